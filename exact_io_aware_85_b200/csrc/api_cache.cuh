// api_cache.cuh — host side of the 4-bit cache operators (kv4.cuh, evict.cuh, key_weights.cuh):
// argument validation, launch plans and the extern "C" entry points declared in include/fa.h.
// Included by api.cu after its helpers.
#pragma once

namespace {

bool head_dim_ok(int d) { return d == 64 || d == 128 || d == 256; }

// Sizes of a cache: C rows per (b, key/value head), a multiple of 128 and at most 2^30.
int check_cache(int B, int Hkv, int C, int d) {
  if (B < 1 || Hkv < 1 || C < 1) return FA_ERR_INVALID_ARG;
  if (!head_dim_ok(d)) return FA_ERR_UNSUPPORTED;
  if (C % fa::kKv4Rows != 0) return FA_ERR_INVALID_ARG;
  if (!sizes_fit(B, Hkv, C, d)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

int launched() {
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? FA_OK : cuda_fail(e);
}

// Chunks per key/value head: one wave of CTAs.
int kv4_splits(int B, int Hkv, int C) { return std::max(1, std::min(C / fa::kKv4Rows, 148 / (B * Hkv))); }

template <int D>
void launch_kv4_decode(const fa::Kv4DecodeArgs& a, cudaStream_t s) {
  fa::fa_kv4_decode_kernel<D><<<dim3(a.nsplit, a.BHkv), 128, 0, s>>>(a);
  const int chunk = 4096;
  fa::fa_kv4_combine_kernel<D><<<dim3(a.acc ? (a.C + chunk - 1) / chunk : 1, a.BHkv), 256, 0, s>>>(a, chunk);
}

}  // namespace

extern "C" {

size_t fa_key_weights_workspace_bytes(int B, int H, int H_kv, int N, int d, int window) {
  if (B < 1 || H < 1 || H_kv < 1 || N < 1 || window < 1 || H % H_kv != 0 || !head_dim_ok(d)) return 0;
  return 256;
}

int fa_key_weights(const void* q, const void* k, const float* lse, float* w, const int* n_rows, int B, int H, int H_kv,
                   int N, int ldw, int d, int causal, int window, float scale, void* workspace, size_t workspace_bytes,
                   void* stream) {
  if (!q || !k || !lse || !w || !workspace) return FA_ERR_INVALID_ARG;
  if (B < 1 || H < 1 || H_kv < 1 || N < 1 || H % H_kv != 0 || window < 1 || ldw < N) return FA_ERR_INVALID_ARG;
  if (!(std::isfinite(scale) && scale > 0.f)) return FA_ERR_INVALID_ARG;
  if (!head_dim_ok(d) || !sizes_fit(B, H, N, d)) return FA_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k) || !aligned4(lse) || !aligned4(w) || !aligned4(n_rows) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return FA_ERR_ALIGNMENT;
  if (workspace_bytes < fa_key_weights_workspace_bytes(B, H, H_kv, N, d, window)) return FA_ERR_INVALID_ARG;
  fa::KeyWeightsArgs a;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.lse = lse;
  a.w = w;
  a.n_rows = n_rows;
  a.N = N;
  a.ldw = ldw;
  a.H = H;
  a.Hkv = H_kv;
  a.g = H / H_kv;
  a.window = std::min(window, N);
  a.causal = causal ? 1 : 0;
  a.ktiles = (N + 127) / 128;
  a.scale_log2 = scale * 1.4426950408889634f;
  const unsigned grid = static_cast<unsigned>(static_cast<long long>(B) * H_kv * a.ktiles);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d == 64) fa::fa_key_weights_kernel<64><<<grid, 128, 0, s>>>(a);
  else if (d == 128) fa::fa_key_weights_kernel<128><<<grid, 128, 0, s>>>(a);
  else fa::fa_key_weights_kernel<256><<<grid, 128, 0, s>>>(a);
  return launched();
}

int fa_evict_keep(const float* w, const int* lens, int* idx, int* count, int B, int H_kv, int C, int keep, int n_recent,
                  int n_sink, void* stream) {
  if (!w || !idx || !count) return FA_ERR_INVALID_ARG;
  if (B < 1 || H_kv < 1 || C < 1 || keep < 1 || n_recent < 0 || n_sink < 0) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(n_recent) + n_sink > keep) return FA_ERR_INVALID_ARG;
  if (C > (1 << 30) || keep > (1 << 30) || static_cast<long long>(B) * H_kv >= (1ll << 31)) return FA_ERR_UNSUPPORTED;
  if (!aligned4(w) || !aligned4(lens) || !aligned4(idx) || !aligned4(count)) return FA_ERR_ALIGNMENT;
  fa::EvictArgs a = {};
  a.w = w;
  a.lens = lens;
  a.out = idx;
  a.count = count;
  a.C = C;
  a.Hkv = H_kv;
  a.n_out = keep;
  a.n_recent = n_recent;
  a.n_sink = n_sink;
  fa::fa_evict_kernel<false><<<B * H_kv, fa::kEvictThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return launched();
}

int fa_evict_slots(const float* acc, const int* pos, int* lens, const int* seen, int* slots, int B, int H_kv, int C,
                   int budget, int T, int n_recent, int n_sink, void* stream) {
  if (!acc || !pos || !lens || !seen || !slots) return FA_ERR_INVALID_ARG;
  if (B < 1 || H_kv < 1 || C < 1 || T < 1 || n_recent < 0 || n_sink < 0) return FA_ERR_INVALID_ARG;
  if (budget < 1 || budget > C || T > budget) return FA_ERR_INVALID_ARG;
  if (C > (1 << 30) || static_cast<long long>(B) * H_kv >= (1ll << 31)) return FA_ERR_UNSUPPORTED;
  if (!aligned4(acc) || !aligned4(pos) || !aligned4(lens) || !aligned4(seen) || !aligned4(slots)) return FA_ERR_ALIGNMENT;
  fa::EvictArgs a = {};
  a.w = acc;
  a.pos = pos;
  a.lens_io = lens;
  a.seen = seen;
  a.out = slots;
  a.C = C;
  a.Hkv = H_kv;
  a.n_out = T;
  a.budget = budget;
  a.n_recent = n_recent;
  a.n_sink = n_sink;
  fa::fa_evict_kernel<true><<<B * H_kv, fa::kEvictThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return launched();
}

int fa_kv4_append(const void* k, const void* v, const float* signs, const float* w, const int* rows, const int* slots,
                  const int* start, const int* n_new, const int* base, void* kc, void* ks, void* vc, void* vs,
                  float* acc, int* pos, int B, int H_kv, int N, int T, int C, int ldw, int d, void* stream) {
  if (!k || !v || !kc || !ks || !vc || !vs) return FA_ERR_INVALID_ARG;
  if (N < 1 || T < 1 || (!rows && T > N) || (slots && start) || (w && ldw < N)) return FA_ERR_INVALID_ARG;
  int st = check_cache(B, H_kv, C, d);
  if (st != FA_OK) return st;
  if (!sizes_fit(B, H_kv, N, d) || !sizes_fit(B, H_kv, T, d)) return FA_ERR_UNSUPPORTED;
  if (!aligned16(k) || !aligned16(v) || !aligned16(kc) || !aligned16(ks) || !aligned16(vc) || !aligned16(vs) ||
      !aligned16(acc) || !aligned16(pos))
    return FA_ERR_ALIGNMENT;
  if (!aligned4(signs) || !aligned4(w) || !aligned4(rows) || !aligned4(slots) || !aligned4(start) || !aligned4(n_new) ||
      !aligned4(base))
    return FA_ERR_ALIGNMENT;
  fa::Kv4AppendArgs a;
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.signs = signs;
  a.w = w;
  a.rows = rows;
  a.slots = slots;
  a.start = start;
  a.n_new = n_new;
  a.base = base;
  a.kc = static_cast<uint8_t*>(kc);
  a.ks = static_cast<__nv_bfloat16*>(ks);
  a.vc = static_cast<uint8_t*>(vc);
  a.vs = static_cast<__nv_bfloat16*>(vs);
  a.acc = acc;
  a.pos = pos;
  a.N = N;
  a.T = T;
  a.C = C;
  a.ldw = ldw;
  a.Hkv = H_kv;
  a.tblocks = (T + 7) / 8;
  const long long blocks = static_cast<long long>(B) * H_kv * a.tblocks;
  if (blocks >= (1ll << 31)) return FA_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(blocks), 2);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d == 64) fa::fa_kv4_append_kernel<64><<<grid, 256, 0, s>>>(a);
  else if (d == 128) fa::fa_kv4_append_kernel<128><<<grid, 256, 0, s>>>(a);
  else fa::fa_kv4_append_kernel<256><<<grid, 256, 0, s>>>(a);
  return launched();
}

int fa_kv4_read(const void* kc, const void* ks, const void* vc, const void* vs, const float* signs, const int* slots,
                const int* lens, void* k, void* v, int B, int H_kv, int T, int C, int first, int d, void* stream) {
  if (!kc || !ks || !vc || !vs || !k || !v) return FA_ERR_INVALID_ARG;
  if (T < 1 || first < 0 || (slots && first != 0)) return FA_ERR_INVALID_ARG;
  int st = check_cache(B, H_kv, C, d);
  if (st != FA_OK) return st;
  if (!sizes_fit(B, H_kv, T, d)) return FA_ERR_UNSUPPORTED;
  if (!aligned16(kc) || !aligned16(ks) || !aligned16(vc) || !aligned16(vs) || !aligned16(k) || !aligned16(v))
    return FA_ERR_ALIGNMENT;
  if (!aligned4(signs) || !aligned4(slots) || !aligned4(lens)) return FA_ERR_ALIGNMENT;
  fa::Kv4ReadArgs a;
  a.kc = static_cast<const uint8_t*>(kc);
  a.ks = static_cast<const __nv_bfloat16*>(ks);
  a.vc = static_cast<const uint8_t*>(vc);
  a.vs = static_cast<const __nv_bfloat16*>(vs);
  a.signs = signs;
  a.slots = slots;
  a.lens = lens;
  a.k = static_cast<__nv_bfloat16*>(k);
  a.v = static_cast<__nv_bfloat16*>(v);
  a.T = T;
  a.C = C;
  a.first = first;
  a.tblocks = (T + 7) / 8;
  const long long blocks = static_cast<long long>(B) * H_kv * a.tblocks;
  if (blocks >= (1ll << 31)) return FA_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(blocks), 2);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d == 64) fa::fa_kv4_read_kernel<64><<<grid, 256, 0, s>>>(a);
  else if (d == 128) fa::fa_kv4_read_kernel<128><<<grid, 256, 0, s>>>(a);
  else fa::fa_kv4_read_kernel<256><<<grid, 256, 0, s>>>(a);
  return launched();
}

size_t fa_decode_kv4_workspace_bytes(int B, int H, int H_kv, int C, int d, int weights) {
  if (B < 1 || H < 1 || H_kv < 1 || H % H_kv != 0 || check_cache(B, H_kv, C, d) != FA_OK) return 0;
  if (H / H_kv > 16 || static_cast<long long>(B) * H_kv > 65535) return 0;
  size_t floats = static_cast<size_t>(kv4_splits(B, H_kv, C)) * B * H * (static_cast<size_t>(d) + 2);
  if (weights) floats += static_cast<size_t>(B) * H * C;
  return (floats * sizeof(float) + 255) / 256 * 256;
}

int fa_decode_kv4(const void* q, const void* kc, const void* ks, const void* vc, const void* vs, const float* signs,
                  const int* lens, void* o, float* lse, float* acc, int B, int H, int H_kv, int C, int d, float scale,
                  void* workspace, size_t workspace_bytes, void* stream) {
  if (!q || !kc || !ks || !vc || !vs || !lens || !o || !lse || !workspace) return FA_ERR_INVALID_ARG;
  if (H < 1 || H_kv < 1 || H % H_kv != 0) return FA_ERR_INVALID_ARG;
  if (!(std::isfinite(scale) && scale > 0.f)) return FA_ERR_INVALID_ARG;
  int st = check_cache(B, H_kv, C, d);
  if (st != FA_OK) return st;
  if (H / H_kv > 16) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * H_kv > 65535) return FA_ERR_UNSUPPORTED;  // key/value heads are gridDim.y
  if (!aligned16(q) || !aligned16(kc) || !aligned16(ks) || !aligned16(vc) || !aligned16(vs) || !aligned16(o) ||
      !aligned16(acc) || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return FA_ERR_ALIGNMENT;
  if (!aligned4(signs) || !aligned4(lens) || !aligned4(lse)) return FA_ERR_ALIGNMENT;
  if (workspace_bytes < fa_decode_kv4_workspace_bytes(B, H, H_kv, C, d, acc != nullptr)) return FA_ERR_INVALID_ARG;
  fa::Kv4DecodeArgs a;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.signs = signs;
  a.kc = static_cast<const uint8_t*>(kc);
  a.ks = static_cast<const __nv_bfloat16*>(ks);
  a.vc = static_cast<const uint8_t*>(vc);
  a.vs = static_cast<const __nv_bfloat16*>(vs);
  a.lens = lens;
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  a.acc = acc;
  a.C = C;
  a.BHkv = B * H_kv;
  a.g = H / H_kv;
  a.nsplit = kv4_splits(B, H_kv, C);
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = a.part_o + static_cast<size_t>(a.nsplit) * B * H * d;
  a.scores = acc ? a.part_ml + static_cast<size_t>(a.nsplit) * B * H * 2 : nullptr;
  a.scale_log2 = scale * 1.4426950408889634f / (signs ? static_cast<float>(d) : 1.f);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d == 64) launch_kv4_decode<64>(a, s);
  else if (d == 128) launch_kv4_decode<128>(a, s);
  else launch_kv4_decode<256>(a, s);
  return launched();
}

}  // extern "C"
