// api_cache.cuh — host side of the 4-bit cache operators (kv4.cuh, evict.cuh, key_weights.cuh):
// argument validation, launch plans and the extern "C" entry points declared in include/fa.h.
// Included by api.cu after its helpers.
#pragma once

namespace {

// rows of k and v enter and leave the cache by 32-byte accesses
bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

bool head_dim_ok(int d) { return d == 64 || d == 128 || d == 256; }

// Sizes of a cache: C rows per (b, key/value head), a multiple of 128 and at most 2^30.
int check_cache(int B, int Hkv, int C, int d) {
  if (B < 1 || Hkv < 1 || C < 1) return FA_ERR_INVALID_ARG;
  if (!head_dim_ok(d)) return FA_ERR_UNSUPPORTED;
  if (C % fa::kKv4Rows != 0) return FA_ERR_INVALID_ARG;
  if (!sizes_fit(B, Hkv, C, d)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// The decoding step's plan, from the sizes alone: one CTA per SM (148), fewer when the caches
// hold fewer blocks; rows of the score buffer padded to an even number of heads.
struct Kv4Plan {
  int nt, gp, grid, slots;
  size_t part_o, part_rl, fac, span, scores, bytes;  // offsets in bytes
};

Kv4Plan kv4_plan(int B, int H, int Hkv, int C, int d, bool weights) {
  Kv4Plan p;
  const int g = H / Hkv;
  const long long bhkv = static_cast<long long>(B) * Hkv;
  p.nt = g > 8 ? 2 : 1;
  p.gp = g == 1 ? 1 : (g + 1) / 2 * 2;
  const int block = fa::kv4_warps(d, p.nt) * 32;
  p.grid = static_cast<int>(std::min<long long>(148, bhkv * ((C + block - 1) / block)));
  p.slots = static_cast<int>(p.grid + bhkv);
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  p.part_o = 0;
  p.part_rl = p.part_o + up(static_cast<size_t>(p.slots) * 8 * p.nt * d * 4);
  p.fac = p.part_rl + up(static_cast<size_t>(p.slots) * 8 * p.nt * 8);
  p.span = p.fac + up(static_cast<size_t>(bhkv) * 8 * p.nt * 4);
  p.scores = p.span + up(static_cast<size_t>(bhkv) * 8);
  p.bytes = p.scores + (weights ? up(static_cast<size_t>(bhkv) * C * p.gp * 4) : 0);
  return p;
}

// A kernel that is launched while the one before it on the stream still runs, and waits for it
// on the device: every kernel here begins with wait_for_earlier(), in every thread block, so that
// a kernel's end is also the end of all kernels before it.  (Calls in a row, launched after the
// one before has ended: one row of 64 heads to evict 6.3 us instead of 3.7, a token's append and
// read 10.4 instead of 6.4, a short decoding step 10.4 instead of 8.5.)
template <typename... Params, typename... Args>
int launch_after(void (*kern)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, static_cast<Params>(args)...);
  return e == cudaSuccess ? FA_OK : cuda_fail(e);
}

template <int D, int NT, bool TWO, bool SPLIT>
int launch_kv4_decode_as(const fa::Kv4DecodeArgs& a, cudaStream_t s) {
  using L = fa::Kv4Cfg<D, NT>;
  auto kern = fa::fa_kv4_decode_kernel<D, NT, TWO, SPLIT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES);
  if (e != cudaSuccess) return cuda_fail(e);
  const int st = launch_after(kern, dim3(a.grid), dim3(L::THREADS), L::BYTES, s, a);
  if (st != FA_OK) return st;
  constexpr int KEYS = 4;  // 8: 75 us, 2: 74 us instead of 70 us for 8 x 32768 rows
  const int chunks = a.acc ? (a.C + 256 * KEYS - 1) / (256 * KEYS) : 1;
  return launch_after(fa::fa_kv4_combine_kernel<D, NT, KEYS>, dim3(chunks, a.BHkv), dim3(256), 0, s, a);
}

template <int D>
int launch_kv4_decode(const fa::Kv4DecodeArgs& a, int nt, cudaStream_t s) {
  if (a.g <= 4) return launch_kv4_decode_as<D, 1, false, true>(a, s);
  if (nt == 1)
    return a.signs ? launch_kv4_decode_as<D, 1, true, false>(a, s) : launch_kv4_decode_as<D, 1, false, false>(a, s);
  return a.signs ? launch_kv4_decode_as<D, 2, true, false>(a, s) : launch_kv4_decode_as<D, 2, false, false>(a, s);
}

// The key weights' plan: CTAs, and the workspace's parts in bytes.
struct KeyWeightsPlan {
  int ranges, grid;
  size_t part, span, bytes;
};

KeyWeightsPlan key_weights_plan(int B, int H, int Hkv, int N, int window) {
  KeyWeightsPlan p;
  p.ranges = (N + 255) / 256;
  const long long items = static_cast<long long>(B) * Hkv * p.ranges;
  const long long subs = (std::min(window, N) + 63ll) / 64 * (H / Hkv);
  p.grid = static_cast<int>(std::min<long long>(148, items * ((subs + 1) / 2)));
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  p.part = 0;
  p.span = up((static_cast<size_t>(p.grid) + items) * 512 * 4);
  p.bytes = p.span + up(static_cast<size_t>(items) * 8);
  return p;
}

template <int D>
int launch_key_weights(const void* q, const void* k, int B, int H, int Hkv, int N, const fa::KeyWeightsArgs& a,
                       cudaStream_t s) {
  using C = fa::KeyWeightsCfg<D>;
  CUtensorMap mq, mk;
  int st;
  const auto dt = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  if ((st = encode_qkv_map(&mq, q, dt, 2, D, N, B * H, CU_TENSOR_MAP_SWIZZLE_128B, 64)) != FA_OK) return st;
  if ((st = encode_qkv_map(&mk, k, dt, 2, D, N, B * Hkv)) != FA_OK) return st;
  auto kern = fa::fa_key_weights_kernel<D>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
  if (e != cudaSuccess) return cuda_fail(e);
  if ((st = launch_after(kern, dim3(a.grid), dim3(fa::kKeyWeightsThreads), C::SMEM_BYTES, s, mq, mk, a)) != FA_OK) return st;
  const long long items = static_cast<long long>(B) * Hkv * a.ranges;
  return launch_after(fa::fa_key_weights_sum_kernel, dim3(static_cast<unsigned>((items + 3) / 4)), dim3(256), 0, s,
                      a);
}

// Eviction: CTAs per head (a cluster of up to eight), while the grid stays within the SMs.
template <bool SLOTS>
int launch_evict(fa::EvictArgs a, int heads, int rows, cudaStream_t s) {
  int S = 1;
  while (S < fa::kEvictMaxCluster && rows > 4096 * S && 2ll * S * heads <= 148) S *= 2;
  a.ctas = S;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(heads) * S);
  cfg.blockDim = dim3(1024);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = S;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const int per = (rows + S - 1) / S;
  const cudaError_t e = per <= 4096   ? cudaLaunchKernelEx(&cfg, fa::fa_evict_kernel<SLOTS, 4>, a)
                        : per <= 8192 ? cudaLaunchKernelEx(&cfg, fa::fa_evict_kernel<SLOTS, 8>, a)
                                      : cudaLaunchKernelEx(&cfg, fa::fa_evict_kernel<SLOTS, 16>, a);
  return e == cudaSuccess ? FA_OK : cuda_fail(e);
}

}  // namespace

extern "C" {

size_t fa_key_weights_workspace_bytes(int B, int H, int H_kv, int N, int d, int window) {
  if (B < 1 || H < 1 || H_kv < 1 || N < 1 || window < 1 || H % H_kv != 0 || !head_dim_ok(d)) return 0;
  if (!sizes_fit(B, H, N, d)) return 0;
  return key_weights_plan(B, H, H_kv, N, window).bytes;
}

int fa_key_weights(const void* q, const void* k, const float* lse, float* w, const int* n_rows, int B, int H, int H_kv,
                   int N, int ldw, int d, int causal, int window, float scale, void* workspace, size_t workspace_bytes,
                   void* stream) {
  if (!q || !k || !lse || !w || !workspace) return FA_ERR_INVALID_ARG;
  if (B < 1 || H < 1 || H_kv < 1 || N < 1 || H % H_kv != 0 || window < 1 || ldw < N) return FA_ERR_INVALID_ARG;
  if (!(std::isfinite(scale) && scale > 0.f)) return FA_ERR_INVALID_ARG;
  if (!head_dim_ok(d) || !sizes_fit(B, H, N, d)) return FA_ERR_UNSUPPORTED;
  if (scale < 8.271806e-25f) return FA_ERR_UNSUPPORTED;  // 2^-80: lse / scale has to be a number
  if (!aligned16(q) || !aligned16(k) || !aligned4(lse) || !aligned4(w) || !aligned4(n_rows) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return FA_ERR_ALIGNMENT;
  if (workspace_bytes < fa_key_weights_workspace_bytes(B, H, H_kv, N, d, window)) return FA_ERR_INVALID_ARG;
  const KeyWeightsPlan p = key_weights_plan(B, H, H_kv, N, window);
  if (static_cast<long long>(B) * H_kv * p.ranges >= (1ll << 31) - 4) return FA_ERR_UNSUPPORTED;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  fa::KeyWeightsArgs a;
  a.lse = lse;
  a.w = w;
  a.n_rows = n_rows;
  a.part = reinterpret_cast<float*>(ws + p.part);
  a.span = reinterpret_cast<int2*>(ws + p.span);
  a.B = B;
  a.N = N;
  a.ldw = ldw;
  a.H = H;
  a.Hkv = H_kv;
  a.g = H / H_kv;
  a.window = std::min(window, N);
  a.causal = causal ? 1 : 0;
  a.ranges = p.ranges;
  a.grid = p.grid;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.neg_inv_scale = -1.f / scale;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d == 64) return launch_key_weights<64>(q, k, B, H, H_kv, N, a, s);
  if (d == 128) return launch_key_weights<128>(q, k, B, H, H_kv, N, a, s);
  return launch_key_weights<256>(q, k, B, H, H_kv, N, a, s);
}

int fa_evict_keep(const float* w, const int* lens, int* idx, int* count, int B, int H_kv, int C, int keep, int n_recent,
                  int n_sink, void* stream) {
  if (!w || !idx || !count) return FA_ERR_INVALID_ARG;
  if (B < 1 || H_kv < 1 || C < 1 || keep < 1 || n_recent < 0 || n_sink < 0) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(n_recent) + n_sink > keep) return FA_ERR_INVALID_ARG;
  if (C > (1 << 30) || keep > (1 << 30) || static_cast<long long>(B) * H_kv >= (1ll << 30)) return FA_ERR_UNSUPPORTED;
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
  return launch_evict<false>(a, B * H_kv, C, static_cast<cudaStream_t>(stream));
}

int fa_evict_slots(const float* acc, const int* pos, int* lens, const int* seen, int* slots, int B, int H_kv, int C,
                   int budget, int T, int n_recent, int n_sink, void* stream) {
  if (!acc || !pos || !lens || !seen || !slots) return FA_ERR_INVALID_ARG;
  if (B < 1 || H_kv < 1 || C < 1 || T < 1 || n_recent < 0 || n_sink < 0) return FA_ERR_INVALID_ARG;
  if (budget < 1 || budget > C || T > budget) return FA_ERR_INVALID_ARG;
  if (C > (1 << 30) || static_cast<long long>(B) * H_kv >= (1ll << 30)) return FA_ERR_UNSUPPORTED;
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
  return launch_evict<true>(a, B * H_kv, budget, static_cast<cudaStream_t>(stream));
}

int fa_kv4_append(const void* k, const void* v, const float* signs, const float* w, const int* rows, const int* slots,
                  const int* start, const int* n_new, const int* base, void* kc, void* ks, void* vc, void* vs,
                  float* acc, int* pos, int B, int H_kv, int N, int T, int C, int ldw, int d, void* stream) {
  if (!k || !v || !kc || !ks || !vc || !vs) return FA_ERR_INVALID_ARG;
  if (N < 1 || T < 1 || (!rows && T > N) || (slots && start) || (w && ldw < N)) return FA_ERR_INVALID_ARG;
  int st = check_cache(B, H_kv, C, d);
  if (st != FA_OK) return st;
  if (!sizes_fit(B, H_kv, N, d) || !sizes_fit(B, H_kv, T, d)) return FA_ERR_UNSUPPORTED;
  if (!aligned32(k) || !aligned32(v) || !aligned16(kc) || !aligned16(ks) || !aligned16(vc) || !aligned16(vs) ||
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
  const int rows_per_block = 32;
  a.tblocks = (T + rows_per_block - 1) / rows_per_block;
  const long long blocks = static_cast<long long>(B) * H_kv * a.tblocks;
  if (blocks >= (1ll << 31)) return FA_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(blocks), 2);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d == 64) return launch_after(fa::fa_kv4_append_kernel<64>, grid, dim3(128), 0, s, a);
  if (d == 128) return launch_after(fa::fa_kv4_append_kernel<128>, grid, dim3(128), 0, s, a);
  return launch_after(fa::fa_kv4_append_kernel<256>, grid, dim3(128), 0, s, a);
}

int fa_kv4_read(const void* kc, const void* ks, const void* vc, const void* vs, const float* signs, const int* slots,
                const int* lens, void* k, void* v, int B, int H_kv, int T, int C, int first, int d, void* stream) {
  if (!kc || !ks || !vc || !vs || !k || !v) return FA_ERR_INVALID_ARG;
  if (T < 1 || first < 0 || (slots && first != 0)) return FA_ERR_INVALID_ARG;
  int st = check_cache(B, H_kv, C, d);
  if (st != FA_OK) return st;
  if (!sizes_fit(B, H_kv, T, d)) return FA_ERR_UNSUPPORTED;
  if (!aligned16(kc) || !aligned16(ks) || !aligned16(vc) || !aligned16(vs) || !aligned32(k) || !aligned32(v))
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
  const int rows_per_block = 32;
  a.tblocks = (T + rows_per_block - 1) / rows_per_block;
  const long long blocks = static_cast<long long>(B) * H_kv * a.tblocks;
  if (blocks >= (1ll << 31)) return FA_ERR_UNSUPPORTED;
  const unsigned grid = static_cast<unsigned>(blocks);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d == 64) return launch_after(fa::fa_kv4_read_kernel<64>, dim3(grid), dim3(128), 0, s, a);
  if (d == 128) return launch_after(fa::fa_kv4_read_kernel<128>, dim3(grid), dim3(128), 0, s, a);
  return launch_after(fa::fa_kv4_read_kernel<256>, dim3(grid), dim3(128), 0, s, a);
}

size_t fa_decode_kv4_workspace_bytes(int B, int H, int H_kv, int C, int d, int weights) {
  if (B < 1 || H < 1 || H_kv < 1 || H % H_kv != 0 || check_cache(B, H_kv, C, d) != FA_OK) return 0;
  if (H / H_kv > 16 || static_cast<long long>(B) * H_kv > 65535) return 0;
  return kv4_plan(B, H, H_kv, C, d, weights != 0).bytes;
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
  const Kv4Plan p = kv4_plan(B, H, H_kv, C, d, acc != nullptr);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.gp = p.gp;
  a.grid = p.grid;
  a.stream = static_cast<size_t>(a.BHkv) * C * (d + 4) > (static_cast<size_t>(96) << 20);  // of 126 MB
  a.part_o = reinterpret_cast<float*>(ws + p.part_o);
  a.part_rl = reinterpret_cast<float2*>(ws + p.part_rl);
  a.fac = reinterpret_cast<float*>(ws + p.fac);
  a.span = reinterpret_cast<int2*>(ws + p.span);
  a.scores = acc ? reinterpret_cast<float*>(ws + p.scores) : nullptr;
  a.scale_log2 = scale * 1.4426950408889634f / (signs ? static_cast<float>(d) : 1.f);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d == 64) return launch_kv4_decode<64>(a, p.nt, s);
  if (d == 128) return launch_kv4_decode<128>(a, p.nt, s);
  return launch_kv4_decode<256>(a, p.nt, s);
}

}  // extern "C"
