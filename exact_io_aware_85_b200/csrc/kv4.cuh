// kv4.cuh — a key/value cache held in 4 bits: writing rows, reading rows back, and one
// decoding step over it.
//
// A row (one token of one key/value head) of d values x is stored as d codes and one scale:
//   y = H diag(signs) x   (keys, when signs are given; H the unnormalised Sylvester
//                          Walsh-Hadamard matrix) or y = x,
//   s = bf16(max|y| / 7),  c = min(7, max(-7, rint(y / s))),  code = c + 8,
// element 2i in the low nibble of byte i, element 2i + 1 in its high nibble.  The rotation
// is the incoherent processing of the FP8 forward ("flash-attention-trading-models", "FA3",
// item 3): it spreads a key's outliers over the row before the row gets its one scale, and
// (H a).(H b) = d a.b, so scores come from a rotated query and a factor 1/d.
#pragma once
#include "sm100.cuh"

namespace fa {

constexpr int kKv4Rows = 128;  // cache capacities are multiples of this many rows

// ---------------------------------------------------------------------------
// rows in
// ---------------------------------------------------------------------------
struct Kv4AppendArgs {
  const __nv_bfloat16* k;  // [B*Hkv, N, d]
  const __nv_bfloat16* v;
  const float* signs;      // [d] or null
  const float* w;          // [B*Hkv, ldw] or null: initial accumulated weight of the source rows
  const int* rows;         // [B*Hkv, T] source rows or null (row t)
  const int* slots;        // [B*Hkv, T] cache rows or null (start + t)
  const int* start;        // [B*Hkv] or null (0)
  const int* n_new;        // [B*Hkv] or null (T)
  const int* base;         // [B] or null (0): position of source row 0
  uint8_t* kc;             // [B*Hkv, C, d/2]
  __nv_bfloat16* ks;       // [B*Hkv, C]
  uint8_t* vc;
  __nv_bfloat16* vs;
  float* acc;              // [B*Hkv, C] or null
  int* pos;                // [B*Hkv, C] or null
  int N, T, C, ldw, Hkv;
  int tblocks;             // blocks per (b, head)
};

// One warp per row; lane l holds elements [l E, (l + 1) E).  blockIdx.y: keys, values.
template <int D>
__global__ void __launch_bounds__(256) fa_kv4_append_kernel(const Kv4AppendArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int bh = blockIdx.x / a.tblocks;
  const int t = (blockIdx.x % a.tblocks) * 8 + warp;
  const bool is_v = blockIdx.y == 1;
  const int n_new = a.n_new ? min(a.n_new[bh], a.T) : a.T;
  if (t >= n_new) return;
  const long long bt = static_cast<long long>(bh) * a.T + t;
  const int src = a.rows ? a.rows[bt] : t;
  const long long dst = a.slots ? a.slots[bt] : (a.start ? static_cast<long long>(a.start[bh]) : 0) + t;
  if (src < 0 || src >= a.N || dst < 0 || dst >= a.C) return;
  const __nv_bfloat16* x = (is_v ? a.v : a.k) + (static_cast<size_t>(bh) * a.N + src) * D + lane * E;
  float y[E];
#pragma unroll
  for (int i = 0; i < E; ++i) y[i] = __bfloat162float(x[i]);
  if (!is_v && a.signs) {
#pragma unroll
    for (int i = 0; i < E; ++i) y[i] *= a.signs[lane * E + i];
#pragma unroll
    for (int h = 1; h < E; h <<= 1)
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (!(i & h)) {
          const float p = y[i], q = y[i + h];
          y[i] = p + q;
          y[i + h] = p - q;
        }
#pragma unroll
    for (int h = 1; h < 32; h <<= 1)
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float o = __shfl_xor_sync(0xffffffffu, y[i], h);
        y[i] = (lane & h) ? o - y[i] : y[i] + o;
      }
  }
  // the largest magnitude by its bits: an infinity or a NaN in the row wins
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < E; ++i) top = max(top, __float_as_uint(y[i]) & 0x7fffffffu);
  top = __reduce_max_sync(0xffffffffu, top);
  const bool finite = top < 0x7f800000u;
  const __nv_bfloat16 sb = finite ? __float2bfloat16_rn(__fdiv_rn(__uint_as_float(top), 7.f))
                                  : __ushort_as_bfloat16(static_cast<unsigned short>(0x7fff));
  const float s = __bfloat162float(sb);
  uint32_t packed = 0;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    float c = 0.f;
    if (finite && s > 0.f) c = fminf(7.f, fmaxf(-7.f, rintf(__fdiv_rn(y[i], s))));
    packed |= static_cast<uint32_t>(static_cast<int>(c) + 8) << (4 * i);
  }
  const size_t row = static_cast<size_t>(bh) * a.C + dst;
  uint8_t* codes = (is_v ? a.vc : a.kc) + row * (D / 2) + lane * (E / 2);
  if constexpr (E == 2) *codes = static_cast<uint8_t>(packed);
  else if constexpr (E == 4) *reinterpret_cast<uint16_t*>(codes) = static_cast<uint16_t>(packed);
  else *reinterpret_cast<uint32_t*>(codes) = packed;
  if (lane == 0) {
    (is_v ? a.vs : a.ks)[row] = sb;
    if (!is_v) {
      if (a.acc) a.acc[row] = a.w ? a.w[static_cast<size_t>(bh) * a.ldw + src] : 0.f;
      if (a.pos) a.pos[row] = (a.base ? a.base[bh / a.Hkv] : 0) + src;
    }
  }
}

// ---------------------------------------------------------------------------
// rows out
// ---------------------------------------------------------------------------
struct Kv4ReadArgs {
  const uint8_t* kc;
  const __nv_bfloat16* ks;
  const uint8_t* vc;
  const __nv_bfloat16* vs;
  const float* signs;
  const int* slots;  // [B*Hkv, T] or null (first + t)
  const int* lens;   // [B*Hkv] or null (C)
  __nv_bfloat16* k;  // [B*Hkv, T, d]
  __nv_bfloat16* v;
  int T, C, first;
  int tblocks;
};

// The codes of a rotated row go back through H as whole numbers (sums of at most 256 codes,
// exact in fp32): x = signs (s / d) H c, rounded once, to bf16.
template <int D>
__global__ void __launch_bounds__(256) fa_kv4_read_kernel(const Kv4ReadArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int bh = blockIdx.x / a.tblocks;
  const int t = (blockIdx.x % a.tblocks) * 8 + warp;
  const bool is_v = blockIdx.y == 1;
  if (t >= a.T) return;
  const long long bt = static_cast<long long>(bh) * a.T + t;
  const long long r = a.slots ? a.slots[bt] : static_cast<long long>(a.first) + t;
  const int len = a.lens ? min(a.lens[bh], a.C) : a.C;
  float y[E];
#pragma unroll
  for (int i = 0; i < E; ++i) y[i] = 0.f;
  if (r >= 0 && r < len) {
    const size_t row = static_cast<size_t>(bh) * a.C + r;
    const uint8_t* codes = (is_v ? a.vc : a.kc) + row * (D / 2) + lane * (E / 2);
#pragma unroll
    for (int i = 0; i < E; ++i) y[i] = static_cast<float>(static_cast<int>((codes[i / 2] >> (4 * (i & 1))) & 15) - 8);
    float s = __bfloat162float((is_v ? a.vs : a.ks)[row]);
    if (!is_v && a.signs) {
#pragma unroll
      for (int h = 1; h < E; h <<= 1)
#pragma unroll
        for (int i = 0; i < E; ++i)
          if (!(i & h)) {
            const float p = y[i], q = y[i + h];
            y[i] = p + q;
            y[i + h] = p - q;
          }
#pragma unroll
      for (int h = 1; h < 32; h <<= 1)
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const float o = __shfl_xor_sync(0xffffffffu, y[i], h);
          y[i] = (lane & h) ? o - y[i] : y[i] + o;
        }
      s *= 1.f / D;
#pragma unroll
      for (int i = 0; i < E; ++i) y[i] *= a.signs[lane * E + i];
    }
#pragma unroll
    for (int i = 0; i < E; ++i) y[i] *= s;
  }
  __nv_bfloat16* out = (is_v ? a.v : a.k) + bt * D + lane * E;
#pragma unroll
  for (int i = 0; i < E; ++i) out[i] = __float2bfloat16_rn(y[i]);
}

// ---------------------------------------------------------------------------
// one decoding step
// ---------------------------------------------------------------------------
struct Kv4DecodeArgs {
  const __nv_bfloat16* q;  // [B*H, d]
  const float* signs;      // [d] or null
  const uint8_t* kc;
  const __nv_bfloat16* ks;
  const uint8_t* vc;
  const __nv_bfloat16* vs;
  const int* lens;         // [B*Hkv]
  __nv_bfloat16* o;        // [B*H, d]
  float* lse;              // [B*H]
  float* acc;              // [B*Hkv, C] or null
  float* part_o;           // [nsplit, B*Hkv, g, d]
  float* part_ml;          // [nsplit, B*Hkv, g, 2]
  float* scores;           // [B*Hkv, C, g] in log2 units, or null
  int C, BHkv, g, nsplit;
  float scale_log2;        // softmax scale * log2(e), / d when rotated
};

__device__ __forceinline__ int kv4_len(const int* lens, int bh, int C) { return max(0, min(lens[bh], C)); }

// One CTA per key chunk of one key/value head, 128-key tiles: a thread takes one key's
// scores, then its columns of the output.
template <int D>
__global__ void __launch_bounds__(128) fa_kv4_decode_kernel(const Kv4DecodeArgs a) {
  constexpr int G = 16;
  __shared__ float q[G][D];
  __shared__ float p[G][128];
  __shared__ float red[4][G];
  const int bh = blockIdx.y, split = blockIdx.x, tid = threadIdx.x, g = a.g;
  const int lane = tid & 31, warp = tid >> 5;
  const int len = kv4_len(a.lens, bh, a.C);
  const int tiles = (len + 127) / 128, per = (tiles + a.nsplit - 1) / a.nsplit;
  const int t0 = min(tiles, split * per), t1 = min(tiles, t0 + per);
  for (int i = tid; i < g * D; i += 128)
    q[i / D][i % D] = __bfloat162float(a.q[static_cast<size_t>(bh) * g * D + i]) * (a.signs ? a.signs[i % D] : 1.f);
  __syncthreads();
  if (a.signs)
    for (int h = 1; h < D; h <<= 1) {
      for (int i = tid; i < g * D / 2; i += 128) {
        const int r = i / (D / 2), j = i % (D / 2), lo = (j / h) * 2 * h + j % h;
        const float x = q[r][lo], y = q[r][lo + h];
        q[r][lo] = x + y;
        q[r][lo + h] = x - y;
      }
      __syncthreads();
    }
  float m[G], l[G], o[G][D / 128 > 0 ? D / 128 : 1];
  for (int h = 0; h < G; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
    for (int c = 0; c < (D / 128 > 0 ? D / 128 : 1); ++c) o[h][c] = 0.f;
  }
  for (int t = t0; t < t1; ++t) {
    const int key = t * 128 + tid;
    const size_t row = static_cast<size_t>(bh) * a.C + key;
    const float ks = key < len ? __bfloat162float(a.ks[row]) * a.scale_log2 : 0.f;
    for (int h = 0; h < g; ++h) {
      float s = -INFINITY;
      if (key < len) {
        s = 0.f;
        for (int i = 0; i < D / 2; ++i) {
          const int c = a.kc[row * (D / 2) + i];
          s = fmaf(q[h][2 * i], static_cast<float>((c & 15) - 8), s);
          s = fmaf(q[h][2 * i + 1], static_cast<float>((c >> 4) - 8), s);
        }
        s *= ks;
        if (a.scores) a.scores[row * g + h] = s;
      }
      float mx = s;
      for (int off = 16; off; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      if (lane == 0) red[warp][h] = mx;
      p[h][tid] = s;
    }
    __syncthreads();
    for (int h = 0; h < g; ++h) {
      const float mn = fmaxf(m[h], fmaxf(fmaxf(red[0][h], red[1][h]), fmaxf(red[2][h], red[3][h])));
      const float al = exp2f(m[h] - mn);
      m[h] = mn;
      l[h] *= al;
      for (int c = 0; c < (D / 128 > 0 ? D / 128 : 1); ++c) o[h][c] *= al;
    }
    __syncthreads();
    for (int h = 0; h < g; ++h) p[h][tid] = key < len ? exp2f(p[h][tid] - m[h]) : 0.f;
    __syncthreads();
    const int nk = min(128, len - t * 128);
    for (int j = 0; j < nk; ++j) {
      const size_t vr = static_cast<size_t>(bh) * a.C + t * 128 + j;
      const float vs = __bfloat162float(a.vs[vr]);
      for (int c = 0; c < (D / 128 > 0 ? D / 128 : 1); ++c) {
        const int col = tid + 128 * c;
        if (col < D) {
          const int b = a.vc[vr * (D / 2) + col / 2];
          const float v = vs * static_cast<float>(((b >> (4 * (col & 1))) & 15) - 8);
          for (int h = 0; h < g; ++h) o[h][c] = fmaf(p[h][j], v, o[h][c]);
        }
      }
      for (int h = 0; h < g; ++h) l[h] += p[h][j];
    }
    __syncthreads();
  }
  const size_t slot = (static_cast<size_t>(split) * a.BHkv + bh) * g;
  for (int h = 0; h < g; ++h) {
    for (int c = 0; c < (D / 128 > 0 ? D / 128 : 1); ++c)
      if (tid + 128 * c < D) a.part_o[(slot + h) * D + tid + 128 * c] = o[h][c];
    if (tid == 0) {
      a.part_ml[(slot + h) * 2] = m[h];
      a.part_ml[(slot + h) * 2 + 1] = l[h];
    }
  }
}

// Joins the chunks of a head by their maxima: O, LSE, and each key's weight summed over the
// query heads that share it.  grid (key chunks, B*Hkv).
template <int D>
__global__ void __launch_bounds__(256) fa_kv4_combine_kernel(const Kv4DecodeArgs a, int chunk) {
  __shared__ float lse2[16];
  const int bh = blockIdx.y, g = a.g, tid = threadIdx.x;
  const int len = kv4_len(a.lens, bh, a.C);
  if (tid < g) {
    float M = -INFINITY, L = 0.f;
    for (int s = 0; s < a.nsplit; ++s) {
      const float* ml = a.part_ml + ((static_cast<size_t>(s) * a.BHkv + bh) * g + tid) * 2;
      M = fmaxf(M, ml[0]);
    }
    for (int s = 0; s < a.nsplit; ++s) {
      const float* ml = a.part_ml + ((static_cast<size_t>(s) * a.BHkv + bh) * g + tid) * 2;
      if (ml[1] != 0.f) L += ml[1] * exp2f(ml[0] - M);
    }
    lse2[tid] = len > 0 ? M + log2f(L) : -INFINITY;
    if (blockIdx.x == 0) a.lse[static_cast<size_t>(bh) * g + tid] = lse2[tid] * 0.69314718055994530942f;
  }
  __syncthreads();
  if (blockIdx.x == 0)
    for (int i = tid; i < g * D; i += 256) {
      const int h = i / D, c = i % D;
      float acc = 0.f;
      if (len > 0)
        for (int s = 0; s < a.nsplit; ++s) {
          const size_t slot = (static_cast<size_t>(s) * a.BHkv + bh) * g + h;
          if (a.part_ml[slot * 2 + 1] != 0.f) acc = fmaf(a.part_o[slot * D + c], exp2f(a.part_ml[slot * 2] - lse2[h]), acc);
        }
      a.o[static_cast<size_t>(bh) * g * D + i] = __float2bfloat16_rn(acc);
    }
  if (a.acc)
    for (int key = blockIdx.x * chunk + tid; key < min(len, (blockIdx.x + 1) * chunk); key += 256) {
      const size_t row = static_cast<size_t>(bh) * a.C + key;
      float w = 0.f;
      for (int h = 0; h < g; ++h) w += exp2f(a.scores[row * g + h] - lse2[h]);
      a.acc[row] += w;
    }
}

}  // namespace fa
