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
#include "early.cuh"
#include "sm100.cuh"

namespace fa {

constexpr int kKv4Rows = 128;  // cache capacities are multiples of this many rows

// D (16x8 fp32) += A (16x16 fp16, row-major) B (16x8 fp16, column-major)
__device__ __forceinline__ void mma_16816_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
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

// A warp takes 8 rows; lane (grp, tq) holds a quarter of row grp, D/4 elements, as pairs.  The
// rotation's bits of the element index divide between the tensor core and the registers: bits 0, 1
// and the two that name the lane's quarter are the 16 x 16 matrix H16, one m16n8k16 MMA pair per 4
// elements (whose operand is the row as it lies in memory, and whose result has the same layout;
// half of its rows stay empty: two rows a lane took twice the registers and left too few warps to
// keep the memory busy, 121 us against 118 for the case below); the others are additions between a
// lane's own pairs.  No shuffles, and a fifth of the instructions of the stages as butterflies.
// Append + read of 262144 rows of d = 128 (K and V, 341 MB, 52 us at the copy rate) take 75 us: the
// butterflies 122 us, this with 16-byte accesses 118, with 32-byte ones 104, without divisions next to
// a border 87, with eight CTAs per SM (64 registers) 81, K and V of a row read together 75.
template <int D>
struct Kv4Rows {
  static constexpr int NE = D / 4, NP = NE / 2, BLOCKS = NE / 4;  // elements, pairs, groups of 4 of a lane and row
  static constexpr int WARPS = 4;                                 // per CTA
  static constexpr int CTAS = D == 256 ? 4 : 8;                   // per SM: 64 (128) registers a thread
  static constexpr int ROWS = 8;                                  // of a warp
};

// volatile, and told to touch memory: the load has to stay behind wait_for_earlier()
__device__ __forceinline__ void ld_global_32(const void* p, uint32_t* r) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void st_global_32(void* p, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// Entry (k, n) of H16, the B operand of its MMAs: -1 to the number of ones of k & n.
__device__ __forceinline__ float kv4_h16(int k, int n) { return (__popc(k & n) & 1) ? -1.f : 1.f; }

// The stages of H between a lane's groups of 4 elements.
template <int D>
__device__ __forceinline__ void kv4_hadamard_groups(float2 (&z)[Kv4Rows<D>::NP]) {
#pragma unroll
  for (int h = 1; h < Kv4Rows<D>::BLOCKS; h <<= 1)
#pragma unroll
    for (int b = 0; b < Kv4Rows<D>::BLOCKS; ++b)
      if (!(b & h))
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float2 p = z[2 * b + x], q = z[2 * (b + h) + x];
          z[2 * b + x] = fadd2(p, q);
          z[2 * (b + h) + x] = fsub2(p, q);
        }
}
// three-input maximum of magnitudes in which a NaN wins
__device__ __forceinline__ float absmax3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(fabsf(b)), "f"(fabsf(c)));
  return d;
}
// sign bits of the pairs of a row: bits 15 and 31 of word i for elements 2 i and 2 i + 1
template <int D>
__device__ __forceinline__ void kv4_sign_masks(const float* signs, uint32_t* masks) {
  for (int i = threadIdx.x; i < D / 2; i += 32 * Kv4Rows<D>::WARPS)
    masks[i] = (signs && signs[2 * i] < 0.f ? 0x8000u : 0u) | (signs && signs[2 * i + 1] < 0.f ? 0x80000000u : 0u);
}

// blockIdx.y: keys, values.  What a row costs in instructions comes close to what it costs in
// bytes: quotients are formed two at a time, and four codes are put together in the mantissa of one
// fp32 number.  (The quotient has to be the rounded one: y / s is often an exact tie of two codes, as
// s and an unrotated y have 8 bits.)
template <int D>
__global__ void __launch_bounds__(32 * Kv4Rows<D>::WARPS, Kv4Rows<D>::CTAS) fa_kv4_append_kernel(const Kv4AppendArgs a) {
  using R = Kv4Rows<D>;
  wait_for_earlier();
  __shared__ __align__(16) uint32_t masks[D / 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, grp = lane >> 2, tq = lane & 3;
  const int bh = blockIdx.x / a.tblocks;
  const int t0 = (blockIdx.x % a.tblocks) * (R::ROWS * R::WARPS) + warp * R::ROWS;
  const bool is_v = blockIdx.y == 1, rotate = !is_v && a.signs;
  const int n_new = a.n_new ? min(a.n_new[bh], a.T) : a.T;
  const int t = t0 + grp;
  const long long bt = static_cast<long long>(bh) * a.T + t;
  bool live = t < n_new;
  const int src = live ? (a.rows ? a.rows[bt] : t) : -1;
  const long long dst = live ? (a.slots ? a.slots[bt] : (a.start ? static_cast<long long>(a.start[bh]) : 0) + t) : -1;
  live = src >= 0 && src < a.N && dst >= 0 && dst < a.C;
  uint32_t w[R::NP];  // the row's pairs of bf16
  const __nv_bfloat16* x = (is_v ? a.v : a.k) + (static_cast<size_t>(bh) * a.N + (live ? src : 0)) * D + tq * 16;
#pragma unroll
  for (int u = 0; u < D / 64; ++u) {
    if (live) ld_global_32(x + 64 * u, &w[8 * u]);
    else
#pragma unroll
      for (int i = 0; i < 8; ++i) w[8 * u + i] = 0u;
  }
  const bool notes = !is_v && tq == 0;  // the lane that writes the row's weight and position
  const float weight = notes && live && a.acc && a.w ? a.w[static_cast<size_t>(bh) * a.ldw + src] : 0.f;
  const int base = notes && a.base ? a.base[bh / a.Hkv] : 0;
  if (rotate) {  // (the row is on its way)
    kv4_sign_masks<D>(a.signs, masks);
    __syncthreads();
  }
  if (t0 >= n_new) return;
  float2 z[R::NP];
  if (rotate) {
#pragma unroll
    for (int i = 0; i < R::NP; ++i) w[i] ^= masks[32 * (i >> 3) + tq * 8 + (i & 7)];
    uint32_t b[2][2];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int k8 = 0; k8 < 2; ++k8)
        b[nt][k8] = pack_bf16x2(kv4_h16(2 * tq + 8 * k8, grp + 8 * nt), kv4_h16(2 * tq + 1 + 8 * k8, grp + 8 * nt));
#pragma unroll
    for (int g = 0; g < R::BLOCKS; ++g)
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        float c[4] = {0.f, 0.f, 0.f, 0.f};
        mma_16816(c, w[2 * g], 0u, w[2 * g + 1], 0u, b[nt][0], b[nt][1]);
        z[2 * g + nt] = make_float2(c[0], c[1]);
      }
    kv4_hadamard_groups<D>(z);
  } else {
#pragma unroll
    for (int i = 0; i < R::NP; ++i)
      z[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < R::NP; ++i) top = absmax3_nan(top, z[i].x, z[i].y);
  top = absmax3_nan(top, __shfl_xor_sync(0xffffffffu, top, 1), 0.f);
  top = absmax3_nan(top, __shfl_xor_sync(0xffffffffu, top, 2), 0.f);
  const bool finite = top < INFINITY;
  const __nv_bfloat16 sb = finite ? __float2bfloat16_rn(__fdiv_rn(top, 7.f))
                                  : __ushort_as_bfloat16(static_cast<unsigned short>(0x7fff));
  const float s = __bfloat162float(sb);
  float2 c[R::NP];  // the codes less 8, whole numbers
  if (finite && s >= 1e-30f) {
    // |y| <= amax, so |c| <= 7 where s is a normal number.  With the rounded reciprocal one step on
    // the remainder (an fma) gives the correctly rounded quotient (Markstein; s has 8 bits).
    const float inv = __frcp_rn(s), kMagic = 12582912.f;  // 1.5 2^23
    const float2 inv2 = make_float2(inv, inv), neg2 = make_float2(-s, -s), magic2 = make_float2(kMagic, kMagic);
#pragma unroll
    for (int i = 0; i < R::NP; ++i) {
      float2 q = fmul2(z[i], inv2);
      q = ffma2(ffma2(q, neg2, z[i]), inv2, q);
      c[i] = fsub2(fadd2(q, magic2), magic2);
    }
  } else {
#pragma unroll
    for (int i = 0; i < R::NP; ++i) {
      const bool some = finite && s > 0.f;
      c[i].x = some ? fminf(7.f, fmaxf(-7.f, rintf(__fdiv_rn(z[i].x, s)))) : 0.f;
      c[i].y = some ? fminf(7.f, fmaxf(-7.f, rintf(__fdiv_rn(z[i].y, s)))) : 0.f;
    }
  }
  uint32_t packed[R::NE / 8];
#pragma unroll
  for (int i = 0; i < R::NE / 8; ++i) {
    uint32_t half[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // c0 + 16 c1 + 256 c2 + 4096 c3, plus 0x8888, in the low bits of 2^23 + ...
      const float2 p = ffma2(c[4 * i + 2 * h + 1], make_float2(256.f, 256.f), c[4 * i + 2 * h]);
      half[h] = __float_as_uint(fmaf(p.y, 16.f, p.x) + (8388608.f + 34952.f));
    }
    packed[i] = __byte_perm(half[0], half[1], 0x5410);
  }
  if (!live) return;
  const size_t row = static_cast<size_t>(bh) * a.C + dst;
  uint8_t* codes = (is_v ? a.vc : a.kc) + row * (D / 2) + tq * 8;
#pragma unroll
  for (int u = 0; u < D / 64; ++u) *reinterpret_cast<uint2*>(codes + 32 * u) = make_uint2(packed[2 * u], packed[2 * u + 1]);
  if (tq == 0) {
    (is_v ? a.vs : a.ks)[row] = sb;
    if (!is_v) {
      if (a.acc) a.acc[row] = weight;
      if (a.pos) a.pos[row] = base + src;
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

// The codes of a rotated row go back through H as whole numbers (exact in fp32): x = signs (s / d)
// H c, rounded once, to bf16.  The nibbles n = c + 8 enter the MMAs as fp16 subnormals, n 2^-24 the
// even ones and n 2^-20 the odd ones, against +-2^14 and +-2^10; H of the eights is 8 d in element 0
// and nothing elsewhere.
template <int D>
__global__ void __launch_bounds__(32 * Kv4Rows<D>::WARPS, Kv4Rows<D>::CTAS) fa_kv4_read_kernel(const Kv4ReadArgs a) {
  using R = Kv4Rows<D>;
  wait_for_earlier();
  __shared__ __align__(16) uint32_t masks[D / 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, grp = lane >> 2, tq = lane & 3;
  const int bh = blockIdx.x / a.tblocks;
  const int t0 = (blockIdx.x % a.tblocks) * (R::ROWS * R::WARPS) + warp * R::ROWS, t = t0 + grp;
  const int len = a.lens ? min(a.lens[bh], a.C) : a.C;
  long long at = -1;
  if (t < a.T) at = a.slots ? a.slots[static_cast<long long>(bh) * a.T + t] : static_cast<long long>(a.first) + t;
  const bool live = at >= 0 && at < len;
  const size_t row = static_cast<size_t>(bh) * a.C + (live ? at : 0);
  // the key's and the value's codes and scales, all on their way together
  uint32_t w[2][R::NE / 8];
  float s[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const uint8_t* codes = (x ? a.vc : a.kc) + row * (D / 2) + tq * 8;
#pragma unroll
    for (int u = 0; u < D / 64; ++u) {
      const uint2 v = *reinterpret_cast<const uint2*>(codes + 32 * u);
      w[x][2 * u] = v.x, w[x][2 * u + 1] = v.y;
    }
    s[x] = __bfloat162float((x ? a.vs : a.ks)[row]);
    if (!live) {  // zeros, whatever the row holds
      s[x] = 0.f;
#pragma unroll
      for (int i = 0; i < R::NE / 8; ++i) w[x][i] = 0x88888888u;
    }
  }
  if (a.signs) {
    kv4_sign_masks<D>(a.signs, masks);
    __syncthreads();
  }
  if (t0 >= a.T) return;
  uint32_t x[R::NP];  // the row's pairs of bf16
  auto store = [&](__nv_bfloat16* to) {
    if (t >= a.T) return;
    __nv_bfloat16* out = to + (static_cast<long long>(bh) * a.T + t) * D + tq * 16;
#pragma unroll
    for (int u = 0; u < D / 64; ++u) st_global_32(out + 64 * u, &x[8 * u]);
  };
  auto plain = [&](const uint32_t (&w)[R::NE / 8], float s) {
    // codes as bf16, (128 + n) - 136, times the scale: a product of 4 and 8 bits, rounded once
    const uint32_t s2 = pack_bf16x2(s, s);
#pragma unroll
    for (int i = 0; i < R::NE / 8; ++i) {
      uint32_t v[4];  // elements (0, 4), (1, 5), (2, 6), (3, 7)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t n = ((w[i] >> (4 * e)) & 0x000f000fu) | 0x43004300u;
        asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(v[e]) : "r"(n), "r"(0xC308C308u));
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(v[e]) : "r"(v[e]), "r"(s2));
      }
      x[4 * i] = __byte_perm(v[0], v[1], 0x5410);
      x[4 * i + 1] = __byte_perm(v[2], v[3], 0x5410);
      x[4 * i + 2] = __byte_perm(v[0], v[1], 0x7632);
      x[4 * i + 3] = __byte_perm(v[2], v[3], 0x7632);
    }
  };
  plain(w[1], s[1]);
  store(a.v);
  if (!a.signs) {
    plain(w[0], s[0]);
  } else {
    float2 z[R::NP];
    uint32_t b[2][2];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int k8 = 0; k8 < 2; ++k8) {
        const float even = 16384.f * kv4_h16(2 * tq + 8 * k8, grp + 8 * nt);
        const float odd = 1024.f * kv4_h16(2 * tq + 1 + 8 * k8, grp + 8 * nt);
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(b[nt][k8]) : "f"(odd), "f"(even));
      }
#pragma unroll
    for (int g = 0; g < R::BLOCKS; ++g) {
      uint32_t p[2];  // bytes 2 g, 2 g + 1 of the lane's codes, a byte in each half
#pragma unroll
      for (int h = 0; h < 2; ++h)
        p[h] = __byte_perm(w[0][g >> 1], 0u, (g & 1) ? (h ? 0x4343 : 0x4242) : (h ? 0x4141 : 0x4040)) & 0x00f0000fu;
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        float c[4] = {0.f, 0.f, 0.f, 0.f};
        mma_16816_f16(c, p[0], 0u, p[1], 0u, b[nt][0], b[nt][1]);
        z[2 * g + nt] = make_float2(c[0], c[1]);
      }
    }
    kv4_hadamard_groups<D>(z);
    if (tq == 0) z[0].x -= 8.f * D / 1024.f;
    float f = s[0] * (1024.f / D);
    if (s[0] > 1e30f) {  // the product of the factors could pass fp32's range
      f = s[0];
#pragma unroll
      for (int i = 0; i < R::NP; ++i) z[i] = fmul2(z[i], make_float2(1024.f / D, 1024.f / D));
    }
#pragma unroll
    for (int i = 0; i < R::NP; ++i) {
      const float2 v = fmul2(z[i], make_float2(f, f));
      x[i] = pack_bf16x2(v.x, v.y) ^ masks[32 * (i >> 3) + tq * 8 + (i & 7)];
    }
  }
  store(a.k);
}

// ---------------------------------------------------------------------------
// one decoding step
// ---------------------------------------------------------------------------
// With codes c, scores are x_j = fac_h ks_j (q_h . c_j) in log2 units, and the output is
// sum_j 2^(x_j - m) vs_j c_j / sum_j 2^(x_j - m): the scales stay outside the products, whose
// cache side is small whole numbers.  The step is bound by reading the cache, (d + 4) bytes a
// row; at the copy rate an SM meets some 45 codes per clock, so what it spends per code decides.
//
//   * Warps work alone: a warp takes 32 keys at a time, holds their running maximum, sum and
//     output for all query heads that share them, and meets the other warps only when the
//     CTA's part of a head ends.  Blocks of 32 keys a warp arrive by bulk copies through a ring.
//   * Products are warp-level m16n8k16 MMAs with the codes on the 16-wide side and the query
//     heads on the 8-wide one.  Which key is which row, and which element which column, is free
//     as long as both operands agree, so every lane reads its codes from shared memory as whole
//     words and unpacks them in place: for K the pairs of a word are consecutive k entries; for
//     V the same element of two keys is, and the eight elements of a word belong to eight MMAs.
//   * Unpacking is one AND for two codes: w & 0xf000f is a pair of fp16 subnormals, n 2^-24 for
//     the nibbles n = c + 8, and w & 0xf000f0 is n 2^-20, exact in the MMA; one shift by 8 serves
//     the other half of the word.  The factor 16 goes into q (for K) or into the result (for V).
//     The 8 leaves K's products through the accumulator's start, -8 sum(q), and V's through one
//     more MMA whose codes are all 8: it gathers 8 sum(P), which is taken off at the end (an
//     absolute error of some 2^-20 sum(p vs), below a bf16 output's rounding unless the weighty
//     rows' codes are all zero in a column).
//     (fp16 1024 + n and an addition instead: 594 instead of about 400 instructions per 32 keys
//     of d = 128, and the same in bf16 for V.)
//   * q in fp16, scaled by a power of two per head so that its largest element is near 2^14: a
//     bf16 element within 2^27 of it is exact (odd ones, a sixteenth, are subnormals first); a
//     rotated query is held as a sum of two fp16 numbers (22 bits).  With at most four heads the
//     second number sits in the MMA's unused columns.
//   * A score's accumulator starts at -8 sum(q) and meets up to 15 sum|q|: what it loses goes by
//     sum|q|, whatever the codes are, d 2^-18 ks sum|q| at most (d / 16 steps, each of which may cut
//     17 numbers at 2^-24 of the largest), measured 2^-17.7 with an element of q 2^14 times the
//     others that meets zeros only.
//   * P times the row's scale, u = p vs, meets V's codes in fp16 too (11 bits, so its rounding
//     stays below that of the bf16 output).  Its range: p = 2^(x - R) with R a running maximum of
//     x + log2 vs instead of x, so that u stays near one and what flushes is 2^-24 of the largest;
//     the softmax's sum is held relative to the same R, which stays within -92 and +125 of the
//     maximum of x: rows whose values are zero or tiny keep their share of the sum.
//   * Work is one list of blocks over all heads' lengths, cut into equal parts, one per CTA:
//     ragged batches fill the GPU evenly.
//
// Measured, both kernels, codes from DRAM: 64 heads of 32768 rows of d = 128, four query heads
// each, weights wanted: 68 us (69 when every lane went on with all 32 keys instead of SPLIT below;
// the bytes 45 at the copy rate; the issue slots are 54 % busy), without weights 53 us (42): the
// scores' store and the second kernel's part in them are 16 us; eight query heads each 84 and 60 us,
// sixteen 178 and 100 us; 64 ragged heads of up to 16384 rows of d = 256, eight query heads each:
// 48 us (21), sixteen 78 us; 8 heads of 1000 rows of d = 64: 8 us, two launches' latency.
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
  float* part_o;           // [grid + B*Hkv, 8 NT d]: slot (CTA + head), in the merge's fragment order
  float2* part_rl;         // [grid + B*Hkv, 8 NT]: R, l
  float* fac;              // [B*Hkv, 8 NT]: factors of the scores
  int2* span;              // [B*Hkv]: the first and the last CTA that worked on a head
  float* scores;           // [B*Hkv, C, gp]: log2 scores less their head's factor, or null
  int C, BHkv, g, gp, grid;
  int stream;              // the cache is larger than the L2
  float scale_log2;        // softmax scale * log2(e), / d when rotated
};

__device__ __forceinline__ int kv4_len(const int* lens, int bh, int C) { return max(0, min(lens[bh], C)); }

constexpr float kKv4Lowest = -3.0e38f;  // the running maximum before the first key

// l 2^x in two steps: a sum of p may hold numbers near 2^97 (rows whose values are zero or tiny
// leave R far below their scores), so that 2^x alone can be 0 where the product counts
__device__ __forceinline__ float kv4_rescale(float l, float x) {
  const float h = ex2_approx(0.5f * x);
  return l * h * h;
}

// Working warps per CTA; one more loads.  As many as the registers of the output and the codes
// leave room for: 128, 168 or 255 a thread.
__host__ __device__ constexpr int kv4_warps(int d, int nt) { return nt == 1 && d <= 128 ? 15 : nt * d <= 256 ? 11 : 7; }

template <int D, int NT>
struct Kv4Cfg {
  static constexpr int NW = kv4_warps(D, NT);
  static constexpr int THREADS = NW * 32 + 32;
  static constexpr int BLOCK = NW * 32;                      // keys per block
  static constexpr int ROW = D / 2;                          // bytes of codes per row
  static constexpr int OFF_V = BLOCK * ROW;
  static constexpr int OFF_KS = 2 * BLOCK * ROW, OFF_VS = OFF_KS + 2 * BLOCK;
  static constexpr int STAGE = OFF_VS + 2 * BLOCK;
  static constexpr int STAGES = 204 * 1024 / STAGE;
  static constexpr int KSTEPS = D / 16;
  static constexpr int MT = D / 16;                          // 16-row tiles of O^T
  static constexpr int MC = 2;                               // ... merged at a time
  static constexpr int OFF_Q = STAGES * STAGE;               // fp16 B fragments: [NT][2][KSTEPS][32] x 8 bytes
  static constexpr int OFF_RED = OFF_Q;                      // the merge's buffer lies over them
  static constexpr int Q_BYTES = NT * 2 * KSTEPS * 32 * 8;
  static constexpr int RED_BYTES = NW * MC * NT * 32 * 16;
  static constexpr int OFF_ML = OFF_Q + (Q_BYTES > RED_BYTES ? Q_BYTES : RED_BYTES);  // [2][NW][8 NT]
  static constexpr int OFF_QRAW = OFF_ML + 2 * NW * 8 * NT * 4;  // bf16 [8 NT][D]: the next head's q
  static constexpr int OFF_SIGN = OFF_QRAW + 8 * NT * D * 2;     // float [D]
  static constexpr int OFF_FAC = OFF_SIGN + D * 4;               // [2][8 NT]
  static constexpr int OFF_BAR = OFF_FAC + 2 * 8 * NT * 4;
  static constexpr int OFF_MISC = OFF_BAR + 2 * STAGES * 8;
  static constexpr int BYTES = OFF_MISC + 256;
  static_assert(STAGES >= 2 && BYTES <= 232448, "shared memory budget");
};

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float bf16_bits_to_float(unsigned short u) {
  return __uint_as_float(static_cast<uint32_t>(u) << 16);
}

// bulk load whose lines are the first to leave the L2
__device__ __forceinline__ uint64_t evict_first_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void bulk_load_hint(void* dst, const void* src, uint32_t bytes, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void cp_async_16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Position in the list of blocks: a head, a block of it, and the head's length.
struct Kv4Cursor {
  int bh, blk, nblk, len;
};

// NT: 8-wide tiles of query heads; TWO: the second halves of a rotated q have MMAs of their own
// (otherwise, for at most four heads, they sit in columns 4-7).  SPLIT: at most four heads, so that a
// score is needed in one of columns n and n + 4 only: the two lanes that hold them add theirs up and
// go on with one 16-key half each, column n with the first, n + 4 with the second (half the
// exponentials and what goes with them; the output's two columns are added up at the end).
template <int D, int NT, bool TWO, bool SPLIT>
__global__ void __launch_bounds__(Kv4Cfg<D, NT>::THREADS, 1) fa_kv4_decode_kernel(const Kv4DecodeArgs a) {
  using L = Kv4Cfg<D, NT>;
  constexpr int NW = L::NW, ST = L::STAGES, NQ = 8 * NT, WORKERS = NW * 32;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int grp = lane >> 2, tq = lane & 3;
  uint64_t* const full = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* const empty = full + ST;
  volatile int* const abort_sh = reinterpret_cast<volatile int*>(smem + L::OFF_MISC);
  int* const scan = reinterpret_cast<int*>(smem + L::OFF_MISC + 16);  // [NW + 1 + 2]
  float* const fac_sh = reinterpret_cast<float*>(smem + L::OFF_FAC);  // [NQ] factors, [NQ] accumulator starts
  float* const wl = reinterpret_cast<float*>(smem + L::OFF_ML);       // [NW][NQ] each
  float* const wr = wl + NW * NQ;
  __nv_bfloat16* const qraw = reinterpret_cast<__nv_bfloat16*>(smem + L::OFF_QRAW);
  float* const sign_sh = reinterpret_cast<float*>(smem + L::OFF_SIGN);
  if (tid == 0) {
    *abort_sh = 0;
    for (int s = 0; s < ST; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], NW);
    }
    fence_mbar_init();
  }
  wait_for_earlier();
  // ---- this CTA's part of the list of blocks -------------------------------------------
  const int per = (a.BHkv + L::THREADS - 1) / L::THREADS;
  const int h0 = min(a.BHkv, tid * per), h1 = min(a.BHkv, h0 + per);
  auto nblocks = [&](int len) { return (len + L::BLOCK - 1) / L::BLOCK; };
  int mine = 0;
  for (int h = h0; h < h1; ++h) mine += nblocks(kv4_len(a.lens, h, a.C));
  int incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  int before = incl - mine, total = 0;
  for (int w = 0; w < NW + 1; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  const int n_cta = max(1, min(a.grid, total));  // the others have nothing to do
  const int u0 = static_cast<int>(min(static_cast<long long>(blockIdx.x) * total / n_cta, static_cast<long long>(total)));
  const int u1 = static_cast<int>(min(static_cast<long long>(blockIdx.x + 1) * total / n_cta, static_cast<long long>(total)));
  if (u0 >= u1) return;
  int* const start = scan + NW + 1;
  if (u0 >= before && u0 < before + mine) {
    int f = before, h = h0;
    while (true) {
      const int n = nblocks(kv4_len(a.lens, h, a.C));
      if (u0 < f + n) break;
      f += n;
      ++h;
    }
    start[0] = h;
    start[1] = u0 - f;
  }
  __syncthreads();
  Kv4Cursor cur;
  cur.bh = start[0];
  cur.blk = start[1];
  cur.len = kv4_len(a.lens, cur.bh, a.C);
  cur.nblk = nblocks(cur.len);
  int left = u1 - u0;  // blocks to go
  auto next_head = [&]() {
    cur.blk = 0;
    do {
      cur.len = kv4_len(a.lens, ++cur.bh, a.C);
      cur.nblk = nblocks(cur.len);
    } while (cur.nblk == 0);
  };

  // A head's query comes by asynchronous copies well before its first block: with the ring full of
  // copies a load waits its turn behind them for microseconds.
  const int g = a.g;
  auto fetch_q = [&](int bh) {
    for (int i = tid; i < g * D / 8; i += WORKERS)
      cp_async_16(qraw + 8 * i, a.q + static_cast<size_t>(bh) * g * D + 8 * i);
  };
  if (warp < NW) {
    fetch_q(cur.bh);
    if (a.signs)
      for (int i = tid; i < D; i += WORKERS) cp_async_4(sign_sh + i, a.signs + i);
  }
  __syncthreads();

  if (warp == NW) {
    // ================= the loading warp: one thread, block after block ======================
    if (lane == 0) {
      // The codes are read once a step; where all of them pass through the L2, they would take the
      // scores' place there, which the second kernel reads.
      const uint64_t policy = evict_first_policy();
      auto load = [&](void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
        if (a.stream) bulk_load_hint(dst, src, bytes, bar, policy);
        else bulk_load(dst, src, bytes, bar);
      };
      int t = 0;
      while (true) {
        const int s = t % ST;
        if (!mbar_wait(&empty[s], ((t / ST) & 1) ^ 1, abort_sh, 31)) break;
        const int key0 = cur.blk * L::BLOCK;
        const int rows = min(L::BLOCK, (cur.len - key0 + 31) & ~31);  // whole 32-row chunks: inside the capacity
        uint8_t* st = smem + s * L::STAGE;
        const size_t row = static_cast<size_t>(cur.bh) * a.C + key0;
        mbar_arrive_expect_tx(&full[s], rows * (2 * L::ROW + 4));
        load(st, a.kc + row * L::ROW, rows * L::ROW, &full[s]);
        load(st + L::OFF_KS, a.ks + row, rows * 2, &full[s]);
        load(st + L::OFF_V, a.vc + row * L::ROW, rows * L::ROW, &full[s]);
        load(st + L::OFF_VS, a.vs + row, rows * 2, &full[s]);
        ++t;
        if (--left == 0) break;
        if (++cur.blk == cur.nblk) next_head();
      }
      // every copy has landed before the block ends
      for (int i = max(0, t - ST); i < t; ++i) mbar_wait_drain(&full[i % ST], (i / ST) & 1, 100000000ull);
    }
    return;
  }

  const bool rotated = a.signs != nullptr;
  constexpr int RW = SPLIT ? 2 : 4;                      // rows of 32 whose scores a lane goes on with
  const int second = SPLIT ? tq >> 1 : 0;                // and which 16 they belong to
  const int col = SPLIT ? 2 * (tq & 1) : 2 * tq;         // their columns: col, col + 1 of a tile
  constexpr int EPL = D / 4 < 32 ? D / 4 : 32;    // elements of a lane's chunk of a key
  constexpr float kTwo24 = 16777216.f;
  bool ok = true;
  int t = 0;  // blocks taken from the ring
  // row r of a 16-key tile is key r ^ ((r >> 1) & 1): the rows that one load touches then
  // alternate between the two halves of a 128-byte line
  const int kr = grp ^ ((grp >> 1) & 1);

  while (left > 0) {
    // ================= one head: q into fragments =======================================
    const int bh = cur.bh;
    __half* const qf = reinterpret_cast<__half*>(smem + L::OFF_Q);
    for (int i = tid; i < L::Q_BYTES / 16; i += WORKERS) reinterpret_cast<uint4*>(qf)[i] = make_uint4(0, 0, 0, 0);
    for (int n = tid; n < 2 * NQ; n += WORKERS) fac_sh[n] = 0.f;
    cp_async_wait_all();
    named_bar_sync(1, WORKERS);
    for (int n = warp; n < g; n += NW) {
      constexpr int E = D / 32;
      const __nv_bfloat16* qrow = qraw + n * D + lane * E;
      float y[E];
#pragma unroll
      for (int i = 0; i < E; ++i) y[i] = __bfloat162float(qrow[i]);
      if (rotated) {
#pragma unroll
        for (int i = 0; i < E; ++i) y[i] *= sign_sh[lane * E + i];
#pragma unroll
        for (int h = 1; h < E; h <<= 1)
#pragma unroll
          for (int i = 0; i < E; ++i)
            if (!(i & h)) {
              const float u = y[i], v = y[i + h];
              y[i] = u + v;
              y[i + h] = u - v;
            }
#pragma unroll
        for (int h = 1; h < 32; h <<= 1)
#pragma unroll
          for (int i = 0; i < E; ++i) {
            const float u = __shfl_xor_sync(0xffffffffu, y[i], h);
            y[i] = (lane & h) ? u - y[i] : y[i] + u;
          }
      }
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < E; ++i) top = max(top, __float_as_uint(y[i]) & 0x7fffffffu);
      top = __reduce_max_sync(0xffffffffu, top);
      // 2^k with |q| 2^k < 2^15 (a query that is not finite, or past 2^110, goes on as infinities)
      const int k = max(-95, min(14 - (static_cast<int>(top >> 23) - 127), 120));
      const float up = __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int j = lane * E + i;
        const int c = j / (4 * EPL), r = j % (4 * EPL), e = r & 7;
        // odd elements meet the nibbles at bits 4-7, which count 16 times
        const float x = (e & 1) ? y[i] * up * 0.0625f : y[i] * up;
        const __half hi = __float2half_rn(x);
        const __half lo = __float2half_rn(x - __half2float(hi));
        const float back = rotated ? __half2float(hi) + __half2float(lo) : __half2float(hi);
        sum += (e & 1) ? back * 16.f : back;
        const int ks = c * (EPL / 4) + ((r % EPL) >> 3) * 2 + ((e & 3) >> 1);
        const int sub = (e & 1) * 2 + (e >> 2), ql = r / EPL;
        const int nt = n >> 3, nc = n & 7;
        qf[((((nt * 2) * L::KSTEPS + ks) * 32 + nc * 4 + ql) << 2) + sub] = hi;
        if (rotated) {
          if (SPLIT) qf[((ks * 32 + (nc + 4) * 4 + ql) << 2) + sub] = lo;
          else qf[((((nt * 2 + 1) * L::KSTEPS + ks) * 32 + nc * 4 + ql) << 2) + sub] = lo;
        }
      }
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      if (lane == 0) {
        // never 0 (a scale below 2^-54 with a query of zeros): rows behind the last get the score -infinity,
        // which has to stay one times f.  2^-149 instead of 0 moves a score, 2^127 f at most, by 2^-22.
        const float f = fmaxf(a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + 24 - k) << 23), __uint_as_float(1u));
        fac_sh[n] = f;
        if (a.scores) a.fac[static_cast<size_t>(bh) * NQ + n] = f;
        fac_sh[NQ + n] = sum * (-8.f / kTwo24);
      }
    }
    named_bar_sync(1, WORKERS);
    float fac[NT][2], x0[NT][2], m_run[NT][2], r_run[NT][2], l_run[NT][2], oacc[NT][L::MT][4], ones[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        fac[j][c] = fac_sh[8 * j + col + c];
        x0[j][c] = fac_sh[NQ + 8 * j + 2 * tq + c];
        m_run[j][c] = r_run[j][c] = kKv4Lowest;
        l_run[j][c] = 0.f;
        ones[j][c] = ones[j][c + 2] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < L::MT; ++i) oacc[j][i][0] = oacc[j][i][1] = oacc[j][i][2] = oacc[j][i][3] = 0.f;
    }
    const uint2* const qfrag = reinterpret_cast<const uint2*>(qf) + lane;
    const int len = cur.len;
    // ================= the head's blocks =================================================
    const int end = min(cur.nblk, cur.blk + left), first = cur.blk;
    const bool ends = end == cur.nblk;
    left -= end - first;
    if (left > 0) {  // the query of the head after this one (everybody has read qraw)
      next_head();
      fetch_q(cur.bh);
    }
    for (int blk = first; blk < end; ++blk, ++t) {
      const int s = t % ST;
      const uint8_t* const st = smem + s * L::STAGE + warp * 32 * L::ROW;
      const int key0 = blk * L::BLOCK + warp * 32;
      ok = ok && __all_sync(0xffffffffu, mbar_wait(&full[s], (t / ST) & 1, abort_sh, 30));
      if (ok && key0 < len) {
        float x[2][NT][4];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            x[u][j][0] = x[u][j][2] = x0[j][0];
            x[u][j][1] = x[u][j][3] = x0[j][1];
          }
#pragma unroll
        for (int c = 0; c < D / (4 * EPL); ++c) {
          uint32_t w[4][EPL / 8];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const uint8_t* p = st + (8 * r + kr) * L::ROW + c * 2 * EPL + tq * (EPL / 2);
            if constexpr (EPL == 32) {
              const uint4 v = *reinterpret_cast<const uint4*>(p);
              w[r][0] = v.x, w[r][1] = v.y, w[r][2] = v.z, w[r][3] = v.w;
            } else {
              const uint2 v = *reinterpret_cast<const uint2*>(p);
              w[r][0] = v.x, w[r][1] = v.y;
            }
          }
#pragma unroll
          for (int i = 0; i < EPL / 8; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int ks = c * (EPL / 4) + 2 * i + h;
              uint32_t lo[4], hi[4];
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const uint32_t v = h ? w[r][i] >> 8 : w[r][i];
                lo[r] = v & 0x000f000fu;
                hi[r] = v & 0x00f000f0u;
              }
#pragma unroll
              for (int j = 0; j < NT; ++j) {
                const uint2 b = qfrag[((j * 2) * L::KSTEPS + ks) * 32];
                mma_16816_f16(x[0][j], lo[0], lo[1], hi[0], hi[1], b.x, b.y);
                mma_16816_f16(x[1][j], lo[2], lo[3], hi[2], hi[3], b.x, b.y);
                if constexpr (TWO) {
                  const uint2 b2 = qfrag[((j * 2 + 1) * L::KSTEPS + ks) * 32];
                  mma_16816_f16(x[0][j], lo[0], lo[1], hi[0], hi[1], b2.x, b2.y);
                  mma_16816_f16(x[1][j], lo[2], lo[3], hi[2], hi[3], b2.x, b2.y);
                }
              }
            }
        }
        float y[NT][2 * RW];  // two columns of each row
        if constexpr (SPLIT) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float mine = second ? x[1][0][i] : x[0][0][i], theirs = second ? x[0][0][i] : x[1][0][i];
            y[0][i] = mine + __shfl_xor_sync(0xffffffffu, theirs, 2);
          }
        } else {
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) y[j][i] = x[i >> 2][j][i & 3];
        }
        float vs[RW];
        const int krow = 16 * second + kr;  // the rows are krow + 8 r
        const unsigned short* const ksp =
            reinterpret_cast<const unsigned short*>(smem + s * L::STAGE + L::OFF_KS) + warp * 32 + krow;
        const bool tail = key0 + 32 > len;
#pragma unroll
        for (int r = 0; r < RW; ++r) {
          const float ks = bf16_bits_to_float(ksp[8 * r]);
          vs[r] = bf16_bits_to_float(ksp[L::BLOCK + 8 * r]);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            y[j][2 * r] *= ks;
            y[j][2 * r + 1] *= ks;
          }
        }
        if (tail) {  // rows behind the last hold anything: neither their codes nor their scales count
#pragma unroll
          for (int r = 0; r < RW; ++r)
            if (key0 + 8 * r + krow >= len) {
              vs[r] = 0.f;
#pragma unroll
              for (int j = 0; j < NT; ++j) y[j][2 * r] = y[j][2 * r + 1] = -INFINITY;
            }
        }
        if (a.scores) {
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const int n = 8 * j + col;
            if (n < g) {
              float* p = a.scores + (static_cast<size_t>(bh) * a.C + key0 + krow) * a.gp + n;
#pragma unroll
              for (int r = 0; r < RW; ++r)
                if (!tail || key0 + 8 * r + krow < len) {
                  if (a.gp == 1) p[8 * r] = y[j][2 * r];
                  else *reinterpret_cast<float2*>(p + 8 * r * a.gp) = make_float2(y[j][2 * r], y[j][2 * r + 1]);
                }
            }
          }
        }
        // ---- p = 2^(x - R) and u = p vs, x = fac times what is stored; R moves only when a u passes
        // 2^12 (or a p 2^97), and then u is at most 2^8 in the second turn -----------------------------
        float p[NT][2 * RW], u[NT][2 * RW];
#pragma unroll 1
        for (int turn = 0; turn < 2; ++turn) {
          float top_p = 0.f, top_u = 0.f;
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int r = 0; r < RW; ++r) {
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                p[j][2 * r + c] = ex2_approx(fmaf(y[j][2 * r + c], fac[j][c], -r_run[j][c]));
                u[j][2 * r + c] = p[j][2 * r + c] * vs[r];
              }
              top_p = fmax3(top_p, p[j][2 * r], p[j][2 * r + 1]);
              top_u = fmax3(top_u, u[j][2 * r], u[j][2 * r + 1]);
            }
          if (turn || !__any_sync(0xffffffffu, top_p > 1.5845633e29f || top_u > 4096.f)) break;
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            float be[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float mx = -INFINITY, ry = -INFINITY;
#pragma unroll
              for (int r = 0; r < RW; ++r) {
                const float z = y[j][2 * r + c] * fac[j][c];
                mx = fmaxf(mx, z);
                ry = fmaxf(ry, z + __log2f(vs[r]));
              }
#pragma unroll
              for (int off = SPLIT ? 2 : 4; off < 32; off <<= 1) {
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                ry = fmaxf(ry, __shfl_xor_sync(0xffffffffu, ry, off));
              }
              const float m_new = fmaxf(m_run[j][c], mx);
              // 2^(m - R) stays a normal number, and the sum of 2^30 p below 2^128
              const float r_new = fminf(fmaxf(fmaxf(r_run[j][c], ry), m_new - 92.f), m_new + 125.f);
              be[c] = ex2_approx(r_run[j][c] - r_new);
              l_run[j][c] = kv4_rescale(l_run[j][c], r_run[j][c] - r_new);
              m_run[j][c] = m_new;
              r_run[j][c] = r_new;
              ones[j][c] *= be[c];
              ones[j][c + 2] *= be[c];
            }
#pragma unroll
            for (int i = 0; i < L::MT; ++i) {
              oacc[j][i][0] *= be[0];
              oacc[j][i][1] *= be[1];
              oacc[j][i][2] *= be[0];
              oacc[j][i][3] *= be[1];
            }
          }
        }
        // ---- u as the B operand -----------------------------------------------------------------
        uint32_t pb[2][NT][2];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int h = 0; h < RW / 2; ++h) {
            l_run[j][0] += p[j][4 * h] + p[j][4 * h + 2];
            l_run[j][1] += p[j][4 * h + 1] + p[j][4 * h + 3];
            pb[h][j][0] = movmatrix_trans(pack_f16x2(u[j][4 * h], u[j][4 * h + 1]));
            pb[h][j][1] = movmatrix_trans(pack_f16x2(u[j][4 * h + 2], u[j][4 * h + 3]));
            mma_16816_f16(ones[j], 0x00080008u, 0x00080008u, 0x00080008u, 0x00080008u, pb[h][j][0], pb[h][j][1]);
          }
        if constexpr (SPLIT) {  // columns 0-3 take the first 16 keys, 4-7 the others
          const uint32_t mask = grp < 4 ? 0u : 0xffffffffu;
          pb[1][0][0] = pb[0][0][0] & mask;
          pb[1][0][1] = pb[0][0][1] & mask;
          pb[0][0][0] &= ~mask;
          pb[0][0][1] &= ~mask;
        }
        // ---- O^T += V^T P^T -----------------------------------------------------------------------
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          constexpr int WPL = D / 64;  // words of a lane per key: octets WPL grp ..
          uint32_t w[4][WPL];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int key = 16 * h + 8 * (r >> 1) + ((2 * tq + (r & 1)) ^ (tq & 1));
            const uint8_t* q = st + L::OFF_V + key * L::ROW + grp * 4 * WPL;
            if constexpr (WPL == 1) {
              w[r][0] = *reinterpret_cast<const uint32_t*>(q);
            } else if constexpr (WPL == 2) {
              const uint2 v = *reinterpret_cast<const uint2*>(q);
              w[r][0] = v.x, w[r][1] = v.y;
            } else {
              const uint4 v = *reinterpret_cast<const uint4*>(q);
              w[r][0] = v.x, w[r][1] = v.y, w[r][2] = v.z, w[r][3] = v.w;
            }
          }
          // element i of a half word of t: bits 0-3 (i even) or 4-7 (i odd) of t or of t >> 8
          auto code = [](uint32_t v, int i) { return (i & 2 ? v >> 8 : v) & (i & 1 ? 0x00f000f0u : 0x000f000fu); };
          if constexpr (WPL == 1) {
            // rows 0-7: element i of octet grp, rows 8-15: element i + 4
            const uint32_t lo0 = __byte_perm(w[0][0], w[1][0], 0x5410), hi0 = __byte_perm(w[0][0], w[1][0], 0x7632);
            const uint32_t lo1 = __byte_perm(w[2][0], w[3][0], 0x5410), hi1 = __byte_perm(w[2][0], w[3][0], 0x7632);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int j = 0; j < NT; ++j)
                mma_16816_f16(oacc[j][i], code(lo0, i), code(hi0, i), code(lo1, i), code(hi1, i), pb[h][j][0], pb[h][j][1]);
          } else {
            // rows 0-7: element i of octet 2 o, rows 8-15: of octet 2 o + 1 (of the lane's WPL octets)
#pragma unroll
            for (int o = 0; o < WPL / 2; ++o)
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                const uint32_t sel = half ? 0x7632 : 0x5410;
                const uint32_t a0 = __byte_perm(w[0][2 * o], w[1][2 * o], sel);
                const uint32_t a1 = __byte_perm(w[0][2 * o + 1], w[1][2 * o + 1], sel);
                const uint32_t a2 = __byte_perm(w[2][2 * o], w[3][2 * o], sel);
                const uint32_t a3 = __byte_perm(w[2][2 * o + 1], w[3][2 * o + 1], sel);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                  for (int j = 0; j < NT; ++j)
                    mma_16816_f16(oacc[j][o * 8 + half * 4 + i], code(a0, i), code(a1, i), code(a2, i), code(a3, i),
                                  pb[h][j][0], pb[h][j][1]);
              }
          }
        }
      }
      __syncwarp();  // every lane has read the stage
      if (lane == 0) mbar_arrive(&empty[s]);
    }
    // ================= merge the warps ====================================================
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float l = l_run[j][c];
#pragma unroll
        for (int off = SPLIT ? 2 : 4; off < 32; off <<= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
        const int n = 8 * j + col + c;
        if (grp == 0 && !second) {
          wl[warp * NQ + n] = l;
          wr[warp * NQ + n] = r_run[j][c];
        }
      }
    named_bar_sync(1, WORKERS);
    const size_t slot = static_cast<size_t>(blockIdx.x) + bh;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int n = 8 * j + col + c;
        float R = kKv4Lowest;
#pragma unroll
        for (int w = 0; w < NW; ++w) R = fmaxf(R, wr[w * NQ + n]);
        const float f = ex2_approx(r_run[j][c] - R) * kTwo24;  // and off the codes' 2^-24
        const float eight = ones[j][c] * f;
#pragma unroll
        for (int i = 0; i < L::MT; ++i) {
          const float fi = (i & 1) ? f * 0.0625f : f;
          oacc[j][i][c] = fmaf(oacc[j][i][c], fi, -eight);
          oacc[j][i][c + 2] = fmaf(oacc[j][i][c + 2], fi, -eight);
          if constexpr (SPLIT) {
            oacc[j][i][c] += __shfl_xor_sync(0xffffffffu, oacc[j][i][c], 2);
            oacc[j][i][c + 2] += __shfl_xor_sync(0xffffffffu, oacc[j][i][c + 2], 2);
          }
        }
      }
    if (tid == 0 && first == 0) a.span[bh].x = blockIdx.x;
    if (tid == 0 && ends) a.span[bh].y = blockIdx.x;
    if (tid < (SPLIT ? 4 : NQ)) {
      float R = kKv4Lowest, l = 0.f;
      for (int w = 0; w < NW; ++w) R = fmaxf(R, wr[w * NQ + tid]);
      for (int w = 0; w < NW; ++w) l += kv4_rescale(wl[w * NQ + tid], wr[w * NQ + tid] - R);
      a.part_rl[slot * NQ + tid] = make_float2(R, l);
    }
    float* const red = reinterpret_cast<float*>(smem + L::OFF_RED);  // [NW][MC][NT][32] float4
    constexpr int RED = L::MC * NT * 128;
#pragma unroll
    for (int i = 0; i < L::MT; i += L::MC) {
#pragma unroll
      for (int c = 0; c < L::MC; ++c)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          reinterpret_cast<float4*>(red)[((warp * L::MC + c) * NT + j) * 32 + lane] =
              make_float4(oacc[j][i + c][0], oacc[j][i + c][1], oacc[j][i + c][2], oacc[j][i + c][3]);
      named_bar_sync(1, WORKERS);
      for (int e = tid; e < RED; e += WORKERS) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) v += red[w * RED + e];
        a.part_o[(slot * L::MT + i) * NT * 128 + e] = v;
      }
      named_bar_sync(1, WORKERS);
    }
  }
}

// Joins the parts of a head by their maxima: O, LSE, and each key's weight summed over the
// query heads that share it.  grid (key chunks of 4 KEYS x 256, B*Hkv); the scores of a thread's
// keys are on their way while the heads' LSE is put together.
template <int D, int NT, int KEYS>
__global__ void __launch_bounds__(256) fa_kv4_combine_kernel(const Kv4DecodeArgs a) {
  constexpr int NQ = 8 * NT, MT = D / 16, CHUNK = 256 * KEYS;
  __shared__ float lse2[NQ], fac[NQ];
  const int bh = blockIdx.y, g = a.g, tid = threadIdx.x, gp = a.gp;
  const int key0 = blockIdx.x * CHUNK + tid;
  wait_for_earlier();
  const int len = kv4_len(a.lens, bh, a.C);
  if (blockIdx.x > 0 && blockIdx.x * CHUNK >= len) return;
  const size_t row = static_cast<size_t>(bh) * a.C + key0;
  float old[KEYS];
  float2 sc[KEYS][2];  // the first four heads' scores
  if (a.acc) {
#pragma unroll
    for (int i = 0; i < KEYS; ++i) {
      const bool in = key0 + 256 * i < len;
      old[i] = in ? a.acc[row + 256 * i] : 0.f;
      sc[i][0] = sc[i][1] = make_float2(0.f, 0.f);
      if (in) {
        const float* p = a.scores + (row + 256 * i) * gp;
        if (gp == 1) sc[i][0].x = p[0];
        else if ((gp & 3) == 0) {
          const float4 v = *reinterpret_cast<const float4*>(p);
          sc[i][0] = make_float2(v.x, v.y), sc[i][1] = make_float2(v.z, v.w);
        } else {
          sc[i][0] = *reinterpret_cast<const float2*>(p);
          if (gp > 2) sc[i][1] = *reinterpret_cast<const float2*>(p + 2);
        }
      }
    }
  }
  // the CTAs that worked on this head (within the grid, should a wait have given up)
  const int2 span = len > 0 ? a.span[bh] : make_int2(0, -1);
  const int i0 = max(span.x, 0), i1 = min(span.y, a.grid - 1);
  const float2* const rl = a.part_rl;
  if (tid < NQ) {
    float R = kKv4Lowest, L = 0.f;
    for (int i = i0; i <= i1; ++i) {
      const float2 p = rl[(static_cast<size_t>(i) + bh) * NQ + tid];
      const float r_new = fmaxf(R, p.x);
      L = kv4_rescale(L, R - r_new) + kv4_rescale(p.y, p.x - r_new);
      R = r_new;
    }
    // heads that are not there weigh nothing
    lse2[tid] = tid >= g ? INFINITY : len > 0 ? R + log2f(L) : -INFINITY;
    fac[tid] = a.acc && tid < g && len > 0 ? a.fac[static_cast<size_t>(bh) * NQ + tid] : 0.f;
    if (blockIdx.x == 0 && tid < g) a.lse[static_cast<size_t>(bh) * g + tid] = lse2[tid] * 0.69314718055994530942f;
  }
  __syncthreads();
  if (blockIdx.x == 0)
    for (int f = tid; f < MT * NT * 32; f += 256) {
      const int lane = f & 31, j = (f >> 5) % NT, i = (f >> 5) / NT;
      const int grp = lane >> 2, n = 8 * j + 2 * (lane & 3);
      if (n >= g) continue;
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int p = i0; p <= i1; ++p) {
        const size_t slot = static_cast<size_t>(p) + bh;
        const float w0 = ex2_approx(rl[slot * NQ + n].x - lse2[n]);
        const float w1 = ex2_approx(rl[slot * NQ + n + 1].x - lse2[n + 1]);
        const float4 v = reinterpret_cast<const float4*>(a.part_o)[slot * MT * NT * 32 + f];
        s.x = fmaf(v.x, w0, s.x);
        s.y = fmaf(v.y, w1, s.y);
        s.z = fmaf(v.z, w0, s.z);
        s.w = fmaf(v.w, w1, s.w);
      }
      // columns of the two rows of a tile (see the V operand)
      int c0, c1;
      if constexpr (D == 64) c0 = 8 * grp + i, c1 = c0 + 4;
      else c0 = 8 * (grp * (D / 64) + 2 * (i >> 3)) + (i & 7), c1 = c0 + 8;
      __nv_bfloat16* o = a.o + (static_cast<size_t>(bh) * g + n) * D;
      o[c0] = __float2bfloat16_rn(s.x);
      o[c1] = __float2bfloat16_rn(s.z);
      if (n + 1 < g) {
        o[D + c0] = __float2bfloat16_rn(s.y);
        o[D + c1] = __float2bfloat16_rn(s.w);
      }
    }
  if (a.acc) {
    auto weight = [&](float x, int h) { return h < g ? ex2_approx(fmaf(x, fac[h], -lse2[h])) : 0.f; };
    float w[KEYS];
#pragma unroll
    for (int i = 0; i < KEYS; ++i) {
      w[i] = weight(sc[i][0].x, 0);
      if (gp > 1) w[i] += weight(sc[i][0].y, 1);
      if (gp > 2) w[i] += weight(sc[i][1].x, 2) + weight(sc[i][1].y, 3);
    }
    for (int h = 4; h < g; h += 2) {
#pragma unroll
      for (int i = 0; i < KEYS; ++i)
        if (key0 + 256 * i < len) {
          const float2 v = *reinterpret_cast<const float2*>(a.scores + (row + 256 * i) * gp + h);
          w[i] += weight(v.x, h) + weight(v.y, h + 1);
        }
    }
#pragma unroll
    for (int i = 0; i < KEYS; ++i)
      if (key0 + 256 * i < len) a.acc[row + 256 * i] = old[i] + w[i];
  }
}

}  // namespace fa
