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
// With codes c, scores are x_j = fac_h ks_j (q_h . c_j) in log2 units, and the output is
// sum_j 2^(x_j - m) vs_j c_j / sum_j 2^(x_j - m): the scales stay outside the products, whose
// cache side is small whole numbers.  The step is bound by reading the cache, (d + 4) bytes a
// row; at the copy rate an SM meets some 45 codes per clock, so what it spends per code decides.
//
//   * Warps work alone: a warp takes 32 keys at a time, holds their running maximum, sum and
//     output for all query heads that share them, and meets the other warps only when the
//     CTA's part of a head ends.  Its rows arrive by bulk copies through a ring of its own.
//   * Products are warp-level m16n8k16 MMAs with the codes on the 16-wide side and the query
//     heads on the 8-wide one.  Which key is which row, and which element which column, is free
//     as long as both operands agree, so every lane reads its codes from shared memory as whole
//     words and unpacks them in place: for K the pairs of a word are consecutive k entries; for
//     V the same element of two keys is, and the eight elements of a word belong to eight MMAs.
//   * Unpacking: (w & 0xf000f) | 0x6400_6400 is the fp16 pair 1024 + code, and the nibbles at
//     bits 4-7 read 1024 + 16 code, so one shift serves four pairs; one packed add or fma leaves
//     the code itself, exact.  V's codes go to bf16 (128 + code), beside P times the row's scale,
//     which needs the exponent range.
//   * q in fp16, scaled by a power of two per head so that its largest element is near 2^14: a
//     bf16 query is exact; a rotated query is held as a sum of two fp16 numbers (22 bits).  With at most four
//     heads the second number sits in the MMA's unused columns.
//   * Work is one list of blocks (32 keys a warp) over all heads' lengths, cut into equal parts,
//     one per CTA: ragged batches fill the GPU evenly.
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
  float* part_ml;          // [grid + B*Hkv, 8 NT, 2]
  int* first;              // [B*Hkv + 1]: blocks before each head
  float* scores;           // [B*Hkv, C, gp] in log2 units, or null
  int C, BHkv, g, gp, grid;
  float scale_log2;        // softmax scale * log2(e), / d when rotated
};

__device__ __forceinline__ int kv4_len(const int* lens, int bh, int C) { return max(0, min(lens[bh], C)); }

constexpr float kKv4Lowest = -3.0e38f;  // the running maximum before the first key

template <int D, int NT>
struct Kv4Cfg {
  static constexpr int NW = (NT == 1 && D <= 128) ? 16 : 8;  // warps: 128 or 255 registers a thread
  static constexpr int THREADS = NW * 32;
  static constexpr int BLOCK = NW * 32;                      // keys per block
  static constexpr int ROW = D / 2;                          // bytes of codes per row
  static constexpr int STAGE = 2 * 32 * ROW + 128;           // K, V codes and scales of 32 rows
  static constexpr int STAGES = 200 * 1024 / (NW * STAGE);
  static constexpr int KSTEPS = D / 16;
  static constexpr int MT = D / 16;                          // 16-row tiles of O^T
  static constexpr int MC = 4;                               // ... merged at a time
  static constexpr int OFF_Q = NW * STAGES * STAGE;          // fp16 B fragments: [NT][2][KSTEPS][32] x 8 bytes
  static constexpr int OFF_RED = OFF_Q;                      // the merge's buffer lies over them
  static constexpr int Q_BYTES = NT * 2 * KSTEPS * 32 * 8;
  static constexpr int RED_BYTES = NW * NT * 32 * 16;        // one 16-row tile of every warp
  static constexpr int OFF_ML = OFF_Q + (Q_BYTES > RED_BYTES ? Q_BYTES : RED_BYTES);  // [2][NW][8 NT]
  static constexpr int OFF_FAC = OFF_ML + 2 * NW * 8 * NT * 4;  // [8 NT]
  static constexpr int OFF_BAR = OFF_FAC + 8 * NT * 4;
  static constexpr int OFF_MISC = OFF_BAR + NW * STAGES * 8;
  static constexpr int BYTES = OFF_MISC + 256;
  static_assert(STAGES >= 2 && BYTES <= 232448, "shared memory budget");
};

__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
// the fp16 pairs (e0, e4), (e1, e5), (e2, e6), (e3, e7) of the eight codes in w, less 8
__device__ __forceinline__ void kv4_unpack_f16(uint32_t w, uint32_t (&r)[4]) {
  const uint32_t w8 = w >> 8;
  const uint32_t magic = 0x64006400u, off = 0xE408E408u /* -1032 */, s16 = 0x2C002C00u /* 1/16 */, o16 = 0xD480D480u /* -72 */;
  uint32_t x;
  x = and_or(w, 0x000f000fu, magic);
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r[0]) : "r"(x), "r"(off));
  x = and_or(w, 0x00f000f0u, magic);
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r[1]) : "r"(x), "r"(s16), "r"(o16));
  x = and_or(w8, 0x000f000fu, magic);
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r[2]) : "r"(x), "r"(off));
  x = and_or(w8, 0x00f000f0u, magic);
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r[3]) : "r"(x), "r"(s16), "r"(o16));
}
// the bf16 pair of code i (0..3) of each half of t, less 8
__device__ __forceinline__ uint32_t kv4_unpack_bf16(uint32_t t, int i) {
  const uint32_t x = and_or(t >> (4 * i), 0x000f000fu, 0x43004300u);
  uint32_t r;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(0xC308C308u) /* -136 */);
  return r;
}
__device__ __forceinline__ void mma_16816_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ float bf16_bits_to_float(unsigned short u) {
  return __uint_as_float(static_cast<uint32_t>(u) << 16);
}

// Position in the list of blocks: a head, a block of it, and the head's length.
struct Kv4Cursor {
  int bh, blk, nblk, len;
};

template <int D, int NT>
__global__ void __launch_bounds__(Kv4Cfg<D, NT>::THREADS, 1) fa_kv4_decode_kernel(const Kv4DecodeArgs a) {
  using L = Kv4Cfg<D, NT>;
  constexpr int NW = L::NW, ST = L::STAGES, NQ = 8 * NT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int grp = lane >> 2, tq = lane & 3;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR) + warp * ST;
  volatile int* const abort_sh = reinterpret_cast<volatile int*>(smem + L::OFF_MISC);
  int* const scan = reinterpret_cast<int*>(smem + L::OFF_MISC + 16);  // [NW + 4]
  float* const fac_sh = reinterpret_cast<float*>(smem + L::OFF_FAC);
  float* const wm = reinterpret_cast<float*>(smem + L::OFF_ML);  // [NW][NQ]
  float* const wl = wm + NW * NQ;
  asm volatile("griddepcontrol.launch_dependents;");
  if (tid == 0) *abort_sh = 0;
  if (lane == 0) {
    for (int s = 0; s < ST; ++s) mbar_init(&bars[s], 1);
    fence_mbar_init();
  }
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
  for (int w = 0; w < NW; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  const int n_cta = max(1, min(a.grid, total));  // the others have nothing to do
  const int u0 = static_cast<int>(min(static_cast<long long>(blockIdx.x) * total / n_cta, static_cast<long long>(total)));
  const int u1 = static_cast<int>(min(static_cast<long long>(blockIdx.x + 1) * total / n_cta, static_cast<long long>(total)));
  if (blockIdx.x == 0) {
    int f = before;
    for (int h = h0; h < h1; ++h) {
      a.first[h] = f;
      f += nblocks(kv4_len(a.lens, h, a.C));
    }
    if (tid == 0) a.first[a.BHkv] = total;
  }
  if (u0 >= u1) return;
  int* const start = scan + NW;
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
  Kv4Cursor cur, nxt;
  cur.bh = start[0];
  cur.blk = start[1];
  cur.len = kv4_len(a.lens, cur.bh, a.C);
  cur.nblk = nblocks(cur.len);
  nxt = cur;
  int left = u1 - u0, ahead = u1 - u0;  // blocks to work on, blocks to load
  auto step = [&](Kv4Cursor& c, int& n) {
    --n;
    if (++c.blk == c.nblk && n > 0) {
      c.blk = 0;
      do {
        c.len = kv4_len(a.lens, ++c.bh, a.C);
        c.nblk = nblocks(c.len);
      } while (c.nblk == 0);
    }
  };
  uint8_t* const ring = smem + warp * ST * L::STAGE;
  int put = 0, got = 0;  // copies started, copies waited for
  // starts the copies of this warp's next block that has keys; every lane follows
  auto load_next = [&]() {
    while (ahead > 0) {
      const int key0 = nxt.blk * L::BLOCK + warp * 32;
      const bool some = key0 < nxt.len;
      if (some && lane == 0) {
        uint8_t* st = ring + (put % ST) * L::STAGE;
        uint64_t* bar = &bars[put % ST];
        const size_t row = static_cast<size_t>(nxt.bh) * a.C + key0;
        mbar_arrive_expect_tx(bar, L::STAGE);
        bulk_load(st, a.kc + row * L::ROW, 32 * L::ROW, bar);
        bulk_load(st + 64 * L::ROW, a.ks + row, 64, bar);
        bulk_load(st + 32 * L::ROW, a.vc + row * L::ROW, 32 * L::ROW, bar);
        bulk_load(st + 64 * L::ROW + 64, a.vs + row, 64, bar);
      }
      step(nxt, ahead);
      if (some) {
        ++put;
        return;
      }
    }
  };
#pragma unroll 1
  for (int s = 0; s < ST; ++s) load_next();

  const int g = a.g;
  const bool rotated = a.signs != nullptr;
  const bool dup = NT == 1 && rotated && g <= 4;  // second halves of q in columns 4-7
  const bool two = rotated && !dup;
  bool ok = true;

  while (left > 0) {
    // ================= one head: q into fragments =======================================
    const int bh = cur.bh;
    __half* const qf = reinterpret_cast<__half*>(smem + L::OFF_Q);
    constexpr int EPL = D / 4 < 32 ? D / 4 : 32;  // elements of a lane's chunk of a key
    for (int i = tid; i < L::Q_BYTES / 16; i += L::THREADS) reinterpret_cast<uint4*>(qf)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    for (int n = warp; n < g; n += NW) {
      constexpr int E = D / 32;
      const __nv_bfloat16* qrow = a.q + (static_cast<size_t>(bh) * g + n) * D + lane * E;
      float y[E];
#pragma unroll
      for (int i = 0; i < E; ++i) y[i] = __bfloat162float(qrow[i]);
      if (rotated) {
#pragma unroll
        for (int i = 0; i < E; ++i) y[i] *= a.signs[lane * E + i];
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
      // 2^k with |q| 2^k < 2^15; a query that is not finite goes through as it is
      int k = 14 - (static_cast<int>(top >> 23) - 127);
      if (top >= 0x7f800000u) k = 0;
      k = min(k, 126);  // 2^k and 2^-k stay normal
      const float up = __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float x = y[i] * up;
        const __half hi = __float2half_rn(x);
        const __half lo = __float2half_rn(x - __half2float(hi));
        const int j = lane * E + i;
        const int c = j / (4 * EPL), r = j % (4 * EPL), e = r & 7;
        const int ks = c * (EPL / 4) + ((r % EPL) >> 3) * 2 + ((e & 3) >> 1);
        const int sub = (e & 1) * 2 + (e >> 2), ql = r / EPL;
        const int nt = n >> 3, col = n & 7;
        qf[((((nt * 2) * L::KSTEPS + ks) * 32 + col * 4 + ql) << 2) + sub] = hi;
        if (rotated) {
          if (dup) qf[((ks * 32 + (col + 4) * 4 + ql) << 2) + sub] = lo;
          else qf[((((nt * 2 + 1) * L::KSTEPS + ks) * 32 + col * 4 + ql) << 2) + sub] = lo;
        }
      }
      if (lane == 0) {
        const float f = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
        fac_sh[n] = f;
        if (dup) fac_sh[n + 4] = f;
      }
    }
    for (int n = tid; n < NQ; n += L::THREADS)
      if (n >= g && !(dup && n >= 4 && n < 4 + g)) fac_sh[n] = 0.f;
    __syncthreads();
    float fac[NT][2], m_run[NT][2], l_run[NT][2], oacc[NT][L::MT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        fac[j][c] = fac_sh[8 * j + 2 * tq + c];
        m_run[j][c] = kKv4Lowest;
        l_run[j][c] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < L::MT; ++i) oacc[j][i][0] = oacc[j][i][1] = oacc[j][i][2] = oacc[j][i][3] = 0.f;
    }
    const uint2* const qfrag = reinterpret_cast<const uint2*>(qf) + lane;
    // ================= the head's blocks =================================================
    do {
      const int key0 = cur.blk * L::BLOCK + warp * 32;
      if (ok && key0 < cur.len) {
        const uint8_t* st = ring + (got % ST) * L::STAGE;
        ok = __all_sync(0xffffffffu, mbar_wait(&bars[got % ST], (got / ST) & 1, abort_sh, 30));
        ++got;
        if (ok) {
          // row r of a 16-key tile is key r ^ ((r >> 1) & 1): the rows that one load touches then
          // alternate between the two halves of a 128-byte line
          const int kr = grp ^ ((grp >> 1) & 1);
          float x[2][NT][4];
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int j = 0; j < NT; ++j) x[t][j][0] = x[t][j][1] = x[t][j][2] = x[t][j][3] = 0.f;
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
            for (int i = 0; i < EPL / 8; ++i) {
              uint32_t u[4][4];
#pragma unroll
              for (int r = 0; r < 4; ++r) kv4_unpack_f16(w[r][i], u[r]);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int ks = c * (EPL / 4) + 2 * i + h;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                  const uint2 b = qfrag[((j * 2) * L::KSTEPS + ks) * 32];
                  mma_16816_f16(x[0][j], u[0][2 * h], u[1][2 * h], u[0][2 * h + 1], u[1][2 * h + 1], b.x, b.y);
                  mma_16816_f16(x[1][j], u[2][2 * h], u[3][2 * h], u[2][2 * h + 1], u[3][2 * h + 1], b.x, b.y);
                  if (two) {
                    const uint2 b2 = qfrag[((j * 2 + 1) * L::KSTEPS + ks) * 32];
                    mma_16816_f16(x[0][j], u[0][2 * h], u[1][2 * h], u[0][2 * h + 1], u[1][2 * h + 1], b2.x, b2.y);
                    mma_16816_f16(x[1][j], u[2][2 * h], u[3][2 * h], u[2][2 * h + 1], u[3][2 * h + 1], b2.x, b2.y);
                  }
                }
              }
            }
          }
          float vs[4];
          const unsigned short* const sc = reinterpret_cast<const unsigned short*>(st + 64 * L::ROW);
          const bool tail = key0 + 32 > cur.len;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int key = 8 * r + kr;
            const float ks = bf16_bits_to_float(sc[key]);
            vs[r] = bf16_bits_to_float(sc[32 + key]);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              float& x0 = x[r >> 1][j][2 * (r & 1)];
              float& x1 = x[r >> 1][j][2 * (r & 1) + 1];
              if (NT == 1 && dup) {
                x0 += __shfl_xor_sync(0xffffffffu, x0, 2);
                x1 += __shfl_xor_sync(0xffffffffu, x1, 2);
              }
              x0 *= ks * fac[j][0];
              x1 *= ks * fac[j][1];
            }
          }
          if (tail) {  // rows behind the last hold anything: neither their codes nor their scales count
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (key0 + 8 * r + kr >= cur.len) {
                vs[r] = 0.f;
#pragma unroll
                for (int j = 0; j < NT; ++j) x[r >> 1][j][2 * (r & 1)] = x[r >> 1][j][2 * (r & 1) + 1] = -INFINITY;
              }
          }
          if (a.scores) {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              const int n = 8 * j + 2 * tq;
              if (n < g) {
                float* p = a.scores + (static_cast<size_t>(bh) * a.C + key0 + kr) * a.gp + n;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                  if (!tail || key0 + 8 * r + kr < cur.len) {
                    if (a.gp == 1) p[8 * r] = x[r >> 1][j][2 * (r & 1)];
                    else *reinterpret_cast<float2*>(p + 8 * r * a.gp) =
                             make_float2(x[r >> 1][j][2 * (r & 1)], x[r >> 1][j][2 * (r & 1) + 1]);
                  }
              }
            }
          }
          // ---- the running maximum moves only when a score passes it by more than 2^8 -------
          bool over = false;
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int c = 0; c < 2; ++c)
              over = over || fmaxf(fmaxf(x[0][j][c], x[0][j][c + 2]), fmaxf(x[1][j][c], x[1][j][c + 2])) > m_run[j][c] + 8.f;
          if (__any_sync(0xffffffffu, over)) {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              float al[2];
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                float mx = fmaxf(fmaxf(x[0][j][c], x[0][j][c + 2]), fmaxf(x[1][j][c], x[1][j][c + 2]));
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                const float m_new = fmaxf(m_run[j][c], mx);
                al[c] = ex2_approx(m_run[j][c] - m_new);
                m_run[j][c] = m_new;
                l_run[j][c] *= al[c];
              }
#pragma unroll
              for (int i = 0; i < L::MT; ++i) {
                oacc[j][i][0] *= al[0];
                oacc[j][i][1] *= al[1];
                oacc[j][i][2] *= al[0];
                oacc[j][i][3] *= al[1];
              }
            }
          }
          // ---- P (times the rows' scales) as the B operand -----------------------------------
          uint32_t pb[2][NT][2];
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              const float p0 = ex2_approx(x[t][j][0] - m_run[j][0]), p1 = ex2_approx(x[t][j][1] - m_run[j][1]);
              const float p2 = ex2_approx(x[t][j][2] - m_run[j][0]), p3 = ex2_approx(x[t][j][3] - m_run[j][1]);
              l_run[j][0] += p0 + p2;
              l_run[j][1] += p1 + p3;
              pb[t][j][0] = movmatrix_trans(pack_bf16x2(p0 * vs[2 * t], p1 * vs[2 * t]));
              pb[t][j][1] = movmatrix_trans(pack_bf16x2(p2 * vs[2 * t + 1], p3 * vs[2 * t + 1]));
            }
          // ---- O^T += V^T P^T ------------------------------------------------------------------
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            constexpr int WPL = D / 64;  // words of a lane per key: octets WPL grp ..
            uint32_t w[4][WPL];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int key = 16 * t + 8 * (r >> 1) + ((2 * tq + (r & 1)) ^ (tq & 1));
              const uint8_t* p = st + 32 * L::ROW + key * L::ROW + grp * 4 * WPL;
              if constexpr (WPL == 1) {
                w[r][0] = *reinterpret_cast<const uint32_t*>(p);
              } else if constexpr (WPL == 2) {
                const uint2 v = *reinterpret_cast<const uint2*>(p);
                w[r][0] = v.x, w[r][1] = v.y;
              } else {
                const uint4 v = *reinterpret_cast<const uint4*>(p);
                w[r][0] = v.x, w[r][1] = v.y, w[r][2] = v.z, w[r][3] = v.w;
              }
            }
            if constexpr (WPL == 1) {
              // rows 0-7: element i of octet grp, rows 8-15: element i + 4
              const uint32_t lo0 = __byte_perm(w[0][0], w[1][0], 0x5410), hi0 = __byte_perm(w[0][0], w[1][0], 0x7632);
              const uint32_t lo1 = __byte_perm(w[2][0], w[3][0], 0x5410), hi1 = __byte_perm(w[2][0], w[3][0], 0x7632);
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                  mma_16816(oacc[j][i], kv4_unpack_bf16(lo0, i), kv4_unpack_bf16(hi0, i), kv4_unpack_bf16(lo1, i),
                            kv4_unpack_bf16(hi1, i), pb[t][j][0], pb[t][j][1]);
            } else {
              // rows 0-7: element i of octet 2 s, rows 8-15: of octet 2 s + 1 (of the lane's WPL octets)
#pragma unroll
              for (int s = 0; s < WPL / 2; ++s)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                  const uint32_t sel = half ? 0x7632 : 0x5410;
                  const uint32_t a0 = __byte_perm(w[0][2 * s], w[1][2 * s], sel);
                  const uint32_t a1 = __byte_perm(w[0][2 * s + 1], w[1][2 * s + 1], sel);
                  const uint32_t a2 = __byte_perm(w[2][2 * s], w[3][2 * s], sel);
                  const uint32_t a3 = __byte_perm(w[2][2 * s + 1], w[3][2 * s + 1], sel);
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const uint32_t f0 = kv4_unpack_bf16(a0, i), f1 = kv4_unpack_bf16(a1, i);
                    const uint32_t f2 = kv4_unpack_bf16(a2, i), f3 = kv4_unpack_bf16(a3, i);
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                      mma_16816(oacc[j][s * 8 + half * 4 + i], f0, f1, f2, f3, pb[t][j][0], pb[t][j][1]);
                  }
                }
            }
          }
          __syncwarp();  // every lane has read the stage
          load_next();
        }
      }
      step(cur, left);
    } while (left > 0 && cur.bh == bh);
    // ================= merge the warps ====================================================
    float mx[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float l = l_run[j][c];
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
        l_run[j][c] = l;
        if (grp == 0) wm[warp * NQ + 8 * j + 2 * tq + c] = m_run[j][c];
      }
    __syncthreads();
    const size_t slot = static_cast<size_t>(blockIdx.x) + bh;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int n = 8 * j + 2 * tq + c;
        float M = kKv4Lowest;
        for (int w = 0; w < NW; ++w) M = fmaxf(M, wm[w * NQ + n]);
        mx[j][c] = M;
        const float f = ex2_approx(m_run[j][c] - M);
        if (grp == 0) wl[warp * NQ + n] = l_run[j][c] * f;
#pragma unroll
        for (int i = 0; i < L::MT; ++i) {
          oacc[j][i][c] *= f;
          oacc[j][i][c + 2] *= f;
        }
      }
    __syncthreads();
    if (warp == 0 && grp == 0) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int n = 8 * j + 2 * tq + c;
          float l = 0.f;
          for (int w = 0; w < NW; ++w) l += wl[w * NQ + n];
          a.part_ml[(slot * NQ + n) * 2] = mx[j][c];
          a.part_ml[(slot * NQ + n) * 2 + 1] = l;
        }
    }
    float4* const red = reinterpret_cast<float4*>(smem + L::OFF_RED);  // [NW][NT][32]
#pragma unroll
    for (int i = 0; i < L::MT; ++i) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
        red[(warp * NT + j) * 32 + lane] = make_float4(oacc[j][i][0], oacc[j][i][1], oacc[j][i][2], oacc[j][i][3]);
      __syncthreads();
      if (tid < NT * 32) {
        float4 s = red[tid];
        for (int w = 1; w < NW; ++w) {
          const float4 v = red[w * NT * 32 + tid];
          s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
        reinterpret_cast<float4*>(a.part_o)[(slot * L::MT + i) * NT * 32 + tid] = s;
      }
      __syncthreads();
    }
  }
  // every copy has landed before the block ends
  if (lane == 0)
    for (; got < put; ++got) mbar_wait_drain(&bars[got % ST], (got / ST) & 1, 100000000ull);
}

// Joins the parts of a head by their maxima: O, LSE, and each key's weight summed over the
// query heads that share it.  grid (key chunks, B*Hkv).
template <int D, int NT>
__global__ void __launch_bounds__(256) fa_kv4_combine_kernel(const Kv4DecodeArgs a, int chunk) {
  constexpr int NQ = 8 * NT, MT = D / 16;
  __shared__ float lse2[NQ];
  const int bh = blockIdx.y, g = a.g, tid = threadIdx.x;
  const int len = kv4_len(a.lens, bh, a.C);
  if (blockIdx.x > 0 && blockIdx.x * chunk >= len) return;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the CTAs that worked on this head
  const long long total = a.first[a.BHkv], b0 = a.first[bh], b1 = a.first[bh + 1];
  int i0 = 0, i1 = -1;
  if (b1 > b0) {
    const long long n_cta = min(static_cast<long long>(a.grid), total);
    i0 = static_cast<int>(((b0 + 1) * n_cta - 1) / total);
    i1 = static_cast<int>((b1 * n_cta - 1) / total);
  }
  if (tid < NQ) {
    float M = kKv4Lowest, L = 0.f;
    for (int i = i0; i <= i1; ++i) M = fmaxf(M, a.part_ml[((static_cast<size_t>(i) + bh) * NQ + tid) * 2]);
    for (int i = i0; i <= i1; ++i) {
      const float* ml = a.part_ml + ((static_cast<size_t>(i) + bh) * NQ + tid) * 2;
      L += ml[1] * ex2_approx(ml[0] - M);
    }
    lse2[tid] = len > 0 ? M + log2f(L) : -INFINITY;
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
        const float w0 = ex2_approx(a.part_ml[(slot * NQ + n) * 2] - lse2[n]);
        const float w1 = ex2_approx(a.part_ml[(slot * NQ + n + 1) * 2] - lse2[n + 1]);
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
    const int gp = a.gp;
    for (int key = blockIdx.x * chunk + tid; key < min(len, (blockIdx.x + 1) * chunk); key += 256) {
      const size_t row = static_cast<size_t>(bh) * a.C + key;
      float w = 0.f;
      for (int h = 0; h < g; ++h) w += ex2_approx(a.scores[row * gp + h] - lse2[h]);
      a.acc[row] += w;
    }
  }
}

}  // namespace fa
