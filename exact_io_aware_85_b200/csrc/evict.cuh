// evict.cuh — eviction from a key/value cache by accumulated attention weight: which rows of a
// prompt stay (keep), and which rows of a full cache new tokens replace (slots).
//
// Both are one selection of the n rows with the largest 32-bit keys: rows get a key in the order
// of their weight (reversed for slots), protected rows (sinks, the recent window) the largest (or
// smallest) key, a radix search finds the n-th key, and of the rows equal to it the first (or
// last) ones make up the count.
//
// Reading the weights takes a microsecond or two; what counts is the chain of steps after it.  A
// head's rows are spread over a cluster of CTAs and stay in their registers (the weights are read
// once).  The key's first eleven bits (sign, exponent, two bits of the mantissa: weights of an
// ordinary spread meet many counters, and a warp whose rows all meet one counter adds once) are
// counted over the cluster in distributed shared memory; the rows that share the n-th key's eleven
// bits, a few per cent, then go to a short list, and every CTA searches the whole list by itself.
// Where many rows share the bits (equal weights), the digits are counted over all rows.  The rows
// taken become one bit each, and a thread lists the rows of a word.
// A cluster barrier takes a microsecond and distributed shared memory gives an SM some 16 bytes a
// clock, so a head gets CTAs only while the grid stays within the SMs (64 heads of 32768 rows with
// all three digits counted over all rows: 128 CTAs 18.3 us, 256 CTAs 27 us, 64 CTAs 40 us).
// Measured: 4096 of 32768 rows in 64 heads 17 us, 512 of 131000 rows in 8 heads 18 us (24 us
// with three counted digits and ranks by ballots), one of 4096 rows in 64 heads 3.5 us.
// One row to take (a decoding step of a full cache) needs no search: one reduction over
// (key, row) pairs.
#pragma once
#include "early.cuh"
#include "sm100.cuh"

namespace fa {

constexpr int kEvictMaxCluster = 8;
constexpr int kEvictList = 4096;  // rows of a CTA that may share the n-th key's first bits

struct EvictArgs {
  const float* w;   // [B*Hkv, C]
  const int* pos;   // slots: [B*Hkv, C]
  const int* lens;  // keep: [B*Hkv] or null (C)
  int* lens_io;     // slots: [B*Hkv]
  const int* seen;  // slots: [B]
  int* out;         // keep: [B*Hkv, keep]; slots: [B*Hkv, T]
  int* count;       // keep: [B*Hkv]
  int C, Hkv, n_out, budget, n_recent, n_sink;
  int ctas;         // CTAs per head (the cluster)
};

// Order of a weight as an unsigned number: -0 counts as 0, a NaN as the largest weight.
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0xfffffffeu;
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint32_t ld_peer_u32(const void* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(peer_smem(p, rank)));
  return v;
}
__device__ __forceinline__ uint64_t ld_peer_u64(const void* p, uint32_t rank) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(peer_smem(p, rank)));
  return v;
}

// exclusive prefix sum of one number per thread over a block of W warps, and the total
template <int W>
__device__ __forceinline__ int block_scan(int x, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, s, off);
    if (lane >= off) s += y;
  }
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  const int ws = lane < W ? warp_sums[lane] : 0;
  int y = ws;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, y, off);
    if (lane >= off) y += z;
  }
  total = __shfl_sync(0xffffffffu, y, 31);
  __syncthreads();
  return s - x + __shfl_sync(0xffffffffu, y - ws, warp);
}

// One cluster per (b, key/value head).  SLOTS: the n lightest rows (the last among equals);
// otherwise the n heaviest (the first among equals).  ITEMS: rows a thread holds.
template <bool SLOTS, int ITEMS>
__global__ void __launch_bounds__(1024) fa_evict_kernel(const EvictArgs a) {
  constexpr int LIST = kEvictList, MAXC = kEvictMaxCluster;
  constexpr int THREADS = 1024, W = THREADS / 32, BINS = 2048 / THREADS;  // warps; counters a thread sums up
  __shared__ __align__(8) int hist[3][2048];
  __shared__ int warp_sums[32], lists[MAXC];
  __shared__ uint32_t gt_bits[32 * ITEMS], eq_bits[32 * ITEMS];  // a tile's rows above and at the n-th key
  __shared__ unsigned long long best_sh[32];
  __shared__ unsigned long long best_cta;
  __shared__ __align__(8) int totals[2];
  __shared__ uint32_t list[LIST];
  __shared__ int listed;
  __shared__ uint32_t sh_digit;
  __shared__ int sh_left;
  const int S = a.ctas, rank = S > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int bh = blockIdx.x / S, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const size_t base = static_cast<size_t>(bh) * a.C;
  int* const out = a.out + static_cast<size_t>(bh) * a.n_out;
  // every CTA of the head has written what the others read / has read what they wrote
  auto all_sync = [&]() {
    if (S > 1) cluster_sync_all();
    else __syncthreads();
  };
  wait_for_earlier();
  int len, n;  // rows looked at, rows to take
  int free_rows = 0, recent_from = 0;
  if (SLOTS) {
    len = max(0, min(a.lens_io[bh], a.budget));
    free_rows = min(a.budget - len, a.n_out);
    n = a.n_out - free_rows;
    recent_from = a.seen[bh / a.Hkv] - a.n_recent;
    if (rank == 0)
      for (int t = tid; t < free_rows; t += THREADS) out[t] = len + t;
  } else {
    len = a.lens ? max(0, min(a.lens[bh], a.C)) : a.C;
    n = min(len, a.n_out);
  }
  // this CTA's rows [lo, hi), in tiles of THREADS ITEMS; a warp's rows of a tile are consecutive
  const int chunk = ((len + S - 1) / S + 31) & ~31;
  const int lo = min(len, rank * chunk), hi = min(len, lo + chunk);
  constexpr int TILE = THREADS * ITEMS;
  const int tiles = (hi - lo + TILE - 1) / TILE;
  uint32_t key[ITEMS];
  auto row_of = [&](int tile, int i) { return lo + tile * TILE + warp * (32 * ITEMS) + i * 32 + lane; };
  auto load = [&](int tile) {
    float w[ITEMS];
    int p[ITEMS];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int j = row_of(tile, i);
      w[i] = j < hi ? a.w[base + j] : 0.f;
      if (SLOTS) p[i] = j < hi ? a.pos[base + j] : 0;
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int j = row_of(tile, i);
      if (SLOTS) key[i] = ~((p[i] < a.n_sink || p[i] >= recent_from) ? 0xffffffffu : weight_key(w[i]));
      else key[i] = (j < a.n_sink || j >= len - a.n_recent) ? 0xffffffffu : weight_key(w[i]);
    }
  };
  for (int i = tid; i < 3 * 2048; i += THREADS) hist[0][i] = 0;
  if (tid == 0) listed = 0;
  if (tiles == 1) load(0);
  __syncthreads();

  if (n == 1) {
    // ---- one row: the largest key, then the last (first) row
    unsigned long long best = 0;
    for (int t = 0; t < tiles; ++t) {
      if (tiles > 1) load(t);
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        const int j = row_of(t, i);
        const uint32_t order = SLOTS ? static_cast<uint32_t>(j) + 1u : ~static_cast<uint32_t>(j);
        if (j < hi) best = max(best, static_cast<unsigned long long>(key[i]) << 32 | order);
      }
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, off));
    if (lane == 0) best_sh[warp] = best;
    __syncthreads();
    if (warp == 0) {
      best = lane < W ? best_sh[lane] : 0;
#pragma unroll
      for (int off = 16; off; off >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, off));
      if (lane == 0) best_cta = best;
    }
    all_sync();
    if (S > 1 && rank == 0 && tid == 0)
      for (int r = 1; r < S; ++r) best = max(best, static_cast<unsigned long long>(ld_peer_u64(&best_cta, r)));
    if (rank == 0 && tid == 0) {
      const uint32_t order = static_cast<uint32_t>(best);
      out[free_rows] = static_cast<int>(SLOTS ? order - 1u : ~order);
    }
    if (S > 1) cluster_sync_all();
  } else if (n > 1) {
    // ---- the n-th key
    uint32_t prefix = 0;
    int left = n;  // rows still to take among those that share the prefix
    // one digit of it from counters c (the largest digit's first): the digit, and what is left
    auto find = [&](const int (&c)[BINS], int shift) {
      int sum = 0;
#pragma unroll
      for (int x = 0; x < BINS; ++x) sum += c[x];
      int tot;
      int above = block_scan<W>(sum, warp_sums, tot);
      if (above < left && left <= above + sum) {
        int x = 0;
#pragma unroll
        for (int y = 0; y < BINS - 1; ++y)
          if (x == y && left > above + c[y]) above += c[y], ++x;
        sh_digit = 2047 - BINS * tid - x;
        sh_left = left - above;
      }
      __syncthreads();
      prefix |= sh_digit << shift;
      left = sh_left;
    };
    // the rows' digit at `shift`, of those that share the prefix above it, into counters h
    auto count_rows = [&](int* h, int shift, int bits) {
      const uint32_t mask = (1u << bits) - 1u;
      for (int t = 0; t < tiles; ++t) {
        if (tiles > 1) load(t);
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
          const bool in = row_of(t, i) < hi && (shift == 21 || (key[i] >> (shift + bits)) == (prefix >> (shift + bits)));
          const uint32_t digit = in ? (key[i] >> shift) & mask : 0xffffffffu;
          if (__all_sync(0xffffffffu, digit == __shfl_sync(0xffffffffu, digit, 0))) {
            if (lane == 0 && in) atomicAdd(&h[digit], 32);
          } else if (in) {
            atomicAdd(&h[digit], 1);
          }
        }
      }
    };
    // all CTAs' counters of this thread's digits
    auto gather = [&](const int* h, int (&c)[BINS]) {
      const int top = 2047 - BINS * tid;
#pragma unroll
      for (int x = 0; x < BINS; ++x) c[x] = S > 1 ? 0 : h[top - x];
      if (S > 1) {
        uint64_t v[MAXC][BINS / 2];  // on their way together
#pragma unroll
          for (int r = 0; r < MAXC; ++r)
#pragma unroll
            for (int x = 0; x < BINS / 2; ++x) v[r][x] = r < S ? ld_peer_u64(&h[top - 2 * x - 1], r) : 0;
#pragma unroll
          for (int x = 0; x < BINS / 2; ++x)
#pragma unroll
            for (int r = 0; r < MAXC; ++r) {
              c[2 * x + 1] += static_cast<int>(v[r][x] & 0xffffffffu);
              c[2 * x] += static_cast<int>(v[r][x] >> 32);
            }
      }
    };
    int c[BINS];
    count_rows(hist[0], 21, 11);
    all_sync();
    gather(hist[0], c);
    find(c, 21);
    // the rows that share these bits, into the list
    for (int t = 0; t < tiles; ++t) {
      if (tiles > 1) load(t);
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        const bool in = row_of(t, i) < hi && (key[i] >> 21) == (prefix >> 21);
        const uint32_t b = __ballot_sync(0xffffffffu, in);
        if (b) {
          int at = 0;
          if (lane == 0) at = atomicAdd(&listed, __popc(b));
          at = __shfl_sync(0xffffffffu, at, 0) + __popc(b & ((1u << lane) - 1u));
          if (in && at < LIST) list[at] = key[i];
        }
      }
    }
    all_sync();
    if (tid < MAXC) lists[tid] = tid >= S ? 0 : S > 1 ? static_cast<int>(ld_peer_u32(&listed, tid)) : listed;
    __syncthreads();
    int m[MAXC], all = 0;
#pragma unroll
    for (int r = 0; r < MAXC; ++r) all += m[r] = lists[r];
    const bool fits = all <= LIST;
    uint32_t mine[LIST / THREADS];  // the whole list, over this CTA's threads
#pragma unroll
    for (int x = 0; x < LIST / THREADS; ++x) {
      int r = 0, at = tid + x * THREADS;
      const bool in = fits && at < all;
#pragma unroll
      for (int y = 0; y < MAXC - 1; ++y)
        if (r == y && at >= m[y]) at -= m[y], ++r;
      mine[x] = !in ? 0u : S > 1 ? ld_peer_u32(&list[at], r) : list[at];
    }
    for (int d = 1; d < 3; ++d) {
      const int shift = d == 1 ? 10 : 0, bits = d == 1 ? 11 : 10;
      if (fits) {
        const uint32_t mask = (1u << bits) - 1u;
#pragma unroll
        for (int x = 0; x < LIST / THREADS; ++x)
          if (tid + x * THREADS < all && (d == 1 || (mine[x] >> 10) == (prefix >> 10)))
            atomicAdd(&hist[d][(mine[x] >> shift) & mask], 1);
        __syncthreads();
#pragma unroll
        for (int x = 0; x < BINS; ++x) c[x] = hist[d][2047 - BINS * tid - x];
      } else {
        count_rows(hist[d], shift, bits);
        all_sync();
        gather(hist[d], c);
      }
      find(c, shift);
    }
    // ---- rows above the key, and `left` of those at it, in ascending order: one bit a row, a
    // thread lists the rows of a word
    auto mark = [&](int t) {
      if (tiles > 1) load(t);
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        const bool in = row_of(t, i) < hi;
        const uint32_t bg = __ballot_sync(0xffffffffu, in && key[i] > prefix);
        const uint32_t be = __ballot_sync(0xffffffffu, in && key[i] == prefix);
        if (lane == 0) gt_bits[warp * ITEMS + i] = bg, eq_bits[warp * ITEMS + i] = be;
      }
      __syncthreads();
    };
    uint32_t g = 0, e = 0;
    auto scan_tile = [&](int& tot) {  // this thread's word; rows before it, above in the low half
      const bool has = tid < 32 * ITEMS;
      g = has ? gt_bits[tid] : 0;
      e = has ? eq_bits[tid] : 0;
      return block_scan<W>(__popc(g) | __popc(e) << 16, warp_sums, tot);
    };
    int gt_cta = 0, eq_cta = 0, before = 0;
    for (int t = 0; t < tiles; ++t) {
      mark(t);
      int tot;
      before = scan_tile(tot);
      gt_cta += tot & 0xffff;
      eq_cta += tot >> 16;
    }
    int gt_before = 0, eq_before = 0, eq_all = eq_cta;
    if (S > 1) {
      if (tid == 0) totals[0] = gt_cta, totals[1] = eq_cta;
      cluster_sync_all();
      eq_all = 0;
      uint64_t v[MAXC];
#pragma unroll
      for (int r = 0; r < MAXC; ++r) v[r] = r < S ? ld_peer_u64(totals, r) : 0;
#pragma unroll
      for (int r = 0; r < MAXC; ++r) {
        const int vg = static_cast<int>(v[r] & 0xffffffffu), ve = static_cast<int>(v[r] >> 32);
        if (r < rank) gt_before += vg, eq_before += ve;
        eq_all += ve;
      }
    }
    const int skip = SLOTS ? eq_all - left : 0;  // equals that are not taken come first
    auto taken = [&](int r) { return SLOTS ? max(0, r - skip) : min(r, left); };  // of the first r equals
    for (int t = 0; t < tiles; ++t) {
      if (tiles > 1) {
        mark(t);
        int tot;
        before = scan_tile(tot);
        gt_before += before & 0xffff;
        eq_before += before >> 16;
        before = tot - before;  // what the next tile has to add
      } else {
        gt_before += before & 0xffff;
        eq_before += before >> 16;
      }
      int at = gt_before, r = eq_before;
      const int row0 = lo + t * TILE + tid * 32;
      for (uint32_t bits = g | e; bits; bits &= bits - 1) {
        const int b = __ffs(bits) - 1;
        if (g >> b & 1) {
          out[free_rows + at + taken(r)] = row0 + b;
          ++at;
        } else {
          if (taken(r + 1) > taken(r)) out[free_rows + at + taken(r)] = row0 + b;
          ++r;
        }
      }
      if (tiles > 1) {
        gt_before += before & 0xffff;
        eq_before += before >> 16;
      }
    }
    if (S > 1) cluster_sync_all();  // no CTA ends while another may read its shared memory
  }
  if (SLOTS) {
    if (S > 1 && n < 1) cluster_sync_all();  // every CTA has read the length
    if (rank == 0 && tid == 0)
      a.lens_io[bh] = static_cast<int>(min(static_cast<long long>(a.budget), static_cast<long long>(len) + a.n_out));
  } else {
    if (rank == 0) {
      for (int t = n + tid; t < a.n_out; t += THREADS) out[t] = -1;
      if (tid == 0) a.count[bh] = n;
    }
  }
}

}  // namespace fa
