// evict.cuh — eviction from a key/value cache by accumulated attention weight: which rows of a
// prompt stay (keep), and which rows of a full cache new tokens replace (slots).
//
// Both are one selection: rows get a 32-bit key in the order of their weight, protected rows
// (sinks, the recent window) the largest key, and a radix search over the key's bytes finds the
// value of the k-th row; rows equal to it are taken in row order until the count is met.
#pragma once
#include "sm100.cuh"

namespace fa {

constexpr int kEvictThreads = 1024;

struct EvictArgs {
  const float* w;   // [B*Hkv, C]
  const int* pos;   // slots: [B*Hkv, C]
  const int* lens;  // keep: [B*Hkv] or null (C)
  int* lens_io;     // slots: [B*Hkv]
  const int* seen;  // slots: [B]
  int* out;         // keep: [B*Hkv, keep]; slots: [B*Hkv, T]
  int* count;       // keep: [B*Hkv]
  int C, Hkv, n_out, budget, n_recent, n_sink;
};

// Order of a weight as an unsigned number: -0 counts as 0, a NaN as the largest weight.
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0xfffffffeu;
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// exclusive prefix sum of one count per thread over the block, and the total
__device__ __forceinline__ int block_scan(int x, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, s, off);
    if (lane >= off) s += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  if (warp == 0) {
    int y = warp_sums[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, y, off);
      if (lane >= off) y += z;
    }
    warp_sums[lane] = y;
  }
  __syncthreads();
  total = warp_sums[31];
  return s - x + (warp ? warp_sums[warp - 1] : 0);
}

// One CTA per (b, key/value head).  SLOTS: take the n lightest rows (last row first among equals);
// otherwise keep the n heaviest (first row first among equals).
template <bool SLOTS>
__global__ void __launch_bounds__(kEvictThreads) fa_evict_kernel(const EvictArgs a) {
  __shared__ int hist[256];
  __shared__ int warp_sums[32];
  __shared__ uint32_t sh_digit;
  __shared__ int sh_left;
  const int bh = blockIdx.x, tid = threadIdx.x;
  const size_t base = static_cast<size_t>(bh) * a.C;
  int* out = a.out + static_cast<size_t>(bh) * a.n_out;
  int len, n;  // rows looked at, rows to take
  int free_rows = 0, recent_from = 0;
  if (SLOTS) {
    len = max(0, min(a.lens_io[bh], a.budget));
    free_rows = min(a.budget - len, a.n_out);
    n = a.n_out - free_rows;
    recent_from = a.seen[bh / a.Hkv] - a.n_recent;
    for (int t = tid; t < free_rows; t += kEvictThreads) out[t] = len + t;
  } else {
    len = a.lens ? max(0, min(a.lens[bh], a.C)) : a.C;
    n = min(len, a.n_out);
  }
  // keys such that the rows to take are those with the largest keys
  auto key_of = [&](int j) -> uint32_t {
    if (SLOTS) {
      const int p = a.pos[base + j];
      return ~((p < a.n_sink || p >= recent_from) ? 0xffffffffu : weight_key(a.w[base + j]));
    }
    return (j < a.n_sink || j >= len - a.n_recent) ? 0xffffffffu : weight_key(a.w[base + j]);
  };
  uint32_t prefix = 0;
  int left = n;  // rows still to take among those that share the prefix
  if (n > 0)
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kEvictThreads) hist[i] = 0;
      __syncthreads();
      for (int j = tid; j < len; j += kEvictThreads) {
        const uint32_t k = key_of(j);
        if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255], 1);
      }
      __syncthreads();
      if (tid == 0) {
        int need = left, dgt = 255;
        while (dgt > 0 && hist[dgt] < need) need -= hist[dgt--];
        sh_digit = dgt;
        sh_left = need;
      }
      __syncthreads();
      prefix |= sh_digit << shift;
      left = sh_left;
      __syncthreads();
    }
  // rows above the threshold, and `left` of those at it, in ascending order
  int total_eq = 0;
  if (SLOTS && n > 0) {  // the last rows among equals: skip the first (equal - left)
    int c = 0, tot;
    for (int j = tid; j < len; j += kEvictThreads) c += key_of(j) == prefix;
    block_scan(c, warp_sums, tot);
    total_eq = tot;
  }
  int done = 0, eq_before = 0;
  if (n > 0)
    for (int j0 = 0; j0 < len; j0 += kEvictThreads) {
      const int j = j0 + tid;
      const uint32_t k = j < len ? key_of(j) : 0u;
      const int eq = j < len && k == prefix;
      int eq_tot, tot;
      const int eq_rank = eq_before + block_scan(eq, warp_sums, eq_tot);
      const int take = j < len && (k > prefix || (eq && (SLOTS ? eq_rank >= total_eq - left : eq_rank < left)));
      const int at = done + block_scan(take, warp_sums, tot);
      if (take) out[free_rows + at] = j;
      done += tot;
      eq_before += eq_tot;
    }
  if (SLOTS) {
    if (tid == 0) a.lens_io[bh] = static_cast<int>(min(static_cast<long long>(a.budget), static_cast<long long>(len) + a.n_out));
  } else {
    for (int t = n + tid; t < a.n_out; t += kEvictThreads) out[t] = -1;
    if (tid == 0) a.count[bh] = n;
  }
}

}  // namespace fa
