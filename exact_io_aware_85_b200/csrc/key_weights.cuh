// key_weights.cuh — how much attention each key of a prompt received:
//   w[b, hk, j] = sum over the query heads h that share hk and the window's query rows i
//                 (i >= j when causal) of exp(scale q_hi . k_j - lse_hi),
// the column sums of the softmax matrix, recomputed from q, k and the forward's logsumexp as
// the backward recomputes P ("flash-attention-trading-models", "Pase hacia atras").
//
// Half of the forward's products and all of its exponentials: S^T = K Q^T on tcgen05 with the
// keys on the tensor-memory lanes, so that one thread holds one key, and the sum over the
// queries runs along its registers.  128 x 128 scores take the tensor core 512 clocks at d = 128
// and the exponential unit 1024, so part of the exponentials are computed on the FMA pipe.
//
// Work is one list of steps (a query tile against 256 keys of a key/value head), ordered by
// key/value head, sequence, key range, query head and query tile, cut into equal parts, one per
// CTA and SM.  K of the next range and Q of the next steps load while the last ones are worked on.
// A part's sums go to the workspace and a second kernel adds the parts of each key in order:
// no atomics, the same bits every time.
//   warps 0-3, 4-7  exponentials and sums of keys 0-127, 128-255 of the range
//   warp 8          TMA producer
//   warp 9          tcgen05.mma issuer and TMEM owner
//   warp 10         log-sum-exps of the step's queries into shared memory
// Tensor memory: two score tiles per key half, 4 x 128 columns.
#pragma once
#include "sm100.cuh"

namespace fa {

struct KeyWeightsArgs {
  const float* lse;        // [B*H, N]
  float* w;                // [B*Hkv, ldw]
  const int* n_rows;       // [B] or null (N)
  float* part;             // [grid + B*Hkv*ranges, 256]: slot (CTA + item)
  long long* first;        // [B*ranges + 1]: steps before each (sequence, range), and of them all
  int B, N, ldw, H, Hkv, g, window, causal, ranges, grid;
  float scale_log2;
};

// D: head dim; QT: query rows per step
template <int D, int QT>
struct KeyWeightsCfg {
  static constexpr int KEYS = 256;
  static constexpr int BOX_K = 128 * 128, TILE_K = (D / 64) * BOX_K;  // 128 keys
  static constexpr int BOX_Q = QT * 128, TILE_Q = (D / 64) * BOX_Q;
  static constexpr int KSLOTS = D <= 128 ? 2 : 1;
  static constexpr int LSLOTS = 8;
  static constexpr int QSLOTS_FIT = (221 * 1024 - KSLOTS * 2 * TILE_K) / TILE_Q;
  static constexpr int QSLOTS = QSLOTS_FIT > 6 ? 6 : QSLOTS_FIT;
  static constexpr int OFF_Q = KSLOTS * 2 * TILE_K;
  static constexpr int OFF_L = OFF_Q + QSLOTS * TILE_Q;  // float [LSLOTS][QT]
  static constexpr int SMEM_BYTES = OFF_L + LSLOTS * QT * 4 + 1024;
  static_assert(QSLOTS >= 2 && SMEM_BYTES <= 231424, "shared memory budget (1 KB is static)");
};

// The rows of a sequence and its window, and the steps of one of its key ranges.
struct KeyWeightsSeq {
  int n, lo;
};
__device__ __forceinline__ KeyWeightsSeq key_weights_seq(const KeyWeightsArgs& a, int b) {
  KeyWeightsSeq s;
  s.n = a.n_rows ? max(0, min(a.n_rows[b], a.N)) : a.N;
  s.lo = max(0, s.n - a.window);
  return s;
}
template <int QT>
__device__ __forceinline__ int key_weights_tiles(const KeyWeightsArgs& a, const KeyWeightsSeq& s, int range, int& base) {
  const int j0 = range * 256;
  base = a.causal ? max(s.lo, j0) : s.lo;
  return j0 < s.n ? (s.n - base + QT - 1) / QT : 0;
}

// Walks the steps of one CTA: every role keeps one of these and they stay in step.
template <int QT>
struct KeyWeightsCursor {
  long long left;
  int hk, e, b, range, n, base, tiles, h, tile;

  __device__ __forceinline__ void set_entry(const KeyWeightsArgs& a) {
    b = e / a.ranges;
    range = e % a.ranges;
    const KeyWeightsSeq s = key_weights_seq(a, b);
    n = s.n;
    tiles = key_weights_tiles<QT>(a, s, range, base);
  }
  // to the next entry with steps (there is one while left > 0)
  __device__ __forceinline__ void next_entry(const KeyWeightsArgs& a) {
    do {
      if (++e == a.B * a.ranges) e = 0, ++hk;
      set_entry(a);
    } while (tiles == 0);
    h = tile = 0;
  }
  // true when the step that ends was the last of its entry here
  __device__ __forceinline__ bool step(const KeyWeightsArgs& a) {
    --left;
    if (++tile == tiles) {
      tile = 0;
      if (++h == a.g) {
        if (left > 0) next_entry(a);
        return true;
      }
    }
    return left == 0;
  }
  __device__ __forceinline__ int i0() const { return base + tile * QT; }
  // does this half of the range see any query of the tile
  __device__ __forceinline__ bool live(const KeyWeightsArgs& a, int half) const {
    const int k0 = range * 256 + half * 128;
    return k0 < n && (!a.causal || i0() + QT > k0);
  }
};

// 2^x of two values on the FMA and integer pipes, like exp2_fma2, but to fp32's accuracy: the
// polynomial of degree 5 that is minimax in relative error for 2^f on [-1/2, 1/2] (Remez exchange),
// with these float32 coefficients at most 2.1e-7 off.  x <= 127.
__device__ __forceinline__ float2 exp2_fma2_f32(float2 x) {
  constexpr float c0 = 1.0000001192092896f, c1 = 0.6931469440460205f, c2 = 0.24022120237350464f,
                  c3 = 0.05550713092088699f, c4 = 0.009675540961325169f, c5 = 0.0013276472454890609f;
  x.x = fmaxf(x.x, -126.f);
  x.y = fmaxf(x.y, -126.f);
  const float2 kRound = make_float2(12582912.f, 12582912.f);  // 1.5 * 2^23
  const float2 t = fadd2(x, kRound);
  const float2 f = fsub2(x, fsub2(t, kRound));
  float2 p = ffma2(make_float2(c5, c5), f, make_float2(c4, c4));
  p = ffma2(p, f, make_float2(c3, c3));
  p = ffma2(p, f, make_float2(c2, c2));
  p = ffma2(p, f, make_float2(c1, c1));
  p = ffma2(p, f, make_float2(c0, c0));
  return make_float2(__uint_as_float(__float_as_uint(p.x) + (__float_as_uint(t.x) << 23)),
                     __uint_as_float(__float_as_uint(p.y) + (__float_as_uint(t.y) << 23)));
}

template <int D, int QT>
__global__ void __launch_bounds__(384, 1)
    fa_key_weights_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                          const KeyWeightsArgs a) {
  using C = KeyWeightsCfg<D, QT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t bar_kf[C::KSLOTS], bar_ke[C::KSLOTS], bar_qf[C::QSLOTS], bar_qe[C::QSLOTS];
  __shared__ uint64_t bar_lf[C::LSLOTS], bar_le[C::LSLOTS], bar_sf[2][2], bar_se[2][2], bar_done;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh, odd_sh[C::LSLOTS];
  __shared__ long long scan[12];
  __shared__ long long start_rem;
  __shared__ int start_e;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  asm volatile("griddepcontrol.launch_dependents;");
  if (warp == 9) {
    tmem_alloc(&tmem_base_sh, 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    abort_sh = 0;
    for (int i = 0; i < C::KSLOTS; ++i) mbar_init(&bar_kf[i], 1), mbar_init(&bar_ke[i], 1);
    for (int i = 0; i < C::QSLOTS; ++i) mbar_init(&bar_qf[i], 1), mbar_init(&bar_qe[i], 1);
    for (int i = 0; i < C::LSLOTS; ++i) mbar_init(&bar_lf[i], 1), mbar_init(&bar_le[i], 8);
    for (int i = 0; i < 4; ++i) mbar_init(&bar_sf[i >> 1][i & 1], 1), mbar_init(&bar_se[i >> 1][i & 1], 4);
    mbar_init(&bar_done, 1);
    fence_mbar_init();
  }
  // ---- this CTA's part of the list ------------------------------------------------------
  const int entries = a.B * a.ranges;
  const int per = (entries + 383) / 384, e0 = min(entries, tid * per), e1 = min(entries, e0 + per);
  auto steps = [&](int e) {
    int base;
    return static_cast<long long>(a.g) *
           key_weights_tiles<QT>(a, key_weights_seq(a, e / a.ranges), e % a.ranges, base);
  };
  long long mine = 0;
  for (int e = e0; e < e1; ++e) mine += steps(e);
  long long incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  long long before = incl - mine, per_head = 0;
  for (int w = 0; w < 12; ++w) {
    if (w < warp) before += scan[w];
    per_head += scan[w];
  }
  const long long total = per_head * a.Hkv;
  const long long n_cta = max(1ll, min(static_cast<long long>(a.grid), total));  // the others have nothing to do
  const long long u0 = min(blockIdx.x * total / n_cta, total), u1 = min((blockIdx.x + 1) * total / n_cta, total);
  if (blockIdx.x == 0) {
    long long f = before;
    for (int e = e0; e < e1; ++e) {
      a.first[e] = f;
      f += steps(e);
    }
    if (tid == 0) a.first[entries] = per_head;
  }
  const long long at = per_head > 0 ? u0 % per_head : 0;
  if (u0 < u1 && at >= before && at < before + mine) {
    long long f = before;
    int e = e0;
    while (true) {
      const long long s = steps(e);
      if (at < f + s) break;
      f += s;
      ++e;
    }
    start_e = e;
    start_rem = at - f;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  KeyWeightsCursor<QT> cur;
  cur.left = u1 - u0;
  if (cur.left > 0) {
    cur.hk = static_cast<int>(u0 / per_head);
    cur.e = start_e;
    cur.set_entry(a);
    cur.h = static_cast<int>(start_rem / cur.tiles);
    cur.tile = static_cast<int>(start_rem % cur.tiles);
  }

  if (warp == 8) {
    // ======================= TMA producer ===================================
    if (lane == 0 && cur.left > 0) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      int kt = 0, qt = 0;
      bool fresh = true;
      while (cur.left > 0) {
        if (fresh) {
          const int s = kt % C::KSLOTS;
          if (!mbar_wait(&bar_ke[s], ((kt / C::KSLOTS) & 1) ^ 1, &abort_sh, 40)) break;
          mbar_arrive_expect_tx(&bar_kf[s], 2 * C::TILE_K);
          for (int x = 0; x < 2 * (D / 64); ++x)
            tma_load_3d(smem + s * 2 * C::TILE_K + x * C::BOX_K, &tmK, &bar_kf[s], (x % (D / 64)) * 64,
                        cur.range * 256 + (x / (D / 64)) * 128, cur.b * a.Hkv + cur.hk);
          ++kt;
        }
        const int s = qt % C::QSLOTS;
        if (!mbar_wait(&bar_qe[s], ((qt / C::QSLOTS) & 1) ^ 1, &abort_sh, 41)) break;
        mbar_arrive_expect_tx(&bar_qf[s], C::TILE_Q);
        for (int x = 0; x < D / 64; ++x)
          tma_load_3d(smem + C::OFF_Q + s * C::TILE_Q + x * C::BOX_Q, &tmQ, &bar_qf[s], x * 64, cur.i0(),
                      (cur.b * a.Hkv + cur.hk) * a.g + cur.h);
        ++qt;
        fresh = cur.step(a);
      }
      // every copy has landed before the CTA ends
      for (int i = max(0, kt - C::KSLOTS); i < kt; ++i)
        mbar_wait_drain(&bar_kf[i % C::KSLOTS], (i / C::KSLOTS) & 1, 100000000ull);
      for (int i = max(0, qt - C::QSLOTS); i < qt; ++i)
        mbar_wait_drain(&bar_qf[i % C::QSLOTS], (i / C::QSLOTS) & 1, 100000000ull);
    }
    __syncwarp();
  } else if (warp == 9) {
    // ======================= tcgen05.mma issuer =============================
    if (lane == 0) {
      constexpr uint32_t idesc = make_idesc(128, QT, kFmtBF16, 0, 0);
      const uint32_t k_addr = smem_u32(smem), q_addr = smem_u32(smem + C::OFF_Q);
      int kt = 0, qt = 0, cnt[2] = {0, 0};
      bool fresh = true, ok = true;
      while (ok && cur.left > 0) {
        const int ks = kt % C::KSLOTS, qs = qt % C::QSLOTS;
        if (fresh && !(ok = mbar_wait(&bar_kf[ks], (kt / C::KSLOTS) & 1, &abort_sh, 42))) break;
        if (!(ok = mbar_wait(&bar_qf[qs], (qt / C::QSLOTS) & 1, &abort_sh, 43))) break;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (!ok || !cur.live(a, half)) continue;
          const int buf = cnt[half] & 1;
          if (!(ok = mbar_wait(&bar_se[half][buf], ((cnt[half] >> 1) & 1) ^ 1, &abort_sh, 44))) continue;
          tc_fence_after();
          const uint32_t ka = k_addr + (ks * 2 + half) * C::TILE_K, qa = q_addr + qs * C::TILE_Q;
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            mma_ss(tmem + (half * 2 + buf) * 128,
                   make_sdesc_sw128(ka + (k >> 2) * C::BOX_K + (k & 3) * 32, 16, 1024),
                   make_sdesc_sw128(qa + (k >> 2) * C::BOX_Q + (k & 3) * 32, 16, 1024), idesc, k > 0);
          mma_commit(&bar_sf[half][buf]);
          ++cnt[half];
        }
        if (!ok) break;
        mma_commit(&bar_qe[qs]);
        ++qt;
        fresh = cur.step(a);
        if (fresh) {
          mma_commit(&bar_ke[ks]);
          ++kt;
        }
      }
      // every MMA of this thread must be finished before TMEM is freed
      mma_commit(&bar_done);
      mbar_wait_drain(&bar_done, 0, 100000000ull);
    }
    __syncwarp();
  } else if (warp == 10) {
    // ======================= -log2-sum-exps =================================
    // A tile whose values are not all finite is marked: its exponentials then go the plain way.
    for (int t = 0; cur.left > 0; ++t) {
      const int s = t % C::LSLOTS;
      if (!__all_sync(0xffffffffu, mbar_wait(&bar_le[s], ((t / C::LSLOTS) & 1) ^ 1, &abort_sh, 45))) break;
      const float* lse = a.lse + (static_cast<size_t>(cur.b * a.Hkv + cur.hk) * a.g + cur.h) * a.N;
      float* to = reinterpret_cast<float*>(smem + C::OFF_L) + s * QT;
      bool odd = false;
#pragma unroll
      for (int x = 0; x < QT / 32; ++x) {
        const int i = cur.i0() + lane + 32 * x;
        const float v = i < cur.n ? -1.4426950408889634f * lse[i] : 0.f;
        odd = odd || !(fabsf(v) < 1e30f);
        to[lane + 32 * x] = v;
      }
      odd = __any_sync(0xffffffffu, odd);
      if (lane == 0) odd_sh[s] = odd;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_lf[s]);
      cur.step(a);
    }
  } else if (warp < 8) {
    // ======================= exponentials and sums ==========================
    const int half = warp >> 2, r = tid & 127;
    const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const float c = a.scale_log2;
    float w = 0.f;
    int cnt = 0;
    bool ok = true;
    for (int t = 0; ok && cur.left > 0; ++t) {
      const int s = t % C::LSLOTS;
      const int i0 = cur.i0(), k0 = cur.range * 256 + half * 128;
      if (!(ok = mbar_wait(&bar_lf[s], (t / C::LSLOTS) & 1, &abort_sh, 46))) break;
      if (cur.live(a, half)) {
        const int buf = cnt & 1;
        if (!(ok = mbar_wait(&bar_sf[half][buf], (cnt >> 1) & 1, &abort_sh, 47))) break;
        tc_fence_after();
        const uint32_t ts = tmem + lane_base + (half * 2 + buf) * 128;
        const float4* const l4 = reinterpret_cast<const float4*>(smem + C::OFF_L) + s * (QT / 4);
        const bool plain = i0 + QT <= cur.n && (!a.causal || i0 >= k0 + 127) && !odd_sh[s];
        float sv[2][32];
        tmem_ld32(ts, *reinterpret_cast<uint32_t(*)[32]>(sv[0]));
        float2 sum[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        const float2 c2 = make_float2(c, c);
#pragma unroll
        for (int ch = 0; ch < QT / 32; ++ch) {
          tmem_wait_ld();
          if (ch + 1 < QT / 32) {
            tmem_ld32(ts + 32 * (ch + 1), *reinterpret_cast<uint32_t(*)[32]>(sv[(ch + 1) & 1]));
          } else {
            // the scores are in registers: their columns are free
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_se[half][buf]);
          }
          const float* const x = sv[ch & 1];
          if (plain) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float4 l = l4[ch * 8 + e];
              const float2 a0 = ffma2(make_float2(x[4 * e], x[4 * e + 1]), c2, make_float2(l.x, l.y));
              const float2 a1 = ffma2(make_float2(x[4 * e + 2], x[4 * e + 3]), c2, make_float2(l.z, l.w));
              // 3 of every 8 pairs on the FMA pipe
              float2 p0, p1;
              if ((e & 3) == 0 || (e & 3) == 2) p0 = exp2_fma2_f32(a0);
              else p0 = make_float2(ex2_approx(a0.x), ex2_approx(a0.y));
              if ((e & 3) == 1) p1 = exp2_fma2_f32(a1);
              else p1 = make_float2(ex2_approx(a1.x), ex2_approx(a1.y));
              sum[e & 1] = fadd2(sum[e & 1], p0);
              sum[2 + (e & 1)] = fadd2(sum[2 + (e & 1)], p1);
            }
          } else {
            const int j = k0 + r;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const int i = i0 + ch * 32 + e;
              const float4 l = l4[ch * 8 + (e >> 2)];
              const float lv = (e & 3) == 0 ? l.x : (e & 3) == 1 ? l.y : (e & 3) == 2 ? l.z : l.w;
              const float p = ex2_approx(fmaf(x[e], c, lv));
              if (i < cur.n && (!a.causal || i >= j)) sum[e & 3].x += p;
            }
          }
        }
        const float2 s01 = fadd2(sum[0], sum[1]), s23 = fadd2(sum[2], sum[3]);
        const float2 st = fadd2(s01, s23);
        w += st.x + st.y;
        ++cnt;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_le[s]);
      const long long item = static_cast<long long>(cur.hk) * entries + cur.e;
      if (cur.step(a)) {
        a.part[(static_cast<long long>(blockIdx.x) + item) * 256 + half * 128 + r] = w;
        w = 0.f;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// w of 256 keys of one key/value head: the sums of the CTAs that had a part of them, in order.
template <int QT>
__global__ void __launch_bounds__(256) fa_key_weights_sum_kernel(const KeyWeightsArgs a) {
  const int entries = a.B * a.ranges;
  const int e = blockIdx.x % entries, hk = blockIdx.x / entries;
  const int b = e / a.ranges, j = (e % a.ranges) * 256 + threadIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long per_head = a.first[entries], f = a.first[e];
  const long long steps = a.first[e + 1] - f;
  float w = 0.f;
  if (steps > 0) {
    const long long total = per_head * a.Hkv, x0 = hk * per_head + f, x1 = x0 + steps;
    const long long n_cta = min(static_cast<long long>(a.grid), total);
    const long long i0 = ((x0 + 1) * n_cta - 1) / total, i1 = (x1 * n_cta - 1) / total;
    for (long long i = i0; i <= i1; ++i) w += a.part[(i + blockIdx.x) * 256 + threadIdx.x];
  }
  const KeyWeightsSeq s = key_weights_seq(a, b);
  if (j < a.N) a.w[(static_cast<size_t>(b) * a.Hkv + hk) * a.ldw + j] = j < s.n ? w : 0.f;
}

}  // namespace fa
