// key_weights.cuh — how much attention each key of a prompt received:
//   w[b, hk, j] = sum over the query heads h that share hk and the window's query rows i
//                 (i >= j when causal) of exp(scale q_hi . k_j - lse_hi),
// the column sums of the softmax matrix, recomputed from q, k and the forward's logsumexp as
// the backward recomputes P ("flash-attention-trading-models", "Pase hacia atras").
//
// Half of the forward's products and all of its exponentials: S^T = K Q^T on tcgen05 with the
// keys on the tensor-memory lanes, so that one thread holds one key, and the sum over the
// queries runs along its registers.  128 keys x 128 queries take the tensor core 512 clocks at
// d = 128 and the exponential unit 1024, which bounds it: 8192 tokens, 32 heads, causal, d = 128 take
// 360 to 380 us, of which the exponential unit alone needs 245 (the MMAs alone would need 167).  A
// window of 64 rows over 8 sequences of 32768 tokens takes 193 us (the unit 119, K from DRAM 88).
// Computing 1 to 3 of 8 exponentials on the FMA pipe instead (a degree-5 polynomial) made it slower
// each time it was tried (p. e. 1 of 4: 381 us), as did 8 instead of 16 warps with whole score tiles
// in registers (460 us).
// Each column's -lse / scale is one more column of Q against a column of ones of K, in three bf16
// pieces: no thread reads log-sum-exps (369 us when they read them from shared memory).
//
// Query rows come in subtiles of 64 rows of one head, and a step takes the next two of them,
// whatever heads they belong to: with a window of 64 rows the heads that share a key/value head
// fill the MMAs together.
//
// Work is one list of steps, ordered by key/value head, sequence, range of 256 keys, query head
// and query tile, cut into equal parts, one per CTA and SM.  K of the next range and Q of the next
// steps load while the last ones are worked on.  A part's sums go to the workspace and a second
// kernel adds the parts of each key in order: no atomics, the same bits every time.
//   warps 0-15   exponentials and sums: warps 0-3 and 8-11 of keys 0-127 of the range, the others
//                of keys 128-255; warps 0-7 of every other step, 8-15 of those between
//   warp 16      TMA producer
//   warps 17-18  tcgen05.mma issuers of the two key halves (17 owns the tensor memory): an MMA takes
//                its issuing thread some 70 clocks, and one thread for both halves held up all
//   warp 19      log-sum-exps of the steps' queries into operand tiles, read a step ahead
// Tensor memory: two score tiles of 128 columns per key half.
#pragma once
#include "early.cuh"
#include "sm100.cuh"

namespace fa {

constexpr int kKeyWeightsThreads = 20 * 32;

struct KeyWeightsArgs {
  const float* lse;        // [B*H, N]
  float* w;                // [B*Hkv, ldw]
  const int* n_rows;       // [B] or null (N)
  float* part;             // [grid + B*Hkv*ranges, 2, 256]: slot (CTA + item)
  int2* span;              // [B*Hkv*ranges]: the first and the last CTA that had a part of an item
  int B, N, ldw, H, Hkv, g, window, causal, ranges, grid;
  float scale_log2, neg_inv_scale;
};

template <int D>
struct KeyWeightsCfg {
  static constexpr int NSUB = 2;                         // 64-row subtiles of a step
  static constexpr int QT = 64 * NSUB;
  static constexpr int NBOX = D / 64;
  static constexpr int BOX_K = 128 * 128, TILE_K = NBOX * BOX_K;  // 128 keys
  static constexpr int BOX_Q = QT * 128;                 // 64 of the d columns of a step's rows
  static constexpr int KSLOTS = D == 64 ? 4 : D == 128 ? 3 : 2;   // places for 128 keys
  static constexpr int QSLOTS = D == 64 ? 8 : D == 128 ? 6 : 5;   // places for boxes of Q
  static constexpr int LSLOTS = 3;
  static constexpr int OFF_Q = KSLOTS * TILE_K;
  static constexpr int TILE_X = 128 * 32;                // 128 rows x 16 bf16: the extra step of K = 16
  static constexpr int OFF_X = OFF_Q + QSLOTS * BOX_Q;   // Q's side, [LSLOTS]
  static constexpr int OFF_ONE = OFF_X + LSLOTS * TILE_X;  // K's side: 1, 1, 1, 0, ...
  static constexpr int SMEM_BYTES = OFF_ONE + TILE_X + 1024;
  static_assert(SMEM_BYTES <= 230400, "shared memory budget (2 KB are static)");
};

// The rows of a sequence and its window, and the 64-row query tiles of one of its key ranges.
struct KeyWeightsSeq {
  int n, lo;
};
__device__ __forceinline__ KeyWeightsSeq key_weights_seq(const KeyWeightsArgs& a, int b) {
  KeyWeightsSeq s;
  s.n = a.n_rows ? max(0, min(a.n_rows[b], a.N)) : a.N;
  s.lo = max(0, s.n - a.window);
  return s;
}
__device__ __forceinline__ int key_weights_tiles(const KeyWeightsArgs& a, const KeyWeightsSeq& s, int range, int& base) {
  const int j0 = range * 256;
  base = a.causal ? max(s.lo, j0) : s.lo;
  return j0 < s.n ? (s.n - base + 63) / 64 : 0;
}

// Walks the steps of one CTA: every role keeps one of these and they stay in step.
template <int NSUB>
struct KeyWeightsCursor {
  int left, hk, e, b, range, n, base, tiles;
  int h, tile;  // of the step's first subtile; the next ones follow

  __device__ __forceinline__ void set_entry(const KeyWeightsArgs& a) {
    b = e / a.ranges;
    range = e % a.ranges;
    const KeyWeightsSeq s = key_weights_seq(a, b);
    n = s.n;
    tiles = key_weights_tiles(a, s, range, base);
  }
  // to the subtile after (h, tile); h reaches g behind the last
  __device__ __forceinline__ void next_sub(int& sh, int& st) const {
    if (++st == tiles) st = 0, ++sh;
  }
  // true when the step that ends was the last of its entry here
  __device__ __forceinline__ bool step(const KeyWeightsArgs& a) {
    --left;
#pragma unroll
    for (int u = 0; u < NSUB; ++u) next_sub(h, tile);
    if (h < a.g) return left == 0;
    if (left > 0) {
      do {
        if (++e == a.B * a.ranges) e = 0, ++hk;
        set_entry(a);
      } while (tiles == 0);
      h = tile = 0;
    }
    return true;
  }
  __device__ __forceinline__ int subs(const KeyWeightsArgs& a) const { return min(NSUB, (a.g - h) * tiles - tile); }
  // has the second half of the range any key
  __device__ __forceinline__ bool second() const { return range * 256 + 128 < n; }
};

// Descriptor of a K-major operand without swizzle: 8-row x 16-byte cores of 128 bytes, the two
// cores of a 16-deep step `lbo` apart, groups of 8 rows `sbo` apart.
__device__ __forceinline__ uint64_t make_sdesc_plain(uint32_t smem_addr, uint32_t lbo, uint32_t sbo) {
  return static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu) | static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16 |
         static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32 | 1ull << 46;
}

template <int D>
__global__ void __launch_bounds__(kKeyWeightsThreads, 1)
    fa_key_weights_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                          const KeyWeightsArgs a) {
  using C = KeyWeightsCfg<D>;
  constexpr int NSUB = C::NSUB, QT = C::QT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t bar_kf[C::KSLOTS], bar_ke[C::KSLOTS], bar_qf[C::QSLOTS], bar_qe[C::QSLOTS];
  __shared__ uint64_t bar_lf[C::LSLOTS], bar_le[C::LSLOTS], bar_sf[2][2], bar_se[2][2], bar_done[2];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  __shared__ long long scan[20];
  __shared__ long long start_rem;
  __shared__ int start_e;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == 17) {
    tmem_alloc(&tmem_base_sh, 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    abort_sh = 0;
    for (int i = 0; i < C::KSLOTS; ++i) mbar_init(&bar_kf[i], 1), mbar_init(&bar_ke[i], 1);
    for (int i = 0; i < C::QSLOTS; ++i) mbar_init(&bar_qf[i], 1), mbar_init(&bar_qe[i], 2);
    for (int i = 0; i < C::LSLOTS; ++i) mbar_init(&bar_lf[i], 1), mbar_init(&bar_le[i], 2);
    for (int i = 0; i < 4; ++i) mbar_init(&bar_sf[i >> 1][i & 1], 1), mbar_init(&bar_se[i >> 1][i & 1], 4);
    mbar_init(&bar_done[0], 1);
    mbar_init(&bar_done[1], 1);
    fence_mbar_init();
  }
  for (int i = tid; i < (C::LSLOTS + 1) * C::TILE_X / 16; i += kKeyWeightsThreads) {
    // row r of a tile: 16 bytes at (r / 8) * 256 + (r % 8) * 16, its second eight columns 128 bytes on
    const bool one = i >= C::LSLOTS * C::TILE_X / 16 && !(i & 8);
    reinterpret_cast<uint4*>(smem + C::OFF_X)[i] = one ? make_uint4(0x3F803F80u, 0x00003F80u, 0u, 0u) : make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  wait_for_earlier();
  // ---- this CTA's part of the list ------------------------------------------------------
  const int entries = a.B * a.ranges;
  const int per = (entries + kKeyWeightsThreads - 1) / kKeyWeightsThreads;
  const int e0 = min(entries, tid * per), e1 = min(entries, e0 + per);
  auto steps = [&](int e) {
    int base;
    const long long t = key_weights_tiles(a, key_weights_seq(a, e / a.ranges), e % a.ranges, base);
    return (t * a.g + NSUB - 1) / NSUB;
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
  for (int w = 0; w < 20; ++w) {
    if (w < warp) before += scan[w];
    per_head += scan[w];
  }
  const long long total = per_head * a.Hkv;
  const long long n_cta = max(1ll, min(static_cast<long long>(a.grid), total));  // the others have nothing to do
  const long long u0 = min(blockIdx.x * total / n_cta, total), u1 = min((blockIdx.x + 1) * total / n_cta, total);
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
  KeyWeightsCursor<NSUB> cur;
  cur.left = static_cast<int>(u1 - u0);
  if (cur.left > 0) {
    cur.hk = static_cast<int>(u0 / per_head);
    cur.e = start_e;
    cur.set_entry(a);
    cur.h = static_cast<int>(start_rem * NSUB / cur.tiles);
    cur.tile = static_cast<int>(start_rem * NSUB % cur.tiles);
  }

  if (warp == 16) {
    // ======================= TMA producer ===================================
    if (lane == 0 && cur.left > 0) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      int kt = 0, qt = 0;  // key halves and boxes of Q loaded
      bool fresh = true, ok = true;
      auto load_k = [&](int half) {
        const int s = kt % C::KSLOTS;
        if (!(ok = mbar_wait(&bar_ke[s], ((kt / C::KSLOTS) & 1) ^ 1, &abort_sh, 40))) return;
        mbar_arrive_expect_tx(&bar_kf[s], C::TILE_K);
        for (int x = 0; x < C::NBOX; ++x)
          tma_load_3d(smem + s * C::TILE_K + x * C::BOX_K, &tmK, &bar_kf[s], x * 64, cur.range * 256 + half * 128,
                      cur.b * a.Hkv + cur.hk);
        ++kt;
      };
      while (cur.left > 0) {
        if (fresh) {
          load_k(0);
          if (!ok) break;
        }
        const int subs = cur.subs(a);
        for (int x = 0; ok && x < C::NBOX; ++x) {
          const int s = qt % C::QSLOTS;
          if (!(ok = mbar_wait(&bar_qe[s], ((qt / C::QSLOTS) & 1) ^ 1, &abort_sh, 41))) break;
          mbar_arrive_expect_tx(&bar_qf[s], subs * 64 * 128);
          int h = cur.h, tile = cur.tile;
          for (int u = 0; u < subs; ++u) {
            tma_load_3d(smem + C::OFF_Q + s * C::BOX_Q + u * 64 * 128, &tmQ, &bar_qf[s], x * 64, cur.base + tile * 64,
                        (cur.b * a.Hkv + cur.hk) * a.g + h);
            cur.next_sub(h, tile);
          }
          ++qt;
        }
        if (ok && fresh && cur.second()) load_k(1);
        if (!ok) break;
        fresh = cur.step(a);
      }
      // every copy has landed before the CTA ends
      for (int i = max(0, kt - C::KSLOTS); i < kt; ++i)
        mbar_wait_drain(&bar_kf[i % C::KSLOTS], (i / C::KSLOTS) & 1, 100000000ull);
      for (int i = max(0, qt - C::QSLOTS); i < qt; ++i)
        mbar_wait_drain(&bar_qf[i % C::QSLOTS], (i / C::QSLOTS) & 1, 100000000ull);
    }
    __syncwarp();
  } else if (warp == 17 || warp == 18) {
    // ======================= tcgen05.mma issuers ============================
    if (lane == 0) {
      const int half = warp - 17;
      const uint64_t kd0 = make_sdesc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t qd0 = make_sdesc_sw128(smem_u32(smem + C::OFF_Q), 16, 1024);
      const uint64_t xd0 = make_sdesc_plain(smem_u32(smem + C::OFF_X), 128, 256);
      const uint64_t one = make_sdesc_plain(smem_u32(smem + C::OFF_ONE), 128, 256);
      int kt = 0, qt = 0, t = 0, cnt[2] = {0, 0};  // key halves and boxes of Q begun, steps, tiles per buffer
      bool fresh = true, ok = true;
      auto tile = [&](uint32_t buf, int& used) {
        const uint32_t idesc = make_idesc(128, 0, kFmtBF16, 0, 0) | (static_cast<uint32_t>(cur.subs(a) * 8) << 17);
        const int ks = (kt + half) % C::KSLOTS;
        if (fresh && !(ok = mbar_wait(&bar_kf[ks], ((kt + half) / C::KSLOTS) & 1, &abort_sh, 42))) return;
        if (!(ok = mbar_wait(&bar_se[half][buf], (used & 1) ^ 1, &abort_sh, 44))) return;
        const uint64_t kd = sdesc_add(kd0, ks * C::TILE_K);
#pragma unroll
        for (int x = 0; x < C::NBOX; ++x) {
          const int qs = (qt + x) % C::QSLOTS;
          if (!(ok = mbar_wait(&bar_qf[qs], ((qt + x) / C::QSLOTS) & 1, &abort_sh, 43))) return;
          tc_fence_after();
          const uint64_t qd = sdesc_add(qd0, qs * C::BOX_Q);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ss(tmem + (half * 2 + buf) * 128, sdesc_add(kd, x * C::BOX_K + k * 32), sdesc_add(qd, k * 32), idesc,
                   x > 0 || k > 0);
          mma_commit(&bar_qe[qs]);
        }
        const int ls = t % C::LSLOTS;
        if (!(ok = mbar_wait(&bar_lf[ls], (t / C::LSLOTS) & 1, &abort_sh, 49))) return;
        tc_fence_after();
        mma_ss(tmem + (half * 2 + buf) * 128, one, sdesc_add(xd0, ls * C::TILE_X), idesc, 1);
        mma_commit(&bar_le[ls]);
        mma_commit(&bar_sf[half][buf]);
        ++used;
      };
      while (cur.left > 0) {
        const int halves = cur.second() ? 2 : 1;
        if (half < halves) {
          if (t & 1) tile(1, cnt[1]);
          else tile(0, cnt[0]);
        } else {
          // no keys in this half: the step's operands are not needed here
          for (int x = 0; ok && x < C::NBOX; ++x) {
            const int qs = (qt + x) % C::QSLOTS;
            ok = mbar_wait(&bar_qf[qs], ((qt + x) / C::QSLOTS) & 1, &abort_sh, 48);
            if (ok) mbar_arrive(&bar_qe[qs]);
          }
          const int ls = t % C::LSLOTS;
          ok = ok && mbar_wait(&bar_lf[ls], (t / C::LSLOTS) & 1, &abort_sh, 50);
          if (ok) mbar_arrive(&bar_le[ls]);
        }
        if (!ok) break;
        qt += C::NBOX;
        ++t;
        const int ks = (kt + half) % C::KSLOTS;
        fresh = cur.step(a);
        if (fresh) {
          if (half < halves) mma_commit(&bar_ke[ks]);
          kt += halves;
        }
      }
      // every MMA of this thread must be finished before TMEM is freed
      mma_commit(&bar_done[half]);
      mbar_wait_drain(&bar_done[half], 0, 100000000ull);
    }
    __syncwarp();
  } else if (warp == 19) {
    // ======================= -log-sum-exps / scale ==========================
    // v = -lse / scale as the sum of three bf16 numbers (24 bits), infinities and NaN as they are.
    // The next step's values are read before this one's are handed out.
    float next[QT / 32];
    auto fetch = [&]() {
      int h = cur.h, tile = cur.tile;
#pragma unroll
      for (int u = 0; u < NSUB; ++u) {
        const float* lse = a.lse + (static_cast<size_t>(cur.b * a.Hkv + cur.hk) * a.g + min(h, a.g - 1)) * a.N;
        const int i = cur.base + tile * 64 + lane;
        next[2 * u] = h < a.g && i < cur.n ? lse[i] : 0.f;
        next[2 * u + 1] = h < a.g && i + 32 < cur.n ? lse[i + 32] : 0.f;
        cur.next_sub(h, tile);
      }
    };
    if (cur.left > 0) fetch();
    for (int t = 0; cur.left > 0; ++t) {
      float v[QT / 32];
#pragma unroll
      for (int x = 0; x < QT / 32; ++x) v[x] = next[x];
      cur.step(a);
      if (cur.left > 0) fetch();
      const int s = t % C::LSLOTS;
      if (!__all_sync(0xffffffffu, mbar_wait(&bar_le[s], ((t / C::LSLOTS) & 1) ^ 1, &abort_sh, 45))) break;
#pragma unroll
      for (int x = 0; x < QT / 32; ++x) {
        const float f = v[x] * a.neg_inv_scale;
        const float hi = __bfloat162float(__float2bfloat16_rn(f));
        const float rest = fabsf(f) < 1e30f ? f - hi : 0.f;
        const float mid = __bfloat162float(__float2bfloat16_rn(rest));
        const int row = lane + 32 * x;
        *reinterpret_cast<uint2*>(smem + C::OFF_X + s * C::TILE_X + (row >> 3) * 256 + (row & 7) * 16) =
            make_uint2(pack_bf16x2(hi, mid), pack_bf16x2(rest - mid, 0.f));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_lf[s]);
    }
  } else {
    // ======================= exponentials and sums ==========================
    const int half = (warp >> 2) & 1, part = warp >> 3, r = tid & 127;
    const uint32_t ts = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + (half * 2 + part) * 128;
    const float c = a.scale_log2;
    float w = 0.f;
    int cnt = 0;
    bool begins = cur.h == 0 && cur.tile == 0;
    for (int t = 0; cur.left > 0; ++t) {
      const int k0 = cur.range * 256 + half * 128;
      if ((t & 1) == part && k0 < cur.n) {
        if (!mbar_wait(&bar_sf[half][part], cnt & 1, &abort_sh, 47)) break;
        ++cnt;
        tc_fence_after();
        int h = cur.h, tile = cur.tile;
        float2 sum[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        const float2 c2 = make_float2(c, c);
#pragma unroll 1
        for (int u = 0; u < QT / 32; ++u) {  // 32 columns at a time
          const int i0 = cur.base + tile * 64 + 32 * (u & 1);
          // columns of a subtile that is there, with queries that see a key of this half
          const bool live = h < a.g && i0 < cur.n && (!a.causal || i0 + 31 >= k0);
          float x[32];
          if (live) {
            tmem_ld32(ts + 32 * u, *reinterpret_cast<uint32_t(*)[32]>(x));
            tmem_wait_ld();
          }
          if (u == QT / 32 - 1) {
            // the scores are in registers: their columns are free
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_se[half][part]);
          }
          if (live) {
            if (i0 + 32 > cur.n || (a.causal && i0 < k0 + 127)) {
              // what lies outside does not count, whatever it holds
              const int j = k0 + r;
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const int i = i0 + e;
                if (i >= cur.n || (a.causal && i < j)) x[e] = -INFINITY;
              }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float2 a0 = fmul2(make_float2(x[4 * e], x[4 * e + 1]), c2);
              const float2 a1 = fmul2(make_float2(x[4 * e + 2], x[4 * e + 3]), c2);
              sum[e & 1] = fadd2(sum[e & 1], make_float2(ex2_approx(a0.x), ex2_approx(a0.y)));
              sum[2 + (e & 1)] = fadd2(sum[2 + (e & 1)], make_float2(ex2_approx(a1.x), ex2_approx(a1.y)));
            }
          }
          if (u & 1) cur.next_sub(h, tile);
        }
        const float2 s01 = fadd2(sum[0], sum[1]), s23 = fadd2(sum[2], sum[3]);
        const float2 st = fadd2(s01, s23);
        w += st.x + st.y;
      }
      const int hk = cur.hk, e = cur.e;
      if (cur.step(a)) {
        const long long item = static_cast<long long>(hk) * entries + e;
        a.part[((static_cast<long long>(blockIdx.x) + item) * 2 + part) * 256 + half * 128 + r] = w;
        w = 0.f;
        if (tid == 0) {
          if (begins) a.span[item].x = blockIdx.x;
          if (cur.left > 0 || cur.h >= a.g) a.span[item].y = blockIdx.x;
        }
        begins = true;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 17) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// w of 256 keys of one key/value head: the sums of the CTAs that had a part of them, in order.
// Four keys a thread, four heads' ranges a block (a block each, with the CTAs found by divisions
// here: 22.7 us instead of 7.0 for 32768 keys in 64 heads, read from DRAM).
__global__ void __launch_bounds__(256) fa_key_weights_sum_kernel(const KeyWeightsArgs a) {
  const int entries = a.B * a.ranges;
  const int item = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  wait_for_earlier();
  if (item >= entries * a.Hkv) return;
  const int e = item % entries, hk = item / entries, b = e / a.ranges, range = e % a.ranges;
  const KeyWeightsSeq s = key_weights_seq(a, b);
  int base;
  const bool any = key_weights_tiles(a, s, range, base) > 0;
  float w[4] = {0.f, 0.f, 0.f, 0.f};
  if (any) {
    const int2 span = a.span[item];
    const int i0 = max(span.x, 0), i1 = min(span.y, a.grid - 1);  // within the grid, should a wait have given up
    for (int i = i0; i <= i1; ++i) {
      const float* const p = a.part + (static_cast<long long>(i) + item) * 512 + lane;
#pragma unroll
      for (int x = 0; x < 4; ++x) w[x] += p[64 * x] + p[64 * x + 256];
    }
  }
  float* const out = a.w + (static_cast<size_t>(b) * a.Hkv + hk) * a.ldw;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int j = range * 256 + 64 * x + lane;
    if (j < a.N) out[j] = j < s.n ? w[x] : 0.f;
  }
}

}  // namespace fa
