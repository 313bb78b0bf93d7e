// key_weights.cuh — how much attention each key of a prompt received:
//   w[b, hk, j] = sum over the query heads h that share hk and the window's query rows i
//                 (i >= j when causal) of exp(scale q_hi . k_j - lse_hi),
// the column sums of the softmax matrix, recomputed from q, k and the forward's logsumexp as
// the backward recomputes P ("flash-attention-trading-models", "Pase hacia atras").
#pragma once
#include "sm100.cuh"

namespace fa {

struct KeyWeightsArgs {
  const __nv_bfloat16* q;  // [B*H, N, d]
  const __nv_bfloat16* k;  // [B*Hkv, N, d]
  const float* lse;        // [B*H, N]
  float* w;                // [B*Hkv, ldw]
  const int* n_rows;       // [B] or null (N)
  int N, ldw, H, Hkv, g, window, causal, ktiles;
  float scale_log2;
};

// One CTA per 128 keys of one key/value head, one thread per key.
template <int D>
__global__ void __launch_bounds__(128) fa_key_weights_kernel(const KeyWeightsArgs a) {
  __shared__ float q[16][D];
  __shared__ float l2[16];
  const int bh = blockIdx.x / a.ktiles, tile = blockIdx.x % a.ktiles, tid = threadIdx.x;
  const int b = bh / a.Hkv, j = tile * 128 + tid;
  const int n = a.n_rows ? max(0, min(a.n_rows[b], a.N)) : a.N;
  const int lo = max(n - a.window, a.causal ? tile * 128 : 0);
  const __nv_bfloat162* k = reinterpret_cast<const __nv_bfloat162*>(a.k + (static_cast<size_t>(bh) * a.N + min(j, a.N - 1)) * D);
  float w = 0.f;
  for (int h = 0; h < a.g; ++h) {
    const size_t qh = static_cast<size_t>(bh) * a.g + h;
    for (int i0 = max(lo, 0); i0 < n; i0 += 16) {
      __syncthreads();
      for (int e = tid; e < 16 * D; e += 128)
        q[e / D][e % D] = i0 + e / D < n ? __bfloat162float(a.q[(qh * a.N + i0 + e / D) * D + e % D]) : 0.f;
      if (tid < 16) l2[tid] = i0 + tid < n ? a.lse[qh * a.N + i0 + tid] * 1.4426950408889634f : INFINITY;
      __syncthreads();
      float s[16];
      for (int r = 0; r < 16; ++r) s[r] = 0.f;
      for (int c = 0; c < D / 2; ++c) {
        const float2 kk = __bfloat1622float2(k[c]);
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] = fmaf(kk.y, q[r][2 * c + 1], fmaf(kk.x, q[r][2 * c], s[r]));
      }
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if (!a.causal || i0 + r >= j) w += exp2f(fmaf(s[r], a.scale_log2, -l2[r]));
    }
  }
  if (j < a.N) a.w[static_cast<size_t>(bh) * a.ldw + j] = j < n ? w : 0.f;
}

}  // namespace fa
