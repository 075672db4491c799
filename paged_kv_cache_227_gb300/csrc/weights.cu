// Attention-weight sums: the second half of pa_decode_weights.
//
// The decode leaves every score s (scaled, log2 units) and each query head's
// log2-sum-exp e in the workspace; the attention weight of cached token t for
// query head g is p_g = 2^(s_tg - e_g), so with the group's G heads
//   weights[i][h][t] = decay * weights[i][h][t] + sum_g p_g,   t < L_i.
// No atomics: one thread owns a token's sum, and the heads are added in order.
//
// Bound: memory (4 G + 8 bytes a token and kv head, against the decode's
// 512); the scores were just written, so they come from L2 when they fit.
#include "pa_internal.h"

namespace pa {

constexpr int kSumThreads = 256;
constexpr int kSumTokens = 4;  // tokens a thread: 1,024 a CTA

__global__ void __launch_bounds__(kSumThreads) weight_sums_kernel(const float* __restrict__ scores,
                                                                  const float* __restrict__ lse,
                                                                  float* __restrict__ weights, float decay,
                                                                  const int32_t* __restrict__ seq_lens, int Hkv, int G,
                                                                  int max_blocks) {
  const int i = blockIdx.z, h = blockIdx.y;
  const int span = max_blocks * kBlock;
  int L = seq_lens[i];
  L = L < 0 ? 0 : (L > span ? span : L);  // (the decode reports a length out of range)
  const long long seg = static_cast<long long>(i) * Hkv + h;
  const float* s = scores + seg * span * G;
  float* w = weights + seg * span;
  float e[PA_MAX_GROUP];
#pragma unroll
  for (int g = 0; g < PA_MAX_GROUP; ++g) e[g] = g < G ? lse[seg * G + g] : 0.f;
#pragma unroll
  for (int k = 0; k < kSumTokens; ++k) {
    const long long t = (static_cast<long long>(blockIdx.x) * kSumTokens + k) * kSumThreads + threadIdx.x;
    if (t >= L) return;
    float sum = 0.f;
#pragma unroll
    for (int g = 0; g < PA_MAX_GROUP; ++g)
      if (g < G) {
        const float x = s[t * G + g];
        sum += x == -INFINITY ? 0.f : exp2f(x - e[g]);  // (a head whose every token is skipped has e = -inf)
      }
    w[t] = fmaf(decay, w[t], sum);
  }
}

int launch_weight_sums(const pa_pool* p, const float* scores, const float* lse, float* weights, float decay,
                       const int32_t* seq_lens, int B, int Hq, int max_blocks, cudaStream_t stream) {
  const int span = max_blocks * kBlock;
  const dim3 grid((span + kSumThreads * kSumTokens - 1) / (kSumThreads * kSumTokens), p->n_kv_heads, B);
  weight_sums_kernel<<<grid, kSumThreads, 0, stream>>>(scores, lse, weights, decay, seq_lens, p->n_kv_heads,
                                                       Hq / p->n_kv_heads, max_blocks);
  return cuda_status(cudaGetLastError());
}

}  // namespace pa
