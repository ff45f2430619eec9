// token_logprobs: per row of logits, with lse = log sum_v exp(l_v):
//   logp    = l[token] - lse
//   entropy = lse - sum_v p_v l_v,  p_v = exp(l_v - lse)
//   top     = the top_k largest logits (equal values: the lower index first),
//             as l - lse and their indices.
//
// This kernel is the plain one: a block per row, a pass for the maximum, one
// for the sums and one more for each alternative.
#include <cstdint>
#include "common.cuh"

namespace slim {

constexpr int LP_THREADS = 256;

__device__ __forceinline__ float lp_ld(const void* p, int64_t i, int dtype) {
  if (dtype == 0) return static_cast<const float*>(p)[i];
  return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
}

// A 64-bit key that orders (value, index): larger value first, then the lower
// index; NaN above everything, -0 equal to +0.
__device__ __forceinline__ uint64_t lp_key(float v, uint32_t idx) {
  v = v + 0.f;
  uint32_t u = v != v ? 0x7FFFFFFFu : __float_as_uint(v);
  u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return ((uint64_t)u << 32) | (uint32_t)~idx;
}
__device__ __forceinline__ float lp_key_value(uint64_t key) {
  const uint32_t u = (uint32_t)(key >> 32);
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7FFFFFFFu) : ~u);
}

template <typename T, typename Op>
__device__ T lp_block(T v, T* red, Op op) {
  __syncthreads();
  red[threadIdx.x] = v;
  __syncthreads();
  for (int o = LP_THREADS / 2; o > 0; o >>= 1) {
    if (threadIdx.x < o) red[threadIdx.x] = op(red[threadIdx.x], red[threadIdx.x + o]);
    __syncthreads();
  }
  return red[0];
}

__global__ void __launch_bounds__(LP_THREADS)
lp_plain_kernel(const void* __restrict__ logits, int dtype, int64_t V, int64_t ld, const int64_t* __restrict__ tokens,
                int top_k, float* __restrict__ logp, float* __restrict__ entropy, float* __restrict__ top_logp,
                int32_t* __restrict__ top_id) {
  __shared__ uint64_t red[LP_THREADS];
  const int64_t row = blockIdx.x, at = row * ld;
  auto max64 = [](uint64_t a, uint64_t b) { return a > b ? a : b; };
  auto add = [](float a, float b) { return a + b; };
  uint64_t best = 0;
  for (int64_t v = threadIdx.x; v < V; v += LP_THREADS) best = max64(best, lp_key(lp_ld(logits, at + v, dtype), (uint32_t)v));
  best = lp_block(best, red, max64);
  const float top = lp_key_value(best);
  const float base = top == -INFINITY ? 0.f : top;
  float S = 0.f, Tsum = 0.f;
  for (int64_t v = threadIdx.x; v < V; v += LP_THREADS) {
    const float d = lp_ld(logits, at + v, dtype) - base, e = expf(d);
    S += e;
    if (e != 0.f) Tsum += e * d;
  }
  S = lp_block(S, reinterpret_cast<float*>(red), add);
  Tsum = lp_block(Tsum, reinterpret_cast<float*>(red), add);
  const float ls = S == 0.f ? 0.f : logf(S);
  if (threadIdx.x == 0) {
    const int64_t t = tokens ? tokens[row] : -1;
    if (logp) logp[row] = t >= 0 && t < V ? lp_ld(logits, at + t, dtype) - base - ls : 0.f;
    if (entropy) entropy[row] = S == 0.f ? 0.f : ls - Tsum / S;
  }
  for (int q = 0; q < top_k; ++q) {
    if (threadIdx.x == 0) {
      top_logp[row * top_k + q] = lp_key_value(best) - base - ls;
      top_id[row * top_k + q] = (int32_t)~(uint32_t)best;
    }
    const uint64_t last = best;
    best = 0;
    for (int64_t v = threadIdx.x; v < V; v += LP_THREADS) {
      const uint64_t key = lp_key(lp_ld(logits, at + v, dtype), (uint32_t)v);
      if (key < last && key > best) best = key;
    }
    best = lp_block(best, red, max64);
  }
}

cudaError_t launch_logprobs(const void* logits, int dtype, int64_t N, int64_t V, int64_t ld, const int64_t* tokens,
                            int top_k, float* logp, float* entropy, float* top_logp, int32_t* top_id, int num_sms,
                            cudaStream_t s) {
  lp_plain_kernel<<<(unsigned)N, LP_THREADS, 0, s>>>(logits, dtype, V, ld, tokens, top_k, logp, entropy, top_logp,
                                                     top_id);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace slim
