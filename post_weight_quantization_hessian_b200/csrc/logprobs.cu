// token_logprobs: per row of logits, with lse = log sum_v exp(l_v):
//   logp    = l[token] - lse
//   entropy = lse - sum_v p_v l_v,  p_v = exp(l_v - lse)
//   top     = the top_k largest logits (equal values: the lower index first),
//             as l - lse and their indices.
//
// One pass over the row. A thread keeps the maximum m of its elements and, relative
// to it, S = sum e^(l - m) and T = sum (l - m) e^(l - m); a larger maximum m'
// rescales both, T' = (T + (m - m') S) e^(m - m'). Partial results join the same
// way, and logp = l - m - log S, entropy = log S - T / S.
//
// The alternatives come from the same pass. Of 32 groups of elements (the lanes of
// all warps) the top_k-th largest maximum is a bound that at least top_k elements
// reach and that few others do (about 30 in all for 20 of 32 groups in random
// order). Only threads whose own maximum reaches it look at their elements again;
// what they collect is ranked by counting, as 64-bit keys of value and index.
// Where the bound is -inf (fewer unmasked elements than that), only the others are
// collected and the lowest masked indices follow them. Rows that put too many
// elements at or above the bound (long ties, all large ones in few groups) and
// rows with a NaN take one scan for each alternative instead.
//
// Bound by the bytes of the logits for many rows (about 5.5 issued operations an
// element in packed pairs); for few rows a cluster of up to 8 CTAs shares a row, as one CTA
// cannot ask for the bytes fast enough, and joins through distributed shared memory.
#include <cstdint>
#include <type_traits>
#include "common.cuh"

namespace slim {

constexpr int LP_MAX_K = 32;
constexpr int LP_CAND = 1024;  // collected elements; more take the scans

// A 64-bit key that orders (value, index): larger value first, then the lower
// index; NaN above everything, -0 equal to +0. No key is 0 or all ones.
__device__ __forceinline__ uint64_t lp_key(float v, uint32_t idx) {
  v = v + 0.f;
  uint32_t u = v != v ? 0x7FC00000u : __float_as_uint(v);
  u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return ((uint64_t)u << 32) | (uint32_t)~idx;
}
__device__ __forceinline__ float lp_key_value(uint64_t key) {
  const uint32_t u = (uint32_t)(key >> 32);
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7FFFFFFFu) : ~u);
}
__device__ __forceinline__ uint64_t lp_max(uint64_t a, uint64_t b) { return a > b ? a : b; }
__device__ __forceinline__ float lp_max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float lp_ex2(float a) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
  return r;
}
__device__ __forceinline__ uint64_t lp_pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void lp_unpair(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t lp_add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t lp_mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t lp_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kFar = -150.f;  // e^-150 is 0 in fp32; keeps 0 * -inf out of T

struct LpStat {
  float m, S, T;
  // Relative to a larger maximum. (An m of -inf goes with S = T = 0.)
  __device__ __forceinline__ void rise(float to) {
    const float dm = fmaxf(m - to, -1e4f), f = lp_ex2(dm * kLog2e);
    T = (T + S * dm) * f;
    S *= f;
    m = to;
  }
  __device__ __forceinline__ void join(LpStat o) {
    if (o.m > m) rise(o.m);
    else if (m > o.m) o.rise(m);
    S += o.S;
    T += o.T;
  }
};

template <typename E>
__device__ __forceinline__ float lp_load(const E* p) {
  if constexpr (sizeof(E) == 4)
    return __ldg(reinterpret_cast<const float*>(p));
  else
    return __uint_as_float((uint32_t)__ldg(reinterpret_cast<const uint16_t*>(p)) << 16);
}
// The kVec elements of a 16-byte vector.
template <typename E, int kVec>
__device__ __forceinline__ void lp_unpack(const uint4& q, float (&v)[kVec]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(E) == 4) {
      v[i] = __uint_as_float(w[i]);
    } else {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}

// The largest of kCount vectors (a NaN counts as nothing). bf16 pairs are compared as pairs.
template <typename E, int kCount>
__device__ __forceinline__ float lp_top(const uint4 (&q)[kCount]) {
  if constexpr (sizeof(E) == 4) {
    float top = -INFINITY;
#pragma unroll
    for (int b = 0; b < kCount; ++b)
      top = fmaxf(top, fmaxf(fmaxf(__uint_as_float(q[b].x), __uint_as_float(q[b].y)),
                             fmaxf(__uint_as_float(q[b].z), __uint_as_float(q[b].w))));
    return top;
  } else {
    uint32_t t = 0xFF80FF80u;  // -inf, -inf
#pragma unroll
    for (int b = 0; b < kCount; ++b) {
      asm("max.bf16x2 %0, %0, %1;" : "+r"(t) : "r"(q[b].x));
      asm("max.bf16x2 %0, %0, %1;" : "+r"(t) : "r"(q[b].y));
      asm("max.bf16x2 %0, %0, %1;" : "+r"(t) : "r"(q[b].z));
      asm("max.bf16x2 %0, %0, %1;" : "+r"(t) : "r"(q[b].w));
    }
    return fmaxf(__uint_as_float(t << 16), __uint_as_float(t & 0xFFFF0000u));
  }
}

template <typename E, int kThreads>
__global__ void __launch_bounds__(kThreads)
lp_kernel(const E* __restrict__ logits, int64_t V, int64_t ld, const int64_t* __restrict__ tokens, int top_k,
          int split, float* __restrict__ logp, float* __restrict__ entropy, float* __restrict__ top_logp,
          int32_t* __restrict__ top_id) {
  constexpr int kVec = 16 / sizeof(E), kWarps = kThreads / 32, kBatch = 4;
  __shared__ LpStat s_stat[kWarps];
  __shared__ LpStat s_cta;
  __shared__ uint64_t s_best[32];
  __shared__ float s_top[kWarps][32];
  __shared__ uint64_t s_cand[LP_CAND];
  __shared__ uint64_t s_out[LP_MAX_K];
  __shared__ float s_bound;
  __shared__ int s_count;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x / split;
  const int rank = (int)(blockIdx.x - row * split);
  const E* x = logits + row * ld;
  // this CTA's part: whole 16-byte vectors, the first CTA also what lies before the
  // first of them, the last one what lies behind the last
  const uint32_t mis = (uint32_t)(reinterpret_cast<uintptr_t>(x) & 15) / sizeof(E);
  const uint32_t head = (uint32_t)min((int64_t)(mis ? kVec - mis : 0), V);
  const uint32_t nvec = (uint32_t)((V - head) / kVec), tail = head + nvec * kVec;
  const uint32_t v0 = (uint32_t)((uint64_t)nvec * rank / split), v1 = (uint32_t)((uint64_t)nvec * (rank + 1) / split);
  const uint4* xv = reinterpret_cast<const uint4*>(x + head);
  int64_t token = -1;
  float given = 0.f;
  if (tid == 0 && rank == 0 && tokens) {
    token = tokens[row];
    if (token >= 0 && token < V) given = lp_load(x + token);
  }
  // a scalar element of this thread: one of the head, before its vectors, or one of the tail, behind them
  const bool in_head = rank == 0 && tid < head;
  const bool in_tail = rank == split - 1 && tid >= 32 && tail + (tid - 32) < V;  // (kVec < 32 of them)
  const int64_t odd = in_head ? tid : (in_tail ? (int64_t)tail + (tid - 32) : -1);
  const float odd_value = odd >= 0 ? lp_load(x + odd) : 0.f;
  auto single = [](float v) {
    return LpStat{v == v ? v : -INFINITY, v == INFINITY || v != v ? NAN : (v == -INFINITY ? 0.f : 1.f), 0.f};
  };
  LpStat st = {-INFINITY, 0.f, 0.f};
  if (odd >= 0) st = single(odd_value);
  // kBatch vectors, kThreads apart; what is past the part counts as -inf
  auto take = [&](auto whole, uint32_t i) {
    constexpr int kCount = kBatch;
    constexpr uint32_t kNone = sizeof(E) == 4 ? 0xFF800000u : 0xFF80FF80u;
    uint4 q[kCount];
    float v[kVec];
#pragma unroll
    for (int b = 0; b < kCount; ++b)
      q[b] = decltype(whole)::value || i + b * kThreads < v1 ? __ldg(xv + i + b * kThreads)
                                                             : make_uint4(kNone, kNone, kNone, kNone);
    const float top = lp_top<E, kCount>(q);
    if (top > st.m) {
      if (st.m == -INFINITY) st.m = top; else st.rise(top);
    }
    const float base = st.m == -INFINITY ? 0.f : -st.m;
    const uint64_t base2 = lp_pair(base, base), l2 = lp_pair(kLog2e, kLog2e);
    uint64_t S2 = 0ull, T2 = 0ull;
#pragma unroll
    for (int b = 0; b < kCount; ++b) {
      lp_unpack<E, kVec>(q[b], v);
#pragma unroll
      for (int j = 0; j < kVec; j += 2) {
        float d0, d1, e0, e1;
        lp_unpair(lp_add2(lp_pair(v[j], v[j + 1]), base2), d0, d1);
        const uint64_t d = lp_pair(lp_max_nan(d0, kFar), lp_max_nan(d1, kFar));
        lp_unpair(lp_mul2(d, l2), e0, e1);
        const uint64_t e = lp_pair(lp_ex2(e0), lp_ex2(e1));
        S2 = lp_add2(S2, e);
        T2 = lp_fma2(e, d, T2);
      }
    }
    float a, b;
    lp_unpair(S2, a, b);
    st.S += a + b;
    lp_unpair(T2, a, b);
    st.T += a + b;
  };
  uint32_t i0 = v0 + tid;
  for (; i0 + (kBatch - 1) * kThreads < v1; i0 += kThreads * kBatch) take(std::true_type{}, i0);
  if (i0 < v1) take(std::false_type{}, i0);
  const bool any = odd >= 0 || v0 + tid < v1;

  // the CTA's statistics, in a fixed order
  LpStat w = st;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    LpStat other = {__shfl_xor_sync(0xffffffffu, w.m, o), __shfl_xor_sync(0xffffffffu, w.S, o),
                    __shfl_xor_sync(0xffffffffu, w.T, o)};
    w.join(other);
  }
  if (lane == 0) s_stat[warp] = w;
  if (top_k) s_top[warp][lane] = any ? st.m : -INFINITY;
  if (tid == 0) s_count = 0;
  __syncthreads();
  if (warp == 0) {
    LpStat c = lane < kWarps ? s_stat[lane] : LpStat{-INFINITY, 0.f, 0.f};
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      LpStat other = {__shfl_xor_sync(0xffffffffu, c.m, o), __shfl_xor_sync(0xffffffffu, c.S, o),
                      __shfl_xor_sync(0xffffffffu, c.T, o)};
      c.join(other);
    }
    if (lane == 0) s_cta = c;
    if (top_k) {
      float g = -INFINITY;
#pragma unroll
      for (int u = 0; u < kWarps; ++u) g = fmaxf(g, s_top[u][lane]);
      int above = 0;
#pragma unroll
      for (int u = 0; u < 32; ++u) {
        const float o = __shfl_sync(0xffffffffu, g, u);
        above += o > g || (o == g && u < lane) ? 1 : 0;
      }
      if (above == top_k - 1) s_bound = g;
    }
  }
  __syncthreads();
  if (top_k) {
    const float bound = s_bound;
    const bool masked = bound == -INFINITY;
    bool scan = s_cta.S != s_cta.S;  // a NaN or +inf
    if (!scan) {
      const bool reaches = any && st.m >= bound && st.m > -INFINITY;
      auto offer = [&](float v, uint32_t idx) {
        if (masked ? v > bound : v >= bound) {
          const int at = atomicAdd(&s_count, 1);  // (the order does not matter: keys are ranked)
          if (at < LP_CAND) s_cand[at] = lp_key(v, idx);
        }
      };
      if (reaches && odd >= 0) offer(odd_value, (uint32_t)odd);
      // the vectors of each such thread, by its whole warp
      for (unsigned todo = __ballot_sync(0xffffffffu, reaches); todo; todo &= todo - 1) {
        const uint32_t owner = warp * 32 + __ffs(todo) - 1;
        for (uint32_t i = v0 + owner + lane * kThreads; i < v1; i += 32 * kThreads) {
          const uint4 q[1] = {__ldg(xv + i)};
          if (lp_top<E, 1>(q) >= bound) {
            float v[kVec];
            lp_unpack<E, kVec>(q[0], v);
#pragma unroll
            for (int j = 0; j < kVec; ++j) offer(v[j], head + i * kVec + j);
          }
        }
      }
      __syncthreads();
      const int count = s_count;
      scan = count > LP_CAND;
      if (!scan) {
        if (tid < LP_MAX_K) s_out[tid] = 0ull;
        __syncthreads();
        for (int c = tid; c < count; c += kThreads) {
          const uint64_t key = s_cand[c];
          int above = 0;
          for (int u = 0; u < count; ++u) above += s_cand[u] > key ? 1 : 0;
          if (above < top_k) s_out[above] = key;
        }
        if (masked && warp == 0) {  // the lowest indices of -inf follow; at most `count` others lie before them
          const int64_t begin = rank == 0 ? 0 : head + (int64_t)v0 * kVec;
          const int64_t end = rank == split - 1 ? V : head + (int64_t)v1 * kVec;
          int have = count;
          for (int64_t i = begin; i < end && have < top_k; i += 32) {
            const bool gone = i + lane < end && lp_load(x + i + lane) == -INFINITY;
            const unsigned mask = __ballot_sync(0xffffffffu, gone);
            const int at = have + __popc(mask & ((1u << lane) - 1));
            if (gone && at < top_k) s_out[at] = lp_key(-INFINITY, (uint32_t)(i + lane));
            have += __popc(mask);
          }
        }
      }
    }
    if (scan) {  // (uniform) one scan for each alternative
      uint64_t last = ~0ull;
      for (int r = 0; r < top_k; ++r) {
        uint64_t best = 0;
        auto offer = [&](float v, uint32_t idx) {
          const uint64_t key = lp_key(v, idx);
          if (key < last && key > best) best = key;
        };
        if (odd >= 0) offer(odd_value, (uint32_t)odd);
        for (uint32_t i = v0 + tid; i < v1; i += kThreads) {
          float v[kVec];
          lp_unpack<E, kVec>(__ldg(xv + i), v);
#pragma unroll
          for (int j = 0; j < kVec; ++j) offer(v[j], head + i * kVec + j);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) best = lp_max(best, __shfl_xor_sync(0xffffffffu, best, o));
        __syncthreads();
        if (lane == 0) s_best[warp] = best;
        __syncthreads();
        best = 0;
        for (int u = 0; u < kWarps; ++u) best = lp_max(best, s_best[u]);
        if (tid == 0) s_out[r] = best;
        last = best;
      }
    }
    __syncthreads();
  }
  // the row's statistics and alternatives, by the first CTA of a cluster
  if (split > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  if (rank == 0) {
    LpStat c = s_cta;
    if (split > 1) {
      const uint32_t at = smem_u32(&s_cta), out = smem_u32(s_out);
      for (int z = 1; z < split; ++z) {
        uint32_t r;
        LpStat o;
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(z));
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(o.m) : "r"(r) : "memory");
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(o.S) : "r"(r + 4) : "memory");
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(o.T) : "r"(r + 8) : "memory");
        c.join(o);
      }
      if (top_k) {
        for (int v = tid; v < split * top_k; v += kThreads) {
          const int z = v / top_k;
          uint32_t r;
          uint64_t key;
          asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(out + (v - z * top_k) * 8), "r"(z));
          asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(key) : "r"(r) : "memory");
          s_cand[v] = key;
        }
        __syncthreads();
        for (int v = tid; v < split * top_k; v += kThreads) {
          const uint64_t key = s_cand[v];
          int above = 0;
          for (int u = 0; u < split * top_k; ++u) above += s_cand[u] > key ? 1 : 0;
          if (key && above < top_k) s_out[above] = key;
        }
        __syncthreads();
      }
    }
    const float base = c.m == -INFINITY ? 0.f : c.m;
    const float log_sum = c.S == 0.f ? 0.f : logf(c.S);  // (NaN stays NaN)
    if (tid == 0) {
      if (logp) logp[row] = token >= 0 && token < V ? given - base - log_sum : 0.f;
      if (entropy) entropy[row] = c.S == 0.f ? 0.f : log_sum - c.T / c.S;
    }
    if (tid < top_k) {
      const uint64_t key = s_out[tid];
      top_logp[row * top_k + tid] = lp_key_value(key) - base - log_sum;
      top_id[row * top_k + tid] = (int32_t)~(uint32_t)key;
    }
  }
  if (split > 1) {  // no CTA leaves while the first may still read its results
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
}

template <typename E, int kThreads>
static cudaError_t launch_lp(const void* logits, int64_t N, int64_t V, int64_t ld, const int64_t* tokens, int top_k,
                             int split, float* logp, float* entropy, float* top_logp, int32_t* top_id,
                             cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(N * split), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = split;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  count_launches(1);
  return cudaLaunchKernelEx(&cfg, lp_kernel<E, kThreads>, static_cast<const E*>(logits), V, ld, tokens, top_k, split,
                            logp, entropy, top_logp, top_id);
}

cudaError_t launch_logprobs(const void* logits, int dtype, int64_t N, int64_t V, int64_t ld, const int64_t* tokens,
                            int top_k, float* logp, float* entropy, float* top_logp, int32_t* top_id, int num_sms,
                            cudaStream_t s) {
  const int64_t bytes = V * (dtype == 0 ? 4 : 2);
  // A row is split until there are two CTAs an SM, while each part is worth the cluster's hand-over: 64 rows of 128000
  // fp32 take 12.5 us in eight parts and 20.2 whole, one row of 32000 bf16 takes 12.0 in eight and 8.4 whole. (Splitting
  // 1024 rows of 100003 fp32 further for an evener last wave: 98 us instead of 92.)
  int split = 1;
  while (split < 8 && N * split < 2 * num_sms && bytes / (2 * split) >= 32768) split *= 2;
  const bool small = bytes / split <= 16384;
#define SLIM_LP(E)                                                                                                    \
  (small ? launch_lp<E, 128>(logits, N, V, ld, tokens, top_k, split, logp, entropy, top_logp, top_id, s)             \
         : launch_lp<E, 256>(logits, N, V, ld, tokens, top_k, split, logp, entropy, top_logp, top_id, s))
  return dtype == 0 ? SLIM_LP(float) : SLIM_LP(uint16_t);
#undef SLIM_LP
}

}  // namespace slim
