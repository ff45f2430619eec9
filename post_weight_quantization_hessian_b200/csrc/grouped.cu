// dequant_grouped_gemm: Y_e = X_e W_hat_e^T for a set of packed layers (the
// experts of a mixture, or one layer), rows grouped by expert with ragged
// counts that are known on the device only.
//
// Per (row r of expert e, output i), with c the column groups of width b:
//   y[r][i] = sum_c scale (sum_j x_j q_j - zero sum_j x_j).
//
// This kernel is the plain one: a thread per output, the codes extracted one
// by one, fp32 sums.
#include <cstdint>
#include "common.cuh"

namespace slim {

// Where the asynchronous kernels of the current device record a failure; read
// and cleared by slim_async_status.
__device__ DevStatus g_async_status;

cudaError_t take_async_status(DevStatus* host, cudaStream_t s) {
  static const DevStatus clear = {};
  cudaError_t e = cudaMemcpyFromSymbolAsync(host, g_async_status, sizeof(DevStatus), 0, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaMemcpyToSymbolAsync(g_async_status, &clear, sizeof(DevStatus), 0, cudaMemcpyHostToDevice, s);
  return e == cudaSuccess ? cudaStreamSynchronize(s) : e;
}

__device__ __forceinline__ float gg_ld(const void* p, int64_t i, int dtype) {
  if (dtype == 0) return static_cast<const float*>(p)[i];
  return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
}
__device__ __forceinline__ uint16_t gg_bf16(float v) {
  uint16_t h;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(v));
  return h;
}

__global__ void __launch_bounds__(128)
gg_plain_kernel(const uint32_t* __restrict__ codes, const uint8_t* __restrict__ bits, const float* __restrict__ scale,
                const float* __restrict__ zero, int E, int64_t m, int64_t n, int group, int64_t rw,
                const void* __restrict__ x, int xdtype, int64_t T, const int32_t* __restrict__ row_index,
                const int32_t* __restrict__ offsets, int64_t R, void* __restrict__ y, int ydtype) {
  const int64_t i = (int64_t)blockIdx.x * 128 + threadIdx.x;
  const int k = (int)(n / group);
  for (int64_t r = blockIdx.y; r < R; r += gridDim.y) {
    int e = 0;
    while (e < E && !(offsets[e] <= r && r < offsets[e + 1])) ++e;
    if (e == E || i >= m) continue;
    const int64_t src = row_index ? row_index[r] : r;
    const bool have = src >= 0 && src < T;
    const uint32_t* w = codes + (e * m + i) * rw;
    const float* sc = scale + (e * m + i) * k;
    const float* ze = zero + (e * m + i) * k;
    int64_t bit = 0;
    float acc = 0.f;
    for (int c = 0; c < k; ++c) {
      const int b = bits[(int64_t)e * k + c];
      if (b < 1 || b > 8) continue;
      float a = 0.f, xs = 0.f;
      for (int j = 0; j < group; ++j, bit += b) {
        const int64_t wi = bit >> 5;
        const uint32_t lo = wi < rw ? w[wi] : 0u, hi = wi + 1 < rw ? w[wi + 1] : 0u;
        const uint32_t q = __funnelshift_r(lo, hi, (uint32_t)bit & 31) & ((1u << b) - 1);
        const float xv = have ? gg_ld(x, src * n + (int64_t)c * group + j, xdtype) : 0.f;
        a = fmaf(xv, (float)q, a);
        xs += xv;
      }
      acc = fmaf(sc[c], fmaf(-ze[c], xs, a), acc);
    }
    if (ydtype == 0)
      static_cast<float*>(y)[r * m + i] = acc;
    else
      static_cast<uint16_t*>(y)[r * m + i] = gg_bf16(acc);
  }
}

size_t grouped_workspace_bytes(int64_t E, int64_t m, int64_t n, int group, int xdtype, int64_t R) { return 0; }

cudaError_t launch_grouped(const uint32_t* codes, const uint8_t* bits, const float* scale, const float* zero,
                           int64_t E, int64_t m, int64_t n, int group, int avg_bits, const void* x, int xdtype,
                           int64_t T, const int32_t* row_index, const int32_t* offsets, int64_t R, void* y,
                           int ydtype, uint8_t* ws, int num_sms, cudaStream_t s) {
  const dim3 grid((unsigned)((m + 127) / 128), (unsigned)(R < 65535 ? R : 65535));
  gg_plain_kernel<<<grid, 128, 0, s>>>(codes, bits, scale, zero, (int)E, m, n, group, n * avg_bits / 32, x, xdtype, T,
                                       row_index, offsets, R, y, ydtype);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace slim
