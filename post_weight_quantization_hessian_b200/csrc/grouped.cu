// dequant_grouped_gemm: Y_e = X_e W_hat_e^T for a set of packed layers (the
// experts of a mixture, or one layer), rows grouped by expert with ragged
// counts that are known on the device only.
//
// Per (row r of expert e, output i), with c the column groups of width b:
//   y[r][i] = sum_c scale (sum_j x_j q_j - zero sum_j x_j).
// The codes enter the tensor cores as exact bf16 values v (decode.cuh), so a
// group's D = sum_j x_j v_j is a sum of exact products in fp32, and the scale
// and zero are applied to D and to xs = sum_j x_j in fp32: no weight is rounded.
#include <algorithm>
#include <cstdint>
#include "common.cuh"
#include "decode.cuh"
#include "tmap.h"

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

// ---------------------------------------------------------------- preparation
// Sums of x over each column group, xs[c][r] (fp32), and where the tensor-core
// kernel cannot read x as it is (gathered rows, fp32), the rows as bf16 in
// grouped order: fp32 as three planes x1 + x2 + x3 that hold all 24 bits.
// A warp takes a row, a block 8 rows; 16-byte loads; the sums of 8 rows are
// collected in shared memory so that their stores cover whole 32-byte sectors.
constexpr int GP_ROWS = 8;

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__global__ void __launch_bounds__(GP_ROWS * 32)
gg_prep_kernel(const void* __restrict__ x, int xdtype, int64_t T, const int32_t* __restrict__ row_index, int64_t R,
               int64_t Rs, int64_t n, int group, uint16_t* __restrict__ xg, int planes, float* __restrict__ xs) {
  extern __shared__ float sums[];  // [k][8]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t r0 = (int64_t)blockIdx.x * GP_ROWS, r = r0 + warp;
  const int k = (int)(n / group), per = group / 8;  // lanes of a group
  int64_t src = r;
  if (row_index) src = r < R ? row_index[r] : -1;
  const bool have = r < R && src >= 0 && src < T;
  for (int64_t j = lane * 8; j < (n + 255) / 256 * 256; j += 256) {
    float v[8];
    uint32_t p[4] = {0, 0, 0, 0};
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = 0.f;
    if (have && j < n) {
      if (xdtype == 1) {
        const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + src * n + j);
        p[0] = q.x; p[1] = q.y; p[2] = q.z; p[3] = q.w;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          v[2 * u] = __uint_as_float(p[u] << 16);
          v[2 * u + 1] = __uint_as_float(p[u] & 0xFFFF0000u);
        }
      } else {
        const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(x) + src * n + j);
        const float4 a = q[0], b = q[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
      }
    }
    float s = ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    for (int o = 1; o < per; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (j < n && lane % per == 0) sums[(j / group) * GP_ROWS + warp] = s;
    if (xg && r < R && j < n) {
      if (xdtype == 1) {
        *reinterpret_cast<uint4*>(xg + r * n + j) = make_uint4(p[0], p[1], p[2], p[3]);
      } else {
#pragma unroll
        for (int pl = 0; pl < 3; ++pl) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            p[u] = pack_bf16(v[2 * u], v[2 * u + 1]);
            v[2 * u] -= __uint_as_float(p[u] << 16);
            v[2 * u + 1] -= __uint_as_float(p[u] & 0xFFFF0000u);
          }
          *reinterpret_cast<uint4*>(xg + ((int64_t)pl * R + r) * n + j) = make_uint4(p[0], p[1], p[2], p[3]);
        }
      }
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < k * GP_ROWS; e += GP_ROWS * 32) {
    const int c = e / GP_ROWS, q = e % GP_ROWS;
    if (r0 + q < R) xs[c * Rs + r0 + q] = sums[e];
  }
}

// ---------------------------------------------------------------- tensor cores
// A persistent CTA per SM takes tiles of 128 outputs x up to 256 rows (an
// expert's rows cut evenly, in multiples of 16, so that a narrow remainder does
// not cost a tile's decoding). The whole depth n is one tile's; per 64 columns
// (a box):
//   warps 8..11  decode the 128 x 64 codes into the A operand in shared memory
//                (thread = output row; K-major, 128-byte swizzle)
//   warp 12      x boxes (64 columns x rows) by TMA, the B operand
//   warp 13      tcgen05.mma M=128 x N=rows x K=16, A x B^T into tensor memory:
//                each group into its own accumulator, two in flight
//   warp 14      windows of 16 code words x 128 rows by TMA
//   warp 15      xs of each group by bulk copies; tensor memory
//   warps 0..7   per group: acc += coef_d D + coef_x xs in packed fp32 pairs,
//                thread = output row, two warps a row set on alternate 32 columns;
//                at the end y (a warp stores 32 consecutive outputs of a row)
// Rows of two neighbouring experts may share an x box: an accumulator column
// depends on its own row of x alone, and only the tile's rows are stored.
constexpr int GT_M = 128, GT_N = 256, GT_K = 64;
constexpr int GT_THREADS = 512;
constexpr int GT_XS = 4, GT_AS = 3, GT_CS = 3, GT_SS = 4;  // ring lengths: x, A, code windows, group sums
constexpr int GT_XBYTES = GT_N * GT_K * 2, GT_ABYTES = GT_M * GT_K * 2;
constexpr int GT_WIN = 16, GT_CBYTES = GT_M * GT_WIN * 4, GT_SBYTES = GT_N * 4;
constexpr int GT_OFF_A = GT_XS * GT_XBYTES;
constexpr int GT_OFF_C = GT_OFF_A + GT_AS * GT_ABYTES;
constexpr int GT_OFF_S = GT_OFF_C + GT_CS * GT_CBYTES;
constexpr int GT_OFF_BAR = GT_OFF_S + GT_SS * GT_SBYTES;
constexpr int GT_OFF_E = GT_OFF_BAR + 512;
constexpr int GT_MAX_E = 1024;
constexpr int GT_SMEM = GT_OFF_E + 2 * (GT_MAX_E + 1) * 4 + 1024;  // + alignment
static_assert(GT_SMEM <= 227 * 1024, "shared memory of a CTA");

struct GtParams {
  const uint32_t* codes;
  const uint8_t* bits;
  const float* scale;
  const float* zero;
  const int32_t* offsets;
  const float* xs;
  void* y;
  int64_t m, n, R, Rs, rw;
  int E, k, group, planes, ydtype, codes_tma, mtiles;
};
struct GtMaps {
  CUtensorMap x256, x32, codes;
};

struct GtTile {
  int e;        // expert
  int64_t m0;   // first output
  int col0;     // first row of x (a multiple of 4; may lie before the expert's first)
  int r0, r1;   // the expert's rows
  int N;        // accumulator columns
};

struct GtRing {  // position in a ring of S slots and the phase that goes with it
  uint32_t slot = 0, phase = 0;
  __device__ __forceinline__ void step(uint32_t S) {
    if (++slot == S) {
      slot = 0;
      phase ^= 1;
    }
  }
};

__device__ __forceinline__ uint64_t gt_pack(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void gt_unpack(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t gt_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void gt_cp4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// Tiles of expert e's rows [r0, r1): count, and the width of each.
__device__ __forceinline__ int gt_row_tiles(int r0, int r1, int& width) {
  if (r1 <= r0) {
    width = 0;
    return 0;
  }
  const int span = r1 - (r0 & ~3), nt = (span + GT_N - 1) / GT_N;
  width = ((span + nt - 1) / nt + 15) & ~15;
  return nt;
}

__device__ __forceinline__ GtTile gt_tile(const GtParams& p, int t, const int* first, const int* off) {
  int lo = 0, hi = p.E;  // the last expert whose first tile is <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= t) lo = mid; else hi = mid;
  }
  GtTile u;
  u.e = lo;
  u.r0 = off[lo];
  u.r1 = off[lo + 1];
  int width;
  gt_row_tiles(u.r0, u.r1, width);
  const int j = (t - first[lo]) / p.mtiles;
  u.m0 = (int64_t)(t - first[lo] - j * p.mtiles) * GT_M;
  u.col0 = (u.r0 & ~3) + j * width;
  const int cols = min(width, u.r1 - u.col0);
  u.N = (cols + 15) & ~15;
  return u;
}

template <bool kCenter>
__global__ void __launch_bounds__(GT_THREADS, 1) gg_tc_kernel(const __grid_constant__ GtMaps tm, const GtParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sx = smem;
  uint8_t* sa = smem + GT_OFF_A;
  uint8_t* sc = smem + GT_OFF_C;
  float* ss = reinterpret_cast<float*>(smem + GT_OFF_S);
  uint64_t* xfull = reinterpret_cast<uint64_t*>(smem + GT_OFF_BAR);
  uint64_t* xempty = xfull + GT_XS;
  uint64_t* afull = xempty + GT_XS;
  uint64_t* aempty = afull + GT_AS;
  uint64_t* cfull = aempty + GT_AS;
  uint64_t* cempty = cfull + GT_CS;
  uint64_t* sfull = cempty + GT_CS;
  uint64_t* sempty = sfull + GT_SS;
  uint64_t* dfull = sempty + GT_SS;
  uint64_t* dempty = dfull + 2;
  uint64_t* done = dempty + 2;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
  int* s_first = reinterpret_cast<int*>(smem + GT_OFF_E);
  int* s_off = s_first + GT_MAX_E + 1;
  DevStatus* st = &g_async_status;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < GT_XS; ++i) { mbar_init(&xfull[i], 1); mbar_init(&xempty[i], 1); }
    for (int i = 0; i < GT_AS; ++i) { mbar_init(&afull[i], 4); mbar_init(&aempty[i], 1); }
    for (int i = 0; i < GT_CS; ++i) { mbar_init(&cfull[i], 1); mbar_init(&cempty[i], 4); }
    for (int i = 0; i < GT_SS; ++i) { mbar_init(&sfull[i], 1); mbar_init(&sempty[i], 8); }
    for (int i = 0; i < 2; ++i) { mbar_init(&dfull[i], 1); mbar_init(&dempty[i], 8); }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm.x256);
    tma_prefetch_desc(&tm.x32);
    if (p.codes_tma) tma_prefetch_desc(&tm.codes);
  }
  if (warp == 15) tmem_alloc(tslot, 512);
  for (int e = tid; e <= p.E; e += GT_THREADS) s_off[e] = max(0, min(p.offsets[e], (int)p.R));
  __syncthreads();
  if (warp == 0) {  // tiles before each expert
    int run = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      int width, v = 0;
      if (e < p.E) v = gt_row_tiles(s_off[e], s_off[e + 1], width) * p.mtiles;
      int incl = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
      }
      if (e < p.E) s_first[e] = run + incl - v;
      run += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) s_first[p.E] = run;
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tslot;
  const int tiles = s_first[p.E];
  const int nbox = (int)((p.n + GT_K - 1) / GT_K);

  if (warp < 8) {
    // ------------------------------------------------------------ epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    const int half = warp >> 2, sub = (warp & 3) * 32;
    GtRing sr, dr;
    bool ok = true;
    for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      const GtTile u = gt_tile(p, t, s_first, s_off);
      const int64_t i = u.m0 + sub + lane;
      const bool row_ok = i < p.m;
      const int64_t srow = ((int64_t)u.e * p.m + (row_ok ? i : p.m - 1)) * p.k;
      const uint8_t* bits = p.bits + (int64_t)u.e * p.k;
      const bool vec = (p.k & 3) == 0 &&
                       ((reinterpret_cast<uintptr_t>(p.scale) | reinterpret_cast<uintptr_t>(p.zero)) & 15) == 0;
      uint64_t acc[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) acc[j] = 0ull;
      float4 s4 = {}, z4 = {}, sn = {}, zn = {};
      auto load4 = [&](int c, float4& a, float4& b) {
        if (vec) {
          if (c < p.k) {
            a = *reinterpret_cast<const float4*>(p.scale + srow + c);
            b = *reinterpret_cast<const float4*>(p.zero + srow + c);
          }
        } else {
          float av[4] = {}, bv[4] = {};
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (c + q < p.k) {
              av[q] = p.scale[srow + c + q];
              bv[q] = p.zero[srow + c + q];
            }
          a = make_float4(av[0], av[1], av[2], av[3]);
          b = make_float4(bv[0], bv[1], bv[2], bv[3]);
        }
      };
      load4(0, sn, zn);
      int bnext = bits[0];
      for (int c = 0; c < p.k; ++c) {
        if ((c & 3) == 0) {
          s4 = sn;
          z4 = zn;
          load4(c + 4, sn, zn);
        }
        const int b = bnext;
        if (c + 1 < p.k) bnext = bits[c + 1];
        const float s = s4.x, z = z4.x;
        s4 = make_float4(s4.y, s4.z, s4.w, 0.f);
        z4 = make_float4(z4.y, z4.z, z4.w, 0.f);
        const bool valid = b >= 1 && b <= 8;
        const float cd = valid ? coef_d<kCenter>(b, s) : 0.f, cx = valid ? coef_x<kCenter>(b, s, z) : 0.f;
        const uint64_t cd2 = gt_pack(cd, cd), cx2 = gt_pack(cx, cx);
        if (!mbar_wait(&sfull[sr.slot], sr.phase, abort_flag, st, 10) ||
            !mbar_wait(&dfull[dr.slot], dr.phase, abort_flag, st, 11)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const float* xs = ss + sr.slot * GT_N;
        const uint32_t dcol = tbase + ((uint32_t)sub << 16) + dr.slot * GT_N;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int col = (2 * q + half) * 32;
          if (col < u.N) {
            uint32_t d[32];
            tmem_ld32(dcol + col, d);
            tc_wait_ld();
            const ulonglong2* x2 = reinterpret_cast<const ulonglong2*>(xs + col);
#pragma unroll
            for (int v = 0; v < 8; ++v) {
              const ulonglong2 xv = x2[v];
              uint64_t& a0 = acc[q * 16 + 2 * v];
              uint64_t& a1 = acc[q * 16 + 2 * v + 1];
              a0 = gt_fma2(cx2, xv.x, gt_fma2(cd2, ((uint64_t)d[4 * v + 1] << 32) | d[4 * v], a0));
              a1 = gt_fma2(cx2, xv.y, gt_fma2(cd2, ((uint64_t)d[4 * v + 3] << 32) | d[4 * v + 2], a1));
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&dempty[dr.slot]);
          mbar_arrive(&sempty[sr.slot]);
        }
        dr.step(2);
        sr.step(GT_SS);
      }
      if (!ok) break;
      if (row_ok) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int col = (2 * q + half) * 32;
          if (col < u.N) {
#pragma unroll
            for (int v = 0; v < 16; ++v) {
              float a, b;
              gt_unpack(acc[q * 16 + v], a, b);
#pragma unroll
              for (int w = 0; w < 2; ++w) {
                const int r = u.col0 + col + 2 * v + w;
                if (r >= u.r0 && r < u.r1 && col + 2 * v + w < u.N) {
                  const float val = w ? b : a;
                  if (p.ydtype == 0) {
                    static_cast<float*>(p.y)[(int64_t)r * p.m + i] = val;
                  } else {
                    uint16_t h;
                    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(val));
                    static_cast<uint16_t*>(p.y)[(int64_t)r * p.m + i] = h;
                  }
                }
              }
            }
          }
        }
      }
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------ decoding
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    const int row = tid - 256;
    GtRing ar;
    uint32_t ci = 0;  // windows taken so far
    bool ok = true;
    const int nwin = (int)((p.rw + GT_WIN - 1) / GT_WIN);
    const uint32_t rbase = smem_u32(sc) + row * (GT_WIN * 4), rswz = (row >> 1) & 3;
    for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      const GtTile u = gt_tile(p, t, s_first, s_off);
      const uint8_t* bits = p.bits + (int64_t)u.e * p.k;
      const int64_t i = u.m0 + row;
      const uint32_t* crow = p.codes + ((int64_t)u.e * p.m + (i < p.m ? i : p.m - 1)) * p.rw;
      int win = -1, wpos = 0;
      uint32_t wslot = 0;
      // rows that are not 16-byte aligned: each thread copies its own words, two windows ahead
      auto copy_window = [&](int w) {
        uint8_t* dst = sc + (w % GT_CS) * GT_CBYTES + row * (GT_WIN * 4);
#pragma unroll 4
        for (int q = 0; q < GT_WIN; ++q)
          if (w * GT_WIN + q < p.rw) gt_cp4(dst + (((q >> 2) ^ rswz) << 4) + (q & 3) * 4, crow + w * GT_WIN + q);
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      if (!p.codes_tma) {
        copy_window(0);
        copy_window(1);
      }
      auto next_window = [&]() {
        ++win;
        if (p.codes_tma) {
          if (win > 0) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&cempty[wslot]);
          }
          wslot = ci % GT_CS;
          const uint32_t ph = (ci / GT_CS) & 1;
          ++ci;
          return mbar_wait(&cfull[wslot], ph, abort_flag, st, 20);
        }
        wslot = win % GT_CS;
        copy_window(win + 2);
        asm volatile("cp.async.wait_group 2;" ::: "memory");
        return true;
      };
      auto word = [&](int wi) -> uint32_t {
        if (wi >= p.rw) return 0u;
        while ((wi / GT_WIN) != win) {
          if (!ok) return 0u;
          ok = next_window();
        }
        uint32_t v;
        const uint32_t a = rbase + wslot * GT_CBYTES + ((((uint32_t)wi >> 2) & 3) ^ rswz) * 16 + (wi & 3) * 4;
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
        return v;
      };
      for (int kb = 0; kb < nbox && ok; ++kb) {
        if (!mbar_wait(&aempty[ar.slot], ar.phase ^ 1, abort_flag, st, 21)) {
          ok = false;
          break;
        }
        uint8_t* arow = sa + ar.slot * GT_ABYTES + row * 128;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          const int col = kb * GT_K + h * 32;
          if (col >= p.n) break;
          const int b = bits[col / p.group];
          uint32_t o[16];
#pragma unroll
          for (int q = 0; q < 16; ++q) o[q] = 0u;
          switch (b) {
#define GT_CASE(B)                                                          \
  case B: {                                                                 \
    uint32_t w[B];                                                          \
    _Pragma("unroll") for (int q = 0; q < B; ++q) w[q] = word(wpos + q);    \
    decode32<B, kCenter>(w, o);                                             \
    wpos += B;                                                              \
  } break;
            GT_CASE(1) GT_CASE(2) GT_CASE(3) GT_CASE(4) GT_CASE(5) GT_CASE(6) GT_CASE(7) GT_CASE(8)
#undef GT_CASE
            default: break;
          }
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<uint4*>(arow + (((h * 4 + q) ^ (row & 7)) << 4)) =
                make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&afull[ar.slot]);
        ar.step(GT_AS);
      }
      if (p.codes_tma) {
        while (ok && win < nwin - 1) ok = next_window();
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&cempty[wslot]);
      } else {
        asm volatile("cp.async.wait_all;" ::: "memory");
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 12 && lane == 0) {
      // ---------------------------------------------------------- x boxes
      uint32_t xi = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
        const GtTile u = gt_tile(p, t, s_first, s_off);
        const int per = u.N > 128 ? 1 : (u.N > 64 ? 2 : 4);  // boxes of a stage
        for (int kb = 0; kb < nbox && ok; kb += per) {
          const int nb = min(per, nbox - kb);
          for (int pl = p.planes - 1; pl >= 0; --pl, ++xi) {
            const uint32_t s = xi % GT_XS;
            if (!mbar_wait(&xempty[s], ((xi / GT_XS) & 1) ^ 1, abort_flag, st, 30)) {
              ok = false;
              break;
            }
            const int y0 = (int)(pl * p.R) + u.col0;
            uint8_t* dst = sx + s * GT_XBYTES;
            if (per == 1) {
              mbar_arrive_expect_tx(&xfull[s], GT_XBYTES);
              tma_load_2d(dst, &tm.x256, &xfull[s], kb * GT_K, y0);
            } else {
              const int nr = (u.N + 31) / 32;
              mbar_arrive_expect_tx(&xfull[s], (uint32_t)(nb * nr * 4096));
              for (int q = 0; q < nb; ++q)
                for (int v = 0; v < nr; ++v)
                  tma_load_2d(dst + q * (GT_XBYTES / per) + v * 4096, &tm.x32, &xfull[s], (kb + q) * GT_K, y0 + 32 * v);
            }
          }
        }
      }
      for (uint32_t j = xi > GT_XS ? xi - GT_XS : 0; j < xi; ++j) mbar_drain(&xfull[j % GT_XS], (j / GT_XS) & 1);
    } else if (warp == 13 && lane == 0) {
      // ---------------------------------------------------------- matrix products
      uint32_t xi = 0;
      GtRing ar, dr;
      bool ok = true;
      const int parts = p.group == 32 ? 2 : 1, ksteps = 4 / parts;
      for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
        const GtTile u = gt_tile(p, t, s_first, s_off);
        const int per = u.N > 128 ? 1 : (u.N > 64 ? 2 : 4);
        const uint32_t idesc = idesc_bf16_f32(GT_M, 16, false, false) + ((uint32_t)(u.N / 8 - 2) << 17);
        for (int kb = 0; kb < nbox && ok; ++kb) {
          if (!mbar_wait(&afull[ar.slot], ar.phase, abort_flag, st, 40)) {
            ok = false;
            break;
          }
          const int sub = kb % per;
          const bool first_sub = sub == 0, last_sub = sub == per - 1 || kb == nbox - 1;
          const uint32_t abase = smem_u32(sa) + ar.slot * GT_ABYTES;
          for (int h = 0; h < parts && ok; ++h) {
            if (kb * GT_K + h * 32 >= p.n) break;
            const bool last_part = h == parts - 1 || kb * GT_K + (h + 1) * 32 >= p.n;
            const bool begins = p.group != 128 || (kb & 1) == 0, ends = p.group != 128 || (kb & 1) == 1;
            if (begins && !mbar_wait(&dempty[dr.slot], dr.phase ^ 1, abort_flag, st, 41)) {
              ok = false;
              break;
            }
            for (int q = 0; q < p.planes; ++q) {
              const uint32_t s = (xi + q) % GT_XS;
              if (first_sub && h == 0 && !mbar_wait(&xfull[s], ((xi + q) / GT_XS) & 1, abort_flag, st, 42)) {
                ok = false;
                break;
              }
              tc_fence_after();
              const uint32_t bbase = smem_u32(sx) + s * GT_XBYTES + sub * (GT_XBYTES / per);
              for (int k16 = 0; k16 < ksteps; ++k16) {
                const uint32_t koff = (uint32_t)(h * ksteps + k16) * 32;
                tc_mma_bf16(tbase + dr.slot * GT_N, sdesc_sw128(abase + koff, 16, 1024),
                            sdesc_sw128(bbase + koff, 16, 1024), idesc, (begins && q == 0 && k16 == 0) ? 0u : 1u);
              }
              if (last_sub && last_part) tc_commit(&xempty[s]);
            }
            if (ok && ends) {
              tc_commit(&dfull[dr.slot]);
              dr.step(2);
            }
          }
          if (!ok) break;
          if (last_sub) xi += p.planes;
          tc_commit(&aempty[ar.slot]);
          ar.step(GT_AS);
        }
      }
      // every issued product completes before tensor memory can be freed, also after an abort
      tc_commit(done);
      mbar_drain(done, 0);
    } else if (warp == 14 && lane == 0 && p.codes_tma) {
      // ---------------------------------------------------------- code windows
      uint32_t ci = 0;
      bool ok = true;
      const int nwin = (int)((p.rw + GT_WIN - 1) / GT_WIN);
      for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
        const GtTile u = gt_tile(p, t, s_first, s_off);
        const int y0 = (int)(u.e * p.m + u.m0);
        for (int w = 0; w < nwin; ++w, ++ci) {
          const uint32_t s = ci % GT_CS;
          if (!mbar_wait(&cempty[s], ((ci / GT_CS) & 1) ^ 1, abort_flag, st, 50)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&cfull[s], GT_CBYTES);
          tma_load_2d(sc + s * GT_CBYTES, &tm.codes, &cfull[s], w * GT_WIN, y0);
        }
      }
      for (uint32_t j = ci > GT_CS ? ci - GT_CS : 0; j < ci; ++j) mbar_drain(&cfull[j % GT_CS], (j / GT_CS) & 1);
    } else if (warp == 15 && lane == 0) {
      // ---------------------------------------------------------- group sums of x
      GtRing sr;
      uint32_t si = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
        const GtTile u = gt_tile(p, t, s_first, s_off);
        for (int c = 0; c < p.k; ++c, ++si) {
          if (!mbar_wait(&sempty[sr.slot], sr.phase ^ 1, abort_flag, st, 60)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&sfull[sr.slot], (uint32_t)u.N * 4);
          bulk_load(ss + sr.slot * GT_N, p.xs + (int64_t)c * p.Rs + u.col0, (uint32_t)u.N * 4, &sfull[sr.slot]);
          sr.step(GT_SS);
        }
      }
      for (uint32_t j = si > GT_SS ? si - GT_SS : 0; j < si; ++j) mbar_drain(&sfull[j % GT_SS], (j / GT_SS) & 1);
    }
    __syncwarp();
  }
  __syncthreads();
  if (warp == 15) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// ---------------------------------------------------------------- host side
struct GroupedPlan {
  int64_t Rs;  // row stride of xs: a tile's columns may reach past R
  int planes;  // bf16 planes copied in grouped order (0: x is read as it is)
  size_t off_xg, bytes;
};

static GroupedPlan grouped_plan(int64_t n, int group, int xdtype, bool gathered, int64_t R) {
  GroupedPlan g{};
  g.Rs = ((R + 3) & ~int64_t(3)) + GT_N;
  g.planes = xdtype == 0 ? 3 : (gathered ? 1 : 0);
  g.off_xg = ((size_t)(n / group) * g.Rs * 4 + 255) & ~size_t(255);
  g.bytes = g.off_xg + (((size_t)g.planes * R * n * 2 + 255) & ~size_t(255));
  return g;
}

size_t grouped_workspace_bytes(int64_t E, int64_t m, int64_t n, int group, int xdtype, bool gathered, int64_t R) {
  return grouped_plan(n, group, xdtype, gathered, R).bytes;
}

template <bool kCenter>
static cudaError_t launch_gt(const GtMaps& tm, const GtParams& p, int num_sms, cudaStream_t s) {
  static std::atomic<uint64_t> attr{0};
  uint64_t bit = 0;
  if (attr_pending(attr, bit)) {
    const cudaError_t e =
        cudaFuncSetAttribute(gg_tc_kernel<kCenter>, cudaFuncAttributeMaxDynamicSharedMemorySize, GT_SMEM);
    if (e != cudaSuccess) return e;
    attr.fetch_or(bit);
  }
  gg_tc_kernel<kCenter><<<num_sms, GT_THREADS, GT_SMEM, s>>>(tm, p);
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_grouped(const uint32_t* codes, const uint8_t* bits, const float* scale, const float* zero,
                           int64_t E, int64_t m, int64_t n, int group, int avg_bits, const void* x, int xdtype,
                           int64_t T, const int32_t* row_index, const int32_t* offsets, int64_t R, void* y,
                           int ydtype, uint8_t* ws, int num_sms, cudaStream_t s) {
  const GroupedPlan g = grouped_plan(n, group, xdtype, row_index != nullptr, R);
  float* xs = reinterpret_cast<float*>(ws);
  uint16_t* xg = g.planes ? reinterpret_cast<uint16_t*>(ws + g.off_xg) : nullptr;
  const int k = (int)(n / group);
  gg_prep_kernel<<<(unsigned)((R + GP_ROWS - 1) / GP_ROWS), GP_ROWS * 32, (size_t)k * GP_ROWS * 4, s>>>(
      x, xdtype, T, row_index, R, g.Rs, n, group, xg, g.planes, xs);
  count_launches(1);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  GtParams p{};
  p.codes = codes; p.bits = bits; p.scale = scale; p.zero = zero; p.offsets = offsets; p.xs = xs; p.y = y;
  p.m = m; p.n = n; p.R = R; p.Rs = g.Rs; p.rw = n * avg_bits / 32;
  p.E = (int)E; p.k = k; p.group = group; p.planes = g.planes ? g.planes : 1; p.ydtype = ydtype;
  p.mtiles = (int)((m + GT_M - 1) / GT_M);
  p.codes_tma = p.rw % 4 == 0;
  GtMaps tm;
  const void* xb = xg ? static_cast<const void*>(xg) : x;
  const uint64_t rows = xg ? (uint64_t)g.planes * R : (uint64_t)T;
  if (!make_tmap_bf16(&tm.x256, xb, (uint64_t)n, rows, GT_K, GT_N) ||
      !make_tmap_bf16(&tm.x32, xb, (uint64_t)n, rows, GT_K, 32))
    return cudaErrorInvalidValue;
  if (p.codes_tma && !make_tmap_u32_sw64(&tm.codes, codes, (uint64_t)p.rw, (uint64_t)(E * m), GT_WIN, GT_M))
    return cudaErrorInvalidValue;
  return ydtype == 0 ? launch_gt<true>(tm, p, num_sms, s) : launch_gt<false>(tm, p, num_sms, s);
}

}  // namespace slim
