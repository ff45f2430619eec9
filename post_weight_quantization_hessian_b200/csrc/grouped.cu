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
#include <type_traits>
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
// Sums of x over each column group, as the bf16 parts that the correction
// columns of the tensor-core kernel take (below), and where that kernel cannot
// read x as it is (gathered rows, fp32), the rows as bf16 in grouped order: fp32
// as three planes x1 + x2 + x3 that hold all 24 bits. A warp takes a row, with
// 16-byte loads and stores; bound by the bytes of x (read, and written if copied).
constexpr int GP_ROWS = 8;

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// v = p1 + p2 + p3, each a bf16 value (8 + 8 + 8 bits).
__device__ __forceinline__ void split3(float v, float& p1, float& p2, float& p3) {
  p1 = __uint_as_float(pack_bf16(v, 0.f) << 16);
  p2 = __uint_as_float(pack_bf16(v - p1, 0.f) << 16);
  p3 = __uint_as_float(pack_bf16(v - p1 - p2, 0.f) << 16);
}
// Correction columns of one group: the products of the parts of a and b that
// matter, side by side. Four columns (a1 b1, a1 b2, a2 b1, a2 b2) leave out about
// 2^-17 of a b, eight (with a1 b3, a3 b1, a2 b3, a3 b2) about 2^-24.
template <int kSlots, bool kFirst>
__device__ __forceinline__ void split_slots(float v, uint32_t (&o)[kSlots / 2]) {
  float p1, p2, p3;
  split3(v, p1, p2, p3);
  if (kFirst) {
    o[0] = pack_bf16(p1, p1);
    o[1] = pack_bf16(p2, p2);
    if constexpr (kSlots == 8) {
      o[2] = pack_bf16(p1, p3);
      o[3] = pack_bf16(p2, p3);
    }
  } else {
    o[0] = pack_bf16(p1, p2);
    o[1] = pack_bf16(p1, p2);
    if constexpr (kSlots == 8) {
      o[2] = pack_bf16(p3, p1);
      o[3] = pack_bf16(p3, p2);
    }
  }
}

template <int kSlots>
__global__ void __launch_bounds__(GP_ROWS * 32)
gg_prep_kernel(const void* __restrict__ x, int xdtype, int64_t T, const int32_t* __restrict__ row_index, int64_t R,
               int64_t n, int group, uint16_t* __restrict__ xg, uint16_t* __restrict__ xs, int64_t xs_stride) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t r = (int64_t)blockIdx.x * GP_ROWS + warp;
  if (r >= R) return;
  const int per = group / 8;  // lanes of a group
  const int64_t src = row_index ? row_index[r] : r;
  const bool have = src >= 0 && src < T;
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
    if (j >= n) continue;
    if (lane % per == 0) {
      uint32_t o[kSlots / 2];
      split_slots<kSlots, false>(s, o);
      uint16_t* dst = xs + r * xs_stride + j / group * kSlots;
      if constexpr (kSlots == 8)
        *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
      else
        *reinterpret_cast<uint2*>(dst) = make_uint2(o[0], o[1]);
    }
    if (xg && xdtype == 1) {
      *reinterpret_cast<uint4*>(xg + r * n + j) = make_uint4(p[0], p[1], p[2], p[3]);
    } else if (xg) {
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

// ---------------------------------------------------------------- tensor cores
// A persistent CTA per SM takes tiles of 128 outputs x up to 256 rows (an
// expert's rows cut evenly, in multiples of 16, so that a narrow remainder does
// not cost a tile's decoding). The whole depth n is one tile's; per 64 columns
// (a box):
//   warps 8..15  decode the 128 x 64 codes into the A operand in shared memory
//                (thread = output row; K-major, 128-byte swizzle), two sets of four
//                warps on alternate boxes
//   warp 16      x boxes (64 columns x rows) by TMA, the B operand
//   warp 17      tcgen05.mma M=128 x N=rows x K=16, A x B^T into tensor memory:
//                each group into its own accumulator, two in flight
//   warp 18      windows of 16 code words x 128 rows by TMA
//   warps 0..7   per group: acc += coef_d D in packed fp32 pairs, thread = output
//                row, two warps a row set on alternate 32 columns; at the end y
//                (a warp stores 32 consecutive outputs of a row)
// The other term, sum over groups of coef_x xs, is a product of its own of depth
// k: its factors are fp32, so each is cut into bf16 parts and the products of the
// parts stand side by side as correction columns (4 a group for a bf16 y, 8 for
// an fp32 y), which the tensor cores add up like one more group. That takes
// 4 / group more tensor time and halves the epilogue's arithmetic, which is what
// bounds groups of 64 and 32.
// Rows of two neighbouring experts may share an x box: an accumulator column
// depends on its own row of x alone, and only the tile's rows are stored.
constexpr int GT_M = 128, GT_N = 256, GT_K = 64;
constexpr int GT_THREADS = 640;
constexpr int GT_XS = 4, GT_AS = 3, GT_CS = 4;  // ring lengths: x, A, code windows
constexpr int GT_XBYTES = GT_N * GT_K * 2, GT_ABYTES = GT_M * GT_K * 2;
constexpr int GT_WIN = 16, GT_CBYTES = GT_M * GT_WIN * 4;
constexpr int GT_OFF_A = GT_XS * GT_XBYTES;
constexpr int GT_OFF_C = GT_OFF_A + GT_AS * GT_ABYTES;
constexpr int GT_OFF_BAR = GT_OFF_C + GT_CS * GT_CBYTES;
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
  void* y;
  int64_t m, n, R, rw;
  int E, k, planes, ydtype, codes_tma, mtiles;
};
struct GtMaps {
  CUtensorMap x256, x32, s256, s32, codes;
};

struct GtTile {
  int e;        // expert
  int64_t m0;   // first output
  int col0;     // first row of x
  int r1;       // end of the expert's rows
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

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
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
// Bounded wait. A poll suspends the warp in hardware for up to 20 us, so that
// waiting warps take no issue slots from the working ones; the limit on polls
// (a healthy phase completes in microseconds) turns a would-be hang into a
// recorded failure. Kept small: it is inlined at every wait, and the roles'
// loops have to stay in the instruction cache together (with a clock and a
// second loop in it the kernel was 289 KB of code and ran 3 to 4 times slower).
constexpr int kWaitPolls = 100000;
__device__ __forceinline__ bool gt_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int where) {
#pragma unroll 1
  for (int it = 0; it < kWaitPolls; ++it) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(20000u)
        : "memory");
    if (ok) return true;
    if (*abort_flag) return false;
  }
  *abort_flag = where;
  return false;
}

// Tiles of the rows [r0, r1): count, and the width of each.
__device__ __forceinline__ int gt_row_tiles(int r0, int r1, int& width) {
  if (r1 <= r0) {
    width = 0;
    return 0;
  }
  const int span = r1 - r0, nt = (span + GT_N - 1) / GT_N;
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
  u.r1 = off[lo + 1];
  int width;
  gt_row_tiles(off[lo], u.r1, width);
  const int j = (t - first[lo]) / p.mtiles;
  u.m0 = (int64_t)(t - first[lo] - j * p.mtiles) * GT_M;
  u.col0 = off[lo] + j * width;
  u.N = (min(width, u.r1 - u.col0) + 15) & ~15;
  return u;
}

template <int G, bool kCenter>
__global__ void __launch_bounds__(GT_THREADS, 1) gg_tc_kernel(const __grid_constant__ GtMaps tm, const GtParams p) {
  constexpr int kSlots = kCenter ? 8 : 4;       // correction columns of a group
  constexpr int kUnits = G / 32;                // 32-code units of a group
  constexpr int kCorr = GT_K / kSlots;          // groups of a correction box
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sx = smem;
  uint8_t* sa = smem + GT_OFF_A;
  uint8_t* sc = smem + GT_OFF_C;
  uint64_t* xfull = reinterpret_cast<uint64_t*>(smem + GT_OFF_BAR);
  uint64_t* xempty = xfull + GT_XS;
  uint64_t* afull = xempty + GT_XS;
  uint64_t* aempty = afull + GT_AS;
  uint64_t* cfull = aempty + GT_AS;
  uint64_t* cempty = cfull + GT_CS;
  uint64_t* dfull = cempty + GT_CS;
  uint64_t* dempty = dfull + 2;
  uint64_t* done = dempty + 2;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
  int* s_first = reinterpret_cast<int*>(smem + GT_OFF_E);
  int* s_off = s_first + GT_MAX_E + 1;

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform: roles' loops run on uniform registers
  if (tid == 0) {
    for (int i = 0; i < GT_XS; ++i) { mbar_init(&xfull[i], 1); mbar_init(&xempty[i], 1); }
    for (int i = 0; i < GT_AS; ++i) { mbar_init(&afull[i], 4); mbar_init(&aempty[i], 1); }
    for (int i = 0; i < GT_CS; ++i) { mbar_init(&cfull[i], 1); mbar_init(&cempty[i], 8); }
    for (int i = 0; i < 2; ++i) { mbar_init(&dfull[i], 1); mbar_init(&dempty[i], 8); }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm.x256);
    tma_prefetch_desc(&tm.x32);
    if (p.codes_tma) tma_prefetch_desc(&tm.codes);
  }
  if (warp == 19) tmem_alloc(tslot, 512);
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
  const int nbox = (int)((p.n + GT_K - 1) / GT_K);     // boxes of codes
  const int ncor = (p.k + kCorr - 1) / kCorr;          // boxes of correction columns

  if (warp < 8) {
    // ------------------------------------------------------------ epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
    const int half = warp >> 2, sub = (warp & 3) * 32;
    GtRing dr;
    bool ok = true;
    for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      const GtTile u = gt_tile(p, t, s_first, s_off);
      const int64_t i = u.m0 + sub + lane;
      const bool row_ok = i < p.m;
      const float* scale = p.scale + ((int64_t)u.e * p.m + (row_ok ? i : p.m - 1)) * p.k;
      const uint8_t* bits = p.bits + (int64_t)u.e * p.k;
      const bool vec = (p.k & 3) == 0 && (reinterpret_cast<uintptr_t>(p.scale) & 15) == 0;
      uint64_t acc[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) acc[j] = 0ull;
      auto load4 = [&](int c) {
        if (vec) return c < p.k ? *reinterpret_cast<const float4*>(scale + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        return make_float4(c < p.k ? scale[c] : 0.f, c + 1 < p.k ? scale[c + 1] : 0.f,
                           c + 2 < p.k ? scale[c + 2] : 0.f, c + 3 < p.k ? scale[c + 3] : 0.f);
      };
      float4 s4 = {}, sn = load4(0);
      int bnext = bits[0];
      for (int c = 0; c <= p.k; ++c) {  // group k: the correction columns
        float cd = 1.f;
        if (c < p.k) {
          if ((c & 3) == 0) {
            s4 = sn;
            sn = load4(c + 4);
          }
          cd = bnext >= 1 && bnext <= 8 ? coef_d<kCenter>(bnext, s4.x) : 0.f;
          s4 = make_float4(s4.y, s4.z, s4.w, 0.f);
          if (c + 1 < p.k) bnext = bits[c + 1];
        }
        const uint64_t cd2 = gt_pack(cd, cd);
        if (!gt_wait(smem_u32(dfull) + 8 * (dr.slot), dr.phase, abort_flag, 11)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t dcol = tbase + ((uint32_t)sub << 16) + dr.slot * GT_N;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int col = (2 * q + half) * 32;
          if (col < u.N) {
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              uint32_t d[16];
              tmem_ld16(dcol + col + 16 * w, d);
              tc_wait_ld16(d);
#pragma unroll
              for (int v = 0; v < 8; ++v)
                acc[q * 16 + w * 8 + v] =
                    gt_fma2(cd2, ((uint64_t)d[2 * v + 1] << 32) | d[2 * v], acc[q * 16 + w * 8 + v]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&dempty[dr.slot]);
        dr.step(2);
      }
      if (!ok) break;
      using out_t = typename std::conditional<kCenter, float, uint16_t>::type;
      const int cols = row_ok ? min(u.N, u.r1 - u.col0) : 0;
      out_t* yp = static_cast<out_t*>(p.y) + (int64_t)(u.col0 + half * 32) * p.m + i;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int left = cols - (2 * q + half) * 32;
        if (left > 0) {
          out_t* yc = yp;
#pragma unroll
          for (int v = 0; v < 32; ++v) {
            float a, b;
            gt_unpack(acc[q * 16 + v / 2], a, b);
            const float val = v & 1 ? b : a;
            if (v < left) {
              if constexpr (kCenter)
                *yc = val;
              else
                *yc = (uint16_t)pack_bf16(val, 0.f);
            }
            yc += p.m;
          }
        }
        yp += 64 * p.m;
      }
    }
  } else if (warp < 16) {
    // ------------------------------------------------------------ decoding
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    const int row = tid & 127, set = (warp - 8) >> 2;  // the two sets of four warps take alternate boxes
    uint32_t ai = 0;  // boxes of all tiles so far
    uint32_t ci = 0;  // windows taken so far
    bool ok = true;
    const int nwin = (int)((p.rw + GT_WIN - 1) / GT_WIN), rw = (int)p.rw;
    const uint32_t cbase = smem_u32(sc) + row * (GT_WIN * 4), cswz = ((row >> 1) & 3) << 4;
    const uint32_t abase = smem_u32(sa) + row * 128, aswz = (row & 7) << 4;
    for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      const GtTile u = gt_tile(p, t, s_first, s_off);
      const uint8_t* bits = p.bits + (int64_t)u.e * p.k;
      const int64_t i = (int64_t)u.e * p.m + (u.m0 + row < p.m ? u.m0 + row : p.m - 1);
      const uint32_t* crow = p.codes + i * p.rw;
      int wpos = 0, have = 0, freed = 0;  // words and windows of this tile: read, arrived, given back
      const uint32_t cslot = ci;  // ring position of the tile's window 0
      // (a set takes the windows of the boxes it leaves to the other set too, so that no warp gives a
      // window back a second time before every warp has given it back once)
      auto take_windows = [&](int upto) {
#pragma unroll 1
        for (; p.codes_tma && have < upto && ok; ++have, ++ci)
          ok = gt_wait(smem_u32(cfull) + 8 * (ci % GT_CS), (ci / GT_CS) & 1, abort_flag, 20);
      };
      auto free_windows = [&](int upto) {
#pragma unroll 1
        for (; p.codes_tma && freed < upto && ok; ++freed) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&cempty[(cslot + freed) % GT_CS]);
        }
      };
      auto begin_box = [&]() {
        if (ok) ok = gt_wait(smem_u32(aempty) + 8 * (ai % GT_AS), ((ai / GT_AS) & 1) ^ 1, abort_flag, 21);
        return abase + (ai % GT_AS) * GT_ABYTES;
      };
      auto end_box = [&]() {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&afull[ai % GT_AS]);
      };
      auto store16 = [&](uint32_t to, int chunk, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + ((chunk * 16) ^ aswz)), "r"(a), "r"(b),
                     "r"(c), "r"(d)
                     : "memory");
      };
      uint32_t bcache = 0;
#pragma unroll 1
      for (int kb = 0; kb < nbox && ok; ++kb, ++ai) {
        // the widths of the box's two units, and the words before and of them
        int b[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c = (2 * kb + h) / kUnits;
          if ((2 * kb + h) % (32 * kUnits) == 0) bcache = c + lane < p.k ? bits[c + lane] : 0;
          b[h] = __shfl_sync(0xffffffffu, bcache, c & 31);
          if (kUnits > 1 && h == 0) b[1] = b[0];
          if (kUnits > 1) break;
        }
        if (b[0] > 8 || wpos + b[0] > rw) b[0] = 0;  // not a width: nothing of this group counts
        if (b[1] > 8 || wpos + b[0] + b[1] > rw) b[1] = 0;
        const int wend = wpos + b[0] + b[1];
        take_windows((wend + GT_WIN - 1) / GT_WIN);
        if ((kb & 1) == set) {
          uint32_t to = 0;
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            uint32_t o[16];
            switch (b[h]) {
#define GT_CASE(B)                                                                                  \
  case B: {                                                                                         \
    uint32_t w[B];                                                                                  \
    _Pragma("unroll") for (int q = 0; q < B; ++q) {                                                 \
      const uint32_t wi = (uint32_t)(wpos + q);                                                     \
      if (p.codes_tma)                                                                              \
        asm volatile("ld.shared.u32 %0, [%1];"                                                      \
                     : "=r"(w[q])                                                                   \
                     : "r"(cbase + ((cslot + wi / GT_WIN) % GT_CS) * GT_CBYTES +                    \
                           (((wi % GT_WIN) * 4) ^ cswz)));                                          \
      else /* rows that are not 16-byte aligned */                                                  \
        w[q] = __ldg(crow + wi);                                                                    \
    }                                                                                               \
    decode32<B, kCenter>(w, o);                                                                     \
  } break;
              GT_CASE(1) GT_CASE(2) GT_CASE(3) GT_CASE(4) GT_CASE(5) GT_CASE(6) GT_CASE(7) GT_CASE(8)
#undef GT_CASE
              default:
#pragma unroll
                for (int q = 0; q < 16; ++q) o[q] = 0u;
            }
            if (h == 0) to = begin_box();
#pragma unroll
            for (int q = 0; q < 4; ++q) store16(to, h * 4 + q, o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
            wpos += b[h];
          }
          end_box();
        }
        wpos = wend;
        free_windows(wpos / GT_WIN);
      }
      take_windows(nwin);
      free_windows(nwin);
      // the correction columns: coef_x of each group in bf16 parts
      const float* sc_row = p.scale + i * p.k;
      const float* ze_row = p.zero + i * p.k;
#pragma unroll 1
      for (int q = 0; q < ncor && ok; ++q, ++ai) {
        if ((q & 1) != set) continue;
        const uint32_t to = begin_box();
#pragma unroll 1
        for (int v = 0; v < kCorr; v += 8) {  // 8 groups' scales and zeros in flight at a time
          float sv[8], zv[8];
#pragma unroll
          for (int w = 0; w < 8; ++w) {
            const int c = min(q * kCorr + v + w, p.k - 1);
            sv[w] = sc_row[c];
            zv[w] = ze_row[c];
          }
#pragma unroll
          for (int w = 0; w < 8; w += 8 / kSlots) {  // a 16-byte chunk
            uint32_t o[4];
#pragma unroll
            for (int z = 0; z < 8 / kSlots; ++z) {
              const int c = q * kCorr + v + w + z;
              const int b = c < p.k ? bits[c] : 0;
              const float cx = b >= 1 && b <= 8 ? coef_x<kCenter>(b, sv[w + z], zv[w + z]) : 0.f;
              uint32_t part[kSlots / 2];
              split_slots<kSlots, true>(cx, part);
#pragma unroll
              for (int y = 0; y < kSlots / 2; ++y) o[z * (kSlots / 2) + y] = part[y];
            }
            store16(to, (v + w) * kSlots / 8, o[0], o[1], o[2], o[3]);
          }
        }
        end_box();
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 32;");
    if (warp == 16 && lane == 0) {
      // ---------------------------------------------------------- x boxes
      uint32_t xi = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
        const GtTile u = gt_tile(p, t, s_first, s_off);
        const int per = u.N > 128 ? 1 : (u.N > 64 ? 2 : 4);  // boxes of a stage
        for (int kb = 0; kb < nbox + ncor && ok;) {
          const bool cor = kb >= nbox;
          const int k0 = cor ? kb - nbox : kb, nb = min(per, (cor ? nbox + ncor : nbox) - kb);
          for (int pl = cor ? 0 : p.planes - 1; pl >= 0; --pl, ++xi) {
            const uint32_t s = xi % GT_XS;
            if (!gt_wait(smem_u32(xempty) + 8 * (s), ((xi / GT_XS) & 1) ^ 1, abort_flag, 30)) {
              ok = false;
              break;
            }
            const int y0 = (int)(pl * p.R) + u.col0;
            uint8_t* dst = sx + s * GT_XBYTES;
            if (per == 1) {
              mbar_arrive_expect_tx(&xfull[s], GT_XBYTES);
              tma_load_2d(dst, cor ? &tm.s256 : &tm.x256, &xfull[s], k0 * GT_K, y0);
            } else {
              const int nr = (u.N + 31) / 32;
              mbar_arrive_expect_tx(&xfull[s], (uint32_t)(nb * nr * 4096));
              for (int q = 0; q < nb; ++q)
                for (int v = 0; v < nr; ++v)
                  tma_load_2d(dst + q * (GT_XBYTES / per) + v * 4096, cor ? &tm.s32 : &tm.x32, &xfull[s],
                              (k0 + q) * GT_K, y0 + 32 * v);
            }
          }
          kb += nb;
        }
      }
      for (uint32_t j = xi > GT_XS ? xi - GT_XS : 0; j < xi; ++j) mbar_drain(&xfull[j % GT_XS], (j / GT_XS) & 1);
    } else if (warp == 17) {
      // ---------------------------------------------------------- matrix products
      // The whole warp runs the loop (uniform control and registers); one elected
      // lane issues. What stands between two products is kept to a few instructions.
      const bool lead = elect_one();
      constexpr uint64_t kDesc = ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
                                 ((uint64_t)2 << 61);  // K-major, 128-byte swizzle (sdesc_sw128)
      const uint32_t a0 = smem_u32(sa) >> 4, x0 = smem_u32(sx) >> 4;
      GtRing xr, ar, dr;
      bool ok = true;
      for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
        const GtTile u = gt_tile(p, t, s_first, s_off);
        const int per = u.N > 128 ? 1 : (u.N > 64 ? 2 : 4);
        const uint32_t xstep = (GT_XBYTES / 16) / per;
        const uint32_t idesc = idesc_bf16_f32(GT_M, 16, false, false) + ((uint32_t)(u.N / 8 - 2) << 17);
        int sub = 0;
        // kSteps products of 16 columns from every plane; fresh: the first of an accumulator
        auto part = [&](auto steps, uint32_t koff, int planes, uint32_t fresh, bool wait_x, bool free_x) {
          constexpr int kSteps = decltype(steps)::value;
          const uint64_t ad = kDesc + (a0 + ar.slot * (GT_ABYTES / 16) + koff);
          const uint32_t d = tbase + dr.slot * GT_N;
          uint32_t slot = xr.slot, phase = xr.phase, acc = fresh ^ 1u;
#pragma unroll 1
          for (int q = 0; q < planes; ++q) {
            if (wait_x) {
              if (!gt_wait(smem_u32(xfull) + 8 * slot, phase, abort_flag, 42)) return false;
              tc_fence_after();
            }
            const uint64_t bd = kDesc + (x0 + slot * (GT_XBYTES / 16) + sub * xstep + koff);
            if (lead) {
#pragma unroll
              for (int k16 = 0; k16 < kSteps; ++k16) tc_mma_bf16(d, ad + 2 * k16, bd + 2 * k16, idesc, k16 ? 1u : acc);
              if (free_x) tc_commit(&xempty[slot]);
            }
            acc = 1u;
            if (++slot == GT_XS) {
              slot = 0;
              phase ^= 1;
            }
          }
          if (free_x) {
            xr.slot = slot;
            xr.phase = phase;
          }
          return true;
        };
        // boxes [0, n) of codes (kParts parts each, begins and ends of groups known) or of correction columns
        auto boxes = [&](auto parts, auto per_group, int n, int planes, bool odd) {
          constexpr int kParts = decltype(parts)::value, kPer = decltype(per_group)::value;
#pragma unroll 1
          for (int kb = 0; kb < n; ++kb) {
            if (!gt_wait(smem_u32(afull) + 8 * ar.slot, ar.phase, abort_flag, 40)) return false;
            const bool last = kb == n - 1, last_sub = sub == per - 1 || last;
            const bool begins = kPer == 0 ? kb == 0 : (kPer == 1 || (kb & 1) == 0);
            const bool ends = kPer == 0 ? last : (kPer == 1 || (kb & 1) == 1);
#pragma unroll
            for (int h = 0; h < kParts; ++h) {
              const bool only = kParts == 1 || (last && odd);
              if (h == 1 && only) break;
              if (begins && !gt_wait(smem_u32(dempty) + 8 * dr.slot, dr.phase ^ 1, abort_flag, 41)) return false;
              tc_fence_after();
              if (!part(std::integral_constant<int, 4 / kParts>{}, (uint32_t)h * 4, planes, begins,
                        sub == 0 && h == 0, last_sub && (h == 1 || only)))
                return false;
              if (ends) {
                if (lead) tc_commit(&dfull[dr.slot]);
                dr.step(2);
              }
            }
            sub = last_sub ? 0 : sub + 1;
            if (lead) tc_commit(&aempty[ar.slot]);
            ar.step(GT_AS);
          }
          return true;
        };
        ok = boxes(std::integral_constant<int, G == 32 ? 2 : 1>{}, std::integral_constant<int, G == 128 ? 2 : 1>{}, nbox,
                   p.planes, (p.k & 1) != 0) &&
             boxes(std::integral_constant<int, 1>{}, std::integral_constant<int, 0>{}, ncor, 1, false);
      }
      // every issued product completes before tensor memory can be freed, also after an abort
      if (lead) {
        tc_commit(done);
        mbar_drain(done, 0);
      }
    } else if (warp == 18 && lane == 0 && p.codes_tma) {
      // ---------------------------------------------------------- code windows
      uint32_t ci = 0;
      bool ok = true;
      const int nwin = (int)((p.rw + GT_WIN - 1) / GT_WIN);
      for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
        const GtTile u = gt_tile(p, t, s_first, s_off);
        const int y0 = (int)(u.e * p.m + u.m0);
        for (int w = 0; w < nwin; ++w, ++ci) {
          const uint32_t s = ci % GT_CS;
          if (!gt_wait(smem_u32(cempty) + 8 * (s), ((ci / GT_CS) & 1) ^ 1, abort_flag, 50)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&cfull[s], GT_CBYTES);
          tma_load_2d(sc + s * GT_CBYTES, &tm.codes, &cfull[s], w * GT_WIN, y0);
        }
      }
      for (uint32_t j = ci > GT_CS ? ci - GT_CS : 0; j < ci; ++j) mbar_drain(&cfull[j % GT_CS], (j / GT_CS) & 1);
    }
    __syncwarp();
  }
  __syncthreads();
  if (tid == 0 && *abort_flag) record_failure(&g_async_status, kStatusTimeout, *abort_flag);
  if (warp == 19) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// ---------------------------------------------------------------- host side
struct GroupedPlan {
  int planes;         // bf16 planes copied in grouped order (0: x is read as it is)
  int64_t xs_stride;  // correction columns of a row, padded to 16 bytes
  size_t off_xg, bytes;
};

// For an fp32 y the correction columns are 8 a group; the plan has room for either.
static GroupedPlan grouped_plan(int64_t n, int group, int xdtype, bool gathered, int64_t R) {
  GroupedPlan g{};
  g.xs_stride = n / group * 8;
  g.planes = xdtype == 0 ? 3 : (gathered ? 1 : 0);
  g.off_xg = ((size_t)R * g.xs_stride * 2 + 255) & ~size_t(255);
  g.bytes = g.off_xg + (((size_t)g.planes * R * n * 2 + 255) & ~size_t(255));
  return g;
}

size_t grouped_workspace_bytes(int64_t E, int64_t m, int64_t n, int group, int xdtype, bool gathered, int64_t R) {
  return grouped_plan(n, group, xdtype, gathered, R).bytes;
}

template <int G, bool kCenter>
static cudaError_t launch_gt(const GtMaps& tm, const GtParams& p, int num_sms, cudaStream_t s) {
  static std::atomic<uint64_t> attr{0};
  uint64_t bit = 0;
  if (attr_pending(attr, bit)) {
    const cudaError_t e =
        cudaFuncSetAttribute(gg_tc_kernel<G, kCenter>, cudaFuncAttributeMaxDynamicSharedMemorySize, GT_SMEM);
    if (e != cudaSuccess) return e;
    attr.fetch_or(bit);
  }
  gg_tc_kernel<G, kCenter><<<num_sms, GT_THREADS, GT_SMEM, s>>>(tm, p);
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_grouped(const uint32_t* codes, const uint8_t* bits, const float* scale, const float* zero,
                           int64_t E, int64_t m, int64_t n, int group, int avg_bits, const void* x, int xdtype,
                           int64_t T, const int32_t* row_index, const int32_t* offsets, int64_t R, void* y,
                           int ydtype, uint8_t* ws, int num_sms, cudaStream_t s) {
  const GroupedPlan g = grouped_plan(n, group, xdtype, row_index != nullptr, R);
  uint16_t* xs = reinterpret_cast<uint16_t*>(ws);
  uint16_t* xg = g.planes ? reinterpret_cast<uint16_t*>(ws + g.off_xg) : nullptr;
  const int k = (int)(n / group);
  const unsigned blocks = (unsigned)((R + GP_ROWS - 1) / GP_ROWS);
  const int slots = ydtype == 0 ? 8 : 4;
  if (slots == 8)
    gg_prep_kernel<8><<<blocks, GP_ROWS * 32, 0, s>>>(x, xdtype, T, row_index, R, n, group, xg, xs, g.xs_stride);
  else
    gg_prep_kernel<4><<<blocks, GP_ROWS * 32, 0, s>>>(x, xdtype, T, row_index, R, n, group, xg, xs, g.xs_stride);
  count_launches(1);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  GtParams p{};
  p.codes = codes; p.bits = bits; p.scale = scale; p.zero = zero; p.offsets = offsets; p.y = y;
  p.m = m; p.n = n; p.R = R; p.rw = n * avg_bits / 32;
  p.E = (int)E; p.k = k; p.planes = g.planes ? g.planes : 1; p.ydtype = ydtype;
  p.mtiles = (int)((m + GT_M - 1) / GT_M);
  p.codes_tma = p.rw % 4 == 0;
  GtMaps tm;
  const void* xb = xg ? static_cast<const void*>(xg) : x;
  const uint64_t rows = xg ? (uint64_t)g.planes * R : (uint64_t)T;
  if (!make_tmap_bf16(&tm.x256, xb, (uint64_t)n, rows, GT_K, GT_N) ||
      !make_tmap_bf16(&tm.x32, xb, (uint64_t)n, rows, GT_K, 32) ||
      !make_tmap_2byte_strided(&tm.s256, xs, (uint64_t)k * slots, (uint64_t)R, (uint64_t)g.xs_stride * 2, GT_K, GT_N) ||
      !make_tmap_2byte_strided(&tm.s32, xs, (uint64_t)k * slots, (uint64_t)R, (uint64_t)g.xs_stride * 2, GT_K, 32))
    return cudaErrorInvalidValue;
  if (p.codes_tma && !make_tmap_u32_sw64(&tm.codes, codes, (uint64_t)p.rw, (uint64_t)(E * m), GT_WIN, GT_M))
    return cudaErrorInvalidValue;
#define SLIM_GT(G) (ydtype == 0 ? launch_gt<G, true>(tm, p, num_sms, s) : launch_gt<G, false>(tm, p, num_sms, s))
  return group == 32 ? SLIM_GT(32) : (group == 64 ? SLIM_GT(64) : SLIM_GT(128));
#undef SLIM_GT
}

}  // namespace slim
