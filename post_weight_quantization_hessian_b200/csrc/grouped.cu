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
#include <cstdlib>
#include <type_traits>
#include "common.cuh"
#include "decode.cuh"
#include "tmap.h"

namespace slim {

// Where the asynchronous kernels of the current device record their first failure
// (where << 32 | code, 0: none), read and cleared by slim_async_status in one
// exchange: a failure that another stream records meanwhile is kept for the next query.
__device__ unsigned long long g_async_status;

__device__ __forceinline__ void record_async(int code, int where) {
  atomicCAS(&g_async_status, 0ull, (unsigned long long)(uint32_t)where << 32 | (uint32_t)code);
}
__global__ void take_status_kernel(unsigned long long* out) { *out = atomicExch(&g_async_status, 0ull); }

// tmp: 8 bytes of device memory. Waits for the stream.
cudaError_t take_async_status(int* code, int* where, uint8_t* tmp, cudaStream_t s) {
  unsigned long long v = 0;
  take_status_kernel<<<1, 1, 0, s>>>(reinterpret_cast<unsigned long long*>(tmp));
  count_launches(1);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = cudaMemcpyAsync(&v, tmp, sizeof(v), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  *code = (int)(uint32_t)v;
  *where = (int)(uint32_t)(v >> 32);
  return e;
}

// ---------------------------------------------------------------- preparation
// Sums of x over each column group, as the bf16 parts that the correction
// columns of the tensor-core kernel take (below), and where that kernel cannot
// read x as it is (gathered rows, fp32), the rows as bf16 in grouped order: fp32
// as three planes x1 + x2 + x3 that hold all 24 bits. A warp takes 512 columns of
// a row, with 16-byte loads and stores; bound by the bytes of x (read, and
// written if copied).
constexpr int GP_ROWS = 8, GP_COLS = 512;

// A value of y: fp32, or rounded once to bf16.
template <typename out_t>
__device__ __forceinline__ out_t as_out(float v) {
  if constexpr (std::is_same<out_t, float>::value)
    return v;
  else
    return (out_t)pack_bf16(v, 0.f);
}
// v = p1 + p2 + p3, each a bf16 value (8 + 8 + 8 bits).
__device__ __forceinline__ void split3(float v, float& p1, float& p2, float& p3) {
  p1 = __uint_as_float(pack_bf16(v, 0.f) << 16);
  p2 = __uint_as_float(pack_bf16(v - p1, 0.f) << 16);
  p3 = __uint_as_float(pack_bf16(v - p1 - p2, 0.f) << 16);
}
// Correction columns of one group: eight products of the parts of a and b side by
// side (a1 b1, a1 b2, a2 b1, a2 b2, a1 b3, a3 b1, a2 b3, a3 b2), all but a3 b3: about
// 2^-32 of a b is left out. (The first four alone leave out 2^-17, which a bf16
// result shows: 2 percent of its values rounded to the wrong side, 6 for x of mean 1.)
constexpr int kSlots = 8;
template <bool kFirst>
__device__ __forceinline__ void split_slots(float v, uint32_t (&o)[kSlots / 2]) {
  float p1, p2, p3;
  split3(v, p1, p2, p3);
  if (kFirst) {
    o[0] = pack_bf16(p1, p1);
    o[1] = pack_bf16(p2, p2);
    o[2] = pack_bf16(p1, p3);
    o[3] = pack_bf16(p2, p3);
  } else {
    o[0] = pack_bf16(p1, p2);
    o[1] = pack_bf16(p1, p2);
    o[2] = pack_bf16(p3, p1);
    o[3] = pack_bf16(p3, p2);
  }
}

__global__ void __launch_bounds__(GP_ROWS * 32)
gg_prep_kernel(const void* __restrict__ x, int xdtype, int64_t T, const int32_t* __restrict__ row_index, int64_t R,
               int64_t n, int group, uint16_t* __restrict__ xg, uint16_t* __restrict__ xs, int64_t xs_stride) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t r = (int64_t)blockIdx.x * GP_ROWS + warp;
  if (r >= R) return;
  const int per = group / 8;  // lanes of a group
  const int64_t src = row_index ? row_index[r] : r;
  const bool have = src >= 0 && src < T;
  const int64_t j0 = (int64_t)blockIdx.y * GP_COLS;
#pragma unroll
  for (int step = 0; step < GP_COLS / 256; ++step) {
    const int64_t j = j0 + step * 256 + lane * 8;
    if (j - lane * 8 >= n) break;
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
    if (xs && lane % per == 0) {
      uint32_t o[kSlots / 2];
      split_slots<false>(s, o);
      uint16_t* dst = xs + r * xs_stride + (uint32_t)j / (uint32_t)group * kSlots;
      *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
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

// ---------------------------------------------------------------- many rows
// Experts with more than kFewRows rows: their codes are decoded once into bf16
// tiles in the workspace (gd_kernel), and a tensor-core kernel (gg_tc_kernel)
// multiplies the tiles with x, in passes over the outputs, and where one tile of
// outputs of every expert is too much over the experts, that bound the
// workspace (kTileBytes). (Passes whose tiles stay in L2, 64 MB, cost more in their
// last waves than they saved: a third more time on 8192 rows over eight 11008 x 4096
// experts.)
// (A kernel that decoded each tile inside the product loop was built first: 265 us
// on 4096 rows of a 4096 x 4096 layer where the two take 151, bound by the decoding
// warps and the barriers between the roles, a wait of 150 cycles each; every 256
// rows decoded the layer again.)
constexpr int GT_M = 128, GT_N = 256, GT_K = 64;
constexpr int GT_MAX_E = 1024;
constexpr int kCorr = GT_K / kSlots;  // groups of a box of correction columns
constexpr int GT_ABYTES = GT_M * GT_K * 2, GT_XBYTES = GT_N * GT_K * 2;
constexpr int kWaitPolls = 100000;  // of a bounded wait: about 2 s

struct GtParams {
  const uint32_t* codes;
  const uint8_t* bits;
  const float* scale;
  const float* zero;
  const int32_t* offsets;
  uint8_t* tiles;  // [slot of the pass][output tile of the pass][box] of 16 KB
  void* y;
  int64_t m, n, R, rw;
  int E, k, planes, few_rows, max_slots;
  int acc_polls;   // limit of the epilogue's wait for an accumulator (normally kWaitPolls)
  int mt0, mtn;    // output tiles of this pass: first, count
  int slot0, slots;  // its slots: first, count at most
};
struct GtMaps {
  CUtensorMap x256, x32, s256, s32;
};

__device__ __forceinline__ int gt_clamp(int v, int64_t R) { return max(0, min(v, (int)R)); }

// The slots of the experts with more than few_rows rows, in order: s_expert[slot].
// At most max_slots of them, which offsets that do not descend never exceed; returns
// how many the pass takes, from slot0 on. One warp.
__device__ __forceinline__ int gt_slots(const GtParams& p, int lane, int* s_expert) {
  int run = 0;
  for (int e0 = 0; e0 < p.E; e0 += 32) {
    const int e = e0 + lane;
    const bool many =
        e < p.E && gt_clamp(p.offsets[e + 1], p.R) - gt_clamp(p.offsets[e], p.R) > p.few_rows;
    const unsigned mask = __ballot_sync(0xffffffffu, many);
    if (many) s_expert[run + __popc(mask & ((1u << lane) - 1))] = e;
    run += __popc(mask);
  }
  return max(0, min(min(run, p.max_slots) - p.slot0, p.slots));
}

// ---------------------------------------------------------------- decoding
// One block: 128 outputs x up to 4 boxes of 64 columns of one slot. A thread
// takes 8 codes (b bytes of the row's stream) and writes the 16 bytes of their
// bf16 values where the product's shared-memory layout wants them (K-major, 128-
// byte swizzle), so that a warp writes 512 consecutive bytes and the product
// loads a whole tile with one bulk copy. Behind the boxes of codes come those of
// the correction columns. Bound by the bytes written (2 a weight: 13 us for a 4096 x
// 4096 layer, 196 us for eight of 11008 x 4096, 4.1 TB/s) and by the latency of the
// loads of codes and zeros where there are few blocks.
constexpr int GD_THREADS = 256, GD_BOXES = 4;

template <int B>
__device__ __forceinline__ uint4 decode8(uint32_t lo, uint32_t hi, uint32_t shift) {
  uint32_t w[(B * 8 + 31) / 32], o[4];
  w[0] = lo;
  if constexpr (B > 4) w[1] = hi;
  decode_codes<B, 8>(w, shift, o);
  return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int G>
__global__ void __launch_bounds__(GD_THREADS) gd_kernel(const GtParams p) {
  constexpr int kUnits = G / 32;
  __shared__ int s_expert[GT_MAX_E];
  __shared__ int s_count, s_before;
  __shared__ uint32_t s_width[GD_BOXES * 2];  // first word << 4 | width, of each 32-column unit
  constexpr int kGroups = GD_BOXES * 2 / kUnits;
  __shared__ uint32_t s_shift[kGroups][GT_M];  // what is added to the codes
  const int tid = threadIdx.x, lane = tid & 31, slot = blockIdx.z;
  if (tid == 0) s_before = 0;
  if (tid < 32) {
    const int c = gt_slots(p, lane, s_expert);
    if (lane == 0) s_count = c;
  }
  __syncthreads();
  if (slot >= s_count) return;
  const int e = s_expert[p.slot0 + slot], nbox = (int)((p.n + GT_K - 1) / GT_K), ncor = (p.k + kCorr - 1) / kCorr;
  const int kb0 = blockIdx.x * GD_BOXES, kb1 = min(kb0 + GD_BOXES, nbox + ncor);
  const uint8_t* bits = p.bits + (int64_t)e * p.k;
  const int64_t m0 = (int64_t)(p.mt0 + blockIdx.y) * GT_M;
  uint8_t* out = p.tiles + ((int64_t)slot * p.mtn + blockIdx.y) * (nbox + ncor) * GT_ABYTES;
  // widths before the block's boxes, then the block's own; its zeros are on the way meanwhile
  int before = 0;
  const int c0 = kb0 * 2 / kUnits;
  constexpr int kZeros = kGroups * GT_M / GD_THREADS;
  float zeros[kZeros];
#pragma unroll
  for (int z = 0; z < kZeros; ++z) {
    const int v = z * GD_THREADS + tid, c = min(c0 + v % kGroups, p.k - 1);
    zeros[z] = __ldg(p.zero + ((int64_t)e * p.m + min(m0 + v / kGroups, p.m - 1)) * p.k + c);
  }
  for (int c = tid; c < min(c0, p.k); c += GD_THREADS) before += bits[c] <= 8 ? bits[c] : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
  if (lane == 0) atomicAdd(&s_before, before);  // (integers: the order does not matter)
  __syncthreads();
  if (tid < 32) {  // lane = unit of the block, which starts with a group (a multiple of 256 columns)
    const int unit = kb0 * 2 + lane, c = unit / kUnits;
    int b = c < p.k && lane < GD_BOXES * 2 ? bits[c] : 0;
    if (b > 8) b = 0;
    int incl = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const int first = s_before * kUnits + incl - b;
    // widths that do not fill a row: nothing outside it is read
    if (lane < GD_BOXES * 2) s_width[lane] = first + b > p.rw ? 0u : (uint32_t)first << 4 | (uint32_t)b;
  }
  __syncthreads();
#pragma unroll
  for (int z = 0; z < kZeros; ++z) {
    const int v = z * GD_THREADS + tid, c = v % kGroups;
    s_shift[c][v / kGroups] = code_shift(s_width[c * kUnits] & 15, zeros[z]);
  }
  __syncthreads();
  const int chunk = tid & 7, h = chunk >> 2;
  for (int kb = kb0; kb < kb1; ++kb) {
    const bool cor = kb >= nbox;
    uint8_t* tile = out + (int64_t)kb * GT_ABYTES;
    const uint32_t en = s_width[(kb - kb0) * 2 + h], b = en & 15, first = en >> 4;
    const int group = ((kb - kb0) * 2 + h) / kUnits;  // of the block's
#pragma unroll 4
    for (int row = tid >> 3; row < GT_M; row += GD_THREADS / 8) {
      const int64_t i = (int64_t)e * p.m + min(m0 + row, p.m - 1);
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (!cor) {
        const uint32_t bit = (chunk & 3) * 8 * b, sh = bit & 31;
        const uint32_t* w = p.codes + i * p.rw + first + (bit >> 5);
        const uint32_t shift = s_shift[group][row];
        uint32_t lo = 0, hi = 0;
        if (b) {  // 8 b bits from bit `sh` on: never past the unit's b words
          const uint32_t w0 = __ldg(w), w1 = sh + 8 * b > 32 ? __ldg(w + 1) : 0u;
          lo = __funnelshift_r(w0, w1, sh);
          if (b > 4) hi = sh + 8 * b > 64 ? __funnelshift_r(w1, __ldg(w + 2), sh) : w1 >> sh;
        }
        switch (b) {
          case 1: v = decode8<1>(lo, hi, shift); break;
          case 2: v = decode8<2>(lo, hi, shift); break;
          case 3: v = decode8<3>(lo, hi, shift); break;
          case 4: v = decode8<4>(lo, hi, shift); break;
          case 5: v = decode8<5>(lo, hi, shift); break;
          case 6: v = decode8<6>(lo, hi, shift); break;
          case 7: v = decode8<7>(lo, hi, shift); break;
          case 8: v = decode8<8>(lo, hi, shift); break;
          default: break;
        }
      } else {
        const int c = (kb - nbox) * kCorr + chunk, bc = c < p.k ? bits[c] : 0;
        float cx = 0.f;
        if (bc >= 1 && bc <= 8) {
          const float z = p.zero[i * p.k + c];
          cx = coef_x(bc, p.scale[i * p.k + c], z, code_shift(bc, z));
        }
        uint32_t o[4];
        split_slots<true>(cx, o);
        v = make_uint4(o[0], o[1], o[2], o[3]);
      }
      *reinterpret_cast<uint4*>(tile + row * 128 + ((chunk ^ (row & 7)) << 4)) = v;
    }
  }
}

// ---------------------------------------------------------------- product
// A persistent CTA per SM takes tiles of 128 outputs x up to 256 rows (an
// expert's rows cut evenly, in multiples of 16). The whole depth is one tile's;
// per box of 64 columns:
//   warp 8       the decoded 128 x 64 tile (one bulk copy) and the x box (TMA)
//   warp 9       tcgen05.mma M=128 x N=rows x K=16, A x B^T into tensor memory:
//                each group into its own accumulator, two in flight
//   warp 10      the gate: arrives on a box's barrier, beside the copies, once the
//                accumulator that the box starts is free. So the issuing warp has
//                one wait a box (a wait is 150 cycles even when nothing is left
//                to wait for; a box's products take 512 at 256 rows)
//   warps 0..7   per group: acc += coef_d D in packed fp32 pairs, thread = output,
//                two warps an output set on alternate 32 rows; at the end y (a
//                warp stores 32 consecutive outputs of a row)
// The other term, sum over groups of coef_x xs, is a product of its own of depth
// k: its factors are fp32, so each is cut into bf16 parts and the products of the
// parts stand side by side as correction columns, 8 a group, which the tensor
// cores add up like one more group. That takes 8 / group more tensor time and
// halves the epilogue's arithmetic, which is what bounds groups of 64 and 32.
// Rows of two neighbouring experts may share an x box: an accumulator column
// depends on its own row of x alone, and only the tile's rows are stored.
// 138 us on 4096 rows of a 4096 x 4096 layer at groups of 128 (996 TFLOP/s), 1100 us
// on 8192 rows over eight 11008 x 4096 experts at groups of 64 (672): what bounds it is
// the chain of an accumulator's hand-over (commit, wait, loads and additions,
// wait), about 1000 cycles a group besides the 256 to 1024 of its products.
constexpr int GT_THREADS = 384;
constexpr int GT_MAX_STAGES = 8;  // of a ring of 192 KB: 4, 6 or 8 for tiles of 256, 128 or 64 rows
constexpr int GT_OFF_BAR = 4 * (GT_ABYTES + GT_XBYTES);
constexpr int GT_OFF_E = GT_OFF_BAR + 256;
constexpr int GT_SMEM = GT_OFF_E + (2 * GT_MAX_E + 1) * 4 + 1024;  // + alignment
static_assert(GT_SMEM <= 227 * 1024, "shared memory of a CTA");

struct GtTile {
  int e, slot;  // expert and its slot
  int mt;       // output tile of the pass
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
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// Bounded wait. A poll suspends the warp in hardware for up to 20 us, so that
// waiting warps take no issue slots from the working ones; the limit on polls
// (a healthy phase completes in microseconds) turns a would-be hang into a
// recorded failure. (%globaltimer is not read here: that costs more than a phase.)
__device__ __forceinline__ bool gt_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int where,
                                        int polls = kWaitPolls) {
#pragma unroll 1
  for (int it = 0; it < polls; ++it) {
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

// Tiles of at most `most` of the rows [r0, r1): count, and the width of each.
__device__ __forceinline__ int gt_row_tiles(int r0, int r1, int most, int& width) {
  const int span = r1 - r0, nt = (span + most - 1) / most;
  width = nt ? ((span + nt - 1) / nt + 15) & ~15 : 0;
  return nt;
}

// first[s]: the row tiles of the slots before s, times the output tiles of the pass.
__device__ __forceinline__ GtTile gt_tile(const GtParams& p, int t, int slots, int most, const int* first,
                                          const int* expert) {
  int lo = 0, hi = slots;  // the last slot whose first tile is <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= t) lo = mid; else hi = mid;
  }
  GtTile u;
  u.slot = lo;
  u.e = expert[lo];
  const int r0 = gt_clamp(p.offsets[u.e], p.R);
  u.r1 = gt_clamp(p.offsets[u.e + 1], p.R);
  int width;
  gt_row_tiles(r0, u.r1, most, width);
  const int j = (t - first[lo]) / p.mtn;
  u.mt = t - first[lo] - j * p.mtn;
  u.col0 = r0 + j * width;
  u.N = (min(width, u.r1 - u.col0) + 15) & ~15;
  return u;
}

template <int G, typename out_t>
__global__ void __launch_bounds__(GT_THREADS, 1) gg_tc_kernel(const __grid_constant__ GtMaps tm, const GtParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + GT_OFF_BAR);
  uint64_t* empty = full + GT_MAX_STAGES;
  uint64_t* dfull = empty + GT_MAX_STAGES;
  uint64_t* dempty = dfull + 2;
  uint64_t* done = dempty + 2;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
  int* s_slots = reinterpret_cast<int*>(tslot + 2);
  volatile uint32_t* s_issued = tslot + 4;   // stages that the copies filled, and that the gate arrived on,
  volatile uint32_t* s_arrived = tslot + 5;  // in all, when their loops ended
  int* s_first = reinterpret_cast<int*>(smem + GT_OFF_E);
  int* s_expert = s_first + GT_MAX_E + 1;

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform: the roles' loops run on uniform registers
  if (tid == 0) {
    for (int i = 0; i < GT_MAX_STAGES; ++i) { mbar_init(&full[i], 2); mbar_init(&empty[i], 1); }
    for (int i = 0; i < 2; ++i) { mbar_init(&dfull[i], 1); mbar_init(&dempty[i], 8); }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm.x256);
    tma_prefetch_desc(&tm.x32);
  }
  if (warp == 11) tmem_alloc(tslot, 512);
  if (warp == 0) {  // slots and the tiles before each
    const int slots = gt_slots(p, lane, s_expert);
    __syncwarp();
    // 256 rows a tile, fewer while the tiles would leave SMs idle: a tile's time hardly falls below 64
    int run = 0, width, most = 2 * GT_N;
    do {
      most /= 2;
      run = 0;
      for (int q0 = 0; q0 < slots; q0 += 32) {
        const int q = q0 + lane;
        int v = 0;
        if (q < slots) {
          const int e = s_expert[p.slot0 + q];
          v = gt_row_tiles(gt_clamp(p.offsets[e], p.R), gt_clamp(p.offsets[e + 1], p.R), most, width) * p.mtn;
        }
        int incl = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int u = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += u;
        }
        if (q < slots) s_first[q] = run + incl - v;
        run += __shfl_sync(0xffffffffu, incl, 31);
      }
    } while (most > 64 && run * 2 <= (int)gridDim.x);
    if (lane == 0) {
      s_first[slots] = run;
      s_slots[0] = slots;
      s_slots[1] = most;
    }
  }
  __syncthreads();
  tc_fence_after();
  s_expert += p.slot0;
  const uint32_t tbase = *tslot;
  const int slots = s_slots[0], most = s_slots[1], tiles = s_first[slots];
  const uint32_t stages = most == 256 ? 4 : (most == 128 ? 6 : 8), stage = GT_ABYTES + most * 128;
  const int nbox = (int)((p.n + GT_K - 1) / GT_K);     // boxes of codes
  const int ncor = (p.k + kCorr - 1) / kCorr;          // boxes of correction columns

  if (warp < 8) {
    // ------------------------------------------------------------ epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int half = warp >> 2, sub = (warp & 3) * 32;
    GtRing dr;
    bool ok = true;
    for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      const GtTile u = gt_tile(p, t, slots, most, s_first, s_expert);
      const int64_t i = (int64_t)(p.mt0 + u.mt) * GT_M + sub + lane;
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
          cd = bnext >= 1 && bnext <= 8 ? coef_d(bnext, s4.x) : 0.f;
          s4 = make_float4(s4.y, s4.z, s4.w, 0.f);
          if (c + 1 < p.k) bnext = bits[c + 1];
        }
        const uint64_t cd2 = gt_pack(cd, cd);
        if (!gt_wait(smem_u32(dfull) + 8 * dr.slot, dr.phase, abort_flag, 11, p.acc_polls)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t dcol = tbase + ((uint32_t)sub << 16) + dr.slot * GT_N;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int col = (2 * q + half) * 32;
          if (col < u.N) {
            uint32_t d[32];
            tmem_ld32(dcol + col, d);
            tc_wait_ld();
#pragma unroll
            for (int v = 0; v < 16; ++v)
              acc[q * 16 + v] = gt_fma2(cd2, ((uint64_t)d[2 * v + 1] << 32) | d[2 * v], acc[q * 16 + v]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&dempty[dr.slot]);
        dr.step(2);
      }
      if (!ok) break;
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
              *yc = as_out<out_t>(val);
            }
            yc += p.m;
          }
        }
        yp += 64 * p.m;
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 8 && lane == 0) {
      // ---------------------------------------------------------- copies
      GtRing r;
      uint32_t issued = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
        const GtTile u = gt_tile(p, t, slots, most, s_first, s_expert);
        const uint8_t* at = p.tiles + ((int64_t)u.slot * p.mtn + u.mt) * (nbox + ncor) * GT_ABYTES;
        const int nr = (u.N + 31) / 32;
        const uint32_t bytes = (u.N > 128 ? GT_XBYTES : nr * 4096) + GT_ABYTES;
        for (int kb = 0; kb < nbox + ncor && ok; ++kb) {
          const bool cor = kb >= nbox;
          // fp32 x: a stage for every plane, the small parts first, each with the decoded tile
          for (int pl = cor ? 0 : p.planes - 1; pl >= 0; --pl, ++issued) {
            if (!gt_wait(smem_u32(empty) + 8 * r.slot, r.phase ^ 1, abort_flag, 30)) {
              ok = false;
              break;
            }
            uint8_t* dst = smem + r.slot * stage;
            uint64_t* bar = &full[r.slot];
            mbar_arrive_expect_tx(bar, bytes);
            bulk_load(dst, at + (int64_t)kb * GT_ABYTES, GT_ABYTES, bar);
            const int x0 = (cor ? kb - nbox : kb) * GT_K, y0 = (int)(pl * p.R) + u.col0;
            dst += GT_ABYTES;
            if (u.N > 128) {
              tma_load_2d(dst, cor ? &tm.s256 : &tm.x256, bar, x0, y0);
            } else {
              for (int v = 0; v < nr; ++v) tma_load_2d(dst + v * 4096, cor ? &tm.s32 : &tm.x32, bar, x0, y0 + 32 * v);
            }
            r.step(stages);
          }
        }
      }
      *s_issued = issued;
    } else if (warp == 10 && lane == 0) {
      // ---------------------------------------------------------- gate
      GtRing r, dr;
      uint32_t arrived = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
        for (int kb = 0; kb < nbox + ncor && ok; ++kb) {
          const bool cor = kb >= nbox;
          // accumulators that the box starts (groups of 32: both of its halves)
          const int starts = cor ? kb == nbox : (G == 128 ? (kb & 1) == 0 : (G == 64 ? 1 : min(2, p.k - 2 * kb)));
          const int planes = cor ? 1 : p.planes;
          for (int q = 0; q < planes && ok; ++q) {
            // its arrival has to fall into the stage's current use
            ok = gt_wait(smem_u32(empty) + 8 * r.slot, r.phase ^ 1, abort_flag, 31);
            if (q == 0 && G != 32)
              for (int v = 0; v < starts && ok; ++v) {
                ok = gt_wait(smem_u32(dempty) + 8 * dr.slot, dr.phase ^ 1, abort_flag, 32);
                dr.step(2);
              }
            if (ok) {
              mbar_arrive(&full[r.slot]);
              ++arrived;
            }
            r.step(stages);
          }
        }
      }
      *s_arrived = arrived;
    } else if (warp == 9) {
      // ---------------------------------------------------------- matrix products
      // The whole warp runs the loop (uniform control and registers); one elected
      // lane issues. What stands between two products is kept to a few instructions.
      const bool lead = elect_one();
      constexpr uint64_t kDesc = ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
                                 ((uint64_t)2 << 61);  // K-major, 128-byte swizzle (sdesc_sw128)
      const uint32_t a0 = smem_u32(smem) >> 4;
      GtRing r, dr;
      bool ok = true;
      for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
        const GtTile u = gt_tile(p, t, slots, most, s_first, s_expert);
        const uint32_t idesc = idesc_bf16_f32(GT_M, 16, false, false) + ((uint32_t)(u.N / 8 - 2) << 17);
        // kPer: boxes of a group (0: all n boxes are one); kParts: groups of a box
        auto boxes = [&](auto per_group, int n, int planes) {
          constexpr int kPer = decltype(per_group)::value;
#pragma unroll 1
          for (int kb = 0; kb < n; ++kb) {
            const bool begins = kPer == 0 ? kb == 0 : (kPer == 1 || (kb & 1) == 0);
            const bool ends = kPer == 0 ? kb == n - 1 : (kPer == 1 || (kb & 1) == 1);
#pragma unroll 1
            for (int q = 0; q < planes; ++q) {
              if (!gt_wait(smem_u32(full) + 8 * r.slot, r.phase, abort_flag, 40)) return false;
              tc_fence_after();
              const uint64_t ad = kDesc + (a0 + r.slot * (stage / 16)), bd = ad + GT_ABYTES / 16;
              if (lead) {
#pragma unroll
                for (int k16 = 0; k16 < 4; ++k16)
                  tc_mma_bf16(tbase + dr.slot * GT_N, ad + 2 * k16, bd + 2 * k16, idesc,
                              k16 == 0 && q == 0 && begins ? 0u : 1u);
                tc_commit(&empty[r.slot]);
                if (ends && q == planes - 1) tc_commit(&dfull[dr.slot]);
              }
              r.step(stages);
            }
            if (ends) dr.step(2);
          }
          return true;
        };
        // groups of 32: a box's two groups in turn, each from every plane; a stage is
        // given back after the second, so the planes of a box are all held at once
        auto boxes32 = [&](int n, int planes) {
#pragma unroll 1
          for (int kb = 0; kb < n; ++kb) {
            const int parts = min(2, p.k - 2 * kb);
            GtRing rs = r;
#pragma unroll 1
            for (int h = 0; h < parts; ++h) {
              if (!gt_wait(smem_u32(dempty) + 8 * dr.slot, dr.phase ^ 1, abort_flag, 41)) return false;
              rs = r;
#pragma unroll 1
              for (int q = 0; q < planes; ++q) {
                if (h == 0 && !gt_wait(smem_u32(full) + 8 * rs.slot, rs.phase, abort_flag, 42)) return false;
                tc_fence_after();
                const uint64_t ad = kDesc + (a0 + rs.slot * (stage / 16) + 4 * h), bd = ad + GT_ABYTES / 16;
                if (lead) {
                  tc_mma_bf16(tbase + dr.slot * GT_N, ad, bd, idesc, q == 0 ? 0u : 1u);
                  tc_mma_bf16(tbase + dr.slot * GT_N, ad + 2, bd + 2, idesc, 1u);
                  if (h == parts - 1) tc_commit(&empty[rs.slot]);
                }
                rs.step(stages);
              }
              if (lead) tc_commit(&dfull[dr.slot]);
              dr.step(2);
            }
            r = rs;
          }
          return true;
        };
        if constexpr (G == 32) {
          ok = boxes32(nbox, p.planes);
          if (ok) ok = gt_wait(smem_u32(dempty) + 8 * dr.slot, dr.phase ^ 1, abort_flag, 41);
        } else {
          ok = boxes(std::integral_constant<int, G == 128 ? 2 : 1>{}, nbox, p.planes);
        }
        if (ok) ok = boxes(std::integral_constant<int, 0>{}, ncor, 1);
      }
      // every issued product completes before tensor memory can be freed, also after an abort
      if (lead) {
        tc_commit(done);
        mbar_drain(done, 0);
      }
    }
    __syncwarp();
  }
  __syncthreads();
  if (*abort_flag && tid == 256) {
    record_async(kStatusTimeout, *abort_flag);
    // Every issued copy lands before the CTA can exit, whichever role gave up. A stage's phase ends with the
    // gate's arrival too: those that it left out are made up first. One limit for all of them.
    const uint32_t issued = *s_issued;
    for (uint32_t j = *s_arrived; j < issued; ++j) mbar_arrive(&full[j % stages]);
    const uint64_t t0 = global_ns();
    for (uint32_t j = issued > stages ? issued - stages : 0; j < issued; ++j)
      while (!mbar_try_wait(&full[j % stages], (j / stages) & 1) && global_ns() - t0 < kWaitLimitNs) {
      }
  }
  if (warp == 11) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// ---------------------------------------------------------------- few rows
// Experts with at most few_rows rows (single tokens, small batches): the packed
// codes are decoded into registers as the A fragments of mma.m16n8k16, whose
// other operand (rows of x) comes from shared memory. What bounds it is issue
// (decoding, about 1.8 operations a code, and the copies' addressing)
// before HBM, not the tensor work, so the warp-level instruction fits: no decoded
// operand passes through shared or tensor memory.
//
// A CTA of 8 warps takes 128 outputs and a range of 256-column chunks; a warp
// takes 32 of the outputs and every other group. The CTAs of a cluster share the
// outputs, split the depth and add their sums through distributed shared memory
// in a fixed order. Codes, x, scales and zeros are one chunk ahead (with a third
// stage fewer CTAs fit an SM: a quarter more time on three 13824 x 5120 experts of
// fp32 rows). Of 64 columns (32 in groups of 32) thread (g, t) of a warp takes the
// 16 (8) codes from 16 t (8 t) on of rows g, g + 8, g + 16, g + 24: as k-steps may
// take the columns in any order that x follows, those are its pairs of four (two)
// k-steps, and x's are consecutive bytes. The sums of x over 32 columns are
// products with rows of ones, a unit of the chunk for each warp.
// 10.7 us for one row of a 4096 x 4096 layer (5.3 MB), 84 for eight rows over five
// 11008 x 4096 experts (71 MB, 0.85 TB/s). (32 rows at a time at groups of 64 and 128
// spill 28 to 76 bytes at the 128 registers of two CTAs an SM.)
constexpr int GS_THREADS = 256, GS_M = 128, GS_K = 256, GS_STAGES = 2;
constexpr int GS_SMEM = 160 * 1024;  // beside 32 KB of tables; groups of 32, 7 bits, 16 rows in three planes take 130
// What the tables in shared memory hold: the widest layer that the entry point accepts.
constexpr int GS_MAX_CHUNKS = (kMaxColumns + GS_K - 1) / GS_K;
// Bytes of a row of x: the 16-byte reads of two rows and four threads meet no bank twice.
__host__ __device__ constexpr int gs_xstride(int group) { return GS_K * 2 + (group == 32 ? 64 : 16); }

struct GsParams {
  const uint32_t* codes;
  const uint8_t* bits;
  const float* scale;
  const float* zero;
  const void* x;             // bf16, [planes][rows][n]
  const int32_t* row_index;  // of x, or null
  const int32_t* offsets;
  void* y;
  int64_t m, n, R, rw, plane;  // plane: values between two planes of x
  int64_t T;
  int E, k, few_rows, mtiles, split;
  int cap, wstride;          // code words of a row in a stage, and their stride
};

__device__ __forceinline__ void gs_cp16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void gs_cp4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void gs_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// kNT: tiles of 8 rows at a time; kPlanes: bf16 planes of x.
template <int G, typename out_t, int kNT, int kPlanes>
__global__ void __launch_bounds__(GS_THREADS, 2) gs_kernel(const GsParams p) {
  constexpr int kUnits = G / 32, kGroups = GS_K / G, kRows = 8 * kNT;
  constexpr int kSub = G == 32 ? 32 : 64, kCodes = kSub / 4;  // columns decoded at a time, and a thread's of a row
  constexpr int GS_XSTRIDE = gs_xstride(G);
  extern __shared__ __align__(16) uint8_t gs_smem[];
  __shared__ int s_expert, s_found;
  __shared__ uint32_t s_width[kMaxGroups];         // first word << 4 | width of each group
  __shared__ int2 s_words[GS_MAX_CHUNKS];          // first and last word of each chunk
  // coef_d and coef_x, and what is added to the codes; a thread's four outputs side by side
  __shared__ __align__(16) float2 s_coef[2][kGroups][GS_M];
  __shared__ __align__(16) uint32_t s_shift[2][kGroups][GS_M];
  __shared__ int s_row[kRows];                     // row of x, -1: zeros
  __shared__ float2 s_sum[GS_K / 32][kRows / 2];   // sums of x over 32 columns, of two rows
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
  const int out0 = (warp & 3) * 32, part = warp >> 2;  // the warp's outputs, and which of the chunk's groups
  const int rank = blockIdx.x % p.split, mt = blockIdx.x / p.split;
  // the expert of this slot among those with 1 .. few_rows rows
  if (warp == 0) {
    int run = 0, mine = -1;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      const int rows = e < p.E ? gt_clamp(p.offsets[e + 1], p.R) - gt_clamp(p.offsets[e], p.R) : 0;
      const unsigned mask = __ballot_sync(0xffffffffu, rows > 0 && rows <= p.few_rows);
      const int at = (int)blockIdx.y - run;
      if (mine < 0 && at >= 0 && at < __popc(mask)) mine = e0 + (int)__fns(mask, 0, at + 1);
      run += __popc(mask);
    }
    if (lane == 0) {
      s_expert = mine;
      s_found = mine >= 0;
    }
  }
  __syncthreads();
  if (!s_found) return;  // (the same for every CTA of a cluster)
  const int e = s_expert, r0 = gt_clamp(p.offsets[e], p.R), r1 = gt_clamp(p.offsets[e + 1], p.R);
  if (warp == 0) {
    const uint8_t* bits = p.bits + (int64_t)e * p.k;
    int run = 0;
#pragma unroll 4
    for (int c0 = 0; c0 < p.k; c0 += 32) {
      const int c = c0 + lane;
      int b = c < p.k ? bits[c] : 0;
      if (b > 8) b = 0;
      int incl = b;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const int first = (run + incl - b) * kUnits;
      if (first + b * kUnits > p.rw) b = 0;  // widths that do not fill a row: nothing outside it is read
      if (c < p.k) s_width[c] = (uint32_t)(first << 4 | b);
      run += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  __syncthreads();
  const int chunks = (int)((p.n + GS_K - 1) / GS_K);
  const bool wide = (p.rw & 3) == 0;  // rows of 16-byte multiples
  for (int ch = tid; ch < chunks; ch += GS_THREADS) {  // words [first, end) of each chunk
    const uint32_t a = s_width[ch * kGroups], z = s_width[min((ch + 1) * kGroups, p.k) - 1];
    const int first = min((int)(a >> 4), (int)p.rw), end = min((int)(z >> 4) + (int)(z & 15) * kUnits, (int)p.rw);
    s_words[ch] = make_int2(wide ? first & ~3 : first, end);
  }
  __syncthreads();
  const int ch0 = chunks * rank / p.split, ch1 = chunks * (rank + 1) / p.split;
  const int64_t m0 = (int64_t)mt * GS_M, base = (int64_t)e * p.m;
  const int mrows = (int)min((int64_t)GS_M, p.m - m0);
  const uint32_t sbase = smem_u32(gs_smem);
  const uint32_t xbytes = kPlanes * kRows * GS_XSTRIDE, stage = xbytes + GS_M * p.wstride * 4;
  // this thread's scales and zeros: an output's, of one half of a chunk's groups
  const int64_t srow = (base + m0 + min(tid & (GS_M - 1), mrows - 1)) * p.k;
  constexpr int kHalf = kGroups / 2;
  const int chalf = (tid / GS_M) * kHalf;
  const int sat = (tid & (GS_M - 32)) + (tid & 7) * 4 + ((tid & 31) >> 3);  // where its output stands in the tables

  for (int q0 = r0; q0 < r1; q0 += kRows) {
    const int rows = min(kRows, r1 - q0), nt = (rows + 7) / 8;
    float acc[2][kNT][4];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int b = 0; b < kNT; ++b)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[a][b][c] = 0.f;
    if (tid < kRows) {
      int src = q0 + tid;
      if (tid < rows && p.row_index) src = p.row_index[src];
      s_row[tid] = tid < rows && src >= 0 && src < p.T ? src : -1;
    }
    __syncthreads();
    const uint32_t* codes0 = p.codes + (base + m0 + (tid >> 3)) * p.rw;
    auto copy_chunk = [&](int ch, int slot) {
      if (ch < ch1) {
        const uint32_t sx = sbase + slot * stage, sw = sx + xbytes;
        const int cols = (int)min((int64_t)GS_K, p.n - (int64_t)ch * GS_K);
        const int c = tid & 31;
        const bool col_ok = c * 8 < cols;
#pragma unroll
        for (int pl = 0; pl < kPlanes; ++pl)
#pragma unroll 2
          for (int r = tid >> 5; r < nt * 8; r += GS_THREADS / 32) {
            const int src = s_row[r];
            const bool have = src >= 0 && col_ok;
            gs_cp16(sx + (pl * kRows + r) * GS_XSTRIDE + c * 16,
                    static_cast<const uint16_t*>(p.x) + pl * p.plane + (have ? src * p.n + ch * GS_K + c * 8 : 0),
                    have ? 16u : 0u);  // 0: zeros
          }
        const int first = s_words[ch].x, end = min(s_words[ch].y, first + p.cap);
        const int row = tid >> 3;  // and every 32nd from it
        constexpr int kStep = GS_THREADS / 8;
        const uint32_t rstep = kStep * p.wstride * 4;
        if (wide) {
          for (int w = (tid & 7) * 4; w < end - first; w += 32) {
            const uint32_t* src = codes0 + first + w;
            uint32_t dst = sw + (row * p.wstride + w) * 4;
#pragma unroll
            for (int i = 0; i < GS_M / kStep; ++i) {
              if (row + kStep * i < mrows) gs_cp16(dst, src, 16u);
              src += kStep * p.rw;
              dst += rstep;
            }
          }
        } else {
          for (int w = tid & 7; w < end - first; w += 8) {
            const uint32_t* src = codes0 + first + w;
            uint32_t dst = sw + (row * p.wstride + w) * 4;
#pragma unroll
            for (int i = 0; i < GS_M / kStep; ++i) {
              if (row + kStep * i < mrows) gs_cp4(dst, src);
              src += kStep * p.rw;
              dst += rstep;
            }
          }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    float sreg[kHalf], zreg[kHalf];
    auto load_scales = [&](int ch) {
#pragma unroll
      for (int c = 0; c < kHalf; ++c) {
        const int at = min(ch * kGroups + chalf + c, p.k - 1);
        sreg[c] = __ldg(p.scale + srow + at);
        zreg[c] = __ldg(p.zero + srow + at);
      }
    };
#pragma unroll
    for (int c = 0; c < GS_STAGES - 1; ++c) copy_chunk(ch0 + c, c);
    if (ch0 < ch1) load_scales(ch0);
    int slot = 0;
    for (int ch = ch0; ch < ch1; ++ch) {
      // coefficients of this chunk (their buffer was last read two chunks ago)
#pragma unroll
      for (int c = 0; c < kHalf; ++c) {
        const int at = ch * kGroups + chalf + c, b = at < p.k ? s_width[at] & 15 : 0;
        const uint32_t shift = code_shift(b, zreg[c]);
        s_shift[ch & 1][chalf + c][sat] = shift;
        s_coef[ch & 1][chalf + c][sat] =
            b ? make_float2(coef_d(b, sreg[c]), coef_x(b, sreg[c], zreg[c], shift)) : make_float2(0.f, 0.f);
      }
      if (ch + 1 < ch1) load_scales(ch + 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(GS_STAGES - 2) : "memory");
      __syncthreads();  // this chunk has arrived for all; the slot of the last one is free
      copy_chunk(ch + GS_STAGES - 1, slot == 0 ? GS_STAGES - 1 : slot - 1);
      const int first = s_words[ch].x;
      const uint32_t sx = sbase + slot * stage + g * GS_XSTRIDE + t4 * kCodes * 2;
      const uint32_t sw = sbase + slot * stage + xbytes + (out0 + g) * p.wstride * 4;
      // the sums of x over the warp's unit of 32 columns (rows of ones: every row of the product is the sum)
#pragma unroll
      for (int q = 0; q < kNT; ++q)
        if (q < nt) {
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int pl = kPlanes - 1; pl >= 0; --pl) {
            uint32_t b0, b1, b2, b3;
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(b0), "=r"(b1), "=r"(b2), "=r"(b3)
                         : "r"(sbase + slot * stage + (pl * kRows + q * 8 + g) * GS_XSTRIDE + warp * 64 + t4 * 16));
            gs_mma(sum, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u, b0, b1);
            gs_mma(sum, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u, b2, b3);
          }
          if (g == 0) s_sum[warp][q * 4 + t4] = make_float2(sum[0], sum[1]);
        }
      __syncthreads();
      const bool fits = s_words[ch].y - first <= p.cap;
#pragma unroll 1
      for (int c = part; c < kGroups; c += 2) {
        if (ch * kGroups + c >= p.k) break;
        const uint32_t en = s_width[ch * kGroups + c], b = en & 15;
        if (b == 0) continue;  // not a width
        float d[2][kNT][4];
#pragma unroll
        for (int q = 0; q < kNT; ++q)
#pragma unroll
          for (int v = 0; v < 4; ++v) d[0][q][v] = d[1][q][v] = 0.f;
        const uint32_t wrel = (en >> 4) - first;
#pragma unroll 1
        for (int u = 0; u < G / kSub; ++u) {
          // the thread's kCodes codes of four rows: kCodes b bits from bit `bit` of the staged row on
          const uint32_t bit = (wrel + u * (kSub / 32) * b) * 32 + t4 * kCodes * b;
          const uint4 shifts = *reinterpret_cast<const uint4*>(&s_shift[ch & 1][c][out0 + g * 4]);
          uint32_t A[4][kCodes / 2];
          switch (b) {
#define GS_CASE(B)                                                                                            \
  case B: {                                                                                                   \
    constexpr int kBits = B * kCodes, kWords = (kBits + 31) / 32;                                             \
    /* the bits start where a multiple of kBits and of 8 can start in a word */                               \
    constexpr bool kShift = kBits % 32 != 0, kMore = kShift && (kBits % 32) + (kBits % 16 ? 24 : 16) > 32;    \
    const uint32_t sh = bit & 31;                                                                             \
    _Pragma("unroll") for (int r = 0; r < 4; ++r) {                                                           \
      uint32_t w[kWords + 1], v[kWords];                                                                      \
      w[kWords] = 0;                                                                                          \
      if (fits) {                                                                                             \
        const uint32_t at = sw + (r * 8 * p.wstride + (bit >> 5)) * 4;                                        \
        _Pragma("unroll") for (int q = 0; q < kWords + (kMore ? 1 : 0); ++q)                                  \
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[q]) : "r"(at + 4 * q));                           \
      } else { /* wider than the stage was made for: straight from global memory */                           \
        const int row = min(out0 + g + 8 * r, mrows - 1);                                                     \
        const uint32_t* src = p.codes + (base + m0 + row) * p.rw;                                             \
        _Pragma("unroll") for (int q = 0; q < kWords + (kMore ? 1 : 0); ++q) {                                \
          const int64_t at = first + (bit >> 5) + q;                                                          \
          w[q] = at < p.rw ? __ldg(src + at) : 0u;                                                            \
        }                                                                                                     \
      }                                                                                                       \
      _Pragma("unroll") for (int q = 0; q < kWords; ++q) v[q] = kShift ? __funnelshift_r(w[q], w[q + 1], sh) : w[q]; \
      decode_codes<B, kCodes>(v, r == 0 ? shifts.x : r == 1 ? shifts.y : r == 2 ? shifts.z : shifts.w, A[r]); \
    }                                                                                                         \
  } break;
            GS_CASE(1) GS_CASE(2) GS_CASE(3) GS_CASE(4) GS_CASE(5) GS_CASE(6) GS_CASE(7) GS_CASE(8)
#undef GS_CASE
            default: break;
          }
          const uint32_t xu = sx + (c * G + u * kSub) * 2;
#pragma unroll
          for (int pl = kPlanes - 1; pl >= 0; --pl)
#pragma unroll
            for (int q = 0; q < kNT; ++q)
              if (q < nt) {
#pragma unroll
                for (int h = 0; h < kCodes / 8; ++h) {
                  uint32_t b0, b1, b2, b3;
                  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                               : "=r"(b0), "=r"(b1), "=r"(b2), "=r"(b3)
                               : "r"(xu + (pl * kRows + q * 8) * GS_XSTRIDE + h * 16));
#pragma unroll
                  for (int a = 0; a < 2; ++a) {
                    gs_mma(d[a][q], A[2 * a][4 * h], A[2 * a + 1][4 * h], A[2 * a][4 * h + 1], A[2 * a + 1][4 * h + 1],
                           b0, b1);
                    gs_mma(d[a][q], A[2 * a][4 * h + 2], A[2 * a + 1][4 * h + 2], A[2 * a][4 * h + 3],
                           A[2 * a + 1][4 * h + 3], b2, b3);
                  }
                }
              }
        }
        const float4* cp = reinterpret_cast<const float4*>(&s_coef[ch & 1][c][out0 + g * 4]);
        const float4 c01 = cp[0], c23 = cp[1];
        const float2 co[4] = {{c01.x, c01.y}, {c01.z, c01.w}, {c23.x, c23.y}, {c23.z, c23.w}};
#pragma unroll
        for (int q = 0; q < kNT; ++q)
          if (q < nt) {
            float2 xs = s_sum[c * kUnits][q * 4 + t4];
#pragma unroll
            for (int u = 1; u < kUnits; ++u) {
              const float2 more = s_sum[c * kUnits + u][q * 4 + t4];
              xs.x += more.x;
              xs.y += more.y;
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              float* to = &acc[r >> 1][q][(r & 1) * 2];
              const float* dd = &d[r >> 1][q][(r & 1) * 2];
              to[0] = fmaf(co[r].x, dd[0], fmaf(co[r].y, xs.x, to[0]));
              to[1] = fmaf(co[r].x, dd[1], fmaf(co[r].y, xs.y, to[1]));
            }
          }
      }
      slot = slot == GS_STAGES - 1 ? 0 : slot + 1;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    // the CTA's sums [row of x][output], then the cluster's in rank order
    float* red = reinterpret_cast<float*>(gs_smem);
#pragma unroll
    for (int turn = 1; turn >= 0; --turn) {  // the second half of the groups, then the first on top
      if (part == turn) {
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int q = 0; q < kNT; ++q)
#pragma unroll
            for (int v = 0; v < 4; ++v)
              if (q < nt) {
                float* to = &red[(q * 8 + t4 * 2 + (v & 1)) * GS_M + out0 + a * 16 + g + (v >> 1) * 8];
                *to = turn ? acc[a][q][v] : *to + acc[a][q][v];
              }
      }
      if (turn) __syncthreads();
    }
    if (p.split > 1) {
      asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    } else {
      __syncthreads();
    }
    for (int v = tid + rank * GS_THREADS; v < rows * GS_M; v += GS_THREADS * p.split) {
      const int r = v / GS_M, o = v % GS_M;
      if (o >= mrows) continue;
      float sum = 0.f;
      for (int z = 0; z < p.split; ++z) {
        float f;
        if (p.split > 1) {
          uint32_t at;
          asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(sbase + v * 4), "r"(z));
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f) : "r"(at) : "memory");
        } else {
          f = red[v];
        }
        sum += f;
      }
      const int64_t to = (int64_t)(q0 + r) * p.m + m0 + o;
      static_cast<out_t*>(p.y)[to] = as_out<out_t>(sum);
    }
    if (p.split > 1) {
      asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    } else {
      __syncthreads();
    }
  }
}

// ---------------------------------------------------------------- host side
// Experts with at most this many rows: the few-rows kernel, whose time grows with every 8 rows and starts again
// every 32 (fp32 x: 16, each in three planes), while the other's is the decoding and the depth's chain. Eight 4096 x 4096
// experts of 16, 24, 32, 48, 64 rows each, the few-rows kernel / the other, in us:
//   bf16, groups of 128: 82/167 108/168 119/168 188/174 209/175    groups of 32: 140/267 163/267 173/267 295/285 312/285
//   fp32, groups of 128: 110/241 184/241 206/242 296/271 384/272   groups of 32: 196/327 355/330 373/335 544/351 714/358
// For a single expert the few-rows kernel is the faster one up to 64 rows (fp32 at groups of 32: 48).
constexpr int kFewRows = 32;
constexpr size_t kTileBytes = size_t(1) << 30;  // decoded tiles of a pass

struct GroupedPlan {
  int planes;          // bf16 planes copied in grouped order (0: x is read as it is)
  int64_t xs_stride;   // correction columns of a row
  int64_t slots, st;   // experts that can have many rows, in all and in a pass
  int64_t mtiles, mt;  // output tiles in all and of a pass
  size_t off_xg, off_tiles, bytes;
};

static GroupedPlan grouped_plan(int64_t E, int64_t m, int64_t n, int group, int xdtype, bool gathered, int64_t R) {
  GroupedPlan g{};
  const int64_t k = n / group, boxes = (n + GT_K - 1) / GT_K + (k + kCorr - 1) / kCorr;
  g.slots = std::min<int64_t>(E, R / (kFewRows + 1));
  g.mtiles = (m + GT_M - 1) / GT_M;
  g.planes = xdtype == 0 ? 3 : (gathered && g.slots ? 1 : 0);
  g.xs_stride = k * kSlots;
  if (g.slots) {
    const size_t each = (size_t)boxes * GT_ABYTES;  // one output tile of a slot: 18 MB at most
    const int64_t fit = (int64_t)(kTileBytes / each);
    g.st = std::min(g.slots, fit);
    g.mt = std::min(g.mtiles, fit / g.st);
    g.off_xg = ((size_t)R * g.xs_stride * 2 + 255) & ~size_t(255);
    g.bytes = each * g.st * g.mt;
  }
  g.off_tiles = g.off_xg + (((size_t)g.planes * R * n * 2 + 255) & ~size_t(255));
  g.bytes += g.off_tiles;
  return g;
}

size_t grouped_workspace_bytes(int64_t E, int64_t m, int64_t n, int group, int xdtype, bool gathered, int64_t R) {
  return grouped_plan(E, m, n, group, xdtype, gathered, R).bytes;
}

template <int G, typename out_t>
static cudaError_t launch_many(const GtMaps& tm, GtParams p, const GroupedPlan& g, int num_sms, cudaStream_t s) {
  static std::atomic<uint64_t> attr{0};
  uint64_t bit = 0;
  if (attr_pending(attr, bit)) {
    const cudaError_t e =
        cudaFuncSetAttribute(gg_tc_kernel<G, out_t>, cudaFuncAttributeMaxDynamicSharedMemorySize, GT_SMEM);
    if (e != cudaSuccess) return e;
    attr.fetch_or(bit);
  }
  const int boxes = (int)((p.n + GT_K - 1) / GT_K) + (p.k + kCorr - 1) / kCorr;
  for (int64_t st = 0; st < g.slots; st += g.st) {
    p.slot0 = (int)st;
    p.slots = (int)std::min(g.st, g.slots - st);
    for (int64_t mt = 0; mt < g.mtiles; mt += g.mt) {
      p.mt0 = (int)mt;
      p.mtn = (int)std::min<int64_t>(g.mt, g.mtiles - mt);
      gd_kernel<G><<<dim3((boxes + GD_BOXES - 1) / GD_BOXES, p.mtn, (unsigned)p.slots), GD_THREADS, 0, s>>>(p);
      gg_tc_kernel<G, out_t><<<num_sms, GT_THREADS, GT_SMEM, s>>>(tm, p);
      count_launches(2);
    }
  }
  return cudaGetLastError();
}

template <int G, typename out_t, int kNT, int kPlanes>
static cudaError_t launch_few(GsParams p, int64_t slots, int avg_bits, int num_sms, cudaStream_t s) {
  static std::atomic<uint64_t> attr{0};
  uint64_t bit = 0;
  if (attr_pending(attr, bit)) {
    const cudaError_t e = cudaFuncSetAttribute(gs_kernel<G, out_t, kNT, kPlanes>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, GS_SMEM);
    if (e != cudaSuccess) return e;
    attr.fetch_or(bit);
  }
  // a stage holds widths of up to avg_bits + 1 on average; 4 more words where the copy starts early
  p.cap = GS_K / 32 * std::min(avg_bits + 1, 8) + 4;
  p.wstride = (p.cap + 7) / 8 * 8 + 4;  // 4 modulo 8: the eight rows of a read meet no bank twice
  const size_t smem = (size_t)GS_STAGES * (kPlanes * 8 * kNT * gs_xstride(G) + GS_M * p.wstride * 4);
  // The depth is split over a cluster until two to four CTAs an SM have work: one row of a 4096 x 4096 layer takes a
  // third of the time split over eight (10.4 us against 32.9), 160 rows over seven 4096 x 11008 experts nine tenths. The
  // host knows how many experts can have rows, not how many have.
  const int64_t tiles = slots * p.mtiles, chunks = (p.n + GS_K - 1) / GS_K;
  int split = 1;
  while (split < 8 && tiles * split * 2 <= (int64_t)num_sms * 4 && chunks >= split * 2) split *= 2;
  p.split = split;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.mtiles * split), (unsigned)slots, 1);
  cfg.blockDim = dim3(GS_THREADS, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = split;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  count_launches(1);
  return cudaLaunchKernelEx(&cfg, gs_kernel<G, out_t, kNT, kPlanes>, p);
}

template <int G, typename out_t>
static cudaError_t launch_few_of(const GsParams& p, int planes, int64_t slots, int64_t R, int avg_bits, int num_sms,
                                 cudaStream_t s) {
  if (planes == 3)
    return R <= 8 ? launch_few<G, out_t, 1, 3>(p, slots, avg_bits, num_sms, s)
                  : launch_few<G, out_t, 2, 3>(p, slots, avg_bits, num_sms, s);
  if (R <= 8) return launch_few<G, out_t, 1, 1>(p, slots, avg_bits, num_sms, s);
  return R <= 16 ? launch_few<G, out_t, 2, 1>(p, slots, avg_bits, num_sms, s)
                 : launch_few<G, out_t, 4, 1>(p, slots, avg_bits, num_sms, s);
}

// The limit of the epilogue's wait, in polls. Tests shorten it by SLIM_TEST_GROUPED_POLLS (0: runs out at once) to
// check that a wait that runs out is reported and leaves the device usable. Nothing else reads it.
static int acc_polls() {
  const char* t = std::getenv("SLIM_TEST_GROUPED_POLLS");
  const int v = t ? std::atoi(t) : kWaitPolls;
  return v >= 0 && v < kWaitPolls ? v : kWaitPolls;
}

cudaError_t launch_grouped(const uint32_t* codes, const uint8_t* bits, const float* scale, const float* zero,
                           int64_t E, int64_t m, int64_t n, int group, int avg_bits, const void* x, int xdtype,
                           int64_t T, const int32_t* row_index, const int32_t* offsets, int64_t R, void* y,
                           int ydtype, uint8_t* ws, int num_sms, cudaStream_t s) {
  const GroupedPlan g = grouped_plan(E, m, n, group, xdtype, row_index != nullptr, R);
  uint16_t* xs = g.slots ? reinterpret_cast<uint16_t*>(ws) : nullptr;
  uint16_t* xg = g.planes ? reinterpret_cast<uint16_t*>(ws + g.off_xg) : nullptr;
  const int k = (int)(n / group);
  cudaError_t e = cudaSuccess;
  if (xs || xg) {
    const dim3 blocks((unsigned)((R + GP_ROWS - 1) / GP_ROWS), (unsigned)((n + GP_COLS - 1) / GP_COLS));
    gg_prep_kernel<<<blocks, GP_ROWS * 32, 0, s>>>(x, xdtype, T, row_index, R, n, group, xg, xs, g.xs_stride);
    count_launches(1);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  const int64_t rw = n * avg_bits / 32;
  // one expert of many rows: the few-rows kernel has nothing to do unless its count is small, which only the
  // device knows, so both run
  GsParams f{};
  f.codes = codes; f.bits = bits; f.scale = scale; f.zero = zero; f.offsets = offsets; f.y = y;
  f.x = xg ? static_cast<const void*>(xg) : x;
  f.row_index = xg ? nullptr : row_index;
  f.T = xg ? R : T; f.plane = R * n;
  f.m = m; f.n = n; f.R = R; f.rw = rw; f.E = (int)E; f.k = k; f.few_rows = kFewRows;
  f.mtiles = (int)((m + GS_M - 1) / GS_M);
  const int planes = xdtype == 0 ? 3 : 1;
  const int64_t few = std::min<int64_t>(E, R);
#define SLIM_GS(G)                                                                  \
  (ydtype == 0 ? launch_few_of<G, float>(f, planes, few, R, avg_bits, num_sms, s)   \
               : launch_few_of<G, uint16_t>(f, planes, few, R, avg_bits, num_sms, s))
  e = group == 32 ? SLIM_GS(32) : (group == 64 ? SLIM_GS(64) : SLIM_GS(128));
#undef SLIM_GS
  if (e != cudaSuccess || g.slots == 0) return e;
  GtParams p{};
  p.codes = codes; p.bits = bits; p.scale = scale; p.zero = zero; p.offsets = offsets; p.y = y;
  p.tiles = ws + g.off_tiles;
  p.m = m; p.n = n; p.R = R; p.rw = rw;
  p.E = (int)E; p.k = k; p.planes = planes; p.few_rows = kFewRows;
  p.max_slots = (int)g.slots;
  p.acc_polls = acc_polls();
  GtMaps tm;
  const void* xb = xg ? static_cast<const void*>(xg) : x;
  const uint64_t rows = xg ? (uint64_t)g.planes * R : (uint64_t)T;
  const uint64_t xs_bytes = (uint64_t)g.xs_stride * 2;
  if (!make_tmap_bf16(&tm.x256, xb, (uint64_t)n, rows, GT_K, GT_N) ||
      !make_tmap_bf16(&tm.x32, xb, (uint64_t)n, rows, GT_K, 32) ||
      !make_tmap_2byte_strided(&tm.s256, xs, (uint64_t)k * kSlots, (uint64_t)R, xs_bytes, GT_K, GT_N) ||
      !make_tmap_2byte_strided(&tm.s32, xs, (uint64_t)k * kSlots, (uint64_t)R, xs_bytes, GT_K, 32))
    return cudaErrorInvalidValue;
#define SLIM_GT(G) (ydtype == 0 ? launch_many<G, float>(tm, p, g, num_sms, s) : launch_many<G, uint16_t>(tm, p, g, num_sms, s))
  return group == 32 ? SLIM_GT(32) : (group == 64 ? SLIM_GT(64) : SLIM_GT(128));
#undef SLIM_GT
}

}  // namespace slim
