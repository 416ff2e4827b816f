// slm_orth.cu - the orthogonalised update (slm_orthogonalize): momentum, normalisation and the
// Newton-Schulz products.
//
// For each [m, n] matrix of a stack, with k = min(m, n):
//     mom <- beta mom + (1 - beta) g,   u = beta mom + (1 - beta) g (or mom, or g without one)
//     X = u / (||u||_F + eps)
//     steps times:  A = X X^T (X^T X when m > n),  B = b A + c A^2,  X <- a X + B X (or X B).
//
// Number formats.  The products run on the tensor cores with fp16 operands (11-bit
// significands; bf16's 8 bits lose 1e-2 to 3e-1 of the result here, because the steps
// multiply small singular directions, and with them the rounding noise, by up to a^steps) and
// fp32 accumulators.  Three choices keep the result within about 1e-3 of the exact iteration:
//   - X is held as hi + lo, two fp16 numbers (22 bits).  Products use hi; the term a X, which
//     carries the small singular directions through, uses both.
//   - A and B are held as a diagonal in fp32 and fp16 off-diagonal entries (zero diagonal).
//     The diagonals of A and B are their largest and nearly equal entries, so that rounding
//     them is one common error, which the polynomial amplifies; apart, they cost one fused
//     multiply-add in the epilogues:  with A = D + R,
//         A^2 = R R + (D_i + D_j) R + D^2,    B X = R_B hi + D_B hi.
//     (D_B multiplies hi, not hi + lo: B must act on one and the same X in all its terms, or
//     the difference's noise reaches directions that B alone would not touch.)
//   - hi, lo and the matrices are stored times a power of two (kScaleX, kScaleA, kScaleB), so
//     that fp16's exponent range covers them: |X|, |A| < 4 and |B| < 16 fit, which the host
//     checks of the coefficients, and entries down to 2^-28 are normal numbers.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "slm_internal.h"
#include "slm_wait.cuh"
#include "sm100.cuh"

namespace slm {
namespace {
using namespace sm100;

constexpr float kScaleX = 16384.f;  // 2^14
constexpr float kScaleA = 16384.f;
constexpr float kScaleB = 4096.f;  // 2^12

template <class T>
__device__ __forceinline__ float ld_elem(const void* p, int64_t i);
template <>
__device__ __forceinline__ float ld_elem<float>(const void* p, int64_t i) {
  return static_cast<const float*>(p)[i];
}
template <>
__device__ __forceinline__ float ld_elem<__nv_bfloat16>(const void* p, int64_t i) {
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
template <>
__device__ __forceinline__ float ld_elem<__half>(const void* p, int64_t i) {
  return __half2float(static_cast<const __half*>(p)[i]);
}

constexpr int kPrepThreads = 256;

// Momentum update and the partial sums of u^2 (64 bits: the squares of fp32 gradients may
// leave fp32's range).  Block (i, b): rows i, i + gridDim.x, ... of matrix b.
template <class T>
__global__ void __launch_bounds__(kPrepThreads) orth_moment(const OrthPrep p) {
  const int64_t b = blockIdx.y;
  double s = 0.0;
  for (int64_t r = blockIdx.x; r < p.m; r += gridDim.x) {
    const int64_t g0 = b * p.grad_batch + r * p.ldg, m0 = (b * p.m + r) * p.n;
    for (int64_t c = threadIdx.x; c < p.n; c += kPrepThreads) {
      float u = ld_elem<T>(p.grad, g0 + c);
      if (p.momentum) {
        const float mom = p.beta * p.momentum[m0 + c] + p.rest * u;
        p.momentum[m0 + c] = mom;
        u = p.nesterov ? p.beta * mom + p.rest * u : mom;
      }
      s += static_cast<double>(u) * static_cast<double>(u);
    }
  }
  __shared__ double part[kPrepThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    double t = 0.0;
    for (int i = 0; i < kPrepThreads / 32; ++i) t += part[i];
    p.sums[b * kOrthSums + blockIdx.x] = t;
  }
}

// X = u / (||u|| + eps) as hi + lo; the norm from the partial sums, added in a fixed order.
template <class T>
__global__ void __launch_bounds__(kPrepThreads) orth_scale(const OrthPrep p, int nsums) {
  __shared__ float inv_sh;
  const int64_t b = blockIdx.y;
  if (threadIdx.x < 32) {
    double t = 0.0;
    for (int i = threadIdx.x; i < nsums; i += 32) t += p.sums[b * kOrthSums + i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (threadIdx.x == 0)
      inv_sh = static_cast<float>(kScaleX / (sqrt(t) + static_cast<double>(p.eps)));
  }
  __syncthreads();
  const float inv = inv_sh;
  for (int64_t r = blockIdx.x; r < p.m; r += gridDim.x) {
    const int64_t g0 = b * p.grad_batch + r * p.ldg, m0 = (b * p.m + r) * p.n;
    const int64_t x0 = (b * p.m + r) * p.ldx;
    for (int64_t c = threadIdx.x; c < p.n; c += kPrepThreads) {
      float u = ld_elem<T>(p.grad, g0 + c);
      if (p.momentum) {
        const float mom = p.momentum[m0 + c];
        u = p.nesterov ? p.beta * mom + p.rest * u : mom;
      }
      const float x = u * inv;
      const __half hi = __float2half_rn(x);
      p.hi[x0 + c] = hi;
      p.lo[x0 + c] = __float2half_rn(x - __half2float(hi));
    }
  }
}

// ----------------------------------------------------------------------------------------
// The products: a persistent 2-SM GEMM (M = 256 rows per CTA pair, BN columns, fp16 operands,
// two TMEM accumulators so that one tile's epilogue overlaps the next tile's MMAs).  Warp 0
// loads, warp 1 issues the MMAs, eight warps run the epilogue, each warpgroup over half of the
// columns.  Operands are K-major or MN-major as they lie in memory, so that no transpose of X
// is ever stored.
//   kGram    R, D of A = X X^T:  a symmetric product, only tiles on and below the diagonal
//            are computed and each is written to its mirrored place too
//   kSquare  R_B, D_B of B = b A + c A^2, symmetric in the same way
//   kUpdate  hi, lo of a X + B X; in the last step the result in bf16
// ----------------------------------------------------------------------------------------
enum OrthOp { kGram = 0, kSquare = 1, kUpdate = 2 };
constexpr int kOrthWG = 2;
constexpr int kOrthThreads = 64 + 128 * kOrthWG;

template <int STAGES>
struct OrthCtl {
  uint64_t full[STAGES], empty[STAGES], tfull[2], tempty[2], fin;
  uint32_t tmem_base;
  int abort;
};

template <int BN>
struct OrthCfg {
  static constexpr int kSliceN = BN / 2;  // columns whose operand rows each CTA holds
  static constexpr uint32_t kABytes = kBM * kBK * 2;
  static constexpr uint32_t kBBytes = kSliceN * kBK * 2;
  static constexpr uint32_t kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = BN == 256 ? 6 : 8;
  static constexpr size_t kSmem =
      1024 + kStages * static_cast<size_t>(kStageBytes) + sizeof(OrthCtl<kStages>);
  static_assert(2 * BN <= 512, "two accumulators in TMEM");
  static_assert(kSmem <= 232448, "shared memory per CTA");
};

// Tile of unit u: matrix z, pair row tile i, column tile j.
template <int BN, bool SYM>
__device__ __forceinline__ void orth_unit(const OrthGemm& g, int u, int& z, int& i, int& j) {
  z = u / g.units_per;
  const int t = u - z * g.units_per;
  if (SYM) {
    // Row tile i has the column tiles 0 .. W (i + 1) - 1, W = 256 / BN; rows before i: W i (i + 1) / 2.
    constexpr int W = 256 / BN;
    i = static_cast<int>((sqrtf(8.f / W * t + 1.f) - 1.f) * 0.5f);
    while (W * i * (i + 1) / 2 > t) --i;
    while (W * (i + 1) * (i + 2) / 2 <= t) ++i;
    j = t - W * i * (i + 1) / 2;
  } else {
    const int per_group = g.group_m * g.num_n;
    const int grp = t / per_group;
    const int r = t - grp * per_group;
    const int gm = min(g.group_m, g.num_m - grp * g.group_m);
    j = r / gm;
    i = grp * g.group_m + (r - j * gm);
  }
}

// 32 consecutive fp16 numbers of a row; `n` of them exist (the rest read as 0).
__device__ __forceinline__ void ld_half32(const __half* p, int n, float (&v)[32]) {
  if (n >= 32) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint4 w = reinterpret_cast<const uint4*>(p)[q];
      const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&a[e]));
        v[8 * q + 2 * e] = f.x;
        v[8 * q + 2 * e + 1] = f.y;
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] = e < n ? __half2float(p[e]) : 0.f;
  }
}
__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_bf162(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void st_half32(__half* p, int n, const float (&v)[32]) {
  if (n >= 32) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      reinterpret_cast<uint4*>(p)[q] =
          make_uint4(pack_half2(v[8 * q], v[8 * q + 1]), pack_half2(v[8 * q + 2], v[8 * q + 3]),
                     pack_half2(v[8 * q + 4], v[8 * q + 5]), pack_half2(v[8 * q + 6], v[8 * q + 7]));
  } else {
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (e < n) p[e] = __float2half_rn(v[e]);
  }
}

// One thread's 32 columns [col, col + 32) of row `row` (row < rows) of matrix z.
template <int OP, bool LAST>
__device__ __forceinline__ void orth_epilogue(const OrthGemm& g, int z, int64_t row, int64_t col,
                                              bool mirror, float (&v)[32]) {
  const int n = static_cast<int>(min(static_cast<int64_t>(32), g.cols - col));
  if (OP == kGram || OP == kSquare) {
    const int64_t at = (static_cast<int64_t>(z) * g.rows + row) * g.ld + col;
    if (OP == kGram) {
      const int e = static_cast<int>(row - col);
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        if (c == e) g.diag_out[static_cast<int64_t>(z) * g.rows + row] = v[c] * (1.f / (kScaleX * kScaleX));
        v[c] = c == e ? 0.f : v[c] * (kScaleA / (kScaleX * kScaleX));
      }
    } else {
      float r[32];
      ld_half32(g.a_in + at, n, r);
      const float* dg = g.diag_in + static_cast<int64_t>(z) * g.rows;
      const float di = dg[row];
      const int e = static_cast<int>(row - col);
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        const float dj = c < n ? dg[col + c] : 0.f;
        const float rr = v[c] * (1.f / (kScaleA * kScaleA));
        if (c == e) {
          g.diag_out[static_cast<int64_t>(z) * g.rows + row] = fmaf(g.c, fmaf(di, di, rr), g.b * di);
          v[c] = 0.f;
        } else {
          const float a = r[c] * (1.f / kScaleA);
          v[c] = kScaleB * fmaf(g.c, fmaf(di + dj, a, rr), g.b * a);
        }
      }
    }
    st_half32(g.a_out + at, n, v);
    if (mirror) {
      // Lanes hold consecutive rows: each column goes out as one run of 32 fp16 numbers.
      __half* dst = g.a_out + (static_cast<int64_t>(z) * g.rows + col) * g.ld + row;
#pragma unroll
      for (int c = 0; c < 32; ++c)
        if (c < n) dst[static_cast<int64_t>(c) * g.ld] = __float2half_rn(v[c]);
    }
  } else {
    const int64_t at = (static_cast<int64_t>(z) * g.rows + row) * g.ld + col;
    float hi[32], lo[32];
    ld_half32(g.hi_in + at, n, hi);
    ld_half32(g.lo + at, n, lo);
    const float* dg = g.diag_in + static_cast<int64_t>(z) * g.diag_n;
    const float drow = g.tall ? 0.f : dg[row];
#pragma unroll
    for (int c = 0; c < 32; ++c) {
      const float db = g.tall ? (c < n ? dg[col + c] : 0.f) : drow;
      v[c] = fmaf(v[c], 1.f / kScaleB, fmaf(db, hi[c], g.a * (hi[c] + lo[c])));
    }
    if (LAST) {
      __nv_bfloat16* out = g.out + (static_cast<int64_t>(z) * g.rows + row) * g.cols + col;
#pragma unroll
      for (int c = 0; c < 32; ++c) v[c] *= 1.f / kScaleX;
      if (g.out_vec && n >= 32) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          reinterpret_cast<uint4*>(out)[q] = make_uint4(
              pack_bf162(v[8 * q], v[8 * q + 1]), pack_bf162(v[8 * q + 2], v[8 * q + 3]),
              pack_bf162(v[8 * q + 4], v[8 * q + 5]), pack_bf162(v[8 * q + 6], v[8 * q + 7]));
      } else {
#pragma unroll
        for (int c = 0; c < 32; ++c)
          if (c < n) out[c] = __float2bfloat16_rn(v[c]);
      }
    } else {
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        hi[c] = __half2float(__float2half_rn(v[c]));
        lo[c] = v[c] - hi[c];
      }
      st_half32(g.hi_out + at, n, hi);
      st_half32(g.lo + at, n, lo);
    }
  }
}

template <int BN, bool A_MN, bool B_MN, int OP, bool LAST>
__global__ void __launch_bounds__(kOrthThreads, 1)
    orth_gemm(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
              const OrthGemm g, const DevCtl ctl) {
  using C = OrthCfg<BN>;
  constexpr int STAGES = C::kStages;
  constexpr uint32_t kIdesc = idesc_f16_f32(2 * kBM, BN, A_MN, B_MN);
  constexpr bool kSym = OP != kUpdate;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  OrthCtl<STAGES>* pc = reinterpret_cast<OrthCtl<STAGES>*>(smem + STAGES * C::kStageBytes);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1;
  const int npairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&pc->full[s], 1);
      mbar_init(&pc->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&pc->tfull[b], 1);
      mbar_init(&pc->tempty[b], 2 * 4 * kOrthWG);  // one arrive per epilogue warp, both CTAs
    }
    mbar_init(&pc->fin, 1);
    pc->abort = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    tmem_alloc_pair(&pc->tmem_base, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();  // both CTAs' barriers exist before either CTA touches the other's
  tc_fence_after();
  const uint32_t tmem = pc->tmem_base;
  volatile int* abort = &pc->abort;

  if (warp == 0) {
    // TMA producer (both CTAs); both CTAs' copies complete on the leader's "full" barrier.
    uint32_t it = 0;
    bool ok = true;
    for (int u = pair; ok && u < g.num_units; u += npairs) {
      int z, i, j;
      orth_unit<BN, kSym>(g, u, z, i, j);
      const int mrow = i * 2 * kBM + static_cast<int>(rank) * kBM;
      const int ncol = j * BN + static_cast<int>(rank) * C::kSliceN;
      for (int kb = 0; kb < g.k_blocks; ++kb, ++it) {
        const int s = it % STAGES;
        if (!wait_warp(&pc->empty[s], ((it / STAGES) & 1u) ^ 1u, abort, ctl)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          uint8_t* st = smem + s * C::kStageBytes;
          uint8_t* bst = st + C::kABytes;
          if (leader) mbar_arrive_expect_tx(&pc->full[s], 2 * C::kStageBytes);
          const int k0 = kb * kBK;
          if (A_MN) {
            tma_load_3d_pair(st, &tmA, &pc->full[s], mrow, k0, z);
            tma_load_3d_pair(st + 8192, &tmA, &pc->full[s], mrow + 64, k0, z);
          } else {
            tma_load_3d_pair(st, &tmA, &pc->full[s], k0, mrow, z);
          }
          if (B_MN) {
#pragma unroll
            for (int q = 0; q < C::kSliceN / 64; ++q)
              tma_load_3d_pair(bst + q * 8192, &tmB, &pc->full[s], ncol + q * 64, k0, z);
          } else {
            tma_load_3d_pair(bst, &tmB, &pc->full[s], k0, ncol, z);
          }
        }
        __syncwarp();
      }
    }
    if (ok) {
      // No remote release of a stage may reach this CTA after it has exited: wait for the
      // releases of the last stages.
      const uint32_t first = it > (uint32_t)STAGES ? it - STAGES : 0u;
      bool tail_ok = true;
      for (uint32_t q = first; tail_ok && q < it; ++q)
        tail_ok = wait_warp(&pc->empty[q % STAGES], (q / STAGES) & 1u, abort, ctl);
      if (!tail_ok)
        for (int q = 0; q < 100; ++q) __nanosleep(1000);
    } else if (leader) {
      // Let the pair's copies in flight land before either CTA leaves the final barrier.
      const uint32_t first = it > (uint32_t)STAGES ? it - STAGES : 0u;
      for (uint32_t q = first; q < it; ++q)
        wait_warp(&pc->full[q % STAGES], (q / STAGES) & 1u, abort, ctl, false);
    } else {
      for (int q = 0; q < 100; ++q) __nanosleep(1000);
    }
  } else if (warp == 1) {
    // MMA issuer (leader only).
    if (leader) {
      uint32_t it = 0, t = 0;
      bool ok = true;
      for (int u = pair; ok && u < g.num_units; u += npairs, ++t) {
        const int b = static_cast<int>(t & 1u);
        if (!wait_warp(&pc->tempty[b], ((t >> 1) & 1u) ^ 1u, abort, ctl)) break;
        tc_fence_after();
        const uint32_t dcol = tmem + b * BN;
        for (int kb = 0; kb < g.k_blocks; ++kb, ++it) {
          const int s = it % STAGES;
          if (!wait_warp(&pc->full[s], (it / STAGES) & 1u, abort, ctl)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (lane == 0) {
            const uint32_t a_addr = smem_u32(smem + s * C::kStageBytes);
            const uint32_t b_addr = a_addr + C::kABytes;
#pragma unroll
            for (int kk = 0; kk < kBK / 16; ++kk) {
              const uint64_t ad = A_MN ? smem_desc_sw128(a_addr + kk * 2048, 8192, 1024)
                                       : smem_desc_sw128(a_addr + kk * 32, 16, 1024);
              const uint64_t bd = B_MN ? smem_desc_sw128(b_addr + kk * 2048, 8192, 1024)
                                       : smem_desc_sw128(b_addr + kk * 32, 16, 1024);
              umma_bf16_pair(dcol, ad, bd, kIdesc, (kb | kk) != 0 ? 1u : 0u);
            }
            umma_commit_pair_mc(&pc->empty[s], 0x3);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (lane == 0) umma_commit_pair_mc(&pc->tfull[b], 0x3);
        __syncwarp();
      }
      // Every MMA must be complete (in both CTAs' TMEM) before TMEM is released.
      if (lane == 0) umma_commit_pair_mc(&pc->fin, 0x1);
      __syncwarp();
      wait_warp(&pc->fin, 0u, abort, ctl, false);
    }
  } else {
    // Epilogue (both CTAs).
    const int q = warp & 3;  // a warp may only touch TMEM lanes [32 * (warp % 4), +32)
    const int wg = (warp - 2) >> 2;
    const uint32_t lane_bits = static_cast<uint32_t>(q * 32) << 16;
    constexpr int kShare = BN / kOrthWG;
    const uint32_t tempty0 = mapa_shared(smem_u32(&pc->tempty[0]), 0);
    const uint32_t tempty1 = mapa_shared(smem_u32(&pc->tempty[1]), 0);
    uint32_t t = 0;
    for (int u = pair; u < g.num_units; u += npairs, ++t) {
      int z, i, j;
      orth_unit<BN, kSym>(g, u, z, i, j);
      const int b = static_cast<int>(t & 1u);
      if (!wait_warp(&pc->tfull[b], (t >> 1) & 1u, abort, ctl)) break;
      tc_fence_after();
      const int64_t row = static_cast<int64_t>(i) * 2 * kBM + rank * kBM + q * 32 + lane;
      const int64_t col0 = static_cast<int64_t>(j) * BN;
      const bool mirror = kSym && col0 + BN <= static_cast<int64_t>(i) * 2 * kBM;
#pragma unroll 1
      for (int c = wg * kShare; c < (wg + 1) * kShare; c += 32) {
        float v[32];
        tmem_ld32(tmem + lane_bits + b * BN + c, v);
        tmem_ld_wait();
        if (row < g.rows && col0 + c < g.cols)
          orth_epilogue<OP, LAST>(g, z, row, col0 + c, mirror, v);
      }
      tc_fence_before();
      __syncwarp();
      // Test hook (fault == 1): withhold the release of the first accumulator.
      if (lane == 0 && !(ctl.fault == 1 && t == 0)) mbar_arrive_cluster(b ? tempty1 : tempty0);
    }
  }

  // Neither CTA leaves while the other may still signal its barriers or use its TMEM.
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

template <int BN, bool A_MN, bool B_MN, int OP, bool LAST>
cudaError_t launch_orth(const CUtensorMap& a, const CUtensorMap& b, const OrthGemm& g,
                        const DevCtl& c, cudaStream_t s) {
  using C = OrthCfg<BN>;
  auto kern = orth_gemm<BN, A_MN, B_MN, OP, LAST>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(kOrthThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // Per device, once (later launches make no such calls, so that they can be captured).
  static int max_clusters[64] = {0};
  if (max_clusters[dev] == 0) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(C::kSmem));
    if (e != cudaSuccess) return e;
    int n = 0;
    cfg.gridDim = dim3(2 * 512, 1, 1);
    if ((e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg)) != cudaSuccess) return e;
    max_clusters[dev] = n > 0 ? n : 1;
  }
  cfg.gridDim = dim3(2 * std::max(1, std::min(g.num_units, max_clusters[dev])), 1, 1);
  return cudaLaunchKernelEx(&cfg, kern, a, b, g, c);
}

template <int BN>
cudaError_t launch_op(int op, bool tall, bool last, const CUtensorMap& a, const CUtensorMap& b,
                      const OrthGemm& g, const DevCtl& c, cudaStream_t s) {
  if (op == kGram)
    return tall ? launch_orth<BN, true, true, kGram, false>(a, b, g, c, s)
                : launch_orth<BN, false, false, kGram, false>(a, b, g, c, s);
  if (op == kSquare) return launch_orth<BN, false, false, kSquare, false>(a, b, g, c, s);
  if (tall)
    return last ? launch_orth<BN, false, false, kUpdate, true>(a, b, g, c, s)
                : launch_orth<BN, false, false, kUpdate, false>(a, b, g, c, s);
  return last ? launch_orth<BN, false, true, kUpdate, true>(a, b, g, c, s)
              : launch_orth<BN, false, true, kUpdate, false>(a, b, g, c, s);
}

}  // namespace

cudaError_t launch_orth_prep(int dtype, const OrthPrep& p, int64_t batch, cudaStream_t s) {
  const int64_t blocks = std::min<int64_t>(p.m, kOrthSums);
  const dim3 g1(static_cast<unsigned>(blocks), static_cast<unsigned>(batch));
  const dim3 g2(static_cast<unsigned>(std::min<int64_t>(p.m, 4096)), static_cast<unsigned>(batch));
  auto run = [&](auto t) {
    using T = decltype(t);
    orth_moment<T><<<g1, kPrepThreads, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    orth_scale<T><<<g2, kPrepThreads, 0, s>>>(p, static_cast<int>(blocks));
    return cudaGetLastError();
  };
  if (dtype == 0) return run(__nv_bfloat16{});
  if (dtype == 1) return run(__half{});
  return run(float{});
}

cudaError_t launch_orth_gemm(int op, int bn, bool tall, bool last, const CUtensorMap& a,
                             const CUtensorMap& b, const OrthGemm& g, const DevCtl& c,
                             cudaStream_t s) {
  return bn == 128 ? launch_op<128>(op, tall, last, a, b, g, c, s)
                   : launch_op<256>(op, tall, last, a, b, g, c, s);
}

}  // namespace slm
