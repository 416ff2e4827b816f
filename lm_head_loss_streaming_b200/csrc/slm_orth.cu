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
// fp32 accumulators.  Three choices keep the result of five steps within about 1.4e-3 of the exact
// iteration (a later step adds 2e-4 to 3e-4; directions that the gradient lacks hold rounding noise,
// which the product of the steps' a multiplies, as in fp32):
//   - X is held as hi + lo, two fp16 numbers (22 bits).  Products use hi; the term a X, which
//     carries the small singular directions through, uses both.
//   - A and B are held as a diagonal in fp32 and fp16 off-diagonal entries (zero diagonal).
//     The diagonals of A and B are their largest and nearly equal entries, so that rounding
//     them is one common error, which the polynomial amplifies; apart, they cost one fused
//     multiply-add in the epilogues:  with A = D + R,
//         A^2 = R R + (D_i + D_j) R + D^2,    B X = R_B hi + D_B hi.
//     (D_B multiplies hi, not hi + lo: B must act on one and the same X in all its terms, or
//     the difference's noise reaches directions that B alone would not touch.  orth_small has
//     room for B (hi + lo) where k <= 128.)
//   - hi, lo and the matrices are stored times a power of two (kScaleX, kScaleA, kScaleB), so
//     that fp16's exponent range covers them: |X|, |A| < 4 and |B| < 16 fit, which the host
//     checks of the coefficients, and entries down to 2^-28 are normal numbers.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "slm_internal.h"
#include "slm_ran_out.cuh"
#include "slm_wait.cuh"
#include "sm100.cuh"

namespace slm {
namespace {
using namespace sm100;

constexpr float kScaleX = 16384.f;  // 2^14
constexpr float kScaleA = 16384.f;
constexpr float kScaleB = 4096.f;  // 2^12

constexpr int kPrepThreads = 256;

// V consecutive elements (V = 8: whole 16-byte pieces; V = 1).
template <class T, int V>
__device__ __forceinline__ void ld_elems(const T* p, float (&v)[V]) {
  if constexpr (V == 1) {
    if constexpr (std::is_same_v<T, float>)
      v[0] = *p;
    else if constexpr (std::is_same_v<T, __half>)
      v[0] = __half2float(*p);
    else
      v[0] = __bfloat162float(*p);
  } else if constexpr (std::is_same_v<T, float>) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 f;
      if constexpr (std::is_same_v<T, __half>)
        f = __half22float2(*reinterpret_cast<const __half2*>(&a[i]));
      else
        f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&a[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}

// Where group `i` of V elements of a matrix lies in the gradient, in the momentum (contiguous)
// and in hi / lo (rows of ldx).
struct OrthAt {
  int64_t grad, mom, x;
};
template <int V>
__device__ __forceinline__ OrthAt orth_at(const OrthPrep& p, int64_t b, int64_t i) {
  const int64_t per_row = p.n / V;
  int64_t r, c;
  if (p.m * per_row < (int64_t(1) << 32)) {
    r = static_cast<uint32_t>(i) / static_cast<uint32_t>(per_row);
    c = static_cast<uint32_t>(i) - static_cast<uint32_t>(r) * static_cast<uint32_t>(per_row);
  } else {
    r = i / per_row;
    c = i - r * per_row;
  }
  c *= V;
  return {b * p.grad_batch + r * p.ldg + c, (b * p.m + r) * p.n + c, (b * p.m + r) * p.ldx + c};
}

// Momentum update and the partial sums of u^2 (64 bits: the squares of fp32 gradients may
// leave fp32's range).  Blocks (., b) share matrix b.
template <class T, int V>
__global__ void __launch_bounds__(kPrepThreads) orth_moment(const OrthPrep p) {
  const int64_t b = blockIdx.y;
  const int64_t groups = p.m * (p.n / V);
  if (blockIdx.x == 0 && b == 0 && threadIdx.x == 0) {
    *p.status = 0;
    *p.counter = 0;
  }
  double s = 0.0;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kPrepThreads + threadIdx.x; i < groups;
       i += static_cast<int64_t>(gridDim.x) * kPrepThreads) {
    const OrthAt at = orth_at<V>(p, b, i);
    float u[V];
    ld_elems<T, V>(static_cast<const T*>(p.grad) + at.grad, u);
    if (p.momentum) {
      float mom[V];
      ld_elems<float, V>(p.momentum + at.mom, mom);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        mom[e] = p.beta * mom[e] + p.rest * u[e];
        u[e] = p.nesterov ? p.beta * mom[e] + p.rest * u[e] : mom[e];
      }
      if constexpr (V == 8) {
        float4* o = reinterpret_cast<float4*>(p.momentum + at.mom);
        o[0] = make_float4(mom[0], mom[1], mom[2], mom[3]);
        o[1] = make_float4(mom[4], mom[5], mom[6], mom[7]);
      } else {
        p.momentum[at.mom] = mom[0];
      }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) s = fma(static_cast<double>(u[e]), static_cast<double>(u[e]), s);
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

// The scale kScaleX / (||u|| + eps) as two factors to multiply by in turn, the first a power of
// two: the scale itself may leave fp32's range where u nearly does.
__device__ __forceinline__ float2 orth_factors(double sum, float eps) {
  const double s = kScaleX / (sqrt(sum) + static_cast<double>(eps));
  const float pre = s > 1e30 ? 0x1p64f : s < 1e-30 ? 0x1p-64f : 1.f;
  return make_float2(pre, static_cast<float>(s / pre));
}

// X = u / (||u|| + eps) as hi + lo; the norm from the partial sums, added in a fixed order.
template <class T, int V>
__global__ void __launch_bounds__(kPrepThreads) orth_scale(const OrthPrep p, int nsums) {
  __shared__ float2 inv_sh;
  const int64_t b = blockIdx.y;
  if (threadIdx.x < 32) {
    double t = 0.0;
    for (int i = threadIdx.x; i < nsums; i += 32) t += p.sums[b * kOrthSums + i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (threadIdx.x == 0)
      inv_sh = orth_factors(t, p.eps);
  }
  __syncthreads();
  const float2 inv = inv_sh;
  const int64_t groups = p.m * (p.n / V);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kPrepThreads + threadIdx.x; i < groups;
       i += static_cast<int64_t>(gridDim.x) * kPrepThreads) {
    const OrthAt at = orth_at<V>(p, b, i);
    float u[V];
    ld_elems<T, V>(static_cast<const T*>(p.grad) + at.grad, u);
    if (p.momentum) {
      float mom[V];
      ld_elems<float, V>(p.momentum + at.mom, mom);
#pragma unroll
      for (int e = 0; e < V; ++e) u[e] = p.nesterov ? p.beta * mom[e] + p.rest * u[e] : mom[e];
    }
    alignas(16) __half hi[V], lo[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float x = u[e] * inv.x * inv.y;
      hi[e] = __float2half_rn(x);
      lo[e] = __float2half_rn(x - __half2float(hi[e]));
    }
    if constexpr (V == 8) {
      *reinterpret_cast<uint4*>(p.hi + at.x) = *reinterpret_cast<const uint4*>(hi);
      *reinterpret_cast<uint4*>(p.lo + at.x) = *reinterpret_cast<const uint4*>(lo);
    } else {
      p.hi[at.x] = hi[0];
      p.lo[at.x] = lo[0];
    }
  }
}

// ----------------------------------------------------------------------------------------
// The products: all of them in one cooperative launch of 2-SM GEMMs (M = 256 rows per CTA pair,
// fp16 operands).  Warp 0 loads, warp 1 issues the MMAs, eight warps run the epilogue, each
// warpgroup over half of a slot's columns (sixteen, with 96 registers a thread, made 2048 x 2048
// 10% slower and 1024 x 1024 6%).  Operands are K-major or MN-major as they lie in memory, so that
// no transpose of X is ever stored.  Per step:
//   kGram    R, D of A = X X^T:  a symmetric product, only blocks on and below the diagonal
//            are computed and each is written to its mirrored place too
//   kSquare  R_B, D_B of B = b A + c A^2, symmetric in the same way
//   kUpdate  hi, lo of a X + B X; in the last step the result in bf16
// A product reads what the one before wrote anywhere, so the CTAs meet between products (a
// counter in the workspace, bounded waits; the cooperative launch makes them all resident).
// A meeting costs about 2 us, a launch of its own with its set-up and drain 7 us.
// Where the Gram product has few tiles over a long K (SPLIT), a tile's K blocks are shared out
// over several pairs, whose fp32 sums go to memory; after another meeting every epilogue warp of
// the launch adds blocks' parts in order and finishes them.  Five steps with and without:
// 300 x 8192 174 and 333 us, 100 x 8192 126 and 286, 1024 x 8192 309 and 474, eight of 100 x 4000
// 188 and 251, 64 x 2048 98 and 120.
// The tensor memory holds two accumulator slots of BNI columns.  NSUB = 1: tiles take the slots
// in turn, so that a tile's epilogue overlaps the next tile's MMAs.  NSUB = 2: a tile of 512
// columns takes both; the operands then cross from L2 at 170 instead of 128 flops per byte, and
// L2 is what bounds these products (about 9.3 TB/s measured over the 74 pairs: 256-column
// tiles reach 1.2 PFLOP/s).  The next tile's MMAs for the first slot start while the epilogue
// still drains the second.
// Where every pair has at most one tile of the update (NSUB = 1; up to 74 tiles of 256 x 256),
// hi and lo of that tile stay in the second slot from step to step, two fp16 numbers per
// 32-bit cell: only hi goes to memory, for the products to read.
// ----------------------------------------------------------------------------------------
enum OrthOp { kGram = 0, kSquare = 1, kUpdate = 2, kJoin = 3 };
constexpr int kOrthWG = 2;
constexpr int kOrthThreads = 64 + 128 * kOrthWG;
// Meeting of the CTAs between products.
__device__ __forceinline__ int ld_acquire_s32(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void red_release_add_s32(int* p, int v) {
  asm volatile("red.release.gpu.global.add.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ void fence_proxy_async_all() {
  asm volatile("fence.proxy.async;" ::: "memory");
}
__device__ __forceinline__ void fence_proxy_async_global() {
  asm volatile("fence.proxy.async.global;" ::: "memory");
}
// Waits (boundedly; lane 0 polls) until `target` arrivals are counted; what the arriving CTAs
// wrote is then visible to this thread's loads and bulk copies.
__device__ __forceinline__ bool wait_met(const int* counter, int target, volatile int* abort,
                                         const DevCtl& ctl) {
  int ok = 1;
  if ((threadIdx.x & 31) == 0) {
    const long long t0 = clock64();
    while (ld_acquire_s32(counter) < target) {
      if (*abort) {
        ok = 0;
        break;
      }
      if (clock64() - t0 > ctl.timeout_cycles) {
        *abort = 1;
        atomicOr(ctl.status, kFlagTimeout);
        ok = 0;
        break;
      }
    }
    fence_proxy_async_global();
  }
  return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

// Staging of an epilogue warp: a block of 32 rows x 32 fp16 columns, 64 bytes per row, with
// 16-byte piece k of row r at k ^ (r / 2 % 4), so that neither a lane per row nor four lanes
// per row conflict.
constexpr int kOrthStage = 2048;
__device__ __forceinline__ int stage_piece(int row, int k) {
  return row * 4 + (k ^ ((row >> 1) & 3));
}

template <int STAGES>
struct OrthCtl {
  uint64_t full[STAGES], empty[STAGES], tfull[2], tempty[2], fin, met, done;
  uint32_t tmem_base;
  int abort;
};

template <int BNI, int NSUB>
struct OrthCfg {
  static constexpr int kTileN = BNI * NSUB;
  static constexpr int kSliceN = BNI / 2;  // columns of a slot whose operand rows each CTA holds
  static constexpr uint32_t kABytes = kBM * kBK * 2;
  static constexpr uint32_t kSliceBytes = kSliceN * kBK * 2;
  static constexpr uint32_t kStageBytes = kABytes + NSUB * kSliceBytes;
  static constexpr int kStages = NSUB == 2 ? 4 : BNI == 256 ? 6 : 8;
  static constexpr size_t kRing = kStages * static_cast<size_t>(kStageBytes);
  static constexpr size_t kSmem =
      1024 + kRing + 4 * kOrthWG * kOrthStage + sizeof(OrthCtl<kStages>);
  static_assert(kSmem <= 232448, "shared memory per CTA");
};

// Tile of unit u: matrix z, pair row tile i, column tile j, and how many of its slots' columns
// are wanted (of a symmetric product, the blocks right of the diagonal are not).
template <int BNI, int NSUB, bool SYM>
__device__ __forceinline__ void orth_unit(const OrthGeom& g, int u, int& z, int& i, int& j,
                                          int& nsub) {
  z = u / g.units_per;
  const int t = u - z * g.units_per;
  nsub = NSUB;
  if (SYM && NSUB == 2) {
    // Row tile i has i / 2 + 1 column tiles; rows before it (i + 1)^2 / 4.
    i = max(0, static_cast<int>(2.f * sqrtf(static_cast<float>(t))) - 1);
    while ((i + 1) * (i + 1) / 4 > t) --i;
    while ((i + 2) * (i + 2) / 4 <= t) ++i;
    j = t - (i + 1) * (i + 1) / 4;
    nsub = min(2, i + 1 - 2 * j);
  } else if (SYM) {
    // Row tile i has W (i + 1) column tiles, W = 256 / BNI; rows before it W i (i + 1) / 2.
    constexpr int W = 256 / BNI;
    i = static_cast<int>((sqrtf(8.f / W * t + 1.f) - 1.f) * 0.5f);
    while (W * i * (i + 1) / 2 > t) --i;
    while (W * (i + 1) * (i + 2) / 2 <= t) ++i;
    j = t - W * i * (i + 1) / 2;
  } else {
    const int per_group = kOrthGroup * g.num_n;
    const int grp = t / per_group;
    const int r = t - grp * per_group;
    const int gm = min(kOrthGroup, g.num_m - grp * kOrthGroup);
    j = r / gm;
    i = grp * kOrthGroup + (r - j * gm);
  }
}

// Part of a product's K blocks that unit u covers: its first block and their number; u becomes the
// tile's number.
template <bool SPLIT>
__device__ __forceinline__ int orth_part(const OrthGeom& g, int& u, int& kb0) {
  kb0 = 0;
  if (!SPLIT) return g.k_blocks;
  const int tiles = g.num_units / g.split, part = u / tiles;
  u -= part * tiles;
  kb0 = part * g.part_blocks;
  return min(g.part_blocks, g.k_blocks - kb0);
}

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half2(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ uint32_t pack_bf162(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// A warp's block, rows [row0, row0 + 32) and columns [col, col + 32) of a matrix at `src` whose
// rows are padded to whole 16-byte pieces: four lanes per row, so that every access covers whole
// 64-byte runs of rows, ...
struct OrthBlock {
  uint4 w[4];
  __device__ __forceinline__ void load(const __half* src, int64_t ld, int row0, int col, int rows,
                                       int cols, int lane) {
    const int c = col + (lane & 3) * 8, row = row0 + (lane >> 2);
    const uint4* at = reinterpret_cast<const uint4*>(src + row * ld + c);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      w[q] = row + q * 8 < rows && c < cols ? at[q * ld] : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void store(void* dst, int64_t ld, int row0, int col, int rows,
                                        int cols, int lane) const {
    const int c = col + (lane & 3) * 8, row = row0 + (lane >> 2);
    uint4* at = reinterpret_cast<uint4*>(static_cast<uint16_t*>(dst) + row * ld + c);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (row + q * 8 < rows && c < cols) at[q * ld] = w[q];
  }
  // ... turned through the staging into a lane per row and back.
  __device__ __forceinline__ void to_rows(uint4* stage, int lane, uint32_t (&r)[16]) const {
#pragma unroll
    for (int q = 0; q < 4; ++q) stage[stage_piece(q * 8 + (lane >> 2), lane & 3)] = w[q];
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint4 v = stage[stage_piece(lane, q)];
      r[4 * q] = v.x;
      r[4 * q + 1] = v.y;
      r[4 * q + 2] = v.z;
      r[4 * q + 3] = v.w;
    }
    __syncwarp();
  }
  __device__ __forceinline__ void from_rows(uint4* stage, int lane, const uint32_t (&r)[16],
                                            bool zero_diagonal = false) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      stage[stage_piece(lane, q)] = make_uint4(r[4 * q], r[4 * q + 1], r[4 * q + 2], r[4 * q + 3]);
    if (zero_diagonal)
      reinterpret_cast<uint16_t*>(stage)[stage_piece(lane, lane >> 3) * 8 + (lane & 7)] = 0;
    __syncwarp();
    read(stage, lane);
  }
  __device__ __forceinline__ void read(const uint4* stage, int lane) {
#pragma unroll
    for (int q = 0; q < 4; ++q) w[q] = stage[stage_piece(q * 8 + (lane >> 2), lane & 3)];
    __syncwarp();
  }
};

// What a block's epilogue reads, fetched a block ahead (behind the MMAs, or the block before).
// FROM: hi and lo of the update come from tensor memory instead.
template <int OP, bool TALL, bool FROM>
struct OrthIn {
  static constexpr bool kCols = OP == kSquare || (OP == kUpdate && TALL);  // D of the columns
  OrthBlock hi, lo;  // kSquare: R in hi
  float dcol;        // lane l: the diagonal's entry of column col + l
  __device__ __forceinline__ void fetch(const OrthView& g, int z, int row0, int col, int lane) {
    if (OP == kGram) return;
    const int64_t base = static_cast<int64_t>(z) * g.rows * g.ld;
    if (OP == kSquare || !FROM) {
      hi.load(g.in + base, g.ld, row0, col, g.rows, g.cols, lane);
      if (OP == kUpdate) lo.load(g.lo + base, g.ld, row0, col, g.rows, g.cols, lane);
    }
    if (kCols)
      dcol = col + lane < g.cols ? g.diag_in[static_cast<int64_t>(z) * g.diag_n + col + lane] : 0.f;
  }
};

// One warp's block of product OP: v holds this lane's row `row`, columns [col, col + 32) of the
// accumulator of matrix z.  (Bulk stores from the staging measured slower: a block waited about
// 0.7 us for the one before to be read.)
// FROM, TO: hi and lo of the update's tile are read from / left in tensor memory at `master`.
template <int OP, bool LAST, bool TALL, bool FROM, bool TO>
__device__ __forceinline__ void orth_epilogue(const OrthView& g, uint4* stage, int z, int row,
                                              int col, int next_col, bool mirror, float drow,
                                              OrthIn<OP, TALL, FROM>& in, uint32_t master,
                                              float (&v)[32]) {
  constexpr bool kCols = OrthIn<OP, TALL, FROM>::kCols;
  const int lane = threadIdx.x & 31;
  const int row0 = row - lane;
  const int64_t base = static_cast<int64_t>(z) * g.rows * g.ld;
  uint32_t hi[16], lo[16];
  OrthBlock blk;
  if (OP != kGram) {
    if (FROM) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t w[16];
        tmem_ld16_raw(master + 16 * half, w);
        tmem_ld_wait();
#pragma unroll
        for (int h = 0; h < 8; ++h) {
          hi[8 * half + h] = __byte_perm(w[2 * h], w[2 * h + 1], 0x5410);
          lo[8 * half + h] = __byte_perm(w[2 * h], w[2 * h + 1], 0x7632);
        }
      }
    } else {
      in.hi.to_rows(stage, lane, hi);
      if (OP == kUpdate) in.lo.to_rows(stage, lane, lo);
    }
    if (kCols) {
      reinterpret_cast<float*>(stage)[lane] = in.dcol;
      __syncwarp();
    }
    if (next_col >= 0) in.fetch(g, z, row0, next_col, lane);
  }
  const float4* d4 = reinterpret_cast<const float4*>(stage);
#pragma unroll
  for (int h = 0; h < 16; ++h) {  // a pair of columns
    const float2 x = make_float2(v[2 * h], v[2 * h + 1]);
    float2 d = both(drow);
    if (kCols) {
      const float4 f = d4[h / 2];
      d = h & 1 ? make_float2(f.z, f.w) : make_float2(f.x, f.y);
    }
    if (OP == kGram) {
      const float2 r = __fmul2_rn(x, both(kScaleA / (kScaleX * kScaleX)));
      hi[h] = pack_half2(r.x, r.y);
    } else if (OP == kSquare) {
      // scaled c (R R + (D_i + D_j) R) + b R
      const float2 t = __ffma2_rn(both(g.c * (kScaleB / kScaleA)), d,
                                  both(fmaf(g.c, drow, g.b) * (kScaleB / kScaleA)));
      const float2 r = __ffma2_rn(unpack_half2(hi[h]), t,
                                  __fmul2_rn(x, both(g.c * (kScaleB / (kScaleA * kScaleA)))));
      hi[h] = pack_half2(r.x, r.y);
    } else {
      const float2 r = __ffma2_rn(x, both(1.f / kScaleB),
                                  __ffma2_rn(unpack_half2(hi[h]), __fadd2_rn(d, both(g.a)),
                                             __fmul2_rn(unpack_half2(lo[h]), both(g.a))));
      if (LAST) {
        hi[h] = pack_bf162(r.x * (1.f / kScaleX), r.y * (1.f / kScaleX));
      } else {
        hi[h] = pack_half2(r.x, r.y);
        const float2 f = unpack_half2(hi[h]);
        lo[h] = pack_half2(r.x - f.x, r.y - f.y);
      }
    }
  }
  if (kCols) __syncwarp();  // the staging is free again
  if (OP != kUpdate && row0 == col) {
    // The block on the diagonal: this lane's diagonal element goes to the fp32 diagonal, a zero
    // takes its place.  (Selected, not branched to: a branch per lane took 3 us.)
    float x = 0.f;
#pragma unroll
    for (int c = 0; c < 32; ++c) x = c == lane ? v[c] : x;
    if (row < g.rows)
      g.diag_out[static_cast<int64_t>(z) * g.diag_n + row] =
          OP == kGram ? x * (1.f / (kScaleX * kScaleX))
                      : fmaf(g.c, fmaf(drow, drow, x * (1.f / (kScaleA * kScaleA))), g.b * drow);
  }
  if (LAST && !g.out_vec) {
    // Rows of the result that do not start on 16-byte boundaries: element stores, a row per
    // instruction.
#pragma unroll
    for (int q = 0; q < 4; ++q)
      stage[stage_piece(lane, q)] = make_uint4(hi[4 * q], hi[4 * q + 1], hi[4 * q + 2], hi[4 * q + 3]);
    __syncwarp();
    const uint16_t* el = reinterpret_cast<const uint16_t*>(stage);
    uint16_t* dst = static_cast<uint16_t*>(g.out) +
                    (static_cast<int64_t>(z) * g.rows + row0) * g.cols + col + lane;
    const int rows = min(32, g.rows - row0);
    if (col + lane < g.cols)
      for (int r = 0; r < rows; ++r)
        dst[static_cast<int64_t>(r) * g.cols] = el[stage_piece(r, lane >> 3) * 8 + (lane & 7)];
    __syncwarp();
    return;
  }
  const int64_t out_ld = LAST ? g.cols : g.ld;
  uint16_t* out = static_cast<uint16_t*>(g.out) + static_cast<int64_t>(z) * g.rows * out_ld;
  blk.from_rows(stage, lane, hi, OP != kUpdate && row0 == col);
  blk.store(out, out_ld, row0, col, g.rows, g.cols, lane);
  if (OP == kUpdate && !LAST) {
    if (TO) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t w[16];
#pragma unroll
        for (int h = 0; h < 8; ++h) {
          w[2 * h] = __byte_perm(hi[8 * half + h], lo[8 * half + h], 0x5410);
          w[2 * h + 1] = __byte_perm(hi[8 * half + h], lo[8 * half + h], 0x7632);
        }
        tmem_st16_raw(master + 16 * half, w);
      }
      tmem_st_wait();
    } else {
      blk.from_rows(stage, lane, lo);
      blk.store(g.lo + base, g.ld, row0, col, g.rows, g.cols, lane);
    }
  }
  if (OP != kUpdate && mirror) {
    // The transpose: column c of the block as row c, a lane per element.
    uint16_t* t = reinterpret_cast<uint16_t*>(stage);
#pragma unroll
    for (int c = 0; c < 32; ++c)
      t[stage_piece(c, lane >> 3) * 8 + (lane & 7)] =
          static_cast<uint16_t>(c & 1 ? hi[c / 2] >> 16 : hi[c / 2]);
    __syncwarp();
    blk.read(stage, lane);
    blk.store(out, out_ld, col, row0, g.cols, g.rows, lane);
  }
}

// SPLIT: the Gram product's K is split (ch.geom[kGram].split > 1).
template <int BNI, int NSUB, bool TALL, bool SPLIT>
__global__ void __launch_bounds__(kOrthThreads, 1)
    orth_chain(const __grid_constant__ OrthChain ch, const __grid_constant__ OrthMaps maps,
               const DevCtl ctl) {
  using C = OrthCfg<BNI, NSUB>;
  constexpr int STAGES = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  OrthCtl<STAGES>* pc =
      reinterpret_cast<OrthCtl<STAGES>*>(smem + C::kRing + 4 * kOrthWG * kOrthStage);
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
    mbar_init(&pc->met, 1);
    mbar_init(&pc->done, 4 * kOrthWG);
    pc->abort = 0;
    fence_barrier_init();
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
  // Phases of a step: the products, and a join after a Gram product whose K is split.
  constexpr int per_step = SPLIT ? 4 : 3;
  const int phases = per_step * ch.steps;
  auto phase_op = [&](int p) {
    const int r = p % per_step;
    return !SPLIT || r == 0 ? r : r == 1 ? static_cast<int>(kJoin) : r - 1;
  };

  if (warp == 0) {
    // TMA producer (both CTAs); both CTAs' copies complete on the leader's "full" barrier.
    uint32_t it = 0;
    bool ok = true;
    auto product = [&](auto opc, int cur) {
      constexpr int OP = decltype(opc)::value;
      constexpr bool A_MN = TALL && OP == kGram;
      constexpr bool B_MN = (TALL && OP == kGram) || (!TALL && OP == kUpdate);
      const OrthGeom& g = ch.geom[OP];
      const CUtensorMap* ma = &maps.a[OP][cur];
      const CUtensorMap* mb = &maps.b[OP][cur];
      for (int u = pair; ok && u < g.num_units; u += npairs) {
        int z, i, j, nsub, tile = u, kb0;
        const int blocks = orth_part<SPLIT && OP == kGram>(g, tile, kb0);
        orth_unit<BNI, NSUB, OP != kUpdate>(g, tile, z, i, j, nsub);
        const int mrow = i * 2 * kBM + static_cast<int>(rank) * kBM;
        for (int kb = kb0; kb < kb0 + blocks; ++kb, ++it) {
          const int s = it % STAGES;
          if (!wait_warp(&pc->empty[s], ((it / STAGES) & 1u) ^ 1u, abort, ctl)) {
            ok = false;
            break;
          }
          if (lane == 0) {
            uint8_t* st = smem + s * C::kStageBytes;
            if (leader)
              mbar_arrive_expect_tx(&pc->full[s], 2 * (C::kABytes + nsub * C::kSliceBytes));
            const int k0 = kb * kBK;
            if (A_MN) {
              tma_load_3d_pair(st, ma, &pc->full[s], mrow, k0, z);
              tma_load_3d_pair(st + 8192, ma, &pc->full[s], mrow + 64, k0, z);
            } else {
              tma_load_3d_pair(st, ma, &pc->full[s], k0, mrow, z);
            }
#pragma unroll
            for (int h = 0; h < NSUB; ++h) {
              if (h >= nsub) break;
              uint8_t* bst = st + C::kABytes + h * C::kSliceBytes;
              const int ncol = j * C::kTileN + h * BNI + static_cast<int>(rank) * C::kSliceN;
              if (B_MN) {
#pragma unroll
                for (int q = 0; q < C::kSliceN / 64; ++q)
                  tma_load_3d_pair(bst + q * 8192, mb, &pc->full[s], ncol + q * 64, k0, z);
              } else {
                tma_load_3d_pair(bst, mb, &pc->full[s], k0, ncol, z);
              }
            }
          }
          __syncwarp();
        }
      }
    };
    for (int p = 0; ok && p < phases; ++p) {
      if (p > 0) {
        // This CTA's part of the product before is in memory; wait for the others' and let the
        // epilogue know.
        ok = wait_warp(&pc->done, (p - 1) & 1, abort, ctl);
        if (ok) {
          if (lane == 0) red_release_add_s32(ch.counter, 1);
          __syncwarp();
          ok = wait_met(ch.counter, p * static_cast<int>(gridDim.x), abort, ctl);
        }
        if (lane == 0) mbar_arrive(&pc->met);
        __syncwarp();
        if (!ok) break;
      }
      const int step = p / per_step, op = phase_op(p);
      if (op == kGram)
        product(std::integral_constant<int, kGram>{}, step & 1);
      else if (op == kSquare)
        product(std::integral_constant<int, kSquare>{}, 0);
      else if (op == kUpdate)
        product(std::integral_constant<int, kUpdate>{}, step & 1);
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
      uint32_t it = 0, t = 0, used0 = 0, used1 = 0;
      bool ok = true;
      auto product = [&](auto opc) {
        constexpr int OP = decltype(opc)::value;
        constexpr bool A_MN = TALL && OP == kGram;
        constexpr bool B_MN = (TALL && OP == kGram) || (!TALL && OP == kUpdate);
        constexpr uint32_t kIdesc = idesc_f16_f32(2 * kBM, BNI, A_MN, B_MN);
        const OrthGeom& g = ch.geom[OP];
        // The MMAs of stage `st` into slot b (operand slice h); first = the tile's first K block.
        auto issue = [&](int st, int h, int b, bool first) {
          const uint32_t a_addr = smem_u32(smem + st * C::kStageBytes);
          const uint32_t b_addr = a_addr + C::kABytes + h * C::kSliceBytes;
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk) {
            const uint64_t ad = A_MN ? smem_desc_sw128(a_addr + kk * 2048, 8192, 1024)
                                     : smem_desc_sw128(a_addr + kk * 32, 16, 1024);
            const uint64_t bd = B_MN ? smem_desc_sw128(b_addr + kk * 2048, 8192, 1024)
                                     : smem_desc_sw128(b_addr + kk * 32, 16, 1024);
            umma_bf16_pair(tmem + b * BNI, ad, bd, kIdesc, (!first || kk != 0) ? 1u : 0u);
          }
        };
        for (int u = pair; u < g.num_units; u += npairs, ++t) {
          int z, i, j, nsub, tile = u, kb0;
          const int blocks = orth_part<SPLIT && OP == kGram>(g, tile, kb0);
          orth_unit<BNI, NSUB, OP != kUpdate>(g, tile, z, i, j, nsub);
          const int b0 = NSUB == 2 || ch.resident ? 0 : static_cast<int>(t & 1u);
          uint32_t& used = b0 ? used1 : used0;
          ok = wait_warp(&pc->tempty[b0], (used & 1u) ^ 1u, abort, ctl);
          if (!ok) return;
          ++used;
          tc_fence_after();
          int kb = 0;
          if (NSUB == 2 && nsub == 2) {
            // The first slot over the stages that are there already, then, once the second
            // slot is free, its MMAs for them, with the stages' releases.
            const int pre = min(STAGES, blocks);
            for (; kb < pre; ++kb) {
              const uint32_t q = it + kb;
              ok = wait_warp(&pc->full[q % STAGES], (q / STAGES) & 1u, abort, ctl);
              if (!ok) return;
              tc_fence_after();
              if (lane == 0) issue(q % STAGES, 0, 0, kb == 0);
              __syncwarp();
            }
            ok = wait_warp(&pc->tempty[1], (used1 & 1u) ^ 1u, abort, ctl);
            if (!ok) return;
            ++used1;
            tc_fence_after();
            for (int q = 0; q < pre; ++q, ++it) {
              if (lane == 0) {
                issue(it % STAGES, 1, 1, q == 0);
                umma_commit_pair_mc(&pc->empty[it % STAGES], 0x3);
              }
              __syncwarp();
            }
          }
          for (; kb < blocks; ++kb, ++it) {
            const int s = it % STAGES;
            ok = wait_warp(&pc->full[s], (it / STAGES) & 1u, abort, ctl);
            if (!ok) return;
            tc_fence_after();
            if (lane == 0) {
              issue(s, 0, b0, kb == 0);
              if (NSUB == 2 && nsub == 2) issue(s, 1, 1, false);
              umma_commit_pair_mc(&pc->empty[s], 0x3);
            }
            __syncwarp();
          }
          if (lane == 0) {
            umma_commit_pair_mc(&pc->tfull[b0], 0x3);
            if (NSUB == 2 && nsub == 2) umma_commit_pair_mc(&pc->tfull[1], 0x3);
          }
          __syncwarp();
        }
      };
      for (int p = 0; ok && p < phases; ++p) {
        const int op = phase_op(p);
        if (op == kGram)
          product(std::integral_constant<int, kGram>{});
        else if (op == kSquare)
          product(std::integral_constant<int, kSquare>{});
        else if (op == kUpdate)
          product(std::integral_constant<int, kUpdate>{});
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
    constexpr int kShare = BNI / kOrthWG, kChunks = kShare / 32;
    uint4* stage = reinterpret_cast<uint4*>(smem + C::kRing + (warp - 2) * kOrthStage);
    const uint32_t tempty0 = mapa_shared(smem_u32(&pc->tempty[0]), 0);
    const uint32_t tempty1 = mapa_shared(smem_u32(&pc->tempty[1]), 0);
    uint32_t t = 0, used0 = 0, used1 = 0;
    bool ok = true;
    // Where block (rows, cols) of 32 x 32 of unit u's partial sums lies.
    auto part_block = [&](int u, int rows, int cols) {
      return reinterpret_cast<float4*>(ch.parts) +
             ((static_cast<int64_t>(u) * 8 + rows) * (BNI / 32) + cols) * 256;
    };
    auto product = [&](auto opc, auto lastc, auto fromc, auto toc, int step) {
      constexpr int OP = decltype(opc)::value;
      constexpr bool LAST = decltype(lastc)::value;
      constexpr bool FROM = decltype(fromc)::value, TO = decltype(toc)::value;
      constexpr bool kSym = OP != kUpdate;
      const OrthGeom& geo = ch.geom[OP];
      const int cur = step & 1;
      const OrthView g{OP == kUpdate ? ch.m : ch.k, OP == kUpdate ? ch.n : ch.k,
                       OP == kUpdate ? ch.ldx : ch.ldk, ch.k,
                       OP == kUpdate ? ch.hi[cur] : ch.mat[0], ch.lo,
                       OP == kSquare ? ch.diag[0] : ch.diag[1],
                       OP == kGram ? ch.diag[0] : ch.diag[1],
                       OP == kGram     ? static_cast<void*>(ch.mat[0])
                       : OP == kSquare ? static_cast<void*>(ch.mat[1])
                       : LAST          ? static_cast<void*>(ch.out)
                                       : static_cast<void*>(ch.hi[cur ^ 1]),
                       ch.co[step][0],
                       ch.co[step][1], ch.co[step][2], ch.out_vec};
      for (int u = pair; ok && u < geo.num_units; u += npairs, ++t) {
        int z, i, j, nsub, tile = u, kb0;
        orth_part<SPLIT && OP == kGram>(geo, tile, kb0);
        orth_unit<BNI, NSUB, kSym>(geo, tile, z, i, j, nsub);
        const int row = i * 2 * kBM + static_cast<int>(rank) * kBM + q * 32 + lane;
        float drow = 0.f;
        if (OP == kSquare || (OP == kUpdate && !TALL))
          if (row < g.rows) drow = g.diag_in[static_cast<int64_t>(z) * g.diag_n + row];
        for (int h = 0; h < nsub; ++h) {
          const int b = NSUB == 2 ? h : ch.resident ? 0 : static_cast<int>(t & 1u);
          uint32_t& used = b ? used1 : used0;
          const int col0 = j * C::kTileN + h * BNI + wg * kShare;
          const bool mirror = kSym && col0 - wg * kShare + BNI <= i * 2 * kBM;
          OrthIn<OP, TALL, FROM> in;
          in.fetch(g, z, row - lane, col0, lane);
          if (!wait_warp(&pc->tfull[b], used & 1u, abort, ctl)) {
            ok = false;
            break;
          }
          ++used;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < kChunks; ++c) {
            float v[32];
            tmem_ld32(tmem + lane_bits + b * BNI + wg * kShare + c * 32, v);
            tmem_ld_wait();
            if (c == kChunks - 1) {
              // The slot is drained once this load has completed.
              tc_fence_before();
              __syncwarp();
              // Test hook (fault == 1): withhold the release of the first accumulator.
              if (lane == 0 && !(ctl.fault == 1 && t == 0))
                mbar_arrive_cluster(b ? tempty1 : tempty0);
            }
            if (SPLIT && OP == kGram) {
              // A part of the sum, for the join: a block's piece e of row r at e * 32 + r.
              float4* const at = part_block(u, static_cast<int>(rank) * 4 + q,
                                            wg * kChunks + c) + lane;
#pragma unroll
              for (int e = 0; e < 8; ++e)
                at[e * 32] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
            } else if (col0 + c * 32 < g.cols)
              orth_epilogue<OP, LAST, TALL, FROM, TO>(g, stage, z, row, col0 + c * 32,
                                            c + 1 < kChunks ? col0 + (c + 1) * 32 : -1, mirror,
                                            drow, in,
                                            tmem + lane_bits + BNI + wg * kShare + c * 32, v);
          }
        }
      }
    };
    // The parts of a split Gram product, added in order; every warp of the launch takes blocks.
    auto join = [&]() {
      const OrthGeom& geo = ch.geom[kGram];
      const OrthView g{ch.k, ch.k, ch.ldk, ch.k, nullptr, nullptr, nullptr, ch.diag[0],
                       ch.mat[0], 0.f, 0.f, 0.f, 0};
      const int tiles = geo.num_units / geo.split, warps = 4 * kOrthWG;
      for (int blk = (warp - 2) * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);
           blk < tiles * (8 * BNI / 32); blk += warps * static_cast<int>(gridDim.x)) {
        const int tile = blk / (8 * BNI / 32), r = blk / (BNI / 32) % 8, c = blk % (BNI / 32);
        int z, i, j, nsub;
        orth_unit<BNI, NSUB, true>(geo, tile, z, i, j, nsub);
        const int row = i * 2 * kBM + r * 32 + lane, col = j * BNI + c * 32;
        if (row - lane >= g.rows || col >= g.cols) continue;
        float v[32] = {};
#pragma unroll 4
        for (int s = 0; s < geo.split; ++s) {
          const float4* const at = part_block(s * tiles + tile, r, c) + lane;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 f = at[e * 32];
            v[4 * e] += f.x;
            v[4 * e + 1] += f.y;
            v[4 * e + 2] += f.z;
            v[4 * e + 3] += f.w;
          }
        }
        OrthIn<kGram, TALL, false> in;
        orth_epilogue<kGram, false, TALL, false, false>(
            g, stage, z, row, col, -1, j * BNI + BNI <= i * 2 * kBM, 0.f, in, 0u, v);
      }
    };
    for (int p = 0; ok && p < phases; ++p) {
      if (p > 0) ok = wait_warp(&pc->met, (p - 1) & 1, abort, ctl);
      if (!ok) break;
      const int step = p / per_step, op = phase_op(p);
      constexpr std::false_type no{};
      constexpr std::true_type yes{};
      constexpr std::integral_constant<int, kUpdate> up{};
      const bool last = step + 1 == ch.steps;
      if (op == kGram) {
        product(std::integral_constant<int, kGram>{}, no, no, no, step);
      } else if (op == kJoin) {
        if constexpr (SPLIT) join();
      } else if (op == kSquare) {
        product(std::integral_constant<int, kSquare>{}, no, no, no, step);
      } else if (NSUB == 1 && ch.resident) {
        if (step == 0)
          product(up, no, no, yes, step);
        else if (!last)
          product(up, no, yes, yes, step);
        else
          product(up, yes, yes, no, step);
      } else if (!last) {
        product(up, no, no, no, step);
      } else {
        product(up, yes, no, no, step);
      }
      if (!ok) break;
      // This warp's part of the product, stored by plain stores and loaded by bulk copies,
      // becomes visible in order by the arrival, which the loading warp passes on at the
      // meeting's scope.
      fence_proxy_async_global();
      __syncwarp();
      if (lane == 0) mbar_arrive(&pc->done);
    }
  }

  // Neither CTA leaves while the other may still signal its barriers or use its TMEM.
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
  if (threadIdx.x == 0 && *abort) record_ran_out();
}

// maps = NULL: only whether the launch would be taken, so that nothing before it is enqueued in vain.
template <int BNI, int NSUB, bool TALL, bool SPLIT>
cudaError_t launch_chain(const OrthChain& ch, const OrthMaps* maps, const DevCtl& c,
                         cudaStream_t s) {
  using C = OrthCfg<BNI, NSUB>;
  auto kern = orth_chain<BNI, NSUB, TALL, SPLIT>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (c.fault == 4) return cudaErrorCooperativeLaunchTooLarge;  // test hook
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  // The CTAs wait for one another: all of them resident, or none.
  attr[1].id = cudaLaunchAttributeCooperative;
  attr[1].val.cooperative = 1;
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
    if (n < 1) return cudaErrorCooperativeLaunchTooLarge;
    max_clusters[dev] = n;
  }
  if (!maps) return cudaSuccess;
  cfg.numAttrs = 2;
  int pairs = 1;
  for (const OrthGeom& g : ch.geom) pairs = std::max(pairs, g.num_units);
  pairs = std::min(pairs, max_clusters[dev]);
  cfg.gridDim = dim3(2 * pairs, 1, 1);
  OrthChain co = ch;
  co.resident = ch.resident && ch.geom[kUpdate].num_units <= pairs;
  return cudaLaunchKernelEx(&cfg, kern, co, *maps, c);
}

// ----------------------------------------------------------------------------------------
// Matrices of up to 256 x 256: everything between the gradient and the result in one CTA pair's
// shared and tensor memory.  Y [k, l] is X, or X^T when m > n, its rows shared out between the
// two CTAs (128 each), zero beyond the matrix.  Per CTA:
//   rows    hi of its 128 rows, K-major: both operands of Y Y^T
//   cols    hi of all 256 rows, its 128 columns, MN-major: its half of the update's B operand
//   mat     its 128 rows of R, then of R_B in place, K-major: both operands of R R, and the
//           update's A operand
//   tensor memory  256 columns of accumulator, 256 of hi and lo, two fp16 numbers per cell
// With k <= 128 the second half of cols' rows holds lo, and B acts on hi + lo: small matrices have
// few roundings to average over, and this halves their error (16 x 23 noise, mean over 20: 1.7e-3
// to 1.0e-3 before the rounding to bf16).
// An epilogue writes the next product's operands where the MMAs read them (a row of `cols` goes to
// the CTA that holds those columns), and a product starts when the epilogue warps of the pair have
// arrived.  A step of 256 x 256 takes 15.5 us: 4.6 of MMAs and their start, 7 of epilogue
// arithmetic (all four schedulers of an SM issue throughout: 128 x 256 numbers each of a Gram
// 1.2 us, a square 1.8, an update 3.6) and 4 of arrivals.  Sixteen warps with every fourth run of
// 16 columns each, so that a narrow matrix uses them all, and global memory by way of shared memory
// 32 B at a time: eight warps of 128 columns, whose lanes read and wrote a row each, took 53 us for
// 64 x 64 and 131 for 256 x 256.  Graph replay, this kernel and orth_chain with its two launches
// before: 64 x 64 45 and 66 us, 16 x 200 64 and 62, 256 x 256 90 and 99, a hundred of 128 x 128 127
// and 145, a hundred of 256 x 256 182 and 225.
// ----------------------------------------------------------------------------------------
constexpr int kSmallWarps = 16;  // epilogue warps per CTA
constexpr int kSmallThreads = 32 + 32 * kSmallWarps;
constexpr int kSmallStride = kSmallWarps / 4 * 16;  // columns from one run of a warp's to the next
constexpr int kSmallBlock = 128 * 128;  // bytes of 128 rows x 64 fp16 columns
constexpr int kSmallStage = 32 * 64 * 4;  // bytes of a warp's fp32 elements, 32 rows x 64
static_assert(kSmallWarps * kSmallStage == 8 * kSmallBlock, "rows and cols, cleared as stages");

struct SmallCtl {
  uint64_t ready[2], tfull, fin;  // ready: in turn, as an arrival may overtake an earlier one
  uint32_t tmem_base;
  int abort;
  double sums[2 * kSmallWarps];
  alignas(16) float d[256];  // D of A, all rows
  float db[128];             // D_B, this CTA's rows
};
constexpr size_t kSmallSmem = 1024 + 12 * kSmallBlock + sizeof(SmallCtl);
static_assert(kSmallSmem <= 232448, "shared memory per CTA");

// Byte offset of 16-byte piece `piece` (8 columns) of row `row` in tiles of `rows` x 64 columns
// with the 128-byte swizzle.
__device__ __forceinline__ uint32_t small_at(int rows, int row, int piece) {
  return static_cast<uint32_t>((piece >> 3) * rows * 128 + row * 128 +
                               (((piece & 7) ^ (row & 7)) << 4));
}
__device__ __forceinline__ void st_cluster_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                              uint32_t d) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}
// wait_warp for a barrier that both CTAs of the pair arrive on after writing shared memory.
__device__ __forceinline__ bool wait_pair(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          const DevCtl& ctl) {
  const uint32_t a = smem_u32(bar);
  bool done = mbar_try_wait_cluster(a, parity);
  if (!done) {
    const long long t0 = clock64();
    while (!(done = mbar_try_wait_cluster(a, parity))) {
      if (*abort) break;
      if (clock64() - t0 > ctl.timeout_cycles) {
        *abort = 1;
        atomicOr(ctl.status, kFlagTimeout);
        break;
      }
    }
  }
  return __all_sync(0xffffffffu, done);
}

// BOTH: k <= 128, and the update multiplies lo too, by the rows of cols behind hi's.
template <class T, bool BOTH>
__global__ void __launch_bounds__(kSmallThreads, 1)
    orth_small(const __grid_constant__ OrthSmall p, const DevCtl ctl) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* rows = smem;                     // 4 tiles of 128 x 64
  uint8_t* cols = smem + 4 * kSmallBlock;   // 2 tiles of 256 x 64
  uint8_t* mat = smem + 8 * kSmallBlock;    // 4 tiles of 128 x 64
  SmallCtl* sc = reinterpret_cast<SmallCtl*>(smem + 12 * kSmallBlock);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int64_t z = blockIdx.x >> 1;
  const bool tall = p.m > p.n;
  const int k = tall ? p.n : p.m, l = tall ? p.m : p.n;
  volatile int* abort = &sc->abort;

  if (threadIdx.x == 0) {
    mbar_init(&sc->ready[0], 2 * kSmallWarps);
    mbar_init(&sc->ready[1], 2 * kSmallWarps);
    mbar_init(&sc->tfull, 1);
    mbar_init(&sc->fin, 1);
    sc->abort = 0;
    if (blockIdx.x == 0) *ctl.status = 0;  // a wait can only run out long after this
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc_pair(&sc->tmem_base, 512);
    tmem_relinquish_pair();
  }
  for (int i = threadIdx.x; i < 4 * kSmallBlock / 16; i += kSmallThreads)
    reinterpret_cast<uint4*>(mat)[i] = make_uint4(0, 0, 0, 0);
  for (int i = threadIdx.x; i < 256; i += kSmallThreads) {
    sc->d[i] = 0.f;
    sc->db[i & 127] = 0.f;
  }
  fence_proxy_async_all();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = sc->tmem_base;
  const int products = 3 * p.steps;

  // Epilogue warps: rows q * 32 + lane of the CTA, 16 columns of every kSmallStride.
  const int q = warp & 3;
  const int col0 = ((warp - 1) >> 2) * 16;
  const int row = q * 32 + lane;                        // of the CTA
  const int grow = static_cast<int>(rank) * 128 + row;  // of Y
  const bool live = grow - lane < k;                    // some row of this warp is Y's
  const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16);
  const uint32_t master = acc + 256;
  float* const stage = reinterpret_cast<float*>(smem + max(warp - 1, 0) * kSmallStage);
  if (warp > 0) {
    // u into the cells, momentum updated, the sum of u^2.  Two runs of 16 elements per load, by way
    // of shared memory, element c of row r at c ^ r.  When m > n a lane's row of Y is a column of
    // the matrix, and the same runs are lanes' rows.
    double sums[2] = {0.0, 0.0};
    const int run = lane & 15, half = lane & 16;
#pragma unroll 1
    for (int c = 0; c < 4 && live; ++c) {
      const int col = col0 + c * kSmallStride;
      if (col >= l) break;
      // Element e of this lane's run: at (i, j), then a row down each, `lim` of them in the matrix.
      const int i = tall ? col : grow - lane + half;
      const int j = tall ? grow - lane + (run + half) : col + run;
      const int lim = j < static_cast<int>(p.n) ? static_cast<int>(p.m) - i : 0;
      // Every load is issued before one is used; those beyond the matrix read its first element.
      const T* const from = static_cast<const T*>(p.grad) + z * p.grad_batch;
      float* const mom = p.momentum ? p.momentum + z * p.m * p.n : nullptr;
      const int jn = i * static_cast<int>(p.n) + j;
      T raw[16];
      float u[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) raw[e] = from[e < lim ? (i + e) * p.ldg + j : 0];
      if (mom) {
#pragma unroll
        for (int e = 0; e < 16; ++e) u[e] = mom[e < lim ? jn + e * static_cast<int>(p.n) : 0];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float g = static_cast<float>(raw[e]);
          const float now = p.beta * u[e] + p.rest * g;
          if (e < lim) mom[jn + e * static_cast<int>(p.n)] = now;
          u[e] = p.nesterov ? p.beta * now + p.rest * g : now;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) u[e] = static_cast<float>(raw[e]);
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float in = e < lim ? u[e] : 0.f;
        sums[e & 1] = fma(static_cast<double>(in), static_cast<double>(in), sums[e & 1]);
        const int r = tall ? run + half : e + half, cc = c * 16 + (tall ? e : run);
        stage[r * 64 + (cc ^ r)] = in;
      }
    }
    __syncwarp();
#pragma unroll 1
    for (int c = 0; c < 4 && live; ++c) {
      if (col0 + c * kSmallStride >= l) break;
      uint32_t w[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(stage[lane * 64 + ((c * 16 + e) ^ lane)]);
      tmem_st16_raw(master + col0 + c * kSmallStride, w);
    }
    tmem_st_wait();
    __syncwarp();
#pragma unroll 4
    for (int i = lane; i < kSmallStage / 16; i += 32)
      reinterpret_cast<uint4*>(stage)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_all();
    double sum = sums[0] + sums[1];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane < 2) {
      double* at = &sc->sums[rank * kSmallWarps + warp - 1];
      const uint32_t dst = mapa_shared(smem_u32(at), lane);
      const unsigned long long bits = __double_as_longlong(sum);
      st_shared_cluster_u32(dst, static_cast<uint32_t>(bits));
      st_shared_cluster_u32(dst + 4, static_cast<uint32_t>(bits >> 32));
    }
  }
  tc_fence_before();
  cluster_sync();  // the sums are there, and both CTAs' shared memory is cleared
  tc_fence_after();

  if (warp == 0) {
    // MMA issuer (leader only).
    if (rank == 0) {
      constexpr uint32_t kSym = idesc_f16_f32(256, 256, false, false);
      constexpr uint32_t kUpd = idesc_f16_f32(256, 256, false, true);
      for (int t = 0; t < products; ++t) {
        if (!wait_pair(&sc->ready[t & 1], (t >> 1) & 1, abort, ctl)) break;
        fence_proxy_async_all();
        tc_fence_after();
        if (lane == 0) {
          const int op = t % 3;
          const uint32_t a = smem_u32(op == kGram ? rows : mat);
          const uint32_t b = op == kUpdate ? smem_u32(cols) : a;
          const int steps = ((op == kGram ? l : k) + 15) / 16;
          for (int kk = 0; kk < steps; ++kk) {
            const uint64_t ad = smem_desc_sw128(a + (kk >> 2) * kSmallBlock + (kk & 3) * 32, 16, 1024);
            const uint64_t bd = op == kUpdate
                                    ? smem_desc_sw128(b + kk * 2048, 2 * kSmallBlock, 1024)
                                    : smem_desc_sw128(b + (kk >> 2) * kSmallBlock + (kk & 3) * 32, 16, 1024);
            umma_bf16_pair(tmem, ad, bd, op == kUpdate ? kUpd : kSym, kk != 0 ? 1u : 0u);
            if (op == kUpdate && BOTH)
              umma_bf16_pair(tmem, ad, smem_desc_sw128(b + (kk + 8) * 2048, 2 * kSmallBlock, 1024),
                             kUpd, 1u);
          }
          umma_commit_pair_mc(&sc->tfull, 0x3);
        }
        __syncwarp();
      }
      if (lane == 0) umma_commit_pair_mc(&sc->fin, 0x1);
      __syncwarp();
      wait_warp(&sc->fin, 0u, abort, ctl, false);
    }
  } else {
    double total = 0.0;
#pragma unroll
    for (int i = 0; i < 2 * kSmallWarps; ++i) total += sc->sums[i];
    const float2 inv = orth_factors(total, p.eps);
    // This warp's operands are written: both CTAs' barriers learn of it.
    auto arrive = [&](int t, bool withhold) {
      fence_proxy_async_all();
      tc_fence_before();
      __syncwarp();
      if (lane < 2 && !withhold) mbar_arrive_cluster(mapa_shared(smem_u32(&sc->ready[t & 1]), lane));
    };
    // 8 pairs of columns from col to the CTA that holds the columns, as its row r, ...
    const uint32_t cols_far = mapa_shared(smem_u32(cols), rank ^ 1);
    auto put_cols = [&](int r, int col, const uint32_t(&w)[8]) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t at = small_at(256, r, (col / 8 + e) & 15);
        if ((col < 128) == (rank == 0))
          *reinterpret_cast<uint4*>(cols + at) =
              make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
        else
          st_cluster_v4(cols_far + at, w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
      }
    };
    // ... and the products' operands: hi, and lo where it takes part.
    auto put = [&](int col, const uint32_t(&hi)[8], const uint32_t(&lo)[8]) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
        *reinterpret_cast<uint4*>(rows + small_at(128, row, col / 8 + e)) =
            make_uint4(hi[4 * e], hi[4 * e + 1], hi[4 * e + 2], hi[4 * e + 3]);
      put_cols(grow, col, hi);
      if (BOTH) put_cols(128 + grow, col, lo);
    };
    auto put_cells = [&](uint32_t at, const uint32_t(&hi)[8], const uint32_t(&lo)[8]) {
      uint32_t w[16];
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        w[2 * h] = __byte_perm(hi[h], lo[h], 0x5410);
        w[2 * h + 1] = __byte_perm(hi[h], lo[h], 0x7632);
      }
      tmem_st16_raw(at, w);
    };
    auto split = [](float2 r, uint32_t& hi, uint32_t& lo) {
      hi = pack_half2(r.x, r.y);
      const float2 f = unpack_half2(hi);
      lo = pack_half2(r.x - f.x, r.y - f.y);
    };
    // X = u / (||u|| + eps).
#pragma unroll 1
    for (int col = col0; col < l && live; col += kSmallStride) {
      uint32_t w[16], hi[8], lo[8];
      tmem_ld16_raw(master + col, w);
      tmem_ld_wait();
#pragma unroll
      for (int h = 0; h < 8; ++h)
        split(make_float2(__uint_as_float(w[2 * h]) * inv.x * inv.y,
                          __uint_as_float(w[2 * h + 1]) * inv.x * inv.y),
              hi[h], lo[h]);
      put_cells(master + col, hi, lo);
      put(col, hi, lo);
    }
    tmem_st_wait();
    arrive(0, false);

    for (int t = 0; t < products; ++t) {
      const int step = t / 3, op = t % 3;
      const float a = p.co[step][0], b = p.co[step][1], cc = p.co[step][2];
      const bool last = t == products - 1;
      // What the other warps wrote for this product's epilogue (diagonals), then its MMAs.
      if (!wait_pair(&sc->ready[t & 1], (t >> 1) & 1, abort, ctl)) break;
      if (!wait_warp(&sc->tfull, t & 1, abort, ctl)) break;
      tc_fence_after();
      const float drow = op == kSquare ? sc->d[grow] : op == kUpdate ? sc->db[row] : 0.f;
      const float on_hi = drow + a, on_lo = BOTH ? on_hi : a;
      const int end = !live ? 0 : op == kUpdate ? l : k;
#pragma unroll 1
      for (int col = col0; col < end; col += kSmallStride) {
        uint32_t v[16], hi[8], lo[8];
        tmem_ld16_raw(acc + col, v);
        if (op == kUpdate) {
          uint32_t w[16];
          tmem_ld16_raw(master + col, w);
          tmem_ld_wait();
#pragma unroll
          for (int h = 0; h < 8; ++h) {
            const float2 x = make_float2(__uint_as_float(v[2 * h]), __uint_as_float(v[2 * h + 1]));
            const float2 r = __ffma2_rn(
                x, both(1.f / kScaleB),
                __ffma2_rn(unpack_half2(__byte_perm(w[2 * h], w[2 * h + 1], 0x5410)),
                           both(on_hi),
                           __fmul2_rn(unpack_half2(__byte_perm(w[2 * h], w[2 * h + 1], 0x7632)),
                                      both(on_lo))));
            if (last)
              hi[h] = pack_bf162(r.x * (1.f / kScaleX), r.y * (1.f / kScaleX));
            else
              split(r, hi[h], lo[h]);
          }
          if (last) {
            // The operands have been read: this warp's part of them takes what it has to turn.
            __nv_bfloat16* const out = p.out + z * p.m * p.n;
            uint32_t* const turn = reinterpret_cast<uint32_t*>(stage);
            if (!tall) {
#pragma unroll
              for (int h = 0; h < 8; ++h) turn[lane * 8 + (h ^ (lane >> 2))] = hi[h];
              __syncwarp();
            }
            const int run = lane & 15, half = lane & 16;
            const int i = tall ? col : grow - lane + half, j = tall ? grow : col + run;
            const int lim = j < static_cast<int>(p.n) ? static_cast<int>(p.m) - i : 0;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int r = e + half;
              const uint32_t two = tall ? hi[e / 2] : turn[r * 8 + ((run >> 1) ^ (r >> 2))];
              const uint16_t bits = static_cast<uint16_t>((tall ? e : run) & 1 ? two >> 16 : two);
              if (e < lim) out[(i + e) * static_cast<int>(p.n) + j] = __ushort_as_bfloat16(bits);
            }
          } else {
            put_cells(master + col, hi, lo);
            put(col, hi, lo);
          }
          __syncwarp();
          continue;
        }
        uint8_t* at[2] = {mat + small_at(128, row, col / 8), mat + small_at(128, row, col / 8 + 1)};
        if (op == kSquare) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint4 w = *reinterpret_cast<const uint4*>(at[e]);
            lo[4 * e] = w.x;
            lo[4 * e + 1] = w.y;
            lo[4 * e + 2] = w.z;
            lo[4 * e + 3] = w.w;
          }
        }
        tmem_ld_wait();
        if (op == kGram) {
#pragma unroll
          for (int h = 0; h < 8; ++h) {
            const float2 x = make_float2(__uint_as_float(v[2 * h]), __uint_as_float(v[2 * h + 1]));
            const float2 r = __fmul2_rn(x, both(kScaleA / (kScaleX * kScaleX)));
            hi[h] = pack_half2(r.x, r.y);
          }
        } else {
          const float2 slope = both(cc * (kScaleB / kScaleA));
          const float2 base = both(fmaf(cc, drow, b) * (kScaleB / kScaleA));
#pragma unroll
          for (int h = 0; h < 8; ++h) {
            const float2 x = make_float2(__uint_as_float(v[2 * h]), __uint_as_float(v[2 * h + 1]));
            const float2 dj = *reinterpret_cast<const float2*>(&sc->d[col + 2 * h]);
            const float2 r = __ffma2_rn(unpack_half2(lo[h]), __ffma2_rn(slope, dj, base),
                                        __fmul2_rn(x, both(cc * (kScaleB / (kScaleA * kScaleA)))));
            hi[h] = pack_half2(r.x, r.y);
          }
        }
        if (col + 16 > grow - lane && col < grow - lane + 32) {
          // The diagonal's elements to fp32, zeros in their place.
          float diag = 0.f;
#pragma unroll
          for (int h = 0; h < 8; ++h) {
            const bool d0 = grow == col + 2 * h, d1 = grow == col + 2 * h + 1;
            diag = d0 ? __uint_as_float(v[2 * h]) : d1 ? __uint_as_float(v[2 * h + 1]) : diag;
            hi[h] = d0 ? hi[h] & 0xffff0000u : d1 ? hi[h] & 0xffffu : hi[h];
          }
          if (grow >= col && grow < col + 16) {
            if (op == kGram) {
              const uint32_t bits = __float_as_uint(diag * (1.f / (kScaleX * kScaleX)));
              const uint32_t da = smem_u32(&sc->d[grow]);
              st_shared_cluster_u32(mapa_shared(da, 0), bits);
              st_shared_cluster_u32(mapa_shared(da, 1), bits);
            } else {
              sc->db[row] =
                  fmaf(cc, fmaf(drow, drow, diag * (1.f / (kScaleA * kScaleA))), b * drow);
            }
          }
          __syncwarp();
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *reinterpret_cast<uint4*>(at[e]) =
              make_uint4(hi[4 * e], hi[4 * e + 1], hi[4 * e + 2], hi[4 * e + 3]);
        __syncwarp();
      }
      if (op == kUpdate && !last) tmem_st_wait();
      // Test hook (fault == 1): withhold one warp's first arrival.
      if (!last) arrive(t + 1, ctl.fault == 1 && t == 0 && warp == 1);
    }
  }

  // Neither CTA leaves while the other may still write its shared memory or use its TMEM.
  tc_fence_before();
  __syncwarp();
  cluster_sync();
  tc_fence_after();
  if (warp == 0) tmem_dealloc_pair(tmem, 512);
  if (threadIdx.x == 0 && *abort) record_ran_out();
}

template <class T, bool BOTH>
cudaError_t small_t(const OrthSmall& p, int64_t batch, const DevCtl& c, cudaStream_t s) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  static bool smem_set[64] = {false};  // per device, once
  if (!smem_set[dev]) {
    e = cudaFuncSetAttribute(orth_small<T, BOTH>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSmallSmem));
    if (e != cudaSuccess) return e;
    smem_set[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(2 * batch), 1, 1);
  cfg.blockDim = dim3(kSmallThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmallSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, orth_small<T, BOTH>, p, c);
}

}  // namespace

cudaError_t launch_orth_small(int dtype, const OrthSmall& p, int64_t batch, const DevCtl& c,
                              cudaStream_t s) {
  auto run = [&](auto t) {
    using T = decltype(t);
    return std::min(p.m, p.n) <= 128 ? small_t<T, true>(p, batch, c, s)
                                     : small_t<T, false>(p, batch, c, s);
  };
  if (dtype == 0) return run(__nv_bfloat16{});
  if (dtype == 1) return run(__half{});
  return run(float{});
}

cudaError_t orth_ran_out(int* flags) { return take_ran_out(flags); }

cudaError_t launch_orth_prep(int dtype, const OrthPrep& p, int64_t batch, cudaStream_t s) {
  auto aligned = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0; };
  const bool vec = p.n % 8 == 0 && p.ldg % 8 == 0 && p.grad_batch % 8 == 0 && aligned(p.grad) &&
                   aligned(p.momentum);
  const int64_t groups = p.m * (vec ? p.n / 8 : p.n);
  const int64_t want = (groups + kPrepThreads - 1) / kPrepThreads;
  const dim3 g1(static_cast<unsigned>(std::min<int64_t>(want, kOrthSums)), static_cast<unsigned>(batch));
  const dim3 g2(static_cast<unsigned>(std::min<int64_t>(want, 4096)), static_cast<unsigned>(batch));
  auto run = [&](auto t) {
    using T = decltype(t);
    if (vec)
      orth_moment<T, 8><<<g1, kPrepThreads, 0, s>>>(p);
    else
      orth_moment<T, 1><<<g1, kPrepThreads, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (vec)
      orth_scale<T, 8><<<g2, kPrepThreads, 0, s>>>(p, static_cast<int>(g1.x));
    else
      orth_scale<T, 1><<<g2, kPrepThreads, 0, s>>>(p, static_cast<int>(g1.x));
    return cudaGetLastError();
  };
  if (dtype == 0) return run(__nv_bfloat16{});
  if (dtype == 1) return run(__half{});
  return run(float{});
}

static cudaError_t orth_chain_call(int bn, bool tall, const OrthChain& ch, const OrthMaps* maps,
                                   const DevCtl& c, cudaStream_t s) {
  auto run = [&](auto tallc, auto splitc) {
    constexpr bool T = decltype(tallc)::value, S = decltype(splitc)::value;
    return bn == 256 ? launch_chain<256, 1, T, S>(ch, maps, c, s)
                     : launch_chain<128, 1, T, S>(ch, maps, c, s);
  };
  constexpr std::false_type no{};
  constexpr std::true_type yes{};
  if (bn == 512)
    return tall ? launch_chain<256, 2, true, false>(ch, maps, c, s)
                : launch_chain<256, 2, false, false>(ch, maps, c, s);
  if (ch.geom[kGram].split > 1) return tall ? run(yes, yes) : run(no, yes);
  return tall ? run(yes, no) : run(no, no);
}

cudaError_t launch_orth_chain(int bn, bool tall, const OrthChain& ch, const OrthMaps& maps,
                              const DevCtl& c, cudaStream_t s) {
  return orth_chain_call(bn, tall, ch, &maps, c, s);
}

cudaError_t ready_orth_chain(int bn, bool tall, const OrthChain& ch, const DevCtl& c) {
  return orth_chain_call(bn, tall, ch, nullptr, c, nullptr);
}

}  // namespace slm
