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

// X = u / (||u|| + eps) as hi + lo; the norm from the partial sums, added in a fixed order.
template <class T, int V>
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
      const float x = u[e] * inv;
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
// warpgroup over half of the columns.  Operands are K-major or MN-major as they lie in memory,
// so that no transpose of X is ever stored.  Per step:
//   kGram    R, D of A = X X^T:  a symmetric product, only blocks on and below the diagonal
//            are computed and each is written to its mirrored place too
//   kSquare  R_B, D_B of B = b A + c A^2, symmetric in the same way
//   kUpdate  hi, lo of a X + B X; in the last step the result in bf16
// A product reads what the one before wrote anywhere, so the CTAs meet between products (a
// counter in the workspace, bounded waits; the cooperative launch makes them all resident).
// A meeting costs about 2 us, a launch of its own with its set-up and drain 7 us: 256 x 256
// matrices, which are all latency, took 116 us of GPU time in 15 launches.
// The tensor memory holds two accumulator slots of BNI columns.  NSUB = 1: tiles take the slots
// in turn, so that a tile's epilogue overlaps the next tile's MMAs.  NSUB = 2: a tile of 512
// columns takes both; the operands then cross from L2 at 170 instead of 128 flops per byte, and
// L2 is what bounds these products (about 9.3 TB/s measured over the 74 pairs: 256-column
// tiles reach 1.2 PFLOP/s).  The next tile's MMAs for the first slot start while the epilogue
// still drains the second.
// ----------------------------------------------------------------------------------------
enum OrthOp { kGram = 0, kSquare = 1, kUpdate = 2 };
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

// Staging of an epilogue warp: two blocks of 32 rows x 32 fp16 columns, 64 bytes per row, in
// the 64-byte swizzle of the store maps (16-byte piece k of row r at k ^ (r / 2 % 4)).
constexpr int kOrthStage = 4096;
__device__ __forceinline__ int stage_piece(int row, int k) {
  return row * 4 + (k ^ ((row >> 1) & 3));
}

template <int STAGES>
struct OrthCtl {
  uint64_t full[STAGES], empty[STAGES], tfull[2], tempty[2], fin, met;
  uint32_t tmem_base;
  int abort, done;
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

// What the epilogue reads for a warp's block of 32 rows x 32 columns: fetched a block ahead, so
// that its latency passes behind the MMAs or the block before.  Four lanes share a row, so that
// every load covers whole 64-byte pieces of rows.
template <int OP>
struct OrthIn {
  static constexpr int kSets = OP == kGram ? 0 : OP == kSquare ? 1 : 2;
  uint4 w[kSets == 0 ? 1 : kSets][4];  // kSquare: R; kUpdate: hi, lo
  float dcol;                          // lane l: the diagonal's entry of column col + l
  __device__ __forceinline__ void fetch(const OrthView& g, int z, int64_t row0, int64_t col,
                                        int lane) {
    if (OP == kGram || col >= g.cols) return;
    if (OP == kSquare || g.tall)
      dcol = col + lane < g.cols ? g.diag_in[static_cast<int64_t>(z) * g.diag_n + col + lane] : 0.f;
    const int64_t c = col + (lane & 3) * 8;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t row = row0 + q * 8 + (lane >> 2);
      const int64_t at = (static_cast<int64_t>(z) * g.rows + row) * g.ld + c;
      const bool in = row < g.rows && c < g.cols;  // rows are padded to whole pieces
      const uint4 none = make_uint4(0, 0, 0, 0);
      w[0][q] = !in ? none
                    : *reinterpret_cast<const uint4*>(g.in + at);
      if (OP == kUpdate) w[kSets - 1][q] = !in ? none : *reinterpret_cast<const uint4*>(g.lo + at);
    }
  }
  // Into the warp's staging blocks.
  __device__ __forceinline__ void put(uint4* stage, int lane) const {
#pragma unroll
    for (int e = 0; e < kSets; ++e)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        stage[e * 128 + stage_piece(q * 8 + (lane >> 2), lane & 3)] = w[e][q];
  }
};

// One warp's block: this lane's row `row`, columns [col, col + 32) of matrix z.  The block's
// inputs lie in the staging blocks; its outputs take their place, each lane its own row, and go
// out by bulk stores, which leave out rows and columns outside the matrix.
template <int OP, bool LAST>
__device__ __forceinline__ void orth_epilogue(const OrthView& g, const CUtensorMap* st0,
                                              const CUtensorMap* st1, uint4* stage, int z,
                                              int64_t row, int64_t col, bool mirror, float drow,
                                              float dcol, float (&v)[32]) {
  const int lane = threadIdx.x & 31;
  uint32_t in[2][16];
#pragma unroll
  for (int e = 0; e < OrthIn<OP>::kSets; ++e)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint4 w = stage[e * 128 + stage_piece(lane, q)];
      in[e][4 * q] = w.x;
      in[e][4 * q + 1] = w.y;
      in[e][4 * q + 2] = w.z;
      in[e][4 * q + 3] = w.w;
    }
  auto put_row = [&](int e, const uint32_t(&w)[16]) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      stage[e * 128 + stage_piece(lane, q)] =
          make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
  };
  uint32_t out[16];
  if (OP == kGram || OP == kSquare) {
    const int e = static_cast<int>(row - col);  // the diagonal's column of the block, if in it
    float d = 0.f;
    if (OP == kGram) {
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        if (c == e) d = v[c] * (1.f / (kScaleX * kScaleX));
        v[c] = c == e ? 0.f : v[c] * (kScaleA / (kScaleX * kScaleX));
      }
    } else {
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        const float dj = __shfl_sync(0xffffffffu, dcol, c);
        const float2 r2 = unpack_half2(in[0][c / 2]);
        const float rr = v[c] * (1.f / (kScaleA * kScaleA));
        const float a = (c & 1 ? r2.y : r2.x) * (1.f / kScaleA);
        if (c == e) d = fmaf(g.c, fmaf(drow, drow, rr), g.b * drow);
        v[c] = c == e ? 0.f : kScaleB * fmaf(g.c, fmaf(drow + dj, a, rr), g.b * a);
      }
    }
#pragma unroll
    for (int c = 0; c < 16; ++c) out[c] = pack_half2(v[2 * c], v[2 * c + 1]);
    if (row < g.rows && e >= 0 && e < 32)
      g.diag_out[static_cast<int64_t>(z) * g.diag_n + row] = d;
    put_row(0, out);
    if (mirror) {
      // The block's transpose: two lanes trade halves, so that each word holds two rows.
      uint32_t* t = reinterpret_cast<uint32_t*>(stage + 128);
      const bool odd = lane & 1;
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const uint32_t q = __shfl_xor_sync(0xffffffffu, out[c], 1);
        const int cc = 2 * c + odd, word = lane >> 1;
        t[stage_piece(cc, word >> 2) * 4 + (word & 3)] =
            odd ? __byte_perm(q, out[c], 0x7632) : __byte_perm(out[c], q, 0x5410);
      }
    }
  } else {
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
      const float2 hi = unpack_half2(in[0][c / 2]), lo = unpack_half2(in[1][c / 2]);
      float d0 = drow, d1 = drow;
      if (g.tall) {
        d0 = __shfl_sync(0xffffffffu, dcol, c);
        d1 = __shfl_sync(0xffffffffu, dcol, c + 1);
      }
      v[c] = fmaf(v[c], 1.f / kScaleB, fmaf(d0, hi.x, g.a * (hi.x + lo.x)));
      v[c + 1] = fmaf(v[c + 1], 1.f / kScaleB, fmaf(d1, hi.y, g.a * (hi.y + lo.y)));
    }
    if (LAST) {
#pragma unroll
      for (int c = 0; c < 16; ++c)
        out[c] = pack_bf162(v[2 * c] * (1.f / kScaleX), v[2 * c + 1] * (1.f / kScaleX));
      put_row(0, out);
      if (!g.out_vec) {
        // Rows of the result that do not start on 16-byte boundaries: element stores, a row
        // per instruction.
        __syncwarp();
        const __nv_bfloat16* el = reinterpret_cast<const __nv_bfloat16*>(stage);
        const int64_t r0 = row - lane;
        __nv_bfloat16* dst = g.out + (static_cast<int64_t>(z) * g.rows + r0) * g.cols + col + lane;
        const int rows = static_cast<int>(min(static_cast<int64_t>(32), g.rows - r0));
        if (col + lane < g.cols)
          for (int r = 0; r < rows; ++r)
            dst[r * g.cols] = el[stage_piece(r, lane >> 3) * 8 + (lane & 7)];
      }
    } else {
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        out[c] = pack_half2(v[2 * c], v[2 * c + 1]);
        const float2 hi = unpack_half2(out[c]);
        v[2 * c] -= hi.x;
        v[2 * c + 1] -= hi.y;
      }
      put_row(0, out);
#pragma unroll
      for (int c = 0; c < 16; ++c) out[c] = pack_half2(v[2 * c], v[2 * c + 1]);
      put_row(1, out);
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0 && !(LAST && !g.out_vec)) {
    const int r0 = static_cast<int>(row), c0 = static_cast<int>(col);
    if (r0 < g.rows) {
      tma_store_3d(st0, stage, c0, r0, z);
      if (OP == kUpdate && !LAST) tma_store_3d(st1, stage + 128, c0, r0, z);
      if (OP != kUpdate && mirror) tma_store_3d(st0, stage + 128, r0, c0, z);
      bulk_commit();
    }
  }
}

template <int BNI, int NSUB, bool TALL>
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
    pc->abort = 0;
    pc->done = 0;
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
  const int products = 3 * ch.steps;

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
        int z, i, j, nsub;
        orth_unit<BNI, NSUB, OP != kUpdate>(g, u, z, i, j, nsub);
        const int mrow = i * 2 * kBM + static_cast<int>(rank) * kBM;
        for (int kb = 0; kb < g.k_blocks; ++kb, ++it) {
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
    for (int p = 0; ok && p < products; ++p) {
      if (p > 0) {
        // Every CTA has finished the product before; let this CTA's epilogue know.
        ok = wait_met(ch.counter, p * static_cast<int>(gridDim.x), abort, ctl);
        if (lane == 0) mbar_arrive(&pc->met);
        __syncwarp();
        if (!ok) break;
      }
      const int cur = (p / 3) & 1;
      if (p % 3 == 0)
        product(std::integral_constant<int, kGram>{}, cur);
      else if (p % 3 == 1)
        product(std::integral_constant<int, kSquare>{}, 0);
      else
        product(std::integral_constant<int, kUpdate>{}, cur);
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
          int z, i, j, nsub;
          orth_unit<BNI, NSUB, OP != kUpdate>(g, u, z, i, j, nsub);
          const int b0 = NSUB == 2 ? 0 : static_cast<int>(t & 1u);
          uint32_t& used = b0 ? used1 : used0;
          ok = wait_warp(&pc->tempty[b0], (used & 1u) ^ 1u, abort, ctl);
          if (!ok) return;
          ++used;
          tc_fence_after();
          int kb = 0;
          if (NSUB == 2 && nsub == 2) {
            // The first slot over the stages that are there already, then, once the second
            // slot is free, its MMAs for them, with the stages' releases.
            const int pre = min(STAGES, g.k_blocks);
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
          for (; kb < g.k_blocks; ++kb, ++it) {
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
      for (int p = 0; ok && p < products; ++p) {
        if (p % 3 == 0)
          product(std::integral_constant<int, kGram>{});
        else if (p % 3 == 1)
          product(std::integral_constant<int, kSquare>{});
        else
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
    auto product = [&](auto opc, auto lastc, int step) {
      constexpr int OP = decltype(opc)::value;
      constexpr bool LAST = decltype(lastc)::value;
      constexpr bool kSym = OP != kUpdate;
      const OrthGeom& geo = ch.geom[OP];
      const int cur = step & 1;
      const OrthView g{OP == kUpdate ? ch.m : ch.k, OP == kUpdate ? ch.n : ch.k,
                       OP == kUpdate ? ch.ldx : ch.ldk, ch.k,
                       OP == kUpdate ? ch.hi[cur] : ch.mat[0], ch.lo,
                       OP == kSquare ? ch.diag[0] : ch.diag[1],
                       OP == kGram ? ch.diag[0] : ch.diag[1], ch.out, ch.co[step][0],
                       ch.co[step][1], ch.co[step][2], TALL, ch.out_vec};
      const CUtensorMap* st0 = OP == kGram ? &maps.mat[0] : OP == kSquare ? &maps.mat[1]
                               : LAST ? &maps.out : &maps.hi[cur ^ 1];
      for (int u = pair; ok && u < geo.num_units; u += npairs, ++t) {
        int z, i, j, nsub;
        orth_unit<BNI, NSUB, kSym>(geo, u, z, i, j, nsub);
        const int64_t row = static_cast<int64_t>(i) * 2 * kBM + rank * kBM + q * 32 + lane;
        const int64_t row0 = row - lane;
        float drow = 0.f;
        if (OP == kSquare || (OP == kUpdate && !TALL))
          if (row < g.rows) drow = g.diag_in[static_cast<int64_t>(z) * g.diag_n + row];
        for (int h = 0; h < nsub; ++h) {
          const int b = NSUB == 2 ? h : static_cast<int>(t & 1u);
          uint32_t& used = b ? used1 : used0;
          const int64_t col0 = static_cast<int64_t>(j) * C::kTileN + h * BNI + wg * kShare;
          const bool mirror =
              kSym && col0 - wg * kShare + BNI <= static_cast<int64_t>(i) * 2 * kBM;
          OrthIn<OP> in;
          in.fetch(g, z, row0, col0, lane);
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
            // The staging blocks are free once the stores of the block before have read them.
            if (lane == 0) bulk_wait_read_all();
            __syncwarp();
            in.put(stage, lane);
            const float dcol = in.dcol;
            if (c + 1 < kChunks) in.fetch(g, z, row0, col0 + (c + 1) * 32, lane);
            tmem_ld_wait();
            if (c == kChunks - 1) {
              // The slot is drained once this load has completed.
              tc_fence_before();
              __syncwarp();
              // Test hook (fault == 1): withhold the release of the first accumulator.
              if (lane == 0 && !(ctl.fault == 1 && t == 0))
                mbar_arrive_cluster(b ? tempty1 : tempty0);
            } else {
              __syncwarp();
            }
            if (col0 + c * 32 < g.cols)
              orth_epilogue<OP, LAST>(g, st0, &maps.lo, stage, z, row, col0 + c * 32, mirror,
                                      drow, dcol, v);
          }
        }
      }
    };
    for (int p = 0; ok && p < products; ++p) {
      if (p > 0) ok = wait_warp(&pc->met, (p - 1) & 1u, abort, ctl);
      if (!ok) break;
      const int step = p / 3;
      if (p % 3 == 0)
        product(std::integral_constant<int, kGram>{}, std::false_type{}, step);
      else if (p % 3 == 1)
        product(std::integral_constant<int, kSquare>{}, std::false_type{}, step);
      else if (step + 1 < ch.steps)
        product(std::integral_constant<int, kUpdate>{}, std::false_type{}, step);
      else
        product(std::integral_constant<int, kUpdate>{}, std::true_type{}, step);
      if (!ok) break;
      // This warp's part of the product is in memory: bulk stores complete, plain stores fenced.
      // The last of the CTA's warps reports (nobody blocks: after a wait that ran out, some
      // warps may never come here).
      if (lane == 0) {
        bulk_wait_all();
        fence_proxy_async_global();
      }
      __threadfence();
      __syncwarp();
      if (lane == 0 && atomicAdd(&pc->done, 1) == 4 * kOrthWG * (p + 1) - 1) {
        __threadfence();
        red_release_add_s32(ch.counter, 1);
      }
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }

  // Neither CTA leaves while the other may still signal its barriers or use its TMEM.
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

template <int BNI, int NSUB, bool TALL>
cudaError_t launch_chain(const OrthChain& ch, const OrthMaps& maps, const DevCtl& c,
                         cudaStream_t s) {
  using C = OrthCfg<BNI, NSUB>;
  auto kern = orth_chain<BNI, NSUB, TALL>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
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
    max_clusters[dev] = n > 0 ? n : 1;
  }
  cfg.numAttrs = 2;
  int units = 1;
  for (const OrthGeom& g : ch.geom) units = std::max(units, g.num_units);
  cfg.gridDim = dim3(2 * std::min(units, max_clusters[dev]), 1, 1);
  return cudaLaunchKernelEx(&cfg, kern, ch, maps, c);
}

}  // namespace

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

cudaError_t launch_orth_chain(int bn, bool tall, const OrthChain& ch, const OrthMaps& maps,
                              const DevCtl& c, cudaStream_t s) {
  if (bn == 512)
    return tall ? launch_chain<256, 2, true>(ch, maps, c, s)
                : launch_chain<256, 2, false>(ch, maps, c, s);
  if (bn == 256)
    return tall ? launch_chain<256, 1, true>(ch, maps, c, s)
                : launch_chain<256, 1, false>(ch, maps, c, s);
  return tall ? launch_chain<128, 1, true>(ch, maps, c, s)
              : launch_chain<128, 1, false>(ch, maps, c, s);
}

}  // namespace slm
