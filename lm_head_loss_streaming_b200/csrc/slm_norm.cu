// slm_norm.cu - norms before and after a draft block, fused with its gate and its residual
// scale, and their backward (slm_block_norm_fwd, slm_block_norm_bwd).
//
// Per row of d channels, with rs = residual_scale, bs = block_scale, wq = w_post + offset,
// wp = w_pre + offset and norm factors i_t = 1 / sqrt(mean(t^2) + eps):
//     yh = y i_y (y without w_post),   r = rs x + bs gate (yh wq),   rh = r i_r,   h = rh wp.
// Backward, with a = bs gate wq, u = dh wp, and the incoming dr and dh:
//     g  = dr + i_r (u - rh c1),        c1 = mean(u rh)
//     dx = rs g,   dy = i_y (a g - yh c2),  c2 = mean(a yh g)
//     dgate = bs yh wq g,   dw_post = sum_rows bs gate yh g,   dw_pre = sum_rows dh rh.
// c2 needs no second reduction after c1, because g is linear in c1:
//     c2 = mean(a yh (dr + i_r u)) - i_r c1 mean(a yh rh),
// so one reduction of three sums per row serves both.  Everything between the loads and the
// stores is fp32: h is made from the unrounded r, and the backward recomputes r from x and y
// (it must read a row of either r or x anyway) instead of taking the rounded one, so that the
// weight gradients, returned in fp32, see no rounding of r.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "f32x2.cuh"
#include "slm_internal.h"
#include "slm_wait.cuh"
#include "sm100.cuh"

namespace slm {
namespace {
using namespace sm100;

template <class T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}
template <>
__device__ __forceinline__ float to_f<__half>(__half v) {
  return __half2float(v);
}
template <class T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f<__half>(float v) {
  return __float2half_rn(v);
}

// Element i of a parameter array (weights, gate) that is either of the rows' type or fp32.
template <class T>
__device__ __forceinline__ float ld_param(const void* p, bool f32, int64_t i) {
  return f32 ? static_cast<const float*>(p)[i] : to_f<T>(static_cast<const T*>(p)[i]);
}

// Sums v over the block, the same total in every thread.
template <int K>
__device__ __forceinline__ void block_sum(float (&v)[K]) {
  __shared__ float part[32][K];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  __syncthreads();  // the previous sum has been read
  if (lane == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) part[warp][k] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float t = lane < nw ? part[lane][k] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    v[k] = t;
  }
}

// ----------------------------------------------------------------------------------------
// The kernels for every width, stride and alignment: one row per block, element loads, the
// row read again (from L1 / L2) for each of its sweeps.
// ----------------------------------------------------------------------------------------
constexpr int kAnyThreads = 256;

template <class T>
__global__ void __launch_bounds__(kAnyThreads) norm_fwd_any(const NormFwd p) {
  const bool wf = p.w_f32, gf = p.gate_f32;
  for (int64_t n = blockIdx.x; n < p.N; n += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + n * p.ldx;
    const T* y = p.y ? static_cast<const T*>(p.y) + n * p.ldy : nullptr;
    const int64_t grow = p.gate ? n / p.rows_per_gate * p.d : 0;
    float iy = 1.f;
    if (p.w_post) {
      float s[1] = {0.f};
      for (int64_t c = threadIdx.x; c < p.d; c += kAnyThreads) {
        const float v = to_f<T>(y[c]);
        s[0] = fmaf(v, v, s[0]);
      }
      block_sum(s);
      iy = rsqrtf(s[0] / static_cast<float>(p.d) + p.eps);
      if (threadIdx.x == 0 && p.rstd_post) p.rstd_post[n] = iy;
    }
    auto stream = [&](int64_t c) {
      float r = p.residual_scale * to_f<T>(x[c]);
      if (y) {
        float v = to_f<T>(y[c]) * iy;
        if (p.w_post) v *= ld_param<T>(p.w_post, wf, c) + p.weight_offset;
        if (p.gate) v *= ld_param<T>(p.gate, gf, grow + c);
        r = fmaf(p.block_scale, v, r);
      }
      return r;
    };
    float ir = 1.f;
    if (p.w_pre) {
      float s[1] = {0.f};
      for (int64_t c = threadIdx.x; c < p.d; c += kAnyThreads) {
        const float r = stream(c);
        s[0] = fmaf(r, r, s[0]);
      }
      block_sum(s);
      ir = rsqrtf(s[0] / static_cast<float>(p.d) + p.eps);
      if (threadIdx.x == 0 && p.rstd_pre) p.rstd_pre[n] = ir;
    }
    // The residual may be written over x: each element is read and written by one thread.
    for (int64_t c = threadIdx.x; c < p.d; c += kAnyThreads) {
      const float r = stream(c);
      if (p.residual) static_cast<T*>(p.residual)[n * p.d + c] = from_f<T>(r);
      if (p.w_pre)
        static_cast<T*>(p.hidden)[n * p.d + c] =
            from_f<T>(r * ir * (ld_param<T>(p.w_pre, wf, c) + p.weight_offset));
    }
  }
}

// One row's element-wise quantities of the backward.
template <class T>
struct BwdElem {
  float xh, yh, gate, wq, wp, rh, dr, dh;
};
template <class T>
__device__ __forceinline__ BwdElem<T> bwd_elem(const NormBwd& p, int64_t n, int64_t c, float iy,
                                               float ir) {
  BwdElem<T> e;
  e.yh = 0.f;
  e.gate = 1.f;
  e.wq = 1.f;
  e.wp = 0.f;
  e.rh = 0.f;
  if (p.y) {
    e.yh = to_f<T>(static_cast<const T*>(p.y)[n * p.ldy + c]) * iy;
    if (p.w_post) e.wq = ld_param<T>(p.w_post, p.w_f32, c) + p.weight_offset;
    if (p.gate) e.gate = ld_param<T>(p.gate, p.gate_f32, n / p.rows_per_gate * p.d + c);
  }
  e.dr = p.d_residual ? to_f<T>(static_cast<const T*>(p.d_residual)[n * p.ld_dr + c]) : 0.f;
  e.dh = 0.f;
  if (p.w_pre) {
    e.dh = to_f<T>(static_cast<const T*>(p.d_hidden)[n * p.ld_dh + c]);
    e.wp = ld_param<T>(p.w_pre, p.w_f32, c) + p.weight_offset;
    const float x = to_f<T>(static_cast<const T*>(p.x)[n * p.ldx + c]);
    e.rh = ir * fmaf(p.block_scale * e.gate * e.wq, e.yh, p.residual_scale * x);
  }
  return e;
}

template <class T>
__global__ void __launch_bounds__(kAnyThreads) norm_bwd_rows_any(const NormBwd p) {
  const float inv_d = 1.f / static_cast<float>(p.d);
  for (int64_t n = blockIdx.x; n < p.N; n += gridDim.x) {
    const float iy = p.w_post ? p.rstd_post[n] : 1.f;
    const float ir = p.w_pre ? p.rstd_pre[n] : 0.f;
    float s[3] = {0.f, 0.f, 0.f};
    if (p.w_pre || p.w_post)
      for (int64_t c = threadIdx.x; c < p.d; c += kAnyThreads) {
        const BwdElem<T> e = bwd_elem<T>(p, n, c, iy, ir);
        const float u = e.dh * e.wp, ay = p.block_scale * e.gate * e.wq * e.yh;
        s[0] = fmaf(u, e.rh, s[0]);
        s[1] = fmaf(ay, fmaf(ir, u, e.dr), s[1]);
        s[2] = fmaf(ay, e.rh, s[2]);
      }
    block_sum(s);
    const float c1 = s[0] * inv_d;
    const float c2 = p.w_post ? (s[1] - ir * c1 * s[2]) * inv_d : 0.f;
    if (threadIdx.x == 0) p.c1[n] = c1;
    for (int64_t c = threadIdx.x; c < p.d; c += kAnyThreads) {
      const BwdElem<T> e = bwd_elem<T>(p, n, c, iy, ir);
      const float g = fmaf(ir, e.dh * e.wp - e.rh * c1, e.dr);
      static_cast<T*>(p.dx)[n * p.d + c] = from_f<T>(p.residual_scale * g);
      if (p.y) {
        const float a = p.block_scale * e.gate * e.wq;
        static_cast<T*>(p.dy)[n * p.d + c] = from_f<T>(iy * (a * g - e.yh * c2));
      }
      if (p.gate && p.rows_per_gate == 1) {
        const float dg = p.block_scale * e.yh * e.wq * g;
        if (p.gate_f32)
          static_cast<float*>(p.dgate)[n * p.d + c] = dg;
        else
          static_cast<T*>(p.dgate)[n * p.d + c] = from_f<T>(dg);
      }
    }
  }
}

// The column sums of row block blockIdx.y: weight gradients into its partial, shared gates'
// gradients into the group's partial (a slice of one group), or straight to the output
// (whole groups).
template <class T>
__global__ void __launch_bounds__(128) norm_bwd_cols_any(const NormBwd p) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
  if (c >= p.d) return;
  const int b = blockIdx.y;
  const NormRows rows = norm_rows(p.plan, b);
  float wpre = 0.f, wpost = 0.f;
  for (int64_t g = rows.g0; g < rows.g1; ++g) {
    float dg = 0.f;
    const int64_t n1 = rows.end(g);
    for (int64_t n = rows.begin(g); n < n1; ++n) {
      const float iy = p.w_post ? p.rstd_post[n] : 1.f;
      const float ir = p.w_pre ? p.rstd_pre[n] : 0.f;
      const BwdElem<T> e = bwd_elem<T>(p, n, c, iy, ir);
      const float gr = fmaf(ir, e.dh * e.wp - e.rh * p.c1[n], e.dr);
      const float by = p.block_scale * e.yh * gr;
      wpre = fmaf(e.dh, e.rh, wpre);
      wpost = fmaf(by, e.gate, wpost);
      dg = fmaf(by, e.wq, dg);
    }
    if (p.plan.shared_gate) {
      if (p.plan.slices > 1)
        p.part_gate[static_cast<int64_t>(b) * p.d + c] = dg;
      else if (p.gate_f32)
        static_cast<float*>(p.dgate)[g * p.d + c] = dg;
      else
        static_cast<T*>(p.dgate)[g * p.d + c] = from_f<T>(dg);
    }
  }
  if (p.w_post) p.part_post[static_cast<int64_t>(b) * p.d + c] = wpost;
  if (p.w_pre) p.part_pre[static_cast<int64_t>(b) * p.d + c] = wpre;
}

// Adds the row blocks' partials in a fixed order: blockIdx.y = 0 dw_post, 1 dw_pre, 2 + g the
// shared gate's row g (its slices' partials).  32 columns per block, 8 threads per column.
template <class T>
__global__ void __launch_bounds__(256) norm_bwd_reduce(const NormBwd p) {
  __shared__ float part[8][33];
  const int col = threadIdx.x & 31, sub = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + col;
  const float* src;
  int n;
  if (blockIdx.y < 2) {
    src = blockIdx.y == 0 ? p.part_post : p.part_pre;
    n = p.plan.blocks;
    if (blockIdx.y == 0 ? !p.w_post : !p.w_pre) return;
  } else {
    src = p.part_gate + static_cast<int64_t>(blockIdx.y - 2) * p.plan.slices * p.d;
    n = p.plan.slices;
  }
  float t = 0.f;
  if (c < p.d)
    for (int i = sub; i < n; i += 8) t += src[static_cast<int64_t>(i) * p.d + c];
  part[sub][col] = t;
  __syncthreads();
  if (sub != 0 || c >= p.d) return;
  for (int i = 1; i < 8; ++i) t += part[i][col];
  if (blockIdx.y == 0)
    p.dw_post[c] = t;
  else if (blockIdx.y == 1)
    p.dw_pre[c] = t;
  else if (p.gate_f32)
    static_cast<float*>(p.dgate)[(blockIdx.y - 2) * p.d + c] = t;
  else
    static_cast<T*>(p.dgate)[(blockIdx.y - 2) * p.d + c] = from_f<T>(t);
}

// ----------------------------------------------------------------------------------------
// 16-byte pieces: 8 bf16 / fp16 or 4 fp32 elements, as packed fp32 pairs.
// ----------------------------------------------------------------------------------------
template <class T>
struct Piece {
  static constexpr int kElems = 16 / sizeof(T);
  static constexpr int kPairs = kElems / 2;
  static __device__ __forceinline__ void unpack(const uint4& w, float2 (&v)[kPairs]) {
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
    if constexpr (std::is_same_v<T, float>) {
      v[0] = make_float2(__uint_as_float(a[0]), __uint_as_float(a[1]));
      v[1] = make_float2(__uint_as_float(a[2]), __uint_as_float(a[3]));
    } else if constexpr (std::is_same_v<T, __nv_bfloat16>) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = make_float2(__uint_as_float(a[i] << 16), __uint_as_float(a[i] & 0xffff0000u));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __half22float2(*reinterpret_cast<const __half2*>(&a[i]));
    }
  }
  static __device__ __forceinline__ uint4 pack(const float2 (&v)[kPairs]) {
    uint32_t a[4];
    if constexpr (std::is_same_v<T, float>) {
      a[0] = __float_as_uint(v[0].x);
      a[1] = __float_as_uint(v[0].y);
      a[2] = __float_as_uint(v[1].x);
      a[3] = __float_as_uint(v[1].y);
    } else if constexpr (std::is_same_v<T, __nv_bfloat16>) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[i].x, v[i].y);
        a[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(v[i].x, v[i].y);
        a[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    return make_uint4(a[0], a[1], a[2], a[3]);
  }
  // Piece `i` of a parameter array of type T or fp32 (T's piece width in both cases).
  static __device__ __forceinline__ void param(const void* p, bool f32, int64_t i,
                                               float2 (&v)[kPairs]) {
    if (!f32 || std::is_same_v<T, float>) {
      unpack(__ldg(static_cast<const uint4*>(p) + i), v);
    } else {
#pragma unroll
      for (int q = 0; q < kPairs / 2; ++q) {
        const float4 f = __ldg(static_cast<const float4*>(p) + i * (kPairs / 2) + q);
        v[2 * q] = make_float2(f.x, f.y);
        v[2 * q + 1] = make_float2(f.z, f.w);
      }
    }
  }
};

// Row data is used once: loaded past L1, which then keeps the weights.
__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ float2 pair(float v) { return make_float2(v, v); }

// Sum over the TPR threads of a row (a warp, or the whole block), in every one of them.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (TPR > 32) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < TPR / 32 ? part[lane] : 0.f;
#pragma unroll
    for (int o = TPR >= 1024 ? 16 : TPR / 64; o > 0; o >>= 1)
      v += __shfl_xor_sync(0xffffffffu, v, o);
    if (TPR < 1024) v = __shfl_sync(0xffffffffu, v, 0);
  }
  return v;
}

// Forward for rows of whole, aligned 16-byte pieces: each row is read once into the registers
// of its TPR threads (NV pieces of x and of y each), and r and h are written from there.
template <class T, int TPR, int NV>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) norm_fwd_vec(const NormFwd p) {
  using P = Piece<T>;
  constexpr int K = P::kPairs;
  constexpr int kRows = TPR < 128 ? 128 / TPR : 1;  // rows per block
  static_assert(TPR == 32 || TPR >= 128, "a row is a warp's or a block's");
  __shared__ float part[2][32];
  const int64_t n = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / TPR;
  const int t = threadIdx.x % TPR;
  if (kRows > 1 && n >= p.N) return;
  const int nvec = static_cast<int>(p.d / P::kElems);
  const uint4* x = reinterpret_cast<const uint4*>(static_cast<const T*>(p.x) + n * p.ldx);
  const uint4* y = reinterpret_cast<const uint4*>(static_cast<const T*>(p.y) + n * p.ldy);
  uint4 xv[NV], yv[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int i = t + v * TPR;
    xv[v] = yv[v] = make_uint4(0, 0, 0, 0);
    if (i < nvec) {
      // x may be written in place by this thread below: not through the read-only path.
      xv[v] = __ldcs(x + i);
      if (p.y) yv[v] = ld_stream(y + i);
    }
  }
  const float inv_d = 1.f / static_cast<float>(p.d);
  float iy = 1.f;
  if (p.w_post) {
    float2 s = pair(0.f);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float2 f[K];
      P::unpack(yv[v], f);
#pragma unroll
      for (int k = 0; k < K; ++k) s = fma2(f[k], f[k], s);
    }
    iy = rsqrtf(fmaf(row_sum<TPR>(s.x + s.y, part[0]), inv_d, p.eps));
    if (t == 0 && p.rstd_post) p.rstd_post[n] = iy;
  }
  const int64_t grow = p.gate ? n / p.rows_per_gate * nvec : 0;
  const float2 cy = pair(p.y ? p.block_scale * iy : 0.f), rs = pair(p.residual_scale);
  float2 r[NV][K];
  float2 s = pair(0.f);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int i = t + v * TPR;
    float2 f[K], w[K];
    P::unpack(xv[v], r[v]);
    P::unpack(yv[v], f);
#pragma unroll
    for (int k = 0; k < K; ++k) f[k] = mul2(f[k], cy);
    if (i < nvec) {
      if (p.w_post) {
        P::param(p.w_post, p.w_f32, i, w);
#pragma unroll
        for (int k = 0; k < K; ++k) f[k] = mul2(f[k], add2(w[k], pair(p.weight_offset)));
      }
      if (p.gate) {
        P::param(p.gate, p.gate_f32, grow + i, w);
#pragma unroll
        for (int k = 0; k < K; ++k) f[k] = mul2(f[k], w[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      r[v][k] = fma2(rs, r[v][k], f[k]);
      s = fma2(r[v][k], r[v][k], s);
    }
    if (i < nvec && p.residual)
      __stcs(reinterpret_cast<uint4*>(static_cast<T*>(p.residual) + n * p.d) + i, P::pack(r[v]));
  }
  if (!p.w_pre) return;
  const float ir = rsqrtf(fmaf(row_sum<TPR>(s.x + s.y, part[1]), inv_d, p.eps));
  if (t == 0 && p.rstd_pre) p.rstd_pre[n] = ir;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int i = t + v * TPR;
    if (i >= nvec) break;
    float2 w[K];
    P::param(p.w_pre, p.w_f32, i, w);
#pragma unroll
    for (int k = 0; k < K; ++k)
      w[k] = mul2(mul2(r[v][k], pair(ir)), add2(w[k], pair(p.weight_offset)));
    __stcs(reinterpret_cast<uint4*>(static_cast<T*>(p.hidden) + n * p.d) + i, P::pack(w));
  }
}

// ----------------------------------------------------------------------------------------
// Backward for rows of whole, aligned 16-byte pieces, in one pass: every row worker (a block,
// or a cluster of CL blocks that share a row's columns) walks its rows with the row data
// coming in through a ring of bulk copies, and keeps the column sums in registers.
//   warp 8      copies the rows' segments into the ring (cp.async.bulk, counted on an mbarrier)
//   warps 0-7   TPR threads per row, NV pieces each; a batch of 256 / TPR rows at a time
// Sweep 1 over a row forms the three sums, sweep 2 the outputs, both from shared memory.
// Only two parameters per column are needed in the loop: a = bs gate wq (bs wq with a gate per
// token) and wp.  The group's sum S = sum yh g serves two gradients, which are taken when the
// group ends:  dgate = bs wq S,  dw_post += bs gate S.
//   GATE   0 none or shared by the rows of a group; 1 per token, of the rows' type; 2 per
//          token, fp32 beside 16-bit rows
// ----------------------------------------------------------------------------------------
constexpr int kRingThreads = 256;  // computing threads; one more warp copies
constexpr int kMaxCluster = 8;

struct RingCtl {
  uint64_t full[4], empty[4], sums;
  int abort;
  float part[2][kMaxCluster * 8][3];
};

template <class T, int TPR, int NV, int GATE>
struct RingCfg {
  static constexpr int kRows = kRingThreads / TPR;      // rows per batch
  static constexpr int kCap = TPR * NV;                 // pieces per row segment, at most
  static constexpr int kSeg = kCap * 16;                // bytes of one array's row segment
  static constexpr int kGateSeg = GATE == 0 ? 0 : GATE == 1 ? kSeg : 2 * kSeg;
  static constexpr int kStage = kRows * (4 * kSeg + kGateSeg);
  static constexpr int kParams = 2 * kCap * Piece<T>::kElems * 4;  // a, wp
  static constexpr int kScratch = kRows > 1 ? kRingThreads * NV * Piece<T>::kElems * 4 : 0;
  static constexpr int kFixed = (static_cast<int>(sizeof(RingCtl)) + 127) / 128 * 128 + kParams + kScratch;
  // Two blocks per SM where two stages fit in half of it, so that one block's reductions
  // overlap the other's arithmetic.
  static constexpr int kHalf = 115712 - 128, kWhole = 232448 - 128;
  static constexpr int kFit2 = (kHalf - kFixed) / kStage, kFit1 = (kWhole - kFixed) / kStage;
  static constexpr int kStages = kFit2 >= 2 ? (kFit2 > 4 ? 4 : kFit2) : (kFit1 > 4 ? 4 : kFit1);
  static constexpr size_t kSmem = 128 + kFixed + static_cast<size_t>(kStages) * kStage;
  static_assert(kStages >= 2, "ring");
};

// wait_warp for a barrier that other blocks of the cluster arrive on after storing to this
// block's shared memory.
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort,
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

__device__ __forceinline__ void consumers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kRingThreads) : "memory");
}

template <class T, int TPR, int NV, int GATE, bool CL>
__global__ void __launch_bounds__(kRingThreads + 32, 2)
    norm_bwd_ring(const NormBwd p, const DevCtl ctl, const int seg) {
  using P = Piece<T>;
  using C = RingCfg<T, TPR, NV, GATE>;
  constexpr int K = P::kPairs, kRows = C::kRows, kCap = C::kCap, S = C::kStages;
  extern __shared__ uint8_t ring_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(ring_raw) + 127) &
                                             ~static_cast<uintptr_t>(127));
  RingCtl* rc = reinterpret_cast<RingCtl*>(base);
  float4* a4 = reinterpret_cast<float4*>(base + (sizeof(RingCtl) + 127) / 128 * 128);
  float4* wp4 = a4 + kCap * (K / 2);      // half h of piece i at [h * kCap + i]
  float4* scratch = wp4 + kCap * (K / 2);
  uint8_t* ring = reinterpret_cast<uint8_t*>(scratch) + C::kScratch;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cs = CL ? static_cast<int>(cluster_size()) : 1;
  const int rank = CL ? static_cast<int>(cluster_ctarank()) : 0;
  const int worker = static_cast<int>(blockIdx.x) / cs;
  const int nvec = static_cast<int>(p.d / P::kElems);
  const int piece0 = rank * seg;
  const int mine = min(seg, nvec - piece0);
  const NormRows rows = norm_rows(p.plan, worker);
  const bool has_y = p.y != nullptr, has_dr = p.d_residual != nullptr, pre = p.w_pre != nullptr;
  volatile int* abort = &rc->abort;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&rc->full[s], 1);
      mbar_init(&rc->empty[s], kRingThreads / 32);
    }
    mbar_init(&rc->sums, cs * (kRingThreads / 32));
    rc->abort = 0;
    fence_barrier_init();
  }
  if (CL)
    cluster_sync();
  else
    __syncthreads();

  if (warp == kRingThreads / 32) {
    // ------------------------------ copies ------------------------------
    const uint32_t bytes = static_cast<uint32_t>(mine) * 16;
    const uint32_t gbytes = GATE == 2 ? 2 * bytes : bytes;
    const int narr = 5;
    const uint32_t row_bytes = bytes * (has_y + has_dr + 2 * pre) + (GATE ? gbytes : 0);
    uint32_t it = 0;
    bool ok = true;
    for (int64_t g = rows.g0; ok && g < rows.g1; ++g) {
      const int64_t n1 = rows.end(g);
      for (int64_t n = rows.begin(g); n < n1; n += kRows, ++it) {
        const int s = it % S;
        if (!wait_warp(&rc->empty[s], ((it / S) & 1u) ^ 1u, abort, ctl)) {
          ok = false;
          break;
        }
        const int valid = static_cast<int>(min(static_cast<int64_t>(kRows), n1 - n));
        if (lane == 0) mbar_arrive_expect_tx(&rc->full[s], row_bytes * valid);
        __syncwarp();
        uint8_t* st = ring + s * C::kStage;
        for (int q = lane; q < valid * narr; q += 32) {
          const int arr = q % narr, rw = q / narr;
          const int64_t row = n + rw;
          const uint8_t* src = nullptr;
          int64_t ld = 0;
          if (arr == 0) {
            src = pre ? static_cast<const uint8_t*>(p.x) : nullptr;
            ld = p.ldx;
          } else if (arr == 1) {
            src = static_cast<const uint8_t*>(p.y);
            ld = p.ldy;
          } else if (arr == 2) {
            src = static_cast<const uint8_t*>(p.d_residual);
            ld = p.ld_dr;
          } else if (arr == 3) {
            src = pre ? static_cast<const uint8_t*>(p.d_hidden) : nullptr;
            ld = p.ld_dh;
          } else if (GATE) {
            src = static_cast<const uint8_t*>(p.gate);
            ld = p.d;
          }
          if (!src) continue;
          if (arr < 4)
            bulk_load(st + arr * kRows * C::kSeg + rw * C::kSeg,
                      src + row * ld * sizeof(T) + static_cast<int64_t>(piece0) * 16, bytes,
                      &rc->full[s]);
          else
            bulk_load(st + 4 * kRows * C::kSeg + rw * C::kGateSeg,
                      src + (row * ld * sizeof(T) + static_cast<int64_t>(piece0) * 16) *
                                (GATE == 2 ? 2 : 1),
                      gbytes, &rc->full[s]);
        }
        __syncwarp();
      }
    }
    if (!ok) {
      // Copies in flight land before the block leaves.
      const uint32_t first = it > static_cast<uint32_t>(S) ? it - S : 0u;
      for (uint32_t q = first; q < it; ++q)
        wait_warp(&rc->full[q % S], (q / S) & 1u, abort, ctl, false);
    }
  } else {
    // ------------------------------ arithmetic ------------------------------
    const int rw = threadIdx.x / TPR, t = threadIdx.x % TPR;
    const float2 zero = pair(0.f);
    const float2 off = pair(p.weight_offset), bs = pair(p.block_scale), rs = pair(p.residual_scale);
    const float inv_d = 1.f / static_cast<float>(p.d);
    float2 acc_s[NV][K], acc_p[NV][K];
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int k = 0; k < K; ++k) acc_s[v][k] = acc_p[v][k] = zero;

    auto put = [&](float4* dst, int i, const float2(&v)[K]) {
#pragma unroll
      for (int h = 0; h < K / 2; ++h)
        dst[h * kCap + i] = make_float4(v[2 * h].x, v[2 * h].y, v[2 * h + 1].x, v[2 * h + 1].y);
    };
    auto get = [&](const float4* src, int i, float2(&v)[K]) {
#pragma unroll
      for (int h = 0; h < K / 2; ++h) {
        const float4 f = src[h * kCap + i];
        v[2 * h] = make_float2(f.x, f.y);
        v[2 * h + 1] = make_float2(f.z, f.w);
      }
    };
    // wq of piece i, and bs times the group's gate.
    auto load_wq = [&](int i, float2(&w)[K]) {
      if (p.w_post) {
        P::param(p.w_post, p.w_f32, piece0 + i, w);
#pragma unroll
        for (int k = 0; k < K; ++k) w[k] = add2(w[k], off);
      } else {
#pragma unroll
        for (int k = 0; k < K; ++k) w[k] = pair(1.f);
      }
    };
    auto load_gs = [&](int64_t g, int i, float2(&w)[K]) {
      if (GATE == 0 && p.gate) {
        P::param(p.gate, p.gate_f32, g * nvec + piece0 + i, w);
#pragma unroll
        for (int k = 0; k < K; ++k) w[k] = mul2(w[k], bs);
      } else {
#pragma unroll
        for (int k = 0; k < K; ++k) w[k] = bs;
      }
    };
    // The column sums of the batch's row lanes, added in a fixed order into lane 0's.
    auto join = [&](float2(&acc)[NV][K]) {
      if (kRows == 1) return;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int h = 0; h < K / 2; ++h)
          scratch[(v * (K / 2) + h) * kRingThreads + threadIdx.x] =
              make_float4(acc[v][2 * h].x, acc[v][2 * h].y, acc[v][2 * h + 1].x, acc[v][2 * h + 1].y);
      consumers_sync();
      if (rw == 0)
        for (int o = 1; o < kRows; ++o)
#pragma unroll
          for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int h = 0; h < K / 2; ++h) {
              const float4 f = scratch[(v * (K / 2) + h) * kRingThreads + threadIdx.x + o * TPR];
              acc[v][2 * h] = add2(acc[v][2 * h], make_float2(f.x, f.y));
              acc[v][2 * h + 1] = add2(acc[v][2 * h + 1], make_float2(f.z, f.w));
            }
      consumers_sync();
    };
    // Pieces of an fp32 output row.
    auto store_f32 = [&](float* dst, int i, const float2(&v)[K], bool add) {
      float4* o = reinterpret_cast<float4*>(dst) + static_cast<int64_t>(piece0 + i) * (K / 2);
#pragma unroll
      for (int h = 0; h < K / 2; ++h) {
        float4 f = make_float4(v[2 * h].x, v[2 * h].y, v[2 * h + 1].x, v[2 * h + 1].y);
        if (add) {
          const float4 q = o[h];
          f = make_float4(f.x + q.x, f.y + q.y, f.z + q.z, f.w + q.w);
        }
        o[h] = f;
      }
    };
    auto store_param_grad = [&](void* dst, bool f32, int64_t row, int i, const float2(&v)[K]) {
      if (f32)
        store_f32(static_cast<float*>(dst) + row * p.d, i, v, false);
      else
        reinterpret_cast<uint4*>(static_cast<T*>(dst) + row * p.d)[piece0 + i] = P::pack(v);
    };

    // wp for the whole run; a per group.
    if (rw == 0)
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int i = t + v * TPR;
        if (i >= mine) break;
        float2 w[K];
        if (pre) {
          P::param(p.w_pre, p.w_f32, piece0 + i, w);
#pragma unroll
          for (int k = 0; k < K; ++k) w[k] = add2(w[k], off);
        } else {
#pragma unroll
          for (int k = 0; k < K; ++k) w[k] = zero;
        }
        put(wp4, i, w);
      }

    uint32_t it = 0;
    float iy = 1.f, ir = 0.f;
    auto factors = [&](int64_t n, float& fy, float& fr) {
      if (n < p.N) {
        fy = p.w_post ? __ldg(p.rstd_post + n) : 1.f;
        fr = pre ? __ldg(p.rstd_pre + n) : 0.f;
      }
    };
    factors(rows.begin(rows.g0) + rw, iy, ir);
    for (int64_t g = rows.g0; g < rows.g1; ++g) {
      if (rw == 0)
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const int i = t + v * TPR;
          if (i >= mine) break;
          float2 w[K], q[K];
          load_wq(i, w);
          load_gs(g, i, q);
#pragma unroll
          for (int k = 0; k < K; ++k) w[k] = has_y ? mul2(w[k], q[k]) : zero;
          put(a4, i, w);
        }
      if (kRows > 1) consumers_sync();
      const int64_t n1 = rows.end(g);
      for (int64_t nb = rows.begin(g); nb < n1; nb += kRows, ++it) {
        const int s = it % S;
        const int64_t n = nb + rw;
        const bool live = n < n1;
        float iy_next = 1.f, ir_next = 0.f;
        factors((nb + kRows < n1 ? nb + kRows : rows.begin(g + 1)) + rw, iy_next, ir_next);
        wait_warp(&rc->full[s], (it / S) & 1u, abort, ctl);
        const uint8_t* st = ring + s * C::kStage + rw * C::kSeg;
        const uint4* sx = reinterpret_cast<const uint4*>(st);
        const uint4* sy = reinterpret_cast<const uint4*>(st + kRows * C::kSeg);
        const uint4* sr = reinterpret_cast<const uint4*>(st + 2 * kRows * C::kSeg);
        const uint4* sh = reinterpret_cast<const uint4*>(st + 3 * kRows * C::kSeg);
        const uint8_t* sg = ring + s * C::kStage + 4 * kRows * C::kSeg + rw * C::kGateSeg;
        const float2 iy2 = pair(iy), ir2 = pair(ir);
        // Everything both sweeps need of piece i.
        auto load = [&](int i, float2(&a)[K], float2(&gate)[K], float2(&yh)[K], float2(&rh)[K],
                        float2(&dh)[K], float2(&u)[K], float2(&tt)[K]) {
          float2 x[K];
          get(a4, i, a);
          get(wp4, i, u);
          if (pre)
            P::unpack(sx[i], x);
          if (GATE == 1) P::unpack(reinterpret_cast<const uint4*>(sg)[i], gate);
          if (GATE == 2) {
#pragma unroll
            for (int h = 0; h < K / 2; ++h) {
              const float4 f = reinterpret_cast<const float4*>(sg)[i * (K / 2) + h];
              gate[2 * h] = make_float2(f.x, f.y);
              gate[2 * h + 1] = make_float2(f.z, f.w);
            }
          }
          if (has_y)
            P::unpack(sy[i], yh);
          else
#pragma unroll
            for (int k = 0; k < K; ++k) yh[k] = zero;
          if (pre)
            P::unpack(sh[i], dh);
          else
#pragma unroll
            for (int k = 0; k < K; ++k) dh[k] = zero;
          if (has_dr)
            P::unpack(sr[i], tt);
          else
#pragma unroll
            for (int k = 0; k < K; ++k) tt[k] = zero;
#pragma unroll
          for (int k = 0; k < K; ++k) {
            yh[k] = mul2(yh[k], iy2);
            const float2 ag = GATE ? mul2(a[k], gate[k]) : a[k];
            rh[k] = pre ? mul2(ir2, fma2(rs, x[k], mul2(ag, yh[k]))) : zero;
            u[k] = mul2(dh[k], u[k]);
            tt[k] = fma2(ir2, u[k], tt[k]);
          }
        };
        float2 s0 = zero, s1 = zero, s2 = zero;
        if (live)
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            const int i = t + v * TPR;
            if (i >= mine) break;
            float2 a[K], gate[K], yh[K], rh[K], dh[K], u[K], tt[K];
            load(i, a, gate, yh, rh, dh, u, tt);
#pragma unroll
            for (int k = 0; k < K; ++k) {
              const float2 ay = mul2(GATE ? mul2(a[k], gate[k]) : a[k], yh[k]);
              s0 = fma2(u[k], rh[k], s0);
              s1 = fma2(ay, tt[k], s1);
              s2 = fma2(ay, rh[k], s2);
            }
          }
        float v3[3] = {s0.x + s0.y, s1.x + s1.y, s2.x + s2.y};
#pragma unroll
        for (int k = 0; k < 3; ++k)
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) v3[k] += __shfl_xor_sync(0xffffffffu, v3[k], o);
        if (CL) {
          // Every warp hands its sums to each block of the cluster; lane c serves block c.
          if (lane < cs) {
            float* slot = rc->part[it & 1][rank * 8 + warp];
            const uint32_t dst = mapa_shared(smem_u32(slot), lane);
#pragma unroll
            for (int k = 0; k < 3; ++k) st_shared_cluster_u32(dst + 4 * k, __float_as_uint(v3[k]));
            mbar_arrive_cluster(mapa_shared(smem_u32(&rc->sums), lane));
          }
          __syncwarp();
          wait_cluster(&rc->sums, it & 1u, abort, ctl);
        } else if (TPR > 32) {
          if (lane == 0)
#pragma unroll
            for (int k = 0; k < 3; ++k) rc->part[it & 1][warp][k] = v3[k];
          consumers_sync();
        }
        if (CL || TPR > 32) {
          const int w0 = CL ? 0 : rw * (TPR / 32), nw = CL ? cs * 8 : TPR / 32;
          v3[0] = v3[1] = v3[2] = 0.f;
          for (int w = 0; w < nw; ++w)
#pragma unroll
            for (int k = 0; k < 3; ++k) v3[k] += rc->part[it & 1][w0 + w][k];
        }
        const float c1 = v3[0] * inv_d;
        const float c2 = p.w_post ? (v3[1] - ir * c1 * v3[2]) * inv_d : 0.f;
        const float2 kg = pair(-ir * c1), ky = pair(-iy * c2);
        if (live)
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            const int i = t + v * TPR;
            if (i >= mine) break;
            float2 a[K], gate[K], yh[K], rh[K], dh[K], u[K], g2[K], o[K];
            load(i, a, gate, yh, rh, dh, u, g2);
#pragma unroll
            for (int k = 0; k < K; ++k) {
              g2[k] = fma2(kg, rh[k], g2[k]);
              o[k] = mul2(rs, g2[k]);
              acc_p[v][k] = fma2(dh[k], rh[k], acc_p[v][k]);
            }
            const int64_t at = n * nvec + piece0 + i;
            __stcs(static_cast<uint4*>(p.dx) + at, P::pack(o));
            if (has_y) {
#pragma unroll
              for (int k = 0; k < K; ++k) {
                const float2 yg = mul2(yh[k], g2[k]);
                const float2 ag = GATE ? mul2(a[k], gate[k]) : a[k];
                acc_s[v][k] = GATE ? fma2(gate[k], yg, acc_s[v][k]) : add2(yg, acc_s[v][k]);
                o[k] = fma2(ky, yh[k], mul2(mul2(iy2, ag), g2[k]));
                if (GATE) g2[k] = mul2(a[k], yg);
              }
              __stcs(static_cast<uint4*>(p.dy) + at, P::pack(o));
              if (GATE) store_param_grad(p.dgate, GATE == 2 || std::is_same_v<T, float>, n, i, g2);
            }
          }
        __syncwarp();
        if (lane == 0) mbar_arrive(&rc->empty[s]);
        iy = iy_next;
        ir = ir_next;
      }
      if (GATE == 0 && (p.w_post || p.gate)) {
        // The group's end: its S into the gate's and the post weight's gradients.
        join(acc_s);
        if (rw == 0)
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            const int i = t + v * TPR;
            if (i >= mine) break;
            float2 w[K], q[K];
            load_wq(i, w);
            load_gs(g, i, q);
#pragma unroll
            for (int k = 0; k < K; ++k) {
              q[k] = mul2(q[k], acc_s[v][k]);
              w[k] = mul2(mul2(w[k], bs), acc_s[v][k]);
            }
            if (p.w_post)
              store_f32(p.part_post + static_cast<int64_t>(worker) * p.d, i, q, g > rows.g0);
            if (p.gate) {
              if (p.plan.slices > 1)
                store_f32(p.part_gate + static_cast<int64_t>(worker) * p.d, i, w, false);
              else
                store_param_grad(p.dgate, p.gate_f32, g, i, w);
            }
          }
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int k = 0; k < K; ++k) acc_s[v][k] = zero;
      }
    }
    if (GATE && p.w_post) {
      join(acc_s);
      if (rw == 0)
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const int i = t + v * TPR;
          if (i >= mine) break;
#pragma unroll
          for (int k = 0; k < K; ++k) acc_s[v][k] = mul2(bs, acc_s[v][k]);
          store_f32(p.part_post + static_cast<int64_t>(worker) * p.d, i, acc_s[v], false);
        }
    }
    if (pre) {
      join(acc_p);
      if (rw == 0)
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const int i = t + v * TPR;
          if (i >= mine) break;
          store_f32(p.part_pre + static_cast<int64_t>(worker) * p.d, i, acc_p[v], false);
        }
    }
  }
  // No block leaves while another of its cluster may still write its sums into it.
  if (CL) {
    __syncwarp();
    cluster_sync();
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <class T, int TPR, int NV>
cudaError_t fwd_vec(const NormFwd& p, cudaStream_t s) {
  constexpr int kRows = TPR < 128 ? 128 / TPR : 1;
  const int64_t grid = (p.N + kRows - 1) / kRows;
  norm_fwd_vec<T, TPR, NV><<<static_cast<unsigned>(grid), TPR < 128 ? 128 : TPR, 0, s>>>(p);
  return cudaGetLastError();
}

template <class T>
cudaError_t fwd_t(const NormFwd& p, cudaStream_t s) {
  constexpr int E = Piece<T>::kElems;
  const int64_t nvec = p.d / E;
  const bool vec = p.d % E == 0 && nvec <= 4096 && p.ldx % E == 0 && (!p.y || p.ldy % E == 0) &&
                   aligned16(p.x) && aligned16(p.y) && aligned16(p.w_post) && aligned16(p.w_pre) &&
                   aligned16(p.gate) && aligned16(p.residual) && aligned16(p.hidden);
  if (!vec) {
    const int64_t grid = std::min<int64_t>(p.N, int64_t(1) << 20);
    norm_fwd_any<T><<<static_cast<unsigned>(grid), kAnyThreads, 0, s>>>(p);
    return cudaGetLastError();
  }
  const bool few = p.N <= 2 * sm_count();
  if (nvec <= 32) return fwd_vec<T, 32, 1>(p, s);
  if (nvec <= 64 && !few) return fwd_vec<T, 32, 2>(p, s);
  if (nvec <= 128) return fwd_vec<T, 128, 1>(p, s);
  if (nvec <= 256) return few ? fwd_vec<T, 256, 1>(p, s) : fwd_vec<T, 128, 2>(p, s);
  if (nvec <= 512) return few ? fwd_vec<T, 512, 1>(p, s) : fwd_vec<T, 256, 2>(p, s);
  if (nvec <= 1024) return few ? fwd_vec<T, 1024, 1>(p, s) : fwd_vec<T, 512, 2>(p, s);
  if (nvec <= 2048) return few ? fwd_vec<T, 1024, 2>(p, s) : fwd_vec<T, 512, 4>(p, s);
  return fwd_vec<T, 1024, 4>(p, s);
}

template <class T>
cudaError_t bwd_sums(const NormBwd& p, cudaStream_t s) {
  const bool gates = p.plan.shared_gate && p.plan.slices > 1;
  if (!p.w_post && !p.w_pre && !gates) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>((p.d + 31) / 32),
                  static_cast<unsigned>(2 + (gates ? p.plan.groups : 0)));
  norm_bwd_reduce<T><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

template <class T, int TPR, int NV, int GATE, bool CL>
cudaError_t bwd_ring(NormBwd p, const DevCtl& c, int cs, cudaStream_t s) {
  using C = RingCfg<T, TPR, NV, GATE>;
  auto kern = norm_bwd_ring<T, TPR, NV, GATE, CL>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(kRingThreads + 32, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // Per device and cluster size, once: how many workers can be resident.
  static int resident[64][4] = {};
  int& most = resident[dev][cs == 1 ? 0 : cs == 2 ? 1 : cs == 4 ? 2 : 3];
  if (most == 0) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(C::kSmem));
    if (e != cudaSuccess) return e;
    int n = 0;
    cfg.gridDim = dim3(static_cast<unsigned>(512 * cs), 1, 1);
    if ((e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg)) != cudaSuccess) return e;
    most = n > 0 ? n : 1;
  }
  const int workers = std::min(most, kNormBlocks);
  p.plan = norm_plan(p.N, p.rows_per_gate, p.gate != nullptr, workers, C::kRows);
  const int nvec = static_cast<int>(p.d / Piece<T>::kElems);
  cfg.gridDim = dim3(static_cast<unsigned>(p.plan.blocks * cs), 1, 1);
  if ((e = cudaLaunchKernelEx(&cfg, kern, p, c, (nvec + cs - 1) / cs)) != cudaSuccess) return e;
  return bwd_sums<T>(p, s);
}

template <class T, int GATE>
cudaError_t bwd_vec(const NormBwd& p, const DevCtl& c, cudaStream_t s) {
  const int64_t nvec = p.d / Piece<T>::kElems;
  if (nvec <= 32) return bwd_ring<T, 32, 1, GATE, false>(p, c, 1, s);
  if (nvec <= 64) return bwd_ring<T, 64, 1, GATE, false>(p, c, 1, s);
  if (nvec <= 128) return bwd_ring<T, 128, 1, GATE, false>(p, c, 1, s);
  if (nvec <= 256) return bwd_ring<T, 256, 1, GATE, false>(p, c, 1, s);
  if (nvec <= 512) return bwd_ring<T, 256, 2, GATE, false>(p, c, 1, s);
  return bwd_ring<T, 256, 2, GATE, true>(p, c, nvec <= 1024 ? 2 : nvec <= 2048 ? 4 : 8, s);
}

template <class T>
cudaError_t bwd_t(const NormBwd& p, const DevCtl& c, cudaStream_t s) {
  constexpr int E = Piece<T>::kElems;
  const bool vec = p.d % E == 0 && p.d / E <= 512 * kMaxCluster && p.ldx % E == 0 &&
                   (!p.y || p.ldy % E == 0) && (!p.d_residual || p.ld_dr % E == 0) &&
                   (!p.d_hidden || p.ld_dh % E == 0) && aligned16(p.x) && aligned16(p.y) &&
                   aligned16(p.d_residual) && aligned16(p.d_hidden) && aligned16(p.w_post) &&
                   aligned16(p.w_pre) && aligned16(p.gate) && aligned16(p.dx) &&
                   aligned16(p.dy) && aligned16(p.dgate);
  if (vec) {
    if (!p.gate || p.plan.shared_gate) return bwd_vec<T, 0>(p, c, s);
    if constexpr (!std::is_same_v<T, float>)
      if (p.gate_f32) return bwd_vec<T, 2>(p, c, s);
    return bwd_vec<T, 1>(p, c, s);
  }
  const int64_t grid = std::min<int64_t>(p.N, int64_t(1) << 20);
  norm_bwd_rows_any<T><<<static_cast<unsigned>(grid), kAnyThreads, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !(p.w_post || p.w_pre || p.plan.shared_gate)) return e;
  const dim3 gc(static_cast<unsigned>((p.d + 127) / 128), static_cast<unsigned>(p.plan.blocks));
  norm_bwd_cols_any<T><<<gc, 128, 0, s>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return bwd_sums<T>(p, s);
}

}  // namespace

NormPlan norm_plan(int64_t N, int64_t rows_per_gate, bool has_gate, int max_blocks, int batch) {
  NormPlan q{};
  q.shared_gate = has_gate && rows_per_gate > 1;
  q.rows = q.shared_gate ? rows_per_gate : N;
  q.groups = q.shared_gate ? N / rows_per_gate : 1;
  // Blocks own either one slice of one group or several whole groups.
  const int64_t most = (q.rows + batch - 1) / batch;  // no slice below a batch of rows
  q.slices = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(most, max_blocks / q.groups)));
  q.blocks = static_cast<int>(q.slices > 1 ? q.groups * q.slices
                                           : std::min<int64_t>(q.groups, max_blocks));
  return q;
}

cudaError_t launch_norm_fwd(int dtype, const NormFwd& p, cudaStream_t s) {
  if (dtype == 0) return fwd_t<__nv_bfloat16>(p, s);
  if (dtype == 1) return fwd_t<__half>(p, s);
  return fwd_t<float>(p, s);
}

cudaError_t launch_norm_bwd(int dtype, const NormBwd& p, const DevCtl& c, cudaStream_t s) {
  if (dtype == 0) return bwd_t<__nv_bfloat16>(p, c, s);
  if (dtype == 1) return bwd_t<__half>(p, c, s);
  return bwd_t<float>(p, c, s);
}

}  // namespace slm
