// slm_norm.cuh - norms before and after a draft block, fused with its gate and its residual
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

#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "slm_internal.h"
#include "slm_norm_rows.h"
#include "slm_ran_out.cuh"
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
// row read again (from L1 / L2) for each of its sweeps.  For arrays whose rows do not start equally
// far from 16-byte boundaries, rows wider than the kernels below take, and in the backward rows
// narrower than a piece; bound by its element
// accesses.  16384 x 4096 bf16: forward 364 us and backward 1778, by pieces 85 and 155.
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
__global__ void __launch_bounds__(kAnyThreads) norm_bwd_rows_any(const NormBwd p, int* status) {
  if (blockIdx.x == 0 && threadIdx.x == 0) *status = 0;
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
        static_cast<T*>(p.dy)[n * p.d + c] = from_f<T>(p.w_post ? iy * (a * g - e.yh * c2) : a * g);
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
      if (p.plan.parts() > 1)
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
    n = p.plan.parts();
    src = p.part_gate + static_cast<int64_t>(blockIdx.y - 2) * n * p.d;
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

// Rows that do not start on a 16-byte boundary: piece i of a row covers the columns
// c .. c + kElems - 1 with c = kElems i - shift, so that every piece but the row's first and last
// is a whole aligned one; those two are taken element by element.  Elements outside [0, d)
// read as 0 and are not written.
template <class T>
struct Edge {
  static constexpr int E = Piece<T>::kElems, K = Piece<T>::kPairs;
  static __device__ __forceinline__ bool is(int c, int d) { return c < 0 || c + E > d; }
  static __device__ __forceinline__ void load(const T* row, int c, int d, float2 (&v)[K]) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int a = c + 2 * k;
      v[k].x = a >= 0 && a < d ? to_f<T>(row[a]) : 0.f;
      v[k].y = a + 1 >= 0 && a + 1 < d ? to_f<T>(row[a + 1]) : 0.f;
    }
  }
  static __device__ __forceinline__ void store(T* row, int c, int d, const float2 (&v)[K]) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int a = c + 2 * k;
      if (a >= 0 && a < d) row[a] = from_f<T>(v[k].x);
      if (a + 1 >= 0 && a + 1 < d) row[a + 1] = from_f<T>(v[k].y);
    }
  }
  static __device__ __forceinline__ void mask(int c, int d, float2 (&v)[K]) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int a = c + 2 * k;
      if (a < 0 || a >= d) v[k].x = 0.f;
      if (a + 1 < 0 || a + 1 >= d) v[k].y = 0.f;
    }
  }
  // Parameters (T or fp32) of columns c .. c + E - 1.
  static __device__ __forceinline__ void param(const void* p, bool f32, int64_t at, int c, int d,
                                               float2 (&v)[K]) {
    if (f32)
      Edge<float>::row(static_cast<const float*>(p) + at, c, d, v);
    else
      row(static_cast<const T*>(p) + at, c, d, v);
  }
  // Inside the array by two aligned loads and a shift (the same for all lanes: their columns
  // are whole pieces apart), near its ends element by element.
  template <int K2>
  static __device__ __forceinline__ void row(const T* q, int c, int d, float2 (&v)[K2]) {
    if (c < 2 * K2 - 1 || c + 4 * K2 > d) {
#pragma unroll
      for (int k = 0; k < K2; ++k) {
        const int a = c + 2 * k;
        v[k].x = a >= 0 && a < d ? to_f<T>(__ldg(q + a)) : 0.f;
        v[k].y = a + 1 >= 0 && a + 1 < d ? to_f<T>(__ldg(q + a + 1)) : 0.f;
      }
      return;
    }
    constexpr int kWords = 2 * K2 * static_cast<int>(sizeof(T)) / 4;  // words of the columns
    const uintptr_t at = reinterpret_cast<uintptr_t>(q + c);
    const uint4* from = reinterpret_cast<const uint4*>(at & ~static_cast<uintptr_t>(15));
    const int off = static_cast<int>(at & 15);
    uint32_t w[kWords + 4];
#pragma unroll
    for (int i = 0; i < kWords / 4 + 1; ++i) {
      const uint4 u = i < kWords / 4 || off != 0 ? __ldg(from + i) : make_uint4(0, 0, 0, 0);
      w[4 * i] = u.x;
      w[4 * i + 1] = u.y;
      w[4 * i + 2] = u.z;
      w[4 * i + 3] = u.w;
    }
    if (off & 8)
#pragma unroll
      for (int i = 0; i < kWords + 2; ++i) w[i] = w[i + 2];
    if (off & 4)
#pragma unroll
      for (int i = 0; i < kWords + 1; ++i) w[i] = w[i + 1];
    if (sizeof(T) == 2 && (off & 2))
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = __byte_perm(w[i], w[i + 1], 0x5432);
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) {
      float2 f[K];
      Piece<T>::unpack(make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]), f);
#pragma unroll
      for (int k = 0; k < K; ++k) v[i * K + k] = f[k];
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
// Packed fp32 pairs: two operations, each rounded as its scalar form, in one instruction.
__device__ __forceinline__ float2 pair(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }

// Sum over a row's threads (a warp, or the whole block), in every one of them.
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (!WARP) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < (blockDim.x >> 5) ? part[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  }
  return v;
}

// Forward by 16-byte pieces: each row is read once into the registers
// of its threads (NV pieces of x and of y each), and r and h are written from there.  A row is a
// block's, as many warps as it has pieces for, or, if short (WARP), one warp's of four.  Bound by
// memory: x and y in, r and h out.  16384 x 4096 bf16 85 us, 6.3 TB/s.  Rows that are not 16-byte
// aligned also align the parameters of every piece of every row and mask its elements, which bounds
// 16-bit ones (16384 x 4097 bf16 222 us, 2.4 TB/s; 16384 x 1001 fp32 with a gate per token, five
// arrays, 67 us, 4.9 TB/s).  One row of 4096 takes 2.9 us.
template <class T, int NV, bool WARP, bool SHIFT>
__global__ void __launch_bounds__(WARP ? 128 : NV == 2 ? 512 : 1024) norm_fwd_vec(const NormFwd p) {
  using P = Piece<T>;
  constexpr int K = P::kPairs;
  __shared__ float part[2][32];
  const int TPR = WARP ? 32 : blockDim.x;  // threads per row
  const int64_t n =
      WARP ? static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5) : static_cast<int64_t>(blockIdx.x);
  const int t = WARP ? threadIdx.x & 31 : threadIdx.x;
  if (WARP && n >= p.N) return;
  // SHIFT: the row starts `shift` elements after an aligned piece (the same in every array).
  const int d = static_cast<int>(p.d);
  const int shift = SHIFT ? static_cast<int>((p.shift0 + n * p.d) % P::kElems) : 0;
  const int nvec = static_cast<int>((p.d + shift + P::kElems - 1) / P::kElems);
  const T* xrow = static_cast<const T*>(p.x) + n * p.ldx;
  const T* yrow = static_cast<const T*>(p.y) + n * p.ldy;
  const uint4* x = reinterpret_cast<const uint4*>(xrow - shift);
  const uint4* y = reinterpret_cast<const uint4*>(yrow - shift);
  uint4 xv[NV], yv[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int i = t + v * TPR;
    xv[v] = yv[v] = make_uint4(0, 0, 0, 0);
    if (i < nvec) {
      const int c = i * P::kElems - shift;
      if (SHIFT && Edge<T>::is(c, d)) {
        float2 f[K];
        Edge<T>::load(xrow, c, d, f);
        xv[v] = P::pack(f);
        if (p.y) {
          Edge<T>::load(yrow, c, d, f);
          yv[v] = P::pack(f);
        }
      } else {
        // x may be written in place by this thread below: not through the read-only path.
        xv[v] = __ldcs(x + i);
        if (p.y) yv[v] = ld_stream(y + i);
      }
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
    iy = rsqrtf(fmaf(row_sum<WARP>(s.x + s.y, part[0]), inv_d, p.eps));
    if (t == 0 && p.rstd_post) p.rstd_post[n] = iy;
  }
  const int64_t grow = p.gate ? n / p.rows_per_gate * p.d : 0;
  // Parameters of piece i, and r or h out of it.
  auto param = [&](const void* q, bool f32, int64_t at, int i, float2(&w)[K]) {
    if (SHIFT)
      Edge<T>::param(q, f32, at, i * P::kElems - shift, d, w);
    else
      P::param(q, f32, at / P::kElems + i, w);
  };
  auto store = [&](void* q, int i, const float2(&w)[K]) {
    T* row = static_cast<T*>(q) + n * p.d;
    const int c = i * P::kElems - shift;
    if (SHIFT && Edge<T>::is(c, d))
      Edge<T>::store(row, c, d, w);
    else
      __stcs(reinterpret_cast<uint4*>(row - shift) + i, P::pack(w));
  };
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
        param(p.w_post, p.w_f32, 0, i, w);
#pragma unroll
        for (int k = 0; k < K; ++k) f[k] = mul2(f[k], add2(w[k], pair(p.weight_offset)));
      }
      if (p.gate) {
        param(p.gate, p.gate_f32, grow, i, w);
#pragma unroll
        for (int k = 0; k < K; ++k) f[k] = mul2(f[k], w[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      r[v][k] = fma2(rs, r[v][k], f[k]);
      s = fma2(r[v][k], r[v][k], s);
    }
    if (i < nvec && p.residual) store(p.residual, i, r[v]);
  }
  if (!p.w_pre) return;
  const float ir = rsqrtf(fmaf(row_sum<WARP>(s.x + s.y, part[1]), inv_d, p.eps));
  if (t == 0 && p.rstd_pre) p.rstd_pre[n] = ir;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int i = t + v * TPR;
    if (i >= nvec) break;
    float2 w[K];
    param(p.w_pre, p.w_f32, 0, i, w);
#pragma unroll
    for (int k = 0; k < K; ++k)
      w[k] = mul2(mul2(r[v][k], pair(ir)), add2(w[k], pair(p.weight_offset)));
    store(p.hidden, i, w);
  }
}

// ----------------------------------------------------------------------------------------
// Backward by 16-byte pieces, in one pass: every row worker (a block,
// or a cluster of blocks that share a row's columns) walks its rows, a batch of 256 / TPR at
// a time.
//   warp 8      copies the batches' row segments into a ring (cp.async.bulk, counted on
//               mbarriers)
//   warps 0-7   TPR threads per row, NV pieces of each array per thread; parameters and column
//               sums stay in registers, as every thread keeps its columns
// Sweep 1 over a batch forms the rows' three sums, sweep 2 the outputs, both from the ring.
// Sweep 1 runs one batch ahead, so that the sums are exchanged behind sweep 2 of the batch
// before: at most one block barrier per batch, and a cluster's exchange is off the critical path.
// Bound by memory for fp32 (8192 x 4096 136 us, 5.9 TB/s), by instructions for 16-bit rows
// (16384 x 4096 bf16 155 us, 5.2 TB/s: twice the conversions and arithmetic per byte, between
// dependent reads of shared memory).  The general kernels, which read global memory twice, take
// 1778 us there; sweeps in step, without the batch between them, took 207.
// Only two parameters per column are needed in the loop: a = bs gate wq (bs wq with a gate per
// token) and wp.  The group's sum S = sum yh g serves two gradients, which are taken when the
// group ends:  dgate = bs wq S,  dw_post += bs gate S.
//   GATE   0 none or shared by the rows of a group; 1 per token, of the rows' type; 2 per
//          token, fp32 beside 16-bit rows
//   SHIFT  rows do not all start on 16-byte boundaries: a worker takes rows n = class (mod
//          `classes`) only, which start equally far from one, so that its threads keep their
//          columns; the copied windows reach into the neighbouring rows, whose elements are
//          masked (rows narrower than a piece go to the general kernels: slm_norm_rows.h)
//   PRE    there is the second norm.  Without it nothing depends on r, which must not be formed: an
//          infinite y would make it infinite, and its zero factors would make NaN of that
// ----------------------------------------------------------------------------------------
constexpr int kRingThreads = 256;  // computing threads (more where one row takes more)
constexpr int kRingMost = 352;     // 11 warps and the copying one: still 168 registers a thread
constexpr int kRingWarps = kRingThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxStages = 6;
constexpr int kPartStride = kMaxCluster * kRingWarps + 8;  // the three sums in banks apart

struct RingCtl {
  uint64_t full[kMaxStages], empty[kMaxStages], sums[4];
  int abort;
  uint32_t issued;  // batches copied, at the end
  float2 factor[kMaxStages][kRingWarps];  // i_y, i_r of the batch's rows
  float part[4][3 * kPartStride];
};

template <class T, int TPR, int NV, int GATE>
struct RingCfg {
  static constexpr int kThreads = TPR > kRingThreads ? TPR : kRingThreads;
  static constexpr int kRows = kThreads / TPR;      // rows per batch
  static constexpr int kSeg = TPR * NV * 16;        // bytes of one array's row segment, at most
  static constexpr int kGateSeg = GATE == 0 ? 0 : GATE == 1 ? kSeg : 2 * kSeg;
  static constexpr int kStage = kRows * (4 * kSeg + kGateSeg);
  static constexpr int kCtl = (static_cast<int>(sizeof(RingCtl)) + 127) / 128 * 128;
  static constexpr int kScratch = kRows > 1 ? kThreads * NV * Piece<T>::kElems * 4 : 0;
  static constexpr int kFit = (232448 - 128 - kCtl - kScratch - kSeg) / kStage;
  static constexpr int kStages = kFit > kMaxStages ? kMaxStages : kFit;
  static constexpr size_t kSmem =
      128 + kCtl + kScratch + kSeg + static_cast<size_t>(kStages) * kStage;
  static_assert(kStages >= 3, "two batches in use, one under way");
};

// Three sums over the warp with six shuffles instead of fifteen: the first two steps also deal
// the sums out, so that lanes 8 k .. 8 k + 7 end with sum k (k = 0, 1, 2).
__device__ __forceinline__ float warp_sum3(float v0, float v1, float v2, int lane) {
  const bool b4 = lane & 16, b3 = lane & 8;
  float k0 = b4 ? v2 : v0, k1 = b4 ? 0.f : v1;
  k0 += __shfl_xor_sync(0xffffffffu, b4 ? v0 : v2, 16);
  k1 += __shfl_xor_sync(0xffffffffu, b4 ? v1 : 0.f, 16);
  float k = b3 ? k1 : k0;
  k += __shfl_xor_sync(0xffffffffu, b3 ? k0 : k1, 8);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) k += __shfl_xor_sync(0xffffffffu, k, o);
  return k;
}

template <class T, int TPR, int NV, int GATE, bool CL, bool SHIFT, bool PRE>
__global__ void __launch_bounds__((TPR > kRingThreads ? TPR : kRingThreads) + 32, 1)
    norm_bwd_ring(const NormBwd p, const DevCtl ctl, const int seg) {
  using P = Piece<T>;
  using C = RingCfg<T, TPR, NV, GATE>;
  constexpr int K = P::kPairs, kRows = C::kRows, S = C::kStages;
  constexpr int kThreads = C::kThreads, kWarps = kThreads / 32;
  static_assert(!CL || TPR == kRingThreads, "a cluster shares one row");
  extern __shared__ uint8_t ring_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(ring_raw) + 127) &
                                             ~static_cast<uintptr_t>(127));
  RingCtl* rc = reinterpret_cast<RingCtl*>(base);
  float4* scratch = reinterpret_cast<float4*>(base + C::kCtl);
  uint8_t* zeros = base + C::kCtl + C::kScratch;  // stands in for the arrays that are absent
  uint8_t* ring = zeros + C::kSeg;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cs = CL ? static_cast<int>(cluster_size()) : 1;
  const int rank = CL ? static_cast<int>(cluster_ctarank()) : 0;
  const int worker = static_cast<int>(blockIdx.x) / cs;
  const NormRows rows = norm_rows(p.plan, worker);
  const int step = SHIFT ? p.plan.classes : 1;  // from one of the worker's rows to the next
  const int shift =
      SHIFT ? static_cast<int>((p.shift0 + rows.begin(rows.g0) * p.d) % P::kElems) : 0;
  const int nvec = static_cast<int>((p.d + shift + P::kElems - 1) / P::kElems);
  const int piece0 = rank * seg;
  const int mine = max(0, min(seg, nvec - piece0));
  const bool has_y = p.y != nullptr, has_dr = p.d_residual != nullptr;
  // Always PRE; as a constant in that variant it changed ptxas's schedule (16384 x 4096 168 us, not 156).
  const bool pre = PRE && p.w_pre != nullptr;
  volatile int* abort = &rc->abort;

  // The status word is cleared here, without a launch for it: a wait can only run out long
  // after the first block has started.
  if (blockIdx.x == 0 && threadIdx.x == 0) *ctl.status = 0;
  for (int i = threadIdx.x; i < C::kSeg / 16; i += kThreads + 32)
    reinterpret_cast<uint4*>(zeros)[i] = make_uint4(0, 0, 0, 0);
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&rc->full[s], 1);
      // Test hook (fault == 1): the first stage (of a cluster's first block) wants a release that no
      // warp gives.  (Withheld in the loop, it cost 16384 x 4096 bf16 15 of its 156 us.)
      mbar_init(&rc->empty[s], kWarps + (ctl.fault == 1 && s == 0 && rank == 0 ? 1 : 0));
    }
    for (int s = 0; s < 4; ++s) mbar_init(&rc->sums[s], 1);
    rc->abort = 0;
    fence_barrier_init();
  }
  if (CL)
    cluster_sync();
  else
    __syncthreads();

  if (warp == kWarps) {
    // ------------------------------ copies ------------------------------
    const int arrays = has_y + has_dr + 2 * pre;
    uint32_t it = 0;
    bool ok = true;
    // The norms' factors of row n + lane step (lanes below kRows), fetched a batch ahead.
    auto factors = [&](int64_t n) {
      float2 f = make_float2(1.f, 0.f);
      const int64_t row = n + lane * step;
      if (lane < kRows && row < p.N) {
        if (p.w_post) f.x = __ldg(p.rstd_post + row);
        if (pre) f.y = __ldg(p.rstd_pre + row);
      }
      return f;
    };
    float2 f = factors(rows.begin(rows.g0));
    for (int64_t g = rows.g0; ok && g < rows.g1; ++g) {
      const int64_t n1 = rows.end(g);
      for (int64_t n = rows.begin(g); n < n1; n += kRows * step, ++it) {
        const int s = it % S;
        if (!wait_warp(&rc->empty[s], ((it / S) & 1u) ^ 1u, abort, ctl)) {
          ok = false;
          break;
        }
        const int valid =
            static_cast<int>(min(static_cast<int64_t>(kRows), (n1 - n + step - 1) / step));
        uint8_t* st = ring + s * C::kStage;
        auto source = [&](int arr, const void*& src, int64_t& ld) {
          src = arr == 0 ? (pre ? p.x : nullptr) : arr == 1 ? p.y : arr == 2 ? p.d_residual
                : arr == 3 ? (pre ? p.d_hidden : nullptr) : GATE ? p.gate : nullptr;
          ld = arr == 0 ? p.ldx : arr == 1 ? p.ldy : arr == 2 ? p.ld_dr : arr == 3 ? p.ld_dh : p.d;
        };
        // Pieces [lo, hi) of row `row` that this block copies whole.
        auto whole = [&](int64_t row, int& lo, int& hi) {
          const NormWindow w = SHIFT ? norm_window(row, p.N, p.d, shift, P::kElems, piece0, mine)
                                     : NormWindow{piece0, piece0 + mine};
          lo = w.lo;
          hi = w.hi;
        };
        uint32_t bytes = 0;
        for (int rw = 0; rw < valid; ++rw) {
          int lo, hi;
          whole(n + rw * step, lo, hi);
          bytes += (hi - lo) * 16;
          if (SHIFT && hi - lo < mine) {
            // Their elements, by plain loads (the first and the last row only).
            for (int q = lane; q < 5 * 2 * P::kElems; q += 32) {
              const int arr = q / (2 * P::kElems), e = q % P::kElems;
              const int piece = q / P::kElems % 2 ? hi : lo - 1;
              const void* src;
              int64_t ld;
              source(arr, src, ld);
              const int64_t c = static_cast<int64_t>(piece) * P::kElems - shift + e;
              if (!src || piece < piece0 || piece >= piece0 + mine || c < 0 || c >= p.d) continue;
              const int64_t at = (n + rw * step) * ld + c;
              uint8_t* dst = st + arr * kRows * C::kSeg;
              const int slot = (rw * mine + piece - piece0) * P::kElems + e;
              if (arr == 4 && GATE == 2)
                reinterpret_cast<float*>(dst)[slot] = static_cast<const float*>(src)[at];
              else
                reinterpret_cast<T*>(dst)[slot] = static_cast<const T*>(src)[at];
            }
          }
        }
        if (lane < kRows) rc->factor[s][lane] = f;
        __syncwarp();
        if (lane == 0)
          mbar_arrive_expect_tx(&rc->full[s], bytes * (arrays + (GATE == 0 ? 0 : GATE == 1 ? 1 : 2)));
        __syncwarp();
        f = factors(n + kRows * step < n1 ? n + kRows * step : rows.begin(g + 1));
        // Rows that lie end to end come as one copy (short rows would be bound by their number).
        for (int q = lane; q < valid * 5; q += 32) {
          const int arr = q % 5, rw = q / 5;
          const void* src;
          int64_t ld;
          source(arr, src, ld);
          const bool dense = !CL && !SHIFT && ld == p.d;
          int lo, hi;
          whole(n + rw * step, lo, hi);
          if (!src || (dense && rw > 0) || hi <= lo) continue;
          const int wide = arr == 4 && GATE == 2 ? 2 : 1;  // fp32 beside 16-bit rows
          const uint32_t size = static_cast<uint32_t>(hi - lo) * 16 * wide;
          const int64_t at = ((n + rw * step) * ld - shift) * static_cast<int64_t>(sizeof(T)) +
                             static_cast<int64_t>(lo) * 16;
          bulk_load(st + arr * kRows * C::kSeg + (rw * mine + lo - piece0) * 16 * wide,
                    static_cast<const uint8_t*>(src) + at * wide, dense ? size * valid : size,
                    &rc->full[s]);
        }
        __syncwarp();
      }
    }
    if (lane == 0) rc->issued = it;
  } else {
    // ------------------------------ arithmetic ------------------------------
    const int rw = threadIdx.x / TPR, t = threadIdx.x % TPR;  // row of the batch, first piece
    const float2 zero = pair(0.f);
    const float2 off = pair(p.weight_offset), bs = pair(p.block_scale), rs = pair(p.residual_scale);
    const float inv_d = 1.f / static_cast<float>(p.d);
    auto param = [&](const void* q, bool f32, int64_t row, int v, float2(&w)[K]) {
      if (SHIFT)
        Edge<T>::param(q, f32, row * p.d,
                       (piece0 + t + v * TPR) * P::kElems - shift, static_cast<int>(p.d), w);
      else
        P::param(q, f32, row * nvec + piece0 + t + v * TPR, w);
    };
    bool col[NV], edge[NV];
    int c0[NV];  // first column of piece v
    const int d = static_cast<int>(p.d);
    float2 acc_s[NV][K], acc_p[NV][K], a[NV][K], wp[NV][K];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      col[v] = t + v * TPR < mine;
      c0[v] = (piece0 + t + v * TPR) * P::kElems - shift;
      edge[v] = SHIFT && col[v] && Edge<T>::is(c0[v], d);
#pragma unroll
      for (int k = 0; k < K; ++k) acc_s[v][k] = acc_p[v][k] = a[v][k] = wp[v][k] = zero;
      if (pre && col[v]) {
        param(p.w_pre, p.w_f32, 0, v, wp[v]);
#pragma unroll
        for (int k = 0; k < K; ++k) wp[v][k] = add2(wp[v][k], off);
      }
    }
    // wq, and bs times the group's gate, of piece t + v TPR.
    auto load_wq = [&](int v, float2(&w)[K]) {
      if (p.w_post) param(p.w_post, p.w_f32, 0, v, w);
#pragma unroll
      for (int k = 0; k < K; ++k) w[k] = p.w_post ? add2(w[k], off) : pair(1.f);
    };
    auto load_gs = [&](int64_t g, int v, float2(&w)[K]) {
      const bool shared = GATE == 0 && p.gate;
      if (shared) param(p.gate, p.gate_f32, g, v, w);
#pragma unroll
      for (int k = 0; k < K; ++k) w[k] = shared ? mul2(w[k], bs) : bs;
    };
    auto consumers_sync = [] {
      asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
    };
    // The column sums of the batch's row lanes, added in a fixed order into lane 0's.
    auto join = [&](float2(&acc)[NV][K]) {
      if (kRows == 1) return;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int h = 0; h < K / 2; ++h)
          scratch[(v * (K / 2) + h) * kThreads + threadIdx.x] = make_float4(
              acc[v][2 * h].x, acc[v][2 * h].y, acc[v][2 * h + 1].x, acc[v][2 * h + 1].y);
      consumers_sync();
      if (rw == 0)
        for (int o = 1; o < kRows; ++o)
#pragma unroll
          for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int h = 0; h < K / 2; ++h) {
              const float4 f = scratch[(v * (K / 2) + h) * kThreads + threadIdx.x + o * TPR];
              acc[v][2 * h] = add2(acc[v][2 * h], make_float2(f.x, f.y));
              acc[v][2 * h + 1] = add2(acc[v][2 * h + 1], make_float2(f.z, f.w));
            }
      consumers_sync();
    };
    // Columns of piece v of a row of fp32 sums.
    auto store_f32 = [&](float* dst, int v, const float2(&w)[K], bool add) {
      if (SHIFT) {
#pragma unroll
        for (int e = 0; e < 2 * K; ++e)
          if (c0[v] + e >= 0 && c0[v] + e < d) {
            float* o = dst + c0[v] + e;
            const float f = e & 1 ? w[e / 2].y : w[e / 2].x;
            *o = add ? *o + f : f;
          }
        return;
      }
      float4* o = reinterpret_cast<float4*>(dst + c0[v]);
#pragma unroll
      for (int h = 0; h < K / 2; ++h) {
        float4 f = make_float4(w[2 * h].x, w[2 * h].y, w[2 * h + 1].x, w[2 * h + 1].y);
        if (add) {
          const float4 q = o[h];
          f = make_float4(f.x + q.x, f.y + q.y, f.z + q.z, f.w + q.w);
        }
        o[h] = f;
      }
    };
    // Piece v of row `row` of an output of the rows' type.
    auto store_row = [&](void* dst, int64_t row, int v, const float2(&w)[K]) {
      T* o = static_cast<T*>(dst) + row * p.d;
      if (edge[v])
        Edge<T>::store(o, c0[v], d, w);
      else
        __stcs(reinterpret_cast<uint4*>(o + c0[v]), P::pack(w));
    };
    auto store_gate_grad = [&](bool f32, int64_t row, int v, const float2(&w)[K]) {
      if (GATE == 1) {
        store_row(p.dgate, row, v, w);
      } else if (GATE == 2 && !edge[v]) {
        // Aligned although the row is not: pieces of 8 start on whole 32 bytes.
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.dgate) + row * p.d + c0[v]);
#pragma unroll
        for (int h = 0; h < K / 2; ++h)
          o[h] = make_float4(w[2 * h].x, w[2 * h].y, w[2 * h + 1].x, w[2 * h + 1].y);
      } else if (f32) {
        store_f32(static_cast<float*>(p.dgate) + row * p.d, v, w, false);
      } else if (SHIFT) {
        // A shared gate's row starts elsewhere than the worker's rows.
        Edge<T>::store(static_cast<T*>(p.dgate) + row * p.d, c0[v], d, w);
      } else {
        store_row(p.dgate, row, v, w);
      }
    };
    // Where this thread's pieces of x, y, dr and dh lie in stage 0, and how far on in the next.
    const uint8_t* arr[4];
    int stride[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const bool there = q == 1 ? has_y : q == 2 ? has_dr : pre;
      arr[q] = (there ? ring + q * kRows * C::kSeg + rw * mine * 16 : zeros) + t * 16;
      stride[q] = there ? C::kStage : 0;
    }
    // This thread's piece v of a stage: y, dr, the gate, i_y a (gate), r and dh.
    auto load = [&](int s, int v, float2 iy, float2(&y)[K], float2(&dr)[K], float2(&gate)[K],
                    float2(&ay)[K], float2(&r)[K], float2(&dh)[K]) {
      P::unpack(*reinterpret_cast<const uint4*>(arr[0] + s * stride[0] + v * TPR * 16), r);
      P::unpack(*reinterpret_cast<const uint4*>(arr[1] + s * stride[1] + v * TPR * 16), y);
      P::unpack(*reinterpret_cast<const uint4*>(arr[2] + s * stride[2] + v * TPR * 16), dr);
      P::unpack(*reinterpret_cast<const uint4*>(arr[3] + s * stride[3] + v * TPR * 16), dh);
      if (GATE) {
        const uint8_t* sg = ring + s * C::kStage + 4 * kRows * C::kSeg +
                            rw * mine * (GATE == 2 ? 32 : 16);
        const int i = t + v * TPR;
        if (GATE == 1) {
          P::unpack(reinterpret_cast<const uint4*>(sg)[i], gate);
        } else {
#pragma unroll
          for (int h = 0; h < K / 2; ++h) {
            const float4 f = reinterpret_cast<const float4*>(sg)[i * (K / 2) + h];
            gate[2 * h] = make_float2(f.x, f.y);
            gate[2 * h + 1] = make_float2(f.z, f.w);
          }
        }
      }
      if (edge[v]) {
        Edge<T>::mask(c0[v], d, r);
        Edge<T>::mask(c0[v], d, y);
        Edge<T>::mask(c0[v], d, dr);
        Edge<T>::mask(c0[v], d, dh);
        if (GATE) Edge<T>::mask(c0[v], d, gate);
      }
#pragma unroll
      for (int k = 0; k < K; ++k) {
        ay[k] = mul2(GATE ? mul2(a[v][k], gate[k]) : a[v][k], iy);
        r[k] = PRE ? fma2(rs, r[k], mul2(ay[k], y[k])) : zero;
      }
    };
    // Sweep 1: sum u r, sum a yh (dr + i_r u), sum a yh r over the rows of the batch, handed on
    // to the warps that share a row (the factor i_r of rh comes in afterwards).
    auto sweep1 = [&](uint32_t it, int s, bool live) {
      wait_warp(&rc->full[s], (it / S) & 1u, abort, ctl);
      float2 s0 = zero, s1 = zero, s2 = zero;
      if (live) {
        const float2 f = rc->factor[s][rw], iy2 = pair(f.x), ir2 = pair(f.y);
#pragma unroll
        for (int v = 0; v < NV; ++v)
          if (col[v]) {
            float2 y[K], dr[K], gate[K], ay[K], r[K], dh[K];
            load(s, v, iy2, y, dr, gate, ay, r, dh);
#pragma unroll
            for (int k = 0; k < K; ++k) {
              const float2 u = mul2(dh[k], wp[v][k]), ayy = mul2(ay[k], y[k]);
              s0 = fma2(u, r[k], s0);
              s1 = fma2(ayy, fma2(ir2, u, dr[k]), s1);
              s2 = fma2(ayy, r[k], s2);
            }
          }
      }
      const float v = warp_sum3(s0.x + s0.y, s1.x + s1.y, s2.x + s2.y, lane);
      if (TPR == 32) return v;
      const int slot = (lane >> 3) * kPartStride + rank * kRingWarps + warp;
      if (CL) {
        // Lane c of each eight serves block c; the stores count themselves on its barrier, so
        // that nothing waits for this thread's earlier stores to global memory.  Four buffers
        // and barriers: a block that sends batch it has received every warp's sums of batch
        // it - 2, which each sent after it had received and read those of batch it - 4.  After a
        // wait that ran out that order is lost, and the block takes no more part: the others' waits
        // run out in turn, on barriers that have counted no batch too many.
        if (!*abort) {
          if (threadIdx.x == 0)
            mbar_arrive_expect_tx(&rc->sums[it & 3], static_cast<uint32_t>(cs * kRingWarps * 12));
          if (lane < 24 && (lane & 7) < cs)
            st_async_cluster(mapa_shared(smem_u32(&rc->part[it & 3][slot]), lane & 7), v,
                             mapa_shared(smem_u32(&rc->sums[it & 3]), lane & 7));
        }
        __syncwarp();
      } else if (lane < 24 && (lane & 7) == 0) {
        rc->part[it & 3][slot] = v;
      }
      return v;
    };

    uint32_t it = 0;
    int s = 0;  // it % S
    for (int64_t g = rows.g0; g < rows.g1; ++g) {
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (col[v] && has_y) {
          float2 w[K], q[K];
          load_wq(v, w);
          load_gs(g, v, q);
#pragma unroll
          for (int k = 0; k < K; ++k) a[v][k] = mul2(w[k], q[k]);
        }
      const int64_t n1 = rows.end(g);
      int64_t n = rows.begin(g) + rw * step;
      const int batches = static_cast<int>(
          max(static_cast<int64_t>(0), (n1 - rows.begin(g) + kRows * step - 1) / (kRows * step)));
      float mysum = batches > 0 ? sweep1(it, s, n < n1) : 0.f;
      for (int b = 0; b < batches; ++b, n += kRows * step, ++it) {
        if (!CL && TPR > 32) consumers_sync();  // the sums of this batch are there
        float sum = mysum;
        const int s_next = s + 1 == S ? 0 : s + 1;
        if (b + 1 < batches) mysum = sweep1(it + 1, s_next, n + kRows * step < n1);
        if (CL) wait_warp(&rc->sums[it & 3], (it >> 2) & 1u, abort, ctl);
        if (TPR > 32) {
          const float* part = rc->part[it & 3] + (lane >> 3) * kPartStride;
          const int w0 = CL ? 0 : rw * (TPR / 32), nw = CL ? cs * kRingWarps : TPR / 32;
          sum = 0.f;
          if (lane < 24)
            for (int w = lane & 7; w < nw; w += 8) sum += part[w0 + w];
#pragma unroll
          for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        }
        const float2 f = rc->factor[s][rw];
        const float iy = f.x, ir = f.y;
        const float c1 = __shfl_sync(0xffffffffu, sum, 0) * ir * inv_d;
        const float s1 = __shfl_sync(0xffffffffu, sum, 8), s2 = __shfl_sync(0xffffffffu, sum, 16);
        const float c2 = p.w_post ? (s1 - ir * ir * c1 * s2) * inv_d : 0.f;
        if (n < n1) {
          const float2 kg = pair(-ir * ir * c1), ky = pair(-iy * iy * c2), py = pair(iy), pr = pair(ir);
#pragma unroll
          for (int v = 0; v < NV; ++v)
            if (col[v]) {
              float2 y[K], g2[K], gate[K], ay[K], r[K], dh[K], o[K];
              load(s, v, py, y, g2, gate, ay, r, dh);
#pragma unroll
              for (int k = 0; k < K; ++k) {
                dh[k] = mul2(dh[k], pr);
                g2[k] = fma2(kg, r[k], fma2(dh[k], wp[v][k], g2[k]));
                o[k] = mul2(rs, g2[k]);
                acc_p[v][k] = fma2(dh[k], r[k], acc_p[v][k]);
              }
              store_row(p.dx, n, v, o);
              if (has_y) {
#pragma unroll
                for (int k = 0; k < K; ++k) {
                  o[k] = mul2(ay[k], g2[k]);
                  if (p.w_post) o[k] = fma2(ky, y[k], o[k]);
                  g2[k] = mul2(py, g2[k]);
                  if (GATE) {
                    const float2 yg = mul2(y[k], g2[k]);
                    acc_s[v][k] = fma2(gate[k], yg, acc_s[v][k]);
                    g2[k] = mul2(a[v][k], yg);
                  } else {
                    acc_s[v][k] = fma2(y[k], g2[k], acc_s[v][k]);
                  }
                }
                store_row(p.dy, n, v, o);
                if (GATE) store_gate_grad(GATE == 2 || std::is_same_v<T, float>, n, v, g2);
              }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&rc->empty[s]);
        s = s_next;
      }
      if (GATE == 0 && (p.w_post || p.gate)) {
        // The group's end: its S into the gate's and the post weight's gradients.
        join(acc_s);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          if (rw == 0 && col[v]) {
            float2 w[K], q[K];
            load_wq(v, w);
            load_gs(g, v, q);
#pragma unroll
            for (int k = 0; k < K; ++k) {
              q[k] = mul2(q[k], acc_s[v][k]);
              w[k] = mul2(mul2(w[k], bs), acc_s[v][k]);
            }
            if (p.w_post)
              store_f32(p.part_post + static_cast<int64_t>(worker) * p.d, v, q, g > rows.g0);
            if (p.gate) {
              if (p.plan.parts() > 1)
                store_f32(p.part_gate + static_cast<int64_t>(worker) * p.d, v, w, false);
              else
                store_gate_grad(p.gate_f32, g, v, w);
            }
          }
#pragma unroll
          for (int k = 0; k < K; ++k) acc_s[v][k] = zero;
        }
      }
    }
    if (GATE && p.w_post) {
      join(acc_s);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
#pragma unroll
        for (int k = 0; k < K; ++k) acc_s[v][k] = mul2(bs, acc_s[v][k]);
        if (rw == 0 && col[v])
          store_f32(p.part_post + static_cast<int64_t>(worker) * p.d, v, acc_s[v], false);
      }
    }
    if (pre) {
      join(acc_p);
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (rw == 0 && col[v])
          store_f32(p.part_pre + static_cast<int64_t>(worker) * p.d, v, acc_p[v], false);
    }
  }
  __syncthreads();
  if (*abort && warp == 0) {
    // After a wait that ran out: copies in flight land (boundedly) before the block leaves.
    const uint32_t last = rc->issued;
    for (uint32_t q = last > static_cast<uint32_t>(S) ? last - S : 0u; q < last; ++q)
      wait_warp(&rc->full[q % S], (q / S) & 1u, abort, ctl, false);
  }
  // By the copying warp: in warp 0's branch above it changed ptxas's schedule of the loop (16384 x 4096
  // bf16 167 us, not 155).
  if (*abort && threadIdx.x == kThreads) record_ran_out();
  // No block leaves while another of its cluster may still write its sums into it: one whose waits
  // all ended has received every sum; to one that gave up, those sent before the barrier may still
  // be on their way, which takes microseconds.
  if (CL) {
    __syncwarp();
    cluster_sync();
    if (*abort)
      for (int q = 0; q < 100; ++q) __nanosleep(1000);
  }
}

// How row arrays lie to the 16-byte pieces: elements from an aligned address to the first row,
// and whether every row of every array starts equally far from one as its fellows.
struct RowFit {
  int elems;        // elements per piece
  int64_t N, d;
  int64_t shift0 = -1;
  bool ok = true;
  void add(const void* p, int64_t ld) {
    if (!p) return;
    const int64_t at = static_cast<int64_t>(reinterpret_cast<uintptr_t>(p) & 15) * elems / 16;
    if (shift0 < 0) shift0 = at;
    ok = ok && at == shift0 && (N == 1 || ld % elems == d % elems);
  }
  bool shifted() const { return shift0 != 0 || d % elems != 0; }
};
// Row classes: after this many rows the distance to the 16-byte boundary comes round again.
inline int row_classes(int64_t N, int64_t d, int elems, bool shift) {
  int classes = 1;
  while (shift && N > 1 && classes * d % elems != 0) classes *= 2;
  return classes;
}
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <class T, int NV, bool WARP>
cudaError_t fwd_vec(const NormFwd& p, int threads, bool shift, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(WARP ? (p.N + 3) / 4 : p.N);
  if (shift)
    norm_fwd_vec<T, NV, WARP, true><<<grid, threads, 0, s>>>(p);
  else
    norm_fwd_vec<T, NV, WARP, false><<<grid, threads, 0, s>>>(p);
  return cudaGetLastError();
}

template <class T>
cudaError_t fwd_t(NormFwd p, cudaStream_t s) {
  constexpr int E = Piece<T>::kElems;
  RowFit fit{E, p.N, p.d};
  fit.add(p.x, p.ldx);
  fit.add(p.y, p.ldy);
  fit.add(p.residual, p.d);
  fit.add(p.hidden, p.d);
  const bool shift = fit.shifted() || !aligned16(p.w_post) || !aligned16(p.w_pre) || !aligned16(p.gate);
  const int64_t nvec = shift ? (p.d + 2 * E - 2) / E : p.d / E;  // the most that a row has
  if (!fit.ok || nvec > 4096) {
    const int64_t grid = std::min<int64_t>(p.N, int64_t(1) << 20);
    norm_fwd_any<T><<<static_cast<unsigned>(grid), kAnyThreads, 0, s>>>(p);
    return cudaGetLastError();
  }
  p.shift0 = static_cast<int>(fit.shift0);
  // Few rows: as many threads per row as there are pieces, for latency (130 x 2048 bf16 2.7 us
  // against 3.3 with two pieces a thread; 296 x 4096 4.0 and 4.5, but 600 x 4096 7.0 and 6.0).
  // Many: two pieces per thread, whose loads are in flight together, or four (16384 rows of 16 bits:
  // width 4608 98 us with two and 100 with four, 5000 114 and 110, 8192 174 and 167; unaligned 4096 x
  // 5001 64 and 52; fp32 rows of 4096 160 and 165).  Short rows: a warp each (65536 x 256 bf16 26 us, by
  // blocks 37; 32768 x 512 21 and 24).
  const bool few = p.N <= 2 * sm_count();
  auto warps = [&](int64_t per) { return static_cast<int>((nvec + 32 * per - 1) / (32 * per) * 32); };
  if (nvec <= 32) return fwd_vec<T, 1, true>(p, 128, shift, s);
  if (nvec <= 64 && !few) return fwd_vec<T, 2, true>(p, 128, shift, s);
  if (nvec <= 1024 && few) return fwd_vec<T, 1, false>(p, warps(1), shift, s);
  if (nvec <= (E == 8 ? 608 : 1024)) return fwd_vec<T, 2, false>(p, warps(2), shift, s);
  return fwd_vec<T, 4, false>(p, warps(4), shift, s);
}

template <class T>
cudaError_t bwd_sums(const NormBwd& p, cudaStream_t s) {
  const bool gates = p.plan.shared_gate && p.plan.parts() > 1;
  if (!p.w_post && !p.w_pre && !gates) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>((p.d + 31) / 32),
                  static_cast<unsigned>(2 + (gates ? p.plan.groups : 0)));
  norm_bwd_reduce<T><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

template <class T, int TPR, int NV, int GATE, bool CL, bool SHIFT, bool PRE>
cudaError_t bwd_ring_t(NormBwd p, const DevCtl& c, int cs, cudaStream_t s) {
  using C = RingCfg<T, TPR, NV, GATE>;
  auto kern = norm_bwd_ring<T, TPR, NV, GATE, CL, SHIFT, PRE>;
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
  cfg.blockDim = dim3(C::kThreads + 32, 1, 1);
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
  constexpr int E = Piece<T>::kElems;
  const int classes = row_classes(p.N, p.d, E, SHIFT);
  p.plan = norm_plan(p.N, p.rows_per_gate, p.gate != nullptr, std::min(most, kNormBlocks), C::kRows,
                     classes);
  const int nvec = static_cast<int>(SHIFT ? (p.d + 2 * E - 2) / E : p.d / E);
  cfg.gridDim = dim3(static_cast<unsigned>(p.plan.blocks * cs), 1, 1);
  if ((e = cudaLaunchKernelEx(&cfg, kern, p, c, (nvec + cs - 1) / cs)) != cudaSuccess) return e;
  return bwd_sums<T>(p, s);
}

template <class T, int TPR, int NV, int GATE, bool CL, bool SHIFT>
cudaError_t bwd_ring(const NormBwd& p, const DevCtl& c, int cs, cudaStream_t s) {
  return p.w_pre ? bwd_ring_t<T, TPR, NV, GATE, CL, SHIFT, true>(p, c, cs, s)
                 : bwd_ring_t<T, TPR, NV, GATE, CL, SHIFT, false>(p, c, cs, s);
}

// Threads per row: as few as keep two pieces each, so that a batch has many rows and few threads
// share a sum (256 threads for every row: 65536 x 256 bf16 379 us instead of 70, 16384 x 2048 114
// instead of 85).  One block for a row as long as its registers and ring do (4096 x 5120 62 us, in
// clusters of two 94; 16384 x 4096 155 and 290), then as few blocks as that leaves (8192 x 16384 396
// us in clusters of four, 689 of eight).
template <class T, int GATE, bool SHIFT>
cudaError_t bwd_vec(const NormBwd& p, int64_t nvec, const DevCtl& c, cudaStream_t s) {
  if (nvec <= 32) return bwd_ring<T, 32, 1, GATE, false, SHIFT>(p, c, 1, s);
  if (nvec <= 64) return bwd_ring<T, 32, 2, GATE, false, SHIFT>(p, c, 1, s);
  if (nvec <= 128) return bwd_ring<T, 64, 2, GATE, false, SHIFT>(p, c, 1, s);
  if (nvec <= 256) return bwd_ring<T, 128, 2, GATE, false, SHIFT>(p, c, 1, s);
  if (nvec <= 512) return bwd_ring<T, 256, 2, GATE, false, SHIFT>(p, c, 1, s);
  if (nvec <= 2 * kRingMost) return bwd_ring<T, kRingMost, 2, GATE, false, SHIFT>(p, c, 1, s);
  return bwd_ring<T, 256, 2, GATE, true, SHIFT>(p, c, nvec <= 1024 ? 2 : nvec <= 2048 ? 4 : 8, s);
}

template <class T>
cudaError_t bwd_t(NormBwd p, const DevCtl& c, cudaStream_t s) {
  constexpr int E = Piece<T>::kElems;
  RowFit fit{E, p.N, p.d};
  fit.add(p.x, p.ldx);
  fit.add(p.y, p.ldy);
  fit.add(p.d_residual, p.ld_dr);
  fit.add(p.d_hidden, p.ld_dh);
  fit.add(p.dx, p.d);
  fit.add(p.dy, p.d);
  const bool token = p.gate && !p.plan.shared_gate;
  const bool wide = token && p.gate_f32 && !std::is_same_v<T, float>;  // fp32 beside 16 bits
  if (token && !wide) {
    fit.add(p.gate, p.d);
    fit.add(p.dgate, p.d);
  }
  const bool shift = fit.shifted() || !aligned16(p.w_post) || !aligned16(p.w_pre) ||
                     !aligned16(p.gate) || !aligned16(p.dgate);
  // Pieces of 8 fp32 gates start on 16-byte boundaries where those of the rows do.
  if (wide) fit.ok = fit.ok && fit.shift0 == 0 && aligned16(p.gate) && aligned16(p.dgate);
  // A shared gate with more groups than can be split by row class (each class of each group has a
  // worker of its own) is left to the general path.
  const int classes = row_classes(p.N, p.d, E, shift);
  if (classes > 1 && p.plan.shared_gate) fit.ok = fit.ok && p.plan.groups * classes <= kNormBlocks;
  const int64_t nvec = shift ? (p.d + 2 * E - 2) / E : p.d / E;  // the most that a row has
  if (fit.ok && norm_ring_takes(p.d, E) && nvec <= 2 * kRingThreads * kMaxCluster) {
    p.shift0 = static_cast<int>(fit.shift0);
    if (!token)
      return shift ? bwd_vec<T, 0, true>(p, nvec, c, s) : bwd_vec<T, 0, false>(p, nvec, c, s);
    if constexpr (!std::is_same_v<T, float>)
      if (wide)
        return shift ? bwd_vec<T, 2, true>(p, nvec, c, s) : bwd_vec<T, 2, false>(p, nvec, c, s);
    return shift ? bwd_vec<T, 1, true>(p, nvec, c, s) : bwd_vec<T, 1, false>(p, nvec, c, s);
  }
  const int64_t grid = std::min<int64_t>(p.N, int64_t(1) << 20);
  norm_bwd_rows_any<T><<<static_cast<unsigned>(grid), kAnyThreads, 0, s>>>(p, c.status);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !(p.w_post || p.w_pre || p.plan.shared_gate)) return e;
  const dim3 gc(static_cast<unsigned>((p.d + 127) / 128), static_cast<unsigned>(p.plan.blocks));
  norm_bwd_cols_any<T><<<gc, 128, 0, s>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return bwd_sums<T>(p, s);
}

}  // namespace
}  // namespace slm
