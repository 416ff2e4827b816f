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

#include "slm_internal.h"

namespace slm {
namespace {

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

template <class T>
cudaError_t fwd_t(const NormFwd& p, cudaStream_t s) {
  const int64_t grid = std::min<int64_t>(p.N, int64_t(1) << 20);
  norm_fwd_any<T><<<static_cast<unsigned>(grid), kAnyThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <class T>
cudaError_t bwd_t(const NormBwd& p, cudaStream_t s) {
  const int64_t grid = std::min<int64_t>(p.N, int64_t(1) << 20);
  norm_bwd_rows_any<T><<<static_cast<unsigned>(grid), kAnyThreads, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !(p.w_post || p.w_pre || p.plan.shared_gate)) return e;
  const dim3 gc(static_cast<unsigned>((p.d + 127) / 128), static_cast<unsigned>(p.plan.blocks));
  norm_bwd_cols_any<T><<<gc, 128, 0, s>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int64_t sums = 2 + (p.plan.shared_gate && p.plan.slices > 1 ? p.plan.groups : 0);
  const dim3 gr(static_cast<unsigned>((p.d + 31) / 32), static_cast<unsigned>(sums));
  norm_bwd_reduce<T><<<gr, 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

NormPlan norm_plan(int64_t N, int64_t rows_per_gate, bool has_gate) {
  NormPlan q{};
  q.shared_gate = has_gate && rows_per_gate > 1;
  q.rows = q.shared_gate ? rows_per_gate : N;
  q.groups = q.shared_gate ? N / rows_per_gate : 1;
  // Blocks own either one slice of one group or several whole groups.
  const int64_t want = std::min<int64_t>(N, kNormBlocks);
  q.slices = static_cast<int>(
      std::max<int64_t>(1, std::min<int64_t>(q.rows, want / std::max<int64_t>(1, q.groups))));
  q.blocks = static_cast<int>(q.slices > 1 ? q.groups * q.slices
                                           : std::min<int64_t>(q.groups, kNormBlocks));
  return q;
}

cudaError_t launch_norm_fwd(int dtype, const NormFwd& p, cudaStream_t s) {
  if (dtype == 0) return fwd_t<__nv_bfloat16>(p, s);
  if (dtype == 1) return fwd_t<__half>(p, s);
  return fwd_t<float>(p, s);
}

cudaError_t launch_norm_bwd(int dtype, const NormBwd& p, cudaStream_t s) {
  if (dtype == 0) return bwd_t<__nv_bfloat16>(p, s);
  if (dtype == 1) return bwd_t<__half>(p, s);
  return bwd_t<float>(p, s);
}

}  // namespace slm
