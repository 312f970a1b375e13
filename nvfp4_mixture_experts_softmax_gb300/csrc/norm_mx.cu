// Residual addition + RMSNorm with MXFP8 output, and its backward pass.
//
// Forward, per row:  h = bf16(x + residual),  r = 1 / sqrt(mean(h^2) + eps),  y = (h * r) * gamma,
// then per 32 elements the E8M0 scale and E4M3 codes of y (the W4A8 layer's activation format,
// quantised from the FP32 y: no BF16 rounding in between) and, if asked for, bf16(y).  h is
// rounded to BF16 before the norm because that is what the residual stream keeps: the norm of
// the stored h is what the backward pass and any later reader recompute.
//
// Backward, with a = gamma * dy:  dx = dh + r * a - h * r^3 * mean(a * h)  (the gradient of x and
// of the residual alike),  dgamma_c = sum over rows of dy * (h * r).  The quantisation is passed
// straight through: dy is the gradient of y.
//
// Both are bound by HBM: every element is read and written once (7.03 bytes an element forward, 9.03
// with y; 6 or 8 backward).  Measured (device time of a call): forward 16384 x 4096 74.6 us = 93% of
// the copy rate, 4096 x 7168 with y 46.9 us (84%), 20000 x 256 9.3 us (74%), 1 x 2048 1.9 us;
// backward 8192 x 2048 with dh 27.8 us (71%), 1999 x 7168 22.2 us (57%), 3906 x 16384 118 us
// (64%).  One block per row, reduced before the next row's loads, took 108, 53.9, 20.6, 2.0 us and
// 50, 33, 134 us.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "ops.h"
#include "rows.cuh"

namespace nvfp4moe {

namespace {

constexpr int kMaxCols = 16384;

// How a row is laid over threads: W warps with J vectors of 8 columns a lane (vector c of lane t:
// c = j * 32 W + t, so four neighbouring lanes share a 32-element block); a block holds G such row
// groups, each of which takes every gridDim * G-th row.
struct RowGrid {
  int J, W, G, blocks;
};

// h = bf16(x + residual) of one vector, and its squares added to sq.
__device__ __forceinline__ uint4 add_vec(uint4 x, uint4 r, bool has_res, float& sq) {
  float f[8];
  unpack8(x, f);
  if (has_res) {
    float g[8];
    unpack8(r, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] += g[i];
    x = pack8(f);
    unpack8(x, f);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) sq = fmaf(f[i], f[i], sq);
  return x;
}

// The next row's x and residual are loaded before the current row is reduced.  64 registers a
// thread: 32 warps an SM with 2 KB each in flight.
template <int J>
__global__ void __launch_bounds__(512, J <= 2 ? 2 : 1) add_rmsnorm_mx_kernel(
    const uint4* x, const uint4* residual, const uint4* __restrict__ gamma, float eps,
    int64_t rows, int cols, int W, int G, uint4* h, uint2* codes, uint8_t* sf, uint4* y,
    float* rrms) {
  __shared__ float red[2 * 16 * 32];
  const int warp = threadIdx.x >> 5, group = warp / W, wrow = warp - group * W;
  const int t = wrow * 32 + (threadIdx.x & 31), span = W * 32;   // thread of the row, vectors apart
  const int nvec = cols / 8;
  const float inv_cols = 1.0f / (float)cols;
  griddep_wait();
  griddep_launch();
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  int64_t row = (int64_t)blockIdx.x * G + group;
  const int64_t step = (int64_t)gridDim.x * G;
  uint4 nx[J], nr[J];
  auto load = [&](int64_t rw) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = j * span + t;
      const bool in = rw < rows && c < nvec;
      nx[j] = in ? x[rw * nvec + c] : zero;
      nr[j] = in && residual ? residual[rw * nvec + c] : zero;
    }
  };
  load(row);
  for (int parity = 0; row < rows; row += step, parity ^= 1) {
    const int64_t base = row * nvec;
    uint4 hv[J];
    float sq = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j) hv[j] = add_vec(nx[j], nr[j], residual != nullptr, sq);
    load(row + step);   // (rows are written by their own group only, after this group read them)
    if (residual) {
#pragma unroll
      for (int j = 0; j < J; ++j)
        if (j * span + t < nvec) h[base + j * span + t] = hv[j];
    }
    sq = row_sum(sq, red, W, wrow, group, G, parity);
    const float r = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(sq * inv_cols, eps)));
    if (rrms && t == 0) rrms[row] = r;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = j * span + t;
      const bool in = c < nvec;
      float v[8], g[8];
      unpack8(hv[j], v);
      unpack8(in ? __ldg(gamma + c) : zero, g);
      uint32_t top = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = __fmul_rn(__fmul_rn(v[i], r), g[i]);
        top = max(top, __float_as_uint(fabsf(v[i])));   // NaN orders above infinity
      }
      if (y && in) y[base + c] = pack8(v);
      if (!codes) continue;
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      if (!in) continue;
      uint32_t sb = mx_scale_byte(__uint_as_float(top), 8);
      uint32_t lo, hi;
      if (top >= 0x7F800000u) {   // a block that holds an infinity or NaN is NaN as a whole
        sb = 255u;
        lo = hi = 0x7F7F7F7Fu;
      } else {
        const float inv = e8m0_to_f32(254u - sb);   // 2^(127 - sb)
        lo = f32_to_e4m3x2(v[0] * inv, v[1] * inv) | f32_to_e4m3x2(v[2] * inv, v[3] * inv) << 16;
        hi = f32_to_e4m3x2(v[4] * inv, v[5] * inv) | f32_to_e4m3x2(v[6] * inv, v[7] * inv) << 16;
      }
      codes[base + c] = make_uint2(lo, hi);
      if ((c & 3) == 0) sf[(base + c) >> 2] = (uint8_t)sb;
    }
  }
}

// A thread owns the same J vectors of 8 columns in all rows of its group and keeps their share of
// dgamma in registers; the groups of a block are joined in order at the end, the blocks by
// dgamma_kernel.  Up to two vectors the next row's dy, h and dh are loaded before the current row is
// reduced (J = 1: 24 warps an SM, J = 2: 16); four vectors (above 8192 columns) fill the registers.
template <int J>
__global__ void __launch_bounds__(J == 1 ? 256 : 512, J == 1 ? 3 : 1) add_rmsnorm_backward_kernel(
    const uint4* dy, const uint4* dh, const uint4* __restrict__ h,
    const float* __restrict__ rrms, const uint4* __restrict__ gamma, int64_t rows, int cols, int W,
    int G, uint4* dx, float4* __restrict__ partial) {
  constexpr bool kAhead = J <= 2;
  extern __shared__ float4 s_dg[];   // [cols / 4] if G > 1
  __shared__ float red[2 * 16 * 32];
  const int warp = threadIdx.x >> 5, group = warp / W, wrow = warp - group * W;
  const int t = wrow * 32 + (threadIdx.x & 31), span = W * 32;
  const int nvec = cols / 8;
  const float inv_cols = __fdiv_rn(1.0f, (float)cols);
  griddep_wait();
  griddep_launch();
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  float dg[J][8];
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) dg[j][i] = 0.0f;
  int64_t row = (int64_t)blockIdx.x * G + group;
  const int64_t step = (int64_t)gridDim.x * G;
  uint4 nd[J], nh[J], ne[J], ng[kAhead ? J : 1];
  float nr = 0.0f;
  auto gamma_of = [&](int j) {
    return j * span + t < nvec ? __ldg(gamma + j * span + t) : zero;
  };
  if constexpr (kAhead) {
#pragma unroll
    for (int j = 0; j < J; ++j) ng[j] = gamma_of(j);
  }
  auto load_dh = [&](int64_t rw) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = j * span + t;
      ne[j] = rw < rows && c < nvec && dh ? dh[rw * nvec + c] : zero;
    }
  };
  auto load = [&](int64_t rw) {
    nr = rw < rows ? __ldg(rrms + rw) : 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = j * span + t;
      const bool in = rw < rows && c < nvec;
      nd[j] = in ? dy[rw * nvec + c] : zero;
      nh[j] = in ? __ldg(h + rw * nvec + c) : zero;
    }
    if (kAhead) load_dh(rw);
  };
  if constexpr (kAhead) load(row);
  for (int parity = 0; row < rows; row += step, parity ^= 1) {
    if constexpr (!kAhead) load(row);
    const float r = nr;
    uint4 qd[J], qh[J], qe[J];
    float a[kAhead ? J : 1][8];   // gamma dy, or computed again from qd
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      qd[j] = nd[j];
      qh[j] = nh[j];
      if (kAhead) qe[j] = ne[j];
      float d[8], hv[8], g[8];
      unpack8(qd[j], d);
      unpack8(qh[j], hv);
      unpack8(kAhead ? ng[kAhead ? j : 0] : gamma_of(j), g);
      const bool in = j * span + t < nvec;   // (an infinite 1/rms must not meet the zeros outside)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float ai = d[i] * g[i];
        if constexpr (kAhead) a[j][i] = ai;
        s = fmaf(ai, hv[i], s);
        if (in) dg[j][i] = fmaf(d[i], hv[i] * r, dg[j][i]);
      }
    }
    if constexpr (kAhead) {
      load(row + step);
    } else {   // dh is not part of the row's sum
      load_dh(row);
#pragma unroll
      for (int j = 0; j < J; ++j) qe[j] = ne[j];
    }
    s = row_sum(s, red, W, wrow, group, G, parity);
    const float m = r * r * (s * inv_cols);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = j * span + t;
      if (c >= nvec) continue;
      float hv[8], e[8], o[8];
      unpack8(qh[j], hv);
      unpack8(qe[j], e);
      if constexpr (kAhead) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = r * fmaf(-hv[i], m, a[j][i]);
      } else {
        float d[8], g[8];
        unpack8(qd[j], d);
        unpack8(gamma_of(j), g);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = r * fmaf(-hv[i], m, d[i] * g[i]);
      }
      if (dh) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] += e[i];
      }
      dx[row * nvec + c] = pack8(o);
    }
  }
  for (int k = 1; k < G; ++k) {   // the other groups' sums to the first's, in order
    __syncthreads();
    if (group == k) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int c = j * span + t;
        if (c >= nvec) continue;
        s_dg[2 * c] = make_float4(dg[j][0], dg[j][1], dg[j][2], dg[j][3]);
        s_dg[2 * c + 1] = make_float4(dg[j][4], dg[j][5], dg[j][6], dg[j][7]);
      }
    }
    __syncthreads();
    if (group == 0) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int c = j * span + t;
        if (c >= nvec) continue;
        const float4 u = s_dg[2 * c], v = s_dg[2 * c + 1];
        dg[j][0] += u.x; dg[j][1] += u.y; dg[j][2] += u.z; dg[j][3] += u.w;
        dg[j][4] += v.x; dg[j][5] += v.y; dg[j][6] += v.z; dg[j][7] += v.w;
      }
    }
  }
  if (group != 0) return;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c = j * span + t;
    if (c >= nvec) continue;
    float4* p = partial + (int64_t)blockIdx.x * (cols / 4) + 2 * c;
    p[0] = make_float4(dg[j][0], dg[j][1], dg[j][2], dg[j][3]);
    p[1] = make_float4(dg[j][4], dg[j][5], dg[j][6], dg[j][7]);
  }
}

// dgamma = sum of the blocks' partial rows: warp w takes rows w, w + 32, ..., then the warps in order.
__global__ void __launch_bounds__(1024) dgamma_kernel(const float* __restrict__ partial, int nb,
                                                      int cols, float* __restrict__ dgamma) {
  __shared__ float red[32][33];
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.0f;
#pragma unroll 10
  for (int b = warp; b < nb; b += 32) s += __ldcg(partial + (int64_t)b * cols + c);
  red[warp][lane] = s;
  __syncthreads();
  // lane w of warp c adds warp w's share of column c
  s = red[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) dgamma[blockIdx.x * 32 + warp] = s;
}

// Few rows: as many warps a row as its vectors fill, for the latency.  Many rows: two vectors a
// lane, at least eight warps a block, 32 warps an SM.
RowGrid forward_grid(int64_t rows, int nvec) {
  RowGrid g;
  const bool few = rows <= 2 * (int64_t)num_sms();
  g.J = nvec > 1024 ? 4 : nvec > 512 || (!few && nvec > 32) ? 2 : 1;
  g.W = (nvec + 32 * g.J - 1) / (32 * g.J);
  g.G = few ? 1 : std::max(1, 8 / g.W);
  const int64_t need = (rows + g.G - 1) / g.G, most = (int64_t)num_sms() * std::max(1, (g.J <= 2 ? 32 : 16) / (g.W * g.G));
  g.blocks = (int)std::min(need, most);
  return g;
}

RowGrid backward_grid(int64_t rows, int nvec) {
  RowGrid g;
  g.J = nvec > 1024 ? 4 : nvec > 256 ? 2 : 1;
  g.W = (nvec + 32 * g.J - 1) / (32 * g.J);
  g.G = std::max(1, 8 / g.W);
  const int64_t need = (rows + g.G - 1) / g.G;
  const int64_t most = (int64_t)num_sms() * std::max(1, (g.J == 1 ? 24 : 16) / (g.W * g.G));
  g.blocks = (int)std::max<int64_t>(1, std::min(need, most));
  return g;
}

}  // namespace
}  // namespace nvfp4moe

using namespace nvfp4moe;

extern "C" {

int moe_add_rmsnorm_quantize_mx(const void* x, const void* residual, const void* gamma, float eps,
                                int64_t rows, int64_t cols, void* h, uint8_t* codes, uint8_t* sf,
                                void* y, float* rrms, moe_stream_t stream) {
  if (rows < 0 || cols <= 0 || cols % 32 != 0 || !(std::isfinite(eps) && eps >= 0.0f))
    return MOE_ERR_INVALID_ARG;
  if (cols > kMaxCols || rows > INT32_MAX) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (rows == 0) return MOE_OK;
  if ((codes == nullptr) != (sf == nullptr) || (!codes && !y)) return MOE_ERR_INVALID_ARG;
  if ((residual == nullptr) != (h == nullptr)) return MOE_ERR_INVALID_ARG;
  if (!x || !gamma) return MOE_ERR_INVALID_ARG;
  for (const void* p : {x, residual, gamma, (const void*)h, (const void*)y})
    if (!is_aligned(p, 16)) return MOE_ERR_INVALID_ARG;
  if (!is_aligned(codes, 8) || !is_aligned(rrms, 4)) return MOE_ERR_INVALID_ARG;
  const RowGrid g = forward_grid(rows, (int)(cols / 8));
  auto k = g.J == 1 ? add_rmsnorm_mx_kernel<1> : g.J == 2 ? add_rmsnorm_mx_kernel<2>
                                                           : add_rmsnorm_mx_kernel<4>;
  const cudaError_t e = launch_pdl(
      k, dim3((unsigned)g.blocks), dim3(g.W * g.G * 32), 0, reinterpret_cast<cudaStream_t>(stream),
      static_cast<const uint4*>(x), static_cast<const uint4*>(residual),
      static_cast<const uint4*>(gamma), eps, rows, (int)cols, g.W, g.G, static_cast<uint4*>(h),
      reinterpret_cast<uint2*>(codes), sf, static_cast<uint4*>(y), rrms);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t moe_add_rmsnorm_backward_workspace_size(int64_t rows, int64_t cols) {
  if (rows < 0 || cols <= 0 || cols > kMaxCols) return 0;
  return align_up(sizeof(float) * (size_t)backward_grid(rows, (int)((cols + 7) / 8)).blocks *
                  (size_t)cols);
}

int moe_add_rmsnorm_backward(const void* dy, const void* dh, const void* h, const float* rrms,
                             const void* gamma, int64_t rows, int64_t cols, void* dx,
                             float* dgamma, void* workspace, size_t ws_bytes,
                             moe_stream_t stream) {
  if (rows < 0 || cols <= 0 || cols % 32 != 0) return MOE_ERR_INVALID_ARG;
  if (cols > kMaxCols || rows > INT32_MAX) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!workspace || ws_bytes < moe_add_rmsnorm_backward_workspace_size(rows, cols))
    return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (!is_aligned(workspace, 16) || !dgamma || !is_aligned(dgamma, 4)) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (rows == 0)
    return cudaMemsetAsync(dgamma, 0, sizeof(float) * cols, s) == cudaSuccess ? MOE_OK
                                                                             : MOE_ERR_CUDA;
  if (!dy || !h || !rrms || !gamma || !dx) return MOE_ERR_INVALID_ARG;
  for (const void* p : {dy, dh, h, gamma, (const void*)dx})
    if (!is_aligned(p, 16)) return MOE_ERR_INVALID_ARG;
  if (!is_aligned(rrms, 4) || dx == h) return MOE_ERR_INVALID_ARG;   // (h is read behind stores to dx)
  const RowGrid g = backward_grid(rows, (int)(cols / 8));
  auto k = g.J == 1   ? add_rmsnorm_backward_kernel<1>
           : g.J == 2 ? add_rmsnorm_backward_kernel<2>
                      : add_rmsnorm_backward_kernel<4>;
  cudaError_t e = launch_pdl(
      k, dim3(g.blocks), dim3(g.W * g.G * 32), g.G > 1 ? sizeof(float) * (size_t)cols : 0, s,
      static_cast<const uint4*>(dy), static_cast<const uint4*>(dh), static_cast<const uint4*>(h),
      rrms, static_cast<const uint4*>(gamma), rows, (int)cols, g.W, g.G, static_cast<uint4*>(dx),
      static_cast<float4*>(workspace));
  if (e == cudaSuccess)
    e = launch_pdl(dgamma_kernel, dim3((unsigned)(cols / 32)), dim3(1024), 0, s,
                   static_cast<const float*>(workspace), g.blocks, (int)cols, dgamma);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
