// Residual addition + layer norm, and its backward pass, BF16 or FP32 throughout.
//
// Forward, per row:  h = x + residual in the tensors' type,  m = mean(h),  v = mean((h - m)^2),
// s = 1 / sqrt(v + eps),  y = (h - m) * s * gamma + beta.  The row stays in registers, so the variance
// is the mean of the squared distances themselves (a second sum over the row): the difference of
// mean(h^2) and m^2 would lose rows whose mean is large against their spread.
//
// Backward, with n = (h - m) * s and a = gamma * dy:  dx = dh + s * (a - mean(a) - n * mean(a * n)),
// dgamma_c = sum over rows of dy * n,  dbeta_c = sum over rows of dy.  Both row sums go over one barrier.
//
// Both are bound by HBM: every element is read and written once.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "ops.h"
#include "rows.cuh"

namespace nvfp4moe {

namespace {

constexpr int kMaxCols = 16384;

// How a row is laid over threads: W warps with J vectors of 8 columns a lane (vector c of lane t:
// c = j * 32 W + t); a block holds G such row groups, each of which takes every gridDim * G-th row.
struct NormGrid {
  int J, W, G, blocks;
};

// The next row is loaded before the current one is reduced.
template <typename V, int J>
__global__ void __launch_bounds__(512, sizeof(V) == 16 && J <= 2 ? 2 : 1) add_layernorm_kernel(
    const V* x, const V* residual, const V* __restrict__ gamma, const V* __restrict__ beta, float eps,
    int64_t rows, int cols, int W, int G, V* h, V* y, float* mean, float* rstd) {
  __shared__ float red[2 * 16 * 32];
  const int warp = threadIdx.x >> 5, group = warp / W, wrow = warp - group * W;
  const int t = wrow * 32 + (threadIdx.x & 31), span = W * 32;   // thread of the row, vectors apart
  const int nvec = cols / 8;
  const float inv_cols = __fdiv_rn(1.0f, (float)cols);
  griddep_wait();
  griddep_launch();
  const V zero = {};
  int64_t row = (int64_t)blockIdx.x * G + group;
  const int64_t step = (int64_t)gridDim.x * G;
  V nx[J], nr[J];
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
  for (; row < rows; row += step) {
    const int64_t base = row * nvec;
    V hv[J];
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float f[8];
      hv[j] = nx[j];
      unpack8(hv[j], f);
      if (residual) {
        float g[8];
        unpack8(nr[j], g);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] += g[i];
        pack(f, hv[j]);
        unpack8(hv[j], f);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) s += f[i];
    }
    load(row + step);   // (rows are written by their own group only, after this group read them)
    if (h) {
#pragma unroll
      for (int j = 0; j < J; ++j)
        if (j * span + t < nvec) h[base + j * span + t] = hv[j];
    }
    const float m = row_sum(s, red, W, wrow, group, G, 0) * inv_cols;
    s = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float f[8];
      unpack8(hv[j], f);
      if (j * span + t < nvec)
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(f[i] - m, f[i] - m, s);
    }
    const float var = row_sum(s, red, W, wrow, group, G, 1) * inv_cols;
    const float r = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(var, eps)));
    if (t == 0) {
      if (mean) mean[row] = m;
      if (rstd) rstd[row] = r;
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = j * span + t;
      if (c >= nvec) continue;
      float v[8], g[8], b[8];
      unpack8(hv[j], v);
      unpack8(gamma[c], g);
      unpack8(beta ? beta[c] : zero, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = fmaf((v[i] - m) * r, g[i], b[i]);
      V o;
      pack(v, o);
      y[base + c] = o;
    }
  }
}

// The sums of two values over the row's warps; as row_sum, over one barrier.
__device__ __forceinline__ float2 row_sum2(float2 v, float2* red, int W, int wrow, int group, int G,
                                           int parity) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  if (W == 1) return v;
  const int lane = threadIdx.x & 31;
  float2* mine = red + (parity * G + group) * 32;
  if (lane == 0) mine[wrow] = v;
  if (G == 1) __syncthreads();
  else asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(W * 32) : "memory");
  float2 s = lane < W ? mine[lane] : make_float2(0.0f, 0.0f);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
    s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
  }
  return s;
}

// A thread owns the same J vectors of 8 columns in all rows of its group and keeps their share of
// dgamma and dbeta in registers; the groups of a block are joined in order at the end, the blocks by
// column_sums_kernel.
template <typename V, int J, bool kAhead>
__global__ void __launch_bounds__(512, 1) add_layernorm_backward_kernel(
    const V* dy, const V* dh, const V* h, const float* __restrict__ mean, const float* __restrict__ rstd,
    const V* __restrict__ gamma, int64_t rows, int cols, int W, int G, V* dx, bool want_beta,
    float4* __restrict__ partial) {
  extern __shared__ float4 s_part[];   // [cols / 4] if G > 1
  __shared__ float2 red[2 * 16 * 32];
  const int warp = threadIdx.x >> 5, group = warp / W, wrow = warp - group * W;
  const int t = wrow * 32 + (threadIdx.x & 31), span = W * 32;
  const int nvec = cols / 8;
  const float inv_cols = __fdiv_rn(1.0f, (float)cols);
  griddep_wait();
  griddep_launch();
  const V zero = {};
  float dg[J][8], db[J][8];
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) dg[j][i] = db[j][i] = 0.0f;
  int64_t row = (int64_t)blockIdx.x * G + group;
  const int64_t step = (int64_t)gridDim.x * G;
  V nd[J], nh[J], ne[J];
  float nm = 0.0f, nr = 0.0f;
  auto load_dh = [&](int64_t rw) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = j * span + t;
      ne[j] = rw < rows && c < nvec && dh ? dh[rw * nvec + c] : zero;
    }
  };
  auto load = [&](int64_t rw) {
    nm = rw < rows ? __ldg(mean + rw) : 0.0f;
    nr = rw < rows ? __ldg(rstd + rw) : 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = j * span + t;
      const bool in = rw < rows && c < nvec;
      nd[j] = in ? dy[rw * nvec + c] : zero;
      nh[j] = in ? h[rw * nvec + c] : zero;
    }
    if (kAhead) load_dh(rw);
  };
  if (kAhead) load(row);
  for (int parity = 0; row < rows; row += step, parity ^= 1) {
    if (!kAhead) load(row);
    const float m = nm, r = nr;
    V qd[J], qh[J], qe[J];
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      qd[j] = nd[j];
      qh[j] = nh[j];
      if (kAhead) qe[j] = ne[j];
      if (j * span + t >= nvec) continue;
      float d[8], hv[8], g[8];
      unpack8(qd[j], d);
      unpack8(qh[j], hv);
      unpack8(gamma[j * span + t], g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = (hv[i] - m) * r, a = d[i] * g[i];
        s.x += a;
        s.y = fmaf(a, n, s.y);
        dg[j][i] = fmaf(d[i], n, dg[j][i]);
        db[j][i] += d[i];
      }
    }
    if constexpr (kAhead) {
      load(row + step);
    } else {   // dh is not part of the row's sums
      load_dh(row);
#pragma unroll
      for (int j = 0; j < J; ++j) qe[j] = ne[j];
    }
    s = row_sum2(s, red, W, wrow, group, G, parity);
    const float ma = s.x * inv_cols, mn = s.y * inv_cols;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = j * span + t;
      if (c >= nvec) continue;
      float d[8], hv[8], e[8], g[8], o[8];
      unpack8(qd[j], d);
      unpack8(qh[j], hv);
      unpack8(qe[j], e);
      unpack8(gamma[c], g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = (hv[i] - m) * r;
        o[i] = r * fmaf(-n, mn, fmaf(d[i], g[i], -ma));
        if (dh) o[i] += e[i];
      }
      V q;
      pack(o, q);
      dx[row * nvec + c] = q;
    }
  }
#pragma unroll
  for (int which = 0; which < 2; ++which) {   // dgamma, then dbeta
    if (which == 1 && !want_beta) break;
    float(&acc)[J][8] = which ? db : dg;
    for (int k = 1; k < G; ++k) {   // the other groups' sums to the first's, in order
      __syncthreads();
      if (group == k) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const int c = j * span + t;
          if (c >= nvec) continue;
          s_part[2 * c] = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
          s_part[2 * c + 1] = make_float4(acc[j][4], acc[j][5], acc[j][6], acc[j][7]);
        }
      }
      __syncthreads();
      if (group == 0) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const int c = j * span + t;
          if (c >= nvec) continue;
          const float4 u = s_part[2 * c], v = s_part[2 * c + 1];
          acc[j][0] += u.x; acc[j][1] += u.y; acc[j][2] += u.z; acc[j][3] += u.w;
          acc[j][4] += v.x; acc[j][5] += v.y; acc[j][6] += v.z; acc[j][7] += v.w;
        }
      }
    }
    if (group != 0) continue;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = j * span + t;
      if (c >= nvec) continue;
      float4* p = partial + ((int64_t)which * gridDim.x + blockIdx.x) * (cols / 4) + 2 * c;
      p[0] = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
      p[1] = make_float4(acc[j][4], acc[j][5], acc[j][6], acc[j][7]);
    }
  }
}

// dgamma (blockIdx.y = 0) and dbeta (1): the sum of the blocks' partial rows.  Warp w takes rows w,
// w + 32, ..., then the warps in order.
__global__ void __launch_bounds__(1024) column_sums_kernel(const float* __restrict__ partial, int nb,
                                                           int cols, float* __restrict__ dgamma,
                                                           float* __restrict__ dbeta) {
  __shared__ float red[32][33];
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const float* part = partial + (int64_t)blockIdx.y * nb * cols;
  float s = 0.0f;
  if (c < cols)
#pragma unroll 10
    for (int b = warp; b < nb; b += 32) s += __ldcg(part + (int64_t)b * cols + c);
  red[warp][lane] = s;
  __syncthreads();
  // lane w of warp c adds warp w's share of column c
  s = red[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const int col = blockIdx.x * 32 + warp;
  if (lane == 0 && col < cols) (blockIdx.y ? dbeta : dgamma)[col] = s;
}

// Few rows: as many warps a row as its vectors fill, for the latency.  Many rows: two vectors a
// lane, at least eight warps a block.
NormGrid forward_grid(int64_t rows, int nvec, bool f32) {
  NormGrid g;
  const bool few = rows <= 2 * (int64_t)num_sms();
  g.J = nvec > 1024 ? 4 : nvec > 512 || (!few && !f32 && nvec > 32) ? 2 : 1;
  g.W = (nvec + 32 * g.J - 1) / (32 * g.J);
  g.G = few ? 1 : std::max(1, 8 / g.W);
  const int64_t need = (rows + g.G - 1) / g.G;
  const int64_t most = (int64_t)num_sms() * std::max(1, (!f32 && g.J <= 2 ? 32 : 16) / (g.W * g.G));
  g.blocks = (int)std::min(need, most);
  return g;
}

// At most kPartBlocks blocks, which the workspace's size goes by: it does not depend on the device.
constexpr int kPartBlocks = 320;
NormGrid backward_grid(int64_t rows, int nvec) {
  NormGrid g;
  g.J = nvec > 1024 ? 4 : nvec > 256 ? 2 : 1;
  g.W = (nvec + 32 * g.J - 1) / (32 * g.J);
  g.G = std::max(1, 8 / g.W);
  const int64_t need = (rows + g.G - 1) / g.G;
  const int64_t most = std::min<int64_t>(kPartBlocks, (int64_t)num_sms() * std::max(1, 16 / (g.W * g.G)));
  g.blocks = (int)std::max<int64_t>(1, std::min(need, most));
  return g;
}

template <typename V>
cudaError_t launch_forward(const void* x, const void* residual, const void* gamma, const void* beta,
                           float eps, int64_t rows, int cols, void* h, void* y, float* mean,
                           float* rstd, cudaStream_t s) {
  const NormGrid g = forward_grid(rows, cols / 8, sizeof(V) == 32);
  auto k = g.J == 1 ? add_layernorm_kernel<V, 1> : g.J == 2 ? add_layernorm_kernel<V, 2>
                                                            : add_layernorm_kernel<V, 4>;
  return launch_pdl(k, dim3((unsigned)g.blocks), dim3(g.W * g.G * 32), 0, s, static_cast<const V*>(x),
                    static_cast<const V*>(residual), static_cast<const V*>(gamma),
                    static_cast<const V*>(beta), eps, rows, cols, g.W, g.G, static_cast<V*>(h),
                    static_cast<V*>(y), mean, rstd);
}

template <typename V>
cudaError_t launch_backward(const void* dy, const void* dh, const void* h, const float* mean,
                            const float* rstd, const void* gamma, int64_t rows, int cols, void* dx,
                            float* dgamma, float* dbeta, void* workspace, cudaStream_t s) {
  const NormGrid g = backward_grid(rows, cols / 8);
  constexpr bool kBf16 = sizeof(V) == 16;
  auto k = g.J == 1   ? add_layernorm_backward_kernel<V, 1, true>
           : g.J == 2 ? add_layernorm_backward_kernel<V, 2, kBf16>
                      : add_layernorm_backward_kernel<V, 4, false>;
  const cudaError_t e = launch_pdl(
      k, dim3(g.blocks), dim3(g.W * g.G * 32), g.G > 1 ? sizeof(float) * (size_t)cols : 0, s,
      static_cast<const V*>(dy), static_cast<const V*>(dh), static_cast<const V*>(h), mean, rstd,
      static_cast<const V*>(gamma), rows, cols, g.W, g.G, static_cast<V*>(dx), dbeta != nullptr,
      static_cast<float4*>(workspace));
  if (e != cudaSuccess) return e;
  return launch_pdl(column_sums_kernel, dim3((unsigned)((cols + 31) / 32), dbeta ? 2 : 1), dim3(1024),
                    0, s, static_cast<const float*>(workspace), g.blocks, cols, dgamma, dbeta);
}

}  // namespace
}  // namespace nvfp4moe

using namespace nvfp4moe;

extern "C" {

int moe_add_layernorm(const void* x, const void* residual, const void* gamma, const void* beta,
                      float eps, int64_t rows, int64_t cols, uint32_t flags, void* h, void* y,
                      float* mean, float* rstd, moe_stream_t stream) {
  if (rows < 0 || cols <= 0 || cols % 8 != 0 || !(std::isfinite(eps) && eps >= 0.0f) ||
      (flags & ~MOE_ROWS_F32))
    return MOE_ERR_INVALID_ARG;
  if (cols > kMaxCols || rows > INT32_MAX) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (rows == 0) return MOE_OK;
  if (!x || !gamma || !y || (residual == nullptr) != (h == nullptr)) return MOE_ERR_INVALID_ARG;
  for (const void* p : {x, residual, gamma, beta, (const void*)h, (const void*)y})
    if (!is_aligned(p, 16)) return MOE_ERR_INVALID_ARG;
  if (!is_aligned(mean, 4) || !is_aligned(rstd, 4)) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = flags & MOE_ROWS_F32
                            ? launch_forward<F32x8>(x, residual, gamma, beta, eps, rows, (int)cols, h,
                                                    y, mean, rstd, s)
                            : launch_forward<uint4>(x, residual, gamma, beta, eps, rows, (int)cols, h,
                                                    y, mean, rstd, s);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t moe_add_layernorm_backward_workspace_size(int64_t rows, int64_t cols) {
  if (rows < 0 || cols <= 0 || cols > kMaxCols) return 0;
  return align_up(2 * sizeof(float) * (size_t)std::min<int64_t>(std::max<int64_t>(rows, 1), kPartBlocks) *
                  (size_t)cols);
}

int moe_add_layernorm_backward(const void* dy, const void* dh, const void* h, const float* mean,
                               const float* rstd, const void* gamma, int64_t rows, int64_t cols,
                               uint32_t flags, void* dx, float* dgamma, float* dbeta, void* workspace,
                               size_t ws_bytes, moe_stream_t stream) {
  if (rows < 0 || cols <= 0 || cols % 8 != 0 || (flags & ~MOE_ROWS_F32)) return MOE_ERR_INVALID_ARG;
  if (cols > kMaxCols || rows > INT32_MAX) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!workspace || ws_bytes < moe_add_layernorm_backward_workspace_size(rows, cols))
    return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (!is_aligned(workspace, 16) || !dgamma || !is_aligned(dgamma, 4) || !is_aligned(dbeta, 4))
    return MOE_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (rows == 0) {
    cudaError_t e = cudaMemsetAsync(dgamma, 0, sizeof(float) * cols, s);
    if (e == cudaSuccess && dbeta) e = cudaMemsetAsync(dbeta, 0, sizeof(float) * cols, s);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  }
  if (!dy || !h || !mean || !rstd || !gamma || !dx) return MOE_ERR_INVALID_ARG;
  for (const void* p : {dy, dh, h, gamma, (const void*)dx})
    if (!is_aligned(p, 16)) return MOE_ERR_INVALID_ARG;
  if (!is_aligned(mean, 4) || !is_aligned(rstd, 4) || dx == h) return MOE_ERR_INVALID_ARG;
  const cudaError_t e =
      flags & MOE_ROWS_F32
          ? launch_backward<F32x8>(dy, dh, h, mean, rstd, gamma, rows, (int)cols, dx, dgamma, dbeta,
                                   workspace, s)
          : launch_backward<uint4>(dy, dh, h, mean, rstd, gamma, rows, (int)cols, dx, dgamma, dbeta,
                                   workspace, s);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
