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
#include <cmath>

#include "common.cuh"
#include "ops.h"

namespace nvfp4moe {

namespace {

constexpr int kMaxCols = 16384;

__device__ __forceinline__ void unpack8(uint4 q, float (&f)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_bits_to_f32(w[i] & 0xFFFFu);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Sum of one value per thread over the block, the same on every thread and in a fixed order.
__device__ __forceinline__ float block_sum(float v, float* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane == 0) red[warp] = v;
  __syncthreads();
  float s = lane < nw ? red[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  __syncthreads();
  return s;
}

// One block per row; a thread owns J vectors of 8 columns, so four neighbouring threads share a
// 32-element block.
template <int J>
__global__ void __launch_bounds__(512) add_rmsnorm_mx_kernel(
    const uint4* x, const uint4* residual, const uint4* __restrict__ gamma, float eps,
    int64_t rows, int cols, uint4* h, uint2* codes, uint8_t* sf, uint4* y, float* rrms) {
  __shared__ float red[32];
  griddep_wait();
  griddep_launch();
  const int nvec = cols / 8;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const int64_t base = row * nvec;
    float v[J][8];
    float sq = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = j * blockDim.x + threadIdx.x;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
      if (c < nvec) {
        unpack8(x[base + c], v[j]);
        if (residual) {
          float f[8];
          unpack8(residual[base + c], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[j][i] += f[i];
          const uint4 p = pack8(v[j]);
          unpack8(p, v[j]);
          if (h) h[base + c] = p;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sq = fmaf(v[j][i], v[j][i], sq);
      }
    }
    sq = block_sum(sq, red);
    const float r = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(sq, (float)cols), eps)));
    if (rrms && threadIdx.x == 0) rrms[row] = r;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = j * blockDim.x + threadIdx.x;
      const bool in = c < nvec;
      float g[8];
      unpack8(in ? __ldg(gamma + c) : make_uint4(0u, 0u, 0u, 0u), g);
      uint32_t top = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[j][i] = __fmul_rn(__fmul_rn(v[j][i], r), g[i]);
        top = max(top, __float_as_uint(fabsf(v[j][i])));   // NaN orders above infinity
      }
      if (y && in) y[base + c] = pack8(v[j]);
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
        lo = f32_to_e4m3x2(v[j][0] * inv, v[j][1] * inv) |
             f32_to_e4m3x2(v[j][2] * inv, v[j][3] * inv) << 16;
        hi = f32_to_e4m3x2(v[j][4] * inv, v[j][5] * inv) |
             f32_to_e4m3x2(v[j][6] * inv, v[j][7] * inv) << 16;
      }
      codes[base + c] = make_uint2(lo, hi);
      if ((c & 3) == 0) sf[(base + c) >> 2] = (uint8_t)sb;
    }
  }
}

// One block takes rows blockIdx, blockIdx + gridDim, ...; a thread owns the same J vectors of 8
// columns in all of them and keeps their share of dgamma in registers.
template <int J>
__global__ void __launch_bounds__(512) add_rmsnorm_backward_kernel(
    const uint4* dy, const uint4* dh, const uint4* __restrict__ h,
    const float* __restrict__ rrms, const uint4* __restrict__ gamma, int64_t rows, int cols,
    uint4* dx, float4* __restrict__ partial) {
  __shared__ float red[32];
  griddep_wait();
  griddep_launch();
  const int nvec = cols / 8;
  const float inv_cols = __fdiv_rn(1.0f, (float)cols);
  float dg[J][8];
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) dg[j][i] = 0.0f;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const int64_t base = row * nvec;
    const float r = __ldg(rrms + row);
    float s = 0.0f;
    uint4 qd[J], qh[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = j * blockDim.x + threadIdx.x;
      const bool in = c < nvec;
      qd[j] = in ? dy[base + c] : make_uint4(0u, 0u, 0u, 0u);
      qh[j] = in ? __ldg(h + base + c) : make_uint4(0u, 0u, 0u, 0u);
      float d[8], hv[8], g[8];
      unpack8(qd[j], d);
      unpack8(qh[j], hv);
      unpack8(in ? __ldg(gamma + c) : make_uint4(0u, 0u, 0u, 0u), g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s = fmaf(d[i] * g[i], hv[i], s);
        if (in) dg[j][i] = fmaf(d[i], hv[i] * r, dg[j][i]);
      }
    }
    s = block_sum(s, red);
    const float m = r * r * (s * inv_cols);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = j * blockDim.x + threadIdx.x;
      if (c >= nvec) continue;
      float d[8], hv[8], g[8], o[8];
      unpack8(qd[j], d);
      unpack8(qh[j], hv);
      unpack8(__ldg(gamma + c), g);
      float e[8];
      if (dh) unpack8(dh[base + c], e);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        o[i] = r * fmaf(-hv[i], m, d[i] * g[i]);
        if (dh) o[i] += e[i];
      }
      dx[base + c] = pack8(o);
    }
  }
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c = j * blockDim.x + threadIdx.x;
    if (c >= nvec) continue;
    float4* p = partial + (int64_t)blockIdx.x * (cols / 4) + 2 * c;
    p[0] = make_float4(dg[j][0], dg[j][1], dg[j][2], dg[j][3]);
    p[1] = make_float4(dg[j][4], dg[j][5], dg[j][6], dg[j][7]);
  }
}

// dgamma = sum of the blocks' partial rows, in block order.
__global__ void __launch_bounds__(256) dgamma_kernel(const float* __restrict__ partial, int nb,
                                                     int cols, float* __restrict__ dgamma) {
  __shared__ float red[8][32];
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.0f;
  for (int b = warp; b < nb; b += 8) s += __ldcg(partial + (int64_t)b * cols + c);
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int w = 1; w < 8; ++w) s += red[w][lane];
    dgamma[c] = s;
  }
}

// Threads for a row of nvec vectors with J of them each: whole warps.
int row_threads(int nvec, int J) { return ((nvec + J - 1) / J + 31) / 32 * 32; }

int backward_blocks(int64_t rows) {
  const int64_t most = 2 * (int64_t)num_sms();
  return (int)(rows < most ? rows : most);
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
  const int nvec = (int)(cols / 8);
  const int J = nvec <= 512 ? 1 : nvec <= 1024 ? 2 : 4;
  const dim3 grid((unsigned)rows), block(row_threads(nvec, J));
  auto k = J == 1 ? add_rmsnorm_mx_kernel<1> : J == 2 ? add_rmsnorm_mx_kernel<2>
                                                       : add_rmsnorm_mx_kernel<4>;
  const cudaError_t e = launch_pdl(
      k, grid, block, 0, reinterpret_cast<cudaStream_t>(stream), static_cast<const uint4*>(x),
      static_cast<const uint4*>(residual), static_cast<const uint4*>(gamma), eps, rows, (int)cols,
      static_cast<uint4*>(h), reinterpret_cast<uint2*>(codes), sf, static_cast<uint4*>(y), rrms);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t moe_add_rmsnorm_backward_workspace_size(int64_t rows, int64_t cols) {
  if (rows < 0 || cols <= 0) return 0;
  return align_up(sizeof(float) * (size_t)backward_blocks(rows) * (size_t)cols);
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
  if (!is_aligned(rrms, 4)) return MOE_ERR_INVALID_ARG;
  const int nvec = (int)(cols / 8);
  const int J = nvec <= 512 ? 1 : nvec <= 1024 ? 2 : 4;
  const int nb = backward_blocks(rows);
  auto k = J == 1 ? add_rmsnorm_backward_kernel<1> : J == 2 ? add_rmsnorm_backward_kernel<2>
                                                             : add_rmsnorm_backward_kernel<4>;
  cudaError_t e = launch_pdl(
      k, dim3(nb), dim3(row_threads(nvec, J)), 0, s, static_cast<const uint4*>(dy),
      static_cast<const uint4*>(dh), static_cast<const uint4*>(h), rrms,
      static_cast<const uint4*>(gamma), rows, (int)cols, static_cast<uint4*>(dx),
      static_cast<float4*>(workspace));
  if (e == cudaSuccess)
    e = launch_pdl(dgamma_kernel, dim3((unsigned)(cols / 32)), dim3(256), 0, s,
                   static_cast<const float*>(workspace), nb, (int)cols, dgamma);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
