// What the row kernels (norm_mx.cu, tokens.cu) share: vectors of eight BF16 elements and sums over the threads
// of a row.
#pragma once
#include "common.cuh"

namespace nvfp4moe {

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

// Sum of one value per thread over the W warps of a row group, the same on every thread and in a
// fixed order.  One barrier: `red` holds two rows' partial sums in turn (a warp that writes a row's
// has passed the barrier of the row before, behind the reads of the one before that).
__device__ __forceinline__ float row_sum(float v, float* red, int W, int wrow, int group, int G,
                                         int parity) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (W == 1) return v;
  const int lane = threadIdx.x & 31;
  float* mine = red + (parity * G + group) * 32;
  if (lane == 0) mine[wrow] = v;
  if (G == 1) __syncthreads();
  else asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(W * 32) : "memory");
  float s = lane < W ? mine[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

}  // namespace nvfp4moe
