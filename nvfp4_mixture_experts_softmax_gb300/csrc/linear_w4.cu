// 4-bit matrix-vector product for decode-sized batches: y[t, n] = sum_k x[t, k] * W[n, k] with W
// in the canonical NVFP4 layout (E2M1 codes [N, K/2], E4M3 scales [N, K/16], one FP32 tensor
// scale) or MXFP4 (codes [N, K/2], E8M0 scales [N, K/32]), x BF16 [T, K], y BF16 or FP32 [T, N].
//
// The weights are read once and decoded to BF16 in registers (exact: an E2M1 value times an
// E4M3 scale has at most 6 significant bits), then multiplied on the tensor cores
// (mma m16n8k16: 16 weight rows x 8 tokens, FP32 accumulators).  The sum over k may run in any
// order as long as both operands agree, so lane t of a quad takes 32 consecutive codes (one
// 16-byte load) of its row and the same 32 columns of x, with no shuffles.
//
// A block owns 16 weight rows; its warps split K and join their accumulators in shared memory, in
// warp order.
#include "ops.h"
#include "w4.cuh"

namespace nvfp4moe {

namespace {

constexpr int kLinWarps = 8;
constexpr int kLinRows = 16;
constexpr int kLinMaxTokens = 64;

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two E4M3 scale bytes -> each times 2^118 as BF16x2 (exact, see e2m1x8_to_bf16x2_scaled_down:
// times an E2M1 value placed at 2^-126 the product is the weight times 2^-8).  NaN stays NaN.
__device__ __forceinline__ void e4m3x2_scales(uint32_t b2, uint32_t (&s)[2]) {
  const float2 f = e4m3x2_to_f32x2(b2);
  const __nv_bfloat162 s0 = __float2bfloat162_rn(f.x * 0x1p118f);
  const __nv_bfloat162 s1 = __float2bfloat162_rn(f.y * 0x1p118f);
  s[0] = *reinterpret_cast<const uint32_t*>(&s0);
  s[1] = *reinterpret_cast<const uint32_t*>(&s1);
}

// Codes word -> four BF16x2 words of the weights (NVFP4: times 2^-8).
template <bool kMx>
__device__ __forceinline__ void decode8(uint32_t w, uint32_t scale, uint32_t (&o)[4]) {
  e2m1x8_to_bf16x2_scaled_down(w, o);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kMx) o[i] = mul_bf16x2(o[i], kBf16x2Pow2_126);
    o[i] = mul_bf16x2(o[i], scale);
  }
}

struct LinearArgs {
  const uint16_t* x;
  const uint8_t* codes;
  const uint8_t* sf;
  const float* ts;
  int T;
  int64_t N;
  int K;
  void* y;
};

template <int NT, bool kMx, bool kF32>
__global__ void __launch_bounds__(kLinWarps * 32) linear_w4_kernel(LinearArgs a) {
  __shared__ float red[kLinWarps][NT][32][4];
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int64_t n0 = (int64_t)blockIdx.x * kLinRows;
  // rows behind the last one read it again and are not stored
  const int64_t r0 = min(n0 + g, a.N - 1), r1 = min(n0 + g + 8, a.N - 1);
  constexpr int kBlk = kMx ? 32 : 16;
  float c[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) c[j][i] = 0.0f;
  for (int k0 = warp * 128; k0 < a.K; k0 += kLinWarps * 128) {
    const int k = k0 + q * 32;
    uint4 w0 = make_uint4(0u, 0u, 0u, 0u), w1 = w0;
    uint32_t s0[2] = {0u, 0u}, s1[2] = {0u, 0u};
    const bool in = k < a.K;
    if (in) {
      w0 = __ldg(reinterpret_cast<const uint4*>(a.codes + r0 * (a.K / 2) + k / 2));
      w1 = __ldg(reinterpret_cast<const uint4*>(a.codes + r1 * (a.K / 2) + k / 2));
      const uint8_t* p0 = a.sf + r0 * (a.K / kBlk) + k / kBlk;
      const uint8_t* p1 = a.sf + r1 * (a.K / kBlk) + k / kBlk;
      if constexpr (kMx) {
        const uint32_t b0 = __ldg(p0), b1 = __ldg(p1);
        s0[0] = s0[1] = b0 == 255u ? 0x7FC07FC0u : e8m0_scale_bf16x2(b0);
        s1[0] = s1[1] = b1 == 255u ? 0x7FC07FC0u : e8m0_scale_bf16x2(b1);
      } else {
        e4m3x2_scales(__ldg(reinterpret_cast<const uint16_t*>(p0)), s0);
        e4m3x2_scales(__ldg(reinterpret_cast<const uint16_t*>(p1)), s1);
      }
    }
    const uint32_t cw0[4] = {w0.x, w0.y, w0.z, w0.w}, cw1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t o0[4], o1[4];
      decode8<kMx>(cw0[i], s0[i / 2], o0);
      decode8<kMx>(cw1[i], s1[i / 2], o1);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int t = j * 8 + g;
        const uint4 xv = in && t < a.T
                             ? __ldg(reinterpret_cast<const uint4*>(a.x + (int64_t)t * a.K + k + 8 * i))
                             : make_uint4(0u, 0u, 0u, 0u);
        mma_bf16(c[j], o0[0], o1[0], o0[1], o1[1], xv.x, xv.y);
        mma_bf16(c[j], o0[2], o1[2], o0[3], o1[3], xv.z, xv.w);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j)
    *reinterpret_cast<float4*>(red[warp][j][lane]) = make_float4(c[j][0], c[j][1], c[j][2], c[j][3]);
  __syncthreads();
  // element (row r, token t) sits in lane (r % 8) * 4 + (t % 8) / 2, register (r / 8) * 2 + t % 2
  const float scale = kMx ? 1.0f : __ldg(a.ts) * 256.0f;
  for (int i = threadIdx.x; i < kLinRows * a.T; i += kLinWarps * 32) {
    const int r = i % kLinRows, t = i / kLinRows;
    const int src = (r & 7) * 4 + ((t & 7) >> 1), reg = (r >> 3) * 2 + (t & 1);
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kLinWarps; ++w) s += red[w][t >> 3][src][reg];
    s *= scale;
    if (n0 + r < a.N) {
      const int64_t at = (int64_t)t * a.N + n0 + r;
      if constexpr (kF32) static_cast<float*>(a.y)[at] = s;
      else static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(s);
    }
  }
}

template <int NT>
cudaError_t launch_linear(const LinearArgs& a, bool mx, bool f32, cudaStream_t s) {
  auto k = mx ? (f32 ? linear_w4_kernel<NT, true, true> : linear_w4_kernel<NT, true, false>)
              : (f32 ? linear_w4_kernel<NT, false, true> : linear_w4_kernel<NT, false, false>);
  return launch_pdl(k, dim3((unsigned)((a.N + kLinRows - 1) / kLinRows)), dim3(kLinWarps * 32), 0,
                    s, a);
}

}  // namespace
}  // namespace nvfp4moe

using namespace nvfp4moe;

extern "C" int moe_linear_w4(const void* x, const uint8_t* codes, const uint8_t* sf,
                             const float* ts, int32_t T, int64_t N, int64_t K, uint32_t flags,
                             void* y, moe_stream_t stream) {
  if (T < 0 || N < 0 || K <= 0 || (flags & ~(MOE_LINEAR_MXFP4 | MOE_LINEAR_F32_OUT)) != 0u)
    return MOE_ERR_INVALID_ARG;
  if (T > kLinMaxTokens || K % 32 != 0 || K > (1 << 20) || N > ((int64_t)1 << 30))
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (T == 0 || N == 0) return MOE_OK;
  const bool mx = (flags & MOE_LINEAR_MXFP4) != 0u, f32 = (flags & MOE_LINEAR_F32_OUT) != 0u;
  if (!x || !codes || !sf || !y || (mx ? ts != nullptr : ts == nullptr)) return MOE_ERR_INVALID_ARG;
  if (!is_aligned(x, 16) || !is_aligned(codes, 16) || !is_aligned(sf, 2) || !is_aligned(ts, 4) ||
      !is_aligned(y, f32 ? 4 : 2))
    return MOE_ERR_INVALID_ARG;
  LinearArgs a{static_cast<const uint16_t*>(x), codes, sf, ts, T, N, (int)K, y};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = T <= 8    ? launch_linear<1>(a, mx, f32, s)
                        : T <= 16 ? launch_linear<2>(a, mx, f32, s)
                        : T <= 32 ? launch_linear<4>(a, mx, f32, s)
                                  : launch_linear<8>(a, mx, f32, s);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
