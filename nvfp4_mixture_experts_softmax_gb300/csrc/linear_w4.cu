// 4-bit matrix-vector product for decode-sized batches: y[t, n] = sum_k x[t, k] * W[n, k] with W
// in the canonical NVFP4 layout (E2M1 codes [N, K/2], E4M3 scales [N, K/16], one FP32 tensor
// scale) or MXFP4 (codes [N, K/2], E8M0 scales [N, K/32]), x BF16 [T, K], y BF16 or FP32 [T, N].
//
// The weights are read once, decoded in registers and multiplied on the tensor cores
// (mma m16n8k16: 16 weight rows x 8 tokens, FP32 accumulators); x sits in shared memory.  The sum
// over k may run in any order as long as both operands agree, so lane q of a quad takes
// consecutive codes of its rows and the same columns of x, with no shuffles.
//
// For few tokens the bound is the instruction stream of the decoding next to HBM: at the copy rate
// an SM has 22 issue slots for 8 codes.  The conversion of two E2M1 codes to F16 is one
// instruction (measured 27 T codes/s over the GPU; placing the bits of a BF16 by hand 13.7; HBM
// delivers 13.4), so weights and x are F16:
//   * an E2M1 value times an E4M3 scale is exact in F16 (at most 6 significant bits, 2^-10 to
//     2688).  So is one times an E8M0 scale of 2^-23 .. 2^13; a warp that meets another scale, in a
//     block that is not all zeros, does its part of the tile again in BF16, where every scale is
//     exact;
//   * a row of x is multiplied by a power of two: 2^6 if its elements are zero or in [2^-23, 2^10),
//     otherwise the one that brings its largest to [2^15, 2^16) (one more pass over x).  From 2^-17 on
//     F16 holds all of BF16's 8 bits; if an element lies lower even so, 2^32 below its row's largest,
//     the whole product is done in BF16, whose exponents are FP32's, without staging x (18432 x 7168,
//     1 / 8 rows 33 / 50 us).
// So every product is exact, whichever type it takes.
// With more tokens the MMAs weigh most (two cycles each on an SM's four tensor cores: 14 us for
// 18432 x 7168 at 32 tokens), so linear_w4_tc.cu takes over.
//
// K is split twice: over the blocks of a cluster, so that a block can keep its share of x in
// shared memory, and over ks warps of a block.  A group of ks warps works on a tile of kMt * 16
// weight rows; the partial sums are joined through (distributed) shared memory in a fixed order.
//
// Measured (device time of a call): 131072 x 4096 NVFP4, 1 token 60 us (5.0 TB/s; a pure read of HBM
// reaches 5.8), 16 tokens 78 us; 18432 x 7168, 1 / 8 tokens 19.5 / 25.5 us; 2048 x 2048, 1 token 3.8
// us.  A block of 16 rows whose eight warps read x from L1 in BF16, without staging, took 77.6, 166,
// 22.2 / 39 and 2.8 us.
#include <algorithm>

#include "common.cuh"
#include "ops.h"
#include "w4.cuh"

namespace nvfp4moe {

namespace {

constexpr int kLinMaxTokens = 64;
constexpr int kLinSmem = 222 * 1024;  // dynamic shared memory of a block, at most
constexpr int kLinRows = 16;          // of x in this kernel
constexpr int kTopGuess = 9;         // largest exponent of an element of x at the first power of two
constexpr int kF16Top = 15;          // exponents of F16
constexpr int kF16Exact = -17;       // from which on it holds 8 significant bits
constexpr int kBf16Top = 60;         // a row's largest in BF16 with NVFP4 weights

// Tiling by the number of 8-token columns NT.  One column: 16-row tiles, 16 warps of 64 registers
// and two blocks an SM, whose many warps hide the latency of the loads.  Two columns: x fills the
// shared memory of an SM, so one block of 16 warps with 128 registers, 32-row tiles (each x
// fragment is used twice) and more loads in flight a warp.
template <int NT>
struct LinTile {
  static constexpr int kMt = NT == 1 ? 1 : 2;        // 16-row MMA tiles of a warp
  static constexpr int kWarps = 16;
  static constexpr int kPerSm = NT == 1 ? 2 : 1;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kRows = kMt * 16;
  static constexpr int kHalves = 2;                  // 128-column parts of a step
  static constexpr int kFly = NT == 1 ? 4 : 8;       // loads of x in flight in a lane
  static constexpr int kStep = kHalves * 128;        // columns of a step
  // join buffer: a warp's kMt * NT accumulator fragments
  static constexpr int kFrags = kMt * NT;
  static constexpr int kJoinBytes = kWarps * kFrags * 512;
};
constexpr int kScaleWindow = 37;     // binades of E8M0 scales that are exact in F16
constexpr int kScaleLow = 104;       // scale byte of the lowest

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight E2M1 codes -> four F16x2 words of their values, codes 2i and 2i+1 in word i.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t (&o)[4]) {
  asm("{\n"
      ".reg .b8 b0, b1, b2, b3;\n"
      "mov.b32 {b0, b1, b2, b3}, %4;\n"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n"
      "}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}

__device__ __forceinline__ void decode8(uint32_t w, uint32_t scale, uint32_t (&o)[4]) {
  e2m1x8_to_f16x2(w, o);
#pragma unroll
  for (int i = 0; i < 4; ++i) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(o[i]) : "r"(scale));
}

// One row's 32 codes of 128 columns in a lane, and their scale bytes (NVFP4 two, MXFP4 one).
struct RowCodes {
  uint4 c;
  uint32_t s;
  __device__ __forceinline__ uint32_t word(int i) const {
    return i == 0 ? c.x : i == 1 ? c.y : i == 2 ? c.z : c.w;
  }
};

// Scale of unit i (8 codes) of 32 as F16x2, from their scale bytes; MXFP4: 2^(byte - 127), outside
// F16's range some finite value (codes that are not zero are then done again), 255 NaN.
template <bool kMx>
__device__ __forceinline__ uint32_t unit_scale(uint32_t bytes, int i) {
  if constexpr (kMx) {
    const int f = (int)bytes - 112;   // F16 exponent field; subnormal below 1
    uint32_t h = f > 0 ? (uint32_t)min(f, 30) << 10 : 0x200u >> min(-f, 31);
    if (bytes == 255u) h = 0x7E00u;
    return h | (h << 16);
  } else {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)bytes));
    return __byte_perm(h2, 0u, (i & 2) ? 0x3232 : 0x1010);
  }
}

// floor(log2) of a finite nonzero BF16 magnitude.
__device__ __forceinline__ int bf16_exponent(uint32_t m) {
  return m >= 0x80u ? (int)(m >> 7) - 127 : 31 - __clz(m) - 133;
}

// 2^e as two factors, e in [-252, 254].
__device__ __forceinline__ float2 pow2_factors(int e) {
  return make_float2(__uint_as_float((uint32_t)(e / 2 + 127) << 23),
                     __uint_as_float((uint32_t)(e - e / 2 + 127) << 23));
}

__device__ __forceinline__ void st_dsmem_float4(const void* local_smem, uint32_t rank,
                                                const float* v) {
  uint32_t ra;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(smem_u32(local_smem)), "r"(rank));
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(ra), "f"(v[0]), "f"(v[1]),
               "f"(v[2]), "f"(v[3])
               : "memory");
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
  int warps;    // warps of a block that multiply; further ones only bring x into shared memory
  int ks;       // warps that split a tile's steps
  int cluster;  // blocks that split K
  int kslice;   // columns of a block, a multiple of the step
  int kc;       // columns of x in shared memory at a time, a multiple of the step
  int iters;    // tiles of a group of ks warps
};

// Columns [k0, k0 + kc) of x, row t times 2^shift[t], to shared memory as F16 (zeros from column ke
// on); sets *bad if an element is not exact there at the first power of two.  A warp takes a row's
// units (8 columns) 32 at a time, kFly loads in flight.  Inside 128 columns, lane q's i-th unit
// (u = 4 q + i) sits at i * 64 + q * 16, so that a quad's loads of one i are 64 consecutive bytes;
// rows are 64 bytes off a multiple of 128, so two rows fill all banks.  Not inlined: the kernel's
// registers are the multiplication's.
template <int kFly>
__device__ __noinline__ void stage_x(const uint16_t* x, int T, int K, int k0, int kc, int ke,
                                     uint8_t* xs, const int* shift, uint32_t* bad) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int units = kc / 8, per = (units + kFly * 32 - 1) / (kFly * 32), stride = kc * 2 + 64;
  for (int v = warp; v < T * per; v += warps) {
    const int t = v / per, u0 = (v - t * per) * (kFly * 32) + lane;
    const uint4* src = reinterpret_cast<const uint4*>(x + (int64_t)t * K + k0);
    uint4 d[kFly];
#pragma unroll
    for (int b = 0; b < kFly; ++b) {
      const int u = u0 + b * 32;
      d[b] = u < units && k0 + u * 8 < ke ? __ldg(src + u) : make_uint4(0u, 0u, 0u, 0u);
    }
    const float f = __uint_as_float((uint32_t)(shift[t] + 127) << 23);
    uint32_t hi = 0u, lo = 0x7FFF7FFFu;
#pragma unroll
    for (int b = 0; b < kFly; ++b) {
      const int u = u0 + b * 32;
      if (u >= units) break;
      uint32_t w[4] = {d[b].x, d[b].y, d[b].z, d[b].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // per half 0x8000 + magnitude - 1: unsigned, zeros are below all others; signed, above
        const uint32_t m = (w[j] | 0x80008000u) - 0x00010001u;
        hi = __vmaxu2(hi, m);
        lo = __vmins2(lo, m);
        const __half2 hh = __floats2half2_rn(__uint_as_float(w[j] << 16) * f,
                                             __uint_as_float(w[j] & 0xFFFF0000u) * f);
        w[j] = *reinterpret_cast<const uint32_t*>(&hh);
      }
      *reinterpret_cast<uint4*>(xs + (size_t)t * stride + (u >> 4) * 256 + (u & 3) * 64 +
                                ((u >> 2) & 3) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    constexpr uint32_t kBelow = 0x8000u + ((uint32_t)(kTopGuess + 128) << 7) - 1u;
    constexpr int kFrom = ((kF16Exact + kTopGuess - kF16Top + 127) << 7) - 1 - 0x8000;
    const bool fits = max(hi >> 16, hi & 0xFFFFu) < kBelow &&
                      min((int)(int16_t)(lo >> 16), (int)(int16_t)(lo & 0xFFFFu)) >= kFrom;
    if (!__all_sync(0xffffffffu, fits) && lane == 0) *bad = 1u;   // (every writer writes the same)
  }
}

// The largest finite magnitude of each row of x over all of K to hi[t] (BF16 bits, 0 before), the
// smallest that is not zero to lo[t] (0xFFFF before).
__device__ __noinline__ void find_range(const uint16_t* x, int T, int K, uint32_t* hi, uint32_t* lo) {
  constexpr int kFly = 4;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int units = K / 8, per = (units + kFly * 32 - 1) / (kFly * 32);
  for (int v = warp; v < T * per; v += warps) {
    const int t = v / per, u0 = (v - t * per) * (kFly * 32) + lane;
    const uint4* row = reinterpret_cast<const uint4*>(x + (int64_t)t * K);
    uint4 d[kFly];
#pragma unroll
    for (int b = 0; b < kFly; ++b)
      d[b] = u0 + b * 32 < units ? __ldg(row + u0 + b * 32) : make_uint4(0u, 0u, 0u, 0u);
    uint32_t top = 0u, low = 0x7FFF7FFFu;
#pragma unroll
    for (int b = 0; b < kFly; ++b) {
      const uint32_t w[4] = {d[b].x, d[b].y, d[b].z, d[b].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        top = __vmaxu2(top, w[j] & 0x7FFF7FFFu);
        low = __vmins2(low, (w[j] | 0x80008000u) - 0x00010001u);   // (see stage_x)
      }
    }
    top = max(top >> 16, top & 0xFFFFu);
    if (top >= 0x7F80u) {   // without the infinities and NaN
      top = 0u;
#pragma unroll
      for (int b = 0; b < kFly; ++b) {
        const uint32_t w[4] = {d[b].x, d[b].y, d[b].z, d[b].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t m = (w[i >> 1] >> (16 * (i & 1))) & 0x7FFFu;
          if (m < 0x7F80u) top = max(top, m);
        }
      }
    }
    const int least = min((int)(int16_t)(low >> 16), (int)(int16_t)(low & 0xFFFFu));
    top = __reduce_max_sync(0xffffffffu, top);
    low = __reduce_min_sync(0xffffffffu, (uint32_t)(least + 0x8001));   // 0x10000: zeros only
    if (lane == 0) {
      atomicMax(hi + t, top);
      atomicMin(lo + t, low);
    }
  }
}

// A warp's part of a tile in BF16: rows row0 + 8 r + g, and of each kc columns from kb to ke those from
// `first` on, 256 at every `step`, as the kernel's sweeps divide them among warps and with their layout of
// lanes; the sums to out (kMt * NT fragments).  x comes from global memory.
// MXFP4: x as it is.  A placed code times 2^124 is a quarter of its value, times an E8M0 scale that is
// exact in BF16 (2^-130 to 1.5 * 2^127): sums are a quarter of y, in range as far as y is.
// NVFP4: a placed code times its scale and 2^118 is 2^-8 of the weight.  A row of x is multiplied by
// 2^shift, which brings its largest to 2^60: sums of 2^20 terms are finite, and only elements 2^-176 of
// the row's largest meet the end of FP32's range.
// Not inlined, for the same reason as stage_x.
template <int NT, bool kMx>
__device__ __noinline__ void sweep_bf16(const uint16_t* x, const uint8_t* codes, const uint8_t* sf,
                                        int T, int64_t N, int K, int64_t row0, int kb, int ke,
                                        int kc, int first, int step, const int* shift, float* out) {
  using L = LinTile<NT>;
  constexpr int kMt = L::kMt;
  const int g = (threadIdx.x & 31) >> 2, q = threadIdx.x & 3;
  float c[kMt][NT][4];
#pragma unroll
  for (int f = 0; f < L::kFrags * 4; ++f) c[f / (NT * 4)][f / 4 % NT][f % 4] = 0.0f;
  uint32_t xscale[NT];   // 2^shift of this lane's rows of x, in both halves
#pragma unroll
  for (int j = 0; j < NT; ++j)
    xscale[j] = kMx ? 0u : (uint32_t)(shift[min(j * 8 + g, T - 1)] + 127) * 0x00800080u;
  for (int k0 = kb; k0 < ke; k0 += kc)
    for (int k = k0 + first, k1 = min(ke, k0 + kc); k < k1; k += step)
#pragma unroll 1
      for (int h = 0; h < L::kHalves; ++h) {
        const int at = min(k + h * 128 + q * 32, k1 - 32);   // (as in the kernel's load)
        const bool in = k + h * 128 + q * 32 < k1;
        RowCodes w[2 * kMt];
#pragma unroll
        for (int r = 0; r < 2 * kMt; ++r) {
          const int64_t n = min(row0 + r * 8 + g, N - 1);
          w[r].c = __ldg(reinterpret_cast<const uint4*>(codes + n * (K / 2) + (at >> 1)));
          if constexpr (kMx) {
            const uint32_t b = __ldg(sf + n * (K / 32) + at / 32);
            w[r].s = b == 255u ? 0x7FC07FC0u : e8m0_scale_bf16x2(b);
          } else {   // both scales, exact in BF16
            const float2 f = e4m3x2_to_f32x2(
                __ldg(reinterpret_cast<const uint16_t*>(sf + n * (K / 16) + at / 16)));
            const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * 0x1p118f, f.y * 0x1p118f);
            w[r].s = *reinterpret_cast<const uint32_t*>(&b);
          }
        }
        float d[kMt][NT][4];   // (see the kernel's kApart)
#pragma unroll
        for (int f = 0; f < L::kFrags * 4; ++f) d[f / (NT * 4)][f / 4 % NT][f % 4] = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t o[2 * kMt][4];
#pragma unroll
          for (int r = 0; r < 2 * kMt; ++r) {
            e2m1x8_to_bf16x2_scaled_down(w[r].word(i), o[r]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              o[r][e] = kMx ? mul_bf16x2(mul_bf16x2(o[r][e], kBf16x2Pow2_124), w[r].s)
                            : mul_bf16x2(o[r][e], __byte_perm(w[r].s, 0u, (i & 2) ? 0x3232 : 0x1010));
          }
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            if (j * 8 >= T) break;
            const int t = min(j * 8 + g, T - 1);   // (sums of tokens behind T are not stored)
            uint4 xv = in ? __ldg(reinterpret_cast<const uint4*>(x + (int64_t)t * K + at + i * 8))
                          : make_uint4(0u, 0u, 0u, 0u);
            if constexpr (!kMx)
              xv = make_uint4(mul_bf16x2(xv.x, xscale[j]), mul_bf16x2(xv.y, xscale[j]),
                              mul_bf16x2(xv.z, xscale[j]), mul_bf16x2(xv.w, xscale[j]));
#pragma unroll
            for (int m = 0; m < kMt; ++m) {
              mma_bf16(d[m][j], o[2 * m][0], o[2 * m + 1][0], o[2 * m][1], o[2 * m + 1][1], xv.x, xv.y);
              mma_bf16(d[m][j], o[2 * m][2], o[2 * m + 1][2], o[2 * m][3], o[2 * m + 1][3], xv.z, xv.w);
            }
          }
        }
#pragma unroll
        for (int f = 0; f < L::kFrags * 4; ++f)
          c[f / (NT * 4)][f / 4 % NT][f % 4] += d[f / (NT * 4)][f / 4 % NT][f % 4];
      }
#pragma unroll
  for (int f = 0; f < L::kFrags * 4; ++f) out[f] = c[f / (NT * 4)][f / 4 % NT][f % 4];
}

template <int NT, bool kMx, bool kF32>
__global__ void __launch_bounds__(LinTile<NT>::kThreads, LinTile<NT>::kPerSm)
linear_w4_kernel(LinearArgs a) {
  using L = LinTile<NT>;
  constexpr int kMt = L::kMt, kHalves = L::kHalves, kStep = L::kStep;
  constexpr int kBlk = kMx ? 32 : 16;
  constexpr bool kRefill = NT > 1;   // load a part of the next step as soon as this one's is used up
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int s_shift[kLinRows];        // rows of x: the power of two they are times
  __shared__ uint32_t s_bad;               // x is not exact in F16 at the first power of two
  __shared__ uint32_t s_hi[kLinRows], s_lo[kLinRows];   // then: a row's largest and smallest magnitude
  __shared__ float2 s_unscale[kLinRows];   // takes a row's sums to y, in two factors
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int slice = warp % a.ks, group = warp / a.ks, groups = a.warps / a.ks;
  const int rank = (int)blockIdx.x % a.cluster, col = (int)blockIdx.x / a.cluster;
  const int cols = (int)gridDim.x / a.cluster;
  const int stride = a.kc * 2 + 64;
  float4* join = reinterpret_cast<float4*>(smem);   // [warps][kFrags][32], if anything is joined
  const bool joins = a.ks > 1 || a.cluster > 1;
  uint8_t* xs = smem + (joins ? L::kJoinBytes : 0);
  const int64_t tiles = (a.N + L::kRows - 1) / L::kRows;
  const int64_t tile0 = (int64_t)col * groups + group;   // this group's first tile
  const int kb = rank * a.kslice, ke = min(a.K, kb + a.kslice);   // this block's columns
  for (int t = threadIdx.x; t < kLinRows; t += blockDim.x) {   // (blocks of one warp exist)
    s_shift[t] = kF16Top - kTopGuess;
    s_hi[t] = 0u;
    s_lo[t] = 0xFFFFu;
  }
  if (threadIdx.x == 0) s_bad = 0u;
  __syncthreads();
  griddep_wait();
  griddep_launch();

  // x at the first power of two; if an element (in any of the cluster's blocks) is not exact there, at
  // the rows' own; if one is not exact there either, not at all.  x that is too long for shared memory
  // is staged again by chunks.
  const int chunks = (a.kslice + a.kc - 1) / a.kc;
  bool direct = false;   // BF16, x from global memory; the same in all blocks of a cluster
  for (int attempt = 0;; ++attempt) {
    for (int chunk = chunks - 1; chunk >= 0; --chunk)
      stage_x<L::kFly>(a.x, a.T, a.K, kb + chunk * a.kc, a.kc, ke, xs, s_shift, &s_bad);
    __syncthreads();
    if (attempt == 1) break;
    bool fits = s_bad == 0u;
    if (a.cluster > 1) {
      cluster_sync();
      fits = (int)threadIdx.x >= a.cluster || ld_dsmem_u32(&s_bad, threadIdx.x) == 0u;
      fits = __syncthreads_and(fits);
      cluster_sync();   // (the others have read this block's flag)
    }
    if (fits) break;
    find_range(a.x, a.T, a.K, s_hi, s_lo);
    __syncthreads();
    bool exact = true;   // infinities and NaN are
    for (int t = threadIdx.x; t < a.T; t += blockDim.x) {
      const uint32_t hi = s_hi[t];
      const int up = hi == 0u ? 0 : min(kF16Top - bf16_exponent(hi), 127);
      s_shift[t] = up;
      exact = exact && (hi == 0u || bf16_exponent(s_lo[t]) + up >= kF16Exact);
    }
    direct = !__syncthreads_and(exact);
    if (direct) {
      if constexpr (!kMx) {
        for (int t = threadIdx.x; t < a.T; t += blockDim.x)
          s_shift[t] = min(s_shift[t] + kBf16Top - kF16Top, 127);
      }
      break;
    }
  }
  // (the thread that writes a row's shift reads it here)
  for (int t = threadIdx.x; t < kLinRows; t += blockDim.x) {
    float2 u = pow2_factors(-s_shift[t]);   // half on either side of the tensor scale
    if constexpr (!kMx) u.y *= __ldg(a.ts);
    s_unscale[t] = u;
  }
  __syncthreads();

  // A tile's rows 8 r + g; rows behind the last one read it again and are not stored.
  const uint8_t *pc, *ps;
  int off[2 * kMt];
  RowCodes st[kHalves][2 * kMt];
  float c[kMt][NT][4];
  // Part h of the step at column k behind k0: a lane's 32 of each 128 columns, so that a quad's
  // 16-byte loads fill whole sectors.  Columns behind k1 read the row's last 32 again, against
  // zeros of x (a NaN there is the row's anyway).
  auto load = [&](int k0, int k1, int k, int h) {
    const int at = min(k0 + k + q * 32 + h * 128, k1 - 32);
#pragma unroll
    for (int r = 0; r < 2 * kMt; ++r) {
      st[h][r].c = __ldg(reinterpret_cast<const uint4*>(pc + (int64_t)off[r] * (a.K / 2) + (at >> 1)));
      const uint8_t* s = ps + (int64_t)off[r] * (a.K / kBlk) + at / kBlk;
      if constexpr (kMx) st[h][r].s = __ldg(s);
      else st[h][r].s = __ldg(reinterpret_cast<const uint16_t*>(s));
    }
  };
  // Token 8 j + g, unit at byte `at`.  Lanes of tokens behind T read the last token (one column) or
  // the uninitialised end of the last column's rows; they only reach sums that are not stored.
  const uint8_t* xrow = xs + (NT == 1 ? min(g, a.T - 1) : g) * stride + q * 16;
  auto x_frag = [&](int j, int at) {
    return *reinterpret_cast<const uint4*>(xrow + j * 8 * stride + at);
  };
  // Adds columns k0 .. k1 of the tile (x of k0 at the start of shared memory) to c.  Returns
  // whether this lane met a scale that F16 does not hold (kMx), in a block that is not all zeros (those
  // may carry any scale).
  auto sweep = [&](int k0, int k1) {
    bool odd = false;
    // The tensor cores truncate, which a chain of 256 MMAs turns into a bias of 1e-6 of the sum.  One
    // column: the MMAs of four steps sum from zero and are added with rounded FP32 additions.  Two: a
    // second set of accumulators costs 15 to 25%, so the split keeps the chains of FP32 output short.
    constexpr bool kApart = NT == 1;
    float d[kApart ? kMt : 1][kApart ? NT : 1][4];
    auto flush = [&](bool add) {
      if constexpr (kApart) {
#pragma unroll
        for (int m = 0; m < kMt; ++m)
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (add) c[m][j][i] += d[m][j][i];
              d[m][j][i] = 0.0f;
            }
      }
    };
    flush(false);
    int chain = 0;
    if constexpr (kRefill) {
#pragma unroll
      for (int h = 0; h < kHalves; ++h) load(k0, k1, slice * kStep, h);
    }
    for (int k = slice * kStep; k < k1 - k0; k += a.ks * kStep) {
      if constexpr (!kRefill) {
#pragma unroll
        for (int h = 0; h < kHalves; ++h) load(k0, k1, k, h);
      }
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        uint32_t sc[2 * kMt];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t o[2 * kMt][4];
#pragma unroll
          for (int r = 0; r < 2 * kMt; ++r) {
            if (i % (kMx ? 4 : 2) == 0) sc[r] = unit_scale<kMx>(st[h][r].s, i);
            if (kMx && i == 0 && st[h][r].s - (uint32_t)kScaleLow >= (uint32_t)kScaleWindow &&
                st[h][r].s != 255u)
              odd = odd || ((st[h][r].c.x | st[h][r].c.y | st[h][r].c.z | st[h][r].c.w) & 0x77777777u) != 0u;
            decode8(st[h][r].word(i), sc[r], o[r]);
          }
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            if (NT > 1 && j * 8 >= a.T) break;
            const uint4 xv = x_frag(j, k * 2 + h * 256 + i * 64);
#pragma unroll
            for (int m = 0; m < kMt; ++m) {
              float (&sum)[4] = kApart ? d[kApart ? m : 0][kApart ? j : 0] : c[m][j];
              mma_f16(sum, o[2 * m][0], o[2 * m + 1][0], o[2 * m][1], o[2 * m + 1][1], xv.x, xv.y);
              mma_f16(sum, o[2 * m][2], o[2 * m + 1][2], o[2 * m][3], o[2 * m + 1][3], xv.z, xv.w);
            }
          }
        }
        if constexpr (kRefill) load(k0, k1, k + a.ks * kStep, h);
      }
      if (kApart && (++chain & 3) == 0) flush(true);
    }
    flush(true);
    return odd;
  };
  // One sum to y: token 8 j + t8, row r16 of MMA tile m.
  auto store = [&](int64_t tile, int m, int j, int t8, int r16, float v) {
    const int t = j * 8 + t8;
    const int64_t n = tile * L::kRows + m * 16 + r16;
    if (t >= a.T || n >= a.N) return;
    if constexpr (kF32) static_cast<float*>(a.y)[(int64_t)t * a.N + n] = v;
    else static_cast<__nv_bfloat16*>(a.y)[(int64_t)t * a.N + n] = __float2bfloat16_rn(v);
  };
  // One column: no clusters, and further warps only if x is staged once, so they are done.
  if (NT == 1 && warp >= a.warps) return;
  const bool active = NT == 1 || warp < a.warps;
  auto all = [&]() {   // the threads that join a tile
    __syncwarp();
    if (a.cluster > 1) cluster_sync();
    else if (active) asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(a.ks * 32) : "memory");
  };

  for (int it = 0; it < a.iters; ++it) {
    const int64_t tile = active ? tile0 + (int64_t)it * cols * groups : tiles;
    {
      const int64_t row = min(tile * L::kRows + g, a.N - 1);
      pc = a.codes + row * (a.K / 2);
      ps = a.sf + row * (a.K / kBlk);
#pragma unroll
      for (int r = 0; r < 2 * kMt; ++r)
        off[r] = (int)(min(tile * L::kRows + g + r * 8, a.N - 1) - row);
    }
#pragma unroll
    for (int m = 0; m < kMt; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) c[m][j][i] = 0.0f;
    bool odd = false;
    if (!direct) {
#pragma unroll 1
      for (int chunk = 0; chunk < chunks; ++chunk) {
        const int k0 = kb + chunk * a.kc;
        if (chunks > 1 && (it > 0 || chunk > 0)) {   // (the first is there)
          __syncthreads();
          stage_x<L::kFly>(a.x, a.T, a.K, k0, a.kc, ke, xs, s_shift, &s_bad);
          __syncthreads();
        }
        if (tile < tiles) odd = sweep(k0, min(ke, k0 + a.kc)) || odd;
      }
    }
    auto again = [&](float up) {   // this warp's part in BF16, times up
      float sums[L::kFrags * 4];
      sweep_bf16<NT, kMx>(a.x, a.codes, a.sf, a.T, a.N, a.K, tile * L::kRows, kb, ke, a.kc,
                          slice * kStep, a.ks * kStep, s_shift, sums);
#pragma unroll
      for (int f = 0; f < L::kFrags * 4; ++f) c[f / (NT * 4)][f / 4 % NT][f % 4] = sums[f] * up;
    };
    if constexpr (!kMx) {
      if (direct && tile < tiles) again(256.0f);
    }
    // to y's scale: x's powers of two and the tensor scale
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 u = s_unscale[j * 8 + q * 2 + (i & 1)];   // (rows behind T: any)
#pragma unroll
        for (int m = 0; m < kMt; ++m) c[m][j][i] = c[m][j][i] * u.x * u.y;
      }
    if constexpr (kMx) {
      if (direct ? tile < tiles : __any_sync(0xffffffffu, odd)) again(4.0f);
    }
    if (!joins) {
      if (tile < tiles) {
#pragma unroll
        for (int m = 0; m < kMt; ++m)
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              store(tile, m, j, q * 2 + (i & 1), g + (i >> 1) * 8, c[m][j][i]);
      }
      continue;
    }
    if (it > 0) all();   // the readers of what stands there are through
    // fragments go round the cluster's blocks: [block][warp][fragments of a block][lane]
    const int per = L::kFrags / a.cluster;
#pragma unroll
    for (int f = 0; f < L::kFrags; ++f) {
      if (!active) break;
      const float* v = c[f % kMt][f / kMt];
      float4* slot = join + ((rank * a.warps + warp) * per + f / a.cluster) * 32 + lane;
      if (a.cluster > 1) st_dsmem_float4(slot, f % a.cluster, v);
      else *slot = make_float4(v[0], v[1], v[2], v[3]);
    }
    all();
    // this block's sums go round the group's threads, neighbours on neighbouring rows: blocks,
    // then warps in order.  Row r, token t of a fragment: lane (r % 8) * 4 + t / 2, register
    // (r / 8) * 2 + t % 2
    const float* base = reinterpret_cast<const float*>(join + group * a.ks * per * 32);
    for (int e = slice * 32 + lane; active && e < per * 128; e += a.ks * 32) {
      const int r = e & 15, t = (e >> 4) & 7, fl = e >> 7;
      const float* at = base + fl * 128 + (r & 7) * 16 + (t >> 1) * 4 + (r >> 3) * 2 + (t & 1);
      float sum = 0.0f;
      for (int b = 0; b < a.cluster; ++b)
#pragma unroll 4
        for (int w = 0; w < a.ks; ++w) sum += at[(b * a.warps + w) * per * 128];
      const int f = fl * a.cluster + rank;
      if (tile < tiles) store(tile, f % kMt, f / kMt, t, r, sum);
    }
  }
}

// Time of a split in us, from measurements on GB300: a step of a warp takes kStepUs[0], or
// kStepUs[1] for each warp of an SM if its warps are many; a join kJoinUs[0] (warps) or [1]
// (cluster); x comes into shared memory at 16 elements a ns.  A split whose x does not fit is taken
// only if none does: windows of x cost more than the split saves (131072 x 7168 at 12 rows 247 us,
// with a cluster 152).
template <int NT>
struct LinCost {
  static constexpr double kStepUs[2] = {1.1, NT == 1 ? 0.0625 : 0.15};
  static constexpr double kJoinUs[2] = {NT == 1 ? 2.0 : 3.0, 5.0};
};

// Two columns with FP32 output: steps of a warp, at most.  16 are 256 MMAs in one chain, whose truncation
// leaves 1e-6 of y with normal data (32 3e-6, 64 6e-6); BF16 output does not need it.
constexpr int kLinChain = 16;

template <int NT, bool kMx, bool kF32>
cudaError_t launch_linear(LinearArgs a, cudaStream_t s) {
  using L = LinTile<NT>;
  using C = LinCost<NT>;
  auto kern = linear_w4_kernel<NT, kMx, kF32>;
  const int64_t tiles = (a.N + L::kRows - 1) / L::kRows;
  const int64_t steps = (a.K + L::kStep - 1) / L::kStep;
  const int rows = NT == 1 ? a.T : (a.T + 7) / 8 * 8;   // of x in shared memory
  // Columns of x that fit beside the join buffer, with `blocks` blocks an SM.  Two blocks leave L1
  // some 30 KB: with 110 KB each 36864 x 7168 at 7 rows takes 66 us, with one block an SM 41.
  auto fitting = [&](bool joins, int blocks) {
    const int room = (blocks == 2 ? 96 * 1024 : kLinSmem) - (joins ? L::kJoinBytes : 0);
    return (room / rows - 64) / 2 / L::kStep * L::kStep;
  };
  // Clusters of four leave SMs of each GPC idle: on 152 SMs 36 fit (the occupancy query's number).
  auto clusters = [](int cl) { return num_sms() / cl - (cl == 4 ? 2 : 0); };
  // The split of K over cluster blocks and warps, and the blocks an SM, that should finish first.
  double best = 0.0;
  int cols = 1, per_sm = 1;
  const int64_t chain = std::max<int64_t>(kLinChain, (steps + 4 * L::kWarps - 1) / (4 * L::kWarps));
  auto consider = [&](int cl, int ks, int blocks) {
    const bool joins = ks > 1 || cl > 1;
    const int64_t sl = (steps + cl - 1) / cl, groups = L::kWarps / ks;
    if (NT > 1 && kF32 && (sl + ks - 1) / ks > chain) return;
    const int64_t slots = (int64_t)blocks * clusters(cl);
    const int64_t rounds = (tiles + groups * slots - 1) / (groups * slots);
    // no more groups a block than these rounds need: the tiles spread over the SMs
    const int64_t even = (tiles + slots * rounds - 1) / (slots * rounds);
    const int64_t busy = (tiles + even * rounds - 1) / (even * rounds);
    const bool fits = fitting(joins, blocks) >= sl * L::kStep;
    if (!fits && blocks > 1) return;
    const double warps = (double)(busy * cl * even * ks) / num_sms();
    double stage = (double)a.T * sl * L::kStep / 16000.0 * (busy > clusters(cl) ? blocks : 1);
    if (!fits) stage *= 100.0 + (double)rounds;
    const double cost = stage + (cl > 1 ? 1.5 : 0.0) +
                        rounds * ((double)((sl + ks - 1) / ks) *
                                      std::max(C::kStepUs[0], C::kStepUs[1] * warps) +
                                  (cl > 1 ? C::kJoinUs[1] : ks > 1 ? C::kJoinUs[0] : 0.0));
    if (best != 0.0 && cost >= best) return;
    best = cost;
    a.ks = ks;
    a.cluster = cl;
    a.iters = (int)rounds;
    a.kslice = (int)sl * L::kStep;
    a.kc = std::min(a.kslice, fitting(joins, blocks));
    cols = (int)busy;
    per_sm = blocks;
    a.warps = (int)even * ks;
  };
  // (a named barrier for each group: at most 8 of them if ks > 1)
  for (int cl = 1; cl <= L::kFrags && cl <= steps; cl *= 2)
    for (int ks = 1; ks <= L::kWarps; ks *= 2)
      for (int blocks = 1; blocks <= L::kPerSm; ++blocks) consider(cl, ks, blocks);
  const size_t smem = (size_t)rows * (a.kc * 2 + 64) +
                      (a.ks > 1 || a.cluster > 1 ? L::kJoinBytes : 0);
  if (smem > 40 * 1024) {   // always to the most: another thread's launch may need more than this one's
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kLinSmem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(cols * a.cluster));
  // a warp for each of a row's visits of stage_x, up to the block's size
  // (one column: only if it is staged once)
  const int visits = NT == 1 && a.kc < a.kslice ? 1 : a.T * ((a.kc / 8 + L::kFly * 32 - 1) / (L::kFly * 32));
  cfg.blockDim = dim3((unsigned)std::max(a.warps, std::min(visits, L::kWarps)) * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[3];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  // Shared memory for these blocks only, the rest is L1: the codes of a row come in 16-byte loads, and
  // a small L1 loses their lines between them (36864 x 7168 at 8 rows: 68 us where the driver makes
  // room for two blocks, 41 with room for one).  Set with the launch, not with the function, whose
  // other launches (another thread's, a graph's) want other sizes.
  attr[1].id = cudaLaunchAttributePreferredSharedMemoryCarveout;
  attr[1].val.sharedMemCarveout =
      (unsigned)std::min<size_t>(100, (per_sm * (smem + 2048) * 100 + 233471) / 233472);
  attr[2].id = cudaLaunchAttributeClusterDimension;
  attr[2].val.clusterDim.x = (unsigned)a.cluster;
  attr[2].val.clusterDim.y = 1;
  attr[2].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.cluster > 1 ? 3 : 2;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int NT>
cudaError_t launch_linear(const LinearArgs& a, bool mx, bool f32, cudaStream_t s) {
  return mx ? (f32 ? launch_linear<NT, true, true>(a, s) : launch_linear<NT, true, false>(a, s))
            : (f32 ? launch_linear<NT, false, true>(a, s) : launch_linear<NT, false, false>(a, s));
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
  LinearArgs a{};
  a.x = static_cast<const uint16_t*>(x);
  a.codes = codes;
  a.sf = sf;
  a.ts = ts;
  a.T = T;
  a.N = N;
  a.K = (int)K;
  a.y = y;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // One column of tokens while x leaves L1 its room; two, whose blocks split K in a cluster, where
  // it does not and a quarter of K fits (18432 x 16384 at 5 / 6 / 8 rows: 48 / 61 / 73 us and 45;
  // 8192 x 28672 at 3 / 4: 43 / 70 and 40; 8192 x 49152 at 4: 103 and 113).
  const bool one = T == 1 || (T <= 8 && ((int64_t)T * K <= 88 * 1024 || K > 40 * 1024));
  const cudaError_t e = linear_w4_tc_faster(T, N, (int)K)
                            ? launch_linear_w4_tc(x, codes, sf, ts, T, N, (int)K, f32, y, s)
                        : one ? launch_linear<1>(a, mx, f32, s)
                              : launch_linear<2>(a, mx, f32, s);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
