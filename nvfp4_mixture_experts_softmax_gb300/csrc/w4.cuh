// Decoding of 4-bit weights to BF16 in registers, shared by the dequantising GEMM and the 4-bit
// matrix-vector product.
#pragma once
#include "common.cuh"

namespace nvfp4moe {

// Eight E2M1 codes (a 32-bit word, the first code in the low nibble) as four BF16x2 words of
// their values times 2^-126, by placing bits: a code's three magnitude bits (e1 e0 m) become the
// two lowest exponent bits and the top mantissa bit of a BF16, its sign bit the sign.  With
// e1 e0 = 0 that is the subnormal m * 2^-127 = (m / 2) * 2^-126, otherwise
// 2^(e - 127) * (1 + m / 2) = 2^(e - 1) * (1 + m / 2) * 2^-126: E2M1's own definition, scaled.
// Word i holds codes 2i (low half) and 2i+1 (high half).
__device__ __forceinline__ void e2m1x8_to_bf16x2_scaled_down(uint32_t w, uint32_t (&o)[4]) {
  const uint32_t ev = w & 0x0F0F0F0Fu;          // codes 0, 2, 4, 6: the low nibble of each byte
  const uint32_t od = (w >> 4) & 0x0F0F0F0Fu;   // codes 1, 3, 5, 7
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // byte 0 <- byte i of ev, byte 2 <- byte i of od, bytes 1 and 3 <- the sign of ev's byte 0
    // (selector 8), which is clear: code 2i in bits 0-3 and code 2i+1 in bits 16-19
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;"
        : "=r"(r)
        : "r"(ev), "r"(od), "r"(0x8080u | (uint32_t)i | ((uint32_t)(4 + i) << 8)));
    // magnitude to bits 6-8 (x 2^6) and sign to bit 15 (x 2^12) of each half; the two shifted
    // copies occupy disjoint bits, so the sum is their union
    o[i] = (r * 4160u) & 0x81C081C0u;
  }
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

constexpr uint32_t kBf16x2Pow2_126 = 0x7E807E80u;   // 2^126 in both halves
constexpr uint32_t kBf16x2Pow2_124 = 0x7D807D80u;   // 2^124 in both halves
constexpr uint32_t kBf16x2Pow2_120 = 0x7B807B80u;   // 2^120 in both halves

constexpr uint32_t kBf16x2Pow2_118 = 0x7A807A80u;   // 2^118 in both halves

// An E4M3 block scale times 2^118 as BF16x2 (exact; at most 448 * 2^118 < 2^127): its seven
// magnitude bits shifted to the top of a BF16's exponent-and-mantissa field are the scale times
// 2^-120 (subnormal E4M3 to subnormal BF16 likewise), then two multiplications by powers of two.
// Times an E2M1 value placed at 2^-126 this gives the product times 2^-8, at least 2^-19: a
// normal BF16, exact, and only a power of two away from the decoded weight.
__device__ __forceinline__ uint32_t e4m3_scale_x2118_bf16x2(uint32_t b) {
  const uint32_t h = ((b & 0x7Fu) << 4) | ((b & 0x80u) << 8);
  return mul_bf16x2(mul_bf16x2(h | (h << 16), kBf16x2Pow2_120), kBf16x2Pow2_118);
}

// An E8M0 block scale 2^(b - 127) as BF16x2: the byte is the BF16 exponent field (b = 0: the
// subnormal 2^-127).
__device__ __forceinline__ uint32_t e8m0_scale_bf16x2(uint32_t b) {
  const uint32_t h = b ? (b << 7) : 0x40u;
  return h | (h << 16);
}

}  // namespace nvfp4moe
