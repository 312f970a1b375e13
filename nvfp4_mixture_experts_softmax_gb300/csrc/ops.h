// What the operators around the layer (norm_mx.cu, router_loss.cu, linear_w4.cu) share, and the
// launcher of the W4A8 layer's entry for already quantised activations.
#pragma once
#include "internal.h"

namespace nvfp4moe {

inline bool is_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// MXFP8 rows (codes [T, H], E8M0 scales [T, H/32]) decoded to BF16 (exact: 4 significant bits
// times a power of two) into every expert row of each token (xb_perm [Rt, H]); a value that is
// not finite raises MOE_ERR_NONFINITE.
cudaError_t launch_mx_decode_perm(const uint8_t* codes, const uint8_t* sf, int T, int H, int k,
                                  int shared, int Rt, const int32_t* inv, void* xb_perm,
                                  int32_t* status, cudaStream_t s);

// The 4-bit matrix-vector product for many rows of x (linear_w4_tc.cu), whether it is the faster one,
// and its launch; ts null: MXFP4.
bool linear_w4_tc_faster(int T, int64_t N, int K);
cudaError_t launch_linear_w4_tc(const void* x, const uint8_t* codes, const uint8_t* sf,
                                const float* ts, int T, int64_t N, int K, bool f32, void* y,
                                cudaStream_t s);

}  // namespace nvfp4moe
