// The router's balance loss and z loss with per-expert counts, and the gradient of the logits.
//
// Over the n tokens that count (mask != 0 and a logit above -infinity), with p the expert
// probabilities of a token - softmax(l), or s / sum(s) with s = sqrt(softplus(l)) for the
// sqrt-softplus router - and lse = log sum exp(l):
//   counts_e = how often e stands in topk_ids,  f_e = counts_e / (n k),  P_e = (1/n) sum_t p_te,
//   balance = E sum_e f_e P_e,   z = (1/n) sum_t lse_t^2.
// The counts are constants of the gradient.  With gb, gz the gradients of the two losses and g_j
// those of the top-k weights w_j (softmax over the k chosen logits, or s / sum of the k chosen s):
//   dl_e = gb (E/n) p_e (f_e - sum_j f_j p_j)                                   (softmax)
//        | gb (E/n) (f_e - sum_j f_j p_j) / sum(s) * ds_e/dl_e                  (sqrt-softplus)
//        + gz (2/n) lse softmax(l)_e
//        + [e = e_j] ( w_j (g_j - sum_i g_i w_i) | (g_j - sum_i g_i w_i) / sum_k(s) * ds/dl ).
// A token that does not count has a zero gradient row.  Everything is FP32: sums of positive terms
// in short chains and trees (FP64 runs at a few instructions a clock here: one double division per
// thread of a block costs it about 5 us).
//
// G lanes of a warp hold one token's row in registers (VPL logits each), so a warp takes 32 / G
// tokens at a time and each row is read once; the next row's loads are issued before the current
// one is reduced.
// Bound by HBM for softmax and many tokens (the logits once, in the backward pass the gradient once),
// by the instruction stream for the sqrt-softplus router (26 instructions a score), by launches and
// the join for small batches.  Measured (device time of a call, 6% of the tokens masked): losses 131072 x
// 256 30.0 us (67% of the copy rate; sqrt-softplus 43.2), 8192 x 256 8.6 us, 64 x 128 3.2 us; gradient
// 131072 x 256 47.2 us (85%; sqrt-softplus 65.6), 100003 x 60 without a mask 13.7 us, 8192 x 256
// sqrt-softplus 6.4 us.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "ops.h"

namespace nvfp4moe {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kJoinCtas = 8;
constexpr int kJoinThreads = 512;

// Expert of logit i of lane `sub` of a G-lane group: VEC consecutive ones per stripe of G * VEC.
template <int G, int VPL, int VEC>
__device__ __forceinline__ int expert_of(int sub, int i) {
  return (i / VEC) * G * VEC + sub * VEC + i % VEC;
}

// What a lane holds of one token: its logits and its first slot's id.
template <int VPL>
struct TokenRow {
  float v[VPL];
  int32_t id;
};

// Whether token t counts as far as the mask (if there is one: MASK) says.
template <bool MASK>
__device__ __forceinline__ bool kept_token(const uint8_t* __restrict__ mask, int64_t t, int64_t T) {
  return t < T && (!MASK || __ldg(mask + t));
}

// Loads of one token's row if it is kept; row: logits + t * E.  Experts behind E, and all of a token
// that is not kept (whose memory is not touched), are -infinity.
template <int G, int VPL, int VEC>
__device__ __forceinline__ void load_row(const float* __restrict__ row,
                                         const int32_t* __restrict__ ids, bool kept, int64_t t,
                                         int E, int k, int sub, TokenRow<VPL>& r) {
  r.id = kept && ids && sub < k ? __ldg(ids + t * k + sub) : -1;
  const int left = kept ? E - sub * VEC : 0;   // experts from this lane's first on
  const float* p = row + sub * VEC;
#pragma unroll
  for (int i = 0; i < VPL; i += VEC) {
    constexpr int kStripe = G * VEC;
    const int o = i / VEC * kStripe;
    if constexpr (VEC == 4) {
      const float4 q = o < left ? __ldg(reinterpret_cast<const float4*>(p + o))
                                : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      r.v[i] = q.x; r.v[i + 1] = q.y; r.v[i + 2] = q.z; r.v[i + 3] = q.w;
    } else {
      r.v[i] = o < left ? __ldg(p + o) : -INFINITY;
    }
  }
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Maximum that keeps a NaN (fmaxf drops it).
__device__ __forceinline__ float nan_max(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
template <int G>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v = nan_max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

__device__ __forceinline__ float ex2(float x) {
  float d;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(x));
  return d;
}
__device__ __forceinline__ float rsqrt_approx(float x) {
  float d;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(x));
  return d;
}
__device__ __forceinline__ float lg2_approx(float x) {
  float d;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(x));
  return d;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float d;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(x));
  return d;
}

// Score s = sqrt(softplus(l)) of the sqrt-softplus router and its slope ds/dl = sigmoid(l)/(2 s),
// from h = e^(-|l|/2) and w = h^2 without a branch or a cancellation:
//   softplus(l) = max(l, 0) + log1p(w),  log1p(w) = w P(w) with P a polynomial on [0, 1];
//   l <= 0: s = h sqrt(P(w)),          slope = h / (2 (1 + w) sqrt(P(w)));
//   l > 0:  s = sqrt(l + w P(w)),      slope = 1 / (2 (1 + w) s).
// P interpolates log1p(w)/w at Chebyshev points of [0, 1] with P(0) = 1: within 2.3 * 2^-24
// relative in FP32.  The library's log1pf(expf(l)) costs about three times the instructions, and
// underflows below l = -103; this score does not before -174.
__device__ __forceinline__ float sqrtsp_score(float l, float& slope) {
  const float h = ex2(fabsf(l) * (-0.5f * kLog2e));
  const float w = h * h;
  float p = -0.004579766187816858f;
  p = fmaf(p, w, 0.025682786479592323f);
  p = fmaf(p, w, -0.06751181185245514f);
  p = fmaf(p, w, 0.11626528203487396f);
  p = fmaf(p, w, -0.15878385305404663f);
  p = fmaf(p, w, 0.19862109422683716f);
  p = fmaf(p, w, -0.2498755156993866f);
  p = fmaf(p, w, 0.3333289325237274f);
  p = fmaf(p, w, -0.4999999701976776f);
  p = fmaf(p, w, 1.0f);
  const float q = l > 0.0f ? fmaf(w, p, l) : p;
  const float root = rsqrt_approx(q) * (l > 0.0f ? 1.0f : h);
  slope = 0.5f * root * rcp_approx(1.0f + w);
  return q * root;
}

struct LossArgs {
  const float* logits;
  const int32_t* ids;
  const uint8_t* mask;
  int64_t T;
  int E, k;
  // partials of block b: probabilities [E], counts [E], then z, n, bad
  float* part_p;
  int32_t* part_c;
  float* part_z;
  int32_t* part_n;
  int32_t* part_bad;
  // outputs
  float* losses;
  int32_t* counts;
  int32_t* tokens;
  float* probs;
  int32_t* status;
};

// One block per SM whose registers hold a row of VPL logits a lane, its successor and the sums: 640
// threads of 96 registers for up to 16 logits a lane, 512 of 128 for 32.  (131072 x 256: 512, 640,
// 768 and 1024 threads take 33.6, 30.6, 29.8 and 31.8 us with softmax, 48.2, 43.1, 44.5 and 49.1
// us with the sqrt-softplus router; 8192 x 256: 7.7, 8.1, 8.5 and 9.5 us.)
template <int VPL>
constexpr int loss_threads() { return VPL <= 16 ? 640 : 512; }

// One block takes every gridDim-th group of rows; its sums go to partials, or, if it is the only
// block, straight to the outputs.
template <int G, int VPL, int VEC, bool SQRTSP, bool MASK>
__global__ void __launch_bounds__(loss_threads<VPL>(), 1) router_loss_kernel(LossArgs a) {
  constexpr int kThreads = loss_threads<VPL>(), kWarps = kThreads / 32;
  constexpr int R = 32 / G;   // rows of a warp at a time
  extern __shared__ float dyn[];
  float* s_p = dyn;                                                     // [warps][E]
  int32_t* s_c = reinterpret_cast<int32_t*>(dyn + kWarps * a.E);         // [E]
  __shared__ float s_z[kWarps];
  __shared__ int32_t s_n[kWarps], s_bad[kWarps];
  __shared__ float s_dot[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % G;
  for (int e = threadIdx.x; e < a.E; e += kThreads) s_c[e] = 0;
  __syncthreads();
  griddep_wait();
  griddep_launch();
  float acc[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) acc[i] = 0.0f;
  float z = 0.0f;
  int32_t n = 0, bad = 0;
  const int64_t step = (int64_t)gridDim.x * kWarps * R;
  int64_t t = ((int64_t)blockIdx.x * kWarps + warp) * R + lane / G;
  const float* row = a.logits + t * a.E;

  auto take = [&](TokenRow<VPL>& r) {
    float top = r.v[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) top = nan_max(top, r.v[i]);
    top = group_max<G>(top);
    float sum = 0.0f, sc = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const float ex = ex2((r.v[i] - top) * kLog2e);
      sum += ex;
      if constexpr (SQRTSP) {
        float slope;
        r.v[i] = sqrtsp_score(r.v[i], slope);
        sc += r.v[i];
      } else {
        r.v[i] = ex;
      }
    }
    sum = group_sum<G>(sum);
    if constexpr (SQRTSP) sc = group_sum<G>(sc);
    else sc = sum;
    if (top != -INFINITY) {   // (also not if the mask took the token out)
      const float lse = fmaf(lg2_approx(sum), kLn2, top);
      z = fmaf(lse, lse, z);   // (the same on the G lanes; one of them is added up)
      ++n;
      const float inv = sc == 0.0f ? 0.0f : rcp_approx(sc);   // scores that all underflowed: 0
#pragma unroll
      for (int i = 0; i < VPL; ++i) acc[i] = fmaf(r.v[i], inv, acc[i]);
      if (sub < a.k) {
        if ((uint32_t)r.id < (uint32_t)a.E) atomicAdd(s_c + r.id, 1);
        else bad = 1;
      }
      for (int j = sub + G; j < a.k; j += G) {
        const int id = __ldg(a.ids + t * a.k + j);
        if ((uint32_t)id < (uint32_t)a.E) atomicAdd(s_c + id, 1);
        else bad = 1;
      }
    }
    t += step;
    row += step * a.E;
  };
  TokenRow<VPL> r0, r1;
  // The mask is read a round ahead of the row whose loads depend on it.
  bool kept = MASK && kept_token<MASK>(a.mask, t, a.T);
  auto load_next = [&](int64_t ahead, TokenRow<VPL>& r) {
    load_row<G, VPL, VEC>(row + ahead * a.E, a.ids, MASK ? kept : t + ahead < a.T, t + ahead, a.E, a.k,
                          sub, r);
    if constexpr (MASK) kept = kept_token<MASK>(a.mask, t + ahead + step, a.T);
  };
  load_next(0, r0);
  while (true) {   // the warp's first row decides: t - lane / G
    if (t - lane / G >= a.T) break;
    load_next(step, r1);
    take(r0);
    if (t - lane / G >= a.T) break;
    load_next(step, r0);
    take(r1);
  }
  if (sub != 0) z = 0.0f, n = 0;
  // rows of one warp, then the warps in order: every sum in a fixed order
#pragma unroll
  for (int i = 0; i < VPL; ++i)
#pragma unroll
    for (int o = G; o < 32; o <<= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    z += __shfl_xor_sync(0xffffffffu, z, o);
    n += __shfl_xor_sync(0xffffffffu, n, o);
    bad |= __shfl_xor_sync(0xffffffffu, bad, o);
  }
  if (lane == 0) {
    s_z[warp] = z;
    s_n[warp] = n;
    s_bad[warp] = bad;
  }
  if (lane < G) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = expert_of<G, VPL, VEC>(sub, i);
      if (e < a.E) s_p[warp * a.E + e] = acc[i];
    }
  }
  __syncthreads();
  z = 0.0f;
  n = bad = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    z += s_z[w];
    n += s_n[w];
    bad |= s_bad[w];
  }
  const bool only = gridDim.x == 1;
  const float inv_n = n > 0 ? 1.0f / (float)n : 0.0f;
  float dot = 0.0f;
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    float p = 0.0f;
#pragma unroll 8
    for (int w = 0; w < kWarps; ++w) p += s_p[w * a.E + e];
    const int32_t c = s_c[e];
    if (only) {
      p *= inv_n;
      a.counts[e] = c;
      a.probs[e] = p;
      dot = fmaf((float)c, p, dot);
    } else {
      a.part_p[(int64_t)blockIdx.x * a.E + e] = p;
      a.part_c[(int64_t)blockIdx.x * a.E + e] = c;
    }
  }
  if (!only) {
    if (threadIdx.x == 0) {
      a.part_z[blockIdx.x] = z;
      a.part_n[blockIdx.x] = n;
      a.part_bad[blockIdx.x] = bad;
    }
    return;
  }
  for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
  if (lane == 0) s_dot[warp] = dot;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kWarps; ++w) dot += s_dot[w];
    a.losses[0] = dot * inv_n * ((float)a.E / (float)a.k);
    a.losses[1] = z * inv_n;
    *a.tokens = n;
    *a.status = bad ? MOE_ERR_INVALID_ARG : MOE_OK;
  }
}

// Joins the blocks' partials in a fixed order: a cluster of kJoinCtas blocks, each with its share
// of the experts, whose warps take 32 experts x every slices-th partial; block 0 then adds the
// blocks' parts of sum_e counts_e P_e through distributed shared memory.
__global__ void __launch_bounds__(kJoinThreads) router_loss_join_kernel(LossArgs a, int nb) {
  constexpr int kWarps = kJoinThreads / 32;
  __shared__ float s_p[kWarps][32];
  __shared__ int32_t s_c[kWarps][32];
  __shared__ float s_dot[4];
  __shared__ float s_part;
  __shared__ float s_z;
  __shared__ int32_t s_n, s_bad;
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = (int)cluster_ctarank();
  const int per = (a.E + kJoinCtas - 1) / kJoinCtas;       // experts of a block, at most 128
  const int chunks = (per + 31) / 32, slices = kWarps / chunks;
  const int chunk = warp % chunks, slice = warp / chunks;
  const int e = rank * per + chunk * 32 + lane;
  const bool mine = chunk * 32 + lane < per && e < a.E;
  float p = 0.0f;
  int32_t c = 0;
  if (mine && slice < slices) {
    for (int b0 = slice; b0 < nb; b0 += 10 * slices) {   // ten partials in flight
      float pv[10];
      int32_t cv[10];
#pragma unroll
      for (int u = 0; u < 10; ++u) {
        const int b = b0 + u * slices;
        pv[u] = b < nb ? __ldcg(a.part_p + (int64_t)b * a.E + e) : 0.0f;
        cv[u] = b < nb ? __ldcg(a.part_c + (int64_t)b * a.E + e) : 0;
      }
#pragma unroll
      for (int u = 0; u < 10; ++u) {
        p += pv[u];
        c += cv[u];
      }
    }
  }
  s_p[warp][lane] = p;
  s_c[warp][lane] = c;
  if (warp == kWarps - 1) {
    float z = 0.0f;
    int32_t n = 0, bad = 0;
    for (int b = lane; b < nb; b += 32) {
      z += __ldcg(a.part_z + b);
      n += __ldcg(a.part_n + b);
      bad |= __ldcg(a.part_bad + b);
    }
    for (int o = 16; o > 0; o >>= 1) {
      z += __shfl_xor_sync(0xffffffffu, z, o);
      n += __shfl_xor_sync(0xffffffffu, n, o);
      bad |= __shfl_xor_sync(0xffffffffu, bad, o);
    }
    if (lane == 0) {
      s_z = z;
      s_n = n;
      s_bad = bad;
    }
  }
  __syncthreads();
  const float inv_n = s_n > 0 ? 1.0f / (float)s_n : 0.0f;
  if (warp < chunks) {   // slice 0: warp == chunk
    for (int q = 1; q < slices; ++q) {
      p += s_p[q * chunks + chunk][lane];
      c += s_c[q * chunks + chunk][lane];
    }
    float dot = 0.0f;
    if (mine) {
      p *= inv_n;
      a.counts[e] = c;
      a.probs[e] = p;
      dot = (float)c * p;
    }
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (lane == 0) s_dot[warp] = dot;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    float d = 0.0f;
    for (int w = 0; w < chunks; ++w) d += s_dot[w];
    s_part = d;
  }
  cluster_sync();
  if (rank == 0 && threadIdx.x == 0) {
    float dot = 0.0f;
    for (int r = 0; r < kJoinCtas; ++r) dot += __uint_as_float(ld_dsmem_u32(&s_part, r));
    a.losses[0] = dot * inv_n * ((float)a.E / (float)a.k);
    a.losses[1] = s_z * inv_n;
    *a.tokens = s_n;
    *a.status = s_bad ? MOE_ERR_INVALID_ARG : MOE_OK;
  }
  cluster_sync();   // block 0 has read the others' shared memory
}

struct LossBwdArgs {
  const float* logits;
  const int32_t* ids;
  const uint8_t* mask;
  int64_t T;
  int E, k;
  const int32_t* counts;
  const int32_t* tokens;
  const float* grad_losses;   // [2] or null
  const float* grad_w;        // [T, k] or null
  float* dlogits;
};

constexpr int kBwdThreads = 256;
constexpr int kBwdWarps = kBwdThreads / 32;
// Blocks per SM: 80 registers a thread hold a softmax row of up to 16 logits a lane and its successor,
// 128 the slopes of the sqrt-softplus scores as well, or 32 logits.  (131072 x 256 softmax: 2, 3
// blocks 54.5, 48.6 us; sqrt-softplus 68.0, 69.1; 32000 x 1021: 71, 89.)
template <int VPL, bool SQRTSP>
constexpr int bwd_blocks() { return VPL <= 16 && !SQRTSP ? 3 : 2; }

template <int G, int VPL, int VEC, bool SQRTSP, bool MASK>
__global__ void __launch_bounds__(kBwdThreads, (bwd_blocks<VPL, SQRTSP>()))
router_loss_backward_kernel(LossBwdArgs a) {
  extern __shared__ float dyn[];
  constexpr int R = 32 / G;
  constexpr int kWidth = G * VPL;                           // E rounded up to the lanes' layout
  float* s_f = dyn;                                         // [kWidth] gb (E / n) f_e
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % G;
  float* s_row = dyn + kWidth * (1 + warp * R + lane / G);  // this token's gradient row
  griddep_wait();
  griddep_launch();
  const int64_t step = (int64_t)gridDim.x * kBwdWarps * R;
  int64_t t = ((int64_t)blockIdx.x * kBwdWarps + warp) * R + lane / G;
  const float* row = a.logits + t * a.E;
  float* out = a.dlogits + t * a.E + sub * VEC;
  const int32_t* ids = a.grad_w ? a.ids : nullptr;
  constexpr bool kAhead = VPL <= 16;   // two rows of 32 logits a lane would spill
  TokenRow<VPL> next;
  bool kept = kAhead && MASK && kept_token<MASK>(a.mask, t, a.T);   // (a round ahead, as above)
  auto load_next = [&](int64_t rows_on) {
    load_row<G, VPL, VEC>(row + rows_on * a.E, ids, MASK ? kept : t + rows_on < a.T, t + rows_on, a.E,
                          a.k, sub, next);
    if constexpr (MASK) kept = kept_token<MASK>(a.mask, t + rows_on + step, a.T);
  };
  if constexpr (kAhead) load_next(0);
  const int32_t n = __ldg(a.tokens);
  const float inv_n = n > 0 ? 1.0f / (float)n : 0.0f;
  const float gb = a.grad_losses ? __ldg(a.grad_losses) : 0.0f;
  const float gz = (a.grad_losses ? __ldg(a.grad_losses + 1) : 0.0f) * 2.0f * inv_n;
  const float fs = gb * inv_n * inv_n * (float)a.E / (float)a.k;
  for (int e = threadIdx.x; e < kWidth; e += kBwdThreads)
    s_f[e] = e < a.E ? fs * (float)__ldg(a.counts + e) : 0.0f;
  __syncthreads();
  auto f_of = [&](int i, float (&f)[VEC]) {   // the VEC shares from logit i on
    if constexpr (VEC == 4) {
      const float4 q = *reinterpret_cast<const float4*>(s_f + expert_of<G, VPL, VEC>(sub, i));
      f[0] = q.x; f[1] = q.y; f[2] = q.z; f[3] = q.w;
    } else {
      f[0] = s_f[expert_of<G, VPL, VEC>(sub, i)];
    }
  };
  while (t - lane / G < a.T) {   // the warp's first row decides
    TokenRow<VPL> r;
    const int64_t ahead = step * a.E;
    if constexpr (kAhead) {
      r = next;
      load_next(step);
    } else {
      load_row<G, VPL, VEC>(row, ids, kept_token<MASK>(a.mask, t, a.T), t, a.E, a.k, sub, r);
      // Without a mask always true: the branch keeps the compiler from moving the arithmetic of the
      // first logits between the loads of the others (32000 x 1024, softmax 51.7 us without it, 48.4
      // with it; sqrt-softplus 64.7 and 61.9).
      kept = MASK || !a.mask || __ldg(a.mask + t);
    }
    // (E, k) slots of the row: the first per lane, with its logit and weight gradient
    float l0 = -INFINITY, g0 = 0.0f;
    if (ids && (uint32_t)r.id < (uint32_t)a.E) {
      l0 = __ldg(row + r.id);
      g0 = __ldg(a.grad_w + t * a.k + sub);
    }
    float top = r.v[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) top = nan_max(top, r.v[i]);
    top = group_max<G>(top);
    // (not if the mask took the token out)
    const bool live = (kAhead || kept) && top != -INFINITY;
    float sum = 0.0f, sc = 0.0f, fp = 0.0f, slope[SQRTSP ? VPL : 1];
#pragma unroll
    for (int i0 = 0; i0 < VPL; i0 += VEC) {
      float f[VEC];
      f_of(i0, f);
#pragma unroll
      for (int c = 0; c < VEC; ++c) {
        const int i = i0 + c;
        const float ex = ex2((r.v[i] - top) * kLog2e);
        sum += ex;
        if constexpr (SQRTSP) {
          const float s = sqrtsp_score(r.v[i], slope[i]);
          sc += s;
          fp = fmaf(f[c], s, fp);
        } else {
          fp = fmaf(f[c], ex, fp);
        }
        r.v[i] = ex;
      }
    }
    sum = group_sum<G>(sum);
    fp = group_sum<G>(fp);
    if constexpr (SQRTSP) sc = group_sum<G>(sc);
    const float inv = rcp_approx(sum);
    const float is = SQRTSP ? (sc == 0.0f ? 0.0f : rcp_approx(sc)) : inv;
    const float zc = gz * fmaf(lg2_approx(sum), kLn2, top) * inv;
    fp *= is;
#pragma unroll
    for (int i0 = 0; i0 < VPL; i0 += VEC) {
      float f[VEC];
      f_of(i0, f);
#pragma unroll
      for (int c = 0; c < VEC; ++c) {
        const int i = i0 + c;
        const float d = SQRTSP ? fmaf(zc, r.v[i], (f[c] - fp) * is * slope[SQRTSP ? i : 0])
                               : r.v[i] * fmaf(is, f[c] - fp, zc);
        r.v[i] = live ? d : 0.0f;
      }
    }
    if (ids) {
      // the top-k weights' own softmax (or normalised scores) over the valid ids
      auto slot = [&](int j, float& l, float& g) {   // slot j >= G of this row
        const int id = live && j < a.k ? __ldg(ids + t * a.k + j) : -1;
        const bool valid = (uint32_t)id < (uint32_t)a.E;
        l = valid ? __ldg(row + id) : -INFINITY;
        g = valid ? __ldg(a.grad_w + t * a.k + j) : 0.0f;
        return valid ? id : -1;
      };
      auto weight = [&](float l, float mx, float& dl) {   // score and its slope by the logit
        if constexpr (SQRTSP) return sqrtsp_score(l, dl);
        const float w = l == -INFINITY ? 0.0f : ex2((l - mx) * kLog2e);
        dl = w;
        return w;
      };
      float mx = l0, l, g, dl0, dl;
      if constexpr (!SQRTSP) {
        for (int j = sub + G; j - sub < a.k; j += G) {
          slot(j, l, g);
          mx = nan_max(mx, l);
        }
        mx = group_max<G>(mx);
      }
      float ws = weight(l0, mx, dl0), wg = ws * g0;
      for (int j = sub + G; j - sub < a.k; j += G) {
        slot(j, l, g);
        const float w = weight(l, mx, dl);
        ws += w;
        wg = fmaf(w, g, wg);
      }
      ws = group_sum<G>(ws);
      wg = group_sum<G>(wg);
      const float iw = ws == 0.0f ? 0.0f : rcp_approx(ws);
      wg *= iw;
#pragma unroll
      for (int i = 0; i < VPL; i += VEC) {
        float* p = s_row + expert_of<G, VPL, VEC>(sub, i);
        if constexpr (VEC == 4)
          *reinterpret_cast<float4*>(p) = make_float4(r.v[i], r.v[i + 1], r.v[i + 2], r.v[i + 3]);
        else
          *p = r.v[i];
      }
      __syncwarp();
      // G slots at a time; where an id stands twice among them, slot by slot, so that it gets both
      // shares in slot order
      int id = live && (uint32_t)r.id < (uint32_t)a.E ? r.id : -1;
      float add = (g0 - wg) * iw * dl0;
      for (int j = sub;;) {
        const bool valid = id >= 0;
        const uint32_t same = __match_any_sync(0xffffffffu, valid ? lane / G * kWidth + id : -1 - lane);
        if (__all_sync(0xffffffffu, (same & (same - 1u)) == 0u)) {
          if (valid) s_row[id] += add;
        } else {
          for (int q = 0; q < G; ++q) {
            if (valid && sub == q) s_row[id] += add;
            __syncwarp();
          }
        }
        __syncwarp();
        j += G;
        if (j - sub >= a.k) break;
        id = slot(j, l, g);
        weight(l, mx, dl);
        add = (g - wg) * iw * dl;
      }
#pragma unroll
      for (int i = 0; i < VPL; i += VEC) {
        const float* p = s_row + expert_of<G, VPL, VEC>(sub, i);
        if constexpr (VEC == 4) {
          const float4 q = *reinterpret_cast<const float4*>(p);
          r.v[i] = q.x; r.v[i + 1] = q.y; r.v[i + 2] = q.z; r.v[i + 3] = q.w;
        } else {
          r.v[i] = *p;
        }
      }
      __syncwarp();
    }
    const int left = t < a.T ? a.E - sub * VEC : 0;
#pragma unroll
    for (int i = 0; i < VPL; i += VEC) {
      const int o = i / VEC * G * VEC;
      if (o >= left) continue;
      if constexpr (VEC == 4)
        *reinterpret_cast<float4*>(out + o) =
            make_float4(r.v[i], r.v[i + 1], r.v[i + 2], r.v[i + 3]);
      else
        out[o] = r.v[i];
    }
    t += step;
    row += ahead;
    out += ahead;
  }
}

// Lanes of one token's row for E experts, and the blocks of the loss kernel.  A batch of at most four
// rounds of one block's warps stays in one block, which then needs no second launch; above, one block
// per SM.
struct LossGrid {
  int lanes, blocks;
  LossGrid(int64_t T, int E) {
    lanes = E <= 64 ? 4 : E <= 128 ? 8 : E <= 256 ? 16 : 32;
    const int64_t round = (E <= 512 ? loss_threads<16>() : loss_threads<32>()) / lanes;
    const int64_t need = (T + round - 1) / round;
    blocks = need <= 4 ? 1 : (int)std::min<int64_t>(need, num_sms());
  }
};

// Calls f with the lane layout for E experts as template arguments.
template <typename F>
cudaError_t with_layout(int E, bool vec, F&& f) {
  using std::integral_constant;
#define NVFP4MOE_LAYOUT(G, VPL)                                                                  \
  (vec ? f(integral_constant<int, G>{}, integral_constant<int, VPL>{},                           \
           integral_constant<int, 4>{})                                                          \
       : f(integral_constant<int, G>{}, integral_constant<int, VPL>{},                           \
           integral_constant<int, 1>{}))
  if (E <= 32) return NVFP4MOE_LAYOUT(4, 8);
  if (E <= 64) return NVFP4MOE_LAYOUT(4, 16);
  if (E <= 128) return NVFP4MOE_LAYOUT(8, 16);
  if (E <= 256) return NVFP4MOE_LAYOUT(16, 16);
  if (E <= 512) return NVFP4MOE_LAYOUT(32, 16);
  return NVFP4MOE_LAYOUT(32, 32);
#undef NVFP4MOE_LAYOUT
}

int check_loss(int32_t T, int32_t E, int32_t k, uint32_t flags) {
  if (T < 0 || E < 1 || k < 1 || k > E) return MOE_ERR_INVALID_ARG;
  if (flags & ~MOE_FLAG_ROUTER_SQRTSOFTPLUS) return MOE_ERR_INVALID_ARG;
  if (E > 1024 || k > 32) return MOE_ERR_UNSUPPORTED_SHAPE;
  if ((int64_t)T * k > INT32_MAX) return MOE_ERR_UNSUPPORTED_SHAPE;   // counts are 32 bits
  return MOE_OK;
}

}  // namespace
}  // namespace nvfp4moe

using namespace nvfp4moe;

extern "C" {

size_t moe_router_loss_workspace_size(int32_t T, int32_t E) {
  if (T < 0 || E < 1) return 0;
  const size_t nb = (size_t)LossGrid(T, E).blocks;
  return kAlign + 2 * align_up(4 * nb * (size_t)E) + 3 * align_up(4 * nb);
}

int moe_router_loss(const float* logits, const int32_t* topk_ids, const uint8_t* mask, int32_t T,
                    int32_t E, int32_t k, uint32_t flags, float* losses, int32_t* counts,
                    int32_t* tokens, float* probs, void* workspace, size_t ws_bytes,
                    moe_stream_t stream) {
  const int st = check_loss(T, E, k, flags);
  if (st != MOE_OK) return st;
  if (!losses || !counts || !tokens || !probs) return MOE_ERR_INVALID_ARG;
  if (!workspace || ws_bytes < moe_router_loss_workspace_size(T, E))
    return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (!is_aligned(workspace, kAlign)) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!logits || !topk_ids)) return MOE_ERR_INVALID_ARG;
  for (const void* p : {(const void*)logits, (const void*)topk_ids, (const void*)losses,
                        (const void*)counts, (const void*)tokens, (const void*)probs})
    if (!is_aligned(p, 4)) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const LossGrid lg(T, E);
  const int nb = lg.blocks;
  uint8_t* w8 = static_cast<uint8_t*>(workspace);
  LossArgs a{};
  a.logits = logits;
  a.ids = topk_ids;
  a.mask = mask;
  a.T = T;
  a.E = E;
  a.k = k;
  size_t o = kAlign;
  a.part_p = reinterpret_cast<float*>(w8 + o);
  o += align_up(4 * (size_t)nb * E);
  a.part_c = reinterpret_cast<int32_t*>(w8 + o);
  o += align_up(4 * (size_t)nb * E);
  a.part_z = reinterpret_cast<float*>(w8 + o);
  o += align_up(4 * (size_t)nb);
  a.part_n = reinterpret_cast<int32_t*>(w8 + o);
  o += align_up(4 * (size_t)nb);
  a.part_bad = reinterpret_cast<int32_t*>(w8 + o);
  const bool vec = E % 4 == 0 && is_aligned(logits, 16);
  const bool sp = (flags & MOE_FLAG_ROUTER_SQRTSOFTPLUS) != 0u;
  a.losses = losses;
  a.counts = counts;
  a.tokens = tokens;
  a.probs = probs;
  a.status = reinterpret_cast<int32_t*>(workspace);
  cudaError_t e = with_layout(E, vec, [&](auto g, auto vpl, auto v) {
    constexpr int G = decltype(g)::value, VPL = decltype(vpl)::value, VEC = decltype(v)::value;
    auto kern = sp ? (mask ? router_loss_kernel<G, VPL, VEC, true, true>
                           : router_loss_kernel<G, VPL, VEC, true, false>)
                   : (mask ? router_loss_kernel<G, VPL, VEC, false, true>
                           : router_loss_kernel<G, VPL, VEC, false, false>);
    constexpr int threads = loss_threads<VPL>();
    const size_t smem = 4 * (size_t)E * (threads / 32 + 1);
    // 48 KB hold the kernel's own few hundred bytes too.  (Always to the layout's most: another
    // thread's launch may need more.)
    if (smem > 40 * 1024) {
      const cudaError_t ea = cudaFuncSetAttribute(
          kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * G * VPL * (threads / 32 + 1));
      if (ea != cudaSuccess) return ea;
    }
    return launch_pdl(kern, dim3(nb), dim3(threads), smem, s, a);
  });
  if (e == cudaSuccess && nb > 1) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kJoinCtas);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kJoinCtas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, router_loss_join_kernel, a, nb);
  }
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int moe_router_loss_backward(const float* logits, const int32_t* topk_ids, const uint8_t* mask,
                             int32_t T, int32_t E, int32_t k, uint32_t flags,
                             const int32_t* counts, const int32_t* tokens,
                             const float* grad_losses, const float* grad_topk_w, float* dlogits,
                             moe_stream_t stream) {
  const int st = check_loss(T, E, k, flags);
  if (st != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  if (!logits || !counts || !tokens || !dlogits || (grad_topk_w && !topk_ids))
    return MOE_ERR_INVALID_ARG;
  for (const void* p : {(const void*)logits, (const void*)topk_ids, (const void*)counts,
                        (const void*)tokens, (const void*)grad_losses, (const void*)grad_topk_w,
                        (const void*)dlogits})
    if (!is_aligned(p, 4)) return MOE_ERR_INVALID_ARG;
  LossBwdArgs a{logits, topk_ids, mask, T, E, k, counts, tokens, grad_losses, grad_topk_w, dlogits};
  const bool vec = E % 4 == 0 && is_aligned(logits, 16) && is_aligned(dlogits, 16);
  const bool sp = (flags & MOE_FLAG_ROUTER_SQRTSOFTPLUS) != 0u;
  const cudaError_t e = with_layout(E, vec, [&](auto g, auto vpl, auto v) {
    constexpr int G = decltype(g)::value, VPL = decltype(vpl)::value, VEC = decltype(v)::value;
    auto kern = sp ? (mask ? router_loss_backward_kernel<G, VPL, VEC, true, true>
                           : router_loss_backward_kernel<G, VPL, VEC, true, false>)
                   : (mask ? router_loss_backward_kernel<G, VPL, VEC, false, true>
                           : router_loss_backward_kernel<G, VPL, VEC, false, false>);
    constexpr int rows = kBwdWarps * (32 / G), width = G * VPL;
    const int64_t most = (int64_t)(sp ? bwd_blocks<VPL, true>() : bwd_blocks<VPL, false>()) * num_sms();
    const int nb = (int)std::min<int64_t>(((int64_t)T + rows - 1) / rows, most);
    return launch_pdl(kern, dim3(nb), dim3(kBwdThreads), 4 * (size_t)width * (1 + rows),
                      reinterpret_cast<cudaStream_t>(stream), a);
  });
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
