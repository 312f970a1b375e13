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
// A token that does not count has a zero gradient row.
//
// G lanes of a warp hold one token's row in registers (VPL logits each), so a warp takes 32 / G
// tokens at a time and the row is read once.
#include <algorithm>
#include <cfloat>

#include "common.cuh"
#include "ops.h"

namespace nvfp4moe {

namespace {

constexpr int kLossThreads = 256;
constexpr int kLossWarps = kLossThreads / 32;

// Logits of one row held by a lane: VEC consecutive ones, then the next VEC 32-lane stripe.
template <int G, int VPL, int VEC>
__device__ __forceinline__ int expert_of(int sub, int i) {
  return (i / VEC) * G * VEC + sub * VEC + i % VEC;
}

template <int G, int VPL, int VEC>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int E, int sub, bool live,
                                         float (&v)[VPL]) {
#pragma unroll
  for (int i = 0; i < VPL; i += VEC) {
    const int e = expert_of<G, VPL, VEC>(sub, i);
    if constexpr (VEC == 4) {
      const float4 q = live && e < E ? __ldg(reinterpret_cast<const float4*>(row + e))
                                     : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      v[i] = q.x; v[i + 1] = q.y; v[i + 2] = q.z; v[i + 3] = q.w;
    } else {
      v[i] = live && e < E ? __ldg(row + e) : -INFINITY;
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

// s = sqrt(softplus(l)) with softplus(l) = l above 20.  Below -15, softplus(l) = e^l (1 - e^l/2
// + ...) is e^l to 2^-22, so s = e^(l/2), which does not underflow before l = -174.
__device__ __forceinline__ float sqrtsp_score(float l) {
  if (l < -15.0f) return expf(0.5f * l);
  return sqrtf(l > 20.0f ? l : log1pf(expf(l)));
}
// ds/dl = sigmoid(l) / (2 s); s / 2 far below zero.
__device__ __forceinline__ float sqrtsp_slope(float l, float s) {
  if (l < -15.0f) return 0.5f * s;
  return 0.5f / ((1.0f + expf(-l)) * s);
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
};

template <int G, int VPL, int VEC, bool SQRTSP>
__global__ void __launch_bounds__(kLossThreads) router_loss_kernel(LossArgs a) {
  extern __shared__ float dyn[];
  float* s_p = dyn;                                            // [E]
  int32_t* s_c = reinterpret_cast<int32_t*>(dyn + a.E);         // [E]
  __shared__ float s_z[kLossWarps];
  __shared__ int32_t s_n[kLossWarps], s_bad[kLossWarps];
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % G;
  for (int e = threadIdx.x; e < a.E; e += kLossThreads) {
    s_p[e] = 0.0f;
    s_c[e] = 0;
  }
  __syncthreads();
  constexpr int R = 32 / G;   // rows of a warp at a time
  float acc[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) acc[i] = 0.0f;
  float z = 0.0f;
  int32_t n = 0, bad = 0;
  const int64_t step = (int64_t)gridDim.x * kLossWarps * R;
  for (int64_t t0 = ((int64_t)blockIdx.x * kLossWarps + warp) * R; t0 < a.T; t0 += step) {
    const int64_t t = t0 + lane / G;
    bool live = t < a.T && (!a.mask || a.mask[t]);
    float v[VPL];
    load_row<G, VPL, VEC>(a.logits + t * a.E, a.E, sub, live, v);
    float top = v[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) top = nan_max(top, v[i]);
    top = group_max<G>(top);
    live = live && top != -INFINITY;
    float sum = 0.0f, sc = 0.0f, ex[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      ex[i] = expf(v[i] - top);
      sum += ex[i];
    }
    sum = group_sum<G>(sum);
    if constexpr (SQRTSP) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        ex[i] = sqrtsp_score(v[i]);
        sc += ex[i];
      }
      sc = group_sum<G>(sc);
    } else {
      sc = sum;
    }
    if (live) {
      const float lse = top + logf(sum);
      if (sub == 0) {
        z = fmaf(lse, lse, z);
        ++n;
      }
      const float inv = sc == 0.0f ? 0.0f : 1.0f / sc;   // scores that all underflowed: no share
#pragma unroll
      for (int i = 0; i < VPL; ++i) acc[i] = fmaf(ex[i], inv, acc[i]);
      for (int j = sub; j < a.k; j += G) {
        const int id = __ldg(a.ids + t * a.k + j);
        if ((uint32_t)id < (uint32_t)a.E) atomicAdd(s_c + id, 1);
        else bad = 1;
      }
    }
  }
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
  for (int w = 0; w < kLossWarps; ++w) {
    if (warp == w && lane < G) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int e = expert_of<G, VPL, VEC>(sub, i);
        if (e < a.E) s_p[e] += acc[i];
      }
    }
    __syncthreads();
  }
  for (int e = threadIdx.x; e < a.E; e += kLossThreads) {
    a.part_p[(int64_t)blockIdx.x * a.E + e] = s_p[e];
    a.part_c[(int64_t)blockIdx.x * a.E + e] = s_c[e];
  }
  if (threadIdx.x == 0) {
    for (int w = 1; w < kLossWarps; ++w) {
      s_z[0] += s_z[w];
      s_n[0] += s_n[w];
      s_bad[0] |= s_bad[w];
    }
    a.part_z[blockIdx.x] = s_z[0];
    a.part_n[blockIdx.x] = s_n[0];
    a.part_bad[blockIdx.x] = s_bad[0];
  }
}

// One block joins the blocks' partials in their order.
__global__ void __launch_bounds__(1024) router_loss_join_kernel(
    LossArgs a, int nb, float* __restrict__ losses, int32_t* __restrict__ counts,
    int32_t* __restrict__ tokens, float* __restrict__ probs, int32_t* status) {
  __shared__ double s_sum[32];
  __shared__ double s_z;
  __shared__ int32_t s_n, s_bad;
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (warp == 0) {
    double z = 0.0;
    int32_t n = 0, bad = 0;
    for (int b = lane; b < nb; b += 32) {
      z += (double)__ldcg(a.part_z + b);
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
  const double inv_n = s_n > 0 ? 1.0 / (double)s_n : 0.0;
  double dot = 0.0;
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
    double p = 0.0;
    int32_t c = 0;
    for (int b = 0; b < nb; ++b) {
      p += (double)__ldcg(a.part_p + (int64_t)b * a.E + e);
      c += __ldcg(a.part_c + (int64_t)b * a.E + e);
    }
    p *= inv_n;
    counts[e] = c;
    probs[e] = (float)p;
    dot += (double)c * p;
  }
  for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
  if (lane == 0) s_sum[warp] = dot;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < (int)(blockDim.x >> 5); ++w) dot += s_sum[w];
    losses[0] = (float)(dot * inv_n / a.k * a.E);
    losses[1] = (float)(s_z * inv_n);
    *tokens = s_n;
    *status = s_bad ? MOE_ERR_INVALID_ARG : MOE_OK;
  }
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

template <int G, int VPL, int VEC, bool SQRTSP>
__global__ void __launch_bounds__(kLossThreads) router_loss_backward_kernel(LossBwdArgs a) {
  extern __shared__ float dyn[];
  constexpr int R = 32 / G;
  float* s_f = dyn;                                       // [E] f_e * gb * E / n
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % G;
  float* s_row = dyn + a.E + (warp * R + lane / G) * a.E;   // this token's gradient row
  griddep_wait();
  griddep_launch();
  const int32_t n = __ldg(a.tokens);
  const float inv_n = n > 0 ? 1.0f / (float)n : 0.0f;
  const float gb = a.grad_losses ? __ldg(a.grad_losses) : 0.0f;
  const float gz = (a.grad_losses ? __ldg(a.grad_losses + 1) : 0.0f) * 2.0f * inv_n;
  const float fs = gb * inv_n * inv_n * (float)a.E / (float)a.k;
  for (int e = threadIdx.x; e < a.E; e += kLossThreads) s_f[e] = fs * (float)__ldg(a.counts + e);
  __syncthreads();
  float f[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = expert_of<G, VPL, VEC>(sub, i);
    f[i] = e < a.E ? s_f[e] : 0.0f;
  }
  const int64_t step = (int64_t)gridDim.x * kLossWarps * R;
  for (int64_t t0 = ((int64_t)blockIdx.x * kLossWarps + warp) * R; t0 < a.T; t0 += step) {
    const int64_t t = t0 + lane / G;
    bool live = t < a.T && (!a.mask || a.mask[t]);
    float v[VPL], ex[VPL];
    const float* row = a.logits + t * a.E;
    load_row<G, VPL, VEC>(row, a.E, sub, live, v);
    float top = v[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) top = nan_max(top, v[i]);
    top = group_max<G>(top);
    live = live && top != -INFINITY;
    float sum = 0.0f, sc = 0.0f, fp = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      ex[i] = expf(v[i] - top);
      sum += ex[i];
      if constexpr (SQRTSP) {
        const float s = sqrtsp_score(v[i]);
        sc += s;
        fp = fmaf(f[i], s, fp);
      } else {
        fp = fmaf(f[i], ex[i], fp);
      }
    }
    sum = group_sum<G>(sum);
    fp = group_sum<G>(fp);
    if constexpr (SQRTSP) sc = group_sum<G>(sc);
    const float inv = 1.0f / sum;
    const float zc = gz * (top + logf(sum)) * inv;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      float d;
      if constexpr (SQRTSP) {
        const float s = sqrtsp_score(v[i]);
        const float is = sc == 0.0f ? 0.0f : 1.0f / sc;
        d = zc * ex[i] + (s == 0.0f ? 0.0f : (f[i] - fp * is) * is * sqrtsp_slope(v[i], s));
      } else {
        d = ex[i] * (zc + inv * (f[i] - fp * inv));
      }
      const int e = expert_of<G, VPL, VEC>(sub, i);
      if (e < a.E) s_row[e] = live ? d : 0.0f;
    }
    __syncwarp();
    if (a.grad_w) {
      // the top-k weights' own softmax (or normalised scores) over the valid ids
      float mx = -INFINITY;
      for (int j = sub; j < a.k; j += G) {
        const int id = live ? __ldg(a.ids + t * a.k + j) : -1;
        if ((uint32_t)id < (uint32_t)a.E) mx = nan_max(mx, __ldg(row + id));
      }
      mx = group_max<G>(mx);
      float ws = 0.0f, wg = 0.0f;
      for (int j = sub; j < a.k; j += G) {
        const int id = live ? __ldg(a.ids + t * a.k + j) : -1;
        if ((uint32_t)id >= (uint32_t)a.E) continue;
        const float l = __ldg(row + id);
        const float s = SQRTSP ? sqrtsp_score(l) : expf(l - mx);
        ws += s;
        wg = fmaf(s, __ldg(a.grad_w + t * a.k + j), wg);
      }
      ws = group_sum<G>(ws);
      wg = group_sum<G>(wg);
      const float iw = ws == 0.0f ? 0.0f : 1.0f / ws;
      // slot by slot, so that an id that stands twice in a row gets both shares in slot order
      for (int j = 0; j < a.k; ++j) {
        if (sub == j % G && live) {
          const int id = __ldg(a.ids + t * a.k + j);
          if ((uint32_t)id < (uint32_t)a.E) {
            const float l = __ldg(row + id);
            const float g = __ldg(a.grad_w + t * a.k + j) - wg * iw;
            if constexpr (SQRTSP) {
              const float s = sqrtsp_score(l);
              if (s != 0.0f) s_row[id] += g * iw * sqrtsp_slope(l, s);
            } else if (l != -INFINITY) {
              s_row[id] += expf(l - mx) * iw * g;
            }
          }
        }
        __syncwarp();
      }
    }
    if (t < a.T) {
#pragma unroll
      for (int i = 0; i < VPL; i += VEC) {
        const int e = expert_of<G, VPL, VEC>(sub, i);
        if (e >= a.E) continue;
        if constexpr (VEC == 4)
          *reinterpret_cast<float4*>(a.dlogits + t * a.E + e) =
              *reinterpret_cast<const float4*>(s_row + e);
        else
          a.dlogits[t * a.E + e] = s_row[e];
      }
    }
    __syncwarp();
  }
}

int loss_blocks(int64_t T) {
  // whole waves of two blocks per SM; a small batch takes a block per eight tokens
  return (int)std::min<int64_t>(std::max<int64_t>((T + kLossWarps - 1) / kLossWarps, 1),
                                2 * (int64_t)num_sms());
}

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
  if (E <= 64) return NVFP4MOE_LAYOUT(8, 8);
  if (E <= 128) return NVFP4MOE_LAYOUT(16, 8);
  if (E <= 256) return NVFP4MOE_LAYOUT(32, 8);
  if (E <= 512) return NVFP4MOE_LAYOUT(32, 16);
  return NVFP4MOE_LAYOUT(32, 32);
#undef NVFP4MOE_LAYOUT
}

int check_loss(int32_t T, int32_t E, int32_t k, uint32_t flags) {
  if (T < 0 || E < 1 || k < 1 || k > E) return MOE_ERR_INVALID_ARG;
  if (flags & ~MOE_FLAG_ROUTER_SQRTSOFTPLUS) return MOE_ERR_INVALID_ARG;
  if (E > 1024 || k > 32) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

}  // namespace
}  // namespace nvfp4moe

using namespace nvfp4moe;

extern "C" {

size_t moe_router_loss_workspace_size(int32_t T, int32_t E) {
  if (T < 0 || E < 1) return 0;
  const size_t nb = (size_t)loss_blocks(T);
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
  const int nb = loss_blocks(T);
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
  cudaError_t e = with_layout(E, vec, [&](auto g, auto vpl, auto v) {
    auto kern = sp ? router_loss_kernel<decltype(g)::value, decltype(vpl)::value,
                                        decltype(v)::value, true>
                   : router_loss_kernel<decltype(g)::value, decltype(vpl)::value,
                                        decltype(v)::value, false>;
    return launch_pdl(kern, dim3(nb), dim3(kLossThreads), 8 * (size_t)E, s, a);
  });
  if (e == cudaSuccess)
    e = launch_pdl(router_loss_join_kernel, dim3(1), dim3(1024), 0, s, a, nb, losses, counts,
                   tokens, probs, reinterpret_cast<int32_t*>(workspace));
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
    constexpr int G = decltype(g)::value;
    auto kern = sp ? router_loss_backward_kernel<G, decltype(vpl)::value, decltype(v)::value, true>
                   : router_loss_backward_kernel<G, decltype(vpl)::value, decltype(v)::value,
                                                 false>;
    const int rows = kLossWarps * (32 / G);
    const int nb = (int)std::min<int64_t>(((int64_t)T + rows - 1) / rows, 4 * (int64_t)num_sms());
    return launch_pdl(kern, dim3(nb), dim3(kLossThreads), 4 * (size_t)E * (1 + rows), (cudaStream_t)stream, a);
  });
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
