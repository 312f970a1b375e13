// Tokens sorted by expert, their rows brought into that order and back, and the gradients.
//
// sort: of the T * k assignments a = t * k + j those that count (token not masked, id in [0, E)) are
// ordered by expert, ties by a: counts, offsets, perm_src (row -> token) and inv (a -> row, -1 for one
// that does not count).  A block takes a chunk of consecutive assignments, a warp 128 of them in
// order; an assignment's rank inside the warp is the number of earlier ones with the same id (a
// warp match a group of 32, a counter in shared memory between groups), and exclusive sums over the
// warps and over the chunks (the plan's scan kernel) make it the row.  Up to 4096 assignments one block of 32
// warps does it all; beyond, chunks of 8 warps keep all SMs at work (262144 assignments: 3.5 us less than 64
// blocks of 32 warps).
//
// permute:          rows[inv[t,j]] = x[t]          its gradient: combine without weights
// combine:          y[t] = sum_j w[t,j] rows[inv[t,j]], FP32 in slot order, rounded once
// combine backward: drows[inv[t,j]] = w[t,j] dy[t],  dw[t,j] = <dy[t], rows[inv[t,j]]>
// All three are traffic alone: a row is read once for its k copies, k rows for one sum, and the backward
// pass makes one pass over the rows for both gradients.  Device times: sort and permute of 32768 x 2048 to 8 experts each
// 189 us (89% of the copy rate; the sort 15 us of it: three launches that each wait for the one before), combine
// 8192 x 7168 from 8 165 us (94%), FP32 307 us (the copy rate), combine backward 16384 x 4096 from 4 165 us, FP32 327 us (the copy
// rate); one token of 2048: sort and permute
// 4.1 us; 64 x 7168 combined 2.8 us.
#include "common.cuh"
#include "ops.h"
#include "route.cuh"
#include "rows.cuh"

namespace nvfp4moe {

namespace {

constexpr int kPerWarp = 128;                 // assignments of a warp, in groups of 32
constexpr int kOneWarps = 32;                 // of the only block
constexpr int kChunkWarps = 8;                // of one of many
constexpr int kChunk = kChunkWarps * kPerWarp;

// Expert of assignment a, or -1 if it does not count; an id that is neither an expert nor -1 raises
// the status.  A masked token's ids are not read.
__device__ __forceinline__ int expert_of(const int32_t* __restrict__ ids,
                                         const uint8_t* __restrict__ mask, int64_t a, int64_t R, int k,
                                         int E, int32_t* status) {
  if (a >= R) return -1;
  if (mask && mask[(uint32_t)a / (uint32_t)k] == 0) return -1;
  const int e = __ldg(ids + a);
  if ((unsigned)e < (unsigned)E) return e;
  if (e != -1) set_status(status, MOE_ERR_INVALID_ARG);
  return -1;
}

// Histogram of a chunk; block 0 also clears the scan's block count.
__global__ void __launch_bounds__(kChunkWarps * 32) sort_count_kernel(
    const int32_t* __restrict__ ids, const uint8_t* __restrict__ mask, int64_t R, int k, int E,
    int32_t* __restrict__ hist, int32_t* __restrict__ scan_count, int32_t* status) {
  __shared__ int32_t s_cnt[1024];
  for (int e = threadIdx.x; e < E; e += blockDim.x) s_cnt[e] = 0;
  griddep_wait();
  griddep_launch();
  if (blockIdx.x == 0 && threadIdx.x == 0) *scan_count = 0;
  __syncthreads();
  const int64_t a0 = (int64_t)blockIdx.x * kChunk + threadIdx.x;
#pragma unroll
  for (int i = 0; i < kChunk / (kChunkWarps * 32); ++i) {
    const int e = expert_of(ids, mask, a0 + i * kChunkWarps * 32, R, k, E, status);
    if (e >= 0) atomicAdd(&s_cnt[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) hist[(int64_t)blockIdx.x * E + e] = s_cnt[e];
}

// kWarps warps a block; kOne: the only block, which also sums the counts.  Dynamic shared memory: kWarps * E uint16.
template <int kWarps, bool kOne>
__global__ void __launch_bounds__(kWarps * 32) sort_place_kernel(
    const int32_t* __restrict__ ids, const uint8_t* __restrict__ mask, int64_t R, int k, int E,
    const int32_t* __restrict__ base, int32_t* __restrict__ counts, int32_t* __restrict__ offsets,
    int32_t* __restrict__ perm_src, int32_t* __restrict__ inv, int32_t* status) {
  extern __shared__ __align__(16) uint16_t s_rank[];   // [warp][E]: counts, then exclusive sums over the warps
  __shared__ int32_t s_base[1024];
  __shared__ int32_t s_scan[32];
  __shared__ int32_t s_total;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < (kWarps * E + 1) / 2; i += blockDim.x)
    reinterpret_cast<uint32_t*>(s_rank)[i] = 0u;
  griddep_wait();
  griddep_launch();
  if (kOne && threadIdx.x == 0) *status = 0;
  __syncthreads();
  uint16_t* mine = s_rank + warp * E;
  const int64_t a0 = (int64_t)blockIdx.x * (kWarps * kPerWarp) + warp * kPerWarp + lane;
  int ex[kPerWarp / 32], rank[kPerWarp / 32];
#pragma unroll
  for (int i = 0; i < kPerWarp / 32; ++i) ex[i] = expert_of(ids, mask, a0 + i * 32, R, k, E, status);
#pragma unroll
  for (int i = 0; i < kPerWarp / 32; ++i) {
    const uint32_t peers = __match_any_sync(0xffffffffu, ex[i]);
    const int before = __popc(peers & ((1u << lane) - 1u));
    if (ex[i] >= 0) rank[i] = mine[ex[i]] + before;
    __syncwarp();
    if (ex[i] >= 0 && before == 0) mine[ex[i]] += (uint16_t)__popc(peers);
    __syncwarp();
  }
  __syncthreads();
  if (!kOne && threadIdx.x == 0) s_total = __ldg(offsets + E);
  for (int e = threadIdx.x; e < (kOne ? 1024 : E); e += kWarps * 32) {   // (kOne: one round of 1024 threads)
    int32_t sum = 0;
    if (e < E)
      for (int w = 0; w < kWarps; ++w) {
        const int c = s_rank[w * E + e];
        s_rank[w * E + e] = (uint16_t)sum;
        sum += c;
      }
    if constexpr (kOne) {
      int32_t total;
      const int32_t off = block_exclusive_scan(sum, s_scan, total);
      if (e < E) {
        s_base[e] = off;
        counts[e] = sum;
        offsets[e] = off;
      }
      if (e == 0) offsets[E] = s_total = total;
    } else {
      s_base[e] = __ldg(offsets + e) + __ldg(base + (int64_t)blockIdx.x * E + e);
    }
  }
  __syncthreads();
  const int64_t total = s_total;
#pragma unroll
  for (int i = 0; i < kPerWarp / 32; ++i) {
    const int64_t a = a0 + i * 32;
    if (a >= R) continue;
    int32_t p = -1;
    if (ex[i] >= 0) {
      p = s_base[ex[i]] + mine[ex[i]] + rank[i];
      perm_src[p] = (int32_t)((uint32_t)a / (uint32_t)k);
    }
    inv[a] = p;
    if (a >= total) perm_src[a] = -1;   // (rows behind the last expert's)
  }
}

// Row of assignment a, or -1.
__device__ __forceinline__ int64_t row_of(const int32_t* __restrict__ inv, int64_t a, int64_t R) {
  const int p = __ldg(inv + a);
  return p >= 0 && p < R ? p : -1;
}

// A row over `span` threads, 256 / span rows a block; blockIdx.y takes pieces of span vectors of a row.
__global__ void __launch_bounds__(256) permute_kernel(const uint4* __restrict__ x,
                                                      const int32_t* __restrict__ inv, int T, int k,
                                                      int64_t R, int nvec, int span,
                                                      uint4* __restrict__ rows) {
  griddep_wait();
  griddep_launch();
  const int sub = threadIdx.x / span, lane = threadIdx.x - sub * span;
  const int64_t t = (int64_t)blockIdx.x * (256 / span) + sub;
  const int c = blockIdx.y * span + lane;
  if (sub >= 256 / span || t >= T || c >= nvec) return;
  uint4 v;
  bool have = false;   // (a token without rows is not read)
  for (int j = 0; j < k; ++j) {
    const int64_t p = row_of(inv, t * k + j, R);
    if (p < 0) continue;
    if (!have) {
      v = __ldg(x + t * nvec + c);
      have = true;
    }
    rows[p * nvec + c] = v;
  }
}

template <bool kF32>
__device__ __forceinline__ void add_scaled(uint4 q, float w, float (&acc)[8]) {
  if constexpr (kF32) {
    acc[0] = fmaf(w, __uint_as_float(q.x), acc[0]);
    acc[1] = fmaf(w, __uint_as_float(q.y), acc[1]);
    acc[2] = fmaf(w, __uint_as_float(q.z), acc[2]);
    acc[3] = fmaf(w, __uint_as_float(q.w), acc[3]);
  } else {
    float f[8];
    unpack8(q, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = fmaf(w, f[i], acc[i]);
  }
}

// One 16-byte vector of a token's sum a thread; four rows are read ahead of their addition.
template <bool kF32>
__global__ void __launch_bounds__(256) combine_kernel(const uint4* __restrict__ rows,
                                                      const int32_t* __restrict__ inv,
                                                      const float* __restrict__ w, int T, int k,
                                                      int64_t R, int nvec, int span, uint4* __restrict__ y) {
  griddep_wait();
  griddep_launch();
  const int sub = threadIdx.x / span, lane = threadIdx.x - sub * span;
  const int64_t t = (int64_t)blockIdx.x * (256 / span) + sub;
  const int c = blockIdx.y * span + lane;
  if (sub >= 256 / span || t >= T || c >= nvec) return;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
  for (int j0 = 0; j0 < k; j0 += 4) {
    uint4 q[4];
    float wj[4];
    bool live[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t a = t * k + j0 + i;
      const int64_t p = j0 + i < k ? row_of(inv, a, R) : -1;
      live[i] = p >= 0;
      if (live[i]) {
        q[i] = __ldg(rows + p * nvec + c);
        wj[i] = w ? __ldg(w + a) : 1.0f;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (live[i]) add_scaled<kF32>(q[i], wj[i], acc);
  }
  uint4 o;
  if constexpr (kF32)
    o = make_uint4(__float_as_uint(acc[0]), __float_as_uint(acc[1]), __float_as_uint(acc[2]), __float_as_uint(acc[3]));
  else
    o = pack8(acc);
  y[t * nvec + c] = o;
}

// A warp an assignment.  The k warps of a token read its dy after one another, from L2 or L1.  drows may be the buffer of
// rows: a thread reads a vector of it before it alone writes it, four vectors ahead.
template <bool kF32>
__global__ void __launch_bounds__(256) combine_backward_kernel(
    const uint4* __restrict__ dy, const uint4* rows, const int32_t* __restrict__ inv,
    const float* __restrict__ w, int64_t A, int k, int64_t R, int nvec, uint4* drows,
    float* __restrict__ dw) {
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31;
  const int64_t a = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (a >= A) return;
  const int64_t p = row_of(inv, a, R);
  if (p < 0) {
    if (lane == 0) dw[a] = 0.0f;
    return;
  }
  const uint4* src = rows + p * nvec;
  const uint4* d = dy + (int64_t)((uint32_t)a / (uint32_t)k) * nvec;
  uint4* dst = drows + p * nvec;
  const float wa = __ldg(w + a);
  float s = 0.0f;
  for (int c0 = lane; c0 < nvec; c0 += 4 * 32) {
    uint4 qd[4], qr[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = c0 + i * 32;
      if (c >= nvec) continue;
      qd[i] = __ldg(d + c);
      qr[i] = src[c];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = c0 + i * 32;
      if (c >= nvec) continue;
      uint4 o;
      if constexpr (kF32) {
        const float fd[4] = {__uint_as_float(qd[i].x), __uint_as_float(qd[i].y), __uint_as_float(qd[i].z), __uint_as_float(qd[i].w)};
        const float fr[4] = {__uint_as_float(qr[i].x), __uint_as_float(qr[i].y), __uint_as_float(qr[i].z), __uint_as_float(qr[i].w)};
#pragma unroll
        for (int e = 0; e < 4; ++e) s = fmaf(fd[e], fr[e], s);
        o = make_uint4(__float_as_uint(wa * fd[0]), __float_as_uint(wa * fd[1]), __float_as_uint(wa * fd[2]),
                       __float_as_uint(wa * fd[3]));
      } else {
        float fd[8], fr[8];
        unpack8(qd[i], fd);
        unpack8(qr[i], fr);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          s = fmaf(fd[e], fr[e], s);
          fd[e] *= wa;
        }
        o = pack8(fd);
      }
      dst[c] = o;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) dw[a] = s;
}

// Threads of a row: a power of two, as many as it has vectors, 32 to 256.
int row_span(int nvec) {
  int span = 32;
  while (span < 256 && span < nvec) span *= 2;
  return span;
}

int routing_check(int64_t T, int32_t k, int64_t cols, int64_t row_bytes) {
  if (T < 0 || k < 1 || cols < 1 || row_bytes % 16 != 0) return MOE_ERR_INVALID_ARG;
  if (k > 32 || T > INT32_MAX / k || row_bytes > (1 << 20)) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

// Chunks, 1 if one block does it all.
int chunks_of(int64_t R) { return R <= kOneWarps * kPerWarp ? 1 : (int)((R + kChunk - 1) / kChunk); }

}  // namespace
}  // namespace nvfp4moe

using namespace nvfp4moe;

extern "C" {

size_t moe_sort_tokens_workspace_size(int32_t T, int32_t E, int32_t k) {
  if (T < 0 || E < 1 || E > 1024 || k < 1 || k > 32 || (int64_t)T * k > INT32_MAX) return 0;
  const size_t n = chunks_of((int64_t)T * k);
  // status; histograms and bases of the chunks; the scan's block count and totals
  return 256 + align_up(sizeof(int32_t) * n * E) * 2 + align_up(sizeof(int32_t) * (E + 1));
}

int moe_sort_tokens(const int32_t* topk_ids, const uint8_t* mask, int32_t T, int32_t E, int32_t k,
                    int32_t* counts, int32_t* offsets, int32_t* perm_src, int32_t* inv, void* workspace,
                    size_t ws_bytes, moe_stream_t stream) {
  if (T < 0 || E < 1 || k < 1) return MOE_ERR_INVALID_ARG;
  if (E > 1024 || k > 32 || (int64_t)T * k > INT32_MAX) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!workspace || ws_bytes < moe_sort_tokens_workspace_size(T, E, k)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (!is_aligned(workspace, 256) || !counts || !offsets) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!topk_ids || !perm_src || !inv)) return MOE_ERR_INVALID_ARG;
  for (const void* p : {(const void*)topk_ids, (const void*)counts, (const void*)offsets, (const void*)perm_src, (const void*)inv})
    if (!is_aligned(p, 4)) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int64_t R = (int64_t)T * k;
  const int n = chunks_of(R);
  int32_t* status = static_cast<int32_t*>(workspace);
  cudaError_t e = cudaSuccess;
  if (n == 1) {
    auto place = sort_place_kernel<kOneWarps, true>;
    const size_t smem = sizeof(uint16_t) * kOneWarps * E + 4;
    // above the default limit (static memory counts too): the most that any E needs, so that no call depends on another's
    if (smem > 40 * 1024)
      e = cudaFuncSetAttribute(place, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(uint16_t) * kOneWarps * 1024 + 4);
    if (e == cudaSuccess)
      e = launch_pdl(place, dim3(1), dim3(kOneWarps * 32), smem, s, topk_ids, mask, R, (int)k, (int)E, (const int32_t*)nullptr, counts,
                     offsets, perm_src, inv, status);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  }
  int32_t* hist = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + 256);
  const size_t part = align_up(sizeof(int32_t) * (size_t)n * E) / sizeof(int32_t);
  int32_t* base = hist + part;
  int32_t* scratch = base + part;
  e = cudaMemsetAsync(status, 0, sizeof(int32_t), s);
  if (e == cudaSuccess)
    e = launch_pdl(sort_count_kernel, dim3(n), dim3(kChunkWarps * 32), 0, s, topk_ids, mask, R, (int)k, (int)E, hist, scratch, status);
  if (e == cudaSuccess) e = launch_plan_scan(hist, n, E, base, counts, offsets, scratch, s);
  if (e == cudaSuccess)
    e = launch_pdl(sort_place_kernel<kChunkWarps, false>, dim3(n), dim3(kChunkWarps * 32), sizeof(uint16_t) * kChunkWarps * E + 4, s,
                   topk_ids, mask, R, (int)k, (int)E, (const int32_t*)base, counts, offsets, perm_src, inv, status);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int moe_permute_rows(const void* x, const int32_t* inv, int32_t T, int32_t k, int64_t row_bytes,
                     int64_t R, void* rows, moe_stream_t stream) {
  const int st = routing_check(T, k, row_bytes, row_bytes);
  if (st != MOE_OK) return st;
  if (R < 0) return MOE_ERR_INVALID_ARG;
  if (R > INT32_MAX) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (T == 0 || R == 0) return MOE_OK;
  if (!x || !inv || !rows || x == rows || !is_aligned(x, 16) || !is_aligned(rows, 16) || !is_aligned(inv, 4)) return MOE_ERR_INVALID_ARG;
  const int nvec = (int)(row_bytes / 16), span = row_span(nvec), per = 256 / span;
  const cudaError_t e = launch_pdl(permute_kernel, dim3((unsigned)(((int64_t)T + per - 1) / per), (unsigned)((nvec + span - 1) / span)),
                                   dim3(256), 0, reinterpret_cast<cudaStream_t>(stream), static_cast<const uint4*>(x), inv,
                                   (int)T, (int)k, R, nvec, span, static_cast<uint4*>(rows));
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int moe_combine_rows(const void* rows, const int32_t* inv, const float* topk_w, int32_t T, int32_t k,
                     int64_t cols, int64_t R, uint32_t flags, void* y, moe_stream_t stream) {
  if (flags & ~MOE_ROWS_F32) return MOE_ERR_INVALID_ARG;
  const bool f32 = flags & MOE_ROWS_F32;
  const int st = routing_check(T, k, cols, cols > 0 && cols < (1 << 20) ? cols * (f32 ? 4 : 2) : 1 << 24);
  if (st != MOE_OK) return st;
  if (R < 0) return MOE_ERR_INVALID_ARG;
  if (R > INT32_MAX) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return MOE_OK;
  if ((!rows && R > 0) || !inv || !y || rows == y || !is_aligned(rows, 16) || !is_aligned(y, 16) || !is_aligned(inv, 4) || !is_aligned(topk_w, 4))
    return MOE_ERR_INVALID_ARG;
  const int nvec = (int)(cols / (f32 ? 4 : 8)), span = row_span(nvec), per = 256 / span;
  const cudaError_t e = launch_pdl(f32 ? combine_kernel<true> : combine_kernel<false>,
                                   dim3((unsigned)(((int64_t)T + per - 1) / per), (unsigned)((nvec + span - 1) / span)), dim3(256), 0,
                                   reinterpret_cast<cudaStream_t>(stream), static_cast<const uint4*>(rows), inv, topk_w, (int)T,
                                   (int)k, R, nvec, span, static_cast<uint4*>(y));
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int moe_combine_rows_backward(const void* dy, const void* rows, const int32_t* inv, const float* topk_w,
                              int32_t T, int32_t k, int64_t cols, int64_t R, uint32_t flags, void* drows,
                              float* dtopk_w, moe_stream_t stream) {
  if (flags & ~MOE_ROWS_F32) return MOE_ERR_INVALID_ARG;
  const bool f32 = flags & MOE_ROWS_F32;
  const int st = routing_check(T, k, cols, cols > 0 && cols < (1 << 20) ? cols * (f32 ? 4 : 2) : 1 << 24);
  if (st != MOE_OK) return st;
  if (R < 0) return MOE_ERR_INVALID_ARG;
  if (R > INT32_MAX) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return MOE_OK;
  if (!dy || dy == drows || !inv || !topk_w || !dtopk_w || ((!rows || !drows) && R > 0)) return MOE_ERR_INVALID_ARG;
  for (const void* p : {dy, rows, (const void*)drows})
    if (!is_aligned(p, 16)) return MOE_ERR_INVALID_ARG;
  if (!is_aligned(inv, 4) || !is_aligned(topk_w, 4) || !is_aligned(dtopk_w, 4)) return MOE_ERR_INVALID_ARG;
  const int64_t A = (int64_t)T * k;
  const cudaError_t e = launch_pdl(f32 ? combine_backward_kernel<true> : combine_backward_kernel<false>,
                                   dim3((unsigned)((A + 7) / 8)), dim3(256), 0, reinterpret_cast<cudaStream_t>(stream),
                                   static_cast<const uint4*>(dy), static_cast<const uint4*>(rows), inv, topk_w, A, (int)k, R,
                                   (int)(cols / (f32 ? 4 : 8)), static_cast<uint4*>(drows), dtopk_w);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
