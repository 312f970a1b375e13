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
// Both are bound by HBM: every element is read and written once.  Device time of a call, share of the copy rate:
// forward with a residual 16384 x 4096 81.8 us (97%), FP32 166 us (95%), 8191 x 7168 71.3 us (97%), 12000 x 5120 83 us (87%),
// 20000 x 256 12.7 us (47%), one row of 2048 1.7 us; backward with dh 16384 x 4096 84 us (94%), FP32 without dh 133 us (89%),
// 8191 x 7168 82.5 us (84%: one group of 14 warps, whose row takes 1.5 us from its arrival to its last store), 12000 x 5120 94 us
// (77%), 20000 x 1024 33 us (73%).  Narrow rows wait: a row is a chain of a read, two reductions, a barrier and a store of about
// 1.5 us (backward 1.8), and an SM works on 16 rows of 256 columns, 8 of 1024 at a time, so that 20000 rows are 8 to 16 such
// chains, one after another.  2.5 to 5 us of the backward pass are the join of the blocks' sums.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "ops.h"

namespace nvfp4moe {

namespace {

constexpr int kMaxCols = 16384;
constexpr int kMostRing = 216 * 1024;   // dynamic shared memory of a launch, at most

// Eight FP32 elements, as uint4 holds eight BF16 ones.
struct F32x8 {
  float4 a, b;
};

// How a row is laid over threads: W warps with J vectors of 8 columns a lane (vector c of lane t:
// c = j * 32 W + t); a block holds G such row groups.
struct NormGrid {
  int J, W, G, blocks;
};

// ---- many rows: rows come through a ring in shared memory ----
//
// A group of W warps takes every gridDim * G-th row.  Its rows are fetched by bulk copies into a ring of
// `slots` rows of its own (all of the row's tensors).  Each row has one barrier over the group, behind which
// all its warps are done with the row before, whose slot is filled again: no other hand-over is needed.  The
// ring keeps 100 KB and more an SM under way without registers for it, so that a lane can hold two vectors of
// everything else; arithmetic goes in pairs (f32x2), as instructions, not bytes, are what is short: one
// vector a lane and scalar arithmetic took 92 and 101 us for 16384 x 4096 and 8191 x 7168 backward, two rows a
// barrier or not.  slots == 1 (rows so wide that two do not fit): the row ends in a barrier before its slot is filled.
//
// A thread whose wait for a row runs out sets the block's `stop`: the block's rows from there on become NaN (h, which is stored
// before the row's barrier, at the end), issuers start no more copies (a row's slot is filled again behind the next row's
// barrier, so a read of `stop` between the row's own barrier and that is in time), the threads that then wait in vain
// give up too, and at the end each issuer waits, again with a limit, for the copies that it did start, before their
// memory is used for anything else or left.

constexpr uint64_t kCopyLimitNs = 1000000000ull;

// The wait for a row that has not landed yet; false if it ran out, here or elsewhere in the block.  Out of line: inside the loop
// over rows its code costs the forward pass of 8191 x 7168 73.5 us instead of 71.1.
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t phase, volatile uint32_t* stop) {
  const uint64_t t0 = global_timer_ns();
  for (;;) {
    if (mbar_try_wait(bar, phase)) return true;
    if (*stop) return false;
    if (global_timer_ns() - t0 > kCopyLimitNs) {
      *stop = 1u;
      return false;
    }
  }
}

struct Ring {
  uint32_t data, bars;     // shared addresses of the group's slots and their barriers
  uint32_t row_bytes;      // of one tensor
  int slots, group, G, W;
  bool issuer;             // the group's thread that starts the copies
  volatile uint32_t* stop; // the block's: a wait has run out

  template <int kN>
  __device__ __forceinline__ uint32_t at(uint32_t s, int tensor) const {
    return data + (s * kN + tensor) * row_bytes;
  }
  template <int kN>
  __device__ __forceinline__ void fetch(uint32_t s, const void* const (&src)[kN], int count, int64_t row) const {
    const uint32_t bar = bars + 8 * s;
    mbar_arrive_expect_tx(bar, (uint32_t)count * row_bytes);
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (i < count) bulk_load(at<kN>(s, i), static_cast<const uint8_t*>(src[i]) + row * row_bytes, row_bytes, bar);
  }
  // The row of a slot has landed; false if the wait ran out.
  __device__ __forceinline__ bool landed(uint32_t s, uint32_t phase) const {
    return mbar_try_wait(bars + 8 * s, phase) || wait_on(bars + 8 * s, phase, stop);
  }
  // The first `issued` rows' copies have ended (the issuer, after a stop): slot s was filled last by row
  // s + k * slots, in phase k.
  __device__ void drain(int issued) const {
    for (int s = 0; s < min(slots, issued); ++s)
      mbar_wait_bounded(bars + 8 * s, (uint32_t)((issued - 1 - s) / slots) & 1u, kCopyLimitNs, nullptr);
  }
  __device__ __forceinline__ void barrier() const {
    if (W == 1) __syncwarp();
    else if (G == 1) __syncthreads();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(W * 32) : "memory");
  }
};

// Slots of a group's ring: as many as keep `want` bytes an SM under way, `least` of them where they fit.  More do harm:
// with 192 KB of reads ahead the forward pass of 16384 x 4096 takes 92 us, with 96 KB 82 us (with 64 KB 105).
int ring_slots(int G, size_t slot_bytes, size_t want, int least) {
  const int fit = (int)(208 * 1024 / G / slot_bytes);
  return std::max(1, std::min({8, fit, std::max(least, (int)(want / G / slot_bytes))}));
}
size_t ring_bytes(int G, int slots, size_t slot_bytes) { return 2048 + (size_t)G * slots * slot_bytes; }

__device__ __forceinline__ Ring make_ring(uint8_t* smem, uint32_t* stop, uint32_t row_bytes, int tensors, int slots, int group, int G, int W,
                                          int t) {
  Ring r;
  r.stop = stop;
  if (threadIdx.x == 0) *stop = 0u;
  r.bars = smem_u32(smem) + (uint32_t)group * slots * 8;   // (32 groups of 8 slots at most: 2 KB)
  r.data = smem_u32(smem) + 2048 + (uint32_t)group * slots * tensors * row_bytes;
  r.row_bytes = row_bytes;
  r.slots = slots;
  r.group = group;
  r.G = G;
  r.W = W;
  r.issuer = t == 0;
  if (r.issuer) {
    for (int i = 0; i < slots; ++i) mbar_init(r.bars + 8 * i, 1);
    fence_barrier_init();
  }
  return r;
}

__device__ __forceinline__ void set_nan(uint4& q) { q = make_uint4(~0u, ~0u, ~0u, ~0u); }
__device__ __forceinline__ void set_nan(F32x8& q) {
  const float v = __int_as_float(0x7FC00000);
  q.a = q.b = make_float4(v, v, v, v);
}
__device__ __forceinline__ void read_vec(uint32_t addr, uint4& q) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "r"(addr) : "memory");
}
__device__ __forceinline__ void read_vec(uint32_t addr, F32x8& q) {
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(q.a.x), "=f"(q.a.y), "=f"(q.a.z), "=f"(q.a.w) : "r"(addr) : "memory");
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(q.b.x), "=f"(q.b.y), "=f"(q.b.z), "=f"(q.b.w) : "r"(addr + 16) : "memory");
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// The sum over the first 16 lanes, one for each of the row's warps, on all lanes.
__device__ __forceinline__ float warps_sum(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return __shfl_sync(0xffffffffu, v, 0);
}

// sum / cols, correctly rounded as a quotient by a corrected reciprocal is (div_rn_by_recip): the mean of a constant row is its
// value, where sum * (1 / cols) is a step off for most cols, and a step of a large value is far from 0 against eps.  A sum that
// is not finite stays.
__device__ __forceinline__ float row_mean(float sum, float cols, float inv_cols) {
  const float q = div_rn_by_recip(sum, cols, inv_cols);
  return isfinite(sum) ? q : sum;
}

// Two FP32 operations an instruction.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{.reg .b64 x, y, z;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\nadd.rn.f32x2 z, x, y;\nmov.b64 {%0, %1}, z;}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{.reg .b64 x, y, z;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\nmul.rn.f32x2 z, x, y;\nmov.b64 {%0, %1}, z;}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{.reg .b64 x, y, w, z;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\nmov.b64 w, {%6, %7};\n"
      "fma.rn.f32x2 z, x, y, w;\nmov.b64 {%0, %1}, z;}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ void unpack(const uint4& q, float2 (&f)[4]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ void unpack(const F32x8& q, float2 (&f)[4]) {
  f[0] = make_float2(q.a.x, q.a.y);
  f[1] = make_float2(q.a.z, q.a.w);
  f[2] = make_float2(q.b.x, q.b.y);
  f[3] = make_float2(q.b.z, q.b.w);
}
__device__ __forceinline__ void pack(const float2 (&f)[4], uint4& q) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[i].x, f[i].y);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  q = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void pack(const float2 (&f)[4], F32x8& q) {
  q.a = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
  q.b = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
}

// A warp's share of a row's mean and variance: elements, their sum, their mean and the sum of squared distances from it.
// The warps' sums and the distances between their means meet behind the row's one barrier.
struct __align__(16) Share {
  float n, sum, mean, dist;
};

template <typename V, int J>
__global__ void __launch_bounds__(512, 1) add_layernorm_kernel(
    const V* x, const V* residual, const V* __restrict__ gamma, const V* __restrict__ beta, float eps,
    int64_t rows, int cols, int W, int G, int slots, V* h, V* y, float* mean, float* rstd) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Share red[2][16];
  __shared__ uint32_t s_stop;
  constexpr bool kWide = J > 3;   // gamma and beta are read again for each row
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group = warp / W, wrow = warp - group * W;
  const int t = wrow * 32 + lane, span = W * 32;   // thread of the row, vectors apart
  const int nvec = cols / 8;
  const float inv_cols = __fdiv_rn(1.0f, (float)cols);
  const int tensors = residual ? 2 : 1;
  const Ring ring = make_ring(smem, &s_stop, (uint32_t)cols * (sizeof(V) / 8), 2, slots, group, G, W, t);
  __syncthreads();
  griddep_wait();
  griddep_launch();
  const int64_t row0 = (int64_t)blockIdx.x * G + group, step = (int64_t)gridDim.x * G;
  const int count = row0 < rows ? (int)((rows - row0 + step - 1) / step) : 0;   // rows of the group
  const void* const src[2] = {x, residual};
  int issued = min(slots, count);   // rows whose copies have been started
  if (ring.issuer)
    for (int n = 0; n < issued; ++n) ring.fetch<2>(n, src, tensors, row0 + n * step);
  const V zero = {};
  auto gain = [&](int c, float2 (&f)[4]) { unpack(c < nvec ? gamma[c] : zero, f); };
  auto bias = [&](int c, float2 (&f)[4]) { unpack(c < nvec && beta ? beta[c] : zero, f); };
  float2 g[kWide ? 1 : J][4], b[kWide ? 1 : J][4];
  int mine = 0;   // elements of the warp
#pragma unroll
  for (int j = 0; j < J; ++j) {
    if constexpr (!kWide) {
      gain(j * span + t, g[j]);
      bias(j * span + t, b[j]);
    }
    mine += 8 * min(max(nvec - (j * span + wrow * 32), 0), 32);
  }
  int lost = count;   // first of the group's rows that was lost
  const float wn = (float)mine, inv_wn = mine ? __fdiv_rn(1.0f, wn) : 0.0f;
  bool ok = true;
  uint32_t phase = 0;
  for (int n = 0, s = 0, par = 0; n < count; ++n, par ^= 1) {   // s: the row's slot
    ok = ok && ring.landed(s, phase);
    const int64_t base = (row0 + n * step) * nvec;
    float2 f[J][4], sum = both(0.0f);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = j * span + t;
      V q = zero;
      if (c < nvec) {
        read_vec(ring.at<2>(s, 0) + c * (uint32_t)sizeof(V), q);
        if (residual) {
          V e;
          float2 d[4];
          unpack(q, f[j]);
          read_vec(ring.at<2>(s, 1) + c * (uint32_t)sizeof(V), e);
          unpack(e, d);
#pragma unroll
          for (int i = 0; i < 4; ++i) f[j][i] = add2(f[j][i], d[i]);
          pack(f[j], q);
          h[base + c] = q;
        }
      }
      unpack(q, f[j]);
#pragma unroll
      for (int i = 0; i < 4; ++i) sum = add2(sum, f[j][i]);
    }
    const float ws = warp_sum(sum.x + sum.y), wm = ws * inv_wn;
    float2 dist = both(0.0f);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      if (j * span + t >= nvec) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 d = add2(f[j][i], both(-wm));
        dist = fma2(d, d, dist);
      }
    }
    const float wd = warp_sum(dist.x + dist.y);
    if (lane == 0) red[par][warp] = Share{wn, ws, wm, wd};
    ring.barrier();
    const bool stopped = *ring.stop;
    if (ring.issuer && n > 0 && slots > 1 && n - 1 + slots < count && !stopped) {   // the slot of the row before
      ring.fetch<2>(s ? s - 1 : slots - 1, src, tensors, row0 + (int64_t)(n - 1 + slots) * step);
      ++issued;
    }
    const Share w = lane < W ? red[par][group * W + lane] : Share{0.0f, 0.0f, 0.0f, 0.0f};
    float m = row_mean(warps_sum(w.sum), (float)cols, inv_cols);
    if (stopped) {
      m = __int_as_float(0x7FC00000);
      lost = min(lost, n);
    }
    const float var = warps_sum(fmaf(w.n * (w.mean - m), w.mean - m, w.dist)) * inv_cols;
    const float r = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(var, eps)));
    if (t == 0) {
      if (mean) mean[row0 + n * step] = m;
      if (rstd) rstd[row0 + n * step] = r;
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = j * span + t;
      if (c >= nvec) continue;
      if constexpr (kWide) {
        gain(c, g[0]);
        bias(c, b[0]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        f[j][i] = fma2(mul2(add2(f[j][i], both(-m)), both(r)), g[kWide ? 0 : j][i], b[kWide ? 0 : j][i]);
      V o;
      pack(f[j], o);
      y[base + c] = o;
    }
    if (slots == 1) {
      ring.barrier();
      if (ring.issuer && n + 1 < count && !*ring.stop) {
        ring.fetch<2>(0, src, tensors, row0 + (int64_t)(n + 1) * step);
        ++issued;
      }
    }
    if (++s == slots) {
      s = 0;
      phase ^= 1u;
    }
  }
  if (*ring.stop && residual) {
    V q;
    set_nan(q);
    for (int n = lost; n < count; ++n)
      for (int c = t; c < nvec; c += span) h[(row0 + n * step) * nvec + c] = q;
  }
  if (ring.issuer && *ring.stop) ring.drain(issued);
}

// A thread owns the same J vectors of 8 columns in all rows of its group and keeps their share of dgamma
// and dbeta in registers; the groups of a block are joined in order at the end, the blocks by column_sums_kernel.
template <typename V, int J>
__global__ void __launch_bounds__(512, 1) add_layernorm_backward_kernel(
    const V* dy, const V* dh, const V* h, const float* __restrict__ mean, const float* __restrict__ rstd,
    const V* __restrict__ gamma, int64_t rows, int cols, int W, int G, int slots, V* dx, bool want_beta,
    float4* __restrict__ partial) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float2 red[2][16];
  __shared__ uint32_t s_stop;
  constexpr bool kKeep = J <= 2;   // a and n stay in registers over the barrier, else they are computed again
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group = warp / W, wrow = warp - group * W;
  const int t = wrow * 32 + lane, span = W * 32;
  const int nvec = cols / 8;
  const float inv_cols = __fdiv_rn(1.0f, (float)cols);
  const int tensors = dh ? 3 : 2;
  const Ring ring = make_ring(smem, &s_stop, (uint32_t)cols * (sizeof(V) / 8), 3, slots, group, G, W, t);
  __syncthreads();
  griddep_wait();
  griddep_launch();
  const int64_t row0 = (int64_t)blockIdx.x * G + group, step = (int64_t)gridDim.x * G;
  const int count = row0 < rows ? (int)((rows - row0 + step - 1) / step) : 0;
  const void* const src[3] = {dy, h, dh};
  int issued = min(slots, count);   // rows whose copies have been started
  if (ring.issuer)
    for (int n = 0; n < issued; ++n) ring.fetch<3>(n, src, tensors, row0 + n * step);
  const V zero = {};
  float2 g[kKeep ? J : 1][4];
  auto gain = [&](int c, float2 (&f)[4]) { unpack(c < nvec ? gamma[c] : zero, f); };
  float2 dg[J][4], db[J][4];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    if constexpr (kKeep) gain(j * span + t, g[j]);
#pragma unroll
    for (int i = 0; i < 4; ++i) dg[j][i] = db[j][i] = both(0.0f);
  }
  // a = gamma dy and n of a vector
  auto terms = [&](uint32_t s, int j, float m, float r, float2 (&d)[4], float2 (&a)[4], float2 (&nv)[4]) {
    const int c = j * span + t;
    V qd, qh;
    read_vec(ring.at<3>(s, 0) + c * (uint32_t)sizeof(V), qd);
    read_vec(ring.at<3>(s, 1) + c * (uint32_t)sizeof(V), qh);
    unpack(qd, d);
    unpack(qh, nv);
    if constexpr (!kKeep) gain(c, g[0]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      nv[i] = mul2(add2(nv[i], both(-m)), both(r));
      a[i] = mul2(d[i], g[kKeep ? j : 0][i]);
    }
  };
  float nm = count > 0 ? __ldg(mean + row0) : 0.0f, nr = count > 0 ? __ldg(rstd + row0) : 0.0f;
  bool ok = true;
  uint32_t phase = 0;
  for (int n = 0, s = 0, par = 0; n < count; ++n, par ^= 1) {
    float m = nm;
    const float r = nr;
    if (n + 1 < count) {   // the next row's statistics
      nm = __ldg(mean + row0 + (int64_t)(n + 1) * step);
      nr = __ldg(rstd + row0 + (int64_t)(n + 1) * step);
    }
    ok = ok && ring.landed(s, phase);
    if (!ok) m = __int_as_float(0x7FC00000);
    const bool more = !*ring.stop;
    float2 a[kKeep ? J : 1][4], nv[kKeep ? J : 1][4], sa = both(0.0f), sn = both(0.0f);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      if (j * span + t >= nvec) continue;
      const int k = kKeep ? j : 0;
      float2 d[4];
      terms(s, j, m, r, d, a[k], nv[k]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sa = add2(sa, a[k][i]);
        sn = fma2(a[k][i], nv[k][i], sn);
        dg[j][i] = fma2(d[i], nv[k][i], dg[j][i]);
        db[j][i] = add2(db[j][i], d[i]);
      }
    }
    const float2 share = make_float2(warp_sum(sa.x + sa.y), warp_sum(sn.x + sn.y));
    if (lane == 0) red[par][warp] = share;
    ring.barrier();
    if (ring.issuer && n > 0 && slots > 1 && n - 1 + slots < count && more) {   // the slot of the row before
      ring.fetch<3>(s ? s - 1 : slots - 1, src, tensors, row0 + (int64_t)(n - 1 + slots) * step);
      ++issued;
    }
    const float2 w = lane < W ? red[par][group * W + lane] : make_float2(0.0f, 0.0f);
    const float ma = warps_sum(w.x) * inv_cols, mn = warps_sum(w.y) * inv_cols;
    const int64_t base = (row0 + n * step) * nvec;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = j * span + t, k = kKeep ? j : 0;
      if (c >= nvec) continue;
      if constexpr (!kKeep) {
        float2 d[4];
        terms(s, j, m, r, d, a[0], nv[0]);
      }
      float2 o[4], e[4];
      V q;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = mul2(both(r), fma2(nv[k][i], both(-mn), add2(a[k][i], both(-ma))));
      if (dh) {
        read_vec(ring.at<3>(s, 2) + c * (uint32_t)sizeof(V), q);
        unpack(q, e);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = add2(o[i], e[i]);
      }
      pack(o, q);
      dx[base + c] = q;
    }
    if (slots == 1) {
      ring.barrier();
      if (ring.issuer && n + 1 < count && !*ring.stop) {
        ring.fetch<3>(0, src, tensors, row0 + (int64_t)(n + 1) * step);
        ++issued;
      }
    }
    if (++s == slots) {
      s = 0;
      phase ^= 1u;
    }
  }
  if (ring.issuer && *ring.stop) ring.drain(issued);
  __syncthreads();
  if (*ring.stop) {
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) dg[j][i] = db[j][i] = both(__int_as_float(0x7FC00000));
  }
  // the other groups' sums to the first's, in order, through the ring's memory
  float4* s_part = reinterpret_cast<float4*>(smem + 2048);   // [cols / 4]
#pragma unroll
  for (int which = 0; which < 2; ++which) {   // dgamma, then dbeta
    if (which == 1 && !want_beta) break;
    float2(&acc)[J][4] = which ? db : dg;
    for (int k = 1; k < G; ++k) {
      __syncthreads();
      if (group == k) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const int c = j * span + t;
          if (c >= nvec) continue;
          s_part[2 * c] = make_float4(acc[j][0].x, acc[j][0].y, acc[j][1].x, acc[j][1].y);
          s_part[2 * c + 1] = make_float4(acc[j][2].x, acc[j][2].y, acc[j][3].x, acc[j][3].y);
        }
      }
      __syncthreads();
      if (group == 0) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const int c = j * span + t;
          if (c >= nvec) continue;
          const float4 u = s_part[2 * c], v = s_part[2 * c + 1];
          acc[j][0] = add2(acc[j][0], make_float2(u.x, u.y));
          acc[j][1] = add2(acc[j][1], make_float2(u.z, u.w));
          acc[j][2] = add2(acc[j][2], make_float2(v.x, v.y));
          acc[j][3] = add2(acc[j][3], make_float2(v.z, v.w));
        }
      }
    }
    if (group != 0) continue;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = j * span + t;
      if (c >= nvec) continue;
      float4* p = partial + ((int64_t)which * gridDim.x + blockIdx.x) * (cols / 4) + 2 * c;
      p[0] = make_float4(acc[j][0].x, acc[j][0].y, acc[j][1].x, acc[j][1].y);
      p[1] = make_float4(acc[j][2].x, acc[j][2].y, acc[j][3].x, acc[j][3].y);
    }
  }
}

// ---- few rows (forward): one row a block, loaded straight into registers ----
//
// h may be the buffer of x or residual: a thread has read its vectors of both before it writes any.
template <typename V, int J>
__global__ void __launch_bounds__(1024, 1) add_layernorm_row_kernel(
    const V* x, const V* residual, const V* __restrict__ gamma,
    const V* __restrict__ beta, float eps, int cols, V* h, V* y, float* mean, float* rstd) {
  __shared__ Share red[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, span = blockDim.x, W = span / 32, nvec = cols / 8;
  const float inv_cols = __fdiv_rn(1.0f, (float)cols);
  griddep_wait();
  griddep_launch();
  const int64_t base = (int64_t)blockIdx.x * nvec;
  const V zero = {};
  V q[J], e[J], g[J], b[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c = j * span + threadIdx.x;
    const bool in = c < nvec;
    q[j] = in ? x[base + c] : zero;
    e[j] = in && residual ? residual[base + c] : zero;
  }
  float2 f[J][4], sum = both(0.0f);
  int mine = 0;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c = j * span + threadIdx.x;
    g[j] = c < nvec ? gamma[c] : zero;
    b[j] = c < nvec && beta ? beta[c] : zero;
    if (residual && c < nvec) {
      float2 d[4];
      unpack(q[j], f[j]);
      unpack(e[j], d);
#pragma unroll
      for (int i = 0; i < 4; ++i) f[j][i] = add2(f[j][i], d[i]);
      pack(f[j], q[j]);
      h[base + c] = q[j];
    }
    unpack(q[j], f[j]);
#pragma unroll
    for (int i = 0; i < 4; ++i) sum = add2(sum, f[j][i]);
    mine += 8 * min(max(nvec - (j * span + warp * 32), 0), 32);
  }
  const float ws = warp_sum(sum.x + sum.y), wm = mine ? __fdiv_rn(ws, (float)mine) : 0.0f;
  float2 dist = both(0.0f);
#pragma unroll
  for (int j = 0; j < J; ++j) {
    if (j * span + (int)threadIdx.x >= nvec) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 d = add2(f[j][i], both(-wm));
      dist = fma2(d, d, dist);
    }
  }
  const float wd = warp_sum(dist.x + dist.y);
  if (lane == 0) red[warp] = Share{(float)mine, ws, wm, wd};
  __syncthreads();
  const Share w = lane < W ? red[lane] : Share{0.0f, 0.0f, 0.0f, 0.0f};
  const float m = row_mean(warp_sum(w.sum), (float)cols, inv_cols);
  const float var = warp_sum(fmaf(w.n * (w.mean - m), w.mean - m, w.dist)) * inv_cols;
  const float r = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(var, eps)));
  if (threadIdx.x == 0) {
    if (mean) mean[blockIdx.x] = m;
    if (rstd) rstd[blockIdx.x] = r;
  }
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c = j * span + threadIdx.x;
    if (c >= nvec) continue;
    float2 gf[4], bf[4];
    unpack(g[j], gf);
    unpack(b[j], bf);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[j][i] = fma2(mul2(add2(f[j][i], both(-m)), both(r)), gf[i], bf[i]);
    V o;
    pack(f[j], o);
    y[base + c] = o;
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
#pragma unroll 5
    for (int b = warp; b < nb; b += 32) s += __ldcg(part + (int64_t)b * cols + c);
  red[warp][lane] = s;
  __syncthreads();
  // lane w of warp c adds warp w's share of column c
  s = warp_sum(red[lane][warp]);
  const int col = blockIdx.x * 32 + warp;
  if (lane == 0 && col < cols) (blockIdx.y ? dbeta : dgamma)[col] = s;
}

// At most kPartBlocks blocks in the backward pass, which the workspace's size goes by: it does not depend on
// the device.
constexpr int kPartBlocks = 192;

// 16 warps a block, two vectors a lane; four above 8192 columns, one up to 256.  A row takes 1.1 us from its arrival to
// its last store, which a second group hides; of 4104 to 6144 columns two vectors a lane would leave one group of 9 to 12
// warps, three leave two of 6 to 8 (12000 x 5120: 93 and 82 us, backward 104 and 93).
NormGrid row_grid(int64_t rows, int nvec) {
  NormGrid g;
  g.J = nvec > 1024 ? 4 : nvec <= 32 ? 1 : nvec > 512 && nvec <= 768 ? 3 : 2;
  g.W = (nvec + 32 * g.J - 1) / (32 * g.J);
  g.G = (int)std::min<int64_t>(16 / g.W, std::max<int64_t>(1, rows / num_sms()));   // every SM before every group
  g.blocks = (int)std::min<int64_t>((rows + g.G - 1) / g.G, std::min(num_sms(), kPartBlocks));
  return g;
}

template <typename V>
cudaError_t launch_forward(const void* x, const void* residual, const void* gamma, const void* beta,
                           float eps, int64_t rows, int cols, void* h, void* y, float* mean,
                           float* rstd, cudaStream_t s) {
  const V *xv = static_cast<const V*>(x), *rv = static_cast<const V*>(residual);
  const V *gv = static_cast<const V*>(gamma), *bv = static_cast<const V*>(beta);
  V *hv = static_cast<V*>(h), *yv = static_cast<V*>(y);
  const int nvec = cols / 8;
  // Rows that are all on the SMs at once, 48 warps each, have nothing to be read ahead of (912 x 2048: 3.2 us against the
  // ring's 4.5, 152 x 7168 2.7 and 2.9; with twice as many rows 6.3 and 6.8, 4.6 and 4.2).
  const int J = nvec > 1024 ? 2 : 1, threads = (nvec + 32 * J - 1) / (32 * J) * 32;
  if (rows * (threads / 32) <= 48 * (int64_t)num_sms()) {
    auto k = J == 1 ? add_layernorm_row_kernel<V, 1> : add_layernorm_row_kernel<V, 2>;
    return launch_pdl(k, dim3((unsigned)rows), dim3(threads), 0, s, xv, rv, gv, bv, eps, cols, hv, yv, mean, rstd);
  }
  const NormGrid g = row_grid(rows, nvec);
  const size_t slot = 2 * (size_t)cols * (sizeof(V) / 8);
  const int slots = ring_slots(g.G, slot, 120 * 1024, 2);
  auto k = g.J == 1   ? add_layernorm_kernel<V, 1>
           : g.J == 2 ? add_layernorm_kernel<V, 2>
           : g.J == 3 ? add_layernorm_kernel<V, 3>
                      : add_layernorm_kernel<V, 4>;
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostRing);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, dim3((unsigned)g.blocks), dim3(g.W * g.G * 32), ring_bytes(g.G, slots, slot), s, xv, rv, gv, bv, eps, rows,
                    cols, g.W, g.G, slots, hv, yv, mean, rstd);
}

template <typename V>
cudaError_t launch_backward(const void* dy, const void* dh, const void* h, const float* mean,
                            const float* rstd, const void* gamma, int64_t rows, int cols, void* dx,
                            float* dgamma, float* dbeta, void* workspace, cudaStream_t s) {
  const NormGrid g = row_grid(rows, cols / 8);
  const size_t slot = 3 * (size_t)cols * (sizeof(V) / 8);
  const int slots = ring_slots(g.G, slot, 144 * 1024, 3);
  auto k = g.J == 1   ? add_layernorm_backward_kernel<V, 1>
           : g.J == 2 ? add_layernorm_backward_kernel<V, 2>
           : g.J == 3 ? add_layernorm_backward_kernel<V, 3>
                      : add_layernorm_backward_kernel<V, 4>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostRing);
  if (e != cudaSuccess) return e;
  e = launch_pdl(k, dim3(g.blocks), dim3(g.W * g.G * 32), ring_bytes(g.G, slots, slot), s, static_cast<const V*>(dy),
                 static_cast<const V*>(dh), static_cast<const V*>(h), mean, rstd, static_cast<const V*>(gamma), rows, cols, g.W, g.G,
                 slots, static_cast<V*>(dx), dbeta != nullptr, static_cast<float4*>(workspace));
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
