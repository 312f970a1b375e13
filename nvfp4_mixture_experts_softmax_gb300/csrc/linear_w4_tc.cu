// 4-bit matrix-vector product for many rows of x (9 or 17 to 64) on the fifth-generation tensor
// cores: 128 weight rows are an MMA's M, the rows of x (rounded up to 16) its N.
//
// The weights are decoded to BF16 in registers and handed to tcgen05.mma through tensor memory as
// its A operand; x comes into shared memory by TMA as B, as it is.  (A through shared memory would
// put 128 x 64 BF16 weights there for every 64 columns, written and read: 22 us for 18432 x 7168
// before anything else.)  An E2M1 value times an E4M3 scale is exact in BF16 (at most 6 significant
// bits), and so is one times an E8M0 scale with a power of two set aside: a quarter of it is at least
// 2^-130 and at most 1.5 * 2^127.  The sums are the tensor core's, FP32.
//
// A block works on 256 weight rows (two accumulators) in steps of 128 columns; a thread decodes its
// row's 64 bytes of a step.  Warps 0-23 decode (w % 4: tensor memory's lane quadrant, w / 4 % 2: the
// accumulator, w / 8: every third step), 24 loads x, 25 allocates tensor memory and issues the MMAs,
// 26 loads the codes.  Three rings join them: codes and x in shared memory, decoded weights in
// tensor memory.  256 rows, because x is read from L2 once a block: at 128 rows (two blocks an SM)
// it was twice the bytes of the codes.
// With few tiles the blocks of a cluster split K; each sums its share of the rows from all blocks'
// accumulators, which they store into its shared memory, in block order.  With more tiles than SMs a
// block works through several; its rings run on, and the warps that decode store a tile before they
// go on to the next.
// The tensor core truncates where it adds: chains of 128 / 256 / 448 / 1024 MMAs of normal data end 4e-7 /
// 1e-6 / 2e-6 / 6e-6 of y off.  FP32 output stays at 1e-6: above kTcChain steps they take turns on two or
// four accumulators (up to 32 or 16 rows: what 64 columns hold), and a tile's K is worked through in parts,
// like further tiles, that are added in FP32 in shared memory; the blocks of a cluster then read one
// another's sums.  BF16 output does not need it.  (36864 x 7168, 24 / 64 rows: 42.9 / 49.4 us, one chain
// 41.2 / 44.)
// Every wait is bounded; a block whose wait ran out stores NaN.
//
// Measured (device time of a call, NVFP4; in brackets warp-level MMAs): 18432 x 7168, 32 rows 25 us
// (41), 64 rows 29 us (86); 36864 x 7168, 64 rows 44 us (165); 2048 x 2048, 64 rows 8.8 us (17.5);
// 18431 x 7168 MXFP4, 15 rows 24.1 us (26.2).  A step of a block takes 0.62 us.  Alone the decoding
// takes 0.59 (some 20 instructions for 8 codes), the MMAs 0.53 at 64 rows (67 cycles each), the loads
// 0.39 (from L2, 32 KB); 16 decoding warps 0.64; a warp whose single lane issues the MMAs 1.11.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <type_traits>

#include "ops.h"
#include "w4.cuh"

namespace nvfp4moe {

namespace {

constexpr int kTcMaxTokens = 64;
constexpr int kTcRows = 256;           // two accumulators of 128 rows
constexpr int kTcCodeStages = 5;       // ring of codes: 128 columns each
constexpr int kTcXStages = 4;          // ring of x: 128 columns each, as two swizzled tiles of 64
constexpr int kTcAStages = 3;          // ring of decoded weights in tensor memory: 128 columns each
constexpr int kTcCodeBytes = kTcRows * 64;
constexpr int kTcChain = 32;           // steps of an accumulator with FP32 output: 256 MMAs in a chain,
constexpr int kTcPart = 28;            // and where that is not enough, 224
constexpr int kTcDecWarps = 24;
constexpr int kTcXWarp = 24;
constexpr int kTcMmaWarp = 25;
constexpr int kTcCodeWarp = 26;
constexpr int kTcThreads = 864;
constexpr uint32_t kTcCols = 512;      // tensor memory: accumulators, then the A ring
constexpr uint32_t kTcACol = 128;

// kind::f16 with FP32 accumulators, BF16 operands, K-major: see the grouped GEMM's descriptor.
__device__ __forceinline__ uint32_t tc_idesc(int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

// D (+)= A B over 64 columns of K for both halves of the tile (128 rows each), by one lane of a
// converged warp.  A in tensor memory: lane = row, 32-bit column = two elements of K, so K = 16 is 8
// columns; the second half's is 64 columns on, its accumulators too.  B: 32 bytes of a 128-byte
// row.  The whole warp runs the loop around this and one lane is elected here: the operands stay in
// uniform registers (issued by a single lane of a diverged warp an MMA costs 43 cycles).
__device__ __forceinline__ void tc_mma_64(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n"
      ".reg .pred p, q, t;\n"
      ".reg .b32 d1, a1, a2, a3, e0, e1, e2, e3;\n"
      ".reg .b64 b1, b2, b3;\n"
      "elect.sync _|q, 0xffffffff;\n"
      "setp.ne.u32 p, %4, 0;\n"
      "setp.eq.u32 t, %3, %3;\n"
      "add.u32 d1, %0, 64;\n"
      "add.u32 a1, %1, 8;\n"
      "add.u32 a2, %1, 16;\n"
      "add.u32 a3, %1, 24;\n"
      "add.u32 e0, %1, 64;\n"
      "add.u32 e1, %1, 72;\n"
      "add.u32 e2, %1, 80;\n"
      "add.u32 e3, %1, 88;\n"
      "add.u64 b1, %2, 2;\n"
      "add.u64 b2, %2, 4;\n"
      "add.u64 b3, %2, 6;\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [d1], [e0], %2, %3, p;\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [d1], [e1], b1, %3, t;\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [d1], [e2], b2, %3, t;\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [d1], [e3], b3, %3, t;\n"
      "}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tc_commit_elected(const uint64_t* bar) {
  asm volatile(
      "{\n"
      ".reg .pred q;\n"
      "elect.sync _|q, 0xffffffff;\n"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n"
      "}" ::"r"(smem_u32(bar))
      : "memory");
}

// 32 registers of each thread -> 32 consecutive columns of its lane.
__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0],"
      " {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16,"
      " %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t dsmem_addr(const void* local_smem, uint32_t rank) {
  uint32_t ra;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(smem_u32(local_smem)), "r"(rank));
  return ra;
}
__device__ __forceinline__ void st_dsmem_f32x4(uint32_t addr, float a, float b, float c, float d) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(a), "f"(b), "f"(c),
               "f"(d)
               : "memory");
}

__device__ __forceinline__ float4 ld_dsmem_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// A wait of at most about a second.  The timer is read only once the first tries have failed: its
// latency would be the ring's.
__device__ __forceinline__ bool tc_wait(const uint64_t* bar, uint32_t parity) {
  const uint32_t b = smem_u32(bar);
  for (int i = 0; i < 128; ++i)
    if (mbar_try_wait(b, parity)) return true;
  return mbar_wait_bounded(b, parity, 1000000000ull, nullptr);
}

struct TcArgs {
  const uint8_t* sf;
  const float* ts;
  int T, tn;        // rows of x, and rounded up to 16
  int64_t N;
  int K;
  int cluster;      // blocks that split K
  int kslice;       // columns of a block, a multiple of 128
  int turns;        // accumulators that the steps take turns on (kTcParts; 1, 2 or 4)
  int parts;        // in which a tile's share of K is worked through (kTcParts)
  int kpart;        // columns of a part, a multiple of 128
  int tiles;        // of 256 weight rows
  bool wide;        // the scales of 128 columns are one aligned load
  void* y;
};

// What a block works through: one tile; several tiles (its rings run on from one to the next); several
// tiles or one, each in parts of its K or with accumulators that take turns (FP32 output of long rows).
// The steps of a block with one tile are 2 to 4% shorter in the kernel for one; a block for each tile
// takes 106 us for 131072 x 4096 at 64 rows (kTcTiles 102), 31.7 for 146704 x 640 at 24 (23.5).
enum TcWork { kTcTile, kTcTiles, kTcParts };
template <bool kMx, bool kF32, TcWork kWork>
__global__ void __launch_bounds__(kTcThreads, 1)
linear_w4_tc_kernel(const __grid_constant__ CUtensorMap tmap_x,
                    const __grid_constant__ CUtensorMap tmap_c, const TcArgs a) {
  constexpr int kBlk = kMx ? 32 : 16;
  constexpr bool kMany = kWork != kTcTile, kParts = kWork == kTcParts;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ uint64_t c_full[kTcCodeStages], c_empty[kTcCodeStages], x_full[kTcXStages],
      x_empty[kTcXStages], a_full[kTcAStages], a_empty[kTcAStages], acc_full, acc_empty, drained;
  __shared__ uint32_t s_tmem, s_issued_x, s_issued_c;
  __shared__ volatile uint32_t s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)blockIdx.x % a.cluster;
  const int first = (int)blockIdx.x / a.cluster;   // tiles first, + gridDim.x, ..
  const int ntile = kMany ? (a.tiles - first + (int)gridDim.x - 1) / (int)gridDim.x : 1;
  auto row0 = [&](int t) { return ((int64_t)first + (int64_t)t * gridDim.x) * kTcRows; };
  // units of work: tiles or their parts
  const int parts = kParts ? a.parts : 1, turns = kParts ? a.turns : 1, nunit = ntile * parts;
  const int kb = rank * a.kslice, ke = min(a.K, kb + a.kslice);
  // steps of 128 columns in a unit; behind K all are zeros
  const int np = parts > 1 ? (kb < a.K ? a.kpart / 128 : 0) : max(0, (ke - kb + 127) / 128);
  const uint32_t x_bytes = (uint32_t)a.tn * 256u;
  uint8_t* x_ring = smem + kTcCodeStages * kTcCodeBytes;
  // Met before the stores into other blocks, which only then need them to have started: a block
  // that holds tensor memory waits for no other block (one that waits for tensor memory on its SM
  // could hold it up).
  if (a.cluster > 1) cluster_arrive();
  if (warp == kTcMmaWarp) {
    tmem_alloc(smem_u32(&s_tmem), kTcCols);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kTcCodeStages; ++i) {
      mbar_init(smem_u32(c_full + i), 1);    // the TMA load (expect_tx)
      mbar_init(smem_u32(c_empty + i), 8);   // the eight warps that read it
    }
    for (int i = 0; i < kTcXStages; ++i) {
      mbar_init(smem_u32(x_full + i), 1);
      mbar_init(smem_u32(x_empty + i), 1);   // the MMA commit
    }
    for (int i = 0; i < kTcAStages; ++i) {
      mbar_init(smem_u32(a_full + i), 8);    // the eight warps that decode it
      mbar_init(smem_u32(a_empty + i), 1);
    }
    mbar_init(smem_u32(&acc_full), 1);              // a tile's MMAs
    mbar_init(smem_u32(&acc_empty), kTcDecWarps);   // its accumulators have been read
    mbar_init(smem_u32(&drained), 1);
    s_issued_x = s_issued_c = 0u;
    s_abort = 0u;
    fence_barrier_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
  griddep_wait();
  griddep_launch();

  // The factors that undo the decoding's power of two, the exact one first where it cannot overflow
  const float ts = kMx ? 4.0f : __ldg(a.ts);
  const bool large = !kMx && fabsf(ts) > 1.0f;
  const float up0 = large ? 256.0f : 1.0f, up = kMx || large ? ts : ts * 256.0f;
  auto store = [&](int t, int64_t n, float v) {
    if (t >= a.T || n >= a.N) return;
    if constexpr (kF32) static_cast<float*>(a.y)[(int64_t)t * a.N + n] = v;
    else static_cast<__nv_bfloat16*>(a.y)[(int64_t)t * a.N + n] = __float2bfloat16_rn(v);
  };
  // A cluster's block sums 256 / cluster of the rows: join[block][row][token], stored by their blocks.
  // Of a tile with parts: this block's sums, [row][token], from which a cluster's blocks load theirs.
  // Rows of tn + 4 words put a warp's 16-byte stores in all banks.
  const int rows = kTcRows / a.cluster, stride = a.tn + 4;
  float* join = reinterpret_cast<float*>(x_ring + kTcXStages * x_bytes);

  if (warp < kTcDecWarps) {
    // ---- decode: one weight row a thread; after a tile's steps its accumulators' store ----
    const int quad = warp & 3, half = (warp >> 2) & 1, set = warp >> 3;
    const int r = half * 128 + quad * 32 + lane;
    auto scales_of = [&](int t) {   // (rows behind the last are not stored)
      return a.sf + min(row0(t) + r, a.N - 1) * (a.K / kBlk);
    };
    const uint8_t* ps = a.sf;
    const uint32_t a_lane = tmem + kTcACol + (uint32_t)half * 64u + ((uint32_t)(quad * 32) << 16);
    const uint8_t* c_lane = smem + r * 64;
    const int swz = (r >> 1) & 3;   // the 64-byte swizzle: a row's chunk index xor (row / 2) % 4
    // The scales of 128 columns: 8 or 4 bytes.  Behind K (where x and the codes are zeros) the row's
    // last ones: a NaN there is the row's anyway.
    uint32_t s[kMx ? 1 : 2];
    int k0 = kb;   // first column of the unit that the scales are loaded of
    auto load_scales = [&](int p) {
      const int at = k0 + p * 128;
      if (a.wide) {
        const uint8_t* q = ps + min(at, a.K - 128) / kBlk;
        if constexpr (kMx) s[0] = __ldg(reinterpret_cast<const uint32_t*>(q));
        else {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(q));
          s[0] = v.x;
          s[1] = v.y;
        }
      } else {
        uint32_t b[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint8_t* q = ps + min(at + u * 32, a.K - 32) / kBlk;
          if constexpr (kMx) b[u] = __ldg(q);
          else b[u] = __ldg(reinterpret_cast<const uint16_t*>(q));
        }
        if constexpr (kMx) s[0] = b[0] | (b[1] << 8) | (b[2] << 16) | (b[3] << 24);
        else {
          s[0] = b[0] | (b[1] << 16);
          s[1] = b[2] | (b[3] << 16);
        }
      }
    };
    bool ok = true;
    // The next unit (`done` before it): lane = weight row, column = token.
    int done = 0;
    auto epilogue = [&]() {
      if (np > 0 && ok) ok = __all_sync(0xffffffffu, tc_wait(&acc_full, (uint32_t)done & 1u));
      tc_fence_after();
      const bool push = a.cluster > 1 && parts == 1;
      if (push) cluster_wait();
      const int part = kParts ? done % parts : 0, t = kParts ? done / parts : done;
      const uint32_t to =
          push ? dsmem_addr(join + (rank * rows + r % rows) * stride, r / rows) : 0u;
      for (int c0 = set * 16; c0 < a.tn; c0 += 48) {
        uint32_t v[16];
        const uint32_t at = tmem + half * 64 + c0 + ((uint32_t)(quad * 32) << 16);
        tmem_ld_32x32b_x16(at, v);
        tmem_ld_wait();
        float f[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = __uint_as_float(v[i]);
        if constexpr (kParts) {
          for (int j = 1; j < min(turns, np); ++j) {
            tmem_ld_32x32b_x16(at + (uint32_t)(j * a.tn), v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) f[i] += __uint_as_float(v[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          f[i] = np == 0 ? 0.0f : f[i] * up0 * up;
          if (!ok) f[i] = __uint_as_float(0x7FC00000u);
        }
        if (push) {
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            st_dsmem_f32x4(to + (uint32_t)(c0 + i) * 4u, f[i], f[i + 1], f[i + 2], f[i + 3]);
        } else {
          if (parts > 1) {
            float4* sum = reinterpret_cast<float4*>(join + r * stride + c0);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (part > 0) {
                const float4 v4 = sum[i];
                f[4 * i] += v4.x;
                f[4 * i + 1] += v4.y;
                f[4 * i + 2] += v4.z;
                f[4 * i + 3] += v4.w;
              }
              if (part < parts - 1 || a.cluster > 1)
                sum[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
            }
          }
          if (part == parts - 1 && a.cluster == 1) {
#pragma unroll
            for (int i = 0; i < 16; ++i) store(c0 + i, row0(t) + r, f[i]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive(smem_u32(&acc_empty));
      ++done;
    };
    int slot = set, cslot = set;
    uint32_t ph = 0u, cph = 0u;
    // this warp's steps are every third of all its block's; unit t, its step p; the next one's
    // scales are loaded a step ahead
    int t = 0, p = 0;
    auto advance = [&](int by) {
      p += by;
      if constexpr (kParts) {
      } else if constexpr (kMany) {
        const int was = t;
        for (; p >= np && t < ntile; ++t) p -= np;
        if (t != was && t < ntile) ps = scales_of(t);
      } else {
        t = p >= np ? 1 : 0;
      }
    };
    if (np > 0) {
      ps = scales_of(0);
      advance(set);
      if (t < nunit) load_scales(p);
    }
    // kParts: unit by unit, so that the loop over steps is that of a single tile
    for (int unit = 0; unit < (kParts ? nunit : 1);) {
      while (np > 0 && (kParts ? p < np && ok : t < nunit)) {
        if constexpr (kWork == kTcTiles) {
          while (done < t) epilogue();
          if (!ok) break;
        }
        uint32_t ss[kMx ? 1 : 2];
#pragma unroll
        for (int u = 0; u < (kMx ? 1 : 2); ++u) ss[u] = s[u];
        advance(3);
        // (behind the last step the last ones again)
        if (kWork != kTcTiles || t < nunit) load_scales(p);
        ok = __all_sync(0xffffffffu, tc_wait(c_full + cslot, cph));
        if (!ok) break;
        const uint8_t* cp = c_lane + cslot * kTcCodeBytes;
        const int cold = cslot;
        cslot += 3;
        if (cslot >= kTcCodeStages) { cslot -= kTcCodeStages; cph ^= 1u; }
        ok = __all_sync(0xffffffffu, tc_wait(a_empty + slot, ph ^ 1u));
        if (!ok) break;
        tc_fence_after();
        // A placed code times its scale: NVFP4 one product (the scale in BF16 times 2^118).  MXFP4 one if
        // the scale times 2^124 is a BF16 (up to 2^3), otherwise (`big`) two.
        auto decode = [&](const bool big) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t out[32];
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              const uint4 w4 = *reinterpret_cast<const uint4*>(cp + (((2 * q + v) ^ swz) << 4));
              const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
              uint32_t sc[2];
              if constexpr (kMx) {
                const uint32_t e = (ss[0] >> ((2 * q + v) * 8)) & 0xFFu;
                sc[0] = sc[1] = !big ? (e + 124u) * 0x00800080u
                                     : e == 255u ? 0x7FC07FC0u : e8m0_scale_bf16x2(e);
              } else {
                const float2 f = e4m3x2_to_f32x2((ss[q] >> (v * 16)) & 0xFFFFu);   // NaN stays NaN
                const __nv_bfloat162 s0 = __float2bfloat162_rn(f.x * 0x1p118f);
                const __nv_bfloat162 s1 = __float2bfloat162_rn(f.y * 0x1p118f);
                sc[0] = *reinterpret_cast<const uint32_t*>(&s0);
                sc[1] = *reinterpret_cast<const uint32_t*>(&s1);
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t o[4];
                e2m1x8_to_bf16x2_scaled_down(w[i], o);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  if (big) o[j] = mul_bf16x2(o[j], kBf16x2Pow2_124);
                  out[v * 16 + i * 4 + j] = mul_bf16x2(o[j], sc[i >> 1]);
                }
              }
            }
            tmem_st_32x32b_x32(a_lane + (uint32_t)slot * 128u + q * 32u, out);
          }
        };
        bool big = false;
        if constexpr (kMx)
          big = __any_sync(0xffffffffu, (ss[0] & ((ss[0] & 0x7F7F7F7Fu) + 0x7D7D7D7Du) & 0x80808080u) != 0u);
        if (kMx && big) decode(true);
        else decode(false);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(c_empty + cold));
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(a_full + slot));
        ph ^= 1u;
      }
      if constexpr (kParts) {
        p -= np;
        if (++unit < nunit) {   // the next unit's first scales come during the epilogue
          ps = scales_of(unit / parts);
          k0 = kb + unit % parts * a.kpart;
          load_scales(p);
        }
        epilogue();
      } else {
        while (done < nunit) epilogue();
        break;
      }
    }
    if (!ok && lane == 0) s_abort = 1u;
  } else if (warp == kTcXWarp || warp == kTcCodeWarp) {
    if (lane == 0) {
      const bool x = warp == kTcXWarp;
      const int stages = x ? kTcXStages : kTcCodeStages;
      uint64_t* full = x ? x_full : c_full;
      uint64_t* empty = x ? x_empty : c_empty;
      int slot = 0;
      uint32_t ph = 0u;
      uint32_t issued = 0u;
      bool ok = true;
      for (int u = 0, t = 0, part = 0; u < nunit && ok; ++u) {
        const int k0 = kb + part * a.kpart;
        for (int i = 0; i < np; ++i) {
          ok = tc_wait(empty + slot, ph ^ 1u);
          if (!ok) break;
          const uint32_t fb = smem_u32(full + slot);
          mbar_arrive_expect_tx(fb, x ? x_bytes : (uint32_t)kTcCodeBytes);
          if (x) {
            const uint32_t to = smem_u32(x_ring) + slot * x_bytes;
            tma_load_2d(to, &tmap_x, k0 + i * 128, 0, fb);
            tma_load_2d(to + x_bytes / 2, &tmap_x, k0 + i * 128 + 64, 0, fb);
          } else {
            tma_load_2d(smem_u32(smem) + slot * kTcCodeBytes, &tmap_c, k0 / 2 + i * 64, (int)row0(t), fb);
          }
          ++issued;
          if (++slot == stages) { slot = 0; ph ^= 1u; }
        }
        if (++part == parts) { part = 0; ++t; }
      }
      if (!ok) s_abort = 1u;
      (x ? s_issued_x : s_issued_c) = issued;
    }
    __syncwarp();
  } else {
    const uint32_t idesc = tc_idesc(a.tn);
    const uint64_t db = smem_desc(smem_u32(x_ring), 16, 1024, kLayoutSwizzle128B);
    int slot = 0, xs = 0;
    uint32_t ph = 0u, xph = 0u;
    bool ok = true;
    for (int t = 0; t < nunit && np > 0 && ok; ++t) {
      ok = __all_sync(0xffffffffu, tc_wait(&acc_empty, ((uint32_t)t & 1u) ^ 1u));
      if (!ok) break;
      tc_fence_after();
      for (int i = 0; i < np; ++i) {
        ok = __all_sync(0xffffffffu, tc_wait(x_full + xs, xph)) &&
             __all_sync(0xffffffffu, tc_wait(a_full + slot, ph));
        if (!ok) break;
        tc_fence_after();
        const uint64_t b0 = db + (uint64_t)((xs * x_bytes) >> 4);
        const uint32_t a0 = tmem + kTcACol + (uint32_t)slot * 128u;
        const uint32_t d = tmem + (kParts ? (uint32_t)(i & (turns - 1)) * (uint32_t)a.tn : 0u);
        tc_mma_64(d, a0, b0, idesc, i >= turns ? 1u : 0u);
        tc_mma_64(d, a0 + 32u, b0 + (x_bytes >> 5), idesc, 1u);
        tc_commit_elected(x_empty + xs);
        tc_commit_elected(a_empty + slot);
        if (++slot == kTcAStages) { slot = 0; ph ^= 1u; }
        if (++xs == kTcXStages) { xs = 0; xph ^= 1u; }
      }
      if (ok) tc_commit_elected(&acc_full);
    }
    if (!ok) {   // the MMAs issued before the wait that ran out
      tc_commit_elected(&drained);
      tc_wait(&drained, 0u);
    }
    if (!ok && lane == 0) s_abort = 1u;
  }

  __syncwarp();
  if (a.cluster > 1 && (warp >= kTcDecWarps || parts > 1)) cluster_wait();
  tc_fence_before();
  __syncthreads();   // every accumulator has been read, every MMA is done (or a wait ran out)
  // After an expired wait TMA loads may still be in flight: the last ring's worth is waited for.
  if (s_abort != 0u && (warp == kTcXWarp || warp == kTcCodeWarp) && lane == 0) {
    const bool x = warp == kTcXWarp;
    const uint32_t n = x ? s_issued_x : s_issued_c, stages = x ? kTcXStages : kTcCodeStages;
    for (uint32_t i = n > stages ? n - stages : 0u; i < n; ++i)
      if (!tc_wait((x ? x_full : c_full) + i % stages, (i / stages) & 1u))
        break;
  }
  if (warp == kTcMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTcCols);
  }
  if (a.cluster > 1) {
    __syncwarp();
    cluster_sync();
    for (int e = threadIdx.x; e < rows * (a.tn / 4); e += kTcThreads) {
      const int r = e % rows, t = e / rows * 4;
      float4 v[8];
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        v[b] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (b >= a.cluster) continue;
        v[b] = parts > 1 ? ld_dsmem_f32x4(dsmem_addr(join + (rank * rows + r) * stride + t, b))
                         : *reinterpret_cast<const float4*>(join + (b * rows + r) * stride + t);
      }
      float4 sum = v[0];
#pragma unroll
      for (int b = 1; b < 8; ++b) {
        sum.x += v[b].x;
        sum.y += v[b].y;
        sum.z += v[b].z;
        sum.w += v[b].w;
      }
      const int64_t n = row0(0) + rank * rows + r;
      store(t, n, sum.x);
      store(t + 1, n, sum.y);
      store(t + 2, n, sum.z);
      store(t + 3, n, sum.w);
    }
    if (parts > 1) cluster_sync();   // (the others have read this block's sums)
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn_linear() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                                     cudaEnableDefault, &q) == cudaSuccess &&
                    q == cudaDriverEntryPointSuccess;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ok ? ptr : nullptr);
  }();
  return fn;
}

// Blocks that split K: while all clusters are resident at once (of 4 blocks 36, of 8 blocks 15 on 152
// SMs: the occupancy query's numbers) and each has two steps.
int tc_cluster(int64_t tiles, int64_t steps) {
  const int most[4] = {num_sms(), num_sms() / 2, num_sms() * 36 / 152, num_sms() * 15 / 152};
  int cluster = 1;
  for (int l = 1; l < 4 && tiles <= most[l] && steps >= 2 << l; ++l) cluster = 1 << l;
  return cluster;
}

// Alignment, the rings of codes and x, and the buffer of a cluster or of a tile's parts.
size_t tc_smem(int tn, bool joins) {
  return 1024 + (size_t)kTcCodeStages * kTcCodeBytes + (size_t)kTcXStages * tn * 256 +
         (joins ? (size_t)(tn + 4) * kTcRows * 4 : 0u);
}

}  // namespace

// From 17 rows always.  From 9 rows where one round of blocks has work for half the SMs, or K is
// short (us, this kernel and the other one at 16 rows: 2048 x 2048 6.1 and 7.4, 18432 x 7168 24 and
// 27, 4096 x 7168 13.2 and 12.0, 131072 x 4096 97 and 78).
bool linear_w4_tc_faster(int T, int64_t N, int K) {
  if (T <= 8 || T > 16) return T > 16;
  const int64_t tiles = (N + kTcRows - 1) / kTcRows;
  return tiles <= num_sms() && (K <= 2048 || 2 * tiles * tc_cluster(tiles, (K + 127) / 128) >= num_sms());
}

cudaError_t launch_linear_w4_tc(const void* x, const uint8_t* codes, const uint8_t* sf,
                                const float* ts, int T, int64_t N, int K, bool f32, void* y,
                                cudaStream_t s) {
  auto encode = encode_fn_linear();
  if (!encode) return cudaErrorNotSupported;
  TcArgs a{sf, ts, T, (T + 15) / 16 * 16, N, K, 1, 0, 1, 1, 0, 0, false, y};
  a.wide = K % 128 == 0 && is_aligned(sf, ts ? 8 : 4);
  CUtensorMap tmap_x, tmap_c;
  const cuuint32_t estr[2] = {1u, 1u};
  {
    const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)T};
    const cuuint64_t strides[1] = {(cuuint64_t)K * 2};
    const cuuint32_t box[2] = {64u, (cuuint32_t)a.tn};   // rows and columns outside are zeros
    if (encode(&tmap_x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(x), dims, strides,
               box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  {
    const cuuint64_t dims[2] = {(cuuint64_t)K / 2, (cuuint64_t)N};
    const cuuint64_t strides[1] = {(cuuint64_t)K / 2};
    const cuuint32_t box[2] = {64u, (cuuint32_t)kTcRows};
    if (encode(&tmap_c, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(codes), dims, strides,
               box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  const int64_t tiles = (N + kTcRows - 1) / kTcRows;
  const int64_t steps = (K + 127) / 128;
  a.cluster = tc_cluster(tiles, steps);
  a.tiles = (int)tiles;
  const int mine = (int)((steps + a.cluster - 1) / a.cluster);
  if (f32 && mine > kTcChain) {   // as many accumulators as needed and as fit into 64 columns, then parts
    while (a.turns * a.tn <= 32 && a.turns * kTcPart < mine) a.turns *= 2;
    a.parts = (mine + kTcPart * a.turns - 1) / (kTcPart * a.turns);
  }
  a.kpart = (mine + a.parts - 1) / a.parts * 128;
  a.kslice = a.kpart * a.parts;   // (whole parts: none reaches into the next block's share)
  auto pick = [&](auto work) {
    constexpr TcWork kWork = decltype(work)::value;
    return ts ? (f32 ? linear_w4_tc_kernel<false, true, kWork> : linear_w4_tc_kernel<false, false, kWork>)
              : (f32 ? linear_w4_tc_kernel<true, true, kWork> : linear_w4_tc_kernel<true, false, kWork>);
  };
  auto kern = tiles > num_sms() ? pick(std::integral_constant<TcWork, kTcTiles>{})
                                : pick(std::integral_constant<TcWork, kTcTile>{});
  if (a.parts > 1 || a.turns > 1)
    kern = ts ? linear_w4_tc_kernel<false, true, kTcParts> : linear_w4_tc_kernel<true, true, kTcParts>;
  const size_t smem = tc_smem(a.tn, a.cluster > 1 || a.parts > 1);
  // (always to the most: another thread's launch may need more than this one's)
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)tc_smem(kTcMaxTokens, true));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.cluster > 1 ? tiles * a.cluster : std::min<int64_t>(tiles, num_sms())));
  cfg.blockDim = dim3(kTcThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)a.cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, tmap_x, tmap_c, a);
}

}  // namespace nvfp4moe
