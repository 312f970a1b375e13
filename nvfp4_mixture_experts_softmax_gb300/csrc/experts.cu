// The experts' products of a BF16 layer that is trained, on rows sorted by expert (segment e: rows
// offsets[e] .. offsets[e+1]):
//   forward      g = x Wg^T, u = x Wu^T, h = bf16(act(g, u)), out = h Wd^T
//   backward     dh = dout Wd, (dg, du) = bf16(dh * act'(g, u)), dx = dg Wg + du Wu
//   weights      dWg = dg^T x, dWu = du^T x, dWd = dout^T h   (FP32)
// One kernel, a mode for each product.  The products accumulate in FP32 in tensor memory, where the tensor cores truncate; the
// row modes leave that as one chain of K / 16 additions, since their results are rounded to BF16 (of K = 4096 0.2% of
// the elements of g and u then round to the other neighbour than the exact sum, 0.035% after FP32 products that round; the
// outputs' error against 64 bits is 1.67e-3 and 1.66e-3).  h, dg and du
// are rounded to BF16 because the tensor cores read them again (and the backward pass as tensors of
// its own), everything else is rounded once, where it is stored.
//
// tcgen05.mma kind::f16 over pairs of CTAs (cta_group::2): a pair computes a tile of 256 x 256, each CTA
// holding 128 rows of A and 128 of B, so that shared memory is written and read half as often as by
// single CTAs with 128 x 256.  Operands come by TMA with the 128-byte swizzle in stages of K = 64, K-major
// where the reduction runs along a row in memory (forward), MN-major where it runs across rows: no
// product transposes anything in memory.  The gate and up products share a tile: CTA 0 brings 128 rows of
// Wg, CTA 1 the same rows of Wu, so that each thread of the epilogue holds g and u of its row.
//
// Tiles of 256 rows of one segment: a tile's rows behind the segment are read and multiplied, but not
// stored (rows do not mix).  In the weights' gradients the rows are the reduction, and a segment's last block has zeros in the
// place of the rows that are not its own, in both operands, brought by the copies as the rows are (WgradMaps below).
//
// What bounds it, device times: with rows enough the tensor cores (one expert, 8192 rows of 4096 x 4096: forward 1.92
// PFLOP/s, gradients of the rows 1.74, of the weights 1.75); 64 experts of uneven size, 65536 rows of 4096 x 1536:
// forward 1.49 ms (1.65 PFLOP/s: an eighth of the row tiles' rows lie behind their segment; 1.70 ms once the power cap
// lowers the clock), weights' gradients 1.95 to 2.0 ms (1.25: 4.8 GB of FP32 results beside the operands' way from L2; 2.09 ms under the power cap),
// added to earlier ones 2.68 ms (the results are read, too); few
// rows an expert: reading the weights (64 tokens to 8 of 128 experts of 2048 x 768 194 us, 6.1 TB/s; one token 27 us;
// gradients of the rows of 8192 tokens to 8 of 256 experts of 2048 x 512 435 us, 5.4 TB/s).
//
// Warps of a CTA: 0-7 epilogue (each a quarter of the rows and half of the columns), 8 and 10 copies (every other
// stage each: a load takes 100 cycles to issue, up to four a stage), 9 tensor memory and, in CTA 0, the MMAs of
// the pair.  Two accumulators (2 x 256 columns) let the epilogue run beside the next tile's products.  Every wait is bounded; one that runs out leaves
// MOE_ERR_DEVICE_TIMEOUT in the status.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "ops.h"

namespace nvfp4moe {

namespace {

enum Mode { kUp, kUpSingle, kDown, kDgradAct, kDgradRows, kWgrad };

constexpr int kTileM = 256, kTileN = 256;       // of a pair
constexpr int kHalf = 128;                      // rows of A and of B a CTA holds
constexpr int kBlockK = 64;
constexpr int kOperandBytes = kHalf * kBlockK * 2;
constexpr int kChunkBytes = kBlockK * 128;      // MN-major: 64 columns (128 bytes) of 64 rows
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kEpiWarps = 8, kCopyWarp = 8, kMmaWarp = 9, kCopyWarp2 = 10;
constexpr int kThreads = 11 * 32;
constexpr int kMaxExperts = 1024;
constexpr int kGroupM = 8;                      // row tiles that are worked through column by column (4, 8, 16: the weights'
                                                // gradients of 64 experts 1974, 1961, 1986 us)
// Rows of the small box.  Of a tile's half that is not full a CTA fetches boxes of so many rows, and zeros in the place of the rows
// behind the segment (boxes of the columns behind the last, from row 0 on: outside the tensor, but not at an address
// outside its memory, as rows behind the last would be): they need less power when they are multiplied, and power is
// what sets the clock under load (64 tokens to 8 of 128 experts 208 and 200 us, 4096 tokens to 8 of 64 experts of 7168 x 2048
// 1980 and 1955 us).  Up to kFewRows rows in all no zeros, and one box where one holds the rows: the time of a few tokens is that of
// their copies' issue (1 token 26.6 us against 34.9, 4 tokens 59.5 against 66.8; from 16 on no difference).
constexpr int kSmallBox = 32;
constexpr int kFewRows = 128;
constexpr uint64_t kLimitNs = 2000000000ull;

// The tensor cores truncate where they add, so the FP32 gradients are cut into chains of about eight blocks (at most
// eleven: 44 additions), of equal length but for one block, which the epilogue adds up in registers, rounding.  A short
// last chain would cost the epilogue as much as a long one.
__device__ __forceinline__ int chain_count(int blocks) { return blocks == 0 ? 0 : max(1, (blocks + 4) / 8); }
__device__ __forceinline__ int chain_blocks(int blocks, int chains, int chain) { return blocks / chains + (chain < blocks % chains); }

// Shared memory: the stages, a slab for each epilogue warp (its 32 rows by 64 or 128 bytes on their way out), barriers,
// segment tables.  The row modes take six stages and 64-byte slabs (1505 us against 1548 for the forward pass of
// 65536 rows of 4096 x 1536), the weights' gradients, whose FP32 output is three quarters of their traffic, five and 128-byte
// slabs (1972 against 2040 us).
template <Mode kMode>
struct Layout {
  static constexpr int kStages = kMode == kWgrad ? 5 : 6;
  static constexpr int kSlabWidth = kMode == kWgrad ? 128 : 64;   // bytes of a row
  static constexpr int kSlabOff = kStages * kStageBytes;
  static constexpr int kBarOff = kSlabOff + kEpiWarps * 32 * kSlabWidth;
  static constexpr int kTableOff = kBarOff + 256;
  static constexpr size_t kBytes = 1024 + kTableOff + 2 * (kMaxExperts + 1) * sizeof(int32_t) + 8;
  static_assert(kBytes <= 232448 && (2 * kStages + 4) * 8 + 12 <= 256, "shared memory");
};

constexpr bool a_mn_major(Mode m) { return m == kWgrad; }
constexpr bool b_mn_major(Mode m) { return m == kDgradAct || m == kDgradRows || m == kWgrad; }

// kind::f16: FP32 accumulator, BF16 operands, their major dimensions (bits 15 and 16: 1 = MN), N / 8, M / 16.
constexpr uint32_t instr_desc(Mode m) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn_major(m) ? 1u : 0u) << 15) |
         ((b_mn_major(m) ? 1u : 0u) << 16) | ((uint32_t)(kTileN >> 3) << 17) | ((uint32_t)(kTileM >> 4) << 24);
}

struct Maps {
  CUtensorMap m[6];     // operands
  CUtensorMap out[3];   // what the epilogue writes, in slabs
};

// The weights' gradients: operands dg, rows, du, dout, h in blocks of 64 rows, and in boxes of 2^i rows for a segment's last
// block.  `have` rows of it are two boxes of the largest 2^i <= have, from the first row and up to the last (one, if
// that is all of them; where they overlap they bring the same), and the zeros behind them are two boxes of zeros alike.
// So a copy reads nothing of the next segment and starts inside its tensor, and only the copy engine writes what the
// pair's products read: at most 16 copies where a full block takes 4.  (Cleared by a warp's stores, whose release
// to the other CTA and acquire cost 1 us an item: 64 experts of 511 rows, 7168 x 2048, 2922 us against 2580.)
constexpr int kHeights = 6;
struct WgradMaps {
  CUtensorMap m[5], part[5][kHeights], zero[kHeights];
  CUtensorMap out[3];
};
template <Mode kMode> struct MapsOf { using T = Maps; };
template <> struct MapsOf<kWgrad> { using T = WgradMaps; };
__device__ const uint4 g_zeros[(1 << (kHeights - 1)) * 8] = {};   // 128 bytes a row

struct Args {
  const int32_t* offsets;
  int32_t* status;
  int E, R;
  int N;          // columns of the output (gate/up: of each)
  int M;          // kWgrad: H and N: I of the down matrix, the other way round for gate and up
  int n_tiles;    // column tiles
  int K;          // columns of A (not kWgrad)
  int nkb;        // blocks of K = 64 of a tile (not kWgrad)
  int half_kb;    // kDgradRows: blocks of the first source
  int nmat;       // kWgrad: 3, or 2 without a gate
  int act;
  float limit, alpha;
  const __nv_bfloat16 *g, *u;            // kDgradAct: the forward pass's
  __nv_bfloat16* o[3];                   // kUp: g, u (may be null), h; kDgradAct: dg, du; else out; as maps.out
  int accumulate;
  int zeros;      // more than kFewRows rows
  int first;      // this launch clears the status
};

struct Tile {
  int seg, m0, rows, n0;   // rows: of the tile (kWgrad: rows of the segment, the reduction)
  int mat, row0;           // kWgrad
};

__device__ __forceinline__ uint32_t leader_addr(uint32_t bar) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(bar));
  return r;
}
// Arrivals on a barrier of either CTA.  Release at CTA scope: what they order are TMA copies, MMAs and reads of
// tensor memory, which complete on their own terms; at cluster scope each arrival would wait for the thread's
// memory accesses (0.8 us a stage of the copies: a third of the rate).  No ordinary store to
// shared memory is read by the other CTA or its MMAs.
__device__ __forceinline__ void arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// As mbar_wait_bounded; gives up as soon as another role of the CTA has.
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, int32_t* status,
                                             volatile uint32_t* abort) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (;;) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    if (global_timer_ns() - t0 > kLimitNs) {
      set_status(status, MOE_ERR_DEVICE_TIMEOUT);
      *abort = 1u;
      return false;
    }
  }
}

// TMA loads into this CTA's shared memory that complete on a barrier of either CTA of the pair, and the arrival that
// announces their bytes; by one elected lane of a converged warp (uniform registers, as for the MMAs: by
// a lane of a diverged one they took 180 cycles each, and four of them a stage set the weight gradients' pace).
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "{\n"
      ".reg .pred q;\n"
      "elect.sync _|q, 0xffffffff;\n"
      "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%2, %3}], [%4];\n"
      "}" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "{\n"
      ".reg .pred q;\n"
      "elect.sync _|q, 0xffffffff;\n"
      "@q cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%2, %3, %4}], [%5];\n"
      "}" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void expect_bytes(uint32_t addr, uint32_t bytes) {
  asm volatile(
      "{\n"
      ".reg .pred q;\n"
      "elect.sync _|q, 0xffffffff;\n"
      "@q mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;\n"
      "}" ::"r"(addr),
      "r"(bytes)
      : "memory");
}

// The MMAs of a block of K = 64 (kStepA, kStepB: 16 of K in units of 16 bytes), and the arrival on `done` in both
// CTAs once they and all before them are complete; by one elected lane of a converged warp, which keeps the
// operands in uniform registers (by a lane of a diverged one each MMA costs 105 cycles to issue, nearly
// the 128 that it runs).
template <uint32_t kStepA, uint32_t kStepB>
__device__ __forceinline__ void mma_block(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate,
                                          uint32_t done) {
  asm volatile(
      "{\n"
      ".reg .pred p, q, t;\n"
      ".reg .b64 a1, a2, a3, b1, b2, b3;\n"
      ".reg .b16 both;\n"
      "elect.sync _|q, 0xffffffff;\n"
      "setp.ne.u32 p, %4, 0;\n"
      "setp.eq.u32 t, %3, %3;\n"
      "mov.b16 both, 3;\n"
      "add.u64 a1, %1, %6;\n"
      "add.u64 a2, a1, %6;\n"
      "add.u64 a3, a2, %6;\n"
      "add.u64 b1, %2, %7;\n"
      "add.u64 b2, b1, %7;\n"
      "add.u64 b3, b2, %7;\n"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], a1, b1, %3, t;\n"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], a2, b2, %3, t;\n"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], a3, b3, %3, t;\n"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%5], both;\n"
      "}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(done), "n"(kStepA), "n"(kStepB)
      : "memory");
}
// The arrival alone, once all MMAs before are complete.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  asm volatile(
      "{\n"
      ".reg .pred q;\n"
      ".reg .b16 both;\n"
      "mov.b16 both, 3;\n"
      "elect.sync _|q, 0xffffffff;\n"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], both;\n"
      "}" ::"r"(bar)
      : "memory");
}

// 32 bytes a thread: whole sectors, although a warp's threads hold different rows.
__device__ __forceinline__ void store_32b(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void load_32b(const void* p, uint32_t* v) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float low_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_bf16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Slabs: a lane writes its row's 64 or 128 bytes (16-byte pieces in the swizzle of that width, so that the lanes' pieces lie in
// different banks), then one lane stores the whole by TMA: whole lines to L2, where 32 bytes a lane and
// row went at 11 bytes a cycle and SM.
template <int kWidth>
__device__ __forceinline__ void slab_put(uint32_t slab, int lane, int piece, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const int at = kWidth == 128 ? piece ^ (lane & 7) : piece ^ ((lane >> 1) & 3);
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(slab + lane * kWidth + (at << 4)), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
// The slab may be written again once the copies before have read it.
__device__ __forceinline__ void slab_begin(int lane) {
  if (lane == 0) bulk_wait_group_read<0>();
  __syncwarp();
}
__device__ __forceinline__ void slab_store_2d(uint32_t slab, int lane, const CUtensorMap* map, int x, int y) {
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x), "r"(y), "r"(slab)
                 : "memory");
    bulk_commit_group();
  }
}
__device__ __forceinline__ void slab_store_3d(uint32_t slab, int lane, const CUtensorMap* map, int x, int y, int z, bool add) {
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    if (add)
      asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x),
                   "r"(y), "r"(z), "r"(slab)
                   : "memory");
    else
      asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x), "r"(y),
                   "r"(z), "r"(slab)
                   : "memory");
    bulk_commit_group();
  }
}

// 32 columns of 32 rows as BF16, `w` two columns a word: by a slab if all 32 rows belong to the segment, else row by
// row (32 bytes a store).
__device__ __forceinline__ void store_bf16x32(const uint32_t (&w)[16], uint32_t slab, int lane, const CUtensorMap* map, int x, int y,
                                              bool whole, __nv_bfloat16* row, bool live) {
  if (whole) {
    slab_begin(lane);
#pragma unroll
    for (int i = 0; i < 4; ++i) slab_put<64>(slab, lane, i, w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    slab_store_2d(slab, lane, map, x, y);
  } else if (live) {
    store_32b(row, w);
    store_32b(row + 16, w + 8);
  }
}

// The activation and its derivatives by g and u, the clamps passing NaN on.  The fast exponential and
// division err by a few 2^-22, far below the BF16 rounding that follows; a very negative argument's
// denominator overflows and the sigmoid is 0.
__device__ __forceinline__ float clamp_up(float v, float L) { return v > L ? L : v; }
__device__ __forceinline__ float clamp_both(float v, float L) { return v > L ? L : v < -L ? -L : v; }

__device__ __forceinline__ float activation(float g, float u, int act, float L, float alpha) {
  if (act == kActRelu2) return u <= 0.0f ? 0.0f : u * u;
  if (act != kActSwiglu) {
    g = clamp_up(g, L);
    u = clamp_both(u, L);
  }
  if (act == kActSwigluOai) return (u + 1.0f) * __fdividef(g, 1.0f + __expf(-(alpha * g)));
  return __fdividef(g, 1.0f + __expf(-g)) * u;
}

__device__ __forceinline__ void activation_grad(float g, float u, float dh, int act, float L, float alpha, float& dg,
                                                float& du) {
  if (act == kActRelu2) {
    dg = 0.0f;
    du = u <= 0.0f ? 0.0f : dh * (2.0f * u);
    return;
  }
  float gc = g, uc = u, a = 1.0f;
  if (act != kActSwiglu) {
    gc = clamp_up(g, L);
    uc = clamp_both(u, L);
  }
  if (act == kActSwigluOai) {
    a = alpha;
    uc += 1.0f;
  }
  const float s = __fdividef(1.0f, 1.0f + __expf(-(a * gc)));
  dg = dh * (uc * (s * (1.0f + a * gc * (1.0f - s))));
  du = dh * (gc * s);
  if (act != kActSwiglu) {   // the clamps' gradient is 0 beyond them, 1 at them
    if (g > L) dg = 0.0f;
    if (fabsf(u) > L) du = 0.0f;
  }
}

template <Mode kMode>
__device__ __forceinline__ Tile tile_at(const Args& p, const int32_t* s_off, const int32_t* s_tile, int item) {
  constexpr int kCols = kMode == kUp ? kHalf : kTileN;
  Tile t;
  int mt, local;   // row tiles of the group's matrix, item within it
  if constexpr (kMode == kWgrad) {
    const int mh = (p.M + kTileM - 1) / kTileM, ni = (p.N + kTileN - 1) / kTileN;   // of H and of I
    const int per = mh * ni;
    const int sm = item / per;
    local = item - sm * per;
    t.seg = sm / p.nmat;
    t.mat = sm - t.seg * p.nmat + 3 - p.nmat;    // 0 gate, 1 up, 2 down
    mt = t.mat == 2 ? mh : ni;
    t.row0 = s_off[t.seg];
    t.rows = s_off[t.seg + 1] - t.row0;
  } else {
    int lo = 0, hi = p.E - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_tile[mid] * p.n_tiles <= item) lo = mid;
      else hi = mid - 1;
    }
    t.seg = lo;
    t.mat = 0;
    mt = s_tile[lo + 1] - s_tile[lo];
    local = item - s_tile[lo] * p.n_tiles;
  }
  const int n_tiles = kMode == kWgrad ? (t.mat == 2 ? (p.N + kTileN - 1) / kTileN : (p.M + kTileN - 1) / kTileN) : p.n_tiles;
  // kGroupM row tiles by all columns, rows fastest: the pairs that run at the same time share both operands
  const int grp = local / (kGroupM * n_tiles);
  const int rem = local - grp * kGroupM * n_tiles;
  const int gm = min(kGroupM, mt - grp * kGroupM);
  const int nt = rem / gm;
  const int m = grp * kGroupM + rem - nt * gm;
  t.n0 = nt * kCols;
  if constexpr (kMode == kWgrad) {
    t.m0 = m * kTileM;
  } else {
    t.m0 = s_off[t.seg] + m * kTileM;
    t.rows = min(kTileM, s_off[t.seg + 1] - t.m0);
    t.row0 = 0;
  }
  return t;
}

// Rows of the segment that an item's reduction runs over (kWgrad), all that the MMA warp needs to know.
template <Mode kMode>
__device__ __forceinline__ int reduction_rows(const Args& p, const int32_t* s_off, int item) {
  if (kMode != kWgrad) return 0;
  const int seg = item / (p.nmat * ((p.M + kTileM - 1) / kTileM) * ((p.N + kTileN - 1) / kTileN));
  return s_off[seg + 1] - s_off[seg];
}

template <Mode kMode>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    experts_kernel(const __grid_constant__ typename MapsOf<kMode>::T maps, const __grid_constant__ Args p) {
  using L = Layout<kMode>;
  constexpr int kStages = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBarOff);   // [stage], CTA 0's: both CTAs' data has landed
  uint64_t* empty = full + kStages;                               // [stage]: the MMAs have read it
  uint64_t* acc_full = empty + kStages;                           // [2]
  uint64_t* acc_empty = acc_full + 2;                             // [2], CTA 0's
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
  volatile uint32_t* s_abort = tmem_slot + 1;
  int32_t* s_bad = reinterpret_cast<int32_t*>(tmem_slot + 2);
  int32_t* s_off = reinterpret_cast<int32_t*>(smem + L::kTableOff);
  int32_t* s_tile = s_off + kMaxExperts + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(full + s), 2);    // one arrival of each CTA, and the bytes
      mbar_init(smem_u32(empty + s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(acc_full + b), 1);
      mbar_init(smem_u32(acc_empty + b), 2 * kEpiWarps);
    }
    *s_abort = 0u;
    *s_bad = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  griddep_wait();
  griddep_launch();
  for (int i = threadIdx.x; i <= p.E; i += kThreads) s_off[i] = p.offsets[i];
  __syncthreads();
  // offsets that do not ascend within the rows: no work, and the status says so
  for (int i = threadIdx.x; i < p.E; i += kThreads)
    if (s_off[i] < 0 || s_off[i + 1] < s_off[i] || s_off[i + 1] > p.R) *s_bad = 1;
  __syncthreads();
  const bool bad = *s_bad != 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (p.first) *p.status = bad ? MOE_ERR_INVALID_ARG : MOE_OK;
  }
  if (kMode != kWgrad && warp == 0 && !bad) {
    // row tiles before each segment: lane l takes a run of segments
    const int per = (p.E + 31) / 32, s0 = min(lane * per, p.E), s1 = min(s0 + per, p.E);
    int c = 0;
    for (int i = s0; i < s1; ++i) c += (s_off[i + 1] - s_off[i] + kTileM - 1) / kTileM;
    int incl = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    int off = incl - c;
    for (int i = s0; i < s1; ++i) {
      s_tile[i] = off;
      off += (s_off[i + 1] - s_off[i] + kTileM - 1) / kTileM;
    }
    if (lane == 31) s_tile[p.E] = incl;
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // the pair's barriers are ready
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t smem0 = smem_u32(smem);
  int total = 0;
  if (!bad)
    total = kMode == kWgrad ? p.E * p.nmat * ((p.M + kTileM - 1) / kTileM) * ((p.N + kTileN - 1) / kTileN)
                            : s_tile[p.E] * p.n_tiles;
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;   // pairs

  // blocks of K = 64 of an item, its chains, and the blocks of one of them
  auto blocks_of = [&](int rows) { return kMode == kWgrad ? (rows + kBlockK - 1) / kBlockK : p.nkb; };
  auto chains_of = [&](int blocks) { return kMode == kWgrad ? chain_count(blocks) : 1; };
  auto part_of = [&](int blocks, int chains, int ch) { return kMode == kWgrad ? chain_blocks(blocks, chains, ch) : blocks; };

  if (warp == kCopyWarp || warp == kCopyWarp2) {
    // ---------------- copies ----------------
    const uint32_t full0 = leader_addr(smem_u32(full));
    uint32_t st = 0, ph = 0, mine_next = warp == kCopyWarp ? 1u : 0u, filled = 0;   // filled: stages, at most all
    bool ok = true;
    for (int item = first; item < total && ok; item += step) {
      const Tile t = tile_at<kMode>(p, s_off, s_tile, item);
      // what of the tile this CTA brings: rows (columns) m of A, n of B, `na`, `nb` chunks of 64 of them
      const int Mm = kMode != kWgrad ? 0 : t.mat == 2 ? p.M : p.N, Nn = kMode != kWgrad ? p.N : t.mat == 2 ? p.N : p.M;
      const int m = t.m0 + (int)rank * kHalf, n = kMode == kUp ? t.n0 : t.n0 + (int)rank * kHalf;
      const int na = m >= Mm ? 0 : m + 64 >= Mm ? 1 : 2, nb = n >= Nn ? 0 : n + 64 >= Nn ? 1 : 2;
      const int mine = t.rows - (int)rank * kHalf;
      const bool part = kMode != kWgrad && mine < kHalf, zeros = part && p.zeros;
      const uint32_t abytes = kMode == kWgrad ? (uint32_t)na * kChunkBytes
                              : !part || zeros ? (uint32_t)kOperandBytes
                              : mine <= 0 ? 0u : mine <= kSmallBox ? kSmallBox * 128u : (uint32_t)kOperandBytes;
      const uint32_t bytes = abytes + (b_mn_major(kMode) ? (uint32_t)nb * kChunkBytes : nb ? (uint32_t)kOperandBytes : 0u);
      const bool small = part && mine > 0 && (zeros || mine <= kSmallBox);
      const int ia = kMode == kWgrad ? (t.mat == 0 ? 0 : t.mat == 1 ? 2 : 3) : small ? 3 : 0;
      const int ib = kMode == kWgrad ? (t.mat == 2 ? 4 : 1) : kMode == kUp && rank == 1 ? 2 : 1;
      const CUtensorMap *ma = maps.m + ia, *mb = maps.m + ib;
      const int nkb = blocks_of(t.rows);
      for (int kb = 0; kb < nkb; ++kb, mine_next ^= 1u, st = st + 1 == kStages ? 0 : st + 1, ph ^= st == 0) {
        filled = min(filled + 1, (uint32_t)kStages);
        if (kMode == kDgradRows && kb == p.half_kb) {   // the second source
          ma = maps.m + (small ? 5 : 2);
          mb = maps.m + 4;
        }
        if (!mine_next) continue;
        ok = __all_sync(0xffffffffu, wait_bounded(smem_u32(empty + st), ph ^ 1u, p.status, s_abort));
        if (!ok) break;
        const uint32_t a = smem0 + st * kStageBytes, b = a + kOperandBytes;
        const uint32_t bar = full0 + 8 * st;
        if constexpr (kMode == kWgrad) {
          const int done = kb * kBlockK, row = t.row0 + done, have = t.rows - done;
          if (have >= kBlockK) {
            expect_bytes(bar, bytes);
            if (na > 0) load_2d(a, ma, m, row, bar);
            if (na > 1) load_2d(a + kChunkBytes, ma, m + 64, row, bar);
            if (nb > 0) load_2d(b, mb, n, row, bar);
            if (nb > 1) load_2d(b + kChunkBytes, mb, n + 64, row, bar);
          } else {
            const int lv = 31 - __clz(have), lz = 31 - __clz(kBlockK - have), hv = 1 << lv, hz = 1 << lz;
            const bool v2 = have > hv, z2 = kBlockK - have > hz;
            expect_bytes(bar, (uint32_t)((na + nb) * ((v2 ? 2 * hv : hv) + (z2 ? 2 * hz : hz)) * 128));
            auto last_block = [&](uint32_t to, const CUtensorMap* map, int x) {
              load_2d(to, map, x, row, bar);
              if (v2) load_2d(to + (have - hv) * 128, map, x, row + have - hv, bar);
              load_2d(to + have * 128, maps.zero + lz, 0, 0, bar);
              if (z2) load_2d(to + (kBlockK - hz) * 128, maps.zero + lz, 0, 0, bar);
            };
            if (na > 0) last_block(a, maps.part[ia] + lv, m);
            if (na > 1) last_block(a + kChunkBytes, maps.part[ia] + lv, m + 64);
            if (nb > 0) last_block(b, maps.part[ib] + lv, n);
            if (nb > 1) last_block(b + kChunkBytes, maps.part[ib] + lv, n + 64);
          }
        } else {
          int k0 = kb * kBlockK;
          if (kMode == kDgradRows && kb >= p.half_kb) k0 -= p.half_kb * kBlockK;
          expect_bytes(bar, bytes);
          if (zeros && mine > 0) {
#pragma unroll
            for (int i = 0; i < kHalf / kSmallBox; ++i)
              load_2d(a + i * kSmallBox * 128, ma, i * kSmallBox < mine ? k0 : p.K, i * kSmallBox < mine ? m + i * kSmallBox : 0, bar);
          } else if (abytes) {
            load_2d(a, ma, mine > 0 ? k0 : p.K, mine > 0 ? m : 0, bar);
          }
          if constexpr (b_mn_major(kMode)) {
            if (nb > 0) load_3d(b, mb, n, k0, t.seg, bar);
            if (nb > 1) load_3d(b + kChunkBytes, mb, n + 64, k0, t.seg, bar);
          } else {
            if (nb > 0) load_3d(b, mb, k0, n, t.seg, bar);
          }
        }
      }
    }
    // The MMAs' arrivals on this CTA's barriers have to come before it may end: each warp waits for the stages that it
    // filled last (d blocks ago), which nobody fills again.
    for (uint32_t d = 1; d <= filled && ok; ++d) {
      if (((d & 1u) ? mine_next ^ 1u : mine_next) == 0u) continue;
      const uint32_t s = st >= d ? st - d : st + kStages - d;
      ok = __all_sync(0xffffffffu, wait_bounded(smem_u32(empty + s), st >= d ? ph : ph ^ 1u, p.status, s_abort));
    }
  } else if (warp == kMmaWarp) {
    // ---------------- products (CTA 0) ----------------
    if (rank == 0) {
      constexpr uint32_t idesc = instr_desc(kMode);
      const uint64_t da0 = smem_desc(smem0, a_mn_major(kMode) ? kChunkBytes : 16, 1024, kLayoutSwizzle128B);
      const uint64_t db0 = smem_desc(smem0 + kOperandBytes, b_mn_major(kMode) ? kChunkBytes : 16, 1024, kLayoutSwizzle128B);
      uint32_t st = 0, ph = 0, unit = 0;
      bool ok = true;
      for (int item = first; item < total && ok; item += step) {
        const int blocks = blocks_of(reduction_rows<kMode>(p, s_off, item)), nch = chains_of(blocks);
        for (int ch = 0; ch < nch && ok; ++ch, ++unit) {
          const int nkb = part_of(blocks, nch, ch);
          const uint32_t buf = unit & 1u;
          ok = __all_sync(0xffffffffu, wait_bounded(smem_u32(acc_empty + buf), ((unit >> 1) & 1u) ^ 1u, p.status, s_abort));
          if (!ok) break;
          tc_fence_after();
          for (int kb = 0; kb < nkb; ++kb) {
            ok = __all_sync(0xffffffffu, wait_bounded(smem_u32(full + st), ph, p.status, s_abort));
            if (!ok) break;
            tc_fence_after();
            const uint64_t so = (uint64_t)(st * (kStageBytes >> 4));
            mma_block<a_mn_major(kMode) ? 128u : 2u, b_mn_major(kMode) ? 128u : 2u>(tmem + buf * kTileN, da0 + so, db0 + so, idesc,
                                                                                    kb != 0 ? 1u : 0u, smem_u32(empty + st));
            if (++st == kStages) { st = 0; ph ^= 1u; }
          }
          if (ok) commit_pair(smem_u32(acc_full + buf));
        }
      }
    }
  } else {
    // ---------------- epilogue: a row a thread, half of the columns a warp ----------------
    const int quad = warp & 3, half = warp >> 2;
    const int slab_row = (int)rank * kHalf + quad * 32;       // first of the warp's rows of the tile
    const uint32_t slab = smem0 + L::kSlabOff + warp * 32 * L::kSlabWidth;
    uint32_t unit = 0;
    bool ok = true;
    for (int item = first; item < total && ok; item += step) {
      const Tile t = tile_at<kMode>(p, s_off, s_tile, item);
      if constexpr (kMode == kWgrad) {
        // the chains' sums meet in registers: 128 columns a thread
        float sum[kHalf];
        const int nch = chains_of(blocks_of(t.rows));
        for (int ch = 0; ch < nch && ok; ++ch, ++unit) {
          const uint32_t buf = unit & 1u;
          ok = __all_sync(0xffffffffu, wait_bounded(smem_u32(acc_full + buf), (unit >> 1) & 1u, p.status, s_abort));
          if (!ok) break;
          tc_fence_after();
          const uint32_t acc = tmem + buf * kTileN + half * kHalf + ((uint32_t)(quad * 32) << 16);
#pragma unroll
          for (int c = 0; c < kHalf / 16; ++c) {
            uint32_t v[16];
            tmem_ld_32x32b_x16(acc + c * 16, v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) sum[c * 16 + i] = ch == 0 ? __uint_as_float(v[i]) : sum[c * 16 + i] + __uint_as_float(v[i]);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_cluster(leader_addr(smem_u32(acc_empty + buf)));
        }
        if (!ok) break;
        const int Mm = t.mat == 2 ? p.M : p.N, Nn = t.mat == 2 ? p.N : p.M;
        if (t.m0 + slab_row >= Mm || (nch == 0 && p.accumulate)) continue;   // (32 rows: all of them or none)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int col = t.n0 + half * kHalf + c * 32;
          if (col >= Nn) break;
          slab_begin(lane);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float* f = sum + c * 32 + 4 * i;
            if (nch == 0) slab_put<128>(slab, lane, i, 0u, 0u, 0u, 0u);   // a segment without rows
            else slab_put<128>(slab, lane, i, __float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
          }
          slab_store_3d(slab, lane, maps.out + t.mat, col, t.m0 + slab_row, t.seg, p.accumulate);
        }
      } else {
        constexpr int kGroups = kMode == kUp ? 2 : 4;    // of 32 columns a warp
        const bool any = slab_row < t.rows, live = slab_row + lane < t.rows, whole = slab_row + 32 <= t.rows;
        const int y = t.m0 + slab_row, col0 = half * kGroups * 32;
        const size_t row = (size_t)(y + lane) * p.N;
        // kDgradAct: g and u, read two groups ahead, the first two before the products are there (read when they are
        // needed, eight waits of a load each made the epilogue as long as the products)
        uint32_t gu[kMode == kDgradAct ? 2 : 1][32];
        auto read_gu = [&](int k, uint32_t (&to)[32]) {
          const int x = t.n0 + col0 + 32 * k;
          if (!live || x >= p.N) return;
          if (p.g) {
            load_32b(p.g + row + x, to);
            load_32b(p.g + row + x + 16, to + 8);
          }
          load_32b(p.u + row + x, to + 16);
          load_32b(p.u + row + x + 16, to + 24);
        };
        if constexpr (kMode == kDgradAct) {
          read_gu(0, gu[0]);
          read_gu(1, gu[1]);
        }
        const uint32_t buf = unit & 1u;
        ok = __all_sync(0xffffffffu, wait_bounded(smem_u32(acc_full + buf), (unit >> 1) & 1u, p.status, s_abort));
        if (!ok) break;
        ++unit;
        tc_fence_after();
        const uint32_t acc = tmem + buf * kTileN + col0 + ((uint32_t)(quad * 32) << 16);
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
          const int x = t.n0 + col0 + 32 * k;
          if (!any || x >= p.N) break;
          uint32_t w0[16], w1[16], w2[16];
#pragma unroll
          for (int q = 0; q < 2; ++q) {      // 16 columns at a time
            uint32_t v[16], vu[16];
            tmem_ld_32x32b_x16(acc + 32 * k + 16 * q, v);
            if constexpr (kMode == kUp) tmem_ld_32x32b_x16(acc + kHalf + 32 * k + 16 * q, vu);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float a = __uint_as_float(v[2 * i]), b = __uint_as_float(v[2 * i + 1]);
              const int o = 8 * q + i;
              if constexpr (kMode == kUp) {
                const float ua = __uint_as_float(vu[2 * i]), ub = __uint_as_float(vu[2 * i + 1]);
                w0[o] = pack2(a, b);
                w1[o] = pack2(ua, ub);
                w2[o] = pack2(activation(a, ua, p.act, p.limit, p.alpha), activation(b, ub, p.act, p.limit, p.alpha));
              } else if constexpr (kMode == kUpSingle) {
                w1[o] = pack2(a, b);
                w2[o] = pack2(activation(0.0f, a, kActRelu2, 0.0f, 0.0f), activation(0.0f, b, kActRelu2, 0.0f, 0.0f));
              } else if constexpr (kMode == kDgradAct) {
                const uint32_t gw = gu[k & 1][o], uw = gu[k & 1][16 + o];
                float ga, gb, ua, ub;
                activation_grad(low_bf16(gw), low_bf16(uw), a, p.act, p.limit, p.alpha, ga, ua);
                activation_grad(high_bf16(gw), high_bf16(uw), b, p.act, p.limit, p.alpha, gb, ub);
                w0[o] = pack2(ga, gb);
                w1[o] = pack2(ua, ub);
              } else {
                w0[o] = pack2(a, b);
              }
            }
          }
          if constexpr (kMode == kDgradAct)
            if (k + 2 < kGroups) read_gu(k + 2, gu[k & 1]);
          if (kMode != kUpSingle && p.o[0]) store_bf16x32(w0, slab, lane, maps.out, x, y, whole, p.o[0] + row + x, live);
          if (kMode <= kUpSingle || kMode == kDgradAct)
            if (p.o[1]) store_bf16x32(w1, slab, lane, maps.out + 1, x, y, whole, p.o[1] + row + x, live);
          if (kMode <= kUpSingle) store_bf16x32(w2, slab, lane, maps.out + 2, x, y, whole, p.o[2] + row + x, live);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(leader_addr(smem_u32(acc_empty + buf)));
      }
    }
    if (lane == 0) bulk_wait_group<0>();   // the slabs' copies, before the CTA may end
  }

  // After a wait ran out, copies into shared memory and MMAs may still be under way: they end within
  // microseconds, the CTA stays ten milliseconds.
  __syncwarp();
  if (*s_abort) {
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 10000000ull) __nanosleep(10000);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // no arrival and no MMA of the pair is under way towards either CTA
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      ptr = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }();
  return fn;
}

// [d2][d1][d0] (d2 = 0: two dimensions) of BF16, or FP32 if kSize is 4; boxes of `width` bytes by `rows`, swizzled.
template <int kSize = 2>
bool make_map(CUtensorMap* m, const void* ptr, int64_t d0, int64_t d1, int64_t d2, int rows, int width = 128) {
  const cuuint64_t dims[3] = {(cuuint64_t)d0, (cuuint64_t)d1, (cuuint64_t)d2};
  const cuuint64_t strides[2] = {(cuuint64_t)d0 * kSize, (cuuint64_t)d0 * d1 * kSize};
  const cuuint32_t box[3] = {(cuuint32_t)(width / kSize), (cuuint32_t)rows, 1}, estr[3] = {1, 1, 1};
  return encoder()(m, kSize == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, d2 ? 3 : 2, const_cast<void*>(ptr), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, width == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <Mode kMode>
cudaError_t launch(const typename MapsOf<kMode>::T& maps, const Args& a, int64_t most_items, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(experts_kernel<kMode>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<kMode>::kBytes);
  if (e != cudaSuccess) return e;
  const int pairs = (int)std::max<int64_t>(1, std::min<int64_t>(most_items, num_sms() / 2));
  return launch_pdl(experts_kernel<kMode>, dim3(2 * pairs), dim3(kThreads), Layout<kMode>::kBytes, s, maps, a);
}

int div_up(int64_t a, int b) { return (int)((a + b - 1) / b); }

// What the three entry points have in common.
struct Shape {
  int64_t R, H, I;
  int E, act;
  bool gated;
};

int check_shape(const int32_t* offsets, int64_t R, int32_t E, int64_t H, int64_t I, uint32_t flags, float limit, float alpha,
                const void* ws, size_t ws_bytes, size_t need, Shape& sh) {
  if (R < 0 || E < 1 || H < 1 || I < 1 || H % 32 || I % 32) return MOE_ERR_INVALID_ARG;
  const uint32_t acts = MOE_FLAG_SWIGLU_CLAMP | MOE_FLAG_ACT_RELU2 | MOE_FLAG_ACT_SWIGLU_OAI;
  if (flags & ~acts) return MOE_ERR_INVALID_ARG;
  sh.act = flags == 0 ? kActSwiglu
           : flags == MOE_FLAG_SWIGLU_CLAMP ? kActSwigluClamp
           : flags == MOE_FLAG_ACT_RELU2 ? kActRelu2
           : flags == MOE_FLAG_ACT_SWIGLU_OAI ? kActSwigluOai : -1;
  if (sh.act < 0) return MOE_ERR_INVALID_ARG;
  if ((sh.act == kActSwigluClamp || sh.act == kActSwigluOai) && !(std::isfinite(limit) && limit >= 0.0f)) return MOE_ERR_INVALID_ARG;
  if (sh.act == kActSwigluOai && !std::isfinite(alpha)) return MOE_ERR_INVALID_ARG;
  if (E > kMaxExperts || R > INT32_MAX - kTileM || H > (1 << 16) || I > (1 << 16)) return MOE_ERR_UNSUPPORTED_SHAPE;
  // tiles are counted in 32 bits, with room for a pair's next one
  const int64_t cols = std::max(H, I) / kHalf + 1;
  if ((R / kTileM + E) * cols > 1 << 30 || 3 * (int64_t)E * cols * cols > 1 << 30) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!ws || ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (!is_aligned(ws, 256) || !offsets || !is_aligned(offsets, 4)) return MOE_ERR_INVALID_ARG;
  sh.R = R;
  sh.H = H;
  sh.I = I;
  sh.E = E;
  sh.gated = sh.act != kActRelu2;
  return MOE_OK;
}

Args base_args(const Shape& sh, const int32_t* offsets, void* ws, float limit, float alpha) {
  Args a = {};
  a.offsets = offsets;
  a.status = static_cast<int32_t*>(ws);
  a.E = sh.E;
  a.R = (int)sh.R;
  a.act = sh.act;
  a.zeros = sh.R > kFewRows;
  a.limit = limit;
  a.alpha = alpha;
  return a;
}

int64_t row_items(const Shape& sh, int n_tiles) { return (sh.R / kTileM + std::min<int64_t>(sh.E, sh.R)) * n_tiles; }

// The row modes' outputs [R, cols], null: not written.
bool row_outputs(Maps& m, Args& a, int64_t R, int64_t cols, void* o0, void* o1, void* o2) {
  void* const o[3] = {o0, o1, o2};
  for (int i = 0; i < 3; ++i) {
    a.o[i] = static_cast<__nv_bfloat16*>(o[i]);
    if (o[i] && !make_map(&m.out[i], o[i], cols, R, 0, 32, 64)) return false;
  }
  return true;
}

constexpr size_t kHeader = 256;   // the status

}  // namespace
}  // namespace nvfp4moe

using namespace nvfp4moe;

extern "C" {

size_t moe_experts_workspace_size(int64_t R, int64_t I) {
  if (R < 0 || I < 0 || R > INT32_MAX || I > (1 << 16)) return 0;
  return kHeader + align_up((size_t)R * (size_t)I * 2);
}

int moe_experts_forward(const void* rows, const int32_t* offsets, int64_t R, int32_t E, int64_t H, int64_t I,
                        const void* w_gate, const void* w_up, const void* w_down, uint32_t flags, float swiglu_limit,
                        float swiglu_alpha, void* g, void* u, void* h, void* out, void* workspace, size_t ws_bytes,
                        moe_stream_t stream) {
  Shape sh;
  const int st = check_shape(offsets, R, E, H, I, flags, swiglu_limit, swiglu_alpha, workspace, ws_bytes,
                             h || R < 0 || I < 0 ? kHeader : moe_experts_workspace_size(R, I), sh);
  if (st != MOE_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (R == 0) return cudaMemsetAsync(workspace, 0, sizeof(int32_t), s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  if (!rows || !w_up || !w_down || !out || (sh.gated && !w_gate)) return MOE_ERR_INVALID_ARG;
  if (sh.gated ? (g == nullptr) != (u == nullptr) : g != nullptr) return MOE_ERR_INVALID_ARG;
  for (const void* p : {rows, sh.gated ? w_gate : nullptr, w_up, w_down})
    if (!is_aligned(p, 16)) return MOE_ERR_INVALID_ARG;
  for (const void* p : {g, u, h, out})
    if (!is_aligned(p, 32)) return MOE_ERR_INVALID_ARG;
  if (!encoder()) return MOE_ERR_CUDA;
  void* hb = h ? h : static_cast<uint8_t*>(workspace) + kHeader;
  Maps m = {};
  Args a = base_args(sh, offsets, workspace, swiglu_limit, swiglu_alpha);
  bool ok = make_map(&m.m[0], rows, H, R, 0, kHalf) && make_map(&m.m[3], rows, H, R, 0, kSmallBox) &&
            make_map(&m.m[1], sh.gated ? w_gate : w_up, H, I, E, kHalf) && make_map(&m.m[2], w_up, H, I, E, kHalf);
  if (!ok) return MOE_ERR_CUDA;
  a.N = (int)I;
  a.K = (int)H;
  a.nkb = div_up(H, kBlockK);
  a.n_tiles = div_up(I, sh.gated ? kHalf : kTileN);
  if (!row_outputs(m, a, R, I, g, u, hb)) return MOE_ERR_CUDA;
  a.first = 1;
  cudaError_t e = sh.gated ? launch<kUp>(m, a, row_items(sh, a.n_tiles), s) : launch<kUpSingle>(m, a, row_items(sh, a.n_tiles), s);
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  ok = make_map(&m.m[0], hb, I, R, 0, kHalf) && make_map(&m.m[3], hb, I, R, 0, kSmallBox) &&
       make_map(&m.m[1], w_down, I, H, E, kHalf);
  if (!ok) return MOE_ERR_CUDA;
  a.N = (int)H;
  a.K = (int)I;
  a.nkb = div_up(I, kBlockK);
  a.n_tiles = div_up(H, kTileN);
  if (!row_outputs(m, a, R, H, out, nullptr, nullptr)) return MOE_ERR_CUDA;
  a.first = 0;
  return launch<kDown>(m, a, row_items(sh, a.n_tiles), s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int moe_experts_backward(const void* dout, const int32_t* offsets, int64_t R, int32_t E, int64_t H, int64_t I,
                         const void* w_gate, const void* w_up, const void* w_down, uint32_t flags, float swiglu_limit,
                         float swiglu_alpha, const void* g, const void* u, void* dg, void* du, void* drows, void* workspace,
                         size_t ws_bytes, moe_stream_t stream) {
  Shape sh;
  const int st = check_shape(offsets, R, E, H, I, flags, swiglu_limit, swiglu_alpha, workspace, ws_bytes, kHeader, sh);
  if (st != MOE_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (R == 0) return cudaMemsetAsync(workspace, 0, sizeof(int32_t), s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  if (!dout || !w_up || !w_down || !u || !du || !drows) return MOE_ERR_INVALID_ARG;
  if (sh.gated ? !w_gate || !g || !dg : g || dg) return MOE_ERR_INVALID_ARG;
  for (const void* p : {dout, sh.gated ? w_gate : nullptr, w_up, w_down})
    if (!is_aligned(p, 16)) return MOE_ERR_INVALID_ARG;
  for (const void* p : {g, u, (const void*)dg, (const void*)du, (const void*)drows})
    if (!is_aligned(p, 32)) return MOE_ERR_INVALID_ARG;
  if (!encoder()) return MOE_ERR_CUDA;
  Maps m = {};
  Args a = base_args(sh, offsets, workspace, swiglu_limit, swiglu_alpha);
  bool ok = make_map(&m.m[0], dout, H, R, 0, kHalf) && make_map(&m.m[3], dout, H, R, 0, kSmallBox) &&
            make_map(&m.m[1], w_down, I, H, E, kBlockK);
  if (!ok) return MOE_ERR_CUDA;
  a.N = (int)I;
  a.K = (int)H;
  a.nkb = div_up(H, kBlockK);
  a.n_tiles = div_up(I, kTileN);
  a.g = static_cast<const __nv_bfloat16*>(g);
  a.u = static_cast<const __nv_bfloat16*>(u);
  if (!row_outputs(m, a, R, I, dg, du, nullptr)) return MOE_ERR_CUDA;
  a.first = 1;
  if (launch<kDgradAct>(m, a, row_items(sh, a.n_tiles), s) != cudaSuccess) return MOE_ERR_CUDA;
  const void* first = sh.gated ? dg : du;
  ok = make_map(&m.m[0], first, I, R, 0, kHalf) && make_map(&m.m[3], first, I, R, 0, kSmallBox) &&
       make_map(&m.m[1], sh.gated ? w_gate : w_up, H, I, E, kBlockK) && make_map(&m.m[2], du, I, R, 0, kHalf) &&
       make_map(&m.m[5], du, I, R, 0, kSmallBox) && make_map(&m.m[4], w_up, H, I, E, kBlockK);
  if (!ok) return MOE_ERR_CUDA;
  a.N = (int)H;
  a.K = (int)I;
  a.half_kb = div_up(I, kBlockK);
  a.nkb = a.half_kb * (sh.gated ? 2 : 1);
  a.n_tiles = div_up(H, kTileN);
  if (!row_outputs(m, a, R, H, drows, nullptr, nullptr)) return MOE_ERR_CUDA;
  a.first = 0;
  return launch<kDgradRows>(m, a, row_items(sh, a.n_tiles), s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int moe_experts_weight_grad(const void* rows, const void* dout, const void* h, const void* dg, const void* du,
                            const int32_t* offsets, int64_t R, int32_t E, int64_t H, int64_t I, uint32_t flags,
                            float* dw_gate, float* dw_up, float* dw_down, void* workspace, size_t ws_bytes,
                            moe_stream_t stream) {
  Shape sh;
  const bool accumulate = flags & MOE_EXPERTS_ACCUMULATE;
  const int st = check_shape(offsets, R, E, H, I, flags & ~MOE_EXPERTS_ACCUMULATE, 0.0f, 0.0f, workspace, ws_bytes, kHeader, sh);
  if (st != MOE_OK) return st;
  if (!dw_up || !dw_down || (sh.gated ? !dw_gate : dw_gate != nullptr)) return MOE_ERR_INVALID_ARG;
  for (const void* p : {dw_gate, dw_up, dw_down})
    if (!is_aligned(p, 32)) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (R == 0) {
    cudaError_t e = cudaMemsetAsync(workspace, 0, sizeof(int32_t), s);
    const size_t n = sizeof(float) * (size_t)E * H * I;
    for (float* p : {dw_gate, dw_up, dw_down})
      if (e == cudaSuccess && p && !accumulate) e = cudaMemsetAsync(p, 0, n, s);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  }
  if (!rows || !dout || !h || !du || (sh.gated ? !dg : dg != nullptr)) return MOE_ERR_INVALID_ARG;
  for (const void* p : {rows, dout, h, dg, du})
    if (!is_aligned(p, 16)) return MOE_ERR_INVALID_ARG;
  if (!encoder()) return MOE_ERR_CUDA;
  WgradMaps m = {};
  void* zeros = nullptr;
  if (cudaGetSymbolAddress(&zeros, g_zeros) != cudaSuccess) return MOE_ERR_CUDA;
  const void* const operands[5] = {sh.gated ? dg : du, rows, du, dout, h};
  bool ok = make_map<4>(&m.out[0], sh.gated ? dw_gate : dw_up, H, I, E, 32) && make_map<4>(&m.out[1], dw_up, H, I, E, 32) &&
            make_map<4>(&m.out[2], dw_down, I, H, E, 32);
  for (int i = 0; i < 5; ++i) {
    const int64_t cols = i == 1 || i == 3 ? H : I;
    ok = ok && make_map(&m.m[i], operands[i], cols, R, 0, kBlockK);
    for (int l = 0; l < kHeights; ++l) ok = ok && make_map(&m.part[i][l], operands[i], cols, R, 0, 1 << l);
  }
  for (int l = 0; l < kHeights; ++l) ok = ok && make_map(&m.zero[l], zeros, 64, 1 << (kHeights - 1), 0, 1 << l);
  if (!ok) return MOE_ERR_CUDA;
  Args a = base_args(sh, offsets, workspace, 0.0f, 0.0f);
  a.M = (int)H;
  a.N = (int)I;
  a.nmat = sh.gated ? 3 : 2;
  a.accumulate = accumulate;
  a.first = 1;
  const int64_t items = (int64_t)E * a.nmat * div_up(H, kTileM) * div_up(I, kTileN);
  return launch<kWgrad>(m, a, items, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
