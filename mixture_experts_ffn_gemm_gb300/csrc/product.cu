// product.cu -- products grouped by expert with ragged sizes, on pairs of SMs (tcgen05 cta_group::2, fp32
// sums in tensor memory), rows r of expert e from offsets[e] to offsets[e + 1]:
//
//   forward  y[r][n]    = sum_k x[r][k] W_e[n][k]        bf16
//   grad_x   dx[r][k]   = sum_n dy[r][n] W_e[n][k]       bf16
//   grad_w   dW_e[n][k] = sum_r dy[r][n] x[r][k]         bf16
//   micro    out[r][n] = g_a g_w[e] sum_blocks S_a S_w sum_{k in block} c_a c_w      4-bit codes and
//            their scales (MOE_MICRO_MX, MOE_MICRO_NV), plain or with SwiGLU
//
// Orientation: the MMA's M side is the weights (256 features a pair, 128 on each SM's lanes), the N side
// the expert's rows, 32 to 256 of them as the tile has.  Rows are what is ragged: with them on the N side
// a tile costs its rows rounded up to 32, where rows on the M side would be rounded up to 128 (at 170 rows
// an expert a quarter of the work), and a decode step's few rows cost an MMA of N = 32.  A pair copies
// 128 features and half of the tile's rows to each SM for an M = 256 product: two thirds of the bytes a
// lone SM's 128 x 256 tile takes from L2, whose copies alone ran as long as its MMAs.
//
// An operand may lie either way in memory: grad_x sums over W's rows, and grad_w over the rows of dy (its M
// side) and x (its N side), so those are "MN-major" boxes of 64 outputs (128 bytes) x 64 steps of the sum;
// the instruction descriptor says which, and nothing is transposed in memory.  A stage holds 64 steps of
// the sum in bf16, or 256 codes: 128 bytes of each row.
//
// Edges: the maps have the operands' true extents and fill with zeros behind them; W has the expert as
// a third coordinate, so that rows behind W_e are zeros and not the next expert's.  grad_w's last block of
// a group runs into the next group's rows: a warp on each SM overwrites those rows of both operands with
// zeros in shared memory before the block is issued (zeros on one side alone would leave 0 x inf).
//
// Microscaled operands: the MMA takes 64 codes of a row and their scales from tensor memory (two e8m0 or
// four e4m3 bytes a row) and multiplies each block's sum by both scales in fp32; nothing is decoded.  Scales
// travel as they lie, in tiles of 128 rows x 4 columns: global to shared memory with the stage,
// shared to tensor memory by tcgen05.cp ahead of the stage's MMAs, into two sets of columns in turn.
// Row tiles start at multiples of 64 rows of their expert, so that a tile of at most 192 rows lies in two
// scale tiles.  Scales of rows outside a group are whatever the buffer holds; they reach only outputs that
// are not stored.
//
// SwiGLU: a W1 and a W3 tile of the same features against the same rows, two sums in tensor memory,
// g and u of an output in one thread; their 2 x 192 columns leave no room for a second pair of sums.  So that the
// next tile's MMAs do not wait for the exponentials, three of a storing warp's six chunks are read into
// registers first and finished after the columns are free (64 experts, 65536 rows, mx: none kept 633 us,
// three 591, four 625: registers).
//
// Sums: the tensor cores cut what falls behind the sum's 24 bits at every MMA, always towards zero, so that
// a long sum drifts by about 2^-25.5 of itself a step (5 x 10^-6 over 448 steps).  For fp32 outputs a sum stays
// in tensor memory for 32 steps (grad_w, whose stores its storing warps barely keep up with, 64: 1024 rows);
// the storing warps add such segments up in fp32, rounded to nearest.  A bf16 output's half step, 2^-9 to 2^-8 of
// it, is twelve times the drift of the 8192 steps that the widest forward and grad_x have, and that a group of
// kLongRows rows has; weight gradients over more rows than that are summed in segments of 1024 steps.
//
// Kernel shape: persistent, warp 0 copies, warp 1 issues (on the pair's even SM), warps 2..9 store, grad_w's
// warp 10 clears: a lane has a feature, so that a warp's store covers 128 (fp32) or 2 x 64 (bf16) consecutive
// bytes of rows.  dW leaves through shared memory and TMA (for ACCUMULATE its fp32 addition, one for each
// element).
//
// Measured (GB300): 8 experts, 32768 rows, 4096 x 7168: 0.98-1.01 ms in bf16 (1.9-1.97 PFLOP/s; the tensor pipe
// 89% busy), 0.315 ms mx, 0.332 ms nv (6.1, 5.8 PFLOP/s).  384 experts of 2048 x 7168, bf16, 16 tokens:
// 0.44-0.48 ms, the weights at the memory's rate; SwiGLU nv, 128 tokens: 0.77 ms, the same; 8192 tokens: SwiGLU mx
// 0.98-1.0 ms, and 7168 x 2048 0.64 ms.  What bounds it: few rows, the weights' bytes; many, the MMAs (bf16: the
// clock that their power leaves); between (170 rows an expert), the weights' bytes with what the epilogue does
// not hide; short sums (2048 and less), the storing warps; grad_w in fp32, operands and dW together between SMs
// and L2.
#include <atomic>
#include <cstring>

#include "internal.h"
#include "product.cuh"

namespace moe {

namespace {

constexpr int kEpilogueWarps = 8;
constexpr int kParts = kEpilogueWarps / 4;  // a tile's chunks of rows go to them in turn
constexpr int kMaxWarps = 2 + kEpilogueWarps + 1;
constexpr int kBox = 128 * 128;  // 128 features x 128 bytes
constexpr int kBox64 = 64 * 128;
constexpr int kBarBytes = 256;
constexpr int kTable = (4 * (kProductMaxGroups + 1)) * 4 + kMaxWarps * 4;
constexpr int kSmemMost = 232448 - 1024 - kBarBytes - kTable;

// Rows of a call above which a bf16 weight gradient, whose groups' sizes the host does not know, is summed in
// segments (see above).  8192 rows of 64 experts, 4096 x 7168: 899 us without them, 989 with them (the storing warps
// hold a tile's sums in registers until the last segment); 133120 rows, 2048 x 2048, 8 and 64 experts: 596 and 651
// without, 598 and 657 with them; 2^23 rows of one expert: 5% too small without.
constexpr int64_t kLongRows = 1 << 17;

enum Op { OP_FORWARD, OP_GRAD_X, OP_GRAD_W, OP_MX, OP_NV };

template <int kOp, bool kSwiGLU, bool kF32, bool kLong = false>
struct Shape {
  static constexpr bool kMicro = kOp == OP_MX || kOp == OP_NV;
  static constexpr int kMaxRows = !kMicro ? 256 : kSwiGLU && kF32 ? 128 : 192;  // rows of a tile
  static constexpr int kBlock = kMicro ? 256 : 64;         // elements of the sum per stage
  static constexpr int kStep = kMicro ? 64 : 16;           // and per MMA
  static constexpr int kSums = kSwiGLU ? 2 : 1;            // W1 and W3, or one
  // blocks summed in tensor memory at a time (see above)
  static constexpr bool kSegmented = kF32 || kLong;
  static constexpr int kSegment = !kSegmented ? 1 << 30 : !kF32 ? 256 : kOp == OP_GRAD_W ? 16 : 8;
  static constexpr int kTiles = kOp == OP_NV ? 4 : kOp == OP_MX ? 2 : 0;  // scale tiles per 128 rows
  static constexpr int kOpA = kSums * kBox;
  static constexpr int kOpB = kMaxRows / 2 * 128;
  static constexpr int kSfA = kTiles * 512;                // of one sum
  static constexpr int kSfB = 2 * kTiles * 512;
  static constexpr int kStage = kOpA + kOpB + kSums * kSfA + kSfB;
  static constexpr int kChunks = kMaxRows / 16 / kParts;   // chunks of 16 rows of a storing warp, at most
  static constexpr int kThreads = 32 * (2 + kEpilogueWarps + (kOp == OP_GRAD_W ? 1 : 0));
  static constexpr int kStaging = kOp == OP_GRAD_W ? kEpilogueWarps * 2048 : 0;
  static constexpr int kFit = (kSmemMost - kStaging) / kStage;
  static constexpr int kStages = kFit > 6 ? 6 : kFit;
  static constexpr int kSmem = 1024 + kStages * kStage + kStaging + kBarBytes + kTable;
  static constexpr int kAccs = kSwiGLU ? 1 : 2;            // tiles whose sums are in tensor memory
  static constexpr int kAccCols = kSums * kMaxRows;
  static constexpr int kSfCols = (kSums * 4 + 8) * kTiles; // columns of a stage's scales
  static constexpr int kSfCol0 = kAccs * kAccCols;
  static_assert(kSfCol0 + 2 * kSfCols <= 512, "tensor memory");
  static_assert(kStage % 1024 == 0 && kStages >= 3 && (4 * kStages + 5) * 8 + 12 <= kBarBytes, "");
};

struct ProductParams {
  CUtensorMap mw;        // weights
  CUtensorMap mrow[8];   // rows, boxes of 16, 32, .. 128: one copy a stage whatever the tile's rows
  CUtensorMap msw, msr;  // scale tiles of the weights and of the rows
  CUtensorMap mout;      // grad_w: dW, boxes of 32 rows x 64 bytes
  const int32_t* offsets;
  const float* a_factor;
  const float* w_factor;
  int32_t E, rows, F, Kc;  // F: features (outputs of a row), Kc: the sum's length (grad_w: N and K)
  int32_t wrows, ktiles;   // micro: an expert's weight rows, scale tiles along K
  void* out;
  int64_t ldo;
  uint32_t* err;
  uint64_t wait_ns;        // the bounded waits' limit
  int32_t stall;           // test hook: blocks after which a pair's odd SM copies nothing more (0: none)
};

// Descriptor of an MN-major operand: boxes of 64 outputs (128 bytes) x 64 rows of the sum, 128-byte
// swizzle; 8-row groups 1024 bytes apart (stride offset), boxes 8192 bytes apart (leading offset).
__device__ __forceinline__ uint64_t mnmajor_desc(uint32_t smem_addr) {
  return sw128_kmajor_desc(smem_addr) | (uint64_t)(kBox64 >> 4) << 16;
}

// Zeros in rows [from, to) of the boxes from `box0` on (each 64 rows of 128 bytes; the swizzle moves
// 16-byte pieces within a row), for the tensor cores to read.  The whole warp.
template <int kBoxes>
__device__ __forceinline__ void clear_rows(uint8_t* box0, int from, int to, int lane) {
  const int n = (to - from) * 8;
#pragma unroll
  for (int b = 0; b < kBoxes; ++b) {
    uint4* r = reinterpret_cast<uint4*>(box0 + b * kBox64 + from * 128);
    for (int i = lane; i < n; i += 32) r[i] = make_uint4(0, 0, 0, 0);
  }
  fence_async_smem();
}

// mbar_wait for a warp that may be any number of blocks ahead of the copies that it waits for: it gives up after
// a limit's time in which no block was copied.
__device__ __forceinline__ bool wait_behind(uint64_t* bar, uint32_t parity, volatile const int* copied,
                                            volatile int* abort, uint32_t* err, uint64_t limit_ns) {
  if (mbar_test(bar, parity)) return true;
  int seen = *copied;
  uint64_t t0 = globaltimer_ns();
  while (!mbar_test(bar, parity)) {
    if (*abort) return false;
    if (globaltimer_ns() - t0 > limit_ns) {
      const int now = *copied;
      if (now == seen) {
        *abort = 1;
        raise_flag(err, kErrTimeout);
        return false;
      }
      seen = now;
      t0 = globaltimer_ns();
    }
  }
  return true;
}

// A 512-byte scale tile: 32 rows of 16 bytes without swizzle, 8-row groups 128 bytes apart.
__device__ __forceinline__ uint64_t scale_tile_desc(uint32_t smem_addr) {
  return (uint64_t)((smem_addr & 0x3FFFFu) >> 4) | (uint64_t)(128u >> 4) << 32 | (uint64_t)1 << 46;
}
// 32 lanes x 4 columns to each of the four lane quarters, in both SMs from their own shared memory.
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

// Block-scaled MMA, e2m1 operands, M = 256: bits [4,6) B's first scale byte, [7,10) and [10,13) formats
// (1 = e2m1), [17,23) N >> 3, 23 scale type (1 = e8m0, 0 = e4m3), [24,29) M >> 4, [29,31) A's first byte.
template <bool kNv>
__device__ __forceinline__ uint32_t idesc_micro(int n, int first) {
  return ((uint32_t)first << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) |
         (kNv ? 0u : 1u << 23) | ((256u >> 4) << 24) | ((uint32_t)first << 29);
}
template <bool kNv>
__device__ __forceinline__ void mma_micro_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                               uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if constexpr (kNv)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], "
        "[%5], p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], "
        "[%5], p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// A chunk of 32 rows of dW x 64 bytes, lane l holding row l's, through 2 KB of shared memory (in the 64-byte
// swizzle) to TMA, which leaves out what lies behind dW's last row or column.  The whole warp.
template <bool kAdd>
__device__ __forceinline__ void store_dw(const CUtensorMap* map, uint8_t* buf, int lane,
                                         const uint32_t (&v)[16], int x, int y, int z) {
  if (lane == 0) tma_store_wait_read();  // the previous chunk has left the buffer
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<uint4*>(buf + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) =
        make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
  fence_async_smem();
  __syncwarp();
  if (lane == 0) tma_store_3d<kAdd>(map, buf, x, y, z);
}

// g / (1 + exp(-g)).  The division is the approximate one (two steps of 2^-23); an exponential that
// overflows gives 0.  fp32 outputs take the accurate exponential.
template <bool kAccurate>
__device__ __forceinline__ float silu(float g) {
  return __fdividef(g, 1.0f + (kAccurate ? expf(-g) : __expf(-g)));
}

template <int kOp, bool kSwiGLU, bool kF32, bool kAdd, bool kLong>
__global__ void __launch_bounds__(Shape<kOp, kSwiGLU, kF32, kLong>::kThreads, 1)
    product_kernel(const __grid_constant__ ProductParams p) {
  using S = Shape<kOp, kSwiGLU, kF32, kLong>;
  constexpr bool kMicro = S::kMicro, kNv = kOp == OP_NV, kGradW = kOp == OP_GRAD_W;
  constexpr bool kAMn = kOp == OP_GRAD_X || kGradW, kBMn = kGradW;
  constexpr int kStage = S::kStage, kStages = S::kStages, kMaxRows = S::kMaxRows;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int tile0 = (int)(blockIdx.x >> 1), tstep = (int)(gridDim.x >> 1);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* staging = smem + kStages * kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + S::kStaging);
  uint64_t* empty = full + kStages;
  // grad_w, blocks that are cleared: this SM's copies have landed; both SMs' rows behind the group are zeros
  uint64_t* landed = empty + kStages;
  uint64_t* cleared = landed + kStages;
  uint64_t* tfull = cleared + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  volatile int* blocks_copied = abort_flag + 1;  // grad_w: this SM's copying warp counts them
  GroupTable tab;
  tab.tile_start = reinterpret_cast<int*>(staging + S::kStaging + kBarBytes);
  tab.row0 = tab.tile_start + kProductMaxGroups + 1;
  tab.nrows = tab.row0 + kProductMaxGroups + 1;
  tab.cut = tab.nrows + kProductMaxGroups + 1;
  int* scratch = tab.cut + kProductMaxGroups + 1;

  const int warp = uniform(threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&landed[s], 1);
      mbar_init(&cleared[s], 2);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * kEpilogueWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    *blocks_copied = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&p.mw);
    if (kMicro) {
      tma_prefetch_map(&p.msw);
      tma_prefetch_map(&p.msr);
    }
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_holder, 512);
    tmem_relinquish_pair();
  }
  wait_for_prior_kernel();
  build_group_table<kMaxRows, kMicro ? 64 : 32>(tab, scratch, p.offsets, p.E, p.rows,
                              kGradW ? 0 : (p.F + 255) / 256,
                              blockIdx.x == 0 ? p.err : nullptr);  // ends with __syncthreads
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both SMs' barriers exist before any remote arrival
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  // grad_w: the features are dW's rows, and in the place of rows there are its columns, 256 to a tile; the
  // sum runs over the group's rows
  const int fts = (p.F + 255) / 256, nts = (p.Kc + kMaxRows - 1) / kMaxRows;
  const int total = kGradW ? p.E * nts * fts : tab.tile_start[p.E];
  // The warp's next tile (each call takes one step of tstep).  grad_w: fts x nts tiles a group; ft by the
  // reciprocal, whose error (512 x 2^-22 at most 512 tiles along K and along N) stays below half a tile's share.
  TileWalk walk;
  const float per_nts = 1.0f / (float)nts;
  int gw_group = 0, gw_local = tile0;
  const auto tile_of = [&](int tile) {
    if constexpr (kGradW) {
      while (gw_local >= nts * fts) {
        gw_local -= nts * fts;
        ++gw_group;
      }
      ProductTile t;
      t.g = gw_group;
      t.ft = (int)(((float)gw_local + 0.5f) * per_nts);
      t.lrow0 = (gw_local - t.ft * nts) * kMaxRows;
      t.row0 = 0;
      t.valid = min(kMaxRows, p.Kc - t.lrow0);
      gw_local += tstep;
      return t;
    } else {
      return walk.at(tile, tab, p.E, lane);
    }
  };
  const auto sum_len = [&](const ProductTile& t) { return kGradW ? uniform(tab.nrows[t.g]) : p.Kc; };
  // grad_w takes the sum's last, shorter block first, so that it is cleared while the MMAs of the tile before
  // still run.  Steps of the sum in block kb, where it starts, and whether rows behind it are read and so
  // cleared.
  const auto block_len = [](int len, int kb) {
    return kGradW ? (kb ? S::kBlock : len - (len - 1) / S::kBlock * S::kBlock)
                  : min(S::kBlock, len - kb * S::kBlock);
  };
  const auto block_start = [](int len, int kb) {
    return kGradW ? (kb ? kb - 1 : (len - 1) / S::kBlock) * S::kBlock : kb * S::kBlock;
  };
  const auto to_clear = [](int steps) { return kGradW && steps % S::kStep != 0; };
  // micro: whether the tile's rows lie in two scale tiles
  const auto two_scale_tiles = [](const ProductTile& t, int n) { return (t.lrow0 & 127) + n > 128; };
  const auto mma_rows = [](const ProductTile& t) { return (t.valid + 31) & ~31; };

  if (warp == 0) {
    uint32_t stage = 0, phase = 0;
    uint32_t full_uses = 0, landed_uses = 0, in_landed = 0;  // a bit a stage: uses (mod 2), the last one's barrier
    int armed = 0;
    uint32_t blocks = 0;
    bool ok = true;
    for (int tile = tile0; tile < total && ok; tile += tstep) {
      const ProductTile t = tile_of(tile);
      const int n = mma_rows(t), len = sum_len(t), g = t.g;
      const int nkb = (len + S::kBlock - 1) / S::kBlock;
      const int f0 = t.ft * 256 + (int)rank * 128;      // this SM's first feature
      const int r0 = t.row0 + (int)rank * (n / 2);      // and row
      const bool two = two_scale_tiles(t, n);
      // bytes of a stage: MN-major rows come in whole boxes
      const uint32_t bytes =
          S::kOpA + (kBMn ? (n / 2 + 63) / 64 * kBox64 : n / 2 * 128) + S::kSums * S::kSfA +
          (two ? S::kSfB : S::kSfB / 2);
      const int w0 = g * p.wrows;                       // micro: the expert's first weight row
      const int st_w = ((w0 >> 7) + g + (f0 >> 7)) * p.ktiles;
      const int st_u = ((w0 >> 7) + g + ((p.F + f0) >> 7)) * p.ktiles;  // its W3
      const int st_r = (((t.row0 - t.lrow0) >> 7) + g + (t.lrow0 >> 7)) * p.ktiles;
      const int gw_n = t.lrow0 + (int)rank * (n / 2), gw_r = kGradW ? uniform(tab.row0[g]) : 0;
      const CUtensorMap* mrow = &p.mrow[n / 32 - 1];
      for (int kb = 0; kb < nkb; ++kb) {
        ok = __all_sync(~0u, mbar_wait(&empty[stage], phase ^ 1u, abort_flag, p.err, p.wait_ns));
        if (!ok) break;
        const bool mute = p.stall && !leader && blocks >= (uint32_t)p.stall;
        if (!mute && elect_one()) {
          uint8_t* sa = smem + stage * kStage;
          uint8_t* sb = sa + S::kOpA;
          // Both SMs' copies complete on the even SM's full[stage]; of a block that is cleared, each
          // SM's on its own landed[stage], where the warp waits that clears it.
          const bool own = to_clear(block_len(len, kb));
          const uint32_t bar = own ? cluster_addr(&landed[stage], rank) : cluster_addr(&full[stage], 0);
          if (own)
            mbar_arrive_expect_tx(&landed[stage], bytes);
          else if (leader)
            mbar_arrive_expect_tx(&full[stage], 2 * bytes);
          const int kx = kb * (kMicro ? 128 : 64);  // bytes or elements: 128 bytes a row
          if constexpr (kMicro) {
            tma_load_2d_pair(sa, &p.mw, bar, kx, w0 + f0);
            if (kSwiGLU) tma_load_2d_pair(sa + kBox, &p.mw, bar, kx, w0 + p.F + f0);
          } else if constexpr (kGradW) {
            const int y = gw_r + block_start(len, kb);
            tma_load_2d_pair(sa, &p.mw, bar, f0, y);
            tma_load_2d_pair(sa + kBox64, &p.mw, bar, f0 + 64, y);
            for (int j = 0; j < n / 2; j += 64)
              tma_load_2d_pair(sb + j * 128, &p.mrow[0], bar, gw_n + j, y);
          } else if constexpr (kAMn) {
            tma_load_3d_pair(sa, &p.mw, bar, f0, kx, g);
            tma_load_3d_pair(sa + kBox64, &p.mw, bar, f0 + 64, kx, g);
          } else {
            tma_load_3d_pair(sa, &p.mw, bar, kx, f0, g);
          }
          if constexpr (!kBMn) tma_load_2d_pair(sb, mrow, bar, kx, r0);
          if constexpr (kMicro) {
            uint8_t* f = sb + S::kOpB;
            const int kt = kb * S::kTiles;
            tma_load_2d_pair(f, &p.msw, bar, 0, st_w + kt);
            if (kSwiGLU) tma_load_2d_pair(f + S::kSfA, &p.msw, bar, 0, st_u + kt);
            f += S::kSums * S::kSfA;
            tma_load_2d_pair(f, &p.msr, bar, 0, st_r + kt);
            if (two) tma_load_2d_pair(f + S::kSfB / 2, &p.msr, bar, 0, st_r + p.ktiles + kt);
          }
        }
        ++blocks;
        if (kGradW && lane == 0) *blocks_copied = (int)blocks;
        __syncwarp();
        const uint32_t bit = 1u << stage;
        if (to_clear(block_len(len, kb))) {
          landed_uses ^= bit;
          in_landed |= bit;
        } else {
          full_uses ^= bit;
          in_landed &= ~bit;
        }
        if (armed < kStages) ++armed;
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok) {  // let the copies of the last stage uses land
      bool counted_there = false;
      for (int i = 0; i < armed; ++i) {
        stage = stage ? stage - 1 : kStages - 1;
        const bool own = in_landed >> stage & 1u;
        if (own || leader)
          mbar_wait(own ? &landed[stage] : &full[stage],
                    (own ? landed_uses : full_uses) >> stage & 1u ^ 1u, nullptr, nullptr, kDrainLimitNs);
        else
          counted_there = true;
      }
      // Copies of the odd SM that count on the even SM's barriers: only that SM can ask those, and it may have
      // stopped before it expected the last of them.  They get the limit itself; both SMs stay until it is over.
      if (counted_there) {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 <= kDrainLimitNs) __nanosleep(1000);
      }
    }
  } else if (warp == 1 && leader) {
    // the whole warp follows the stages, one thread issues; a stage's barrier of each kind has its phase bit
    uint32_t stage = 0, acc = 0, acc_phase = 0, buf = 0, full_phase = 0, cleared_phase = 0;
    bool ok = true;
    // descriptors of stage 0; a stage, a step of the sum and a tile lie at fixed distances (in 16 bytes)
    const uint32_t s0 = smem_u32(smem);
    const uint64_t a0 = kAMn ? mnmajor_desc(s0) : sw128_kmajor_desc(s0);
    const uint64_t b0 = kBMn ? mnmajor_desc(s0 + S::kOpA) : sw128_kmajor_desc(s0 + S::kOpA);
    const uint64_t f0 = scale_tile_desc(s0 + S::kOpA + S::kOpB);
    constexpr uint32_t kStepA = (kAMn ? 2048 : 32) >> 4, kStepB = (kBMn ? 2048 : 32) >> 4;
    for (int tile = tile0; tile < total && ok; tile += tstep) {
      const ProductTile t = tile_of(tile);
      const int n = mma_rows(t), len = sum_len(t);
      const int nkb = (len + S::kBlock - 1) / S::kBlock;
      if (kGradW && nkb == 0) continue;  // a group without rows: the epilogue writes zeros
      const bool two = two_scale_tiles(t, n);
      const uint32_t b_col = (t.lrow0 & 127) >> 5;  // micro: the tile's first row's scale column
      const uint32_t idesc0 = kMicro ? idesc_micro<kNv>(n, 0)
                                     : idesc_bf16_f32_pair(n) | (kAMn ? 1u << 15 : 0u) | (kBMn ? 1u << 16 : 0u);
      const uint32_t idesc_second = idesc_micro<kNv>(0, 2) - idesc_micro<kNv>(0, 0);
      for (int k0 = 0; k0 < nkb; k0 += S::kSegment) {  // a segment of the sum, into sums that have been read
        ok = __all_sync(~0u, mbar_wait_cluster(&tempty[acc], acc_phase ^ 1u, abort_flag, p.err, p.wait_ns));
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem_base + acc * S::kAccCols;
        const int k1 = nkb - k0 < S::kSegment ? nkb : k0 + S::kSegment;
        for (int kb = k0; kb < k1; ++kb) {
          const int left = block_len(len, kb);
          const int steps = (left + S::kStep - 1) / S::kStep;
          if (to_clear(left)) {
            ok = __all_sync(~0u, mbar_wait_cluster(&cleared[stage], cleared_phase >> stage & 1u,
                                                   abort_flag, p.err, p.wait_ns));
            cleared_phase ^= 1u << stage;
          } else {
            ok = __all_sync(~0u, mbar_wait(&full[stage], full_phase >> stage & 1u, abort_flag, p.err, p.wait_ns));
            full_phase ^= 1u << stage;
          }
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t at = (uint64_t)(stage * (kStage >> 4));
            const uint64_t sa = a0 + at, sb = b0 + at;
            if constexpr (kMicro) {
              const uint64_t fa = f0 + at, fb = fa + (S::kSums * S::kSfA >> 4);
              const uint32_t ta = tmem_base + S::kSfCol0 + buf * S::kSfCols;
              const uint32_t tb = ta + S::kSums * 4 * S::kTiles;
#pragma unroll
              for (int i = 0; i < S::kTiles; ++i) {
#pragma unroll
                for (int m = 0; m < S::kSums; ++m)
                  copy_scales(ta + 4 * (m * S::kTiles + i), fa + ((m * S::kSfA + i * 512) >> 4));
                copy_scales(tb + 8 * i, fb + (i * 512 >> 4));
                if (two) copy_scales(tb + 8 * i + 4, fb + ((S::kSfB / 2 + i * 512) >> 4));
              }
#pragma unroll
              for (int s = 0; s < 4; ++s) {
                if (s == steps) break;
                const int i = kNv ? s : s >> 1;  // scale tile, and first byte in its columns
                const uint32_t id = kNv ? idesc0 : idesc0 + (s & 1) * idesc_second;
#pragma unroll
                for (int m = 0; m < S::kSums; ++m)
                  mma_micro_pair<kNv>(d + m * kMaxRows, sa + ((m * kBox >> 4) + s * kStepA), sb + s * kStepB, id,
                                      ta + 4 * (m * S::kTiles + i), tb + b_col + 8 * i, kb != k0 || s);
              }
            } else {
#pragma unroll
              for (int s = 0; s < 4; ++s) {
                if (s == steps) break;
                mma_bf16_pair(d, sa + s * kStepA, sb + s * kStepB, idesc0, kb != k0 || s);
              }
            }
            commit_both(&empty[stage]);  // frees the stage on both SMs
          }
          __syncwarp();
          buf ^= 1u;
          if (++stage == kStages) stage = 0;
        }
        if (!ok) break;
        if (elect_one()) commit_both(&tfull[acc]);
        __syncwarp();
        if (S::kAccs == 2) acc ^= 1u;
        if (acc == 0) acc_phase ^= 1u;
      }
    }
    if (elect_one()) mma_commit_pair_own(drain);  // every MMA issued above has completed once this arrives
    __syncwarp();
    mbar_wait(drain, 0, nullptr, nullptr, kDrainLimitNs);
  } else if (kGradW && warp == 2 + kEpilogueWarps) {
    // clears this SM's rows behind the group, as soon as a block that has some has landed; it does not wait
    // for the others, of which there may be a whole group's
    uint32_t stage = 0, phase = 0;
    bool ok = true;
    for (int tile = tile0; tile < total && ok; tile += tstep) {
      const int len = sum_len(tile_of(tile));
      for (int kb = 0; kb * S::kBlock < len; ++kb) {
        const int left = block_len(len, kb);
        if (to_clear(left)) {
          ok = __all_sync(~0u, wait_behind(&landed[stage], phase >> stage & 1u, blocks_copied, abort_flag, p.err,
                                           p.wait_ns));
          if (!ok) break;
          phase ^= 1u << stage;
          clear_rows<4>(smem + stage * kStage, left, (left + S::kStep - 1) / S::kStep * S::kStep, lane);
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(cluster_addr(&cleared[stage], 0));
        }
        if (++stage == kStages) stage = 0;
      }
    }
  } else if (warp > 1) {
    const int quarter = warp & 3, part = (warp - 2) >> 2;
    uint32_t acc = 0, acc_phase = 0;
    const float ga = kNv && p.a_factor ? *p.a_factor : 1.0f;
    for (int tile = tile0; tile < total; tile += tstep) {
      const ProductTile t = tile_of(tile);
      const int len = sum_len(t);
      const bool none = kGradW && len == 0;
      if (kAdd && none) continue;
      // A sum is zero or 2^-20 to 2^40.  Where the factors' product keeps the scaled sum a plain number, one
      // multiplication does; else its magnitude may leave fp32 though the result does not, and the sums are
      // taken times the smaller factor first (a normal number, as a factor is at least 2^-100), then times the
      // other (too large only if the result is).  8192 tokens, W2: 711 us, both multiplications always 715; 2048 x
      // 2048 in fp32: 209 and 217.
      float alpha = 1.0f, before = 1.0f;
      const auto read_factors = [&] {
        if constexpr (kNv) {
          const float gw = p.w_factor ? p.w_factor[t.g] : 1.0f;
          alpha = ga * gw;
          if (!(fabsf(alpha) >= 0x1p-100f && fabsf(alpha) <= 0x1p87f)) {
            before = fabsf(ga) < fabsf(gw) ? ga : gw;
            alpha = fabsf(ga) < fabsf(gw) ? gw : ga;
          }
        }
      };
      const auto scale_before = [&](uint32_t (&sums)[16]) {
        if (kNv && before != 1.0f) {
#pragma unroll
          for (int i = 0; i < 16; ++i) sums[i] = __float_as_uint(__uint_as_float(sums[i]) * before);
        }
      };
      const auto scaled = [&](uint32_t sum) { return __uint_as_float(sum) * alpha; };
      const int feat0 = t.ft * 256 + (int)rank * 128 + quarter * 32;  // this warp's first feature
      // this warp's chunks of 16 columns (of 32: grad_w in bf16)
      const auto col = [&](int ch) { return (kParts * ch + part) * (kGradW && !kF32 ? 32 : 16); };
      const int end = t.valid;
      uint8_t* buf = staging + (warp - 2) * 2048;                     // grad_w
      if constexpr (S::kSegmented) {
        // Segments of the sum, added up here in fp32 (rounded to nearest, where the tensor cores cut).
        constexpr int kPieces = kGradW && !kF32 ? 2 : 1;  // of 16 columns, in a chunk
        constexpr int kChunks = S::kChunks / kPieces;
        float sum[S::kSums][S::kChunks * 16];
#pragma unroll
        for (int m = 0; m < S::kSums; ++m)
#pragma unroll
          for (int i = 0; i < S::kChunks * 16; ++i) sum[m][i] = 0.0f;
        const auto release = [&] {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(cluster_addr(&tempty[acc], 0));
          if (S::kAccs == 2) acc ^= 1u;
          if (acc == 0) acc_phase ^= 1u;
        };
        const auto read = [&](int c, uint32_t (&g)[S::kSums][16]) {
          const uint32_t tb = tmem_base + acc * S::kAccCols + ((uint32_t)(quarter * 32) << 16);
#pragma unroll
          for (int m = 0; m < S::kSums; ++m) tmem_ld16(tb + m * kMaxRows + c, g[m]);
          tmem_ld_wait();
        };
        bool ok = true;
        int at = 0;
        for (; len - at > S::kSegment * S::kBlock; at += S::kSegment * S::kBlock) {  // all but the last
          ok = __all_sync(~0u, mbar_wait(&tfull[acc], acc_phase, abort_flag, p.err, p.wait_ns));
          if (!ok) break;
          tc_fence_after();
          if (feat0 < p.F) {
#pragma unroll
            for (int ch = 0; ch < kChunks; ++ch) {
              if (col(ch) < end) {
#pragma unroll
                for (int h = 0; h < kPieces; ++h) {
                  uint32_t g[S::kSums][16];
                  read(col(ch) + 16 * h, g);
#pragma unroll
                  for (int m = 0; m < S::kSums; ++m)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                      sum[m][16 * (kPieces * ch + h) + i] += __uint_as_float(g[m][i]);
                }
              }
            }
          }
          release();
        }
        if (!ok) break;
        if (!none) {
          if (!__all_sync(~0u, mbar_wait(&tfull[acc], acc_phase, abort_flag, p.err, p.wait_ns))) break;
          tc_fence_after();
        }
        if (feat0 < p.F) {
          read_factors();  // here, not in front of the segments, whose sums leave no register for them
#pragma unroll
          for (int ch = 0; ch < kChunks; ++ch) {
            const int c = col(ch);
            if (c >= end) continue;
            uint32_t g[S::kSums][16];
            if constexpr (kPieces == 2) {
              uint32_t v[16];
#pragma unroll
              for (int h = 0; h < kPieces; ++h) {
                float* part_sum = &sum[0][16 * (kPieces * ch + h)];
                if (!none) {
                  read(c + 16 * h, g);
#pragma unroll
                  for (int i = 0; i < 16; ++i) part_sum[i] += __uint_as_float(g[0][i]);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) v[8 * h + i] = pack_bf16x2(part_sum[2 * i], part_sum[2 * i + 1]);
              }
              store_dw<false>(&p.mout, buf, lane, v, t.lrow0 + c, feat0, t.g);
              continue;
            }
            if (!none) {
              read(c, g);
#pragma unroll
              for (int m = 0; m < S::kSums; ++m)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  g[m][i] = __float_as_uint(sum[m][16 * ch + i] + __uint_as_float(g[m][i]));
#pragma unroll
              for (int m = 0; m < S::kSums; ++m) scale_before(g[m]);
            }
            if constexpr (kGradW) {
              if (none) {
#pragma unroll
                for (int i = 0; i < 16; ++i) g[0][i] = 0u;
              }
              store_dw<kAdd>(&p.mout, buf, lane, g[0], t.lrow0 + c, feat0, t.g);
            } else {
              float* dst = static_cast<float*>(p.out) + ((int64_t)t.row0 + c) * p.ldo + feat0 + lane;
              if (feat0 + lane < p.F) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  float f = kMicro ? scaled(g[0][i]) : __uint_as_float(g[0][i]);
                  if constexpr (kSwiGLU) f = silu<true>(f) * scaled(g[S::kSums - 1][i]);
                  if (c + i < t.valid) dst[i * p.ldo] = f;
                }
              }
            }
          }
        }
        if (!none) release();
        continue;
      }
      read_factors();
      if (!none && !__all_sync(~0u, mbar_wait(&tfull[acc], acc_phase, abort_flag, p.err, p.wait_ns))) break;
      tc_fence_after();
      const uint32_t tb = tmem_base + acc * S::kAccCols + ((uint32_t)(quarter * 32) << 16);
      // Outputs f of 16 rows from column c on, a lane's feature.  Lanes in twos: of four rows the even one takes both
      // features of the first two, the odd one those of the others, with one exchange of two rows' bf16 (8192
      // tokens, W2: 634 us mx; an exchange of fp32 for every row and each store with its condition: 681).
      const auto store_rows = [&](const float (&f)[16], int c) {
        const int odd = lane & 1;
        uint32_t v[8];
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
          const uint32_t lo = pack_bf16x2(f[2 * k], f[2 * k + 1]), hi = pack_bf16x2(f[2 * k + 2], f[2 * k + 3]);
          const uint32_t own = odd ? hi : lo, got = __shfl_xor_sync(~0u, odd ? lo : hi, 1);
          v[k] = __byte_perm(own, got, odd ? 0x1054 : 0x5410);
          v[k + 1] = __byte_perm(own, got, odd ? 0x3276 : 0x7632);
        }
        const int r = c + 2 * odd;
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + ((int64_t)t.row0 + r) * p.ldo + feat0 + (lane & ~1);
        const auto row = [](int k) { return 4 * (k / 2) + k % 2; };
        if (c + 16 <= t.valid && feat0 + 32 <= p.F) {
#pragma unroll
          for (int k = 0; k < 8; ++k) *reinterpret_cast<uint32_t*>(dst + row(k) * p.ldo) = v[k];
        } else {
          const int rows = feat0 + (lane & ~1) < p.F ? t.valid - r : 0;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (row(k) < rows) *reinterpret_cast<uint32_t*>(dst + row(k) * p.ldo) = v[k];
        }
      };
      const auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(cluster_addr(&tempty[acc], 0));
        if (S::kAccs == 2) acc ^= 1u;
        if (acc == 0) acc_phase ^= 1u;
      };
      if constexpr (kSwiGLU) {
        constexpr int kKeep = 3;
        const auto finish = [&](uint32_t (&g)[16], uint32_t (&u)[16], int c) {
          scale_before(g);
          scale_before(u);
          float f[16];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            f[i] = silu<false>(scaled(g[i])) * scaled(u[i]);
          store_rows(f, c);
        };
        uint32_t kg[kKeep][16], ku[kKeep][16];
        if (feat0 < p.F) {
#pragma unroll
          for (int k = 0; k < kKeep; ++k)
            if (col(k) < end) {
              tmem_ld16(tb + col(k), kg[k]);
              tmem_ld16(tb + kMaxRows + col(k), ku[k]);
            }
          tmem_ld_wait();
#pragma unroll 1
          for (int c = col(kKeep); c < end; c += 16 * kParts) {
            uint32_t g[16], u[16];
            tmem_ld16(tb + c, g);
            tmem_ld16(tb + kMaxRows + c, u);
            tmem_ld_wait();
            finish(g, u, c);
          }
        }
        release();
        if (feat0 < p.F) {
#pragma unroll
          for (int k = 0; k < kKeep; ++k)
            if (col(k) < end) finish(kg[k], ku[k], col(k));
        }
        continue;
      }
      if (feat0 < p.F) {
#pragma unroll 1
        for (int c = col(0); c < end; c += kGradW ? 64 : 16 * kParts) {
          if constexpr (kGradW) {
            // a lane has a row of dW: chunks of 32 rows x 64 bytes
            uint32_t g[32], v[16];
            if (!none) {
              tmem_ld16(tb + c, reinterpret_cast<uint32_t(&)[16]>(g[0]));
              tmem_ld16(tb + c + 16, reinterpret_cast<uint32_t(&)[16]>(g[16]));
              tmem_ld_wait();
            }
#pragma unroll
            for (int i = 0; i < 16; ++i)
              v[i] = none ? 0u : pack_bf16x2(__uint_as_float(g[2 * i]), __uint_as_float(g[2 * i + 1]));
            store_dw<false>(&p.mout, buf, lane, v, t.lrow0 + c, feat0, t.g);
          } else {
            uint32_t g[16];
            float f[16];
            tmem_ld16(tb + c, g);
            tmem_ld_wait();
            scale_before(g);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              f[i] = kMicro ? scaled(g[i]) : __uint_as_float(g[i]);
            store_rows(f, c);
          }
        }
      }
      if (!none) release();
    }
    if (kGradW && lane == 0) tma_store_wait_all();
  }
  allow_next_kernel();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no arrival at the peer and no MMA into its tensor memory from here on
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

template <int kOp, bool kSwiGLU, bool kF32, bool kAdd = false, bool kLong = false>
cudaError_t launch(const ProductParams& p, int sms, cudaStream_t st, const char* label) {
  using S = Shape<kOp, kSwiGLU, kF32, kLong>;
  auto kern = product_kernel<kOp, kSwiGLU, kF32, kAdd, kLong>;
  static std::atomic<uint64_t> set{0};  // devices whose attribute is set
  const cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kern), S::kSmem, &set);
  if (e != cudaSuccess) return e;
  LaunchScope ls(label, st);
  return launch_pairs(kern, sms, S::kThreads, S::kSmem, st, p);
}

template <int kOp>
cudaError_t launch_micro(const ProductParams& p, bool swiglu, bool f32, int sms, cudaStream_t st) {
  if (swiglu)
    return f32 ? launch<kOp, true, true>(p, sms, st, "micro_product_swiglu")
               : launch<kOp, true, false>(p, sms, st, "micro_product_swiglu");
  return f32 ? launch<kOp, false, true>(p, sms, st, "micro_product")
             : launch<kOp, false, false>(p, sms, st, "micro_product");
}

}  // namespace

// Maps of boxes of 16, 32, .. rows, as far as a tile of a group can need them.
static bool make_row_maps(CUtensorMap* m, int count, int el, const void* base, uint64_t cols,
                          uint64_t rows, uint64_t ld, uint32_t box_cols) {
  for (int i = 0; i < count && (uint64_t)i * 32 < rows; ++i)
    if (!make_map_2d(&m[i], el, base, cols, rows, ld, box_cols, 16 * (i + 1))) return false;
  return true;
}

cudaError_t launch_grouped_product(const GroupedProduct& g, int sms, cudaStream_t st) {
  ProductParams p;
  memset(&p, 0, sizeof p);
  const bool fwd = g.kind == MOE_PRODUCT_FORWARD, grad_w = g.kind == MOE_PRODUCT_GRAD_W;
  p.F = fwd || grad_w ? g.N : g.K;
  p.Kc = fwd || grad_w ? g.K : g.N;
  if (grad_w) {  // dy on the feature side, x on the other
    const int el = g.out_dtype == MOE_F32 ? 4 : 2;
    if (!make_map_2d(&p.mw, 2, g.a, g.N, g.rows, g.ld_a, 64, 64) ||
        !make_map_2d(&p.mrow[0], 2, g.b, g.K, g.rows, g.ld_b, 64, 64) ||
        !make_map_3d(&p.mout, el, g.out, g.K, g.N, g.E, 64 / el, 32))
      return cudaErrorInvalidValue;
  } else if (!make_map_3d(&p.mw, 2, g.b, g.K, g.N, g.E, 64, fwd ? 128 : 64) ||
             !make_row_maps(p.mrow, 8, 2, g.a, p.Kc, g.rows, g.ld_a, 64))
    return cudaErrorInvalidValue;
  p.offsets = g.offsets;
  p.E = g.E;
  p.rows = (int32_t)g.rows;
  p.out = g.out;
  p.ldo = g.ldo;
  p.err = g.err;
  p.wait_ns = g.test_stall ? 20000000ull : g.test_short_waits ? 10000000ull : kWaitLimitNs;
  p.stall = g.test_stall ? 3 : 0;
  const bool f32 = g.out_dtype == MOE_F32;
  if (grad_w) {
    if (g.accumulate) return launch<OP_GRAD_W, false, true, true>(p, sms, st, "grouped_grad_w");
    if (f32) return launch<OP_GRAD_W, false, true>(p, sms, st, "grouped_grad_w");
    return g.rows > kLongRows ? launch<OP_GRAD_W, false, false, false, true>(p, sms, st, "grouped_grad_w")
                              : launch<OP_GRAD_W, false, false>(p, sms, st, "grouped_grad_w");
  }
  if (fwd)
    return f32 ? launch<OP_FORWARD, false, true>(p, sms, st, "grouped_forward")
               : launch<OP_FORWARD, false, false>(p, sms, st, "grouped_forward");
  return f32 ? launch<OP_GRAD_X, false, true>(p, sms, st, "grouped_grad_x")
             : launch<OP_GRAD_X, false, false>(p, sms, st, "grouped_grad_x");
}

cudaError_t launch_micro_product(const MicroProduct& g, int sms, cudaStream_t st) {
  ProductParams p;
  memset(&p, 0, sizeof p);
  const bool nv = g.format == MOE_MICRO_NV;
  p.wrows = g.swiglu ? 2 * g.N : g.N;
  const int per = nv ? 64 : 128;  // channels of a scale tile
  p.ktiles = (g.K + per - 1) / per;
  const uint64_t half = (uint64_t)g.K / 2, wrows = (uint64_t)g.E * p.wrows;
  const uint32_t tiles = nv ? Shape<OP_NV, false, false>::kTiles : Shape<OP_MX, false, false>::kTiles;
  if (!make_map_2d(&p.mw, 1, g.w, half, wrows, half, 128, 128) ||
      !make_row_maps(p.mrow, Shape<OP_MX, false, false>::kMaxRows / 32, 1, g.a, half, g.rows, half, 128) ||
      !make_map_tiles(&p.msw, g.w_scales, (wrows / 128 + g.E) * p.ktiles, tiles) ||
      !make_map_tiles(&p.msr, g.a_scales, ((uint64_t)g.rows / 128 + g.E) * p.ktiles, tiles))
    return cudaErrorInvalidValue;
  p.offsets = g.offsets;
  p.a_factor = g.a_factor;
  p.w_factor = g.w_factor;
  p.E = g.E;
  p.rows = (int32_t)g.rows;
  p.F = g.N;
  p.Kc = g.K;
  p.out = g.out;
  p.ldo = g.ldo;
  p.err = g.err;
  p.wait_ns = kWaitLimitNs;
  const bool f32 = g.out_dtype == MOE_F32;
  return nv ? launch_micro<OP_NV>(p, g.swiglu, f32, sms, st)
            : launch_micro<OP_MX>(p, g.swiglu, f32, sms, st);
}

}  // namespace moe
