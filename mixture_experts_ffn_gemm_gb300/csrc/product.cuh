// product.cuh -- helpers of the products grouped by expert (product.cu): the tile table over ragged groups,
// copies and commits of a pair of SMs, the launch in pairs.
#pragma once

#include "common.cuh"
#include "launch_order.cuh"

namespace moe {

constexpr int kProductMaxGroups = 1023;

// Groups of rows [offsets[g], offsets[g+1]) as every thread of the kernel sees them: each bound is
// clamped into [0, rows] and behind the group's start, so that no tile leaves the buffers whatever
// the offsets hold; a bound that had to be moved raises kErrIndex.
struct GroupTable {
  int* tile_start;  // [G + 1] first tile of each group; [G]: all tiles
  int* row0;        // [G]     first row
  int* nrows;       // [G]     rows
  int* cut;         // [G]     row tiles * 16 + (rows of one) / 32
};

// A group's row tiles: as few as hold `rows` in at most kMaxRows each, of about the same size (a tile of few
// rows takes as long as its weights' copies do), cut at multiples of kCut rows.
template <int kMaxRows, int kCut>
__device__ __forceinline__ int cut_rows(int rows) {
  const int n = (rows + kMaxRows - 1) / kMaxRows;
  return n * 16 + (n ? ((rows + n - 1) / n + kCut - 1) / kCut * (kCut / 32) : 0);
}

// Block-wide (scratch: an int a warp); ends with __syncthreads().  A group has
// feat_tiles tiles for each of its row tiles.
template <int kMaxRows, int kCut>
__device__ __forceinline__ void build_group_table(const GroupTable& t, int* scratch,
                                                  const int32_t* offsets, int G, int rows,
                                                  int feat_tiles, uint32_t* err) {
  const int nt = blockDim.x;
  const int per = (G + nt - 1) / nt;
  const int lo = threadIdx.x * per;
  const int hi = min(G, lo + per);
  int local = 0;
  for (int g = lo; g < hi; ++g) {
    const int a = offsets[g], z = offsets[g + 1];
    const int a2 = min(max(a, 0), rows);
    const int z2 = min(max(z, a2), rows);
    if (a2 != a || z2 != z) raise_flag(err, kErrIndex);
    t.row0[g] = a2;
    t.nrows[g] = z2 - a2;
    const int cut = cut_rows<kMaxRows, kCut>(z2 - a2);
    t.cut[g] = cut;
    const int n = (cut >> 4) * feat_tiles;
    t.tile_start[g] = n;  // count for now
    local += n;
  }
  // inclusive scan of the threads' sums: within the warps, then over the warps' totals
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int sum = local;
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(~0u, sum, off);
    if (lane >= off) sum += v;
  }
  if (lane == 31) scratch[warp] = sum;
  __syncthreads();
  int run = sum - local;  // tiles before this thread's first group
  for (int w = 0; w < warp; ++w) run += scratch[w];
  if (threadIdx.x == nt - 1) t.tile_start[G] = run + local;
  for (int g = lo; g < hi; ++g) {
    const int n = t.tile_start[g];
    t.tile_start[g] = run;
    run += n;
  }
  __syncthreads();
}

struct ProductTile {
  int g;      // group
  int row0;   // first row of the tile
  int valid;  // rows of the tile inside the group, 1..kMaxRows
  int ft;     // feature tile
  int lrow0;  // row0 within the group
};

// One thread of the (converged) warp.  The compiler knows that the branch holds a single thread, and keeps
// what tcgen05 and TMA instructions take from uniform registers there; after `lane == 0` it moves every
// operand into them, one by one, for each instruction.
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(yes));
  return yes != 0;
}

// The same value in every lane, as the compiler is to see it.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(~0u, v, 0); }

// The tiles of one warp, in increasing order.  A group's tiles are numbered feature tile by feature tile, the
// row tiles inside: neighbouring SMs share one weight tile, and the weights stream from memory once.
// A step looks at the starts of the next 32 groups at once (a search from the first group would cost a tile of
// a short sum as much as its MMAs).  The whole warp takes part, and all of it gets the same values.
struct TileWalk {
  int g = 0;
  __device__ __forceinline__ ProductTile at(int tile, const GroupTable& t, int G, int lane) {
    for (;;) {  // g: the last group that starts at `tile` or before
      const int next = g + 1 + lane;
      const uint32_t past = __ballot_sync(~0u, next < G && t.tile_start[min(next, G)] <= tile);
      g += __popc(past);
      if (past != ~0u) break;
    }
    ProductTile p;
    p.g = g;
    const int cut = uniform(t.cut[g]), local = tile - uniform(t.tile_start[g]);
    const int rows = uniform(t.nrows[g]), rpt = (cut & 15) * 32, nrt = cut >> 4;
    p.ft = local;
    p.lrow0 = 0;
    if (nrt > 1) {
      p.ft = local / nrt;
      p.lrow0 = (local - p.ft * nrt) * rpt;
    }
    p.row0 = uniform(t.row0[g]) + p.lrow0;
    p.valid = min(rpt, rows - p.lrow0);
    return p;
  }
};

// TMA copy of a 3D box into this CTA's shared memory of a pair, completion counted on the barrier at
// shared::cluster address `bar_cluster`.
__device__ __forceinline__ void tma_load_3d_pair(void* smem_dst, const CUtensorMap* map,
                                                 uint32_t bar_cluster, int32_t x, int32_t y,
                                                 int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Bulk tensor store of a 3D box from shared memory (kAdd: fp32 addition onto what is there), tracked in
// the thread's bulk async group.
template <bool kAdd>
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* smem_src, int32_t x,
                                             int32_t y, int32_t z) {
  if constexpr (kAdd)
    asm volatile(
        "cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], "
        "[%1];\n\tcp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(map)),
        "r"(smem_u32(smem_src)), "r"(x), "r"(y), "r"(z)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];\n\t"
        "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(map)),
        "r"(smem_u32(smem_src)), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// Arrive once on the barrier at `bar`'s offset in both CTAs of the pair when every pair MMA and copy into
// tensor memory that this thread issued before has completed.
__device__ __forceinline__ void commit_both(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}

// Arrive once on this CTA's `bar` alone when every pair MMA this thread issued before has completed.
__device__ __forceinline__ void mma_commit_pair_own(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
      : "memory");
}

// Writes made by this thread through the generic proxy are visible to the async proxy (TMA, tcgen05).
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Launch of a kernel whose CTAs work in pairs (clusters of two), one CTA per SM.  Its CTAs may start while a
// kernel before it that allows it (allow_next_kernel) still runs: barriers and tensor memory are set up
// meanwhile (a quantisation and the product of eight rows: 20.5 -> 18.5 us, replayed from a graph 16.0 -> 15.0;
// with the quantisation launched the same way 15.7 and 14.7).
template <typename Kernel, typename Params>
inline cudaError_t launch_pairs(Kernel kern, int sms, int threads, int smem, cudaStream_t st,
                                const Params& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(sms & ~1));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  // the kernel waits for the one before it by itself (wait_for_prior_kernel)
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace moe
