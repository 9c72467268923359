// product.cuh -- device helpers shared by the products grouped by expert (grouped.cu: bf16,
// micro_gemm.cu: microscaled 4-bit operands): the tile table over ragged groups, copies, and the
// stores of an output chunk.
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kProductMaxGroups = 1023;

// Groups of rows [offsets[g], offsets[g+1]) as every thread of the kernel sees them: each bound is
// clamped into [0, rows] and behind the group's start, so that no tile leaves the buffers whatever
// the offsets hold; a bound that had to be moved raises kErrIndex.
struct GroupTable {
  int* tile_start;  // [G + 1] first tile of each group; [G]: all tiles
  int* row0;        // [G]     first row
  int* nrows;       // [G]     rows
};

// Block-wide (blockDim.x threads, scratch of as many ints); ends with __syncthreads().
__device__ __forceinline__ void build_group_table(const GroupTable& t, int* scratch,
                                                  const int32_t* offsets, int G, int rows, int rpt,
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
    const int n = (z2 - a2 + rpt - 1) / rpt * feat_tiles;
    t.tile_start[g] = n;  // count for now
    local += n;
  }
  scratch[threadIdx.x] = local;
  __syncthreads();
  for (int off = 1; off < nt; off <<= 1) {  // inclusive scan of the threads' sums
    const int v = threadIdx.x >= off ? scratch[threadIdx.x - off] : 0;
    __syncthreads();
    scratch[threadIdx.x] += v;
    __syncthreads();
  }
  int run = scratch[threadIdx.x] - local;
  for (int g = lo; g < hi; ++g) {
    const int n = t.tile_start[g];
    t.tile_start[g] = run;
    run += n;
  }
  if (threadIdx.x == nt - 1) t.tile_start[G] = scratch[nt - 1];
  __syncthreads();
}

struct ProductTile {
  int g;      // group
  int row0;   // first row of the tile
  int valid;  // rows of the tile inside the group, 1..rpt
  int ft;     // feature tile
  int lrow0;  // row0 within the group
};

// A group's tiles are numbered feature tile by feature tile, the row tiles inside: neighbouring CTAs
// share one weight tile, and the weights stream from memory once.
__device__ __forceinline__ ProductTile decode_product_tile(int tile, const GroupTable& t, int G,
                                                           int rpt) {
  int lo = 0, hi = G - 1;  // largest g with tile_start[g] <= tile (empty groups share starts)
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.tile_start[mid] <= tile)
      lo = mid;
    else
      hi = mid - 1;
  }
  const int rows = t.nrows[lo];
  const int nrt = (rows + rpt - 1) / rpt;
  const int local = tile - t.tile_start[lo];
  ProductTile p;
  p.g = lo;
  p.ft = local / nrt;
  p.lrow0 = (local - p.ft * nrt) * rpt;
  p.row0 = t.row0[lo] + p.lrow0;
  p.valid = min(rpt, rows - p.lrow0);
  return p;
}

__device__ __forceinline__ void tma_load_3d(void* smem_dst, const CUtensorMap* map, uint64_t* bar,
                                            int32_t x, int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Writes made by this thread through the generic proxy are visible to the async proxy (TMA, tcgen05).
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// One epilogue warp writes a chunk of 32 rows x 128 bytes, lane l holding row l's bytes in v: through
// a 4 KB buffer (16-byte pieces XOR-swizzled by row % 8, no bank conflicts either way), so that a store
// instruction covers four whole 128-byte rows.  Rows from `rows` on and 16-byte pieces from `pieces`
// on are not written.  kAdd: fp32 values are added onto what is there.
template <bool kAdd>
__device__ __forceinline__ void store_chunk(uint8_t* buf, int lane, const uint4 (&v)[8], uint8_t* row0,
                                            int64_t pitch, int rows, int pieces) {
  __syncwarp();  // the previous chunk has been read back
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *reinterpret_cast<uint4*>(buf + lane * 128 + ((j ^ (lane & 7)) << 4)) = v[j];
  __syncwarp();
  const int j = lane & 7;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = i * 4 + (lane >> 3);
    uint4 w = *reinterpret_cast<const uint4*>(buf + r * 128 + ((j ^ (r & 7)) << 4));
    if (r < rows && j < pieces) {
      uint4* dst = reinterpret_cast<uint4*>(row0 + r * pitch + j * 16);
      if (kAdd) {
        const uint4 o = *dst;
        w.x = __float_as_uint(__uint_as_float(w.x) + __uint_as_float(o.x));
        w.y = __float_as_uint(__uint_as_float(w.y) + __uint_as_float(o.y));
        w.z = __float_as_uint(__uint_as_float(w.z) + __uint_as_float(o.z));
        w.w = __float_as_uint(__uint_as_float(w.w) + __uint_as_float(o.w));
      }
      *dst = w;
    }
  }
}

}  // namespace moe
