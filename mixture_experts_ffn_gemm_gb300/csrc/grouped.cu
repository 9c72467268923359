// grouped.cu -- products grouped by expert with ragged sizes and their gradients, bf16 operands, fp32
// accumulation in tensor memory (tcgen05), rows [offsets[e], offsets[e+1]) of expert e:
//
//   forward   y[r][n]    = sum_k x[r][k]  W_e[n][k]       both operands contiguous along the sum
//   grad_x    dx[r][k]   = sum_n dy[r][n] W_e[n][k]       W_e's rows run along the sum
//   grad_w    dW_e[n][k] = sum_r dy[r][n] x[r][k]         both operands' rows run along the sum
//
// Tensor memory takes an operand either way: a box of 64 elements (128 bytes, one swizzle row) by R rows
// is "K-major" where the 64 elements run along the sum, and "MN-major" where the rows do; two bits of
// the instruction descriptor say which.  So no operand is transposed in memory in any direction.
//
// Kernel shape: persistent, one CTA per SM, warp 0 copies (TMA), warp 1 issues the MMAs, warps 2..5 store
// (their tile's tensor memory is read while the next tile is summed).  Tiles of 128 x 256 outputs, blocks
// of 64 along the sum.  Edges: the maps have the operands' true extents, so that copies fill with zeros
// behind N, K and the last row of the buffers; W's map has the expert as a third coordinate, so that
// rows behind W_e are zeros and not the next expert's.  grad_w sums over a group's rows, whose last block
// runs into the next group's rows: the MMA warp overwrites those rows of both operands with zeros in
// shared memory (zeros on one side alone would leave 0 x inf) before it issues the block.
#include <atomic>
#include <cstring>

#include "internal.h"
#include "product.cuh"

namespace moe {

namespace {

constexpr int kThreads = 192;
constexpr int kBK = 64;               // elements of the sum per stage
constexpr int kBox64 = 64 * 128;      // a box of 64 rows x 128 bytes
constexpr int kOpA = 128 * 128;       // 128 outputs x 64
constexpr int kOpB = 256 * 128;       // 256 outputs x 64
constexpr int kStage = kOpA + kOpB;
constexpr int kStages = 4;
constexpr int kStaging = 4 * 4096;
constexpr int kBarBytes = 256;
constexpr int kTable = (3 * (kProductMaxGroups + 1)) * 4 + kThreads * 4;
constexpr int kSmem = 1024 + kStages * kStage + kStaging + kBarBytes + kTable;
static_assert(kSmem <= 232448, "shared memory of one CTA");

struct GroupedParams {
  CUtensorMap ma;   // the operand whose rows (or columns) are the tile's 128 outputs
  CUtensorMap mb;   // the operand of the tile's 256 outputs
  const int32_t* offsets;
  int32_t E, rows, N, K;
  void* out;
  int64_t ldo;
  uint32_t* err;
};

// Descriptor of an MN-major operand: boxes of 64 outputs (128 bytes) x 64 rows of the sum, 128-byte
// swizzle; 8-row groups 1024 bytes apart (stride offset), boxes 8192 bytes apart (leading offset).
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(kBox64 >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

template <int kKind, bool kF32, bool kAdd>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_product_kernel(const __grid_constant__ GroupedParams p) {
  constexpr bool kGradW = kKind == MOE_PRODUCT_GRAD_W;
  constexpr bool kAMn = kGradW;
  constexpr bool kBMn = kKind != MOE_PRODUCT_FORWARD;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* staging = smem + kStages * kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + kStaging);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  GroupTable tab;
  tab.tile_start = reinterpret_cast<int*>(staging + kStaging + kBarBytes);
  tab.row0 = tab.tile_start + kProductMaxGroups + 1;
  tab.nrows = tab.row0 + kProductMaxGroups + 1;
  int* scratch = tab.nrows + kProductMaxGroups + 1;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 128);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&p.ma);
    tma_prefetch_map(&p.mb);
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  const int F = kKind == MOE_PRODUCT_FORWARD ? p.N : p.K;  // outputs along the 256 side
  const int fts = (F + 255) / 256;
  const int mts = (p.N + 127) / 128;                       // grad_w: tiles along N
  build_group_table(tab, scratch, p.offsets, p.E, p.rows, 128, kGradW ? 0 : fts,
                    blockIdx.x == 0 ? p.err : nullptr);  // ends with __syncthreads
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const int total = kGradW ? p.E * mts * fts : tab.tile_start[p.E];
  const int Kc = kKind == MOE_PRODUCT_GRAD_X ? p.N : p.K;  // the sum's length (grad_w: the rows)

  // grad_w: group, tile along N, tile along K; its sum runs over the group's rows
  auto tile_of = [&](int tile) {
    if constexpr (!kGradW) return decode_product_tile(tile, tab, p.E, 128);
    ProductTile t;
    t.g = tile / (mts * fts);
    const int local = tile - t.g * (mts * fts);
    t.ft = local / mts;
    t.lrow0 = (local - t.ft * mts) * 128;  // first n
    t.row0 = tab.row0[t.g];
    t.valid = min(128, p.N - t.lrow0);
    return t;
  };
  auto sum_len = [&](const ProductTile& t) { return kGradW ? tab.nrows[t.g] : Kc; };

  if (warp == 0) {
    if (lane == 0) {
      uint32_t stage = 0, phase = 0;
      int armed = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
        const ProductTile t = tile_of(tile);
        const int nkb = (sum_len(t) + kBK - 1) / kBK;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, p.err)) {
            ok = false;
            break;
          }
          uint8_t* sa = smem + stage * kStage;
          uint8_t* sb = sa + kOpA;
          mbar_arrive_expect_tx(&full[stage], kStage);
          const int kx = kb * kBK;
          if constexpr (kGradW) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
              tma_load_2d(sa + j * kBox64, &p.ma, &full[stage], t.lrow0 + j * 64, t.row0 + kx);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              tma_load_2d(sb + j * kBox64, &p.mb, &full[stage], t.ft * 256 + j * 64, t.row0 + kx);
          } else {
            tma_load_2d(sa, &p.ma, &full[stage], kx, t.row0);
            if constexpr (kBMn) {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                tma_load_3d(sb + j * kBox64, &p.mb, &full[stage], t.ft * 256 + j * 64, kx, t.g);
            } else {
              tma_load_3d(sb, &p.mb, &full[stage], kx, t.ft * 256, t.g);
            }
          }
          if (armed < kStages) ++armed;
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {  // let the copies of the last stage uses land
        for (int i = 0; i < armed; ++i) {
          if (stage == 0) {
            stage = kStages;
            phase ^= 1u;
          }
          --stage;
          mbar_wait(&full[stage], phase, nullptr, nullptr, kDrainLimitNs);
        }
      }
    }
  } else if (warp == 1) {
    // the whole warp follows the stages (it clears rows in grad_w); lane 0 issues
    constexpr uint32_t kIdesc =
        idesc_bf16_f32<128, 256>() | (kAMn ? 1u << 15 : 0u) | (kBMn ? 1u << 16 : 0u);
    uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
      const ProductTile t = tile_of(tile);
      const int len = sum_len(t);
      const int nkb = (len + kBK - 1) / kBK;
      if (nkb == 0) continue;  // grad_w of a group without rows: the epilogue writes zeros
      if (!__all_sync(~0u, mbar_wait(&tempty[acc], acc_phase ^ 1u, abort_flag, p.err))) break;
      tc_fence_after();
      const uint32_t d = tmem_base + acc * 256;
      for (int kb = 0; kb < nkb; ++kb) {
        ok = __all_sync(~0u, mbar_wait(&full[stage], phase, abort_flag, p.err));
        if (!ok) break;
        uint8_t* sa = smem + stage * kStage;
        const int left = min(kBK, len - kb * kBK);
        const int steps = (left + 15) / 16;
        if (kGradW && (left & 15)) {
          // rows left .. 16 * steps - 1 of the six boxes: 8 16-byte pieces each
          const int n = (16 * steps - left) * 8;
          for (int i = lane; i < 6 * n; i += 32) {
            const int box = i / n, q = i - box * n;
            *reinterpret_cast<uint4*>(sa + box * kBox64 + left * 128 + q * 16) =
                make_uint4(0, 0, 0, 0);
          }
          fence_async_smem();
        }
        __syncwarp();
        tc_fence_after();
        if (lane == 0) {
          const uint32_t a0 = smem_u32(sa), b0 = a0 + kOpA;
          for (int s = 0; s < steps; ++s) {
            const uint64_t ad = kAMn ? sw128_mnmajor_desc(a0 + s * 2048) : sw128_kmajor_desc(a0 + s * 32);
            const uint64_t bd = kBMn ? sw128_mnmajor_desc(b0 + s * 2048) : sw128_kmajor_desc(b0 + s * 32);
            mma_bf16(d, ad, bd, kIdesc, (kb | s) != 0);
          }
          mma_commit(&empty[stage]);
        }
        __syncwarp();
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      if (lane == 0) mma_commit(&tfull[acc]);
      __syncwarp();
      acc ^= 1u;
      if (acc == 0) acc_phase ^= 1u;
    }
    if (lane == 0) {  // every MMA issued above has completed once this commit arrives
      mma_commit(drain);
      mbar_wait(drain, 0, nullptr, nullptr, kDrainLimitNs);
    }
    __syncwarp();
  } else {
    const int quarter = warp & 3;
    uint8_t* buf = staging + (warp - 2) * 4096;
    uint32_t acc = 0, acc_phase = 0;
    constexpr int kEl = kF32 ? 4 : 2;           // bytes of an output
    constexpr int kChunk = 128 / kEl;           // columns of a chunk
    for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
      const ProductTile t = tile_of(tile);
      const bool none = kGradW && sum_len(t) == 0;
      if (kAdd && none) continue;
      if (!none) {
        const bool ok = __all_sync(~0u, mbar_wait(&tfull[acc], acc_phase, abort_flag, p.err));
        if (!ok) break;
        tc_fence_after();
      }
      const uint32_t tb = tmem_base + acc * 256 + ((uint32_t)(quarter * 32) << 16);
      const int vrows = t.valid - quarter * 32;
      const int cols = min(256, F - t.ft * 256);
      const int64_t orow = (kGradW ? (int64_t)t.g * p.N + t.lrow0 : (int64_t)t.row0) + quarter * 32;
      uint8_t* dst = static_cast<uint8_t*>(p.out) + (orow * p.ldo + (int64_t)t.ft * 256) * kEl;
      if (vrows > 0) {
#pragma unroll 1
        for (int c = 0; c < cols; c += kChunk) {
          uint4 v[8];
          if (none) {
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = make_uint4(0, 0, 0, 0);
          } else if constexpr (kF32) {
            uint32_t a[16], b[16];
            tmem_ld16(tb + c, a);
            tmem_ld16(tb + c + 16, b);
            tmem_ld_wait();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              v[q] = make_uint4(a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]);
              v[4 + q] = make_uint4(b[4 * q], b[4 * q + 1], b[4 * q + 2], b[4 * q + 3]);
            }
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t a[16], b[16];
              tmem_ld16(tb + c + 32 * h, a);
              tmem_ld16(tb + c + 32 * h + 16, b);
              tmem_ld_wait();
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                v[4 * h + q] = make_uint4(
                    pack_bf16x2(__uint_as_float(a[8 * q]), __uint_as_float(a[8 * q + 1])),
                    pack_bf16x2(__uint_as_float(a[8 * q + 2]), __uint_as_float(a[8 * q + 3])),
                    pack_bf16x2(__uint_as_float(a[8 * q + 4]), __uint_as_float(a[8 * q + 5])),
                    pack_bf16x2(__uint_as_float(a[8 * q + 6]), __uint_as_float(a[8 * q + 7])));
                v[4 * h + 2 + q] = make_uint4(
                    pack_bf16x2(__uint_as_float(b[8 * q]), __uint_as_float(b[8 * q + 1])),
                    pack_bf16x2(__uint_as_float(b[8 * q + 2]), __uint_as_float(b[8 * q + 3])),
                    pack_bf16x2(__uint_as_float(b[8 * q + 4]), __uint_as_float(b[8 * q + 5])),
                    pack_bf16x2(__uint_as_float(b[8 * q + 6]), __uint_as_float(b[8 * q + 7])));
              }
            }
          }
          store_chunk<kAdd>(buf, lane, v, dst + c * kEl, p.ldo * kEl, vrows,
                            (cols - c) * kEl / 16);
        }
      }
      if (!none) {
        tc_fence_before();
        mbar_arrive(&tempty[acc]);
        acc ^= 1u;
        if (acc == 0) acc_phase ^= 1u;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

template <int kKind, bool kF32, bool kAdd>
cudaError_t launch(const GroupedParams& p, int grid, cudaStream_t st, const char* label) {
  auto kern = grouped_product_kernel<kKind, kF32, kAdd>;
  static std::atomic<uint64_t> set{0};  // devices whose attribute is set
  const cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kern), kSmem, &set);
  if (e != cudaSuccess) return e;
  LaunchScope ls(label, st);
  kern<<<grid, kThreads, kSmem, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_grouped_product(const GroupedProduct& g, int sms, cudaStream_t st) {
  GroupedParams p;
  memset(&p, 0, sizeof p);
  const int kind = g.kind;
  const uint64_t E = g.E, N = g.N, K = g.K, R = g.rows;
  bool ok;
  if (kind == MOE_PRODUCT_GRAD_W) {
    ok = make_map_2d(&p.ma, 2, g.a, N, R, g.ld_a, 64, 64) &&
         make_map_2d(&p.mb, 2, g.b, K, R, g.ld_b, 64, 64);
  } else {
    const bool fwd = kind == MOE_PRODUCT_FORWARD;
    ok = make_map_2d(&p.ma, 2, g.a, fwd ? K : N, R, g.ld_a, 64, 128) &&
         make_map_3d(&p.mb, 2, g.b, K, N, E, 64, fwd ? 256 : 64);
  }
  if (!ok) return cudaErrorInvalidValue;
  p.offsets = g.offsets;
  p.E = g.E;
  p.rows = (int32_t)g.rows;
  p.N = g.N;
  p.K = g.K;
  p.out = g.out;
  p.ldo = g.ldo;
  p.err = g.err;
  const bool f32 = g.out_dtype == MOE_F32;
  if (kind == MOE_PRODUCT_FORWARD)
    return f32 ? launch<MOE_PRODUCT_FORWARD, true, false>(p, sms, st, "grouped_forward")
               : launch<MOE_PRODUCT_FORWARD, false, false>(p, sms, st, "grouped_forward");
  if (kind == MOE_PRODUCT_GRAD_X)
    return f32 ? launch<MOE_PRODUCT_GRAD_X, true, false>(p, sms, st, "grouped_grad_x")
               : launch<MOE_PRODUCT_GRAD_X, false, false>(p, sms, st, "grouped_grad_x");
  if (g.accumulate) return launch<MOE_PRODUCT_GRAD_W, true, true>(p, sms, st, "grouped_grad_w");
  return f32 ? launch<MOE_PRODUCT_GRAD_W, true, false>(p, sms, st, "grouped_grad_w")
             : launch<MOE_PRODUCT_GRAD_W, false, false>(p, sms, st, "grouped_grad_w");
}

}  // namespace moe
