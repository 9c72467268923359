// micro_gemm.cu -- products grouped by expert of microscaled 4-bit operands on the tensor cores
// (tcgen05 block-scaled MMA, fp32 sums in tensor memory), with a plain or a SwiGLU epilogue.
//
//   out[r][n] = g_a g_w[e] sum_blocks S_a S_w sum_{k in block} c_a c_w
//
// The MMA takes 64 channels of e2m1 codes of 128 rows and 256 weight rows, and their scales from tensor
// memory: two e8m0 scales a row (MOE_MICRO_MX, blocks of 32) or four e4m3 scales (MOE_MICRO_NV, blocks
// of 16).  It multiplies each block's sum by both scales in fp32, so nothing is decoded on the way.
//
// Kernel shape: persistent, one CTA per SM; warp 0 copies (codes by TMA with 128-byte swizzle: 256 channels a
// stage; scales as they lie, by bulk copies of whole 512-byte tiles), warp 1 moves each stage's scales
// into tensor memory (tcgen05.cp, every tile to the four quarters of the lanes) and issues the MMAs,
// warps 2..5 store.  Scales of rows outside a group are whatever the buffer holds; they reach only
// outputs that are not stored.
#include <atomic>
#include <cstring>

#include "internal.h"
#include "product.cuh"

namespace moe {

namespace {

constexpr int kThreads = 192;
constexpr int kOpA = 128 * 128;  // 128 rows x 256 codes
constexpr int kOpB = 256 * 128;
constexpr int kStaging = 4 * 4096;
constexpr int kBarBytes = 256;
constexpr int kTable = (3 * (kProductMaxGroups + 1)) * 4 + kThreads * 4;

template <bool kNv>
struct Shape {
  static constexpr int kTiles = kNv ? 4 : 2;          // scale tiles of 4 columns per 256 channels
  static constexpr int kSfA = kTiles * 512;
  static constexpr int kSfB = 2 * kTiles * 512;
  static constexpr int kStage = kOpA + kOpB + kSfA + kSfB;
  static constexpr int kStages = 3;
  static constexpr int kSmem = 1024 + kStages * kStage + kStaging + kBarBytes + kTable;
  static constexpr int kSfCols = 12 * kTiles;         // tensor memory columns of a stage's scales
  static_assert(kStage % 1024 == 0 && kSmem <= 232448, "shared memory of one CTA");
};

struct MicroGemmParams {
  CUtensorMap ma;  // codes of the rows
  CUtensorMap mw;  // codes of the weights
  const int32_t* offsets;
  const uint8_t* a_scales;
  const uint8_t* w_scales;
  const float* a_factor;
  const float* w_factor;
  int32_t E, rows, N, K, wrows, ktiles;  // wrows: weight rows of an expert
  void* out;
  int64_t ldo;
  uint32_t* err;
};

// Copy of `bytes` (a multiple of 16) to shared memory, counted on the barrier.
__device__ __forceinline__ void bulk_load(void* smem_dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(smem_dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// A 512-byte scale tile: 32 rows of 16 bytes without swizzle, 8-row groups 128 bytes apart.
__device__ __forceinline__ uint64_t scale_tile_desc(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(128u >> 4) << 32;
  d |= (uint64_t)1 << 46;
  return d;
}
// 32 lanes x 4 columns to each of the four lane quarters.
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

// Block-scaled MMA, e2m1 operands: bits [4,6) B's first scale byte, [7,10) and [10,13) formats (1 = e2m1),
// [17,23) N >> 3, 23 scale type (1 = e8m0, 0 = e4m3), [24,29) M >> 4, [29,31) A's first scale byte.
template <bool kNv>
__device__ __forceinline__ constexpr uint32_t idesc_micro(int n, int first) {
  return ((uint32_t)first << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) |
         (kNv ? 0u : 1u << 23) | ((128u >> 4) << 24) | ((uint32_t)first << 29);
}
template <bool kNv>
__device__ __forceinline__ void mma_micro(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if constexpr (kNv)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], "
        "[%5], p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], "
        "[%5], p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

template <bool kNv, bool kSwiGLU, bool kF32>
__global__ void __launch_bounds__(kThreads, 1)
    micro_product_kernel(const __grid_constant__ MicroGemmParams p) {
  using S = Shape<kNv>;
  constexpr int kFeat = kSwiGLU ? 128 : 256;  // output columns of a tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* staging = smem + S::kStages * S::kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + kStaging);
  uint64_t* empty = full + S::kStages;
  uint64_t* tfull = empty + S::kStages;
  uint64_t* tempty = tfull + 1;
  uint64_t* drain = tempty + 1;
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
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(tfull, 1);
    mbar_init(tempty, 128);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&p.ma);
    tma_prefetch_map(&p.mw);
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  build_group_table(tab, scratch, p.offsets, p.E, p.rows, 128, (p.N + kFeat - 1) / kFeat,
                    blockIdx.x == 0 ? p.err : nullptr);  // ends with __syncthreads
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const int total = tab.tile_start[p.E];
  const int nkb = (p.K + 255) / 256;

  if (warp == 0) {
    if (lane == 0) {
      uint32_t stage = 0, phase = 0;
      int armed = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
        const ProductTile t = decode_product_tile(tile, tab, p.E, 128);
        const int64_t wfirst = (int64_t)t.g * p.wrows;  // the expert's first weight row
        const int64_t wtile = (wfirst >> 7) + t.g;      // and first scale tile
        const int n0 = t.ft * kFeat;
        // weight rows of the tile's two halves within the expert, and whether the second exists
        const int h0 = n0, h1 = kSwiGLU ? p.N + n0 : n0 + 128;
        const bool two = kSwiGLU || h1 < p.N;
        const uint8_t* sa = p.a_scales + ((int64_t)((tab.row0[t.g] >> 7) + t.g + (t.lrow0 >> 7)) *
                                          p.ktiles) * 512;
        const uint8_t* sb0 = p.w_scales + (wtile + (h0 >> 7)) * p.ktiles * 512;
        const uint8_t* sb1 = p.w_scales + (wtile + (h1 >> 7)) * p.ktiles * 512;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, p.err)) {
            ok = false;
            break;
          }
          uint8_t* s = smem + stage * S::kStage;
          const int nt = min(S::kTiles, p.ktiles - kb * S::kTiles);
          const uint32_t sf = nt * 512;
          mbar_arrive_expect_tx(&full[stage], kOpA + kOpB + (two ? 3 : 2) * sf);
          tma_load_2d(s, &p.ma, &full[stage], kb * 128, t.row0);
          tma_load_2d(s + kOpA, &p.mw, &full[stage], kb * 128, (int)(wfirst + h0));
          tma_load_2d(s + kOpA + kOpB / 2, &p.mw, &full[stage], kb * 128, (int)(wfirst + h1));
          uint8_t* f = s + kOpA + kOpB;
          const int64_t ko = (int64_t)kb * S::kTiles * 512;
          bulk_load(f, sa + ko, sf, &full[stage]);
          bulk_load(f + S::kSfA, sb0 + ko, sf, &full[stage]);
          if (two) bulk_load(f + S::kSfA + S::kSfB / 2, sb1 + ko, sf, &full[stage]);
          if (armed < S::kStages) ++armed;
          if (++stage == S::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {  // let the copies of the last stage uses land
        for (int i = 0; i < armed; ++i) {
          if (stage == 0) {
            stage = S::kStages;
            phase ^= 1u;
          }
          --stage;
          mbar_wait(&full[stage], phase, nullptr, nullptr, kDrainLimitNs);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      uint32_t stage = 0, phase = 0, acc_phase = 0, buf = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
        if (!mbar_wait(tempty, acc_phase ^ 1u, abort_flag, p.err)) break;
        tc_fence_after();
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait(&full[stage], phase, abort_flag, p.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + stage * S::kStage);
          const uint32_t sb = sa + kOpA, fa = sb + kOpB, fb = fa + S::kSfA;
          const uint32_t ta = tmem_base + 256 + buf * S::kSfCols, tb = ta + 4 * S::kTiles;
          const int nt = min(S::kTiles, p.ktiles - kb * S::kTiles);
          for (int i = 0; i < nt; ++i) {
            copy_scales(ta + 4 * i, scale_tile_desc(fa + i * 512));
            copy_scales(tb + 8 * i, scale_tile_desc(fb + i * 512));
            copy_scales(tb + 8 * i + 4, scale_tile_desc(fb + S::kSfB / 2 + i * 512));
          }
          const int steps = min(4, (p.K - kb * 256) / 64);
          for (int s = 0; s < steps; ++s) {
            const int tile4 = kNv ? s : s >> 1;
            mma_micro<kNv>(tmem_base, sw128_kmajor_desc(sa + s * 32), sw128_kmajor_desc(sb + s * 32),
                           idesc_micro<kNv>(256, kNv ? 0 : (s & 1) * 2), ta + 4 * tile4,
                           tb + 8 * tile4, (kb | s) != 0);
          }
          mma_commit(&empty[stage]);
          buf ^= 1u;
          if (++stage == S::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        mma_commit(tfull);
        acc_phase ^= 1u;
      }
      mma_commit(drain);  // every MMA issued above has completed once this arrives
      mbar_wait(drain, 0, nullptr, nullptr, kDrainLimitNs);
    }
    __syncwarp();
  } else {
    const int quarter = warp & 3;
    uint8_t* buf = staging + (warp - 2) * 4096;
    uint32_t acc_phase = 0;
    constexpr int kEl = kF32 ? 4 : 2;
    constexpr int kChunk = 128 / kEl;
    const float ga = kNv && p.a_factor ? __ldg(p.a_factor) : 1.0f;
    for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
      const ProductTile t = decode_product_tile(tile, tab, p.E, 128);
      const float alpha = kNv && p.w_factor ? ga * __ldg(p.w_factor + t.g) : ga;
      if (!__all_sync(~0u, mbar_wait(tfull, acc_phase, abort_flag, p.err))) break;
      tc_fence_after();
      const uint32_t tb = tmem_base + ((uint32_t)(quarter * 32) << 16);
      const int vrows = t.valid - quarter * 32;
      const int cols = min(kFeat, p.N - t.ft * kFeat);
      uint8_t* dst = static_cast<uint8_t*>(p.out) +
                     (((int64_t)t.row0 + quarter * 32) * p.ldo + (int64_t)t.ft * kFeat) * kEl;
      if (vrows > 0) {
#pragma unroll 1
        for (int c = 0; c < cols; c += kChunk) {
          uint4 v[8];
#pragma unroll
          for (int h = 0; h < kChunk / 16; ++h) {
            uint32_t g[16];
            float f[16];
            tmem_ld16(tb + c + 16 * h, g);
            if constexpr (kSwiGLU) {
              uint32_t u[16];
              tmem_ld16(tb + 128 + c + 16 * h, u);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float x = alpha * __uint_as_float(g[i]);
                f[i] = (kF32 ? silu_accurate(x) : silu_fast(x)) * (alpha * __uint_as_float(u[i]));
              }
            } else {
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) f[i] = alpha * __uint_as_float(g[i]);
            }
            if constexpr (kF32) {
#pragma unroll
              for (int q = 0; q < 4; ++q)
                v[4 * h + q] = make_uint4(__float_as_uint(f[4 * q]), __float_as_uint(f[4 * q + 1]),
                                          __float_as_uint(f[4 * q + 2]), __float_as_uint(f[4 * q + 3]));
            } else {
#pragma unroll
              for (int q = 0; q < 2; ++q)
                v[2 * h + q] =
                    make_uint4(pack_bf16x2(f[8 * q], f[8 * q + 1]), pack_bf16x2(f[8 * q + 2], f[8 * q + 3]),
                               pack_bf16x2(f[8 * q + 4], f[8 * q + 5]), pack_bf16x2(f[8 * q + 6], f[8 * q + 7]));
            }
          }
          store_chunk<false>(buf, lane, v, dst + c * kEl, p.ldo * kEl, vrows, (cols - c) * kEl / 16);
        }
      }
      tc_fence_before();
      mbar_arrive(tempty);
      acc_phase ^= 1u;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

template <bool kNv, bool kSwiGLU, bool kF32>
cudaError_t launch(const MicroGemmParams& p, int grid, cudaStream_t st) {
  using S = Shape<kNv>;
  auto kern = micro_product_kernel<kNv, kSwiGLU, kF32>;
  static std::atomic<uint64_t> set{0};
  const cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kern), S::kSmem, &set);
  if (e != cudaSuccess) return e;
  LaunchScope ls(kSwiGLU ? "micro_product_swiglu" : "micro_product", st);
  kern<<<grid, kThreads, S::kSmem, st>>>(p);
  return cudaGetLastError();
}

template <bool kNv>
cudaError_t launch_format(const MicroGemmParams& p, bool swiglu, bool f32, int grid, cudaStream_t st) {
  if (swiglu) return f32 ? launch<kNv, true, true>(p, grid, st) : launch<kNv, true, false>(p, grid, st);
  return f32 ? launch<kNv, false, true>(p, grid, st) : launch<kNv, false, false>(p, grid, st);
}

}  // namespace

cudaError_t launch_micro_product(const MicroProduct& g, int sms, cudaStream_t st) {
  MicroGemmParams p;
  memset(&p, 0, sizeof p);
  p.wrows = g.swiglu ? 2 * g.N : g.N;
  const uint64_t half = (uint64_t)g.K / 2;
  if (!make_map_2d(&p.ma, 1, g.a, half, (uint64_t)g.rows, half, 128, 128) ||
      !make_map_2d(&p.mw, 1, g.w, half, (uint64_t)g.E * p.wrows, half, 128, 128))
    return cudaErrorInvalidValue;
  p.offsets = g.offsets;
  p.a_scales = g.a_scales;
  p.w_scales = g.w_scales;
  p.a_factor = g.a_factor;
  p.w_factor = g.w_factor;
  p.E = g.E;
  p.rows = (int32_t)g.rows;
  p.N = g.N;
  p.K = g.K;
  const int per = g.format == MOE_MICRO_NV ? 64 : 128;  // channels of a scale tile
  p.ktiles = (g.K + per - 1) / per;
  p.out = g.out;
  p.ldo = g.ldo;
  p.err = g.err;
  const bool f32 = g.out_dtype == MOE_F32;
  return g.format == MOE_MICRO_NV ? launch_format<true>(p, g.swiglu, f32, sms, st)
                                  : launch_format<false>(p, g.swiglu, f32, sms, st);
}

}  // namespace moe
