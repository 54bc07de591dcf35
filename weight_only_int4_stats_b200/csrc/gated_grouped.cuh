// K8: the gated product of rows grouped by expert, H = silu(X W_gate[e]^T) * (X W_up[e]^T), with
// full-precision (fp16) weights: the calibration input of the experts' down projections.
//
// Tensor-bound. One tile is 128 rows of both weights (two A tiles and two TMEM accumulators)
// against up to BN tokens of one expert; units (expert, row tile, token tile) go round the
// persistent CTAs in gemm_fused.cuh's order, and the whole MMA warp walks the issue loop.
// Measured: 16384 rows over 8 experts of [14336, 4096] 3.36 ms with even experts, 1147 TFLOP/s, and
// 3.51 to 3.64 with uneven ones, run for long under the power limit; 1003 rows over 16 experts of
// [1536, 2048] 39 to 41 us, where 189 MB of weights would take 29 us. The tensor pipe works 77 % of the
// time in tiles of 64 (4096 rows over 4 experts of [4096, 4096], 201 us); the rest are the last round of
// CTAs and the waits for stages, of which each CTA reads its own (3.1 GB through L2 there).
//   warp 0       TMA producer of X and both weights, in stages of 64 k
//   warp 1       TMEM allocator and MMA issuer
//   warps 2, 3   idle
//   warps 4..11  epilogue: two warps per TMEM lane quarter, each half of the token columns (with
//                BN = 256 the accumulators fill TMEM, so the next tile waits for this one's
//                epilogue: eight warps and the fast exponential and division keep that short)
// kStack: 64 rows of each weight in one A tile of 128 (gate above up) and one accumulator, so that
// there is room for a second one and the epilogue overlaps the next tile even with BN = 256, and
// half as much work a tile fills the last round of CTAs better; X is read twice as often. Which
// calls take it stands at the launch. The up half of the accumulator lies in other warps' TMEM
// lanes than the gate half, so the warps of a pair trade tokens through shared memory.
#pragma once
#include "common.cuh"
#include "fused.cuh"
#include "gemm_fused.cuh"

namespace awq {

constexpr int kGgThreads = 12 * 32;
constexpr int kGgEpiWarp0 = 4;

template <int BN, bool kStack>
struct GgLayout {
  static constexpr int kRows = kStack ? 64 : 128;            // of each weight in a tile
  static constexpr int kXBytes = BN * kTcBK * 2;
  static constexpr int kABytes = kRows * kTcBK * 2;          // of one weight
  static constexpr int kStage = kXBytes + 2 * kABytes;
  static constexpr int kStages = kStack ? (BN == 256 ? 4 : BN == 128 ? 6 : 8)
                                        : (BN == 256 ? 3 : BN == 128 ? 4 : 5);
  static constexpr int kAccCols = kStack ? BN : 2 * BN;      // of a tile's accumulators
  static constexpr int kBufs = 2 * kAccCols <= 512 ? 2 : 1;
  static constexpr uint32_t kCols = kAccCols * kBufs;
  static constexpr int kXchgOff = kStages * kStage;          // kStack: up values on their way
  static constexpr int kBarOff = kXchgOff + (kStack ? 2 * 4 * 16 * 32 * 4 : 0);
  static constexpr int kTabOff = kBarOff + 256;
  static constexpr int kSmem = kTabOff + static_cast<int>(sizeof(GroupTable)) + 1024;
  static_assert(kSmem <= kTcSmemMax && (2 * kStages + 4) * 8 + 8 <= 256, "shared memory");
};

template <int BN, bool kStack>
__global__ void __launch_bounds__(kGgThreads, 1)
    gated_grouped_kernel(const __grid_constant__ CUtensorMap tmap_x,
                         const __grid_constant__ CUtensorMap tmap_g,
                         const __grid_constant__ CUtensorMap tmap_u, const FusedArgs args) {
  using L = GgLayout<BN, kStack>;
  constexpr int S = L::kStages, B = L::kBufs;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint64_t* empty = full + S;
  uint64_t* dfull = empty + S;
  uint64_t* dempty = dfull + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(dempty + 2);
  GroupTable* tab = reinterpret_cast<GroupTable*>(smem + L::kTabOff);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int G = static_cast<int>(args.K / kGroup);

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&dfull[i], 1);
      mbar_init(&dempty[i], 8);   // every epilogue warp
    }
    fence_barrier_init();
    tma_prefetch_desc(&tmap_x);
    tma_prefetch_desc(&tmap_g);
    tma_prefetch_desc(&tmap_u);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, L::kCols);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_launch_dependents();
  build_group_table(tab->off, tab->tile, args.offsets, args.E, args.M, BN);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const unsigned units =
      static_cast<unsigned>(args.row_tiles) * static_cast<unsigned>(tab->tile[args.E]);

  if (warp == 0) {
    // ------------------------------------------------------------------ producer
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (unsigned u = blockIdx.x; u < units && ok; u += gridDim.x) {
        const TfUnit t = tf_unit<BN>(u, args, tab, G);
        const int arow = static_cast<int>(t.e * args.N) + (kStack ? t.row0 / 2 : t.row0);
        for (int i = 0; i < 2 * G; ++i) {
          ok = mbar_wait(&empty[s], ph ^ 1);
          if (!ok) break;
          uint8_t* st = smem + s * L::kStage;
          mbar_arrive_expect_tx(&full[s], L::kStage);
          tma_load_2d(st, &tmap_x, &full[s], i * kTcBK, t.m0);
          tma_load_2d(st + L::kXBytes, &tmap_g, &full[s], i * kTcBK, arow);
          tma_load_2d(st + L::kXBytes + L::kABytes, &tmap_u, &full[s], i * kTcBK, arow);
          if (++s == S) { s = 0; ph ^= 1; }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    int s = 0, buf = 0;
    uint32_t ph = 0, dph = 0;
    bool ok = true;
    for (unsigned u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const TfUnit t = tf_unit<BN>(u, args, tab, G);
      const uint32_t idesc = f16_idesc(kTcBM, (t.cols + 15) / 16 * 16);
      const uint32_t d = tmem + buf * L::kAccCols;
      ok = __all_sync(0xffffffffu, mbar_wait(&dempty[buf], dph ^ 1));
      for (int i = 0; i < 2 * G && ok; ++i) {
        ok = __all_sync(0xffffffffu, mbar_wait(&full[s], ph));
        if (!ok) break;
        tc_fence_after();
        const uint32_t st = smem_u32(smem) + s * L::kStage;
        const uint64_t xd = sw128_kmajor_desc(st);
        const uint64_t gd = sw128_kmajor_desc(st + L::kXBytes);
        const uint64_t ud = sw128_kmajor_desc(st + L::kXBytes + L::kABytes);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            tc_mma_f16(d, gd + 2 * k, xd + 2 * k, idesc, (i | k) != 0 ? 1u : 0u);
            if (!kStack) tc_mma_f16(d + BN, ud + 2 * k, xd + 2 * k, idesc, (i | k) != 0 ? 1u : 0u);
          }
          tc_commit(&empty[s]);
          if (i == 2 * G - 1) tc_commit(&dfull[buf]);
        }
        __syncwarp();
        if (++s == S) { s = 0; ph ^= 1; }
      }
      if (++buf == B) { buf = 0; dph ^= 1; }
    }
  } else if (warp >= kGgEpiWarp0) {
    // ------------------------------------------------------------------ epilogue
    const int half = (warp - kGgEpiWarp0) >> 2;
    const int quarter = warp & 3;
    // kStack: quarters 0 and 1 hold gate, 2 and 3 the same rows' up
    const int row = 32 * (kStack ? quarter & 1 : quarter) + lane;
    const uint32_t td = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
    float* xchg = reinterpret_cast<float*>(smem + L::kXchgOff) + (2 * half + (quarter & 1)) * 512 + lane;
    __half* H = static_cast<__half*>(args.Y);
    int buf = 0, parity = 0;
    uint32_t ph = 0;
    // after a wait that ran out the warps still walk their tiles, without waiting or storing, so
    // that a pair of kStack does not part at its named barrier
    bool ok = true;
    for (unsigned u = blockIdx.x; u < units; u += gridDim.x) {
      const TfUnit t = tf_unit<BN>(u, args, tab, G);
      const int64_t n = (kStack ? t.row0 / 2 : t.row0) + row;
      const bool live = n < args.N && AWQ_IN_BOUNDS(t.m0 + t.cols <= args.M && t.e < args.E);
      ok = ok && __all_sync(0xffffffffu, mbar_wait(&dfull[buf], ph));
      tc_fence_after();
#pragma unroll 1
      for (int c0 = 16 * half; c0 < t.cols; c0 += 32) {
        uint32_t g[16], v[16];
        tmem_ld_32x32b_x16(td + buf * L::kAccCols + c0, g);
        if constexpr (kStack) {
          // up's warp hands over the first 8 tokens, gate's the last 8, and each finishes its 8;
          // the buffer alternates, so one barrier a turn also tells that the values before the
          // last have been read
          tmem_ld_wait();
          float* x = xchg + parity * 2048;
          parity ^= 1;
          if (quarter >= 2) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j * 32] = __uint_as_float(g[j]);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = g[8 + j];
          } else {
#pragma unroll
            for (int j = 8; j < 16; ++j) x[j * 32] = __uint_as_float(g[j]);
          }
          named_bar_sync(1 + 2 * half + (quarter & 1), 64);
          if (quarter >= 2) {
#pragma unroll
            for (int j = 0; j < 8; ++j) g[j] = __float_as_uint(x[(8 + j) * 32]);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __float_as_uint(x[j * 32]);
          }
        } else {
          tmem_ld_32x32b_x16(td + buf * L::kAccCols + BN + c0, v);
          tmem_ld_wait();
        }
        const int c1 = kStack && quarter >= 2 ? c0 + 8 : c0;
        if (ok && live) {
          __half* h = H + static_cast<int64_t>(t.m0 + c1) * args.N + n;
#pragma unroll
          for (int j = 0; j < (kStack ? 8 : 16); ++j)
            if (c1 + j < t.cols)
              h[j * args.N] = __float2half_rn(activate(__uint_as_float(g[j]), kActSilu) *
                                              __uint_as_float(v[j]));
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(&dempty[buf]);
      if (++buf == B) { buf = 0; ph ^= 1; }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kCols);
  }
}

}  // namespace awq
