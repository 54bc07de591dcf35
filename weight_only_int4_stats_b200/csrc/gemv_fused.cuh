// K6: W4A16 products of few tokens per weight, with the fused epilogue, for one packed weight or
// for rows grouped by expert.
//
// HBM-bound: each packed weight of an expert with rows is read once and serves at most 8
// tokens, so the weights stream through shared memory and meet the tokens in registers, in
// mma.sync m16n8k16 (weights as the 16-row A operand, tokens as the 8-column B operand), as in
// the streaming decode kernel of gemv.cuh. What bounds it beside HBM is the instructions that
// make MMA operands of packed codes, so there are as few of them as can be:
//     y = sum_g s_g (sum_{k in g} q_k x_k - z_g sum_{k in g} x_k),
// and a code q in the low bits of an fp16 is the subnormal q 2^-24, exactly: the pairs
// (k0, k1) and (k4, k5) of a word are one mask each (after a shift by 8 for the second), the
// pairs (k2, k3) and (k6, k7), four bits higher, are q 2^-20. The two kinds go to MMAs of their
// own, and the sums are joined in fp32 (lo + hi / 16). No zero point is subtracted per weight:
// prepare_rows_kernel, launched first, writes each group's sum of x beside the tokens.
// That kernel also makes fp16 of bf16 activations (scaled by a power of two per row, so nothing
// a product could notice is lost), multiplies by inv_s in fp32 with one rounding, and lays the
// rows out as the B fragments are read.
// fp16 activations with inv_s come as two rows, x' = hi + lo (22 bits), whose products are added at
// the end, since one rounded row would err as much as the output's own rounding does.
//  * Work is a list of tiles (expert, block of up to 8 rows of X, 16 kRB weight rows)
//    that each CTA takes a contiguous range of; the experts' row counts come from the device.
//  * The tokens come through the same ring as the weights, chunk by chunk, one bulk copy per
//    row, so no CTA waits to stage X and X may be of any length.
//  * Scales and zero points are read from global memory one unit ahead (the producer warp
//    prefetches them to L2 a ring's depth ahead), so N may be any number.
// Measured on 8 experts of [14336, 4096], 4 rows each: 57.7 us, 4.3 TB/s of packed weights (the
// ring alone, without the arithmetic, streams about 5.3); 128 experts of [1536, 2048], 128 rows on 80 of
// them, 37.8 us with their preparation, 3.5 TB/s. Issue slots are half used: what is left is the
// latency of a consumer warp's chain, four warps a scheduler, and some 200 integer operations a
// unit that are not masks. Subtracting the zero point per weight instead took 47 us in the second
// case, units half as large 49 us, and a load converted where it is issued (the warp then waits
// for it there) 45 us.
// A unit (ring slot) is 8 kGW (row block, group) pairs: 16 kRB rows x 8 kGW / kRB groups. More
// rows per tile read X less often, fewer give more tiles: see the launch.
#pragma once
#include "common.cuh"
#include "fused.cuh"
#include "gemv.cuh"
#include "prepare.cuh"

namespace awq {

constexpr int kSfMaxSlots = 8;
constexpr int kGW = 4;   // groups of a unit that each consumer warp takes

struct StreamArgs {
  int64_t N, K;
  int T;                  // rows of X and Y
  int E;
  const int* offsets;     // [E + 1], or NULL for one expert with every row
  const __half* scales;   // [E, K / 128, N]
  const uint8_t* zeros;
  const uint8_t* xprep;   // what prepare_rows_kernel wrote of X
  FusedEpi epi;
  void* Y;
  int slots;              // ring depth
  int xrows;              // rows of X of a block (at most 8) and of a slot
  int split;              // 1: a token is two rows of X, the parts of x = hi + lo
};

// Shared memory from a 1024-byte aligned base: per slot the packed codes, then the token rows;
// barriers; two reduction buffers; the experts' table.
template <int kRB>
struct SfLayout {
  static constexpr int kChunkG = kG4Warps * kGW / kRB;     // groups per unit
  // a token's chunk: per group [8-k chunk j][32-k quarter c] of 8 fp16 in the order k0 k1 k4 k5
  // k2 k3 k6 k7, then the groups' sums;
  // 64 bytes more than a multiple of 128, so that the two tokens whose fragments a quarter-warp
  // reads at once lie in different banks
  static constexpr int kXChunk = kChunkG * 256 + (kChunkG * 4 + 63) / 64 * 64 +
                                 (kChunkG > 16 ? 64 : 0);
  static_assert(kXChunk % 128 == 64, "bank offset of the next token");
  static constexpr int kWBytes = kG4Warps * kGW * 1024;
  static constexpr int kRed = kG4Warps * 4 * 32 * 4;
  __host__ __device__ static int slot_bytes(int xrows) {
    return kWBytes + (xrows * kXChunk + 1023) / 1024 * 1024;
  }
  __host__ __device__ static int bar_off(int slots, int xrows) { return slots * slot_bytes(xrows); }
  __host__ __device__ static int red_off(int slots, int xrows) {
    return bar_off(slots, xrows) + 2 * kSfMaxSlots * 8;
  }
  __host__ __device__ static int tab_off(int slots, int xrows) {
    return red_off(slots, xrows) + 2 * kRed;
  }
  __host__ __device__ static int total(int slots, int xrows, int E) {
    return tab_off(slots, xrows) + 2 * (E + 1) * 4 + 1024;
  }
};

// A tile: expert, first token row of the block and its tokens, row tile of the expert's weight.
struct TileCursor {
  int e, m0, rows, nt;
};
// Moves the cursor to tile idx of all experts'.
__device__ __forceinline__ void tile_at(TileCursor& t, const int* off, const int* tile, int E,
                                        int64_t idx, int ntiles, int tok) {
  const auto first = [&](int e) { return static_cast<int64_t>(tile[e]) * ntiles; };
  if (idx < first(t.e) || idx >= first(t.e + 1)) {   // the last expert that starts at or before idx
    int lo = 0, n = E;
    while (n > 1) {
      const int half = n >> 1;
      if (first(lo + half) <= idx) {
        lo += half;
        n -= half;
      } else {
        n = half;
      }
    }
    t.e = lo;
  }
  const unsigned local = static_cast<unsigned>(idx - first(t.e));
  const int mb = static_cast<int>(local / static_cast<unsigned>(ntiles));
  t.nt = static_cast<int>(local) - mb * ntiles;
  t.m0 = off[t.e] + mb * tok;
  const int left = off[t.e + 1] - t.m0;
  t.rows = left < tok ? left : tok;
}

// From tile idx - 1 to tile idx: mostly the next row tile of the same block.
__device__ __forceinline__ void next_tile(TileCursor& t, const int* off, const int* tile, int E,
                                          int64_t idx, int ntiles, int tok) {
  if (t.nt + 1 < ntiles) ++t.nt;
  else tile_at(t, off, tile, E, idx, ntiles, tok);
}

__device__ __forceinline__ void lds128(uint32_t (&v)[4], uint32_t addr) {
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr));
}
__device__ __forceinline__ float lds32f(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
// D = A B, fp16 (mma_16816 adds to D).
__device__ __forceinline__ void mma_16816_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                               uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

template <int kRB, bool kBf16, int kBits>
__global__ void __launch_bounds__(kG4Threads, 2) stream_fused_kernel(
    const __grid_constant__ CUtensorMap tmap_w, const StreamArgs a) {
  using L = SfLayout<kRB>;
  using A = act_t<kBf16>;
  constexpr int kRows = kGemvRows * kRB;
  constexpr int kRowW = L::kChunkG * kGroup * kBits / 32;   // packed words of one row in a unit
  constexpr int kBoxes = kRowW / 32;                        // 128-byte boxes of a unit
  static_assert(kRowW % 32 == 0 && (kRB == 1 || kRB == 2 || kRB == 4), "whole boxes");
  constexpr int kBox = kRows * 128;
  constexpr uint32_t kWTx = kRows * kRowW * 4;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  const int S = a.slots;
  const int slot_bytes = L::slot_bytes(a.xrows);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::bar_off(S, a.xrows));
  uint64_t* empty = full + kSfMaxSlots;
  float* red = reinterpret_cast<float*>(smem + L::red_off(S, a.xrows));
  int* off = reinterpret_cast<int*>(smem + L::tab_off(S, a.xrows));
  int* tile = off + a.E + 1;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int Ki = static_cast<int>(a.K);
  const int G = Ki / kGroup;
  const int C = (G + L::kChunkG - 1) / L::kChunkG;
  const int ntiles = static_cast<int>((a.N + kRows - 1) / kRows);
  const int tokens = a.xrows >> a.split;   // of a block

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kG4Warps * 32);
    }
    fence_barrier_init();
    tma_prefetch_desc(&tmap_w);
  }
  // The kernel before this one is prepare_rows_kernel, which lets this one start only after its
  // own predecessors have completed: offsets, weights and scales are there, and only what it
  // writes has to be waited for.
  build_group_table(off, tile, a.offsets, a.E, a.T, tokens);
  __syncthreads();
  const int64_t total = static_cast<int64_t>(tile[a.E]) * ntiles;
  const int64_t P = gridDim.x, bx = blockIdx.x;
  const int64_t t0 = bx * (total / P) + (bx < total % P ? bx : total % P);
  const int64_t t1 = t0 + total / P + (bx < total % P ? 1 : 0);
  const int64_t units = (t1 - t0) * C;
  TileCursor cur{};

  if (warp == kG4Warps) {
    // ---------------------------------------------------------------- producer
    int slot = 0, chunk = 0;
    uint32_t ph = 0;
    int64_t idx = t0;
    auto weights = [&]() {   // lane 0: the unit's packed codes
      uint8_t* wb = smem + slot * slot_bytes;
      mbar_arrive_expect_tx(&full[slot], kWTx + static_cast<uint32_t>(cur.rows << a.split) * L::kXChunk);
      const int32_t row = static_cast<int32_t>(cur.e * a.N + static_cast<int64_t>(cur.nt) * kRows);
#pragma unroll
      for (int b = 0; b < kBoxes; ++b)
        tma_load_2d(wb + b * kBox, &tmap_w, &full[slot], chunk * kRowW + b * 32, row);
    };
    auto activations = [&]() {   // lane m: row m's chunk
      const int row = (cur.m0 << a.split) + lane;
      if (lane < cur.rows << a.split && AWQ_IN_BOUNDS(row < a.T << a.split && lane < a.xrows))
        bulk_load_1d(smem + slot * slot_bytes + L::kWBytes + lane * L::kXChunk,
                     a.xprep + (static_cast<int64_t>(row) * C + chunk) * L::kXChunk, L::kXChunk,
                     &full[slot]);
    };
    auto prefetch_sz = [&]() {   // scales (lanes 0..15) and zero points (16..31) of the unit
      const int g = chunk * L::kChunkG + (lane & 15);
      if ((lane & 15) < L::kChunkG && g < G) {   // (a row run of up to 256 bytes: its first line)
        const int64_t i = (static_cast<int64_t>(cur.e) * G + g) * a.N +
                          static_cast<int64_t>(cur.nt) * kRows;
        const void* p = lane < 16 ? static_cast<const void*>(a.scales + i)
                                  : static_cast<const void*>(a.zeros + i);
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
      }
    };
    auto advance = [&]() {
      if (++slot == S) { slot = 0; ph ^= 1; }
      if (++chunk == C) {
        chunk = 0;
        if (++idx < t1) next_tile(cur, off, tile, a.E, idx, ntiles, tokens);
      }
    };
    if (t0 < t1) tile_at(cur, off, tile, a.E, idx, ntiles, tokens);
    int64_t u = 0;
    const int64_t n_early = units < S ? units : S;
    for (; u < n_early; ++u) {   // the weights of the (empty) ring's units
      if (lane == 0) weights();
      prefetch_sz();
      advance();
    }
    pdl_wait();
    pdl_launch_dependents();
    slot = chunk = 0;
    ph = 0;
    idx = t0;
    if (t0 < t1) tile_at(cur, off, tile, a.E, idx, ntiles, tokens);
    for (int64_t v = 0; v < n_early; ++v) {   // and their activations
      activations();
      advance();
    }
    for (; u < units; ++u) {
      if (!__all_sync(0xffffffffu, mbar_wait(&empty[slot], ph ^ 1))) break;
      if (lane == 0) weights();
      __syncwarp();   // the transaction count is set before any of the copies can complete it
      activations();
      prefetch_sz();
      advance();
    }
    return;
  }

  // ------------------------------------------------------------------ consumers
  const float* factors = reinterpret_cast<const float*>(
      a.xprep + static_cast<int64_t>(a.T << a.split) * C * L::kXChunk);
  const int r = lane >> 2, c = lane & 3;
  const int rw = (r >> 1) + 4 * (r & 1);   // weight row of the MMA's row r (see gemv.cuh)
  const int rb = warp % kRB;               // this warp's row block, and its kGW groups
  const int gp = kGW * (warp / kRB);
  // Shared-memory addresses of this lane's operands in a slot at address 0; a slot starts on
  // 1024 bytes, so the swizzle's bits are the same in all of them. Codes: row `ra` of boxes of
  // kRows rows x 128 bytes, the row's 16-byte chunks xor-swizzled by ra % 8 (row ra + 8, 1024
  // bytes on, has the same pattern).
  const int ra = rb * kGemvRows + rw;
  uint32_t wofs[kGW][kBits == 4 ? 1 : 3];
#pragma unroll
  for (int q = 0; q < kGW; ++q) {
    const int gl = gp + q;
#pragma unroll
    for (int i = 0; i < (kBits == 4 ? 1 : 3); ++i) {
      const int w = kBits == 4 ? gl * 16 + 4 * c : gl * 12 + 3 * c + i;
      wofs[q][i] = static_cast<uint32_t>((w >> 5) * kBox + ra * 128 +
                                         ((((w >> 2) & 7) ^ (ra & 7)) << 4) + (w & 3) * 4);
    }
  }
  // A token that the block does not have reads another row: its column is not stored.
  const auto token_row = [&](int m) {
    return static_cast<uint32_t>(L::kWBytes + (m < a.xrows ? m : a.xrows - 1) * L::kXChunk);
  };
  const uint32_t xofs = token_row(r) + gp * 256 + c * 16;   // token r, the warp's first group
  const uint32_t sofs[2] = {token_row(2 * c) + L::kChunkG * 256 + gp * 4,   // sums of tokens 2c
                            token_row(2 * c + 1) + L::kChunkG * 256 + gp * 4};   // and 2c + 1
  bool ok = true;
  float total_acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};

  // Scales and zero points: of the 4 lanes that share the rows ra and ra + 8, lane c reads row
  // ra + 8 (c % 2) (the last one if it is past N) of the warp's groups c / 2, c / 2 + 2, ...; a
  // scale and a zero point travel as one fp16 pair and are exchanged within the four lanes.
  uint32_t psz = 0;   // walks the units of a tile (E G N < 2^31: see the launch)
  const uint32_t N32 = static_cast<uint32_t>(a.N);
  auto sz_tile = [&](const TileCursor& t) {
    const uint32_t n = static_cast<uint32_t>(t.nt) * kRows + ra + 8 * (c & 1);
    psz = static_cast<uint32_t>(t.e * G + gp + (c >> 1)) * N32 + (n < N32 ? n : N32 - 1);
  };
  // Loaded values are kept as they come and combined when they are used, a unit later: a
  // conversion beside the load would wait for it there.
  struct Raw {
    unsigned short s[kGW / 2];
    unsigned char z[kGW / 2];
  };
  auto load_sz = [&](Raw& z, int chunk) {
#pragma unroll
    for (int i = 0; i < kGW / 2; ++i) {
      z.s[i] = 0;
      z.z[i] = 0;
      if (chunk * L::kChunkG + gp + 2 * i + (c >> 1) < G) {
        z.s[i] = reinterpret_cast<const unsigned short*>(a.scales)[psz + 2 * i * N32];
        z.z[i] = a.zeros[psz + 2 * i * N32];
      }
    }
    psz += L::kChunkG * N32;
  };

  int slot = 0, chunk = 0, parity = 0;
  uint32_t ph = 0;
  int64_t idx = t0;
  TileCursor nxt{};
  Raw raw, raw_next;
  if (t0 < t1) {
    tile_at(cur, off, tile, a.E, idx, ntiles, tokens);
    nxt = cur;
    sz_tile(cur);
    load_sz(raw, 0);
  }
  const uint32_t smem_base = smem_u32(smem);
  pdl_wait();
  for (int64_t u = 0; u < units; ++u) {
    // the next unit's scales and zero points travel while this unit is awaited and computed
    const bool last = chunk == C - 1;
    if (u + 1 < units) {
      if (last) {
        next_tile(nxt, off, tile, a.E, idx + 1, ntiles, tokens);
        sz_tile(nxt);
      }
      load_sz(raw_next, last ? 0 : chunk + 1);
    }
    // what the epilogue reads of the outputs that this lane stores, ahead of the last unit
    const bool finisher = last && warp < kRB;
    FusedIn<kBf16> fin;
    // the lane's tokens are 2c and 2c + 1 of the block, or c with both parts
    const int fm = a.split ? c : 2 * c;
    float fs[2];        // their factors
    const int64_t fn = static_cast<int64_t>(cur.nt) * kRows + ra;
    FusedEpi epi = a.epi;
    if (finisher) {
      if (epi.bias != nullptr) epi.bias = static_cast<const A*>(epi.bias) + cur.e * a.N;
      const int64_t y = cur.m0 * a.N;
      if (epi.mul != nullptr) epi.mul = static_cast<const A*>(epi.mul) + y;
      if (epi.residual != nullptr) epi.residual = static_cast<const A*>(epi.residual) + y;
      fin.load(epi, fn, fm, a.N, cur.rows);
#pragma unroll
      for (int i = 0; i < 2; ++i) fs[i] = fm + i < cur.rows ? factors[cur.m0 + fm + i] : 0.0f;
    }
    ok = __all_sync(0xffffffffu, ok && mbar_wait(&full[slot], ph));
    uint32_t sz[kGW / 2];   // (scale, zero point) of this unit as fp16 pairs
#pragma unroll
    for (int i = 0; i < kGW / 2; ++i)   // 0x6400 | z is 1024 + z
      sz[i] = h2_as_u32(__halves2half2(
          __ushort_as_half(raw.s[i]),
          __hsub(__ushort_as_half(static_cast<unsigned short>(0x6400u | raw.z[i])),
                 __ushort_as_half(0x6400u))));
    const uint32_t sb = smem_base + static_cast<uint32_t>(slot * slot_bytes);
#pragma unroll
    for (int q = 0; q < kGW; ++q) {
      const uint32_t szA = __shfl_sync(0xffffffffu, sz[q >> 1], (lane & 28) + 2 * (q & 1));
      const uint32_t szB = __shfl_sync(0xffffffffu, sz[q >> 1], (lane & 28) + 2 * (q & 1) + 1);
      if (!ok || chunk * L::kChunkG + gp + q >= G) continue;
      uint32_t wA[4], wB[4];
      if constexpr (kBits == 4) {
        lds128(wA, sb + wofs[q][0]);
        lds128(wB, sb + wofs[q][0] + 1024);
      } else {
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          wA[i] = lds32(sb + wofs[q][i]);
          wB[i] = lds32(sb + wofs[q][i] + 1024);
        }
      }
      float lo[4], hi[4];   // sums of q x 2^-24 and of q x 2^-20
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t va[4], vb[4];   // the pairs of rows ra and ra + 8
        if constexpr (kBits == 4) {
          code_pairs(wA[j], va);
          code_pairs(wB[j], vb);
        } else {
          code3_pairs(wA[0], wA[1], wA[2], j, va);
          code3_pairs(wB[0], wB[1], wB[2], j, vb);
        }
        uint32_t xv[4];
        lds128(xv, sb + xofs + q * 256 + j * 64);
        const uint32_t a0[4] = {va[0], vb[0], va[2], vb[2]};
        const uint32_t a1[4] = {va[1], vb[1], va[3], vb[3]};
        if (j == 0) {
          mma_16816_zero(lo, a0, xv[0], xv[1]);
          mma_16816_zero(hi, a1, xv[2], xv[3]);
        } else {
          mma_16816<false>(lo, a0, xv[0], xv[1]);
          mma_16816<false>(hi, a1, xv[2], xv[3]);
        }
      }
      const float2 fA = __half22float2(u32_as_h2(szA)), fB = __half22float2(u32_as_h2(szB));
      constexpr float kHi = kBits == 4 ? 0.0625f : 1.0f;   // 3-bit codes all have one place
      const float s0 = lds32f(sb + sofs[0] + q * 4), s1 = lds32f(sb + sofs[1] + q * 4);
      const float d0 = fmaf(-fA.y, s0, fmaf(kHi, hi[0], lo[0]));
      const float d1 = fmaf(-fA.y, s1, fmaf(kHi, hi[1], lo[1]));
      const float d2 = fmaf(-fB.y, s0, fmaf(kHi, hi[2], lo[2]));
      const float d3 = fmaf(-fB.y, s1, fmaf(kHi, hi[3], lo[3]));
      total_acc[0] = fmaf(fA.x, d0, total_acc[0]);
      total_acc[1] = fmaf(fA.x, d1, total_acc[1]);
      total_acc[2] = fmaf(fB.x, d2, total_acc[2]);
      total_acc[3] = fmaf(fB.x, d3, total_acc[3]);
    }
    if (ok) mbar_arrive(&empty[slot]);
    if (++slot == S) { slot = 0; ph ^= 1; }
    raw = raw_next;
    ++chunk;

    if (last) {
      // Tile complete: the sums of the warps that share a row block, in warp order. The buffer
      // alternates, so the next tile's barrier is the only one that a writer has to pass
      // before it may overwrite what is read here.
      float* rd = red + parity * (L::kRed / 4);
      parity ^= 1;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        rd[(warp * 4 + i) * 32 + lane] = total_acc[i];
        total_acc[i] = 0.0f;
      }
      named_bar_sync(1 + rb, kG4Warps / kRB * 32);   // the warps of the row block
      if (finisher && ok) {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = 0.0f;
#pragma unroll
          for (int w = 0; w < kG4Warps / kRB; ++w) v[i] += rd[((w * kRB + rb) * 4 + i) * 32 + lane];
        }
        if (a.split) {
          v[0] += v[1];
          v[2] += v[3];
        }
        // (the codes came in as q 2^-24; the products by 2^24 and the factor, one after the other,
        // leave fp32's range only where the result does)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int m = fm + (i & 1);
          const int64_t n = fn + 8 * (i >> 1);
          if (m < cur.rows && n < a.N && !(a.split && (i & 1)) && AWQ_IN_BOUNDS(cur.m0 + m < a.T))
            static_cast<A*>(a.Y)[(static_cast<int64_t>(cur.m0) + m) * a.N + n] =
                float_to_act<kBf16>(fin.apply(epi, v[i] * 16777216.0f * fs[i & 1], i));
        }
      }
      chunk = 0;
      ++idx;
      cur = nxt;
    }
  }
}

}  // namespace awq
