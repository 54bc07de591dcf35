// K7: W4A16 GEMM on the 5th-generation tensor cores with the fused epilogue, for one packed
// weight or for rows grouped by expert.
//
// As in gemm_tc.cuh the MMA's M side is 128 weight rows and its N side up to BN tokens, with
// the output in TMEM as 128 lanes (weight rows) x token columns, and the work units (expert, row
// tile, token tile, K slice) go round the persistent CTAs. What differs is where the
// dequantized weights go: not through shared memory but straight into TMEM, as the MMA's A
// operand (lane = weight row, each 32-bit column two consecutive k). In gemm_tc.cuh a 128 x 128
// group of weights costs shared memory a 32 KB write, a 32 KB read by the tensor core and, in
// the packed reads, bank conflicts; with few tokens per weight that is what bounds it (1.7 TB/s
// of packed weights at 16 to 64 tokens). Here a builder thread owns one weight row: it reads
// the row's codes of a block (at 4 bits without bank conflicts), dequantizes in registers and
// stores the block's columns of its lane.
//   warp 0       TMA producer of X
//   warp 1       TMEM allocator and single-thread tcgen05.mma issuer
//   warp 2       TMA producer of packed codes, prefetch of scales and zero points
//   warp 3       producer of inv_s, into the packed codes' slots (idle without it)
//   warps 4..19  builders: four sets of four warps (a warp reaches the TMEM lanes of its quarter,
//                warp % 4); the sets take the K blocks in turn, so that four chains of
//                shared-memory reads, arithmetic, TMEM stores and barriers run at once
//   warps 20..27 epilogue: two warps per quarter, each half of the token columns
// X comes in blocks of 128 k (a group). A stages hold a group too, or half of one with BN = 192.
// TMEM: two accumulators of BN columns and kNA A stages. BN stops at 192 so that both accumulators
// fit beside four A stages and a tile's epilogue always overlaps the next tile's products. (A
// set's turn comes round after four A stages, and a barrier's parity tells only neighbouring
// phases apart: a stage must not come round sooner, so kNA >= the sets.)
// Waiting on a barrier whose phase is already complete still takes about 100 cycles, so a step is as
// long as it can be: the MMA issuer takes a whole group. (Polling the next group's barriers ahead
// of a group's MMAs was slower: [14336, 4096] with 4096 tokens 442 us against 428.)
// The products are fp16: bf16 activations come from prepare_rows_kernel as fp16, scaled by a power
// of two per row (with inv_s already in), and the epilogue takes the row's factor off. bf16
// weights would need (q - z) * scale in two bf16 parts to be rounded only once (19 operations a
// word of 8 codes, 45 with inv_s, against 13), and the dequantization is what bounds this kernel.
// Measured: 8 experts of [14336, 4096] with 128 rows 93 us, 2.7 TB/s of packed weights; with 2048
// rows 279 us, 863 TFLOP/s, in a short run and 329 run for long; [14336, 4096] x 4096 tokens 434 us,
// 1110 TFLOP/s, short and 491 long, where the plain product takes 398 and 458 and, with bias and
// gelu as two more passes, 578 and 647. Few rows: the dequantization (13 operations a word of 8
// codes; 24 at 3 bits) on 4 warps a scheduler, and their barriers. Many rows: the tensor pipe works
// 58 % of the time (4096 tokens), since a group's weights are dequantized again for every 192 tokens,
// the MMA issuer spends about 200 cycles a group waiting and counting, and each CTA reads its own X;
// run for long, the 1000 W power limit takes the SM clock to 1.45 GHz besides (2.2 ms for 8 experts
// of [4096, 14336] with 16384 rows).
// Packed codes: 4 bits: boxes of 128 rows x 128 bytes (two groups) with the 128-byte swizzle;
// 3 bits: one box of 3 or 5 groups (an odd multiple of 48 bytes per row: eight consecutive rows begin
// in eight different bank groups, but the 8-byte reads of sixteen rows at once meet two to a bank).
#pragma once
#include "common.cuh"
#include "fused.cuh"
#include "gemm_tc.cuh"
#include "gemv.cuh"
#include "prepare.cuh"

namespace awq {

constexpr int kTfSets = 4;
constexpr int kTfBuildWarp0 = 4;
constexpr int kTfEpiWarp0 = kTfBuildWarp0 + 4 * kTfSets;
constexpr int kTfThreads = (kTfEpiWarp0 + 8) * 32;

template <int BN, int kBits>
struct TfLayout {
  static_assert(BN == 32 || BN == 64 || BN == 128 || BN == 192, "token tiles");
  static constexpr int kXHalf = BN * kTcBK * 2;                   // 64 k of X
  static constexpr int kXBytes = 2 * kXHalf;
  static constexpr int kXStages = BN >= 128 ? 3 : BN == 64 ? 4 : 6;
  static constexpr int kHB = BN == 192 ? 1 : 2;                   // 64-k halves of an A stage
  static constexpr int kACols = kHB * 32;                         // TMEM columns of an A stage
  static constexpr int kNA = BN >= 128 ? 4 : 6;
  static constexpr int kAccCol = 0;
  static constexpr int kACol = 2 * BN;
  static_assert(kACol + kNA * kACols <= 512 && kNA >= kTfSets, "TMEM columns");
  static constexpr int kPG = kBits == 4 ? (BN == 192 ? 2 : 4) : (BN == 192 ? 3 : 5);
  static constexpr int kRowBytes = kBits == 4 ? 128 : kPG * 48;   // of a box
  static constexpr int kBoxes = kBits == 4 ? kPG / 2 : 1;
  static constexpr int kBoxBytes = kTcBM * kRowBytes;
  static constexpr int kPBytes = (kBoxes * kBoxBytes + 1023) / 1024 * 1024;
  static constexpr int kInvBytes = kPG * kGroup * 4;
  static constexpr int kBarBytes = 512;
  static constexpr int kFit = (kTcSmemMax - 1024 - kBarBytes - static_cast<int>(sizeof(GroupTable)) -
                               kXStages * kXBytes) / (kPBytes + kInvBytes);
  static constexpr int kPSlots = kFit < 6 ? kFit : 6;
  static_assert(kPSlots >= 2, "packed ring");
  static constexpr int kPOff = kXStages * kXBytes;
  static constexpr int kIOff = kPOff + kPSlots * kPBytes;
  static constexpr int kBarOff = kIOff + kPSlots * kInvBytes;
  static constexpr int kTabOff = kBarOff + kBarBytes;
  static constexpr int kSmem = kTabOff + static_cast<int>(sizeof(GroupTable)) + 1024;
  static_assert((2 * kXStages + 2 * kNA + 2 * kPSlots + 4) * 8 + 8 <= kBarBytes, "barriers");
};

// D[tmem] (+)= A[tmem] * B[smem desc]^T, 16-bit inputs, fp32 accumulator, one CTA.
__device__ __forceinline__ void tc_mma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                              uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Whether the phase of that parity is complete, at once (mbar_try_wait may suspend the thread for
// a while when it is not).
__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// mbar_wait on two barriers at once: their first polls are in flight together.
__device__ __forceinline__ bool mbar_wait_all(uint64_t* b0, uint32_t p0, uint64_t* b1, uint32_t p1) {
  const bool r0 = mbar_test_wait(b0, p0), r1 = mbar_test_wait(b1, p1);
  return (r0 || mbar_wait(b0, p0)) && (r1 || mbar_wait(b1, p1));
}

// mbar_wait for a warp that has time: it looks only now and then, so that its polling takes no
// issue slots from the warps that set the pace.
__device__ __forceinline__ bool mbar_wait_lazy(uint64_t* bar, uint32_t parity) {
  for (int i = 0; i < 64; ++i) {
    if (mbar_test_wait(bar, parity)) return true;
    __nanosleep(256);
  }
  return mbar_wait(bar, parity);
}

// True in one lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// 32 lanes x 16 consecutive 32-bit columns from registers (thread i: lane base + i).
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

struct FusedArgs {
  int64_t M, N, K;          // rows of X and Y; weight rows of an expert
  int E;
  int row_tiles;            // 128-row tiles of an expert's weight
  int k_splits;             // > 1: a unit takes a slice of K's groups
  const int* offsets;       // [E + 1], or NULL for one expert with every row
  const __half* scales;     // [E, K / 128, N]
  const uint8_t* zeros;
  const float* inv_s;       // [E, K] or NULL
  const float* factors;     // [M]: factors of prepared activations, or NULL
  float* partial;           // [k_splits, M, N]
  FusedEpi epi;
  void* Y;
};

// A work unit: K slice, expert, row tile and token tile, and the slice's groups.
struct TfUnit {
  int e, row0, m0, cols;      // expert, first weight row, first token, its tokens (at most BN)
  int g0, groups, ksplit;
};
// Unit u (32-bit: see the launch). Units of a slice sweep the token tiles of 16 row tiles at a
// time (so the units in flight share a few weight and token tiles in L2).
template <int BN>
__device__ __forceinline__ TfUnit tf_unit(unsigned u, const FusedArgs& a, const GroupTable* tab, int G) {
  TfUnit t;
  const unsigned rt = static_cast<unsigned>(a.row_tiles);
  const unsigned tiles = rt * static_cast<unsigned>(tab->tile[a.E]);
  t.ksplit = 0;
  if (a.k_splits > 1) {
    t.ksplit = static_cast<int>(u / tiles);
    u -= t.ksplit * tiles;
  }
  int lo = 0, n = a.E;   // the last expert that starts at or before the unit
  while (n > 1) {
    const int half = n >> 1;
    if (rt * static_cast<unsigned>(tab->tile[lo + half]) <= u) {
      lo += half;
      n -= half;
    } else {
      n = half;
    }
  }
  t.e = lo;
  u -= rt * static_cast<unsigned>(tab->tile[lo]);
  const unsigned mt = static_cast<unsigned>(tab->tile[lo + 1] - tab->tile[lo]);
  const unsigned per = kTcRasterRows * mt;
  const unsigned grp = u / per, in = u - grp * per;
  const unsigned first = grp * kTcRasterRows;
  const unsigned here = rt - first < kTcRasterRows ? rt - first : kTcRasterRows;
  const unsigned m = in / here;
  t.row0 = static_cast<int>(first + in - m * here) * kTcBM;
  t.m0 = tab->off[lo] + static_cast<int>(m) * BN;
  const int left = tab->off[lo + 1] - t.m0;
  t.cols = left < BN ? left : BN;
  t.g0 = static_cast<int>(static_cast<int64_t>(t.ksplit) * G / a.k_splits);
  t.groups = static_cast<int>(static_cast<int64_t>(t.ksplit + 1) * G / a.k_splits) - t.g0;
  return t;
}

// Two fp32 products in one instruction.
__device__ __forceinline__ float2 mul_f32x2(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(static_cast<uint64_t>(__float_as_uint(a.y)) << 32 | __float_as_uint(a.x)),
        "l"(static_cast<uint64_t>(__float_as_uint(b.y)) << 32 | __float_as_uint(b.x)));
  return make_float2(__uint_as_float(static_cast<uint32_t>(d)),
                     __uint_as_float(static_cast<uint32_t>(d >> 32)));
}

// 32 weights (one 32-k quarter of a group: 4 words at 4 bits, 3 at 3 bits) of a row to 16 MMA
// operand pairs: exact q - z, then the scale with one rounding to fp16; with inv_s (this
// quarter's) scale * inv_s[k] in fp32 and the product rounded once. (A factor rounded to fp16
// before the product would make three roundings with the output's, sqrt(3) of one, where this
// has sqrt(2): 2.9e-4 of an fp16 output's norm against 2.1e-4 of the output's rounding alone. The
// MMA takes 16-bit operands: a weight of more bits would be two of them, and twice the dequantization
// and MMAs. Under a bf16 output, rounded at 2^-9, an fp16 weight's 2^-12 does not show.)
template <int kBits, bool kInv>
__device__ __forceinline__ void dequant32(const uint32_t* w, uint32_t z, uint32_t sc, float scf,
                                          const float* inv, uint32_t (&o)[16]) {
  const uint32_t bias = (0x6400u | z) * 0x00010001u;
  if constexpr (kBits == 4) {
    const __half2 hi = u32_as_h2((0xD400u | (z << 4)) * 0x00010001u);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t v[4];
      dequant_word_qz(w[j], u32_as_h2(bias), hi, v);
#pragma unroll
      for (int q = 0; q < 4; ++q) o[4 * j + q] = v[q];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t v[4];
      raw3_chunk<false>(w[0], w[1], w[2], j, v);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        o[4 * j + q] = h2_as_u32(__hsub2(u32_as_h2(v[q]), u32_as_h2(bias)));
    }
  }
  if constexpr (!kInv) {
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j] = h2_as_u32(__hmul2(u32_as_h2(o[j]), u32_as_h2(sc)));
  } else {
    const float2 ss = make_float2(scf, scf);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float4 s = reinterpret_cast<const float4*>(inv)[j];
      float2 f = mul_f32x2(__half22float2(u32_as_h2(o[2 * j])), mul_f32x2(ss, make_float2(s.x, s.y)));
      o[2 * j] = float2_to_act2<false>(f.x, f.y);
      f = mul_f32x2(__half22float2(u32_as_h2(o[2 * j + 1])), mul_f32x2(ss, make_float2(s.z, s.w)));
      o[2 * j + 1] = float2_to_act2<false>(f.x, f.y);
    }
  }
}

// 16 token columns of one weight row through the epilogue, the activation known at compile time.
// y: the row's first output of the columns, nc of them are its expert's tokens. With bf16 outputs
// lane j holds the factor of token j's prepared activations. The epilogue warps share the issue
// slots with the builders, so what is absent costs nothing here: written with a multiply and an
// add of a default for each output it took 35,000 cycles a tile of 192 tokens, as much as the
// tile's products.
template <bool kBf16, int kAct>
__device__ __forceinline__ void fused_columns(const FusedArgs& a, int64_t y, int nc, bool live,
                                              float bias, float factor, uint32_t (&v)[16]) {
  using A = act_t<kBf16>;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    float x = __uint_as_float(v[j]);
    if constexpr (kBf16) x = fmaf(x, __shfl_sync(0xffffffffu, factor, j), bias);
    else x += bias;
    v[j] = __float_as_uint(activate(x, kAct));
  }
  if (!live) return;
  if (a.epi.mul != nullptr) {
    const A* p = static_cast<const A*>(a.epi.mul) + y;
    A m[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) m[j] = j < nc ? p[j * a.N] : A(0.0f);
#pragma unroll
    for (int j = 0; j < 16; ++j)
      v[j] = __float_as_uint(__uint_as_float(v[j]) * act_to_float<kBf16>(m[j]));
  }
  if (a.epi.residual != nullptr) {
    const A* p = static_cast<const A*>(a.epi.residual) + y;
    A r[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) r[j] = j < nc ? p[j * a.N] : A(0.0f);
#pragma unroll
    for (int j = 0; j < 16; ++j)
      v[j] = __float_as_uint(__uint_as_float(v[j]) + act_to_float<kBf16>(r[j]));
  }
  A* p = static_cast<A*>(a.Y) + y;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    if (j < nc) *p = float_to_act<kBf16>(__uint_as_float(v[j]));
    p += a.N;
  }
}

// A warp's share of a tile's token columns (alternate 16), from its TMEM lanes at td.
template <bool kBf16, int kAct>
__device__ __forceinline__ void fused_tile(const FusedArgs& a, const TfUnit& t, int64_t n, bool live,
                                           float bias, int half, int lane, uint32_t td) {
#pragma unroll 1
  for (int c0 = 16 * half; c0 < t.cols; c0 += 32) {
    float factor = 0.0f;
    if (kBf16 && c0 + (lane & 15) < t.cols) factor = a.factors[t.m0 + c0 + (lane & 15)];
    uint32_t v[16];
    tmem_ld_32x32b_x16(td + c0, v);
    tmem_ld_wait();
    fused_columns<kBf16, kAct>(a, static_cast<int64_t>(t.m0 + c0) * a.N + n,
                               t.cols - c0, live, bias, factor, v);
    __syncwarp();   // the next TMEM load is the whole warp's
  }
}

// The same for a slice of K: partial sums, times the factors.
template <bool kBf16>
__device__ __forceinline__ void partial_tile(const FusedArgs& a, const TfUnit& t, int64_t n, bool live,
                                             int half, int lane, uint32_t td) {
#pragma unroll 1
  for (int c0 = 16 * half; c0 < t.cols; c0 += 32) {
    float factor = 1.0f;
    if (kBf16 && c0 + (lane & 15) < t.cols) factor = a.factors[t.m0 + c0 + (lane & 15)];
    uint32_t v[16];
    tmem_ld_32x32b_x16(td + c0, v);
    tmem_ld_wait();
    if constexpr (kBf16) {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        v[j] = __float_as_uint(__uint_as_float(v[j]) * __shfl_sync(0xffffffffu, factor, j));
    }
    if (live) {
      float* p = a.partial + (static_cast<int64_t>(t.ksplit) * a.M + t.m0 + c0) * a.N + n;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        if (j < t.cols - c0) *p = __uint_as_float(v[j]);
        p += a.N;
      }
    }
    __syncwarp();
  }
}

// kBf16: the type of Y and the epilogue's operands. kInv: inv_s goes into the weights.
template <int BN, bool kBf16, int kBits, bool kInv>
__global__ void __launch_bounds__(kTfThreads, 1)
    tc_fused_kernel(const __grid_constant__ CUtensorMap tmap_x,
                    const __grid_constant__ CUtensorMap tmap_w, const FusedArgs args, const int early) {
  using L = TfLayout<BN, kBits>;
  constexpr int NX = L::kXStages, NA = L::kNA, P = L::kPSlots, kPG = L::kPG;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  uint64_t* xfull = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint64_t* xempty = xfull + NX;
  uint64_t* afull = xempty + NX;
  uint64_t* aempty = afull + NA;
  uint64_t* pfull = aempty + NA;
  uint64_t* pempty = pfull + P;
  uint64_t* dfull = pempty + P;
  uint64_t* dempty = dfull + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(dempty + 2);
  GroupTable* tab = reinterpret_cast<GroupTable*>(smem + L::kTabOff);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int G = static_cast<int>(args.K / kGroup);

  if (threadIdx.x == 0) {
    for (int i = 0; i < NX; ++i) {
      mbar_init(&xfull[i], 1);
      mbar_init(&xempty[i], 1);
    }
    for (int i = 0; i < NA; ++i) {
      mbar_init(&afull[i], 4);    // the warps of a builder set
      mbar_init(&aempty[i], 1);
    }
    for (int i = 0; i < P; ++i) {
      mbar_init(&pfull[i], kInv ? 2 : 1);   // the codes' producer, and that of inv_s
      mbar_init(&pempty[i], 4 * kTfSets);   // every builder warp
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&dfull[i], 1);
      mbar_init(&dempty[i], 8);   // every epilogue warp
    }
    fence_barrier_init();
    tma_prefetch_desc(&tmap_x);
    tma_prefetch_desc(&tmap_w);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  // With `early` (one weight, whose codes, scales and zero points the preceding kernel does not
  // write) only what that kernel may have written waits for it, each in the warps that touch it: X,
  // inv_s, bias, mul, residual, Y, partial sums.
  if (!early) pdl_wait();
  build_group_table(tab->off, tab->tile, args.offsets, args.E, args.M, BN);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const unsigned units = static_cast<unsigned>(args.row_tiles) *
                         static_cast<unsigned>(tab->tile[args.E]) * args.k_splits;

  if (warp == 0) {
    // ------------------------------------------------------------------ X producer
    pdl_wait();
    pdl_launch_dependents();
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (unsigned u = blockIdx.x; u < units && ok; u += gridDim.x) {
        const TfUnit t = tf_unit<BN>(u, args, tab, G);
        for (int i = 0; i < t.groups; ++i) {
          ok = mbar_wait(&xempty[s], ph ^ 1);
          if (!ok) break;
          mbar_arrive_expect_tx(&xfull[s], L::kXBytes);
#pragma unroll
          for (int h = 0; h < 2; ++h)
            tma_load_2d(smem + s * L::kXBytes + h * L::kXHalf, &tmap_x, &xfull[s],
                        (2 * (t.g0 + i) + h) * kTcBK, t.m0);
          if (++s == NX) { s = 0; ph ^= 1; }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    // The whole warp walks the loop, so that what the instructions take (descriptors, TMEM
    // addresses) is the same in every lane and lives in uniform registers; one elected lane
    // issues. (A loop that only lane 0 ran issued one MMA in about 80 cycles, whatever its N.)
    const bool leader = elect_one();
    const uint64_t xd0 = sw128_kmajor_desc(smem_u32(smem));
    int s = 0, as = 0, buf = 0;
    uint32_t ph = 0, aph = 0, dph = 0;
    bool ok = true;
    for (unsigned u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const TfUnit t = tf_unit<BN>(u, args, tab, G);
      // a tile multiplies only the tokens it has (N goes in steps of 16): the rest of its BN rows
      // of X belong to another expert or lie past the end
      const uint32_t idesc = f16_idesc(kTcBM, (t.cols + 15) / 16 * 16);
      const uint32_t d = tmem + L::kAccCol + buf * BN;
      ok = __all_sync(0xffffffffu, mbar_wait(&dempty[buf], dph ^ 1));   // the epilogue has read it
      for (int i = 0; i < t.groups && ok; ++i) {
        ok = mbar_wait(&xfull[s], ph) && mbar_wait(&afull[as], aph) &&
             (L::kHB == 2 || mbar_wait(&afull[as + 1], aph));   // (kHB = 1: as is even)
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint64_t xd = xd0 + static_cast<uint64_t>(s * (L::kXBytes >> 4));
        const uint32_t a = tmem + L::kACol + as * L::kACols;
        uint64_t* xe = &xempty[s];
        uint64_t* ae = &aempty[as];
        if (++s == NX) { s = 0; ph ^= 1; }
        as += 2 / L::kHB;
        if (as == NA) { as = 0; aph ^= 1; }
        if (leader) {
#pragma unroll
          for (int k = 0; k < 4; ++k)   // 16 k each: 8 columns of A, 32 bytes of X
            tc_mma_f16_ta(d, a + 8 * k, xd + 2 * k, idesc, (i | k) != 0 ? 1u : 0u);
          if (L::kHB == 1) tc_commit(ae);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma_f16_ta(d, a + 32 + 8 * k, xd + (L::kXHalf >> 4) + 2 * k, idesc, 1u);
          tc_commit(L::kHB == 1 ? ae + 1 : ae);
          tc_commit(xe);
          if (i == t.groups - 1) tc_commit(&dfull[buf]);
        }
        __syncwarp();
      }
      if (++buf == 2) { buf = 0; dph ^= 1; }
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------------ packed producer
    int ps = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (unsigned u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const TfUnit t = tf_unit<BN>(u, args, tab, G);
      for (int i = 0; i < t.groups; i += kPG) {   // a slot holds kPG groups of a unit
        ok = __all_sync(0xffffffffu, mbar_wait(&pempty[ps], ph ^ 1));
        if (!ok) break;
        const int g = t.g0 + i;
        if (lane == 0) {
          // groups past K are zero codes that nothing uses; a box is always counted whole
          const int32_t arow = static_cast<int32_t>(t.e * args.N) + t.row0;
          mbar_arrive_expect_tx(&pfull[ps], L::kBoxes * L::kBoxBytes);
#pragma unroll
          for (int b = 0; b < L::kBoxes; ++b)
            tma_load_2d(smem + L::kPOff + ps * L::kPBytes + b * L::kBoxBytes, &tmap_w, &pfull[ps],
                        kBits == 4 ? (g + 2 * b) * 16 : g * 12, arow);
        }
        // scales (256 bytes a group) and zero points (128) of the slot towards L2
        const int pg = g + lane / 4;
        if (lane / 4 < kPG && pg < G) {
          const int64_t n = t.row0 + (lane % 4 == 1 ? 64 : 0);
          const int64_t x = (static_cast<int64_t>(t.e) * G + pg) * args.N + n;
          if (n < args.N && lane % 4 < 3)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(
                lane % 4 < 2 ? static_cast<const void*>(args.scales + x)
                             : static_cast<const void*>(args.zeros + x)));
        }
        if (++ps == P) { ps = 0; ph ^= 1; }
      }
    }
  } else if (kInv && warp == 3) {
    // ------------------------------------------------------------------ inv_s producer
    // The factors are no part of the packed weight: the preceding kernel may have written them, so
    // they wait for it where the codes need not.
    pdl_wait();
    if (lane == 0) {
      int ps = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (unsigned u = blockIdx.x; u < units && ok; u += gridDim.x) {
        const TfUnit t = tf_unit<BN>(u, args, tab, G);
        for (int i = 0; i < t.groups; i += kPG) {   // the slots of the packed producer
          ok = mbar_wait(&pempty[ps], ph ^ 1);
          if (!ok) break;
          const int g = t.g0 + i;
          const uint32_t bytes = static_cast<uint32_t>((G - g < kPG ? G - g : kPG) * kGroup * 4);
          mbar_arrive_expect_tx(&pfull[ps], bytes);
          if (AWQ_IN_BOUNDS(g < G && t.e < args.E))
            bulk_load_1d(smem + L::kIOff + ps * L::kInvBytes,
                         args.inv_s + (static_cast<int64_t>(t.e) * G + g) * kGroup, bytes, &pfull[ps]);
          if (++ps == P) { ps = 0; ph ^= 1; }
        }
      }
    }
  } else if (warp >= kTfBuildWarp0 && warp < kTfEpiWarp0) {
    // ------------------------------------------------------------------ builders
    const int set = (warp - kTfBuildWarp0) >> 2;
    const int row = 32 * (warp & 3) + lane;
    const uint32_t ta = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + L::kACol;
    constexpr int kPerG = 2 / L::kHB;   // K blocks of a group
    const uint32_t N32 = static_cast<uint32_t>(args.N);
    // Scale and zero point of this thread's row (rows past N read the last one): index of those
    // of K block i of a unit; the set's next block of the unit is a fixed step on.
    const uint32_t sz_step = (kTfSets / kPerG) * N32;
    auto sz_index = [&](const TfUnit& t, int i) {
      const uint32_t n = static_cast<uint32_t>(t.row0 + row);
      return static_cast<uint32_t>(t.e * G + t.g0 + i / kPerG) * N32 + (n < N32 ? n : N32 - 1);
    };
    uint32_t sz = 0;
    auto load_sz = [&](unsigned short& s, unsigned char& z) {
      s = reinterpret_cast<const unsigned short*>(args.scales)[sz];
      z = args.zeros[sz];
    };
    unsigned short s_cur = 0, s_far = 0;   // of the block at hand; of the set's next block
    unsigned char z_cur = 0, z_far = 0;
    unsigned u = blockIdx.x;
    TfUnit t{}, tn{};       // the unit at hand and the CTA's next one
    if (u < units) t = tf_unit<BN>(u, args, tab, G);
    int i = set;            // K block (A stage) of the unit
    int slot_i = 0;         // the ring's current slot is the unit's slot_i-th
    int ps = 0, as = set % NA;
    uint32_t ph = 0, aph = (set / NA) & 1;
    bool seen = false;      // the current slot's filling has been awaited
    // moves on to slot `to` of the unit: this warp is done with every slot before it (a slot none
    // of whose groups the set has is awaited too, so that each arrival belongs to its filling)
    auto release_to = [&](int to) {
      bool ok = true;
      for (; slot_i < to && ok; ++slot_i) {
        if (!seen) ok = __all_sync(0xffffffffu, mbar_wait(&pfull[ps], ph));
        if (ok && lane == 0) mbar_arrive(&pempty[ps]);
        if (++ps == P) { ps = 0; ph ^= 1; }
        seen = false;
      }
      return ok;
    };
    bool ok = true;
    // the first unit may have fewer blocks than the set's number
    while (u < units && i >= kPerG * t.groups && ok) {
      ok = release_to((t.groups + kPG - 1) / kPG);
      slot_i = 0;
      i -= kPerG * t.groups;
      u += gridDim.x;
      if (u < units) t = tf_unit<BN>(u, args, tab, G);
    }
    if (u < units) {
      sz = sz_index(t, i);
      load_sz(s_far, z_far);
    }
    while (u < units && ok) {
      // the set's next block: in this unit, or in the first later one that has it
      unsigned un = u;
      int in = i + kTfSets;
      const bool same = in < kPerG * t.groups;
      s_cur = s_far;
      z_cur = z_far;
      if (same) {
        sz += sz_step;
        load_sz(s_far, z_far);
      } else {
        tn = t;
        while (un < units && in >= kPerG * tn.groups) {
          in -= kPerG * tn.groups;
          un += gridDim.x;
          if (un < units) tn = tf_unit<BN>(un, args, tab, G);
        }
        if (un < units) {
          sz = sz_index(tn, in);
          load_sz(s_far, z_far);
        }
      }
      {
        const int gi = i / kPerG % kPG, h = i % kPerG;   // group of the slot, half of the group
        ok = release_to(i / kPerG / kPG) &&
             __all_sync(0xffffffffu, mbar_wait_all(&pfull[ps], ph, &aempty[as], aph ^ 1));
        if (!ok) break;
        seen = true;
        tc_fence_after();
        const uint8_t* box = smem + L::kPOff + ps * L::kPBytes;
        const float* inv = reinterpret_cast<const float*>(smem + L::kIOff + ps * L::kInvBytes) +
                           gi * kGroup + h * kTcBK;   // read with kInv
        const float scf = __half2float(__ushort_as_half(s_cur));
        const uint32_t sc = static_cast<uint32_t>(s_cur) * 0x00010001u;
#pragma unroll
        for (int hh = 0; hh < L::kHB; ++hh) {   // 64 k: 32 columns
          uint32_t wd[2 * kBits];
          const int hg = L::kHB == 2 ? hh : h;   // half of the group
          if constexpr (kBits == 4) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const uint4 p = *reinterpret_cast<const uint4*>(
                  box + (gi >> 1) * L::kBoxBytes + row * 128 +
                  ((((gi & 1) * 4 + 2 * hg + q) ^ (row & 7)) << 4));
              wd[4 * q] = p.x;
              wd[4 * q + 1] = p.y;
              wd[4 * q + 2] = p.z;
              wd[4 * q + 3] = p.w;
            }
          } else {
#pragma unroll
            for (int q = 0; q < 3; ++q) {
              const uint2 p = *reinterpret_cast<const uint2*>(box + row * L::kRowBytes + gi * 48 +
                                                              hg * 24 + q * 8);
              wd[2 * q] = p.x;
              wd[2 * q + 1] = p.y;
            }
          }
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t o[16];
            dequant32<kBits, kInv>(wd + q * kBits, z_cur, sc, scf, inv + 64 * hh + 32 * q, o);
            tmem_st_32x32b_x16(ta + as * L::kACols + hh * 32 + q * 16, o);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&afull[as]);
        if (same) ok = release_to(in / kPerG / kPG);   // the codes and factors have been read
        as += kTfSets;
        if (as >= NA) { as -= NA; aph ^= 1; }
      }
      if (!same) {   // the rest of this unit's slots, and those of units without a group of the set
        while (u != un && ok) {
          ok = release_to((t.groups + kPG - 1) / kPG);
          slot_i = 0;
          u += gridDim.x;
          if (u < units) t = u == un ? tn : tf_unit<BN>(u, args, tab, G);
          else break;
        }
        if (un >= units) break;
      }
      i = in;
    }
  } else if (warp >= kTfEpiWarp0) {
    // ------------------------------------------------------------------ epilogue
    pdl_wait();
    const int half = (warp - kTfEpiWarp0) >> 2;
    const int row = 32 * (warp & 3) + lane;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    int buf = 0;
    uint32_t ph = 0;
    for (unsigned u = blockIdx.x; u < units; u += gridDim.x) {
      const TfUnit t = tf_unit<BN>(u, args, tab, G);
      const int64_t n = t.row0 + row;
      const bool live = n < args.N && AWQ_IN_BOUNDS(t.m0 + t.cols <= args.M && t.e < args.E);
      const float bias = live ? fused_bias<kBf16>(args.epi, t.e * args.N + n) : 0.0f;
      const uint32_t td = tmem + lanes + L::kAccCol + buf * BN;
      if (!__all_sync(0xffffffffu, mbar_wait_lazy(&dfull[buf], ph))) break;
      tc_fence_after();
      if (args.k_splits > 1) {
        partial_tile<kBf16>(args, t, n, live, half, lane, td);
      } else {
        switch (args.epi.act) {
          case kActRelu: fused_tile<kBf16, kActRelu>(args, t, n, live, bias, half, lane, td); break;
          case kActSilu: fused_tile<kBf16, kActSilu>(args, t, n, live, bias, half, lane, td); break;
          case kActGelu: fused_tile<kBf16, kActGelu>(args, t, n, live, bias, half, lane, td); break;
          case kActGeluTanh:
            fused_tile<kBf16, kActGeluTanh>(args, t, n, live, bias, half, lane, td);
            break;
          default: fused_tile<kBf16, kActNone>(args, t, n, live, bias, half, lane, td);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&dempty[buf]);
      if (++buf == 2) { buf = 0; ph ^= 1; }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The epilogue on the sum over the K slices of the fp32 partial sums, slices added in order. One
// CTA per 256 outputs of a row of Y; the first loads of the epilogue's operands are in flight
// with those of the partial sums.
template <bool kBf16>
__global__ void __launch_bounds__(256) splitk_fused_kernel(const FusedArgs args) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (n >= args.N) return;
  const int64_t i = static_cast<int64_t>(blockIdx.y) * args.N + n, MN = args.M * args.N;
  FusedIn<kBf16> in;
  in.load(args.epi, n, blockIdx.y, args.N, static_cast<int>(args.M));
  float acc = args.partial[i];
  for (int s = 1; s < args.k_splits; ++s) acc += args.partial[s * MN + i];
  static_cast<act_t<kBf16>*>(args.Y)[i] = float_to_act<kBf16>(in.apply(args.epi, acc, 0));
}

}  // namespace awq
