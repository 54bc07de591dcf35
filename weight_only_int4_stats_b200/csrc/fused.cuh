// What the products with a fused epilogue and the expert kernels share: the epilogue itself,
//     Y[m, n] = act(P[m, n] + bias[n]) * mul[m, n] + residual[m, n],
// in fp32 with one rounding to Y's type, and the table of the experts' rows that each CTA makes
// from the offsets on the device.
#pragma once
#include "common.cuh"

namespace awq {

// Activations (the values of AWQ_ACT_*).
enum Act : int { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };

// The epilogue's parts in the activations' type; NULL where a part is absent.
struct FusedEpi {
  const void* bias;       // [E, N]
  const void* mul;        // [rows, N]
  const void* residual;   // [rows, N]
  int act;                // Act
};

// act(v) in fp32. A NaN stays one (with relu too); silu and gelu as their formulas give it, the
// tanh form by (1 + tanh u) / 2 = 1 / (1 + exp(-2u)). The fast division is within 2 fp32 roundings, the
// fast exponential of x within 2 + |1.17 x|: at most 106 of them, 2^-17 of the value, before the
// exponential overflows at 88.7, and there v / inf is the limit 0 (from 2^126 on the fast division
// gives it too: silu's -1e-36 of v < -87.3).
__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case kActRelu: return v < 0.0f ? 0.0f : v;
    case kActSilu: return __fdividef(v, 1.0f + __expf(-v));
    case kActGelu: return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
    case kActGeluTanh:   // 2 u = 2 sqrt(2 / pi) (v + 0.044715 v^3)
      return __fdividef(v, 1.0f + __expf(-1.5957691216057308f * fmaf(0.044715f * v * v, v, v)));
    default: return v;
  }
}

template <bool kBf16>
__device__ __forceinline__ float act_to_float(act_t<kBf16> v) {
  if constexpr (kBf16) return __bfloat162float(v);
  else return __half2float(v);
}
template <bool kBf16>
__device__ __forceinline__ float fused_bias(const FusedEpi& f, int64_t i) {
  return f.bias == nullptr ? 0.0f
                           : act_to_float<kBf16>(static_cast<const act_t<kBf16>*>(f.bias)[i]);
}
// The epilogue of the four outputs a lane has of an m16n8 accumulator tile: weight rows n, n + 8
// (value i / 2) of tokens m, m + 1 (value i % 2). load() only loads: nothing waits for the values
// until apply() uses them. mul and residual are read by the thread that writes the output, before
// it does, so either may be Y itself.
template <bool kBf16>
struct FusedIn {
  using A = act_t<kBf16>;
  A bias[2], mul[4], res[4];
  __device__ __forceinline__ void load(const FusedEpi& f, int64_t n, int m, int64_t N, int M) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool live = n + 8 * (i >> 1) < N && m + (i & 1) < M;
      const int64_t y = (m + (i & 1)) * N + n + 8 * (i >> 1);
      if ((i & 1) == 0)
        bias[i >> 1] = live && f.bias != nullptr
                           ? static_cast<const A*>(f.bias)[n + 8 * (i >> 1)] : A(0.0f);
      mul[i] = live && f.mul != nullptr ? static_cast<const A*>(f.mul)[y] : A(1.0f);
      res[i] = live && f.residual != nullptr ? static_cast<const A*>(f.residual)[y] : A(0.0f);
    }
  }
  __device__ __forceinline__ float apply(const FusedEpi& f, float v, int i) const {
    return fmaf(activate(v + act_to_float<kBf16>(bias[i >> 1]), f.act), act_to_float<kBf16>(mul[i]),
                act_to_float<kBf16>(res[i]));
  }
};

// Rows grouped by expert: expert e's rows are offsets[e] .. offsets[e + 1] - 1 of X and Y. The
// offsets live on the device (a router wrote them), so each CTA makes its own table of them.
constexpr int kMaxExperts = 1024;
struct GroupTable {
  int off[kMaxExperts + 1];    // first row of each expert, then the end of the last
  int tile[kMaxExperts + 1];   // token tiles before each expert, then their total
};

// Fills off[0 .. E] and tile[0 .. E] for token tiles of bn rows: the whole CTA calls it, and
// synchronises before it reads them. An offset outside 0 .. rows, or below one before it, is taken
// as the nearest value in order, so no row outside X and Y is ever touched. offsets NULL: one
// expert with all rows. (All offsets are loaded at once and then summed up from shared memory: a
// warp that loads as it goes waits 600 cycles for every 32 experts.)
__device__ __forceinline__ void build_group_table(int* off, int* tile, const int* offsets, int E,
                                                  int64_t rows, int bn) {
  const int M = static_cast<int>(rows);
  if (offsets == nullptr) {
    if (threadIdx.x == 0) {
      off[0] = 0;
      off[1] = M;
      tile[0] = 0;
      tile[1] = (M + bn - 1) / bn;
    }
    return;
  }
  for (int e = static_cast<int>(threadIdx.x); e <= E; e += static_cast<int>(blockDim.x)) {
    const int v = offsets[e];
    off[e] = v < 0 ? 0 : v > M ? M : v;
  }
  __syncthreads();
  if (threadIdx.x >= 32) return;
  const int lane = threadIdx.x;
  int high = 0, tiles = 0;   // the last offset so far, the tiles before it
  for (int base = 0; base <= E; base += 32) {
    const int e = base + lane;
    int v = e <= E ? off[e] : M;
    int before = __shfl_up_sync(0xffffffffu, v, 1);
    if (lane == 0) before = high;
    if (__any_sync(0xffffffffu, v < before)) {   // out of order: the running maximum
      if (lane == 0 && v < high) v = high;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int w = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o && w > v) v = w;
      }
      before = __shfl_up_sync(0xffffffffu, v, 1);
      if (lane == 0) before = high;
      if (e <= E) off[e] = v;
    }
    // the tiles of expert e - 1 end where expert e's begin
    int sum = e == 0 || e > E ? 0 : (v - before + bn - 1) / bn;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int w = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += w;
    }
    if (e <= E) tile[e] = tiles + sum;
    high = __shfl_sync(0xffffffffu, v, 31);
    tiles += __shfl_sync(0xffffffffu, sum, 31);
  }
}

}  // namespace awq
