// K1: per-input-channel activation magnitude s_x[k] = (1/M) sum_m |x[m, k]|.
//
// robotsatlas.com "AWQ", "How it works" and "Components: Activation saliency analysis":
// the calibration set is passed through the layer and the activation magnitude of every
// input channel is measured. The statistic is the mean absolute value over all tokens.
//
// HBM-bound column reduction. Pass 1: a CTA of 32 column lanes x 8 row lanes covers 256
// channels (one 16-byte load of 8 fp16 per lane and row) over a slice of the rows and
// accumulates |x| in fp64; the 8 row lanes are combined in a fixed order and the slice's
// partial sums go to the workspace. Pass 2 adds the slices in order and divides by M.
// fp64 accumulation of fp16 inputs is exact whenever the running sums span fewer than 53
// bits, so the result does not depend on the split.
#pragma once
#include "common.cuh"
#include "fused.cuh"

namespace awq {

constexpr int kStatsCols = 256;   // channels per CTA (32 lanes x 8 fp16)
constexpr int kStatsRowLanes = 8;

__global__ void __launch_bounds__(256) act_stats_partial_kernel(const __half* __restrict__ X,
                                                                int64_t M, int64_t K,
                                                                int64_t rows_per_split,
                                                                double* __restrict__ part) {
  const int lane = threadIdx.x & 31;
  const int rl = threadIdx.x >> 5;                       // row lane 0..7
  const int64_t col0 = static_cast<int64_t>(blockIdx.x) * kStatsCols + lane * 8;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * rows_per_split;
  const int64_t r1 = min(M, r0 + rows_per_split);
  double acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0;
  if (col0 < K) {
    const __half* p = X + col0;
    int64_t r = r0 + rl;
    // four independent 16-byte loads in flight per iteration
    for (; r + 3 * kStatsRowLanes < r1; r += 4 * kStatsRowLanes) {
      uint4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        v[u] = AWQ_IN_BOUNDS(r + u * kStatsRowLanes < M && col0 + 8 <= K)
                   ? ldg_nc_v4(p + (r + u * kStatsRowLanes) * K)
                   : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const __half2* h = reinterpret_cast<const __half2*>(&v[u]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float2 f = __half22float2(h[i]);
          acc[2 * i] += fabs(static_cast<double>(f.x));
          acc[2 * i + 1] += fabs(static_cast<double>(f.y));
        }
      }
    }
    for (; r < r1; r += kStatsRowLanes) {
      uint4 v = AWQ_IN_BOUNDS(r < M && col0 + 8 <= K) ? ldg_nc_v4(p + r * K)
                                                       : make_uint4(0u, 0u, 0u, 0u);
      const __half2* h = reinterpret_cast<const __half2*>(&v);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float2 f = __half22float2(h[i]);
        acc[2 * i] += fabs(static_cast<double>(f.x));
        acc[2 * i + 1] += fabs(static_cast<double>(f.y));
      }
    }
  }
  __shared__ double red[kStatsRowLanes][kStatsCols];
#pragma unroll
  for (int i = 0; i < 8; ++i) red[rl][lane * 8 + i] = acc[i];
  __syncthreads();
  // 256 threads: thread t finalises channel t of the tile, adding row lanes in order.
  const int t = threadIdx.x;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kStatsCols + t;
  if (c < K) {
    double s = 0.0;
#pragma unroll
    for (int j = 0; j < kStatsRowLanes; ++j) s += red[j][t];
    if (AWQ_IN_BOUNDS(blockIdx.y < gridDim.y)) part[static_cast<int64_t>(blockIdx.y) * K + c] = s;
  }
}

__global__ void act_stats_finish_kernel(const double* __restrict__ part, int splits, int64_t M,
                                        int64_t K, float* __restrict__ s_x) {
  const int64_t k = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (k >= K) return;
  double s = 0.0;
  for (int j = 0; j < splits; ++j) s += part[static_cast<int64_t>(j) * K + k];
  s_x[k] = __double2float_rn(s / static_cast<double>(M));
}

// Split count so that the grid covers the GPU several times over.
inline int act_stats_splits(int64_t M, int64_t K, int num_sms) {
  const int64_t col_tiles = (K + kStatsCols - 1) / kStatsCols;
  int64_t want = (static_cast<int64_t>(num_sms) * 8 + col_tiles - 1) / col_tiles;
  int64_t by_rows = (M + 63) / 64;                       // at least 64 rows per slice
  int64_t s = want < by_rows ? want : by_rows;
  if (s < 1) s = 1;
  if (s > 65535) s = 65535;
  return static_cast<int>(s);
}

// ---------------------------------------------------------------------------------------
// The statistic of each expert: s_x[e, k] = mean over e's rows of |x[row, k]|, rows sorted by
// expert, expert e's from offsets[e] to offsets[e + 1] (0 for an expert without rows).
//
// Rows are cut into slices of equal length wherever the experts begin, so the work is balanced
// whatever the routing, and no launch waits for the offsets on the host. A slice that holds
// rows of several experts sums each of them apart. The partial sums of slice y and expert e go
// to slot y + e of the workspace: along the rows either the slice or the expert moves on, so
// the slots of (slice, expert) pairs that share rows are all different, and there are at most
// slices + E of them.
//
// The sums are of doubles made from the fp16 bits by a shift: |x|'s exponent and mantissa at the
// top of a double with exponent field e stand for |x| 2^-1008, exactly, subnormals too (both
// formats are IEEE's), so a conversion instruction, a quarter as fast as the additions, is
// saved and the finish multiplies by 2^1008. Infinities and NaN do not survive the shift (their
// field is an ordinary exponent of a double); each channel's largest |x| remembers them.
//
// HBM-bound: 131072 rows of 4096 channels over 8 experts take 158 us replayed on the same rows,
// 6.8 TB/s, and 171 a call on rows that change, 6.3 (254 us with the conversions). The small calls are
// bound by their two launches and slices cut short at each expert (5000 x 2048 over 64 experts: 11.4 us
// on the device for 3.2 us of traffic).
constexpr int kStatsBatch = 4;   // rows of a lane in flight
inline int64_t grouped_stats_rows(int64_t T, int64_t K, int num_sms) {
  const int64_t splits = act_stats_splits(T, K, num_sms);
  return (T + splits - 1) / splits;
}
inline int64_t grouped_stats_slices(int64_t T, int64_t K, int num_sms) {
  const int64_t rows = grouped_stats_rows(T, K, num_sms);
  return (T + rows - 1) / rows;
}

// offsets[e] as a row of X: a value outside 0 .. T is taken as the nearest end.
__device__ __forceinline__ int64_t row_offset(const int* __restrict__ offsets, int e, int64_t T) {
  const int64_t v = offsets[e];
  return v < 0 ? 0 : v > T ? T : v;
}

__global__ void __launch_bounds__(256) act_stats_grouped_partial_kernel(
    const __half* __restrict__ X, int64_t T, int64_t K, const int* __restrict__ offsets, int E,
    int64_t rows, double* __restrict__ part) {
  const int lane = threadIdx.x & 31;
  const int rl = threadIdx.x >> 5;
  const int64_t col0 = static_cast<int64_t>(blockIdx.x) * kStatsCols + lane * 8;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kStatsCols + threadIdx.x;
  const int64_t y0 = static_cast<int64_t>(blockIdx.y) * rows;
  const int64_t y1 = min(T, y0 + rows);
  __shared__ double red[kStatsRowLanes][kStatsCols];
  __shared__ int off[kMaxExperts + 1];   // the offsets as rows of X, loaded at once
  pdl_wait();
  pdl_launch_dependents();
  for (int i = threadIdx.x; i <= E; i += 256) off[i] = static_cast<int>(row_offset(offsets, i, T));
  __syncthreads();
  // the first expert that ends behind the slice's first row: every one before it ends earlier
  int e = 0;
  for (int n = E; n > 0;) {
    const int half = n >> 1;
    if (off[e + half + 1] <= y0) {
      e += half + 1;
      n -= half + 1;
    } else {
      n = half;
    }
  }
  for (; e < E; ++e) {
    const int64_t a = off[e];
    if (a >= y1) break;
    const int64_t r0 = max(a, y0), r1 = min(static_cast<int64_t>(off[e + 1]), y1);
    if (r0 >= r1) continue;   // no rows of this expert
    double acc[8];
    __half2 big[4];   // the largest |x| of each channel so far; a NaN stays one
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) big[i] = __float2half2_rn(0.0f);
    const auto add = [&](const uint4& v) {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[2 * i] += __hiloint2double(static_cast<int>((w[i] << 10) & 0x01FFFC00u), 0);
        acc[2 * i + 1] += __hiloint2double(static_cast<int>((w[i] >> 6) & 0x01FFFC00u), 0);
        big[i] = __hmax2_nan(big[i], __habs2(u32_as_h2(w[i])));
      }
    };
    if (col0 < K) {
      const __half* p = X + col0;
      int64_t r = r0 + rl;
      for (; r + (kStatsBatch - 1) * kStatsRowLanes < r1; r += kStatsBatch * kStatsRowLanes) {
        uint4 v[kStatsBatch];   // independent loads in flight
#pragma unroll
        for (int u = 0; u < kStatsBatch; ++u)
          v[u] = AWQ_IN_BOUNDS(r + u * kStatsRowLanes < T && col0 + 8 <= K)
                     ? ldg_nc_v4(p + (r + u * kStatsRowLanes) * K) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int u = 0; u < kStatsBatch; ++u) add(v[u]);
      }
      for (; r < r1; r += kStatsRowLanes)
        add(AWQ_IN_BOUNDS(r < T && col0 + 8 <= K) ? ldg_nc_v4(p + r * K) : make_uint4(0u, 0u, 0u, 0u));
    }
    // an infinity's or NaN's bits were added as if of a number: the sum is what they make of it
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(big[i]);
      if (!(f.x <= 65504.0f)) acc[2 * i] = static_cast<double>(f.x);
      if (!(f.y <= 65504.0f)) acc[2 * i + 1] = static_cast<double>(f.y);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) red[rl][lane * 8 + i] = acc[i];
    __syncthreads();
    if (c < K) {
      double s = 0.0;
#pragma unroll
      for (int j = 0; j < kStatsRowLanes; ++j) s += red[j][threadIdx.x];
      if (AWQ_IN_BOUNDS(blockIdx.y + static_cast<int64_t>(e) < gridDim.y + static_cast<int64_t>(E)))
        part[(blockIdx.y + static_cast<int64_t>(e)) * K + c] = s;
    }
    __syncthreads();
  }
}

__global__ void act_stats_grouped_finish_kernel(const double* __restrict__ part, int64_t T,
                                                int64_t K, const int* __restrict__ offsets,
                                                int64_t rows, float* __restrict__ s_x) {
  const int64_t k = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int e = blockIdx.y;
  // (the offsets were there before the kernel that writes the partial sums could start)
  const int64_t a = row_offset(offsets, e, T), b = row_offset(offsets, e + 1, T);
  pdl_wait();
  pdl_launch_dependents();
  if (k >= K) return;
  double s = 0.0;
  if (a < b) {
#pragma unroll 8   // independent loads, added in order
    for (int64_t y = a / rows; y <= (b - 1) / rows; ++y) s += part[(y + e) * K + k];
    s = s * 0x1p1008 / static_cast<double>(b - a);   // see the scale of the sums above
  }
  s_x[e * K + k] = __double2float_rn(s);
}

}  // namespace awq
