// Activations made ready for the products with a fused epilogue.
#pragma once
#include "common.cuh"

namespace awq {

// Prepared activations: x' = x inv_s[k] 2^p as fp16, one rounding, p such that the row's largest
// |x inv_s| lies in [2^14, 2^15) (a value 2^-29 of that and more keeps all of its bits; a row with
// an infinity or a NaN is taken as it is, p = 0), and the row's factor 2^-p. Every finite fp32
// row has such a p, so nothing overflows; from 2^-113 of the largest down p stays at 126, where both
// powers are normal numbers and a bf16 value of any size is an fp16 one. (x inv_s of a bf16 row is
// rounded to 11 bits here; its output to 8, beside which that does not show, so it takes no
// second part.) One CTA per row.
//  * kFragments, for the streaming kernel (gemv_fused.cuh): chunks of chunk_groups groups, each
//    group [8-k chunk j][32-k quarter c] of 8 values as the MMA fragments are read, then the
//    groups' sums of x' times 2^-24 (the codes come in as q 2^-24; the kernel takes that off, since
//    a factor times 2^24 could leave fp32's range). With split = 1 a row is two: x' rounded, then
//    the rounding's remainder, rounded.
//  * else plain rows [T, K], for the tensor-core kernel (gemm_fused.cuh).
// The factors [T] follow the rows.
constexpr int kPrepThreads = 256;
constexpr int kPrepKeep = 4;   // 8-value chunks of a thread kept between the two passes

template <bool kBf16>
__device__ __forceinline__ void prep_load(float (&f)[8], const uint4* X, const float* inv_s, int64_t i) {
  const uint4 v = X[i];
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 p = act2_to_float2<kBf16>(w[e]);
    f[2 * e] = p.x;
    f[2 * e + 1] = p.y;
  }
  if (inv_s != nullptr) {
    const float4 s0 = reinterpret_cast<const float4*>(inv_s)[2 * i];
    const float4 s1 = reinterpret_cast<const float4*>(inv_s)[2 * i + 1];
    const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= s[e];
  }
}

template <bool kBf16, bool kFragments>
__global__ void __launch_bounds__(kPrepThreads) prepare_rows_kernel(
    const uint4* __restrict__ X, int T, int64_t K, const float* __restrict__ inv_s,
    const int* __restrict__ offsets, int E, int chunk_groups, int chunk_bytes, int split,
    uint8_t* __restrict__ out) {
  pdl_wait();
  pdl_launch_dependents();
  const int row = blockIdx.x;
  const int tid = threadIdx.x;
  if (inv_s != nullptr && offsets != nullptr) {
    // the row's expert: how many of them end at or before it (every thread counts a few)
    int e = 0;
    for (int base = 0; base < E; base += kPrepThreads) {
      const int i = base + tid;
      e += __syncthreads_count(i < E && offsets[i + 1] <= row);
    }
    if (e >= E) return;   // a row of no expert
    inv_s += static_cast<int64_t>(e) * K;
  }
  const int nch = static_cast<int>(K / 8);
  const int chunks = (nch / 16 + chunk_groups - 1) / chunk_groups;
  X += static_cast<int64_t>(row) * nch;
  float big = 0.0f;
  bool finite = true;
  const auto look = [&](const float (&f)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      big = fmaxf(big, fabsf(f[e]));
      finite = finite && fabsf(f[e]) <= 3.4028235e38f;
    }
  };
  float keep[kPrepKeep][8];   // the row's first 8192 values stay in registers
#pragma unroll
  for (int j = 0; j < kPrepKeep; ++j) {
    const int i = tid + j * kPrepThreads;
    if (i < nch) {
      prep_load<kBf16>(keep[j], X, inv_s, i);
      look(keep[j]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) keep[j][e] = 0.0f;
    }
  }
  for (int i = tid + kPrepKeep * kPrepThreads; i < nch; i += kPrepThreads) {
    float f[8];
    prep_load<kBf16>(f, X, inv_s, i);
    look(f);
  }
  __shared__ float part[kPrepThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
  if ((tid & 31) == 0) part[tid >> 5] = big;
  finite = __syncthreads_and(finite);
#pragma unroll
  for (int w = 0; w < kPrepThreads / 32; ++w) big = fmaxf(big, part[w]);
  // 2^14 <= big 2^p < 2^15, from big's exponent: p >= -113, and up to 126 both powers are normal
  int p = finite && big > 0.0f ? 14 - (static_cast<int>(__float_as_uint(big) >> 23) - 127) : 0;
  p = p > 126 ? 126 : p;
  const float up = __uint_as_float(static_cast<uint32_t>(127 + p) << 23);
  const int64_t row_bytes = static_cast<int64_t>(chunks) * chunk_bytes;
  uint8_t* base = out + (static_cast<int64_t>(row) << split) * row_bytes;
  const auto store = [&](int i, float (&f)[8]) {   // a whole warp: groups are 16 lanes each
    const bool live = i < nch;
    const int g = i >> 4, ch = i & 15;   // 8-k chunk ch of the group: quarter ch / 4, j = ch % 4
    const int gl = g % chunk_groups;
    uint8_t* c = base + static_cast<int64_t>(g / chunk_groups) * chunk_bytes;
    for (int part = 0; part <= split; ++part) {   // the rounded value, then what it left
      uint32_t v[4];
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x0 = part == 0 ? f[2 * e] * up : f[2 * e];
        const float x1 = part == 0 ? f[2 * e + 1] * up : f[2 * e + 1];
        v[e] = float2_to_act2<false>(x0, x1);
        const float2 h = act2_to_float2<false>(v[e]);
        sum += h.x + h.y;
        f[2 * e] = x0 - h.x;
        f[2 * e + 1] = x1 - h.y;
      }
      if (!kFragments) {
        if (live && AWQ_IN_BOUNDS(row < T))
          reinterpret_cast<uint4*>(out)[static_cast<int64_t>(row) * nch + i] =
              make_uint4(v[0], v[1], v[2], v[3]);
        break;
      }
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      uint8_t* cp = c + part * row_bytes;
      if (live && AWQ_IN_BOUNDS(row < T)) {
        *reinterpret_cast<uint4*>(cp + gl * 256 + (ch & 3) * 64 + (ch >> 2) * 16) =
            make_uint4(v[0], v[2], v[1], v[3]);   // the pairs of the two MMAs
        if (ch == 0)
          *reinterpret_cast<float*>(cp + chunk_groups * 256 + gl * 4) = sum * 5.9604644775390625e-8f;
      }
    }
  };
  const int padded = (nch + 31) / 32 * 32;
#pragma unroll
  for (int j = 0; j < kPrepKeep; ++j)
    if (tid + j * kPrepThreads < padded) store(tid + j * kPrepThreads, keep[j]);
  for (int i = tid + kPrepKeep * kPrepThreads; i < padded; i += kPrepThreads) {
    float f[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (i < nch) prep_load<kBf16>(f, X, inv_s, i);
    store(i, f);
  }
  if (tid == 0) {
    const int64_t rows_bytes =
        kFragments ? (static_cast<int64_t>(T) << split) * row_bytes : static_cast<int64_t>(T) * K * 2;
    reinterpret_cast<float*>(out + rows_bytes)[row] =
        __uint_as_float(static_cast<uint32_t>(127 - p) << 23);
  }
}

}  // namespace awq
