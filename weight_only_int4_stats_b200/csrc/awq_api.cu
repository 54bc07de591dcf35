// Host side of the C ABI declared in include/awq.h: argument checks, workspace carving,
// TMA descriptor encoding and kernel dispatch. All kernels live in the *.cuh files of this
// directory and are compiled into this one translation unit for sm_100a.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <mutex>

#include "awq.h"
#include "act_stats.cuh"
#include "common.cuh"
#include "gated_grouped.cuh"
#include "gemm_tc.cuh"
#include "gemv.cuh"
#include "gemm_fused.cuh"
#include "gemv_fused.cuh"
#include "quantize.cuh"
#include "search.cuh"

namespace {

using awq::ASrc;
using awq::Epi;

constexpr int64_t kMaxDim = (int64_t{1} << 31) - 1;
constexpr int kMaxDevices = 64;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
size_t align256(size_t v) { return (v + 255) & ~size_t{255}; }

awq_status launch_status() {
  cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? AWQ_OK : AWQ_ERR_CUDA;
}

// Per-device caches below are atomics: host threads may call the library concurrently, and
// a value computed twice is the same value, so a racing first call only repeats work.
int num_sms() {
  static std::atomic<int> cache[kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 148;
  int v = cache[dev].load(std::memory_order_acquire);
  if (v == 0) {
    if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0)
      v = 148;
    cache[dev].store(v, std::memory_order_release);
  }
  return v;
}

// cuTensorMapEncodeTiled through the runtime's driver entry point (no link-time libcuda).
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// 2-D row-major tensor [rows, cols] of `elem` bytes per element; box [box_rows, box_cols].
bool make_tmap_2d(CUtensorMap* map, const void* base, CUtensorMapDataType dt, int elem,
                  int64_t rows, int64_t cols, int box_rows, int box_cols, bool swizzle128) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * elem};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(map, dt, 2, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE,
                  swizzle128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

template <int BN, ASrc kA, Epi kEpi, bool kBf16, int kBlkT>
awq_status launch_tc_blk(const void* Xop, int64_t M, const void* Aop, int64_t a_rows,
                         const awq::TcArgs& args, cudaStream_t st, const void* Aop2) {
  using L = awq::TcLayout<BN, kA, kBlkT>;
  static std::atomic<bool> attr_set[kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return AWQ_ERR_CUDA;
  auto kern = awq::tc_gemm_kernel<BN, kA, kEpi, kBf16, kBlkT>;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem) !=
        cudaSuccess)
      return AWQ_ERR_CUDA;
    attr_set[dev].store(true, std::memory_order_release);
  }
  CUtensorMap tx, ta;
  // B operand rows M x (K, or 2K for the two-part normalised Gram matrix) columns
  if (!make_tmap_2d(&tx, Xop, kBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                    : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                    2, M, kA == ASrc::kGram ? 2 * args.K : args.K, BN, awq::kTcBK, true))
    return AWQ_ERR_CUDA;
  if (kA == ASrc::kSplit16 || kA == ASrc::kGram) {   // [a_rows, 2K]: hi part, then lo part
    if (!make_tmap_2d(&ta, Aop, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, a_rows, 2 * args.K,
                      awq::kTcBM, awq::kTcBK, true))
      return AWQ_ERR_CUDA;
  } else if (kA == ASrc::kPair16 || kA == ASrc::kFp16x1) {   // [a_rows, K] fp16 (kPair16:
                                                                  // the second map goes in ts)
    if (!make_tmap_2d(&ta, Aop, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, a_rows, args.K, awq::kTcBM,
                      awq::kTcBK, true))
      return AWQ_ERR_CUDA;
  } else if (kA == ASrc::kPacked4) {   // kPG groups of 16 words (64 bytes) per row per load
    if (!make_tmap_2d(&ta, Aop, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, a_rows, args.K / 8,
                      awq::kTcBM, L::kPRowBytes / 4, false))
      return AWQ_ERR_CUDA;
  } else {   // 3-bit: kPG groups of 12 words (48 bytes) per row per load
    if (!make_tmap_2d(&ta, Aop, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, a_rows, 3 * args.K / 32,
                      awq::kTcBM, L::kPRowBytes / 4, false))
      return AWQ_ERR_CUDA;
  }
  // scales [G, N] fp16 and zeros [G, N] u8 as TMA tiles of kPG groups x 128 rows, when the
  // row stride of the zeros (N bytes) meets the 16-byte rule; otherwise the maps go unused
  CUtensorMap ts = ta, tz = ta;
  awq::TcArgs a = args;
  a.sz_tma = 0;
  if (kA == ASrc::kPair16 &&
      !make_tmap_2d(&ts, Aop2, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, a_rows, args.K, awq::kTcBM,
                    awq::kTcBK, true))
    return AWQ_ERR_CUDA;
  if ((kA == ASrc::kPacked4 || kA == ASrc::kPacked3) && args.N % 16 == 0) {
    const int64_t G = args.K / awq::kGroup;
    if (!make_tmap_2d(&ts, args.scales, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, G, args.N, L::kPG,
                      awq::kTcBM, false) ||
        !make_tmap_2d(&tz, args.zeros, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, G, args.N, L::kPG,
                      awq::kTcBM, false))
      return AWQ_ERR_CUDA;
    a.sz_tma = 1;
  }
  a.m_tiles = static_cast<int>((M + BN - 1) / BN);
  a.row_tiles = static_cast<int>((a_rows + awq::kTcBM - 1) / awq::kTcBM);
  a.rows_total = a_rows;
  if (a.k_splits < 1) a.k_splits = 1;
  const int64_t units = static_cast<int64_t>(a.m_tiles) * a.row_tiles * a.k_splits;
  const int64_t sms = num_sms();
  // persistent, one CTA per SM; the fp32-store epilogue instead takes one CTA per output tile,
  // so that a tile's contraction slices are consecutive units of the same CTA
  const int64_t want = kEpi == Epi::kStoreF32 ? units / a.k_splits : sms;
  const unsigned grid = static_cast<unsigned>(units < want ? units : want);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(awq::kTcThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(L::kSmem);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, tx, ta, ts, tz, a) != cudaSuccess) return AWQ_ERR_CUDA;
  return launch_status();
}

// Packed sources take stages of two 64-k blocks where the builders or the single MMA-issuing
// thread set the pace: token tiles up to 128, and inv_s folded into the weights. Plain
// BN = 256 keeps four one-block stages (two two-block stages, all that fit, measured slower
// there: 1294 -> 1172 TFLOP/s on [28672, 8192] at M = 4096).
template <int BN, ASrc kA, Epi kEpi, bool kBf16 = false>
awq_status launch_tc(const void* Xop, int64_t M, const void* Aop, int64_t a_rows,
                     const awq::TcArgs& args, cudaStream_t st, const void* Aop2 = nullptr) {
  constexpr bool kPk = kA == ASrc::kPacked4 || kA == ASrc::kPacked3;
  if constexpr (kPk && BN == 256) {
    if (args.inv_s == nullptr)
      return launch_tc_blk<BN, kA, kEpi, kBf16, 1>(Xop, M, Aop, a_rows, args, st, Aop2);
    return launch_tc_blk<BN, kA, kEpi, kBf16, 2>(Xop, M, Aop, a_rows, args, st, Aop2);
  } else {
    return launch_tc_blk<BN, kA, kEpi, kBf16, kPk ? 2 : 1>(Xop, M, Aop, a_rows, args, st, Aop2);
  }
}

template <ASrc kA, Epi kEpi, bool kBf16 = false>
awq_status launch_tc_bn(const void* Xop, int64_t M, const void* Aop, int64_t a_rows,
                        const awq::TcArgs& args, cudaStream_t st, const void* Aop2 = nullptr) {
  if (M <= 32) return launch_tc<32, kA, kEpi, kBf16>(Xop, M, Aop, a_rows, args, st, Aop2);
  if (M <= 64) return launch_tc<64, kA, kEpi, kBf16>(Xop, M, Aop, a_rows, args, st, Aop2);
  if (M <= 128) return launch_tc<128, kA, kEpi, kBf16>(Xop, M, Aop, a_rows, args, st, Aop2);
  return launch_tc<256, kA, kEpi, kBf16>(Xop, M, Aop, a_rows, args, st, Aop2);
}

// Streaming decode GEMM (M <= 16), launched with programmatic dependent launch.
constexpr int kSmemLimit = 232448;   // 227 KB per CTA on sm_100
static_assert(awq::kGemvWeightsReady == AWQ_GEMM_WEIGHTS_READY, "flag values must agree");
static_assert((AWQ_GEMM_WEIGHTS_READY & AWQ_GEMM_BF16) == 0, "flags are distinct bits");

// Two CTAs of the streaming kernel fit on one SM when each takes at most half of its 228 KB
// (less 1 KB reserved per CTA): the next launch's CTAs then start beside this one's.
constexpr int kCoResidentSmem = (233472 - 2 * 1024) / 2;

// The streaming kernel's shared-memory plan for a shape: the deepest ring (6 down to 2 slots)
// that leaves room for a co-resident CTA, else the deepest that fits one CTA.
bool gemv_config(int64_t M, int64_t N, int64_t K, awq::G4Smem* out) {
  if (M < 1 || M > 16 || N % 16 != 0 || K / awq::kGroup > 65535) return false;
  const int nt = M <= 8 ? 1 : 2;
  for (int budget : {kCoResidentSmem, kSmemLimit})
    for (int slots = awq::kGSMaxSlots; slots >= 2; --slots) {
      const awq::G4Smem l = awq::G4Smem::make(static_cast<int>(M), K, nt, slots);
      if (l.total(nt) <= budget) {
        *out = l;
        return true;
      }
    }
  return false;
}

// Whether the streaming decode kernel takes this shape: N in whole 16-row tiles and X (plus the
// small sums, the reduction buffer and a two-slot ring) within one CTA's shared memory.
bool gemv_stream_fits(int64_t M, int64_t N, int64_t K) {
  awq::G4Smem l;
  return gemv_config(M, N, K, &l);
}

template <int kNTiles, bool kOffset, bool kBf16, int kBits, bool kFused>
awq_status launch_gemv_stream_t(const void* x, int64_t M, const uint32_t* qweight,
                                const __half* scales, const uint8_t* zeros, int64_t N, int64_t K,
                                const float* inv_s, unsigned flags, void* y, cudaStream_t st,
                                const awq::FusedEpi& epi) {
  using A = awq::act_t<kBf16>;
  static std::atomic<bool> attr_set[kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return AWQ_ERR_CUDA;
  auto kern = awq::gemv_stream_kernel<kNTiles, kOffset, kBf16, kBits, kFused>;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit) !=
        cudaSuccess)
      return AWQ_ERR_CUDA;
    attr_set[dev].store(true, std::memory_order_release);
  }
  awq::G4Smem lay;
  if (!gemv_config(M, N, K, &lay)) return AWQ_ERR_UNSUPPORTED;
  // packed codes [N, K * bits / 32] words in boxes of 16 rows x 32 words (128 B, swizzled);
  // scales [G, N] fp16 and zero points [G, N] uint8 in boxes of 16 groups x 16 rows
  CUtensorMap tw, ts, tz;
  if (!make_tmap_2d(&tw, qweight, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, N, K * kBits / 32,
                    awq::kGemvRows, 32, true) ||
      !make_tmap_2d(&ts, scales, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, K / awq::kGroup, N,
                    awq::kG4Groups, awq::kGemvRows, false) ||
      !make_tmap_2d(&tz, zeros, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, K / awq::kGroup, N,
                    awq::kG4Groups, awq::kGemvRows, false))
    return AWQ_ERR_CUDA;
  const int64_t tiles = N / awq::kGemvRows;
  // Two CTAs per SM (each its own tile range and ring) when both fit, for M <= 8: a CTA's
  // per-unit chain is latency-bound and a second CTA runs a second chain (measured 21.5
  // against 23.3 us on the three decode shapes at M = 1). At M <= 16 (two token tiles) one
  // CTA per SM keeps the ring and X of the larger tiles (two were slower there).
  const int per_sm = kNTiles == 1 && lay.total(kNTiles) <= kCoResidentSmem ? 2 : 1;
  const int64_t ctas = static_cast<int64_t>(num_sms()) * per_sm;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles < ctas ? tiles : ctas));
  cfg.blockDim = dim3(awq::kG4Threads);
  cfg.dynamicSmemBytes = static_cast<size_t>(lay.total(kNTiles));
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, tw, ts, tz, static_cast<const A*>(x),
                         static_cast<int>(M), N, K, inv_s, static_cast<A*>(y), lay,
                         flags, epi) != cudaSuccess)
    return AWQ_ERR_CUDA;
  return launch_status();
}

template <bool kBf16, int kBits, bool kFused>
awq_status launch_gemv_stream_m(const void* x, int64_t M, const uint32_t* qweight,
                                const __half* scales, const uint8_t* zeros, int64_t N, int64_t K,
                                const float* inv_s, unsigned flags, void* y, cudaStream_t st,
                                const awq::FusedEpi& epi) {
  if (M == 1)
    return launch_gemv_stream_t<1, true, kBf16, kBits, kFused>(x, M, qweight, scales, zeros, N, K,
                                                               inv_s, flags, y, st, epi);
  if constexpr (!kFused) {   // (the fused calls have at most 8 tokens: see fused_plan)
    if (M > 8)
      return launch_gemv_stream_t<2, false, kBf16, kBits, false>(x, M, qweight, scales, zeros, N, K,
                                                                 inv_s, flags, y, st, epi);
  }
  return launch_gemv_stream_t<1, false, kBf16, kBits, kFused>(x, M, qweight, scales, zeros, N, K,
                                                              inv_s, flags, y, st, epi);
}

// Returns AWQ_ERR_UNSUPPORTED when the shape does not suit the streaming kernel; the caller
// then uses the register-streaming kernel (fp16, 4-bit, M <= 8) or the tensor-core path.
template <bool kFused = false>
awq_status launch_gemv_stream(const void* x, int64_t M, const uint32_t* qweight,
                              const __half* scales, const uint8_t* zeros, int64_t N, int64_t K,
                              int bits, const float* inv_s, unsigned flags, void* y,
                              cudaStream_t st, const awq::FusedEpi& epi = {}) {
  if (!gemv_stream_fits(M, N, K)) return AWQ_ERR_UNSUPPORTED;
  const bool bf16 = (flags & AWQ_GEMM_BF16) != 0;
  if (bits == 3)
    return bf16 ? launch_gemv_stream_m<true, 3, kFused>(x, M, qweight, scales, zeros, N, K, inv_s,
                                                        flags, y, st, epi)
                : launch_gemv_stream_m<false, 3, kFused>(x, M, qweight, scales, zeros, N, K, inv_s,
                                                         flags, y, st, epi);
  return bf16 ? launch_gemv_stream_m<true, 4, kFused>(x, M, qweight, scales, zeros, N, K, inv_s,
                                                      flags, y, st, epi)
              : launch_gemv_stream_m<false, 4, kFused>(x, M, qweight, scales, zeros, N, K, inv_s,
                                                       flags, y, st, epi);
}

int tc_bn_for(int64_t M) { return M <= 32 ? 32 : M <= 64 ? 64 : M <= 128 ? 128 : 256; }

// Split-K for the tensor-core GEMM when the output has too few 128 x BN tiles to occupy the
// GPU (batched decode, small prefill). The persistent kernel runs one CTA per SM and hands
// out (tile, K slice) units round-robin, so the busiest SM does ceil(tiles * s / sms) units
// of K / s each: pick the split s that minimises that, i.e. ceil(tiles * s / sms) / s, with
// at least two 128-wide groups per slice and the partial traffic within about the packed
// weight bytes. A later s must win by more than 12% per extra slice: each slice adds a
// pipeline fill, an epilogue and 8 bytes of fp32 partial sums per output to reduce. On the
// batched shapes 12% measured best among 2, 6, 12, 40 and 60% (e.g. [14336, 4096] at M = 32
// runs unsplit, 26.6 -> 24.3 us; [4096, 14336] takes 4 slices instead of 9).
int splitk_for(int64_t M, int64_t N, int64_t K, int64_t bn = 0) {
  if (bn == 0) bn = tc_bn_for(M);
  const int64_t tiles = ((N + awq::kTcBM - 1) / awq::kTcBM) * ((M + bn - 1) / bn);
  const int64_t sms = num_sms();
  if (tiles >= sms) return 1;
  int64_t s_max = (K / awq::kGroup) / 2;
  const int64_t by_traffic = K / (8 * M);
  if (s_max > by_traffic) s_max = by_traffic;
  if (s_max > 16) s_max = 16;
  int best = 1;
  double best_cost = 1.0;
  for (int64_t s = 2; s <= s_max; ++s) {
    const double cost =
        static_cast<double>((tiles * s + sms - 1) / sms) / static_cast<double>(s);
    if (cost * (1.0 + 0.12 * static_cast<double>(s - best)) < best_cost) {
      best = static_cast<int>(s);
      best_cost = cost;
    }
  }
  return best;
}

bool bad_dim(int64_t v) { return v < 0 || v > kMaxDim; }

}  // namespace

extern "C" {

const char* awq_status_string(awq_status status) {
  switch (status) {
    case AWQ_OK: return "AWQ_OK";
    case AWQ_ERR_INVALID_ARG: return "AWQ_ERR_INVALID_ARG";
    case AWQ_ERR_UNSUPPORTED: return "AWQ_ERR_UNSUPPORTED";
    case AWQ_ERR_WORKSPACE: return "AWQ_ERR_WORKSPACE";
    case AWQ_ERR_CUDA: return "AWQ_ERR_CUDA";
    case AWQ_ERR_TIMEOUT: return "AWQ_ERR_TIMEOUT";
    case AWQ_ERR_BOUNDS: return "AWQ_ERR_BOUNDS";
  }
  return "AWQ_ERR_UNKNOWN";
}

int awq_abi_version(void) { return 2; }

awq_status awq_check_error(void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cudaStreamSynchronize(st) != cudaSuccess) return AWQ_ERR_CUDA;
  unsigned int word = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&word, awq::g_status_word, sizeof(word)) != cudaSuccess)
    return AWQ_ERR_CUDA;
  if (word != 0 && cudaMemcpyToSymbol(awq::g_status_word, &zero, sizeof(zero)) != cudaSuccess)
    return AWQ_ERR_CUDA;
  if (word & awq::kDevErrBounds) return AWQ_ERR_BOUNDS;
  if (word & awq::kDevErrTimeout) return AWQ_ERR_TIMEOUT;
  return AWQ_OK;
}

awq_status awq_selftest_bounds(int* buf, void* stream) {
#ifdef AWQ_DEBUG_BOUNDS
  if (buf == nullptr || (reinterpret_cast<uintptr_t>(buf) & 15u) != 0) return AWQ_ERR_INVALID_ARG;
  awq::bounds_selftest_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(buf, 4);
  return launch_status();
#else
  (void)buf;
  (void)stream;
  return AWQ_ERR_UNSUPPORTED;   // the release build has no bounds checks
#endif
}

awq_status awq_trace_reset(void) {
#ifdef AWQ_TRACE
  static_assert(awq::kTraceWords == AWQ_TRACE_WORDS, "trace record size");
  const unsigned zero = 0;
  if (cudaMemcpyToSymbol(awq::g_trace_ctas, &zero, sizeof(zero)) != cudaSuccess)
    return AWQ_ERR_CUDA;
  return AWQ_OK;
#else
  return AWQ_ERR_UNSUPPORTED;   // only the trace build records a timeline
#endif
}

awq_status awq_trace_read(unsigned long long* out, int64_t max_ctas, int64_t* n_ctas) {
#ifdef AWQ_TRACE
  if (out == nullptr || n_ctas == nullptr || max_ctas < 0) return AWQ_ERR_INVALID_ARG;
  unsigned count = 0;
  if (cudaMemcpyFromSymbol(&count, awq::g_trace_ctas, sizeof(count)) != cudaSuccess)
    return AWQ_ERR_CUDA;
  int64_t n = count < static_cast<unsigned>(awq::kTraceCtas) ? count : awq::kTraceCtas;
  if (n > max_ctas) n = max_ctas;
  if (n > 0 &&
      cudaMemcpyFromSymbol(out, awq::g_trace,
                           static_cast<size_t>(n) * awq::kTraceWords * sizeof(unsigned long long)) !=
          cudaSuccess)
    return AWQ_ERR_CUDA;
  *n_ctas = count;
  return AWQ_OK;
#else
  (void)out;
  (void)max_ctas;
  (void)n_ctas;
  return AWQ_ERR_UNSUPPORTED;
#endif
}

awq_status awq_selftest_timeout(int* waited_out, void* stream) {
  if (waited_out == nullptr || (reinterpret_cast<uintptr_t>(waited_out) & 3u) != 0)
    return AWQ_ERR_INVALID_ARG;
  awq::timeout_selftest_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(
      50ull * 1000 * 1000, waited_out);
  return launch_status();
}

// ------------------------------------------------------------------ act_stats
size_t awq_act_stats_workspace_size(int64_t M, int64_t K) {
  if (M <= 0 || K <= 0) return 0;
  const int splits = awq::act_stats_splits(M, K, num_sms());
  return static_cast<size_t>(splits) * static_cast<size_t>(K) * sizeof(double);
}

awq_status awq_act_stats(const awq_f16* X, int64_t M, int64_t K, float* s_x, void* workspace,
                         size_t ws_bytes, void* stream) {
  if (bad_dim(M) || bad_dim(K) || M == 0) return AWQ_ERR_INVALID_ARG;
  if (K == 0) return AWQ_OK;
  if (K % 8 != 0) return AWQ_ERR_INVALID_ARG;
  if (!X || !s_x || !aligned16(X) || !aligned16(s_x)) return AWQ_ERR_INVALID_ARG;
  const int splits = awq::act_stats_splits(M, K, num_sms());
  const size_t need = static_cast<size_t>(splits) * static_cast<size_t>(K) * sizeof(double);
  if (!workspace || ws_bytes < need || !aligned16(workspace)) return AWQ_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  double* part = static_cast<double*>(workspace);
  const int64_t rows_per_split = (M + splits - 1) / splits;
  dim3 g1(static_cast<unsigned>((K + awq::kStatsCols - 1) / awq::kStatsCols),
          static_cast<unsigned>(splits));
  awq::act_stats_partial_kernel<<<g1, 256, 0, st>>>(reinterpret_cast<const __half*>(X), M, K,
                                                   rows_per_split, part);
  awq_status s = launch_status();
  if (s != AWQ_OK) return s;
  awq::act_stats_finish_kernel<<<static_cast<unsigned>((K + 255) / 256), 256, 0, st>>>(
      part, splits, M, K, s_x);
  return launch_status();
}

}  // extern "C"

// ------------------------------------------------------------------ act_stats without allocation
// Scratch for awq_act_stats_noalloc: the fp64 partial sums live in this file-scope device
// array instead of a caller workspace. Every GPU that loads the library holds it until the
// process exits. In host code the name is only a stand-in for the symbol, so its device
// address is looked up once per device (with that device current) and cached.
namespace {
constexpr int64_t kNoAllocScratchDoubles = int64_t{1} << 17;   // 1 MiB
constexpr int64_t kNoAllocMaxK = 65536;                       // >= 2 row slices per call
static __device__ __align__(256) double g_noalloc_scratch[kNoAllocScratchDoubles];

double* g_noalloc_ptr[kMaxDevices] = {nullptr};
std::mutex g_noalloc_mu;

awq_status noalloc_scratch(double** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return AWQ_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_noalloc_mu);
  if (g_noalloc_ptr[dev] == nullptr) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_noalloc_scratch) != cudaSuccess || p == nullptr)
      return AWQ_ERR_CUDA;
    g_noalloc_ptr[dev] = static_cast<double*>(p);
  }
  *out = g_noalloc_ptr[dev];
  return AWQ_OK;
}
}  // namespace

extern "C" {

awq_status awq_act_stats_noalloc(const awq_f16* X, int64_t M, int64_t K, float* s_x,
                                 void* stream) {
  if (bad_dim(M) || bad_dim(K) || M == 0) return AWQ_ERR_INVALID_ARG;
  if (K == 0) return AWQ_OK;
  if (K % 8 != 0 || K > kNoAllocMaxK) return AWQ_ERR_INVALID_ARG;
  if (!X || !s_x || !aligned16(X) || !aligned16(s_x)) return AWQ_ERR_INVALID_ARG;
  double* part = nullptr;
  awq_status s = noalloc_scratch(&part);
  if (s != AWQ_OK) return s;
  int splits = awq::act_stats_splits(M, K, num_sms());
  const int64_t cap = kNoAllocScratchDoubles / K;
  if (splits > cap) splits = static_cast<int>(cap);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // Pass 1 writes every (slice, channel) partial it later reads, so nothing of an earlier
  // call's contents is used and the array needs no clearing.
  const int64_t rows_per_split = (M + splits - 1) / splits;
  dim3 g1(static_cast<unsigned>((K + awq::kStatsCols - 1) / awq::kStatsCols),
          static_cast<unsigned>(splits));
  awq::act_stats_partial_kernel<<<g1, 256, 0, st>>>(reinterpret_cast<const __half*>(X), M, K,
                                                   rows_per_split, part);
  if ((s = launch_status()) != AWQ_OK) return s;
  awq::act_stats_finish_kernel<<<static_cast<unsigned>((K + 255) / 256), 256, 0, st>>>(
      part, splits, M, K, s_x);
  return launch_status();
}

// ------------------------------------------------------------------ quantize_pack
awq_status awq_quantize_pack(const awq_f16* W, int64_t N, int64_t K, const float* s, int bits,
                             int group, uint32_t* qweight, awq_f16* scales, uint8_t* zeros,
                             void* stream) {
  if (bad_dim(N) || bad_dim(K) || K == 0) return AWQ_ERR_INVALID_ARG;
  if (group != awq::kGroup || K % awq::kGroup != 0) return AWQ_ERR_INVALID_ARG;
  if (bits != 4 && bits != 3) return AWQ_ERR_INVALID_ARG;
  if (N == 0) return AWQ_OK;
  if (!W || !qweight || !scales || !zeros) return AWQ_ERR_INVALID_ARG;
  if (!aligned16(W) || !aligned16(qweight) || !aligned16(scales) || !aligned16(zeros) ||
      (s && !aligned16(s)))
    return AWQ_ERR_INVALID_ARG;
  if ((K / awq::kGroup) > 65535) return AWQ_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  dim3 grid(static_cast<unsigned>((N + awq::kQuantRowsPerCta - 1) / awq::kQuantRowsPerCta),
            static_cast<unsigned>(K / awq::kGroup));
  const __half* w = reinterpret_cast<const __half*>(W);
  __half* sc = reinterpret_cast<__half*>(scales);
  if (bits == 4)
    awq::quantize_pack_kernel<4><<<grid, 256, 0, st>>>(w, N, K, s, qweight, sc, zeros);
  else
    awq::quantize_pack_kernel<3><<<grid, 256, 0, st>>>(w, N, K, s, qweight, sc, zeros);
  return launch_status();
}

// ------------------------------------------------------------------ search
namespace {
// The error operand E is built and reduced for a chunk of grid points at a time, so the
// workspace stays bounded whatever the layer: at most this many bytes of E per chunk (at
// least one grid point per chunk).
constexpr size_t kSearchChunkBytes = size_t{1} << 30;
// Column tile of the Gram-form loss GEMM (its N side is channels).
constexpr int kGramBN = 128;

// The loss is evaluated in its Gram form e G e^T (G = X^T X, N K^2 per grid point plus K^2 M
// once) when that is cheaper than the direct ||E X^T||^2 (N K M per grid point) with margin:
// the Gram MMAs cost 1.5 times the direct ones per product (three instead of two), so when
// M >= 2K.
bool search_uses_gram(int64_t M, int64_t K) { return M >= 2 * K; }

struct SearchWs {
  int chunk;   // grid points per chunk
  bool gram;
  int64_t M_pad;
  size_t table, inv, err, part, rows, xt, g, g2, rms, total;
};
SearchWs search_ws_layout(int64_t M, int64_t N, int64_t K, int n_alpha) {
  const int64_t N_pad = round_up(N, awq::kTcBM);
  SearchWs w;
  w.gram = search_uses_gram(M, K);
  w.M_pad = round_up(M, awq::kGroup);
  const int64_t m_tiles = w.gram ? K / kGramBN : (M + tc_bn_for(M) - 1) / tc_bn_for(M);
  const size_t per_point = static_cast<size_t>(N_pad) * 2 * K * sizeof(__half);   // hi, lo
  int64_t chunk = static_cast<int64_t>(kSearchChunkBytes / per_point);
  if (chunk < 1) chunk = 1;
  if (chunk > n_alpha) chunk = n_alpha;
  w.chunk = static_cast<int>(chunk);
  w.table = 0;
  w.inv = align256(static_cast<size_t>(n_alpha) * K * sizeof(float));
  w.err = w.inv + align256(static_cast<size_t>(n_alpha) * K * sizeof(float));
  w.part = w.err + align256(static_cast<size_t>(chunk) * per_point);
  w.rows = w.part + align256(static_cast<size_t>(chunk) * N_pad * m_tiles * sizeof(double));
  w.xt = w.rows + align256(static_cast<size_t>(n_alpha) * N * sizeof(double));
  size_t end = w.xt;
  if (w.gram) {   // X^T [K, M_pad] fp16, G [K, K] fp32, G' [K, 2K] fp16 parts, rms [K]
    w.g = w.xt + align256(static_cast<size_t>(K) * w.M_pad * sizeof(__half));
    w.g2 = w.g + align256(static_cast<size_t>(K) * K * sizeof(float));
    w.rms = w.g2 + align256(static_cast<size_t>(K) * 2 * K * sizeof(__half));
    end = w.rms + align256(static_cast<size_t>(K) * sizeof(float));
  }
  w.total = end;
  return w;
}
}  // namespace

size_t awq_search_scale_workspace_size(int64_t M, int64_t N, int64_t K, int n_alpha) {
  if (M <= 0 || N <= 0 || K <= 0 || n_alpha <= 0) return 0;
  return search_ws_layout(M, N, K, n_alpha).total;
}

awq_status awq_search_scale(const awq_f16* W, int64_t N, int64_t K, const awq_f16* X,
                            int64_t M, const float* s_x, const float* alphas, int n_alpha,
                            int bits, int group, const float* s_table, double* losses,
                            int32_t* best_idx, float* best_s, float* best_inv_s,
                            double* row_losses, void* workspace, size_t ws_bytes,
                            void* stream) {
  if (bad_dim(N) || bad_dim(K) || bad_dim(M) || N == 0 || K == 0 || M == 0)
    return AWQ_ERR_INVALID_ARG;
  if (group != awq::kGroup || K % awq::kGroup != 0) return AWQ_ERR_INVALID_ARG;
  if (bits != 4 && bits != 3) return AWQ_ERR_INVALID_ARG;
  if (n_alpha < 1 || n_alpha > 64) return AWQ_ERR_INVALID_ARG;
  if (!W || !X || !losses || !best_idx || !best_s) return AWQ_ERR_INVALID_ARG;
  if (!s_table && (!s_x || !alphas)) return AWQ_ERR_INVALID_ARG;
  if (!aligned16(W) || !aligned16(X) || !aligned16(losses) || !aligned16(best_idx) ||
      !aligned16(best_s) || (s_x && !aligned16(s_x)) || (alphas && !aligned16(alphas)) ||
      (s_table && !aligned16(s_table)) || (row_losses && !aligned16(row_losses)) ||
      (best_inv_s && !aligned16(best_inv_s)))
    return AWQ_ERR_INVALID_ARG;
  const int64_t N_pad = round_up(N, awq::kTcBM);
  if (N_pad / awq::kTcBM > 65535 || K / awq::kGroup > 65535) return AWQ_ERR_INVALID_ARG;
  const SearchWs lay = search_ws_layout(M, N, K, n_alpha);
  if (static_cast<int64_t>(lay.chunk) * N_pad / awq::kTcBM > 65535) return AWQ_ERR_INVALID_ARG;
  if (lay.gram && (K / 32 > 65535 || lay.M_pad / 32 > 2147483647LL)) return AWQ_ERR_INVALID_ARG;
  if (!workspace || ws_bytes < lay.total || !aligned16(workspace)) return AWQ_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  float* table = reinterpret_cast<float*>(ws + lay.table);
  __half* E = reinterpret_cast<__half*>(ws + lay.err);
  double* part = reinterpret_cast<double*>(ws + lay.part);
  const __half* x = reinterpret_cast<const __half*>(X);
  awq_status s;

  const float* S = s_table;
  if (S == nullptr) {
    dim3 g(static_cast<unsigned>((K + 255) / 256), static_cast<unsigned>(n_alpha));
    awq::scale_candidates_kernel<<<g, 256, 0, st>>>(s_x, alphas, n_alpha, K, table);
    if ((s = launch_status()) != AWQ_OK) return s;
    S = table;
  }
  float* inv = reinterpret_cast<float*>(ws + lay.inv);
  {
    const int64_t total = static_cast<int64_t>(n_alpha) * K;
    awq::inv_table_kernel<<<static_cast<unsigned>((total + 255) / 256), 256, 0, st>>>(S, total, inv);
    if ((s = launch_status()) != AWQ_OK) return s;
  }
  // Gram form: X^T (tokens contiguous, padded to whole groups), G = X^T X on the tensor
  // cores, the channels' root mean squares, and G normalised to two fp16 parts
  float* rms = nullptr;
  const __half* G2 = nullptr;
  if (lay.gram) {
    __half* XT = reinterpret_cast<__half*>(ws + lay.xt);
    float* G = reinterpret_cast<float*>(ws + lay.g);
    __half* G2w = reinterpret_cast<__half*>(ws + lay.g2);
    rms = reinterpret_cast<float*>(ws + lay.rms);
    dim3 gt(static_cast<unsigned>(lay.M_pad / 32), static_cast<unsigned>((K + 31) / 32));
    awq::transpose_pad_kernel<<<gt, 256, 0, st>>>(x, M, K, lay.M_pad, XT);
    if ((s = launch_status()) != AWQ_OK) return s;
    awq::TcArgs ga{};
    ga.M = K;            // B rows: channels j
    ga.N = K;
    ga.N_pad = K;
    ga.K = lay.M_pad;    // the contraction runs over tokens
    ga.G = G;
    ga.upper_only = 1;   // G is symmetric: the tiles at or above the diagonal suffice
    // the contraction over tokens in slices of about 2048 (128 accumulation steps each)
    ga.k_splits = static_cast<int>(lay.M_pad / 2048 > 1 ? lay.M_pad / 2048 : 1);
    s = launch_tc<256, ASrc::kFp16x1, Epi::kStoreF32>(XT, K, XT, K, ga, st);
    if (s != AWQ_OK) return s;
    awq::gram_rms_kernel<<<static_cast<unsigned>((K + 255) / 256), 256, 0, st>>>(G, K, M, rms);
    if ((s = launch_status()) != AWQ_OK) return s;
    dim3 gn(static_cast<unsigned>((K + 255) / 256), static_cast<unsigned>(K));
    awq::gram_normalize_kernel<<<gn, 256, 0, st>>>(G, K, G2w);
    if ((s = launch_status()) != AWQ_OK) return s;
    G2 = G2w;
  }
  const int bn = lay.gram ? kGramBN : tc_bn_for(M);
  const int m_tiles = lay.gram ? static_cast<int>(K / kGramBN) : static_cast<int>((M + bn - 1) / bn);
  double* rl = row_losses != nullptr ? row_losses : reinterpret_cast<double*>(ws + lay.rows);
  const __half* w = reinterpret_cast<const __half*>(W);
  for (int a0 = 0; a0 < n_alpha; a0 += lay.chunk) {
    const int na = n_alpha - a0 < lay.chunk ? n_alpha - a0 : lay.chunk;
    const float* Sa = S + static_cast<int64_t>(a0) * K;
    const float* Ia = inv + static_cast<int64_t>(a0) * K;
    {
      dim3 g(static_cast<unsigned>(N_pad / awq::kQuantRowsPerCta),
             static_cast<unsigned>(K / awq::kGroup), static_cast<unsigned>(na));
      if (bits == 4)
        awq::search_build_error_kernel<4><<<g, 256, 0, st>>>(w, N, K, N_pad, Sa, Ia, rms, E);
      else
        awq::search_build_error_kernel<3><<<g, 256, 0, st>>>(w, N, K, N_pad, Sa, Ia, rms, E);
      if ((s = launch_status()) != AWQ_OK) return s;
    }
    {
      awq::TcArgs args{};
      args.M = lay.gram ? K : M;
      args.N = N;
      args.N_pad = N_pad;
      args.K = K;
      args.row_part = part;
      args.m_tiles = m_tiles;
      args.k_splits = 1;
      args.E2 = E;
      s = lay.gram ? launch_tc<kGramBN, ASrc::kGram, Epi::kGramDot>(G2, K, E, na * N_pad, args, st)
                   : launch_tc_bn<ASrc::kSplit16, Epi::kRowSumSq>(X, M, E, na * N_pad, args, st);
      if (s != AWQ_OK) return s;
    }
    {
      const int64_t n = static_cast<int64_t>(na) * N;
      awq::search_row_loss_kernel<<<static_cast<unsigned>((n + awq::kReduceThreads - 1) /
                                                          awq::kReduceThreads),
                                    awq::kReduceThreads, 0, st>>>(
          part, N, N_pad, na, m_tiles, lay.gram ? static_cast<double>(M) : 1.0,
          rl + static_cast<int64_t>(a0) * N);
      if ((s = launch_status()) != AWQ_OK) return s;
    }
  }
  awq::search_reduce_kernel<<<n_alpha, awq::kReduceThreads, 0, st>>>(rl, N, losses);
  if ((s = launch_status()) != AWQ_OK) return s;
  awq::search_pick_kernel<<<static_cast<unsigned>((K + 255) / 256), 256, 0, st>>>(
      losses, n_alpha, S, inv, K, best_idx, best_s, best_inv_s);
  return launch_status();
}

// ------------------------------------------------------------------ gated MLP input
awq_status awq_silu_mul_gemm(const awq_f16* X, int64_t M, const awq_f16* W_gate,
                             const awq_f16* W_up, int64_t I, int64_t K, awq_f16* H,
                             void* stream) {
  if (bad_dim(M) || bad_dim(I) || bad_dim(K) || K == 0) return AWQ_ERR_INVALID_ARG;
  if (K % awq::kGroup != 0) return AWQ_ERR_INVALID_ARG;
  if (M == 0 || I == 0) return AWQ_OK;
  if (!X || !W_gate || !W_up || !H) return AWQ_ERR_INVALID_ARG;
  if (!aligned16(X) || !aligned16(W_gate) || !aligned16(W_up) || !aligned16(H))
    return AWQ_ERR_INVALID_ARG;
  if ((I + awq::kTcBM - 1) / awq::kTcBM > 65535) return AWQ_ERR_INVALID_ARG;
  awq::TcArgs args{};
  args.M = M;
  args.N = I;
  args.N_pad = I;
  args.K = K;
  args.Y = reinterpret_cast<__half*>(H);
  args.m_tiles = static_cast<int>((M + tc_bn_for(M) - 1) / tc_bn_for(M));
  args.k_splits = 1;
  return launch_tc_bn<ASrc::kPair16, Epi::kSiluMul>(X, M,
                                                    W_gate, I, args,
                                                    static_cast<cudaStream_t>(stream), W_up);
}

// ------------------------------------------------------------------ GEMM
size_t awq_gemm_workspace_size(int64_t M, int64_t N, int64_t K, int bits) {
  if (M <= 0 || K <= 0 || N <= 0) return 0;
  // the streaming kernel needs none; a call that it cannot take (an X too large for it, or
  // N % 16 != 0) may take the tensor-core path below: with bf16 activations, at 3 bits or past 8
  // rows (the size covers either type)
  (void)bits;
  if (M <= 16 && gemv_stream_fits(M, N, K)) return 0;
  const int splits = splitk_for(M, N, K);
  return splits > 1 ? align256(static_cast<size_t>(splits) * M * N * sizeof(float)) : 0;
}

awq_status awq_gemm_w4a16(const awq_f16* X, int64_t M, const uint32_t* qweight,
                          const awq_f16* scales, const uint8_t* zeros, int64_t N, int64_t K,
                          int bits, int group, const float* inv_s, unsigned flags, awq_f16* Y,
                          void* workspace, size_t ws_bytes, void* stream) {
  if (bad_dim(M) || bad_dim(N) || bad_dim(K) || K == 0) return AWQ_ERR_INVALID_ARG;
  if (group != awq::kGroup || K % awq::kGroup != 0) return AWQ_ERR_INVALID_ARG;
  if (bits != 4 && bits != 3) return AWQ_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return AWQ_OK;
  if (!X || !qweight || !scales || !zeros || !Y) return AWQ_ERR_INVALID_ARG;
  if (!aligned16(X) || !aligned16(qweight) || !aligned16(scales) || !aligned16(zeros) ||
      !aligned16(Y) || (inv_s && !aligned16(inv_s)))
    return AWQ_ERR_INVALID_ARG;
  if ((flags & ~static_cast<unsigned>(AWQ_GEMM_WEIGHTS_READY | AWQ_GEMM_BF16)) != 0)
    return AWQ_ERR_INVALID_ARG;
  const bool bf16 = (flags & AWQ_GEMM_BF16) != 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const __half* sc = reinterpret_cast<const __half*>(scales);

  if (M <= 16) {
    awq_status r = launch_gemv_stream(X, M, qweight, sc, zeros, N, K, bits, inv_s, flags, Y, st);
    if (r != AWQ_ERR_UNSUPPORTED) return r;
    // the streaming kernel cannot hold X (or N % 16 != 0): register streaming for fp16 4-bit
    // with M <= 8, the tensor-core path below otherwise
    if (M <= 8 && !bf16 && bits == 4) {
      const unsigned grid = static_cast<unsigned>((N + awq::kGemvRows - 1) / awq::kGemvRows);
      awq::gemv_w4a16_kernel<1><<<grid, awq::kGemvWarps * 32, 0, st>>>(
          reinterpret_cast<const __half*>(X), static_cast<int>(M), qweight, sc, zeros, N, K,
          inv_s, reinterpret_cast<__half*>(Y));
      return launch_status();
    }
  }
  if ((N + awq::kTcBM - 1) / awq::kTcBM > 65535) return AWQ_ERR_INVALID_ARG;
  const int splits = splitk_for(M, N, K);
  const size_t part_bytes =
      splits > 1 ? align256(static_cast<size_t>(splits) * M * N * sizeof(float)) : 0;
  if (part_bytes > 0 && (!workspace || ws_bytes < part_bytes || !aligned16(workspace)))
    return AWQ_ERR_WORKSPACE;
  float* partial = splits > 1 ? static_cast<float*>(workspace) : nullptr;
  awq::TcArgs args{};
  args.M = M;
  args.N = N;
  args.N_pad = N;
  args.K = K;
  args.scales = sc;
  args.zeros = zeros;
  args.Y = Y;
  args.m_tiles = static_cast<int>((M + tc_bn_for(M) - 1) / tc_bn_for(M));
  args.k_splits = splits;
  args.partial = partial;
  args.inv_s = inv_s;   // folded into the dequantized weights by the builders
  awq_status r;
  if (bf16)
    r = bits == 3 ? launch_tc_bn<ASrc::kPacked3, Epi::kStoreY, true>(X, M, qweight, N, args, st)
                  : launch_tc_bn<ASrc::kPacked4, Epi::kStoreY, true>(X, M, qweight, N, args, st);
  else
    r = bits == 3 ? launch_tc_bn<ASrc::kPacked3, Epi::kStoreY>(X, M, qweight, N, args, st)
                  : launch_tc_bn<ASrc::kPacked4, Epi::kStoreY>(X, M, qweight, N, args, st);
  if (r != AWQ_OK || splits == 1) return r;
  const int64_t MN = M * N;
  const unsigned rgrid = static_cast<unsigned>((MN / 4 + 1 + 255) / 256);
  if (bf16)
    awq::splitk_reduce_kernel<true><<<rgrid, 256, 0, st>>>(
        partial, splits, MN, reinterpret_cast<__nv_bfloat16*>(Y));
  else
    awq::splitk_reduce_kernel<false><<<rgrid, 256, 0, st>>>(partial, splits, MN,
                                                            reinterpret_cast<__half*>(Y));
  return launch_status();
}

}  // extern "C"

// ------------------------------------------------------------------ fused epilogue, experts
namespace {
bool bad_ptr16(const void* p) { return p != nullptr && !aligned16(p); }

template <typename... KArgs, typename... Args>
awq_status launch_pdl(void (*kern)(KArgs...), dim3 grid, int threads, int smem, cudaStream_t st,
                      Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess) return AWQ_ERR_CUDA;
  return launch_status();
}

// The tensor-core kernel's token tile. Each token tile dequantizes the weight again, so: one that
// holds all rows where it can, and equal ones where it cannot; with experts half as much again as
// the mean row count, which differs from expert to expert (8 experts of [14336, 4096] with 512
// rows, 52 to 75 each: 143 us with tiles of 64, 113 with 128).
int tensor_bn(int64_t T, int64_t E) {
  const int64_t tiles = (T + 191) / 192;
  const int64_t rows = E == 1 ? (T + tiles - 1) / tiles : (T + E - 1) / E * 3 / 2;
  return rows <= 32 ? 32 : rows <= 64 ? 64 : rows <= 128 ? 128 : 192;
}

// Which product kernel a call takes, from its shape alone, and the streaming kernel's variant.
struct FusedPlan {
  enum Kind { kDecode, kStream, kTensor } kind;
  int rb, xrows, slots;   // kStream; split: each token as two rows of X
  int split;
  int splits;             // kTensor: K slices, and where their partial sums start
  size_t prepared;
  size_t workspace;
};

template <int kRB, bool kBf16, int kBits>
awq_status launch_stream(const FusedPlan& plan, const void* X, const float* inv_s,
                         const uint32_t* qweight, awq::StreamArgs a, void* workspace,
                         cudaStream_t st) {
  using L = awq::SfLayout<kRB>;
  static std::atomic<bool> attr_set[kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return AWQ_ERR_CUDA;
  auto kern = awq::stream_fused_kernel<kRB, kBf16, kBits>;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit) !=
        cudaSuccess)
      return AWQ_ERR_CUDA;
    attr_set[dev].store(true, std::memory_order_release);
  }
  constexpr int kRows = awq::kGemvRows * kRB;
  a.xrows = plan.xrows;
  a.slots = plan.slots;
  a.split = plan.split;
  CUtensorMap tw;
  if (!make_tmap_2d(&tw, qweight, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, a.E * a.N, a.K * kBits / 32,
                    kRows, 32, true))
    return AWQ_ERR_CUDA;
  // X in the kernel's layout first, in the workspace
  const awq_status r = launch_pdl(
      awq::prepare_rows_kernel<kBf16, true>, dim3(static_cast<unsigned>(a.T)), awq::kPrepThreads, 0, st,
      static_cast<const uint4*>(X), a.T, a.K, inv_s, a.offsets, a.E, L::kChunkG, L::kXChunk, a.split,
      static_cast<uint8_t*>(workspace));
  if (r != AWQ_OK) return r;
  a.xprep = static_cast<const uint8_t*>(workspace);
  // at most this many tiles: T rows in blocks, one more for each expert with rows
  const int tokens = a.xrows >> a.split;
  const int64_t blocks = a.offsets == nullptr ? (a.T + tokens - 1) / tokens
                                              : a.T / tokens + (a.T < a.E ? a.T : a.E);
  const int64_t tiles = (a.N + kRows - 1) / kRows * blocks;
  const int smem = L::total(a.slots, a.xrows, a.E);
  const int64_t ctas = static_cast<int64_t>(num_sms()) * (smem <= kCoResidentSmem ? 2 : 1);
  return launch_pdl(kern, dim3(static_cast<unsigned>(tiles < ctas ? tiles : ctas)), awq::kG4Threads,
                    smem, st, tw, a);
}

template <bool kBf16, int kBits>
awq_status launch_stream_plan(const FusedPlan& p, const void* X, const float* inv_s,
                              const uint32_t* qweight, const awq::StreamArgs& a, void* ws,
                              cudaStream_t st) {
  if (p.rb == 4) return launch_stream<4, kBf16, kBits>(p, X, inv_s, qweight, a, ws, st);
  if (p.rb == 2) return launch_stream<2, kBf16, kBits>(p, X, inv_s, qweight, a, ws, st);
  return launch_stream<1, kBf16, kBits>(p, X, inv_s, qweight, a, ws, st);
}

template <int kRB>
void plan_stream(FusedPlan& p, int64_t T, int64_t E, int64_t K) {
  using L = awq::SfLayout<kRB>;
  p.kind = FusedPlan::kStream;
  p.rb = kRB;
  p.slots = awq::kSfMaxSlots;
  for (int budget : {kCoResidentSmem, kSmemLimit}) {
    p.slots = awq::kSfMaxSlots;
    while (p.slots >= 2 && L::total(p.slots, p.xrows, static_cast<int>(E)) > budget) --p.slots;
    if (p.slots >= 2) break;
  }
  const int64_t chunks = (K / awq::kGroup + L::kChunkG - 1) / L::kChunkG;
  p.workspace = align256(static_cast<size_t>(T) * ((chunks * L::kXChunk << p.split) + sizeof(float)));
}

// The decode kernel (one launch, no workspace) for the shortest dense calls: at M = 1, 4 and 8 it
// took 5.6, 7.0 and 8.6 us on [4096, 4096] where the streaming kernel behind its preparation
// took 6.6, 9.1 and 9.4; on [11008, 4096] they are equal (12.3 and 12.4 at M = 1, 14.1 and 13.5
// at 8), on [4096, 11008] the streaming kernel is faster at M = 8 (16.9 against 20.2).
// The streaming kernel up to 8 rows of an expert on average: 8 experts of [14336, 4096] with 64
// rows took 80 us there and 100 on the tensor-core kernel, with 128 rows 138 (in blocks of 16
// tokens) and 101.
// inv_s: the decode kernel rounds x * inv_s to 16 bits, so a call with it goes to the others; fp16
// activations then take two rows each in the streaming kernel, in blocks of 4 tokens. From 5 tokens
// to 8 two blocks read each weight: us there and on the tensor-core kernel, 8 rows, 4 bits:
// [4096, 4096] 10.3 and 11.5, [14336, 4096] 20.2 and 24.8, [4096, 14336] 25.9 and 24.2; 3 bits:
// [4096, 4096] 12.9 and 11.7, [14336, 4096] 32.3 and 24.8; 64 rows over 8 experts of [14336, 4096] 104
// and 154, 1024 over 128 of [1536, 2048] 101 and 136. All go to the streaming kernel, where nothing is
// rounded before the output (error 2.1e-4 against 2.9e-4 with the weights as fp16).
FusedPlan fused_plan(int64_t T, int64_t E, int64_t N, int64_t K, bool grouped, bool inv, bool bf16) {
  FusedPlan p{};
  if (!grouped && !inv && (T <= 2 || (T <= 8 && N <= (int64_t{1} << 25) / K)) &&
      gemv_stream_fits(T, N, K)) {
    p.kind = FusedPlan::kDecode;
    return p;
  }
  p.split = inv && !bf16 ? 1 : 0;
  const int most = 8 >> p.split;   // tokens of a block
  if (T <= 8 * E) {
    p.xrows = static_cast<int>(T < most ? T : most) << p.split;
    const int64_t blocks = grouped ? T / most + (T < E ? T : E) : (T + most - 1) / most;
    // 64 weight rows a tile read the tokens least often; 32 with few tokens (one token of two
    // experts [14336, 4096]: 18.7 us against 20.0), and fewer where there are too few tiles
    int rb = p.xrows <= 4 ? 2 : 4;
    while (rb > 1 && (N + 16 * rb - 1) / (16 * rb) * blocks < num_sms()) rb /= 2;
    if (rb == 4) plan_stream<4>(p, T, E, K);
    else if (rb == 2) plan_stream<2>(p, T, E, K);
    else plan_stream<1>(p, T, E, K);
    return p;
  }
  p.kind = FusedPlan::kTensor;
  // prepared activations (bf16) and their factors, then the partial sums of K slices
  p.prepared = bf16 ? align256(static_cast<size_t>(T) * (2 * K + sizeof(float))) : 0;
  p.splits = grouped ? 1 : splitk_for(T, N, K, tensor_bn(T, 1));
  p.workspace = p.prepared +
                (p.splits > 1 ? align256(static_cast<size_t>(p.splits) * T * N * sizeof(float)) : 0);
  return p;
}

template <int BN, bool kBf16, int kBits, bool kInv>
awq_status launch_tensor_bn(const void* X, const uint32_t* qweight, awq::FusedArgs a, int early,
                            cudaStream_t st) {   // X fp16, whatever Y's type
  using L = awq::TfLayout<BN, kBits>;
  static std::atomic<bool> attr_set[kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return AWQ_ERR_CUDA;
  auto kern = awq::tc_fused_kernel<BN, kBf16, kBits, kInv>;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem) !=
        cudaSuccess)
      return AWQ_ERR_CUDA;
    attr_set[dev].store(true, std::memory_order_release);
  }
  CUtensorMap tx, tw;
  if (!make_tmap_2d(&tx, X, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, a.M, a.K, BN, awq::kTcBK, true) ||
      !make_tmap_2d(&tw, qweight, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, a.E * a.N, a.K * kBits / 32,
                    awq::kTcBM, L::kRowBytes / 4, kBits == 4))
    return AWQ_ERR_CUDA;
  a.row_tiles = static_cast<int>((a.N + awq::kTcBM - 1) / awq::kTcBM);
  const int64_t tiles = a.offsets == nullptr ? (a.M + BN - 1) / BN
                                             : a.M / BN + (a.M < a.E ? a.M : a.E);
  const int64_t units = a.row_tiles * tiles * a.k_splits;
  if (units > kMaxDim) return AWQ_ERR_INVALID_ARG;   // the kernel counts them in 32 bits
  const int64_t sms = num_sms();
  return launch_pdl(kern, dim3(static_cast<unsigned>(units < sms ? units : sms)), awq::kTfThreads,
                    L::kSmem, st, tx, tw, a, early);
}

template <bool kBf16, int kBits, bool kInv = false>
awq_status launch_tensor(const void* X, const uint32_t* qweight, const awq::FusedArgs& a, int early,
                         cudaStream_t st) {
  switch (tensor_bn(a.M, a.E)) {
    case 32: return launch_tensor_bn<32, kBf16, kBits, kInv>(X, qweight, a, early, st);
    case 64: return launch_tensor_bn<64, kBf16, kBits, kInv>(X, qweight, a, early, st);
    case 128: return launch_tensor_bn<128, kBf16, kBits, kInv>(X, qweight, a, early, st);
    default: return launch_tensor_bn<192, kBf16, kBits, kInv>(X, qweight, a, early, st);
  }
}

// What the products with a fused epilogue share: argument checks past the shapes, and the
// launch. E experts with N rows each; offsets NULL for one expert with every row of X.
awq_status fused_gemm(const void* X, int64_t T, const int32_t* offsets, int64_t E,
                      const uint32_t* qweight, const awq_f16* scales, const uint8_t* zeros,
                      int64_t N, int64_t K, int bits, int group, const float* inv_s,
                      const awq_f16* bias, int act, const awq_f16* mul, const awq_f16* residual,
                      unsigned flags, awq_f16* Y, void* workspace, size_t ws_bytes,
                      cudaStream_t st) {
  if (bad_dim(T) || bad_dim(N) || bad_dim(K) || K == 0) return AWQ_ERR_INVALID_ARG;
  if (group != awq::kGroup || K % awq::kGroup != 0) return AWQ_ERR_INVALID_ARG;
  if (bits != 4 && bits != 3) return AWQ_ERR_INVALID_ARG;
  if (act < awq::kActNone || act > awq::kActGeluTanh) return AWQ_ERR_INVALID_ARG;
  if ((flags & ~static_cast<unsigned>(AWQ_GEMM_WEIGHTS_READY | AWQ_GEMM_BF16)) != 0)
    return AWQ_ERR_INVALID_ARG;
  if (T == 0 || N == 0) return AWQ_OK;
  if (!X || !qweight || !scales || !zeros || !Y) return AWQ_ERR_INVALID_ARG;
  if (!aligned16(X) || !aligned16(qweight) || !aligned16(scales) || !aligned16(zeros) ||
      !aligned16(Y) || bad_ptr16(inv_s) || bad_ptr16(bias) || bad_ptr16(mul) ||
      bad_ptr16(residual))
    return AWQ_ERR_INVALID_ARG;
  // TMA coordinates (weight rows, scale rows) and indices of scales are 32-bit
  if (E * N > kMaxDim || E * (K / awq::kGroup) > kMaxDim / N) return AWQ_ERR_INVALID_ARG;
  const bool bf16 = (flags & AWQ_GEMM_BF16) != 0;
  const awq::FusedEpi epi{bias, mul, residual, act};
  const FusedPlan plan = fused_plan(T, E, N, K, offsets != nullptr, inv_s != nullptr, bf16);
  if (plan.workspace > 0 && (!workspace || ws_bytes < plan.workspace || !aligned16(workspace)))
    return AWQ_ERR_WORKSPACE;
  if (plan.kind == FusedPlan::kDecode)
    return launch_gemv_stream<true>(X, T, qweight, reinterpret_cast<const __half*>(scales), zeros,
                                    N, K, bits, inv_s, flags, Y, st, epi);
  if (plan.kind == FusedPlan::kStream) {
    awq::StreamArgs a{};
    a.N = N;
    a.K = K;
    a.T = static_cast<int>(T);
    a.E = static_cast<int>(E);
    a.offsets = offsets;
    a.scales = reinterpret_cast<const __half*>(scales);
    a.zeros = zeros;
    a.epi = epi;
    a.Y = Y;
    if (bf16)
      return bits == 3 ? launch_stream_plan<true, 3>(plan, X, inv_s, qweight, a, workspace, st)
                       : launch_stream_plan<true, 4>(plan, X, inv_s, qweight, a, workspace, st);
    return bits == 3 ? launch_stream_plan<false, 3>(plan, X, inv_s, qweight, a, workspace, st)
                     : launch_stream_plan<false, 4>(plan, X, inv_s, qweight, a, workspace, st);
  }
  awq::FusedArgs args{};
  args.M = T;
  args.N = N;
  args.K = K;
  args.scales = reinterpret_cast<const __half*>(scales);
  args.zeros = zeros;
  args.Y = Y;
  args.k_splits = plan.splits;
  args.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + plan.prepared);
  args.inv_s = inv_s;
  args.offsets = offsets;
  args.E = static_cast<int>(E);
  args.epi = epi;
  awq_status r;
  // (behind the preparation the weights of any call are there: see the kernel)
  int early = offsets == nullptr && (flags & AWQ_GEMM_WEIGHTS_READY) != 0;
  if (bf16) {
    r = launch_pdl(awq::prepare_rows_kernel<true, false>, dim3(static_cast<unsigned>(T)),
                   awq::kPrepThreads, 0, st, static_cast<const uint4*>(X), static_cast<int>(T), K,
                   inv_s, offsets, static_cast<int>(E), 1, 0, 0, static_cast<uint8_t*>(workspace));
    if (r != AWQ_OK) return r;
    X = workspace;
    args.factors = reinterpret_cast<const float*>(static_cast<uint8_t*>(workspace) + T * K * 2);
    args.inv_s = nullptr;
    early = 1;
  }
  if (bf16)
    r = bits == 3 ? launch_tensor<true, 3>(X, qweight, args, early, st)
                  : launch_tensor<true, 4>(X, qweight, args, early, st);
  else if (inv_s != nullptr)
    r = bits == 3 ? launch_tensor<false, 3, true>(X, qweight, args, early, st)
                  : launch_tensor<false, 4, true>(X, qweight, args, early, st);
  else
    r = bits == 3 ? launch_tensor<false, 3>(X, qweight, args, early, st)
                  : launch_tensor<false, 4>(X, qweight, args, early, st);
  if (r != AWQ_OK || plan.splits == 1) return r;
  const dim3 grid(static_cast<unsigned>((N + 255) / 256), static_cast<unsigned>(T));
  return bf16 ? launch_pdl(awq::splitk_fused_kernel<true>, grid, 256, 0, st, args)
              : launch_pdl(awq::splitk_fused_kernel<false>, grid, 256, 0, st, args);
}

template <int BN, bool kStack>
awq_status launch_gated_tiles(const void* X, const void* gate, const void* up, awq::FusedArgs a,
                        cudaStream_t st) {
  using L = awq::GgLayout<BN, kStack>;
  static std::atomic<bool> attr_set[kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return AWQ_ERR_CUDA;
  auto kern = awq::gated_grouped_kernel<BN, kStack>;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem) !=
        cudaSuccess)
      return AWQ_ERR_CUDA;
    attr_set[dev].store(true, std::memory_order_release);
  }
  CUtensorMap tx, tg, tu;
  if (!make_tmap_2d(&tx, X, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, a.M, a.K, BN, awq::kTcBK, true) ||
      !make_tmap_2d(&tg, gate, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, a.E * a.N, a.K, L::kRows,
                    awq::kTcBK, true) ||
      !make_tmap_2d(&tu, up, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, a.E * a.N, a.K, L::kRows,
                    awq::kTcBK, true))
    return AWQ_ERR_CUDA;
  a.row_tiles = static_cast<int>((a.N + L::kRows - 1) / L::kRows);
  const int64_t units = a.row_tiles * (a.M / BN + (a.M < a.E ? a.M : a.E));
  if (units > kMaxDim) return AWQ_ERR_INVALID_ARG;   // the kernel counts them in 32 bits
  const int64_t sms = num_sms();
  return launch_pdl(kern, dim3(static_cast<unsigned>(units < sms ? units : sms)), awq::kGgThreads,
                    L::kSmem, st, tx, tg, tu, a);
}

// Tiles for experts of few rows: 128 rows of both weights, or 64 where those take clearly fewer
// rounds of the CTAs, counted with one token tile an expert (us in tiles of 128 and of 64, rows
// unevenly spread: 1003 rows over 16 experts of [1536, 2048] 44 and 39, 2400 rows 62 and 52, 634 over
// 24 of [334, 1536] 16.4 and 12.6, 572 over 83 of [444, 3328] 88 and 78; but 1200 over 8 of
// [4096, 4096] 115 and 129, 27 over 14 of [2456, 512] 12.2 and 16.2, 4241 over 38 of [1315, 5888]
// 252 and 293, where the rounds only double and X is read twice as often). A twelfth more token
// tiles in the count, for experts that need a second one, chose the slower side in 20 of the 23 drawn
// shapes where it made a difference, by up to a third.
template <int BN>
awq_status launch_gated(const void* X, const void* gate, const void* up, const awq::FusedArgs& a,
                        cudaStream_t st) {
  const int64_t sms = num_sms();
  const int64_t active = a.M < a.E ? a.M : a.E;
  const int64_t whole = ((a.N + 127) / 128 * active + sms - 1) / sms;
  const int64_t half = ((a.N + 63) / 64 * active + sms - 1) / sms;
  return 10 * half < 16 * whole ? launch_gated_tiles<BN, true>(X, gate, up, a, st)
                                : launch_gated_tiles<BN, false>(X, gate, up, a, st);
}

bool bad_groups(int64_t E, const int32_t* offsets) {
  return E < 1 || E > awq::kMaxExperts || offsets == nullptr ||
         (reinterpret_cast<uintptr_t>(offsets) & 3u) != 0;
}
}  // namespace

extern "C" {

size_t awq_gemm_epilogue_workspace_size(int64_t M, int64_t N, int64_t K, int bits,
                                        int with_inv_s, unsigned flags) {
  if (M <= 0 || K <= 0 || N <= 0) return 0;
  (void)bits;
  return fused_plan(M, 1, N, K, false, with_inv_s != 0, (flags & AWQ_GEMM_BF16) != 0).workspace;
}

awq_status awq_gemm_w4a16_epilogue(const awq_f16* X, int64_t M, const uint32_t* qweight,
                                   const awq_f16* scales, const uint8_t* zeros, int64_t N,
                                   int64_t K, int bits, int group, const float* inv_s,
                                   const awq_f16* bias, int act, const awq_f16* mul,
                                   const awq_f16* residual, unsigned flags, awq_f16* Y,
                                   void* workspace, size_t ws_bytes, void* stream) {
  return fused_gemm(X, M, nullptr, 1, qweight, scales, zeros, N, K, bits, group, inv_s, bias, act,
                    mul, residual, flags, Y, workspace, ws_bytes,
                    static_cast<cudaStream_t>(stream));
}

size_t awq_gemm_grouped_workspace_size(int64_t T, int64_t E, int64_t N, int64_t K, int bits,
                                       int with_inv_s, unsigned flags) {
  if (T <= 0 || E <= 0 || K <= 0 || N <= 0) return 0;
  (void)bits;
  if (E > awq::kMaxExperts) return 0;
  return fused_plan(T, E, N, K, true, with_inv_s != 0, (flags & AWQ_GEMM_BF16) != 0).workspace;
}

awq_status awq_gemm_w4a16_grouped(const awq_f16* X, int64_t T, const int32_t* offsets, int64_t E,
                                  const uint32_t* qweight, const awq_f16* scales,
                                  const uint8_t* zeros, int64_t N, int64_t K, int bits, int group,
                                  const float* inv_s, const awq_f16* bias, int act,
                                  const awq_f16* mul, const awq_f16* residual, unsigned flags,
                                  awq_f16* Y, void* workspace, size_t ws_bytes, void* stream) {
  if (bad_groups(E, offsets)) return AWQ_ERR_INVALID_ARG;
  return fused_gemm(X, T, offsets, E, qweight, scales, zeros, N, K, bits, group, inv_s, bias, act,
                    mul, residual, flags, Y, workspace, ws_bytes,
                    static_cast<cudaStream_t>(stream));
}

awq_status awq_silu_mul_gemm_grouped(const awq_f16* X, int64_t T, const int32_t* offsets,
                                     int64_t E, const awq_f16* W_gate, const awq_f16* W_up,
                                     int64_t I, int64_t K, awq_f16* H, void* stream) {
  if (bad_groups(E, offsets)) return AWQ_ERR_INVALID_ARG;
  if (bad_dim(T) || bad_dim(I) || bad_dim(K) || K == 0) return AWQ_ERR_INVALID_ARG;
  if (K % awq::kGroup != 0) return AWQ_ERR_INVALID_ARG;
  if (T == 0 || I == 0) return AWQ_OK;
  if (!X || !W_gate || !W_up || !H) return AWQ_ERR_INVALID_ARG;
  if (!aligned16(X) || !aligned16(W_gate) || !aligned16(W_up) || !aligned16(H))
    return AWQ_ERR_INVALID_ARG;
  if (E * I > kMaxDim) return AWQ_ERR_INVALID_ARG;
  awq::FusedArgs args{};
  args.M = T;
  args.N = I;
  args.K = K;
  args.Y = H;
  args.k_splits = 1;
  args.offsets = offsets;
  args.E = static_cast<int>(E);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // the token tile: the smallest that holds an expert of half as many rows again as the mean
  const int64_t rows = (T + E - 1) / E * 3 / 2;
  if (rows <= 64) return launch_gated<64>(X, W_gate, W_up, args, st);
  if (rows <= 128) return launch_gated<128>(X, W_gate, W_up, args, st);
  if (rows <= 256) return launch_gated<256>(X, W_gate, W_up, args, st);
  // Many rows: tiles of 64, whose one accumulator leaves room for a second one, so that epilogues
  // overlap (us in tiles of 128 and of 64, calls run for 0.3 s each in turn: 16384 rows over 8 experts
  // of [14336, 4096] 3720 and 3587, 6144 rows 1673 and 1473, 16384 rows of one [11008, 4096] 2547 and
  // 2427, 8192 over 8 of [14336, 1024] 678 and 461; the other way at the deepest K and many rows alone:
  // 65536 over 8 of [4096, 8192] 7630 and 7913, 16384 rows 2095 and 2080).
  return launch_gated_tiles<256, true>(X, W_gate, W_up, args, st);
}

// ------------------------------------------------------------------ act_stats of each expert
size_t awq_act_stats_grouped_workspace_size(int64_t T, int64_t E, int64_t K) {
  if (T <= 0 || E <= 0 || K <= 0) return 0;
  return static_cast<size_t>(awq::grouped_stats_slices(T, K, num_sms()) + E) *
         static_cast<size_t>(K) * sizeof(double);
}

awq_status awq_act_stats_grouped(const awq_f16* X, int64_t T, const int32_t* offsets, int64_t E,
                                 int64_t K, float* s_x, void* workspace, size_t ws_bytes,
                                 void* stream) {
  if (bad_groups(E, offsets)) return AWQ_ERR_INVALID_ARG;
  if (bad_dim(T) || bad_dim(K)) return AWQ_ERR_INVALID_ARG;
  if (K == 0) return AWQ_OK;
  if (K % 8 != 0) return AWQ_ERR_INVALID_ARG;
  if (!s_x || !aligned16(s_x) || (T > 0 && (!X || !aligned16(X)))) return AWQ_ERR_INVALID_ARG;
  const size_t need = awq_act_stats_grouped_workspace_size(T, E, K);
  if (need > 0 && (!workspace || ws_bytes < need || !aligned16(workspace)))
    return AWQ_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  double* part = static_cast<double*>(workspace);
  const int64_t rows = T > 0 ? awq::grouped_stats_rows(T, K, num_sms()) : 1;
  if (T > 0) {
    const int64_t slices = awq::grouped_stats_slices(T, K, num_sms());
    dim3 g1(static_cast<unsigned>((K + awq::kStatsCols - 1) / awq::kStatsCols),
            static_cast<unsigned>(slices));
    const awq_status s = launch_pdl(awq::act_stats_grouped_partial_kernel, g1, 256, 0, st,
                                    reinterpret_cast<const __half*>(X), T, K, offsets,
                                    static_cast<int>(E), rows, part);
    if (s != AWQ_OK) return s;
  }
  dim3 g2(static_cast<unsigned>((K + 255) / 256), static_cast<unsigned>(E));
  return launch_pdl(awq::act_stats_grouped_finish_kernel, g2, 256, 0, st,
                    static_cast<const double*>(part), T, K, offsets, rows, s_x);
}

}  // extern "C"
