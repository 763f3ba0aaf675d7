// lm_ops.cu -- C entry points of the 8-bit operators of a token model (vocoder_lm_* in
// include/vocoder.h): argument checks, choice of tiles and splits, launches.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>
#include <new>
#include <string>

#include "vocoder.h"
#include "lm_attention.cuh"
#include "lm_cache.cuh"
#include "lm_linear.cuh"
#include "lm_prompt.cuh"
#include "lm_rows.cuh"

#define VOC_API extern "C" __attribute__((visibility("default")))

namespace voc {
std::string &last_error_slot();  // vocoder.cu: the thread's error without a context
}

namespace {

constexpr long long kWaitBudget = 4000000000LL;  // cycles (~2 s) before a wait gives up
constexpr int kMaxDevices = 64;

// Set by a kernel that gave up a wait; read and cleared by calls with VOC_FLAG_SYNC.
__device__ int g_timeout;

voc_status fail(voc_status st, const char *msg) noexcept {
  try {
    voc::last_error_slot() = msg;
  } catch (...) {
  }
  return st;
}
voc_status cuda_fail(cudaError_t e, const char *what) noexcept {
  try {
    voc::last_error_slot() = std::string(what) + ": " + cudaGetErrorString(e);
  } catch (...) {
  }
  return e == cudaErrorMemoryAllocation ? VOC_OOM : VOC_CUDA_ERROR;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

struct Device {
  std::once_flag once;
  cudaError_t err = cudaSuccess;
  int sms = 0;
  int *timeout = nullptr;
  int clusters[9] = {};  // clusters of 1..8 CTAs of the split-K product that run at once
};
Device g_devices[kMaxDevices];

template <typename K>
void allow_smem(cudaError_t &e, K kernel, size_t bytes) {
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(bytes));
}
constexpr size_t kLinSmem = 220 * 1024;       // one CTA of the split-K product on an SM
constexpr size_t kLinSmemTwo = 108 * 1024;    // two

// Clusters of `size` CTAs (along z) of `kernel` that run at once.
template <typename K>
cudaError_t count_clusters(int *out, K kernel, int threads, size_t smem, int size) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1, 1, size);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = size;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaOccupancyMaxActiveClusters(out, kernel, &cfg);
}

// The current device, set up on first use (shared-memory limits of the kernels, SM count).
voc_status device(Device **out) {
  int d = 0;
  cudaError_t e = cudaGetDevice(&d);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (d >= kMaxDevices) return fail(VOC_UNSUPPORTED, "lm: device index");
  Device &dev = g_devices[d];
  std::call_once(dev.once, [&] {
    using namespace voc;
    cudaError_t &er = dev.err;
    er = cudaDeviceGetAttribute(&dev.sms, cudaDevAttrMultiProcessorCount, d);
    void *t = nullptr;
    if (er == cudaSuccess) er = cudaGetSymbolAddress(&t, g_timeout);
    dev.timeout = static_cast<int *>(t);
    allow_smem(er, attn_rows_kernel<__half, 64, 1>, attn_smem<64, 1>());
    allow_smem(er, attn_rows_kernel<__half, 64, 2>, attn_smem<64, 2>());
    allow_smem(er, attn_rows_kernel<__half, 128, 1>, attn_smem<128, 1>());
    allow_smem(er, attn_rows_kernel<__half, 128, 2>, attn_smem<128, 2>());
    allow_smem(er, attn_rows_kernel<__nv_bfloat16, 64, 1>, attn_smem<64, 1>());
    allow_smem(er, attn_rows_kernel<__nv_bfloat16, 64, 2>, attn_smem<64, 2>());
    allow_smem(er, attn_rows_kernel<__nv_bfloat16, 128, 1>, attn_smem<128, 1>());
    allow_smem(er, attn_rows_kernel<__nv_bfloat16, 128, 2>, attn_smem<128, 2>());
    allow_smem(er, attn_prompt_kernel<__half, 64>, PromptSmem<64>::kBytes);
    allow_smem(er, attn_prompt_kernel<__half, 128>, PromptSmem<128>::kBytes);
    allow_smem(er, attn_prompt_kernel<__nv_bfloat16, 64>, PromptSmem<64>::kBytes);
    allow_smem(er, attn_prompt_kernel<__nv_bfloat16, 128>, PromptSmem<128>::kBytes);
    allow_smem(er, linear_many_kernel<float>, kManySmem);
    allow_smem(er, linear_many_kernel<__half>, kManySmem);
    allow_smem(er, linear_many_kernel<__nv_bfloat16>, kManySmem);
    allow_smem(er, linear_few_kernel<float>, kLinSmem);
    allow_smem(er, linear_few_kernel<__half>, kLinSmem);
    allow_smem(er, linear_few_kernel<__nv_bfloat16>, kLinSmem);
    for (int size = 1; size <= 8 && er == cudaSuccess; ++size)
      er = count_clusters(&dev.clusters[size], linear_few_kernel<__nv_bfloat16>, kLinThreads,
                          kLinSmem, size);
  });
  if (dev.err != cudaSuccess) return cuda_fail(dev.err, "lm: device set-up");
  *out = &dev;
  return VOC_OK;
}

// Launch with programmatic stream serialization (see pdl_wait), in clusters of `cluster` CTAs
// along z where that is above 1.
template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, int cluster,
                   voc_stream_t stream, const Args &...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = cluster;
    cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// With VOC_FLAG_SYNC: wait for the stream and report a kernel that gave up a wait.
voc_status finish(const Device &dev, voc_stream_t stream, unsigned flags) {
  if (!(flags & VOC_FLAG_SYNC)) return VOC_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int t = 0;
  cudaError_t e = cudaMemcpyAsync(&t, dev.timeout, sizeof t, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_fail(e, "lm: synchronise");
  if (t) {
    e = cudaMemsetAsync(dev.timeout, 0, sizeof t, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return cuda_fail(e, "lm: synchronise");
    return fail(VOC_DEVICE_TIMEOUT, "lm: a kernel gave up a wait");
  }
  return VOC_OK;
}

bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool known_flags(unsigned f) { return (f & ~static_cast<unsigned>(VOC_FLAG_SYNC)) == 0; }

// Threads of a row: as few as hold it in registers, and more of them while there are too few rows
// to fill the GPU (up to a chunk of values per thread).  Measured, without / with more: 8 x 1024 2.8 /
// 2.2 us, 256 x 4096 3.6 / 3.1 us.
int row_threads(int sms, long long rows, int d, int chunk) {
  int t = 32;
  while (t * voc::kRowValues < d) t *= 2;
  while (t < voc::kRowThreads && t * chunk < d && rows * t < sms * 256ll) t *= 2;
  return t;
}

template <typename T, int MODE, int VB, int CH, bool ANY>
cudaError_t launch_rows_ch(int tpr, const voc::LmRowsArgs &a, voc_stream_t stream) {
  const int threads = std::max(128, tpr);
  const long long per = threads / tpr;
  return launch(voc::rows_kernel<T, MODE, VB, CH, ANY>,
                dim3(static_cast<unsigned>((a.rows + per - 1) / per)), dim3(threads), 0, 1, stream,
                a, tpr);
}

// As many vectors per thread as the row needs, up to kRowValues values, in steps of an eighth of these
// (a vector where that is more; vectors that hold nothing cost instructions all the same: a row of 4100
// takes 19.3 us with 5 vectors of 4 a thread, 20.9 with 6).  `d`: values that the vectors have to cover.
template <typename T, int MODE, int VB, bool ANY, int CH>
cudaError_t launch_rows_need(int need, int tpr, const voc::LmRowsArgs &a, voc_stream_t stream) {
  constexpr int step = std::max(1, voc::kRowValues / (VB / static_cast<int>(sizeof(T))) / 8);
  if constexpr (CH > step)
    if (need <= CH - step)
      return launch_rows_need<T, MODE, VB, ANY, CH - step>(need, tpr, a, stream);
  return launch_rows_ch<T, MODE, VB, CH, ANY>(tpr, a, stream);
}
template <typename T, int MODE, int VB, bool ANY>
cudaError_t launch_rows_vec(int sms, int d, const voc::LmRowsArgs &a, voc_stream_t stream) {
  constexpr int n = VB / static_cast<int>(sizeof(T)), most = voc::kRowValues / n;
  const int tpr = row_threads(sms, a.rows, d, n);
  const int need = (d + n * tpr - 1) / (n * tpr);
  return launch_rows_need<T, MODE, VB, ANY, most>(need, tpr, a, stream);
}

// The widest access that the width, the strides and the buffers allow in every row; below 8 bytes each
// row and buffer by its own.
template <typename T, int MODE>
cudaError_t launch_rows(int sms, const voc::LmRowsArgs &a, voc_stream_t stream) {
  constexpr int most = voc::kRowThreads * voc::kRowValues;
  constexpr int lead = 16 / static_cast<int>(sizeof(T)) - 1;  // places before a row's first value
  auto fits = [&](size_t vb) {  // rows start on vb bytes, codes on as many values
    const long long n = static_cast<long long>(vb / sizeof(T));
    return a.d <= most && a.d % n == 0 && a.ldx % n == 0 && (!a.res || a.ldr % n == 0) &&
           (!a.sum || a.lds % n == 0) && a.ldo % n == 0 && aligned(a.x, vb) &&
           aligned(a.res, vb) && aligned(a.sum, vb) && aligned(a.w, vb) && aligned(a.out, n);
  };
  if (fits(16)) return launch_rows_vec<T, MODE, 16, false>(sms, a.d, a, stream);
  if (fits(8)) return launch_rows_vec<T, MODE, 8, false>(sms, a.d, a, stream);
  if (a.d + lead <= most) return launch_rows_vec<T, MODE, 16, true>(sms, a.d + lead, a, stream);
  return launch(voc::rows_any_kernel<T, MODE>, dim3(static_cast<unsigned>(a.rows)),
                dim3(voc::kAnyThreads), 0, 1, stream, a);
}

template <int MODE>
cudaError_t launch_rows(int sms, int dtype, const voc::LmRowsArgs &a, voc_stream_t stream) {
  if (dtype == VOC_LM_F32) return launch_rows<float, MODE>(sms, a, stream);
  if (dtype == VOC_LM_F16) return launch_rows<__half, MODE>(sms, a, stream);
  return launch_rows<__nv_bfloat16, MODE>(sms, a, stream);
}

}  // namespace

VOC_API voc_status vocoder_lm_rows_fp8(const void *x, long long ldx, const void *residual,
                                       long long ldr, const void *weight, int dtype, int mode,
                                       long long rows, int d, float eps, void *sum_out,
                                       long long lds, void *out8, long long ldo, float *scale,
                                       voc_stream_t stream, unsigned flags) {
  if (dtype != VOC_LM_BF16 && dtype != VOC_LM_F16 && dtype != VOC_LM_F32)
    return fail(VOC_INVALID_ARG, "rows: dtype");
  if (mode != VOC_LM_RMS && mode != VOC_LM_NONE && mode != VOC_LM_GATED)
    return fail(VOC_INVALID_ARG, "rows: mode");
  if (rows < 0 || rows > 0x7fffffffll || d < 1 || d > (1 << 24))
    return fail(VOC_INVALID_ARG, "rows: sizes");
  if (!known_flags(flags)) return fail(VOC_INVALID_ARG, "rows: flags");
  if (mode == VOC_LM_RMS && !weight) return fail(VOC_INVALID_ARG, "rows: weight is NULL");
  if (mode != VOC_LM_RMS && weight) return fail(VOC_INVALID_ARG, "rows: weight without RMS");
  if (mode == VOC_LM_RMS && !(eps >= 0.f && std::isfinite(eps)))
    return fail(VOC_INVALID_ARG, "rows: eps");
  if (mode == VOC_LM_GATED && residual)
    return fail(VOC_INVALID_ARG, "rows: residual with a gated product");
  if ((sum_out != nullptr) && !residual)
    return fail(VOC_INVALID_ARG, "rows: sum_out without residual");
  const long long width = mode == VOC_LM_GATED ? 2ll * d : d;
  if (ldx < width || ldo < d || (residual && ldr < d) || (sum_out && lds < d))
    return fail(VOC_INVALID_ARG, "rows: a row stride is below the width");
  if (rows > 0 && (!x || !out8 || !scale)) return fail(VOC_INVALID_ARG, "rows: NULL buffer");
  const size_t e = dtype == VOC_LM_F32 ? 4 : 2;
  if (!aligned(x, e) || !aligned(residual, e) || !aligned(weight, e) || !aligned(sum_out, e) ||
      !aligned(scale, 4))
    return fail(VOC_INVALID_ARG, "rows: a buffer is not aligned to its type");
  Device *dev;
  if (voc_status st = device(&dev); st != VOC_OK) return st;
  if (rows == 0) return finish(*dev, stream, flags);
  voc::LmRowsArgs a{x, residual, weight, sum_out, static_cast<uint8_t *>(out8), scale,
                    rows, ldx, ldr, lds, ldo, d, eps};
  cudaError_t err;
  if (mode == VOC_LM_RMS)
    err = launch_rows<voc::kRowsRms>(dev->sms, dtype, a, stream);
  else if (mode == VOC_LM_NONE)
    err = launch_rows<voc::kRowsNone>(dev->sms, dtype, a, stream);
  else
    err = launch_rows<voc::kRowsGated>(dev->sms, dtype, a, stream);
  if (err != cudaSuccess) return cuda_fail(err, "launch rows");
  return finish(*dev, stream, flags);
}

// ------------------------------------------------------------------ product
namespace {

// [rows][k] bytes with row stride ld, read in boxes of 128 bytes x `box` rows, 128-byte swizzle;
// what lies outside reads as 0.
voc_status encode_rows(CUtensorMap *map, const void *base, long long rows, long long k,
                       long long ld, int box) {
  auto enc = encode_fn();
  if (!enc) return fail(VOC_CUDA_ERROR, "linear: cuTensorMapEncodeTiled entry point unavailable");
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld)};
  const cuuint32_t b[2] = {128u, static_cast<cuuint32_t>(box)};
  const cuuint32_t es[2] = {1u, 1u};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides,
                   b, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(VOC_CUDA_ERROR, "linear: cuTensorMapEncodeTiled failed");
  return VOC_OK;
}

// Whether a product runs on 256 x 256 tiles of CTA pairs: above 128 tokens and with more than 32 such
// tiles.  Measured (tokens x K x N, us, pairs / split K), 48 tiles: 144 x 4096 x 12288 16.6 / 17.2, 256 of
// them 16.8 / 22.6, 700 x 4096 x 4096 15.1 / 19.3, 2000 x 1024 x 1536 8.1 / 10.6; 40: 1280 x 8192 x 2048
// 23.5 / 32.5; 32: 300 x 4096 x 4096 14.5 / 11.6, 512 14.6 / 14.2, 1000 x 8192 x 2048 23.0 / 20.0, 144 x
// 1024 x 8192 7.7 / 7.0, but 256 of them 7.9 / 9.7; 24: 700 x 8192 x 2048 22.9 / 18.6, but 1000 x 1024 x
// 1536 7.6 / 9.1; 16: 256 x 4096 x 4096 14.2 / 11.3.  (With few chunks of K the pairs win from about 18
// tiles on.)
bool many_tokens(int M, int N) {
  const long long jobs = static_cast<long long>((M + voc::kManyTile - 1) / voc::kManyTile) *
                         ((N + voc::kManyTile - 1) / voc::kManyTile);
  return M > 128 && jobs > 32;
}

template <typename T>
cudaError_t launch_many(int sms, const CUtensorMap &xm, const CUtensorMap &wm,
                        const voc::LmLinearArgs &a, voc_stream_t stream) {
  const long long jobs = static_cast<long long>((a.M + voc::kManyTile - 1) / voc::kManyTile) *
                         ((a.N + voc::kManyTile - 1) / voc::kManyTile);
  const unsigned pairs = static_cast<unsigned>(std::min<long long>(sms / 2, jobs));
  return launch(voc::linear_many_kernel<T>, dim3(2 * pairs), dim3(voc::kManyThreads),
                voc::kManySmem, 1, stream, xm, wm, a);
}

template <typename T>
cudaError_t launch_few(const CUtensorMap &xm, const CUtensorMap &wm, const voc::LmLinearArgs &a,
                       int split, size_t smem, voc_stream_t stream) {
  const dim3 grid((a.N + voc::kLinRows - 1) / voc::kLinRows, (a.M + a.nt - 1) / a.nt, split);
  return launch(voc::linear_few_kernel<T>, grid, dim3(voc::kLinThreads), smem, split, stream,
                xm, wm, a);
}

}  // namespace

VOC_API voc_status vocoder_lm_linear_fp8(const void *x8, long long ldx, const float *x_scale,
                                         const void *w8, long long ldw, const float *w_scale,
                                         const float *bias, int M, int N, int K, void *out,
                                         long long ldo, int out_dtype, voc_stream_t stream,
                                         unsigned flags) {
  if (out_dtype != VOC_LM_BF16 && out_dtype != VOC_LM_F16 && out_dtype != VOC_LM_F32)
    return fail(VOC_INVALID_ARG, "linear: out_dtype");
  if (M < 0 || N < 0 || K < 1 || M > (1 << 28) || N > (1 << 28) || K > (1 << 28))
    return fail(VOC_INVALID_ARG, "linear: sizes");
  if (!known_flags(flags)) return fail(VOC_INVALID_ARG, "linear: flags");
  if (ldx < K || ldw < K || ldo < N)
    return fail(VOC_INVALID_ARG, "linear: a row stride is below the width");
  if (ldx % 16 || ldw % 16)
    return fail(VOC_INVALID_ARG, "linear: row strides of x8 and w8 must be multiples of 16");
  if (M > 0 && N > 0 && (!x8 || !w8 || !x_scale || !w_scale || !out))
    return fail(VOC_INVALID_ARG, "linear: NULL buffer");
  if (!aligned(x8, 16) || !aligned(w8, 16))
    return fail(VOC_INVALID_ARG, "linear: x8 and w8 must be 16-byte aligned");
  if (!aligned(x_scale, 4) || !aligned(w_scale, 4) || !aligned(bias, 4) ||
      !aligned(out, out_dtype == VOC_LM_F32 ? 4 : 2))
    return fail(VOC_INVALID_ARG, "linear: a buffer is not aligned to its type");
  Device *dev;
  if (voc_status st = device(&dev); st != VOC_OK) return st;
  if (M == 0 || N == 0) return finish(*dev, stream, flags);
  voc::LmLinearArgs a{};
  a.xs = x_scale, a.ws = w_scale, a.bias = bias, a.out = out, a.ldo = ldo;
  a.M = M, a.N = N, a.K = K;
  a.budget = kWaitBudget;
  a.timeout = dev->timeout;
  a.chunks = (K + voc::kLinK - 1) / voc::kLinK;
  CUtensorMap xm, wm;
  cudaError_t e;
  if (many_tokens(M, N)) {
    if (voc_status st = encode_rows(&xm, x8, M, K, ldx, 128); st != VOC_OK) return st;
    if (voc_status st = encode_rows(&wm, w8, N, K, ldw, 128); st != VOC_OK) return st;
    if (out_dtype == VOC_LM_F32)
      e = launch_many<float>(dev->sms, xm, wm, a, stream);
    else if (out_dtype == VOC_LM_F16)
      e = launch_many<__half>(dev->sms, xm, wm, a, stream);
    else
      e = launch_many<__nv_bfloat16>(dev->sms, xm, wm, a, stream);
    if (e != cudaSuccess) return cuda_fail(e, "launch linear");
    return finish(*dev, stream, flags);
  }
  // Equal tiles of up to 256 tokens (few: up to 32 of 256 x 256), down to 32 as long as all their
  // parts of K have SMs: a tile's way out grows with its tokens.  Measured (tokens x K x N, us, as large
  // as they go / so): 444 x 592 x 65 8.9 / 4.3, 172 x 1536 x 694 8.0 / 5.7, 500 x 4096 x 256 10.5 / 6.5.
  const int n_tiles = (N + voc::kLinRows - 1) / voc::kLinRows;
  const int most = std::max(1, std::min(8, a.chunks / 2));  // parts of K
  const int m_tiles =
      std::max((M + 255) / 256, std::min((M + 31) / 32, dev->sms / most / n_tiles));
  a.nt = ((M + m_tiles - 1) / m_tiles + 15) / 16 * 16;
  a.tmem_cols = 32;
  while (a.tmem_cols < a.nt) a.tmem_cols *= 2;
  // Up to 64 tokens leave room for two CTAs on an SM (measured, one / two, N x K = 12288 x 4096: 33
  // tokens 13.8 / 12.5 us, 64 tokens 14.5 / 13.5; 4096 x 4096: 16 tokens 5.9 / 5.7, 64 tokens 6.8 /
  // 7.8).  K is split over up to 8 CTAs as long as all clusters run at once, and each keeps 4 stages of
  // K once every SM has a CTA.  Measured at 33 tokens, 12288 x 4096 (96 tiles): split 1 14.7, 2 12.5,
  // 3 12.8 (does not fit), 4 17.2 us; 8 tokens, 2048 x 8192 (16 tiles): split 1 21.9, 4 7.9, 8 5.9 us.
  const int stage = (voc::kLinRows + a.nt) * voc::kLinK;
  const int tiles = n_tiles * ((M + a.nt - 1) / a.nt);
  const int per_sm = a.nt <= 64 ? 2 : 1;
  const size_t smem = per_sm == 2 ? kLinSmemTwo : kLinSmem;
  a.stages = std::min<int>(12, static_cast<int>((smem - 1024) / stage));
  int split = most;
  while (split > 1 && (per_sm * dev->clusters[split] < tiles ||
                       (tiles * split > dev->sms && a.chunks / split < 4)))
    --split;
  if (voc_status st = encode_rows(&xm, x8, M, K, ldx, a.nt); st != VOC_OK) return st;
  if (voc_status st = encode_rows(&wm, w8, N, K, ldw, voc::kLinRows); st != VOC_OK) return st;
  if (out_dtype == VOC_LM_F32)
    e = launch_few<float>(xm, wm, a, split, smem, stream);
  else if (out_dtype == VOC_LM_F16)
    e = launch_few<__half>(xm, wm, a, split, smem, stream);
  else
    e = launch_few<__nv_bfloat16>(xm, wm, a, split, smem, stream);
  if (e != cudaSuccess) return cuda_fail(e, "launch linear");
  return finish(*dev, stream, flags);
}

// ------------------------------------------------------------------ cache and attention
namespace {

// What append and attention ask of the cache and of the batch.
voc_status check_cache(const void *kc, const void *vc, const float *ks, const float *vs,
                       int n_pages, int kv_heads, int head_dim, int dtype, const int *table,
                       long long ldt, int table_cols, const int *lens, const int *cu, int n_seq,
                       int n_tokens, int max_q) {
  if (dtype != VOC_LM_BF16 && dtype != VOC_LM_F16) return fail(VOC_INVALID_ARG, "cache: dtype");
  if (head_dim != 64 && head_dim != 128)
    return fail(VOC_UNSUPPORTED, "cache: head_dim must be 64 or 128");
  if (n_pages < 1 || kv_heads < 1 || kv_heads > 4096 || table_cols < 1 || ldt < table_cols)
    return fail(VOC_INVALID_ARG, "cache: sizes");
  if (n_seq < 0 || n_seq > 65535 || n_tokens < 0 || max_q < 0)
    return fail(VOC_INVALID_ARG, "cache: batch sizes");
  if (n_seq == 0 && n_tokens > 0) return fail(VOC_INVALID_ARG, "cache: tokens without sequences");
  if (n_seq > 0 && !cu && static_cast<long long>(n_seq) * max_q != n_tokens)
    return fail(VOC_INVALID_ARG, "cache: without cu_q every sequence has max_q tokens");
  if (max_q > n_tokens) return fail(VOC_INVALID_ARG, "cache: max_q above the number of tokens");
  if (!kc || !vc || !ks || !vs || (n_seq > 0 && (!table || !lens)))
    return fail(VOC_INVALID_ARG, "cache: NULL buffer");
  if (!aligned(kc, 16) || !aligned(vc, 16) || !aligned(ks, 4) || !aligned(vs, 4) ||
      !aligned(table, 4) || !aligned(lens, 4) || !aligned(cu, 4))
    return fail(VOC_INVALID_ARG, "cache: alignment");
  return VOC_OK;
}

template <typename T, int D>
cudaError_t launch_append(dim3 grid, const voc::LmAppendArgs &a, voc_stream_t stream) {
  const dim3 block(voc::AppendShape<D>::kThreads);
  if (a.max_q < voc::kBlockTokens)
    return launch(voc::append_kernel<T, D, true>, grid, block, 0, 1, stream, a);
  return launch(voc::append_kernel<T, D, false>, grid, block, 0, 1, stream, a);
}

}  // namespace

VOC_API voc_status vocoder_lm_kv_append(void *k_cache, void *v_cache, float *k_scale,
                                        float *v_scale, int n_pages, int kv_heads, int head_dim,
                                        const void *k, long long ldk, long long hsk, const void *v,
                                        long long ldv, long long hsv, int dtype,
                                        const int *page_table, long long ldt, int table_cols,
                                        const int *kv_lens, const int *cu_q, int n_seq,
                                        int n_tokens, int max_q, voc_stream_t stream,
                                        unsigned flags) {
  if (voc_status st = check_cache(k_cache, v_cache, k_scale, v_scale, n_pages, kv_heads, head_dim,
                                  dtype, page_table, ldt, table_cols, kv_lens, cu_q, n_seq,
                                  n_tokens, max_q);
      st != VOC_OK)
    return st;
  if (!known_flags(flags)) return fail(VOC_INVALID_ARG, "append: flags");
  if (n_tokens > 0 && (!k || !v)) return fail(VOC_INVALID_ARG, "append: NULL buffer");
  if (!aligned(k, 16) || !aligned(v, 16) || ldk % 8 || hsk % 8 || ldv % 8 || hsv % 8)
    return fail(VOC_INVALID_ARG, "append: k and v must be 16-byte aligned, strides multiples of 8");
  Device *dev;
  if (voc_status st = device(&dev); st != VOC_OK) return st;
  if (n_tokens == 0 || max_q == 0) return finish(*dev, stream, flags);
  voc::LmAppendArgs a{static_cast<uint8_t *>(k_cache), static_cast<uint8_t *>(v_cache), k_scale,
                      v_scale, k, v, ldk, hsk, ldv, hsv, page_table, kv_lens, cu_q, ldt, n_pages,
                      table_cols, kv_heads, n_seq, n_tokens, max_q, 0};
  // Blocks that max_q tokens can touch, for every sequence, or (prompts of different lengths) all that
  // n_tokens can touch.
  const long long each = (max_q - 1 + voc::kBlockTokens - 1) / voc::kBlockTokens + 1ll;
  const long long all = n_tokens / voc::kBlockTokens + 2ll * n_seq;
  dim3 grid(static_cast<unsigned>(max_q == 1 ? 1 : each), kv_heads, n_seq);
  if (max_q > 1 && n_seq <= voc::kFlatSeqs && all < each * n_seq) {
    a.flat = 1;
    grid = dim3(static_cast<unsigned>(all), kv_heads, 1);
  }
  cudaError_t e;
  if (dtype == VOC_LM_F16)
    e = head_dim == 64 ? launch_append<__half, 64>(grid, a, stream)
                       : launch_append<__half, 128>(grid, a, stream);
  else
    e = head_dim == 64 ? launch_append<__nv_bfloat16, 64>(grid, a, stream)
                       : launch_append<__nv_bfloat16, 128>(grid, a, stream);
  if (e != cudaSuccess) return cuda_fail(e, "launch append");
  return finish(*dev, stream, flags);
}

namespace {

// From kPromptRows rows (queries that share a key head) of a sequence the attention runs on tiles of
// 256 rows (prompt kernel), below on tiles of 8 or 16 (row kernel).  Measured, 8 sequences of 4000
// tokens, 8 heads of 128 channels (us, row / prompt kernel): 16 rows 27.2 / 40.0, 32 rows 40.0 / 41.3,
// 36 rows 51.2 / 41.4; 8 of 15504: 32 rows 105 / 126, 36 rows 145 / 127; one of 15504: 32 rows 25.6 /
// 25.8, 36 rows 29.9 / 26.0.
// Up to kShortBlocks blocks of keys the row kernel takes more rows too, as long as all its tiles run at
// once: the prompt kernel has about 10 us before its first and after its last product.  Measured, 256
// rows x 4 heads of 128 channels: 500 tokens 10.7 / 19.8, 1000 tokens 15.1 / 20.0; 64 rows x 16 heads:
// 1000 tokens 15.1 / 18.4, 2000 tokens (beyond the limit) 24.1 / 15.8; tiles for two turns, 300 rows x
// 8 heads, 4 queries each, 1000 tokens: 34.2 / 25.0.
constexpr int kPromptRows = 33;
constexpr int kShortBlocks = 16;
// A tile of the row kernel is a CTA's, unless equal shares of all units (kTileCost) spare the busiest
// CTA this many: a share that starts inside a tile and the join of its parts cost about as much.
// Measured (us, whole tiles / shares), 128 tiles of 64 channels: 16 blocks 8.0 / 11.6, 32 blocks 13.6 /
// 14.2, 63 blocks 24.0 / 19.6; 16 tiles: 16 blocks 7.9 / 8.0, 32 blocks 12.8 / 8.3; 256 tiles of 128
// channels: 16 blocks 15.9 / 23.1, 63 blocks 43.2 / 50.6; 16 sequences of 1 to 10012 tokens 65.4 / 22.2.
constexpr int kShareGain = 20;

struct AttnPlan {
  bool prompt = false;
  int tile = 8;       // rows of a tile of the row kernel
  int row_tiles = 0;  // of a sequence, at the kernel's own tile size
  int flat_tiles = 0; // prompt kernel: tiles of all sequences, or 0: row_tiles for each
  int splits = 1;     // prompt kernel: parts of the keys
  int ctas = 0;       // row kernel: CTAs that share the work; 0: a CTA has whole tiles
  size_t slots = 0;   // partial rows in the workspace
  size_t ws_bytes = 0;
};

// Partial rows in the workspace: a channel's sum each, the maximum and the sum of the weights.
size_t part_bytes(size_t slots, int head_dim) { return slots * (head_dim * sizeof(float) + 8); }

// Row kernel: a CTA per tile, or equal shares for two CTAs per SM (kShareGain).  Prompt kernel: long
// keys are split while there are fewer tiles than SMs, into parts of 4 blocks or more, and no more than
// 1.5 sqrt(blocks) of them, beyond which the parts' join costs what the shorter parts save.  Measured,
// 256 rows x 4 heads: 1100 tokens whole 28.1, 2 parts 25.4, 4 parts 20.9 us; 8000 tokens whole 123, 15
// parts 27.0, 17 26.2; 64 rows, 16000 tokens: 23 parts 21.9, 31 22.1; 8 chunks over a window of 250 (8
// blocks): whole 15.2, 2 parts 18.7.
// Its CTAs look for their tiles, which n_tokens bounds, so that sequences with few new tokens cost
// none (flat_tiles); splits grow as n_tokens falls, and parts are never more than one per SM.
AttnPlan plan_attention(int sms, int n_seq, long long n_tokens, int max_q, int heads, int kv_heads,
                        int head_dim, int max_kv, int window) {
  AttnPlan p;
  const long long rows = static_cast<long long>(heads / kv_heads) * max_q;
  const long long heads_all = static_cast<long long>(n_seq) * kv_heads;
  long long keys = max_kv;
  if (window > 0) keys = std::min<long long>(keys, static_cast<long long>(window) + max_q);
  const long long blocks = keys / voc::kBlockTokens + 1, slots = 2ll * sms;
  p.tile = rows <= 8 ? 8 : 16;
  const long long row_tiles = (rows + p.tile - 1) / p.tile, tiles = heads_all * row_tiles;
  const long long live =  // tiles that have rows, at most
      std::min(tiles, (n_tokens * (heads / kv_heads) / p.tile + n_seq) * kv_heads);
  const bool brief = rows >= kPromptRows && blocks <= kShortBlocks && live <= slots;
  p.prompt = rows >= kPromptRows && !brief;
  if (p.prompt) {
    p.row_tiles = static_cast<int>((rows + voc::kPrRows - 1) / voc::kPrRows);
    long long all = static_cast<long long>(n_seq) * p.row_tiles;
    if (n_seq <= voc::kFlatTiles) {
      all = std::min(all, n_tokens * (heads / kv_heads) / voc::kPrRows + n_seq);
      p.flat_tiles = static_cast<int>(all);
      const long long fits = blocks > kShortBlocks ? std::min(sms / (all * kv_heads), blocks / 4) : 1;
      while (p.splits < fits && 4ll * (p.splits + 1) * (p.splits + 1) <= 9 * blocks) ++p.splits;
      if (p.splits > 1)
        p.slots = static_cast<size_t>(all) * kv_heads * p.splits * voc::kPrRows;
    }
  } else {
    p.row_tiles = static_cast<int>(row_tiles);
    const long long units = tiles * (blocks + voc::kTileCost);
    const long long alone =  // the busiest CTA's units
        (tiles + slots - 1) / slots * (blocks + voc::kTileCost);
    const long long shared = std::max<long long>((units + slots - 1) / slots, voc::kShareMin);
    if (!brief && n_seq <= voc::kShareSeqs && alone >= shared + kShareGain && units < (1ll << 30)) {
      p.ctas = static_cast<int>(std::min(slots, (units + voc::kShareMin - 1) / voc::kShareMin));
      p.slots = 2ull * p.ctas * p.tile;
    }
  }
  p.ws_bytes = part_bytes(p.slots, head_dim);
  return p;
}

template <typename T, int D, int NT>
cudaError_t launch_rows_attention(const voc::LmAttnArgs &a, int row_tiles, voc_stream_t stream) {
  const dim3 grid = a.ctas ? dim3(a.ctas) : dim3(row_tiles, a.kv_heads, a.n_seq);
  cudaError_t e = launch(voc::attn_rows_kernel<T, D, NT>, grid, dim3(voc::kAttnThreads),
                         voc::attn_smem<D, NT>(), 1, stream, a);
  if (e != cudaSuccess || !a.ctas) return e;
  return launch(voc::attn_join_kernel<T, D, 8 * NT>,
                dim3(a.group * a.max_q, a.kv_heads, a.n_seq), dim3(D), 0, 1, stream, a);
}

template <typename T, int D>
cudaError_t launch_attention(const voc::LmAttnArgs &a, const AttnPlan &plan, voc_stream_t stream) {
  if (!plan.prompt)
    return plan.tile == 8 ? launch_rows_attention<T, D, 1>(a, plan.row_tiles, stream)
                          : launch_rows_attention<T, D, 2>(a, plan.row_tiles, stream);
  const dim3 grid = a.flat ? dim3(plan.flat_tiles, a.kv_heads, a.splits)
                           : dim3(plan.row_tiles, a.kv_heads, a.n_seq);
  cudaError_t e = launch(voc::attn_prompt_kernel<T, D>, grid, dim3(voc::kPrThreads),
                         voc::PromptSmem<D>::kBytes, 1, stream, a);
  if (e != cudaSuccess || a.splits == 1) return e;
  return launch(voc::attn_join_tiles_kernel<T, D>,
                dim3(plan.flat_tiles, a.kv_heads, voc::kPrRows / voc::kJoinRows),
                dim3(32 * voc::kJoinRows), 0, 1, stream, a);
}

}  // namespace

VOC_API size_t vocoder_lm_attention_ws_bytes(int n_seq, int max_q, int heads, int kv_heads,
                                             int head_dim, int max_kv, int window) {
  if (n_seq < 1 || max_q < 1 || kv_heads < 1 || heads < kv_heads || heads % kv_heads ||
      (head_dim != 64 && head_dim != 128) || max_kv < 0 || window < 0)
    return 0;
  Device *dev;
  if (device(&dev) != VOC_OK) return 0;
  // the number of tokens is not known here: the fewest, which have the most parts, stand for any
  const AttnPlan p =
      plan_attention(dev->sms, n_seq, max_q, max_q, heads, kv_heads, head_dim, max_kv, window);
  return p.splits > 1 ? part_bytes(static_cast<size_t>(dev->sms) * voc::kPrRows, head_dim) : p.ws_bytes;
}

VOC_API voc_status vocoder_lm_attention(
    const void *q, long long ldq, long long hsq, int dtype, int heads, const void *k_cache,
    const void *v_cache, const float *k_scale, const float *v_scale, int n_pages, int kv_heads,
    int head_dim, const int *page_table, long long ldt, int table_cols, const int *kv_lens,
    const int *cu_q, int n_seq, int n_tokens, int max_q, int max_kv, float softmax_scale,
    int causal, int window, void *out, long long ldo, long long hso, void *ws, size_t ws_bytes,
    voc_stream_t stream, unsigned flags) {
  if (voc_status st = check_cache(k_cache, v_cache, k_scale, v_scale, n_pages, kv_heads, head_dim,
                                  dtype, page_table, ldt, table_cols, kv_lens, cu_q, n_seq,
                                  n_tokens, max_q);
      st != VOC_OK)
    return st;
  if (!known_flags(flags)) return fail(VOC_INVALID_ARG, "attention: flags");
  if (heads < kv_heads || heads % kv_heads || heads > 65536)
    return fail(VOC_INVALID_ARG, "attention: heads must be a multiple of kv_heads");
  if (static_cast<long long>(heads / kv_heads) * max_q > (1ll << 30))
    return fail(VOC_UNSUPPORTED, "attention: too many rows of a key head");
  if (max_kv < 0 || window < 0 || (causal != 0 && causal != 1))
    return fail(VOC_INVALID_ARG, "attention: max_kv, window or causal");
  if (!std::isfinite(softmax_scale)) return fail(VOC_INVALID_ARG, "attention: softmax_scale");
  if (n_tokens > 0 && (!q || !out)) return fail(VOC_INVALID_ARG, "attention: NULL buffer");
  if (!aligned(q, 2) || !aligned(out, 2) || !aligned(ws, 16))
    return fail(VOC_INVALID_ARG, "attention: alignment");
  Device *dev;
  if (voc_status st = device(&dev); st != VOC_OK) return st;
  if (n_tokens == 0 || max_q == 0) return finish(*dev, stream, flags);
  AttnPlan plan =
      plan_attention(dev->sms, n_seq, n_tokens, max_q, heads, kv_heads, head_dim, max_kv, window);
  // lengths are on the device and may exceed max_kv: what the page table can hold bounds them
  if (static_cast<double>(n_seq) * kv_heads * plan.row_tiles * (table_cols + 1.0 + voc::kTileCost) >= 0x1p30)
    plan.ctas = 0;
  if (plan.ws_bytes && (!ws || ws_bytes < plan.ws_bytes))
    return fail(VOC_WORKSPACE_TOO_SMALL, "attention: workspace below vocoder_lm_attention_ws_bytes");
  voc::LmAttnArgs a{};
  a.q = q, a.out = out, a.ldq = ldq, a.hsq = hsq, a.ldo = ldo, a.hso = hso;
  a.kc = static_cast<const uint8_t *>(k_cache), a.vc = static_cast<const uint8_t *>(v_cache);
  a.ks = k_scale, a.vs = v_scale;
  a.table = page_table, a.lens = kv_lens, a.cu = cu_q, a.ldt = ldt;
  a.n_pages = n_pages, a.table_cols = table_cols;
  a.heads = heads, a.kv_heads = kv_heads, a.group = heads / kv_heads;
  a.n_seq = n_seq, a.n_tokens = n_tokens, a.max_q = max_q;
  a.scale_log2 = softmax_scale * 1.44269504f;
  a.causal = causal, a.window = window;
  a.splits = plan.splits, a.flat = plan.flat_tiles, a.ctas = plan.ctas;
  if (plan.slots) {
    a.part_o = static_cast<float *>(ws);
    a.part_ml = reinterpret_cast<float2 *>(a.part_o + plan.slots * head_dim);
  }
  a.budget = kWaitBudget;
  a.timeout = dev->timeout;
  cudaError_t e;
  if (dtype == VOC_LM_F16)
    e = head_dim == 64 ? launch_attention<__half, 64>(a, plan, stream)
                       : launch_attention<__half, 128>(a, plan, stream);
  else
    e = head_dim == 64 ? launch_attention<__nv_bfloat16, 64>(a, plan, stream)
                       : launch_attention<__nv_bfloat16, 128>(a, plan, stream);
  if (e != cudaSuccess) return cuda_fail(e, "launch attention");
  return finish(*dev, stream, flags);
}
