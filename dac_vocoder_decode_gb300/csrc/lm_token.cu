// lm_token.cu -- C entry points of what a token model runs beside its 8-bit operators (vocoder_lm_rotate,
// vocoder_lm_adapters, vocoder_lm_logprobs in include/vocoder.h): argument checks, choice of launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "vocoder.h"
#include "lm_adapters.cuh"
#include "lm_host.cuh"
#include "lm_logprobs.cuh"
#include "lm_rotate.cuh"

using namespace voc::lm;

// ------------------------------------------------------------------ heads turned by position
namespace {

template <typename T, int L, bool NEAR>
cudaError_t launch_rotate(int sms, voc::LmRotateArgs &a, voc_stream_t stream) {
  constexpr int at_once = 32 / L, warps = voc::kRotThreads / 32;
  int turns = 0;
  for (int i = 0; i < 2; ++i) turns += a.groups[i] = (a.heads[i] + at_once - 1) / at_once;
  // A warp takes all heads of a token, whose angles it then computes once, or as few as fill the GPU with 32
  // warps an SM.
  const long long want = std::max<long long>(1, sms * 32ll / a.tokens);
  int parts = static_cast<int>(std::min<long long>({want, turns, 65535}));
  a.per = (turns + parts - 1) / parts;
  parts = (turns + a.per - 1) / a.per;
  return launch(voc::rotate_kernel<T, L, NEAR>,
                dim3(static_cast<unsigned>((a.tokens + warps - 1) / warps), static_cast<unsigned>(parts)),
                dim3(voc::kRotThreads), 0, 1, stream, a);
}
template <typename T, bool NEAR>
cudaError_t launch_rotate(int sms, voc::LmRotateArgs &a, voc_stream_t stream) {
  const int lanes = a.d / 16;
  if (lanes <= 1) return launch_rotate<T, 1, NEAR>(sms, a, stream);
  if (lanes <= 2) return launch_rotate<T, 2, NEAR>(sms, a, stream);
  if (lanes <= 4) return launch_rotate<T, 4, NEAR>(sms, a, stream);
  if (lanes <= 8) return launch_rotate<T, 8, NEAR>(sms, a, stream);
  return launch_rotate<T, 16, NEAR>(sms, a, stream);
}

}  // namespace

VOC_API voc_status vocoder_lm_rotate(const void *q, long long ldq, long long hsq, int heads,
                                     const void *k, long long ldk, long long hsk, int kv_heads,
                                     int head_dim, int dtype, const void *q_weight,
                                     const void *k_weight, float eps, const int *positions,
                                     long long ldp, int axes, const long long *turns, const int *axis,
                                     int pairs, int neighbours, long long n_tokens, void *q_out,
                                     long long ldqo, long long hsqo, void *k_out, long long ldko,
                                     long long hsko, voc_stream_t stream, unsigned flags) {
  if (dtype != VOC_LM_BF16 && dtype != VOC_LM_F16) return fail(VOC_INVALID_ARG, "rotate: dtype");
  if (head_dim < 16 || head_dim > 256 || head_dim % 16)
    return fail(VOC_UNSUPPORTED, "rotate: head_dim must be a multiple of 16 up to 256");
  if (pairs < 0 || 2 * static_cast<long long>(pairs) > head_dim || pairs % 8)
    return fail(VOC_UNSUPPORTED, "rotate: pairs must be a multiple of 8, and of no more than head_dim channels");
  if (heads < 0 || kv_heads < 0 || heads > 65536 || kv_heads > 65536 || heads + kv_heads < 1)
    return fail(VOC_INVALID_ARG, "rotate: heads");
  if (n_tokens < 0 || n_tokens > 0x7fffffffll / (static_cast<long long>(heads) + kv_heads))
    return fail(VOC_INVALID_ARG, "rotate: number of tokens");
  if (axes < 1 || axes > 16 || (axes > 1 && ldp < n_tokens))
    return fail(VOC_INVALID_ARG, "rotate: axes or the stride of positions");
  if (neighbours != 0 && neighbours != 1) return fail(VOC_INVALID_ARG, "rotate: neighbours");
  if (!known_flags(flags)) return fail(VOC_INVALID_ARG, "rotate: flags");
  if ((q_weight || k_weight) && !(eps >= 0.f && std::isfinite(eps)))
    return fail(VOC_INVALID_ARG, "rotate: eps");
  if (n_tokens > 0 && ((heads && (!q || !q_out)) || (kv_heads && (!k || !k_out)) ||
                       (pairs && (!positions || !turns))))
    return fail(VOC_INVALID_ARG, "rotate: NULL buffer");
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_out, 16) || !aligned(k_out, 16) ||
      !aligned(q_weight, 16) || !aligned(k_weight, 16) || ldq % 8 || hsq % 8 || ldk % 8 || hsk % 8 ||
      ldqo % 8 || hsqo % 8 || ldko % 8 || hsko % 8)
    return fail(VOC_INVALID_ARG,
                "rotate: heads and weights must be 16-byte aligned, strides multiples of 8");
  if (!aligned(positions, 4) || !aligned(axis, 8) || !aligned(turns, 16))
    return fail(VOC_INVALID_ARG, "rotate: positions, axis (8 bytes) or turns (16) are not aligned");
  Device *dev;
  if (voc_status st = device(&dev); st != VOC_OK) return st;
  if (n_tokens == 0) return finish(*dev, stream, flags);
  voc::LmRotateArgs a{};
  a.x[0] = q, a.w[0] = q_weight, a.out[0] = q_out;
  a.x[1] = k, a.w[1] = k_weight, a.out[1] = k_out;
  a.ldx[0] = ldq, a.hsx[0] = hsq, a.ldo[0] = ldqo, a.hso[0] = hsqo, a.heads[0] = heads;
  a.ldx[1] = ldk, a.hsx[1] = hsk, a.ldo[1] = ldko, a.hso[1] = hsko, a.heads[1] = kv_heads;
  a.pos = positions, a.axis = axis, a.ldp = ldp, a.axes = axes;
  a.turns = reinterpret_cast<const unsigned long long *>(turns);
  a.pairs = pairs, a.d = head_dim, a.tokens = n_tokens, a.eps = eps;
  cudaError_t e;
  if (dtype == VOC_LM_F16)
    e = neighbours ? launch_rotate<__half, true>(dev->sms, a, stream)
                   : launch_rotate<__half, false>(dev->sms, a, stream);
  else
    e = neighbours ? launch_rotate<__nv_bfloat16, true>(dev->sms, a, stream)
                   : launch_rotate<__nv_bfloat16, false>(dev->sms, a, stream);
  if (e != cudaSuccess) return cuda_fail(e, "launch rotate");
  return finish(*dev, stream, flags);
}

// ------------------------------------------------------------------ low-rank adapters
namespace {

// Shared-memory limits of the adapters' kernels on the current device.
struct AdapterSetup {
  std::once_flag once;
  cudaError_t err = cudaSuccess;
};
AdapterSetup g_adapters[kMaxDevices];

template <typename W, typename Y>
void allow_adapters(cudaError_t &e) {
  using namespace voc;
  allow_smem(e, adapters_kernel<W, Y, 16>, AdapterSmem<16, kAdParts<W, Y>>::kBytes);
  allow_smem(e, adapters_kernel<W, Y, 32>, AdapterSmem<32, kAdParts<W, Y>>::kBytes);
  allow_smem(e, adapters_kernel<W, Y, 64>, AdapterSmem<64, kAdParts<W, Y>>::kBytes);
  allow_smem(e, adapters_kernel<W, Y, 128>, AdapterSmem<128, kAdParts<W, Y>>::kBytes);
}
cudaError_t set_up_adapters() {
  int d = 0;
  cudaError_t e = cudaGetDevice(&d);
  if (e != cudaSuccess) return e;
  AdapterSetup &s = g_adapters[d];  // device() has looked at the index
  std::call_once(s.once, [&] {
    allow_adapters<__half, __half>(s.err);
    allow_adapters<__half, float>(s.err);
    allow_adapters<__nv_bfloat16, __nv_bfloat16>(s.err);
    allow_adapters<__nv_bfloat16, float>(s.err);
  });
  return s.err;
}

template <typename W, typename Y, int R>
cudaError_t launch_adapters(int sms, const voc::LmAdaptersArgs &a, voc_stream_t stream) {
  const int tiles = (a.M + voc::kAdTokens - 1) / voc::kAdTokens;
  const int most = std::min({a.M, a.pool + 1, voc::kAdTokens});  // adapters of a tile
  // Clusters of a tile, which share its adapters: some 512 of all tiles.  Measured, for 64 / 128 / 256 / 512 / 1024 /
  // 2048 of them, 1024 -> 1536, rank 16: 4000 tokens of 64 adapters in no order 260 / 243 / 232 / 214 / 218 / 233
  // us, 768 tokens 79 / 78 / 81 / 90 / 98 / 98, 15504 of 8 adapters 93 / 93 / 93 / 93 / 91 / 84; 15504 x 4096 ->
  // 4096, rank 64, runs of 4: 159 / 159 / 158 / 124 / 124 / 124.
  const int turns = std::max(1, std::min(most, 512 / tiles));
  // CTAs of a cluster, as long as the tiles' clusters fill two CTAs an SM: measured, 1 / 2 / 4 CTAs, 15504 x 4096 x
  // 4096 of rank 64 136 / 143 / 150 us, 15423 x 1001 x 1540 of rank 32 54 / 62 / 72.
  int split = 8;
  while (split > 1 && static_cast<long long>(tiles) * split > 2 * sms) split /= 2;
  return launch(voc::adapters_kernel<W, Y, R>, dim3(tiles, turns, split), dim3(voc::kAdThreads),
                voc::AdapterSmem<R, voc::kAdParts<W, Y>>::kBytes, split, stream, a);
}
template <typename W, typename Y>
cudaError_t launch_adapters(int sms, const voc::LmAdaptersArgs &a, voc_stream_t stream) {
  if (a.rank <= 16) return launch_adapters<W, Y, 16>(sms, a, stream);
  if (a.rank <= 32) return launch_adapters<W, Y, 32>(sms, a, stream);
  if (a.rank <= 64) return launch_adapters<W, Y, 64>(sms, a, stream);
  return launch_adapters<W, Y, 128>(sms, a, stream);
}

}  // namespace

VOC_API voc_status vocoder_lm_adapters(const void *x8, long long ldx, const float *x_scale,
                                       const void *y, long long ldy, int y_dtype, const void *a,
                                       long long lda, long long sa, const void *b, long long ldb,
                                       long long sb, int dtype, const float *scale, const int *ranks,
                                       int rank, int pool, const int *ids, int M, int N, int K,
                                       void *out, long long ldo, voc_stream_t stream,
                                       unsigned flags) {
  if (dtype != VOC_LM_BF16 && dtype != VOC_LM_F16) return fail(VOC_INVALID_ARG, "adapters: dtype");
  if (y_dtype != dtype && y_dtype != VOC_LM_F32)
    return fail(VOC_INVALID_ARG, "adapters: y_dtype must be the adapters' type or f32");
  if (M < 0 || N < 0 || K < 1 || M > (1 << 28) || N > (1 << 24) || K > (1 << 28))
    return fail(VOC_INVALID_ARG, "adapters: sizes");  // 32-bit counters of a tile's values
  if (rank < 8 || rank > 128 || rank % 8)
    return fail(VOC_UNSUPPORTED, "adapters: rank must be a multiple of 8 up to 128");
  if (pool < 1) return fail(VOC_INVALID_ARG, "adapters: pool");
  if (!known_flags(flags)) return fail(VOC_INVALID_ARG, "adapters: flags");
  if (ldx < K || ldy < N || ldo < N || lda < K || ldb < rank)
    return fail(VOC_INVALID_ARG, "adapters: a row stride is below the width");
  if (ldx > 0x7fffffff || ldy > 0x7fffffff || ldo > 0x7fffffff || lda > 0x7fffffff || ldb > 0x7fffffff)
    return fail(VOC_UNSUPPORTED, "adapters: a row stride above 2^31 - 1");
  if (ldx % 16) return fail(VOC_INVALID_ARG, "adapters: the row stride of x8 must be a multiple of 16");
  if (lda % 8 || ldb % 8 || sa % 8 || sb % 8)
    return fail(VOC_INVALID_ARG, "adapters: strides of a and b must be multiples of 8");
  if (M > 0 && N > 0 && (!x8 || !x_scale || !y || !a || !b || !scale || !ids || !out))
    return fail(VOC_INVALID_ARG, "adapters: NULL buffer");
  if (!aligned(x8, 16) || !aligned(a, 16) || !aligned(b, 16))
    return fail(VOC_INVALID_ARG, "adapters: x8, a and b must be 16-byte aligned");
  const size_t e = y_dtype == VOC_LM_F32 ? 4 : 2;
  if (!aligned(x_scale, 4) || !aligned(scale, 4) || !aligned(ids, 4) || !aligned(ranks, 4) ||
      !aligned(y, e) || !aligned(out, e))
    return fail(VOC_INVALID_ARG, "adapters: a buffer is not aligned to its type");
  if (y == out && ldy != ldo)
    return fail(VOC_INVALID_ARG, "adapters: out in y's place needs y's row stride");
  Device *dev;
  if (voc_status st = device(&dev); st != VOC_OK) return st;
  if (M == 0 || N == 0) return finish(*dev, stream, flags);
  cudaError_t err = set_up_adapters();
  if (err != cudaSuccess) return cuda_fail(err, "adapters: device set-up");
  const voc::LmAdaptersArgs args{static_cast<const uint8_t *>(x8), x_scale, y, a, b, scale, ids, ranks,
                                 out, ldx, ldy, ldo, lda, sa, ldb, sb, M, N, K, rank, pool};
  if (dtype == VOC_LM_F16)
    err = y_dtype == VOC_LM_F32 ? launch_adapters<__half, float>(dev->sms, args, stream)
                                : launch_adapters<__half, __half>(dev->sms, args, stream);
  else
    err = y_dtype == VOC_LM_F32
              ? launch_adapters<__nv_bfloat16, float>(dev->sms, args, stream)
              : launch_adapters<__nv_bfloat16, __nv_bfloat16>(dev->sms, args, stream);
  if (err != cudaSuccess) return cuda_fail(err, "launch adapters");
  return finish(*dev, stream, flags);
}

// ------------------------------------------------------------------ log probabilities
namespace {

template <typename T, bool TOP>
cudaError_t launch_logprobs(int sms, const voc::LmLogprobsArgs &a, voc_stream_t stream) {
  // A warp has a row of up to 4096 values where there are more than four rows an SM, a CTA another, several CTAs while
  // there are SMs for them and a CTA keeps 4096 values.  Measured, a warp / a CTA a row of 2048 bf16 values: without
  // alternatives 300 rows 2.5 / 2.6 us, 640 2.8 / 3.3, 4800 6.4 / 16.4; with 5 5.0 / 4.4, 5.3 / 5.4, 10.6 / 29.1;
  // with 20 8.4 / 4.9, 8.7 / 6.2, 1200 rows 9.6 / 10.5, 4800 17.2 / 33.8.  (So with 20 of 16-bit rows the border comes
  // early: the CTA is ahead up to some seven rows an SM, at 640 x 4096 with 7.2 of 12.8 us.  f32 rows, 640 x 2048:
  // 3.6 / 6.2, 7.1 / 9.6, 11.2 / 10.4.)  A CTA's loop has whole batches from 6144 values of 16 bits on and one vector
  // at a time below: 4800 rows of 4097 / 5000 / 6200 / 8192 bf16 values 24 / 25 / 31 / 23 us (of 4096, a warp
  // each, 9.2).
  if (a.vocab <= 4096 && a.rows > 4 * sms)
    return launch(voc::logprobs_kernel<T, 32, TOP>,
                  dim3(static_cast<unsigned>((a.rows + voc::kLpWarps - 1) / voc::kLpWarps)),
                  dim3(32 * voc::kLpWarps), 0, 1, stream, a);
  int split = 1;
  while (split < 8 && 2 * split * a.rows <= 2 * sms && a.vocab / (2 * split) >= 4096) split *= 2;
  return launch(voc::logprobs_kernel<T, voc::kLpWide, TOP>,
                dim3(static_cast<unsigned>(a.rows), 1, split), dim3(voc::kLpWide), 0, split, stream, a);
}
template <typename T>
cudaError_t launch_logprobs(int sms, const voc::LmLogprobsArgs &a, voc_stream_t stream) {
  return a.k ? launch_logprobs<T, true>(sms, a, stream) : launch_logprobs<T, false>(sms, a, stream);
}

}  // namespace

VOC_API voc_status vocoder_lm_logprobs(const void *logits, long long ldl, int dtype, long long rows,
                                       int vocab, float temperature, const long long *tokens,
                                       float *logprob, float *entropy, int top, float *top_logprobs,
                                       long long *top_tokens, voc_stream_t stream, unsigned flags) {
  if (dtype != VOC_LM_BF16 && dtype != VOC_LM_F16 && dtype != VOC_LM_F32)
    return fail(VOC_INVALID_ARG, "logprobs: dtype");
  if (rows < 0 || rows > 0x7fffffffll || vocab < 1 || vocab > (1 << 28))
    return fail(VOC_INVALID_ARG, "logprobs: sizes");
  if (!(temperature >= 0x1p-20f && temperature <= 0x1p20f))
    return fail(VOC_INVALID_ARG, "logprobs: temperature must lie between 2^-20 and 2^20");
  if (top < 0 || top > vocab) return fail(VOC_INVALID_ARG, "logprobs: top");
  if (top > voc::kLpMaxTop) return fail(VOC_UNSUPPORTED, "logprobs: more than 32 alternatives");
  if (!known_flags(flags)) return fail(VOC_INVALID_ARG, "logprobs: flags");
  if (ldl < vocab) return fail(VOC_INVALID_ARG, "logprobs: a row stride is below the width");
  if ((tokens == nullptr) != (logprob == nullptr))
    return fail(VOC_INVALID_ARG, "logprobs: tokens and logprob go together");
  if (rows > 0 && (!logits || (top && (!top_logprobs || !top_tokens))))
    return fail(VOC_INVALID_ARG, "logprobs: NULL buffer");
  if (!aligned(logits, dtype == VOC_LM_F32 ? 4 : 2) || !aligned(tokens, 8) || !aligned(logprob, 4) ||
      !aligned(entropy, 4) || !aligned(top_logprobs, 4) || !aligned(top_tokens, 8))
    return fail(VOC_INVALID_ARG, "logprobs: a buffer is not aligned to its type");
  Device *dev;
  if (voc_status st = device(&dev); st != VOC_OK) return st;
  if (rows == 0 || (!logprob && !entropy && !top)) return finish(*dev, stream, flags);
  voc::LmLogprobsArgs a{logits, tokens, logprob, entropy, top_logprobs, top_tokens, rows, ldl, vocab, top,
                        static_cast<float>(1.4426950408889634 / temperature), 2.f / temperature};
  cudaError_t e;
  if (dtype == VOC_LM_F32)
    e = launch_logprobs<float>(dev->sms, a, stream);
  else if (dtype == VOC_LM_F16)
    e = launch_logprobs<__half>(dev->sms, a, stream);
  else
    e = launch_logprobs<__nv_bfloat16>(dev->sms, a, stream);
  if (e != cudaSuccess) return cuda_fail(e, "launch logprobs");
  return finish(*dev, stream, flags);
}
