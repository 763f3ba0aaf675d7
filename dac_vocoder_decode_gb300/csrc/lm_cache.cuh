// lm_cache.cuh -- append of new tokens to the e4m3 cache of a token model.
//
// K [page][head][64 tokens][d] and V [page][head][d][64 tokens], e4m3, with one scale per (page,
// head) for each.  V is kept with the tokens innermost: the attention's second product sums over
// tokens, and both products then read their operand along the summed axis.
//
// The scales are powers of two, 2^e with the smallest e >= -96 for which max|v| <= 448 * 2^e.
// e4m3 keeps three mantissa bits at any magnitude, so a power of two costs no precision above the
// subnormals, and when a later token of the block needs a larger scale, moving the block's codes
// over is exact (again but for subnormals), so that appending token by token leaves nearly what
// appending the whole block at once leaves.
//
// Infinities saturate to 448 * scale and do not set the scale.  A NaN in a token's key or value
// makes its whole key row NaN and is stored as 0 in the value: every query that sees the token
// gets NaN, and no query that does not see it can meet a NaN through 0 * NaN.
#pragma once
#include "lm_common.cuh"

namespace voc {

struct LmAppendArgs {
  uint8_t *kc, *vc;
  float *ks, *vs;
  const void *k, *v;
  long long ldk, hsk, ldv, hsv;  // token and head strides of k and v, in elements
  const int *table, *lens, *cu;
  long long ldt;
  int n_pages, table_cols, heads, n_seq, n_tokens, max_q;
};

// First and number of the new tokens of sequence b in the batch (clamped to what there is).
struct SeqSpan {
  int first, count;
};
__device__ __forceinline__ SeqSpan seq_span(const int *cu, int b, int n_seq, int n_tokens,
                                            int max_q) {
  SeqSpan s;
  if (cu) {
    const int lo = min(max(cu[b], 0), n_tokens), hi = min(max(cu[b + 1], lo), n_tokens);
    s.first = lo;
    s.count = min(hi - lo, max_q);
  } else {
    s.count = n_tokens / n_seq;
    s.first = b * s.count;
  }
  return s;
}

// Smallest e >= -96 with a <= 448 * 2^e, for finite a >= 0: 448 = 0.875 * 2^9.
__device__ __forceinline__ int block_exponent(float a) {
  if (a < 0x1p-100f) return kScaleMinExp;
  const uint32_t u = __float_as_uint(a);
  const int x = static_cast<int>(u >> 23) - 126;  // a = f * 2^x with f in [0.5, 1)
  return max(kScaleMinExp, x - ((u & 0x7fffffu) <= 0x600000u ? 9 : 8));
}

// One CTA per (touched block, head, sequence).  Registers hold the block's new tokens (64 x D
// values of K and of V over 256 threads), so k and v are read once; the transposed V goes through
// shared memory.
template <typename T, int D>
__global__ void __launch_bounds__(256) append_kernel(const LmAppendArgs p) {
  constexpr int kChunks = D / 8;                        // 8-value chunks of a token's row
  constexpr int kPer = kBlockTokens * kChunks / 256;    // chunks per thread: 2 (D 64) or 4 (D 128)
  __shared__ float red[32];
  __shared__ uint32_t bad[2];                           // tokens of the block with a NaN
  __shared__ __align__(16) uint8_t vt[D][kBlockTokens];
  const int tid = threadIdx.x;
  pdl_wait();
  const int b = blockIdx.z, head = blockIdx.y;
  const SeqSpan span = seq_span(p.cu, b, p.n_seq, p.n_tokens, p.max_q);
  const long long len = p.lens[b];
  const long long p0 = len - span.count;  // position of the first new token
  const long long start = p0 > 0 ? p0 : 0;
  const long long blk = start / kBlockTokens + blockIdx.x;
  const long long base = blk * kBlockTokens;
  if (span.count <= 0 || base >= len || blk >= p.table_cols) return;
  const int page = p.table[b * p.ldt + blk];
  if (page < 0 || page >= p.n_pages) return;
  const int lo = static_cast<int>(start > base ? start - base : 0);
  const int hi = static_cast<int>(len - base < kBlockTokens ? len - base : kBlockTokens);
  const bool fresh = lo == 0;
  if (tid < 2) bad[tid] = 0;
  __syncthreads();

  float kv[2][kPer][8];
  uint32_t m[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int c = tid + 256 * i, tok = c / kChunks, ch = c % kChunks;
#pragma unroll
    for (int j = 0; j < 8; ++j) kv[0][i][j] = kv[1][i][j] = 0.f;
    if (tok >= lo && tok < hi) {
      const long long row = span.first + (base + tok - p0);
      const T *src[2] = {static_cast<const T *>(p.k) + row * p.ldk + head * p.hsk + ch * 8,
                         static_cast<const T *>(p.v) + row * p.ldv + head * p.hsv + ch * 8};
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        float f[8];
        Vec16<T>::unpack(*reinterpret_cast<const uint4 *>(src[t]), f);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t a = abs_bits(f[j]);
          if (a < kInfBits) m[t] = max(m[t], a);
          if (a > kInfBits) {
            atomicOr(&bad[tok / 32], 1u << (tok % 32));
            f[j] = 0.f;
          }
          kv[t][i][j] = f[j];
        }
      }
    }
  }
  const long long slot = static_cast<long long>(page) * p.heads + head;
  uint8_t *kb = p.kc + slot * (kBlockTokens * D), *vb = p.vc + slot * (kBlockTokens * D);
  float *scales[2] = {p.ks + slot, p.vs + slot};
  float inv[2], move[2] = {1.f, 1.f};
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const uint32_t a = group_max<256>(m[t], red);
    float s = pow2(block_exponent(__uint_as_float(a)));
    if (!fresh) {
      const float old = *scales[t];
      if (old > s) s = old;
      move[t] = old / s;
    }
    inv[t] = 1.f / s;
    __syncthreads();  // everybody has read the old scale
    if (tid == 0) *scales[t] = s;
  }

#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int c = tid + 256 * i, tok = c / kChunks, ch = c % kChunks;
    const bool is_new = tok >= lo && tok < hi;
    uint2 *dst = reinterpret_cast<uint2 *>(kb + tok * D + ch * 8);
    if (is_new || fresh) {
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = kv[0][i][j] * inv[0];
      uint2 w = make_uint2(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]));
      if (bad[tok / 32] >> (tok % 32) & 1u) w = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
      *dst = w;
    } else if (move[0] != 1.f) {
      const uint2 o = *dst;
      const uint32_t w[2] = {o.x, o.y};
      uint32_t r[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float2 a = e4m3x2_to_f32(w[j] & 0xffff), c2 = e4m3x2_to_f32(w[j] >> 16);
        r[j] = e4m3x4(a.x * move[0], a.y * move[0], c2.x * move[0], c2.y * move[0]);
      }
      *dst = make_uint2(r[0], r[1]);
    }
    if (is_new || fresh) {
#pragma unroll
      for (int j = 0; j < 8; ++j) vt[ch * 8 + j][tok] = e4m3(kv[1][i][j] * inv[1]);
    }
  }
  __syncthreads();
  // V: 4 tokens of one channel at a time; a block without earlier tokens is stored whole
  const bool moved = move[1] != 1.f;
  for (int c = tid; c < D * (kBlockTokens / 4); c += 256) {
    const int d = c / (kBlockTokens / 4), t4 = c % (kBlockTokens / 4) * 4;
    uint32_t *dst = reinterpret_cast<uint32_t *>(vb + d * kBlockTokens + t4);
    const uint32_t n = *reinterpret_cast<const uint32_t *>(&vt[d][t4]);
    if (fresh || (t4 >= lo && t4 + 4 <= hi)) {
      *dst = n;
    } else if (moved || (t4 + 4 > lo && t4 < hi)) {
      const uint32_t o = *dst;
      uint32_t r = o;
      if (moved) {
        const float2 a = e4m3x2_to_f32(o & 0xffff), c2 = e4m3x2_to_f32(o >> 16);
        r = e4m3x4(a.x * move[1], a.y * move[1], c2.x * move[1], c2.y * move[1]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (t4 + j >= lo && t4 + j < hi) r = (r & ~(0xffu << 8 * j)) | (n & (0xffu << 8 * j));
      *dst = r;
    }
  }
}

}  // namespace voc
