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
  int flat;  // CTAs count through the sequences' touched blocks (else blockIdx.z is the sequence)
};
constexpr int kFlatSeqs = 64;  // sequences up to which they do

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

// Finite 16-bit values: the first bits that are not, and the value of |bits|.
template <typename T>
struct Bits16;
template <>
struct Bits16<__half> {
  static constexpr uint32_t kInf = 0x7c00u;
  static __device__ __forceinline__ float value(uint32_t b) {
    return __half2float(__ushort_as_half(static_cast<unsigned short>(b)));
  }
};
template <>
struct Bits16<__nv_bfloat16> {
  static constexpr uint32_t kInf = 0x7f80u;
  static __device__ __forceinline__ float value(uint32_t b) { return __uint_as_float(b << 16); }
};

// Four codes times `f`, rounded again.
__device__ __forceinline__ uint32_t move_codes(uint32_t w, float f) {
  const float2 a = e4m3x2_to_f32(w & 0xffff), b = e4m3x2_to_f32(w >> 16);
  return e4m3x4(a.x * f, a.y * f, b.x * f, b.y * f);
}

template <int D>
struct AppendShape {
  static constexpr int kThreads = 2 * D;  // 16 groups of 4 tokens x D / 8 groups of 8 channels
};

// One CTA per (touched block, head, sequence); a thread holds 4 tokens x 8 channels of k and of v
// as they were read, so both are read once.  A warp covers 32 tokens x 32 channels: its loads and
// its stores of K rows and of V rows (4 tokens of a channel are one word) all fill 32-byte sectors,
// without a pass through shared memory.
// Measured: prompts of 13423 tokens, 8 heads of 128 channels (95 MB): 23.0 us, 4.1 TB/s: the chain of
// lengths, page and tokens, block maximum, stores, covered by the 4 CTAs of an SM only in part.  8
// single tokens 3.2 us, the same chain.
// FEW: for single tokens and short chunks, whose time is the chain of dependent reads: words of V that
// new and earlier tokens share are read beside the scales, at the cost of registers that whole blocks
// have a better use for (8 single tokens 5.8 -> 3.9 us; prompts 22.9 -> 26.6 us).
template <typename T, int D, bool FEW>
__global__ void __launch_bounds__(AppendShape<D>::kThreads, FEW ? 1 : 1024 / AppendShape<D>::kThreads)
    append_kernel(const LmAppendArgs p) {
  constexpr int kThreads = AppendShape<D>::kThreads, kWarps = kThreads / 32;
  __shared__ uint32_t red[2][kWarps];
  __shared__ uint32_t bad[2];  // tokens of the block with a NaN
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int t4 = (warp % 2) * 32 + lane / 4 * 4, ch = (warp / 2) * 32 + lane % 4 * 8;
  pdl_wait();
  pdl_launch_dependents();
  const int head = blockIdx.y;
  int b = blockIdx.z, nth = blockIdx.x;  // the sequence, and which of its touched blocks
  if (p.flat) {
    // Without empty CTAs for the blocks that shorter sequences do not have: each warp finds the CTA's
    // block in the running count of touched blocks, 32 sequences at a time.
    b = -1;
    for (int i0 = 0, before = 0; i0 < p.n_seq && b < 0; i0 += 32) {
      int touched = 0;
      if (i0 + lane < p.n_seq) {
        const SeqSpan s = seq_span(p.cu, i0 + lane, p.n_seq, p.n_tokens, p.max_q);
        const long long end = p.lens[i0 + lane], from = max(0ll, end - s.count);
        if (s.count > 0 && end > 0)
          touched = static_cast<int>((end - 1) / kBlockTokens - from / kBlockTokens) + 1;
      }
      int upto = touched;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int u = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += u;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, before + upto > static_cast<int>(blockIdx.x));
      if (past) {
        const int at = __ffs(past) - 1;
        b = i0 + at;
        nth = blockIdx.x - before - __shfl_sync(0xffffffffu, upto - touched, at);
      }
      before += __shfl_sync(0xffffffffu, upto, 31);
    }
    if (b < 0) return;
  }
  const SeqSpan span = seq_span(p.cu, b, p.n_seq, p.n_tokens, p.max_q);
  const long long len = p.lens[b];
  const long long p0 = len - span.count;  // position of the first new token
  const long long start = p0 > 0 ? p0 : 0;
  const long long blk = start / kBlockTokens + nth;
  const long long base = blk * kBlockTokens;
  if (span.count <= 0 || base >= len || blk >= p.table_cols) return;
  const int page = p.table[b * p.ldt + blk];  // used only after the tokens' loads are under way
  const int lo = static_cast<int>(start > base ? start - base : 0);
  const int hi = static_cast<int>(len - base < kBlockTokens ? len - base : kBlockTokens);
  const bool fresh = lo == 0;
  uint4 raw[2][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    raw[0][i] = raw[1][i] = make_uint4(0, 0, 0, 0);
    if (t4 + i >= lo && t4 + i < hi) {
      const long long row = span.first + (base + t4 + i - p0);
      raw[0][i] = *reinterpret_cast<const uint4 *>(static_cast<const T *>(p.k) + row * p.ldk +
                                                   head * p.hsk + ch);
      raw[1][i] = *reinterpret_cast<const uint4 *>(static_cast<const T *>(p.v) + row * p.ldv +
                                                   head * p.hsv + ch);
    }
  }
  if (page < 0 || page >= p.n_pages) return;
  const long long slot = static_cast<long long>(page) * p.heads + head;
  const float old[2] = {fresh ? 0.f : p.ks[slot], fresh ? 0.f : p.vs[slot]};
  uint8_t *kb = p.kc + slot * (kBlockTokens * D), *vb = p.vc + slot * (kBlockTokens * D);
  const bool some = t4 + 4 > lo && t4 < hi, all = fresh || (t4 >= lo && t4 + 4 <= hi);
  uint32_t kept[8];
  if (FEW && some && !all) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      kept[j] = *reinterpret_cast<const uint32_t *>(vb + (ch + j) * kBlockTokens + t4);
  }
  uint32_t m[2] = {0, 0};  // largest |value| of k and v, two at a time in the words' halves
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w[4] = {raw[t][i].x, raw[t][i].y, raw[t][i].z, raw[t][i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) m[t] = __vmaxu2(m[t], w[j] & 0x7fff7fffu);
    }
  auto block_max = [&]() {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int o = 16; o; o >>= 1) m[t] = __vmaxu2(m[t], __shfl_xor_sync(0xffffffffu, m[t], o));
      if (lane == 0) red[t][warp] = m[t];
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m[t] = __vmaxu2(m[t], red[t][w]);
      m[t] = max(m[t] & 0xffffu, m[t] >> 16);
    }
  };
  if (tid < 2) bad[tid] = 0;
  block_max();
  if (m[0] >= Bits16<T>::kInf || m[1] >= Bits16<T>::kInf) {  // an infinity or NaN in the block
    __syncthreads();
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      m[t] = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t w[4] = {raw[t][i].x, raw[t][i].y, raw[t][i].z, raw[t][i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t fin = w[j] & 0x7fff7fffu;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t half = fin >> 16 * h & 0xffffu;
            if (half >= Bits16<T>::kInf) fin &= ~(0xffffu << 16 * h);
            if (half > Bits16<T>::kInf) {
              atomicOr(&bad[(t4 + i) / 32], 1u << (t4 + i) % 32);
              w[j] &= ~(0xffffu << 16 * h);
            }
          }
          m[t] = __vmaxu2(m[t], fin);
        }
        raw[t][i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    block_max();
  }
  float inv[2], move[2];
  float *scales[2] = {p.ks + slot, p.vs + slot};
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    // `old` was read before block_max's barrier, so the store cannot overtake another's read
    float s = pow2(block_exponent(Bits16<T>::value(m[t])));
    move[t] = 1.f;
    if (!fresh && old[t] > s) s = old[t];
    if (!fresh) move[t] = old[t] / s;
    inv[t] = 1.f / s;
    if (tid == 0) *scales[t] = s;
  }

#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int tok = t4 + i;
    uint2 *dst = reinterpret_cast<uint2 *>(kb + tok * D + ch);
    if (fresh || (tok >= lo && tok < hi)) {
      float f[8];
      Vec16<T>::unpack(raw[0][i], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= inv[0];
      uint2 w = make_uint2(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]));
      if (bad[tok / 32] >> (tok % 32) & 1u) w = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
      *dst = w;
    } else if (move[0] != 1.f) {
      const uint2 o = *dst;
      *dst = make_uint2(move_codes(o.x, move[0]), move_codes(o.y, move[0]));
    }
  }
  if (some || fresh || move[1] != 1.f) {
    uint32_t mine = 0;  // bytes of the words that are new
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (t4 + i >= lo && t4 + i < hi) mine |= 0xffu << 8 * i;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float f[4][2];  // channels 2j and 2j + 1 of the four tokens
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w[4] = {raw[1][i].x, raw[1][i].y, raw[1][i].z, raw[1][i].w};
        unpack2<T>(w[j], f[i][0], f[i][1]);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t *dst = reinterpret_cast<uint32_t *>(vb + (ch + 2 * j + h) * kBlockTokens + t4);
        uint32_t w =
            e4m3x4(f[0][h] * inv[1], f[1][h] * inv[1], f[2][h] * inv[1], f[3][h] * inv[1]);
        if (!all) {
          uint32_t o = FEW && some ? kept[2 * j + h] : *dst;
          if (move[1] != 1.f) o = move_codes(o, move[1]);
          w = (w & mine) | (o & ~mine);
        }
        *dst = w;
      }
    }
  }
}

}  // namespace voc
