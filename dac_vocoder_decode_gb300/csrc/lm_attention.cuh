// lm_attention.cuh -- attention of a token model's newest tokens over the e4m3 cache
// (lm_cache.cuh has its layout).
//
// For a query at position p with the visible keys j (causal: j <= p; window w: j > p - w)
//   s_j = (q . k_j) c, c = softmax_scale * log2(e);  o = sum_j 2^(s_j) v_j / sum_j 2^(s_j),
// zeros where no key is visible.  One pass over the keys with the running maximum and sum of the
// softmax.  The scale of a block's values goes into the exponent: with u_j = s_j + log2(vs_j) and
// m = max u_j, the weights 2^(u_j - m) <= 1 multiply the stored codes and the sum takes
// 2^(u_j - m) / vs_j, so accumulators of blocks with different scales add up without a rescale.
#pragma once
#include "lm_cache.cuh"

namespace voc {

constexpr int kAttnWarps = 8;                      // consumer warps; one more warp copies
constexpr int kAttnThreads = 32 * (kAttnWarps + 1);
constexpr int kAttnRows = 16;                      // rows of a tile (one MMA's M)
constexpr int kPShift = 14;                        // weights are kept times 2^14 in 16 bits

struct LmAttnArgs {
  const void *q;
  void *out;
  long long ldq, hsq, ldo, hso;
  const uint8_t *kc, *vc;
  const float *ks, *vs;
  const int *table, *lens, *cu;
  long long ldt;
  int n_pages, table_cols, heads, kv_heads, group, n_seq, n_tokens, max_q;
  float scale_log2;  // softmax_scale * log2(e)
  int causal, window;
  int row_tiles, splits;
  float *part_o;     // [tile][split][16][D], splits > 1
  float2 *part_ml;   // [tile][split][16]
  long long budget;
  int *timeout;
};

// m16n8k16, f16 operands, f32 accumulators.
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  uint32_t u;
  memcpy(&u, &h, 4);
  return u;
}

// Scale of a 16-bit query row (a power of two) that brings its largest finite value to
// [2^14, 2^15): f16 then holds bf16 and f16 values exactly, but for what lies 2^-28 below it.
__device__ __forceinline__ int query_exponent(uint32_t amax) {
  if (amax == 0) return 0;
  const int e = 14 - (static_cast<int>(amax >> 23) - 127);
  return min(max(e, -110), 110);
}

// The keys that the rows [r0, r1) of a sequence's tile can see, and those of one row.
struct KeySpan {
  long long lo, hi;
};
__device__ __forceinline__ KeySpan visible(const LmAttnArgs &p, long long pos, long long len) {
  KeySpan s;
  s.hi = p.causal ? min(len, pos + 1) : len;
  s.lo = p.window > 0 ? max(0ll, pos - p.window + 1) : 0;
  return s;
}

template <int D>
__host__ __device__ constexpr int attn_stages() { return D == 128 ? 12 : 24; }
template <int D>
__host__ __device__ constexpr size_t attn_smem() {
  return static_cast<size_t>(attn_stages<D>()) * 2 * kBlockTokens * D + 1024;
}

// 16 rows (queries that share a key head) of one sequence over one part of its keys.  K and V
// blocks come through a ring of shared-memory stages, one bulk copy each; two warps share a
// block, 32 keys each, so that a stage is held for half the time.  Both products are 16-bit MMAs:
// e4m3 converts exactly to f16, and the weights keep 11 bits there (as e4m3 they would keep 4).
// The order in which a thread holds channels and keys is chosen so that its operands are whole
// words of the stored rows: the sums do not depend on it.
template <typename T, int D>
__global__ void __launch_bounds__(kAttnThreads, 1) attn_rows_kernel(const LmAttnArgs p) {
  constexpr int kStages = attn_stages<D>();
  constexpr int kBytes = kBlockTokens * D;
  constexpr int kSteps = D / 16;   // MMA steps over the channels
  constexpr int kTilesD = D / 8;   // output column tiles
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(8) uint64_t full[kStages], empty[kStages];
  __shared__ int abort_flag;
  __shared__ float2 ml[kAttnWarps][kAttnRows];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int g = lane / 4, t = lane % 4;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(full + i), 1);
      mbar_init(smem_u32(empty + i), 2);
    }
    abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  pdl_wait();

  const int b = blockIdx.z, hk = blockIdx.y / p.row_tiles, rt = blockIdx.y % p.row_tiles;
  const int split = blockIdx.x;
  const SeqSpan span = seq_span(p.cu, b, p.n_seq, p.n_tokens, p.max_q);
  const int rows = span.count * p.group;
  const int r0 = rt * kAttnRows;
  if (r0 >= rows) return;  // the whole block
  const int r_last = min(rows, r0 + kAttnRows) - 1;
  const long long len = max(0ll, min(static_cast<long long>(p.lens[b]),
                                     static_cast<long long>(p.table_cols) * kBlockTokens));
  const long long p0 = static_cast<long long>(p.lens[b]) - span.count;
  const long long key_lo = visible(p, p0 + r0 / p.group, len).lo;
  const long long key_hi = visible(p, p0 + r_last / p.group, len).hi;
  const long long blk0 = key_lo / kBlockTokens;
  const long long n_blk = key_hi > key_lo ? (key_hi - 1) / kBlockTokens + 1 - blk0 : 0;
  const long long per = (n_blk + p.splits - 1) / p.splits;
  const int first = static_cast<int>(blk0 + min(n_blk, split * per));
  const int count = static_cast<int>(min(n_blk, (split + 1) * per) - min(n_blk, split * per));
  const int *table = p.table + b * p.ldt;

  float o[kTilesD][4];
#pragma unroll
  for (int i = 0; i < kTilesD; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

  if (warp == kAttnWarps) {
    if (lane == 0) {
      int done = 0;
      for (int i = 0; i < count; ++i) {
        const int st = i % kStages;
        if (i >= kStages &&
            !mbar_wait(smem_u32(empty + st), (i / kStages - 1) & 1, p.budget, &abort_flag)) {
          *static_cast<volatile int *>(&abort_flag) = 1;
          break;
        }
        const int page = table[first + i];
        if (page < 0 || page >= p.n_pages) {
          mbar_arrive(smem_u32(full + st));
        } else {
          const long long at = (static_cast<long long>(page) * p.kv_heads + hk) * kBytes;
          const uint32_t bar = smem_u32(full + st), dst = smem_u32(smem + st * 2 * kBytes);
          mbar_arrive_expect_tx(bar, 2 * kBytes);
          bulk_load(dst, p.kc + at, kBytes, bar);
          bulk_load(dst + kBytes, p.vc + at, kBytes, bar);
        }
        done = i + 1;
      }
      if (*static_cast<volatile int *>(&abort_flag)) {  // leave with no copy in flight
        const int never = 0;
        for (int i = max(0, done - kStages); i < done; ++i)
          mbar_wait(smem_u32(full + i % kStages), (i / kStages) & 1, p.budget, &never);
        if (p.timeout) *p.timeout = 1;
      }
    }
  } else {
    // queries: rows g and g + 8 of the tile, scaled into f16
    uint32_t qa[kSteps][4];
    float qc[2];
    int row_tok[2];
    KeySpan see[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = min(r0 + g + 8 * h, r_last);  // spare rows repeat the last one
      row_tok[h] = r / p.group;
      see[h] = visible(p, p0 + row_tok[h], len);
      const T *src = static_cast<const T *>(p.q) + (span.first + row_tok[h]) * p.ldq +
                     (hk * p.group + r % p.group) * p.hsq;
      float f[D / 4];
      uint32_t a = 0;
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float v = to_f32(src[64 * (s / 4) + 16 * t + 4 * (s % 4) + j]);
          f[4 * s + j] = v;
          if (abs_bits(v) < kInfBits) a = max(a, abs_bits(v));
        }
      a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
      a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
      const int e = query_exponent(a);
      const float up = pow2(e);
      qc[h] = p.scale_log2 * pow2(-e);
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        qa[s][h] = f16x2(f[4 * s] * up, f[4 * s + 1] * up);
        qa[s][2 + h] = f16x2(f[4 * s + 2] * up, f[4 * s + 3] * up);
      }
    }
    const int half = warp % 2;
    for (int i = warp / 2; i < count; i += kAttnWarps / 2) {
      const int st = i % kStages;
      const bool landed = mbar_wait(smem_u32(full + st), (i / kStages) & 1, p.budget, &abort_flag);
      if (!__all_sync(0xffffffffu, landed)) {
        *static_cast<volatile int *>(&abort_flag) = 1;
        break;
      }
      const int page = table[first + i];
      const long long base = static_cast<long long>(first + i) * kBlockTokens + 32 * half;
      if (page >= 0 && page < p.n_pages && base < key_hi && base + 32 > key_lo) {
        const long long slot = static_cast<long long>(page) * p.kv_heads + hk;
        const float ks = p.ks[slot], vs = fmaxf(p.vs[slot], kScaleMin);
        const float lvs = log2f(vs), ivs = 1.f / vs;
        const uint32_t kb = smem_u32(smem + st * 2 * kBytes), vb = kb + kBytes;
        // scores: column 2t + e of tile j is key 8t + 2j + e
        float sc[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
          for (int x = 0; x < 4; ++x) sc[j][x] = 0.f;
          const uint32_t row = kb + (32 * half + 8 * (g >> 1) + 2 * j + (g & 1)) * D + 16 * t;
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            const uint4 w = lds128(row + 64 * c);
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int s = 0; s < 4; ++s)
              mma_f16(sc[j], qa[4 * c + s], e4m3x2_to_f16x2(ww[s] & 0xffff),
                      e4m3x2_to_f16x2(ww[s] >> 16));
          }
        }
        // u = s + log2(vs), -inf where the row does not see the key
        const bool whole = base >= max(see[0].lo, see[1].lo) && base + 32 <= min(see[0].hi, see[1].hi);
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int h = x / 2;
            float u = fmaf(sc[j][x], qc[h] * ks, lvs);
            if (!whole) {
              const long long key = base + 8 * t + 2 * j + x % 2;
              if (key < see[h].lo || key >= see[h].hi) u = -INFINITY;
            }
            sc[j][x] = u;
            top[h] = fmaxf(top[h], u);
          }
        float alpha[2], off[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
          top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
          const float nm = fmaxf(m[h], top[h]);
          alpha[h] = m[h] == nm ? 1.f : exp2f(m[h] - nm);
          m[h] = nm;
          off[h] = (nm == -INFINITY ? 0.f : nm) - kPShift;
        }
        float sum[2] = {0.f, 0.f};
        uint32_t pa[2][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float w[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            w[x] = exp2f(sc[j][x] - off[x / 2]);
            sum[x / 2] += w[x];
          }
          pa[j / 2][2 * (j % 2)] = f16x2(w[0], w[1]);
          pa[j / 2][2 * (j % 2) + 1] = f16x2(w[2], w[3]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) l[h] = l[h] * alpha[h] + sum[h] * ivs;
        if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
          for (int n = 0; n < kTilesD; ++n) {
            o[n][0] *= alpha[0], o[n][1] *= alpha[0];
            o[n][2] *= alpha[1], o[n][3] *= alpha[1];
          }
        }
        // codes of keys outside the tile's span count as zero, whatever they hold
        uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
        if (base < key_lo || base + 32 > key_hi) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const long long key = base + 8 * t + j;
            if (key < key_lo || key >= key_hi) keep[j / 4] &= ~(0xffu << 8 * (j % 4));
          }
        }
#pragma unroll
        for (int n = 0; n < kTilesD; ++n) {
          uint32_t v0, v1;
          asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                       : "=r"(v0), "=r"(v1)
                       : "r"(vb + (8 * n + g) * kBlockTokens + 32 * half + 8 * t)
                       : "memory");
          v0 &= keep[0], v1 &= keep[1];
          mma_f16(o[n], pa[0], e4m3x2_to_f16x2(v0 & 0xffff), e4m3x2_to_f16x2(v0 >> 16));
          mma_f16(o[n], pa[1], e4m3x2_to_f16x2(v1 & 0xffff), e4m3x2_to_f16x2(v1 >> 16));
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(empty + st));
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    }
    if (t == 0) {
      ml[warp][g] = make_float2(m[0], l[0]);
      ml[warp][g + 8] = make_float2(m[1], l[1]);
    }
  }
  __syncthreads();  // the ring is free: every copy has been waited for
  // join the warps: each scales its rows to the common maximum
  float *acc = reinterpret_cast<float *>(smem);  // [warp][16][D]
  if (warp < kAttnWarps) {
    float f[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float top = -INFINITY;
      for (int w = 0; w < kAttnWarps; ++w) top = fmaxf(top, ml[w][g + 8 * h].x);
      f[h] = top == -INFINITY ? 0.f : exp2f(m[h] - top);
    }
#pragma unroll
    for (int n = 0; n < kTilesD; ++n) {
      float *row = acc + (warp * kAttnRows + g) * D + 8 * n + 2 * t;
      *reinterpret_cast<float2 *>(row) = make_float2(o[n][0] * f[0], o[n][1] * f[0]);
      *reinterpret_cast<float2 *>(row + 8 * D) = make_float2(o[n][2] * f[1], o[n][3] * f[1]);
    }
  }
  __syncthreads();
  const long long tile = (static_cast<long long>(b) * p.kv_heads + hk) * p.row_tiles + rt;
  for (int i = tid; i < kAttnRows * D; i += kAttnThreads) {
    const int r = i / D, d = i % D;
    float top = -INFINITY;
    for (int w = 0; w < kAttnWarps; ++w) top = fmaxf(top, ml[w][r].x);
    float sum = 0.f, v = 0.f;
    for (int w = 0; w < kAttnWarps; ++w) {
      // a warp that saw no key has a sum of 0, or NaN where it met NaN alone
      sum += ml[w][r].x == -INFINITY ? ml[w][r].y : ml[w][r].y * exp2f(ml[w][r].x - top);
      v += acc[(w * kAttnRows + r) * D + d];
    }
    if (p.splits > 1) {
      const long long at = (tile * p.splits + split) * kAttnRows + r;
      p.part_o[at * D + d] = v;
      if (d == 0) p.part_ml[at] = make_float2(top, sum);
    } else if (r0 + r <= r_last) {
      const int tok = (r0 + r) / p.group, h = hk * p.group + (r0 + r) % p.group;
      static_cast<T *>(p.out)[(span.first + tok) * p.ldo + h * p.hso + d] =
          from_f32<T>(sum == 0.f ? 0.f : v / sum);
    }
  }
}

// Joins the parts of a row: one warp per row.
template <typename T, int D>
__global__ void __launch_bounds__(128) attn_join_kernel(const LmAttnArgs p) {
  pdl_wait();
  const int lane = threadIdx.x % 32;
  const int b = blockIdx.z, hk = blockIdx.y;
  const SeqSpan span = seq_span(p.cu, b, p.n_seq, p.n_tokens, p.max_q);
  const int row = blockIdx.x * 4 + threadIdx.x / 32;
  if (row >= span.count * p.group) return;
  const long long tile =
      (static_cast<long long>(b) * p.kv_heads + hk) * p.row_tiles + row / kAttnRows;
  const long long at = tile * p.splits * kAttnRows + row % kAttnRows;
  float top = -INFINITY;
  for (int s = 0; s < p.splits; ++s) top = fmaxf(top, p.part_ml[at + s * kAttnRows].x);
  float sum = 0.f, v[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) v[i] = 0.f;
  for (int s = 0; s < p.splits; ++s) {
    const float2 x = p.part_ml[at + s * kAttnRows];
    if (x.x == -INFINITY) {  // nothing visible in this part, or NaN alone
      sum += x.y;
      continue;
    }
    const float f = exp2f(x.x - top);
    sum += x.y * f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
      v[i] += f * p.part_o[(at + s * kAttnRows) * D + lane + 32 * i];
  }
  const int tok = row / p.group, h = hk * p.group + row % p.group;
  T *dst = static_cast<T *>(p.out) + (span.first + tok) * p.ldo + h * p.hso;
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
    dst[lane + 32 * i] = from_f32<T>(sum == 0.f ? 0.f : v[i] / sum);
}

}  // namespace voc
