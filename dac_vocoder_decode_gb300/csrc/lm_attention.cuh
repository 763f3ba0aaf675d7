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

constexpr int kAttnWarps = 4;                      // consumer warps; one more warp copies
constexpr int kAttnThreads = 32 * (kAttnWarps + 1);
constexpr float kLazy = 8.f;    // log2 of how far the weights' maximum may run ahead
constexpr float kPShift = 7.f;  // weights are kept times 2^7 in 16 bits, so below 2^15
constexpr int kShareSeqs = 512;   // sequences up to which CTAs take equal shares of the work
constexpr int kPrRows = 256;      // rows of a tile of the prompt kernel
constexpr int kFlatTiles = 512;   // sequences up to which its CTAs count through the tiles
constexpr int kShareMin = 4;      // units of the smallest share
// Units that a tile counts beside its blocks, for what its first and last steps take.  Measured with 0,
// 4, 8 and 16: 16 sequences of 1 to 10012 tokens 61.5, 24.9, 22.2 and 22.5 us, 8 of 4000 with 16 rows
// 32.0, 29.9, 27.4 and 28.2.
constexpr int kTileCost = 8;

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
  int splits;        // prompt kernel: parts of a tile's keys
  int flat;          // prompt kernel: tiles that CTAs count through, or 0: blockIdx.z is the sequence
  int ctas;          // row kernel: CTAs that share the work, or 0 (one tile each)
  float *part_o;     // partial outputs [slot][row][D] and their maxima and sums [slot][row]
  float2 *part_ml;
  long long budget;
  int *timeout;
};

// The transpose of an 8 x 8 matrix of 16-bit values spread over the warp (row lane/4, columns
// 2 (lane%4) and the next).
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

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
// [2^14, 2^15), or below where that is under 2^-96: f16 then holds bf16 and f16 values exactly, but for
// what lies 2^-28 below it.  bf16's largest values take 2^-113.
__device__ __forceinline__ int query_exponent(uint32_t amax) {
  if (amax == 0) return 0;
  const int e = 14 - (static_cast<int>(amax >> 23) - 127);
  return min(max(e, -113), 110);
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

// Tiles of the prompt kernel for one sequence.
__device__ __forceinline__ int prompt_tiles(const LmAttnArgs &p, const SeqSpan &s) {
  return (s.count * p.group + kPrRows - 1) / kPrRows;
}

// What the row kernel does for one sequence: its rows, the blocks [blk0, blk0 + blocks) that any of
// them sees, and the work in blocks over all key heads and row tiles.
struct SeqWork {
  SeqSpan span;
  long long len, p0;
  int rows, tiles;
  int blk0, blocks;
  int units;
};
// Units of one of its tiles: the first kTileCost stand for the way to its first product and from its
// last one, a unit for each block follows (one for a tile without keys: it has zeros to write).
__device__ __forceinline__ int tile_units(const SeqWork &w) {
  return kTileCost + max(w.blocks, 1);
}
template <int ROWS>
__device__ __forceinline__ SeqWork seq_work(const LmAttnArgs &p, int b) {
  SeqWork w;
  w.span = seq_span(p.cu, b, p.n_seq, p.n_tokens, p.max_q);
  w.len = max(0ll, min(static_cast<long long>(p.lens[b]),
                       static_cast<long long>(p.table_cols) * kBlockTokens));
  w.p0 = static_cast<long long>(p.lens[b]) - w.span.count;
  w.rows = w.span.count * p.group;
  w.tiles = (w.rows + ROWS - 1) / ROWS;
  const long long lo = visible(p, w.p0, w.len).lo;
  const long long hi = visible(p, w.p0 + w.span.count - 1, w.len).hi;
  w.blk0 = static_cast<int>(lo / kBlockTokens);
  w.blocks = hi > lo ? static_cast<int>((hi - 1) / kBlockTokens) + 1 - w.blk0 : 0;
  w.units = tile_units(w) * p.kv_heads * w.tiles;
  return w;
}

// Share of the total work: CTA c has the units [c q, (c + 1) q) in the order (sequence, key head, row
// tile, block), a tile's blocks behind its first kTileCost units.  The host shares only where the
// units fit 30 bits.
__device__ __forceinline__ int share_of(int total, int ctas) {
  return max((total + ctas - 1) / ctas, kShareMin);
}

// Ring stages: as many as leave room for two CTAs on an SM.
template <int D, int NT>
__host__ __device__ constexpr int attn_stages() { return D == 128 ? (NT == 1 ? 6 : 5) : 12; }
template <int D, int NT>
__host__ __device__ constexpr size_t attn_smem() {
  return static_cast<size_t>(attn_stages<D, NT>()) * 2 * kBlockTokens * D +
         sizeof(float) * (kAttnWarps / 2) * 8 * NT * (D + 4) + 128;
}

// One piece of a CTA's share: blocks [first, first + count) of one (sequence, key head, row tile).
struct Segment {
  SeqWork w;
  int b, hk, rt, first, count;
  bool begins, ends;  // the tile's work starts / ends in this CTA
  bool none;          // the share ends before the tile's first block
};

// Rows (queries that share a key head) in tiles of 8 NT, for the few rows of single tokens.  K and
// V blocks come through a ring of shared-memory stages, one bulk copy each; two warps share a
// block, 32 keys each.  The products are taken transposed, S^T = K Q^T and O^T = V^T P^T, so that
// keys and channels fill the MMA's 16 rows and 8 query rows its columns: with few rows the other
// way round would leave most of each product empty.  e4m3 converts exactly to f16, and the weights
// keep 11 bits there (as e4m3 they would keep 4).  The order in which a thread holds channels and
// keys makes its operands whole words of the stored rows; the sums do not depend on it.
//
// A CTA takes a tile, or the CTAs take equal shares of all blocks of all sequences, whatever their
// lengths, and a tile that several CTAs share is joined by attn_join_kernel.  Two CTAs per SM.
//
// Bound by the cache's bytes: 8 sequences of 15504 tokens, 8 key heads of 128 channels (254 MB), 4
// queries a head: 48 us with the join, 5.3 TB/s; in its middle the kernel reads about 7, and some
// 11 us are the launch, the first blocks' way in, CTAs that end at different times, and the join.  With
// 16-row tiles the same call took 59 us (twice the products and registers): 8 rows and fewer have
// tiles of their own.  With the products the other way round and a fixed split of each tile it took
// 76 us.  One sequence of 250 tokens: 4.2 us, latency.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(kAttnThreads, 2) attn_rows_kernel(const LmAttnArgs p) {
  constexpr int kStages = attn_stages<D, NT>();
  constexpr int kBytes = kBlockTokens * D;
  constexpr int kRows = 8 * NT;
  constexpr int kSteps = D / 16;   // MMA steps over the channels, and output tiles of 16 channels
  constexpr int kLd = D + 4;       // row stride of the join buffer: a warp's stores spread over banks
  extern __shared__ __align__(128) uint8_t smem[];
  float *acc = reinterpret_cast<float *>(smem + kStages * 2 * kBytes);  // [two warps][row][kLd]
  __shared__ __align__(8) uint64_t full[kStages], empty[kStages];
  __shared__ int prefix[kShareSeqs + 1];
  __shared__ float2 ml[kAttnWarps][kRows], row_ml[kRows];  // maximum and sum: by warp, together
  __shared__ int abort_flag;
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
  pdl_wait();
  pdl_launch_dependents();
  int lo, hi;  // this CTA's units
  if (p.ctas) {
    for (int i = tid; i < p.n_seq; i += kAttnThreads) prefix[i + 1] = seq_work<kRows>(p, i).units;
    __syncthreads();
    if (warp == 0) {  // running sums, 32 at a time
      int base = 0;
      for (int i0 = 0; i0 < p.n_seq; i0 += 32) {
        int v = i0 + lane < p.n_seq ? prefix[i0 + lane + 1] : 0;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
          const int u = __shfl_up_sync(0xffffffffu, v, o);
          if (lane >= o) v += u;
        }
        if (i0 + lane < p.n_seq) prefix[i0 + lane + 1] = base + v;
        base += __shfl_sync(0xffffffffu, v, 31);
      }
      if (lane == 0) prefix[0] = 0;
    }
    __syncthreads();
    const int total = prefix[p.n_seq], q = share_of(total, p.ctas);
    lo = min(total, static_cast<int>(blockIdx.x) * q);
    hi = min(total, lo + q);
  } else {
    __syncthreads();
    lo = 0, hi = 1;
  }
  if (lo >= hi) return;  // the whole block
  // the piece of work that starts at unit `at`, and the unit after it
  auto segment = [&](int at, int &next) {
    Segment s;
    if (p.ctas) {
      int a = 0, z = p.n_seq - 1;
      while (a < z) {
        const int mid = (a + z + 1) / 2;
        if (prefix[mid] <= at)
          a = mid;
        else
          z = mid - 1;
      }
      s.b = a;
      s.w = seq_work<kRows>(p, a);
      const int per = tile_units(s.w);
      const int tile = (at - prefix[a]) / per;
      const int begin = (at - prefix[a]) % per;
      const int end = min(per, begin + (hi - at));
      s.hk = tile / s.w.tiles, s.rt = tile % s.w.tiles;
      const int from = max(begin - kTileCost, 0), upto = end - kTileCost;  // the tile's blocks
      s.begins = from == 0, s.ends = end == per;
      s.none = upto <= 0;
      s.first = s.w.blk0 + from;
      s.count = s.none ? 0 : min(upto, s.w.blocks) - from;
      next = at + (end - begin);
    } else {
      s.b = blockIdx.z, s.hk = blockIdx.y, s.rt = blockIdx.x;
      s.w = seq_work<kRows>(p, s.b);
      s.begins = s.ends = true;
      s.none = false;
      s.first = s.w.blk0;
      s.count = s.rt < s.w.tiles ? s.w.blocks : 0;
      next = hi;
    }
    return s;
  };

  if (warp == kAttnWarps) {
    // ---------------------------------------------------------------- copies
    int it = 0;
    bool ok = true;
    for (int at = lo, next; at < hi && ok; at = next) {
      const Segment s = segment(at, next);
      const int *table = p.table + s.b * p.ldt;
      // pages of 32 blocks at a time, a lane each, the next 32 while these are copied
      auto fetch = [&](int i) { return i + lane < s.count ? table[s.first + i + lane] : -1; };
      int page = fetch(0);
      for (int i0 = 0; i0 < s.count && ok; i0 += 32) {
        const int next_page = fetch(i0 + 32);
        for (int j = 0; j < 32 && i0 + j < s.count; ++j, ++it) {
          const int st = it % kStages;
          const int pg = __shfl_sync(0xffffffffu, page, j);
          if (it >= kStages) {
            const bool free = mbar_wait(smem_u32(empty + st), (it / kStages - 1) & 1, p.budget,
                                        &abort_flag);
            if (!__all_sync(0xffffffffu, free)) {
              *static_cast<volatile int *>(&abort_flag) = 1;
              ok = false;
              break;
            }
          }
          if (lane == 0) {
            const uint32_t bar = smem_u32(full + st), dst = smem_u32(smem + st * 2 * kBytes);
            if (pg < 0 || pg >= p.n_pages) {
              mbar_arrive(bar);
            } else {
              const long long from = (static_cast<long long>(pg) * p.kv_heads + s.hk) * kBytes;
              mbar_arrive_expect_tx(bar, 2 * kBytes);
              bulk_load(dst, p.kc + from, kBytes, bar);
              bulk_load(dst + kBytes, p.vc + from, kBytes, bar);
            }
          }
        }
        page = next_page;
      }
    }
    if (!ok && lane == 0) {  // leave with no copy in flight
      const int never = 0;
      for (int i = max(0, it - kStages); i < it; ++i)
        mbar_wait(smem_u32(full + i % kStages), (i / kStages) & 1, p.budget, &never);
      if (p.timeout) *p.timeout = 1;
    }
    return;
  }

  // ------------------------------------------------------------------ products
  const int pair = warp / 2, half = warp % 2;
  int it = 0;
  bool ok = true;
  for (int at = lo, next; at < hi; at = next) {
    const Segment s = segment(at, next);
    const int r0 = s.rt * kRows, r_last = min(s.w.rows, r0 + kRows) - 1;
    if (r0 > r_last || s.none) continue;  // whole-tile launches cover max_q tokens
    // scales of this warp's blocks (every other one): loaded one of them ahead of their use, the
    // pages two ahead
    const int *table = p.table + s.b * p.ldt + s.first;
    const int i_first = (it ^ pair) & 1;
    auto page_at = [&](int i) {
      const int page = i < s.count ? table[i] : -1;
      return page >= 0 && page < p.n_pages ? page : -1;
    };
    float ks = 1.f, vs = 1.f;
    auto load_scales = [&](int page) {
      const long long slot = static_cast<long long>(page) * p.kv_heads + s.hk;
      ks = page >= 0 ? p.ks[slot] : 1.f, vs = page >= 0 ? p.vs[slot] : 1.f;
    };
    int page = page_at(i_first), page2 = page_at(i_first + 2);
    load_scales(page);
    // queries as the second operand: row g of each 8 rows, two halves of f16 per step
    uint32_t qb[NT][kSteps][2];
    float qc[NT][2];
    int see_lo[NT][2], see_hi[NT][2];  // of rows 2t and 2t + 1, relative to the segment's first key
    const long long key0 = static_cast<long long>(s.first) * kBlockTokens;
    const long long key_lo = visible(p, s.w.p0 + r0 / p.group, s.w.len).lo;
    const long long key_hi = visible(p, s.w.p0 + r_last / p.group, s.w.len).hi;
    auto rel = [&](long long key) {
      return static_cast<int>(max(-1ll, min(key - key0, 0x7fffffffll)));
    };
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = min(r0 + 8 * n + g, r_last);  // spare rows repeat the last one
      const T *src = static_cast<const T *>(p.q) +
                     (s.w.span.first + r / p.group) * p.ldq + (s.hk * p.group + r % p.group) * p.hsq;
      const bool vec = (reinterpret_cast<uintptr_t>(src) & 15) == 0;
      uint4 raw[D / 64][2];
      uint32_t a = 0;
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const T *at16 = src + 64 * c + 16 * t + 8 * h;
          if (vec) {
            raw[c][h] = *reinterpret_cast<const uint4 *>(at16);
          } else {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint16_t *u = reinterpret_cast<const uint16_t *>(at16) + 2 * j;
              w[j] = u[0] | static_cast<uint32_t>(u[1]) << 16;
            }
            raw[c][h] = make_uint4(w[0], w[1], w[2], w[3]);
          }
          float f[8];
          Vec16<T>::unpack(raw[c][h], f);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (abs_bits(f[j]) < kInfBits) a = max(a, abs_bits(f[j]));
        }
      a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
      a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
      const int e = query_exponent(a);
      const float up = p.scale_log2 < 0.f ? -pow2(e) : pow2(e);  // scores are scaled by >= 0
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float f[8];
          Vec16<T>::unpack(raw[c][h], f);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            qb[n][4 * c + 2 * h + j / 2][j % 2] = f16x2(f[2 * j] * up, f[2 * j + 1] * up);
        }
      const float mine = fabsf(p.scale_log2) * pow2(-e);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        qc[n][x] = __shfl_sync(0xffffffffu, mine, 4 * (2 * t + x));
        const int rr = min(r0 + 8 * n + 2 * t + x, r_last);
        const KeySpan k = visible(p, s.w.p0 + rr / p.group, s.w.len);
        see_lo[n][x] = rel(k.lo), see_hi[n][x] = rel(k.hi);
      }
    }
    const int all_lo = rel(visible(p, s.w.p0 + r_last / p.group, s.w.len).lo);   // seen by every row
    const int all_hi = rel(visible(p, s.w.p0 + r0 / p.group, s.w.len).hi);
    const int any_lo = rel(key_lo), any_hi = rel(key_hi);                        // seen by some row

    float o[NT][kSteps][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[n][i][j] = 0.f;
      m[n][0] = m[n][1] = -INFINITY, l[n][0] = l[n][1] = 0.f;
    }

    for (int i = i_first; i < s.count; i += 2) {
      const int st = (it + i) % kStages;
      const int base = i * kBlockTokens + 32 * half;  // relative to key0
      const bool use = page >= 0 && base < any_hi && base + 32 > any_lo;
      const float k_scale = ks, v_scale = fmaxf(vs, kScaleMin);
      page = page2;
      load_scales(page);
      page2 = page_at(i + 4);
      if (ok) {
        ok = mbar_wait(smem_u32(full + st), ((it + i) / kStages) & 1, p.budget, &abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) *static_cast<volatile int *>(&abort_flag) = 1;
      }
      if (ok && use) {
        const float lvs = log2f(v_scale), ivs = 1.f / v_scale;
        const uint32_t kb = smem_u32(smem + st * 2 * kBytes), vb = kb + kBytes;
        // scores: row g (g + 8) of tile j is key 8 (g / 2) + 4 j + g % 2 (+ 2)
        float sc[NT][2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) sc[n][j][x] = 0.f;
          const uint32_t row = kb + (32 * half + 8 * (g >> 1) + 4 * j + (g & 1)) * D + 16 * t;
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            const uint4 w0 = lds128(row + 64 * c), w1 = lds128(row + 2 * D + 64 * c);
            const uint32_t a0[4] = {w0.x, w0.y, w0.z, w0.w}, a1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t a[4] = {e4m3x2_to_f16x2(a0[k] & 0xffff), e4m3x2_to_f16x2(a1[k] & 0xffff),
                                     e4m3x2_to_f16x2(a0[k] >> 16), e4m3x2_to_f16x2(a1[k] >> 16)};
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mma_f16(sc[n][j], a, qb[n][4 * c + k][0], qb[n][4 * c + k][1]);
            }
          }
        }
        if (base < all_lo || base + 32 > all_hi) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const int key = base + 8 * (g >> 1) + 4 * j + (g & 1) + x / 2 * 2;
                if (key < see_lo[n][x % 2] || key >= see_hi[n][x % 2]) sc[n][j][x] = -INFINITY;
              }
        }
        // u = s + log2(vs); the maximum is raised only when some weight would leave f16
        bool raise = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float c = fmaxf(qc[n][x] * k_scale, 1e-37f);  // above 0: masked scores stay -inf
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              sc[n][j][x] = fmaf(sc[n][j][x], c, lvs);
              sc[n][j][x + 2] = fmaf(sc[n][j][x + 2], c, lvs);
            }
            const float top = fmaxf(fmaxf(sc[n][0][x], sc[n][0][x + 2]),
                                    fmaxf(sc[n][1][x], sc[n][1][x + 2]));
            raise |= top > m[n][x] + kLazy;
          }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float top = fmaxf(fmaxf(sc[n][0][x], sc[n][0][x + 2]),
                                fmaxf(sc[n][1][x], sc[n][1][x + 2]));
#pragma unroll
              for (int z = 4; z < 32; z *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, z));
              const float nm = fmaxf(m[n][x], top);
              const float alpha = m[n][x] == nm ? 1.f : ex2(m[n][x] - nm);
              m[n][x] = nm;
              l[n][x] *= alpha;
#pragma unroll
              for (int i2 = 0; i2 < kSteps; ++i2) o[n][i2][x] *= alpha, o[n][i2][x + 2] *= alpha;
            }
        }
        uint32_t pb[NT][2][2];  // weights as the second operand: keys by row
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float off[2], sum[2] = {0.f, 0.f};
#pragma unroll
          for (int x = 0; x < 2; ++x) off[x] = (m[n][x] == -INFINITY ? 0.f : m[n][x]) - kPShift;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float w[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              w[x] = ex2(sc[n][j][x] - off[x % 2]);
              sum[x % 2] += w[x];
            }
            pb[n][j][0] = transpose8(f16x2(w[0], w[1]));
            pb[n][j][1] = transpose8(f16x2(w[2], w[3]));
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) l[n][x] = fmaf(sum[x], ivs, l[n][x]);
        }
        // codes of keys that no row sees count as zero, whatever they hold
        uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
        if (base < any_lo || base + 32 > any_hi) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int key = base + 8 * t + j;
            if (key < any_lo || key >= any_hi) keep[j / 4] &= ~(0xffu << 8 * (j % 4));
          }
        }
#pragma unroll
        for (int i2 = 0; i2 < kSteps; ++i2) {
          uint32_t v[2][2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                         : "=r"(v[x][0]), "=r"(v[x][1])
                         : "r"(vb + (16 * i2 + 8 * x + g) * kBlockTokens + 32 * half + 8 * t)
                         : "memory");
            v[x][0] &= keep[0], v[x][1] &= keep[1];
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t a[4] = {e4m3x2_to_f16x2(v[0][j] & 0xffff),
                                   e4m3x2_to_f16x2(v[1][j] & 0xffff),
                                   e4m3x2_to_f16x2(v[0][j] >> 16), e4m3x2_to_f16x2(v[1][j] >> 16)};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_f16(o[n][i2], a, pb[n][j][0], pb[n][j][1]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(empty + st));
    }
    it += s.count;

    // join the warps: each scales its rows to the common maximum
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int z = 4; z < 32; z *= 2) l[n][x] += __shfl_xor_sync(0xffffffffu, l[n][x], z);
        if (g == 0) ml[warp][8 * n + 2 * t + x] = make_float2(m[n][x], l[n][x]);
      }
    asm volatile("bar.sync 1, 128;" ::: "memory");
    if (tid < kRows) {
      float top = -INFINITY, sum = 0.f;
      for (int w = 0; w < kAttnWarps; ++w) top = fmaxf(top, ml[w][tid].x);
      for (int w = 0; w < kAttnWarps; ++w)
        // a warp that saw no key has a sum of 0, or NaN where it met NaN alone
        sum += ml[w][tid].x == -INFINITY ? ml[w][tid].y : ml[w][tid].y * ex2(ml[w][tid].x - top);
      row_ml[tid] = make_float2(top, sum);
    }
    // warps 2 and 3 hand their parts to 0 and 1, which add their own
#pragma unroll
    for (int turn = 1; turn >= 0; --turn) {
      if (warp / 2 == turn) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float top = -INFINITY;
            for (int w = 0; w < kAttnWarps; ++w) top = fmaxf(top, ml[w][8 * n + 2 * t + x].x);
            const float f = top == -INFINITY ? 0.f : ex2(m[n][x] - top);
            float *row = acc + (warp % 2 * kRows + 8 * n + 2 * t + x) * kLd + g;
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
              row[16 * i] = fmaf(o[n][i][x], f, turn ? 0.f : row[16 * i]);
              row[16 * i + 8] = fmaf(o[n][i][x + 2], f, turn ? 0.f : row[16 * i + 8]);
            }
          }
      }
      asm volatile("bar.sync 1, 128;" ::: "memory");
    }
    for (int i = tid; i < kRows * D / 4; i += 32 * kAttnWarps) {
      const int r = i / (D / 4), d = i % (D / 4) * 4;
      if (r0 + r > r_last) break;
      const float4 a0 = *reinterpret_cast<const float4 *>(acc + r * kLd + d);
      const float4 a1 = *reinterpret_cast<const float4 *>(acc + (kRows + r) * kLd + d);
      const float v[4] = {a0.x + a1.x, a0.y + a1.y, a0.z + a1.z, a0.w + a1.w};
      if (s.begins && s.ends) {
        const int tok = (r0 + r) / p.group, h = s.hk * p.group + (r0 + r) % p.group;
        T *dst = static_cast<T *>(p.out) + (s.w.span.first + tok) * p.ldo + h * p.hso + d;
        const float sum = row_ml[r].y, inv = 1.f / sum;
        float f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = sum == 0.f ? 0.f : v[j] * inv;
        if (reinterpret_cast<uintptr_t>(dst) % 8 == 0) {
          *reinterpret_cast<uint2 *>(dst) = make_uint2(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]));
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) dst[j] = from_f32<T>(f[j]);
        }
      } else {  // slot 2c: the tile began in an earlier CTA, 2c + 1: it begins here
        const long long slot = (2ll * blockIdx.x + (s.begins ? 1 : 0)) * kRows + r;
        *reinterpret_cast<float4 *>(p.part_o + slot * D + d) = make_float4(v[0], v[1], v[2], v[3]);
        if (d == 0) p.part_ml[slot] = row_ml[r];
      }
    }
    asm volatile("bar.sync 1, 128;" ::: "memory");  // the buffers are free for the next piece
  }
}

// Joins the parts of a row kernel's tile, one CTA of D threads per row, a channel each.  Bound by its
// chain of reads, lengths, maxima and values: with barriers between the latter it took 3 us more.
template <typename T, int D, int ROWS>
__global__ void __launch_bounds__(D) attn_join_kernel(const LmAttnArgs p) {
  constexpr int kWarps = D / 32;
  __shared__ int counts[2][kWarps];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int b = blockIdx.z, hk = blockIdx.y, row = blockIdx.x;
  // Lengths and counts too are read after the wait: they may come from the kernel before the one that
  // this one follows, and nothing else makes that one's stores visible here.
  pdl_wait();
  pdl_launch_dependents();
  const SeqSpan span = seq_span(p.cu, b, p.n_seq, p.n_tokens, p.max_q);
  // the work before this sequence and in all, as attn_rows_kernel counts it
  int both[2] = {0, 0};
  for (int i = tid; i < p.n_seq; i += D) {
    const int u = seq_work<ROWS>(p, i).units;
    both[1] += u;
    if (i < b) both[0] += u;
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
#pragma unroll
    for (int o = 16; o; o /= 2) both[k] += __shfl_xor_sync(0xffffffffu, both[k], o);
    if (lane == 0) counts[k][warp] = both[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    both[k] = 0;
    for (int w = 0; w < kWarps; ++w) both[k] += counts[k][w];
  }
  const SeqWork w = seq_work<ROWS>(p, b);
  const int per = tile_units(w);
  const int q = share_of(both[1], p.ctas);
  const int at = both[0] + (hk * w.tiles + row / ROWS) * per;
  const int c0 = (at + kTileCost) / q, c1 = (at + per - 1) / q;
  if (row >= span.count * p.group || c0 == c1) return;  // c0 == c1: one CTA had the whole tile
  const int parts = c1 - c0 + 1;
  auto slot_of = [&](int s) {
    return (s == 0 ? 2ll * c0 + 1 : 2ll * (c0 + s)) * ROWS + row % ROWS;
  };
  // Every warp weighs the parts for itself, a lane each, without a barrier.  The first values are
  // fetched beside the maxima: what the join takes is its chain of reads.
  constexpr int kEarly = 8;
  float early[kEarly], top = -INFINITY;
  for (int s = lane; s < parts; s += 32) top = fmaxf(top, p.part_ml[slot_of(s)].x);
#pragma unroll
  for (int s = 0; s < kEarly; ++s) early[s] = s < parts ? p.part_o[slot_of(s) * D + tid] : 0.f;
#pragma unroll
  for (int o = 16; o; o /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  float sum = 0.f, v = 0.f;
  for (int s0 = 0; s0 < parts; s0 += 32) {
    float f = 0.f;
    if (s0 + lane < parts) {
      const float2 x = p.part_ml[slot_of(s0 + lane)];
      // a part that saw no key has a sum of 0, or NaN where it met NaN alone
      f = x.x == -INFINITY ? 0.f : ex2(x.x - top);
      sum += x.x == -INFINITY ? x.y : x.y * f;
    }
    if (s0 == 0) {
#pragma unroll
      for (int s = 0; s < kEarly; ++s) v = fmaf(__shfl_sync(0xffffffffu, f, s), early[s], v);
    }
    const int n = min(32, parts - s0);
#pragma unroll 8
    for (int s = s0 ? 0 : kEarly; s < n; ++s)
      v = fmaf(__shfl_sync(0xffffffffu, f, s), p.part_o[slot_of(s0 + s) * D + tid], v);
  }
#pragma unroll
  for (int o = 16; o; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const int tok = row / p.group, h = hk * p.group + row % p.group;
  static_cast<T *>(p.out)[(span.first + tok) * p.ldo + h * p.hso + tid] =
      from_f32<T>(sum == 0.f ? 0.f : v / sum);
}

// The sequence that the prompt kernel's tile `index` (counted over all sequences) is of, or -1, and
// which of its tiles that is.  For whole warps.
__device__ __forceinline__ int find_tile(const LmAttnArgs &p, int index, int lane, int &nth) {
  int b = -1;
  for (int i0 = 0, before = 0; i0 < p.n_seq && b < 0; i0 += 32) {
    const int tiles =
        i0 + lane < p.n_seq
            ? prompt_tiles(p, seq_span(p.cu, i0 + lane, p.n_seq, p.n_tokens, p.max_q)) : 0;
    int upto = tiles;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int u = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += u;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, before + upto > index);
    if (past) {
      const int at = __ffs(past) - 1;
      b = i0 + at;
      nth = index - before - __shfl_sync(0xffffffffu, upto - tiles, at);
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  return b;
}

// Joins the parts of the prompt kernel's tiles, a warp per row.  One CTA per row of the longest chunk
// and sequence took 25 us for 8 chunks of 1 to 200 tokens, most of them for rows that are not there.
constexpr int kJoinRows = 8;
template <typename T, int D>
__global__ void __launch_bounds__(32 * kJoinRows) attn_join_tiles_kernel(const LmAttnArgs p) {
  constexpr int kPer = D / 32;  // channels of a lane
  const int lane = threadIdx.x % 32, hk = blockIdx.y;
  int nth = 0;
  pdl_wait();  // ahead of the counts too (attn_join_kernel)
  pdl_launch_dependents();
  const int b = find_tile(p, blockIdx.x, lane, nth);
  if (b < 0) return;
  const SeqSpan span = seq_span(p.cu, b, p.n_seq, p.n_tokens, p.max_q);
  const int local = blockIdx.z * kJoinRows + threadIdx.x / 32, row = nth * kPrRows + local;
  if (row >= span.count * p.group) return;
  const long long tile = static_cast<long long>(blockIdx.x) * p.kv_heads + hk;
  auto slot_of = [&](int s) { return (tile * p.splits + s) * kPrRows + local; };
  float top = -INFINITY;
  for (int s = lane; s < p.splits; s += 32) top = fmaxf(top, p.part_ml[slot_of(s)].x);
#pragma unroll
  for (int o = 16; o; o /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  float sum = 0.f, v[kPer] = {};
  for (int s0 = 0; s0 < p.splits; s0 += 32) {
    float f = 0.f;
    if (s0 + lane < p.splits) {
      const float2 x = p.part_ml[slot_of(s0 + lane)];
      // a part that saw no key has a sum of 0, or NaN where it met NaN alone
      f = x.x == -INFINITY ? 0.f : ex2(x.x - top);
      sum += x.x == -INFINITY ? x.y : x.y * f;
    }
    const int n = min(32, p.splits - s0);
#pragma unroll 4
    for (int s = 0; s < n; ++s) {
      const float g = __shfl_sync(0xffffffffu, f, s);
      const float *from = p.part_o + slot_of(s0 + s) * D + kPer * lane;
      float o[kPer];
      if constexpr (kPer == 4) {
        const float4 w = *reinterpret_cast<const float4 *>(from);
        o[0] = w.x, o[1] = w.y, o[2] = w.z, o[3] = w.w;
      } else {
        const float2 w = *reinterpret_cast<const float2 *>(from);
        o[0] = w.x, o[1] = w.y;
      }
#pragma unroll
      for (int k = 0; k < kPer; ++k) v[k] = fmaf(g, o[k], v[k]);
    }
  }
#pragma unroll
  for (int o = 16; o; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const int tok = row / p.group, h = hk * p.group + row % p.group;
  T *dst = static_cast<T *>(p.out) + (span.first + tok) * p.ldo + h * p.hso + kPer * lane;
#pragma unroll
  for (int k = 0; k < kPer; ++k) v[k] = sum == 0.f ? 0.f : v[k] / sum;
  if (reinterpret_cast<uintptr_t>(dst) % 4 == 0) {
#pragma unroll
    for (int k = 0; k < kPer; k += 2)
      reinterpret_cast<uint32_t *>(dst)[k / 2] = pack2<T>(v[k], v[k + 1]);
  } else {
#pragma unroll
    for (int k = 0; k < kPer; ++k) dst[k] = from_f32<T>(v[k]);
  }
}

}  // namespace voc
