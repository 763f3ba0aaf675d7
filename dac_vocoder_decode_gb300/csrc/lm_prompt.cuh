// lm_prompt.cuh -- the attention of lm_attention.cuh for many queries of a sequence at once, on
// the 5th-generation tensor cores.
//
// A CTA takes 256 rows (queries that share a key head) as two tiles of 128 and walks over its keys
// one cache block of 64 at a time:
//   warps 0..3, 4..7   one thread per row of the first / second row tile: softmax of the scores
//   warps 8..11        convert K and V codes to f16 (exact) in shared memory
//   warps 12, 13       issue the scores' products S = Q K^T of the first / second row tile
//   warps 14, 15       issue the outputs' products O += P V of the first / second row tile
// One warp for both products of a row tile was the slowest part: its waits, commits and issues, one
// after the other, took longer than the products.
// The softmax threads take a tile's scores into registers and give them free at once, and P has a
// place of its own, so a row tile's next scores are computed while its softmax is at work: neither
// waits for the other in turn.  First operands come from tensor memory where it has room for them (at
// 128 channels it is full with 2 x (128 O + 64 S + 32 P) + 64 Q columns: the second tile's Q stays in
// shared memory), since a 128-row operand in shared memory costs each step 4 KB of its bandwidth
// beside the conversions' stores.
// Operands are 16-bit: the codes are exact in f16 and the weights keep 11 bits, where an e4m3
// product would round queries and weights to 4.
//
// The weights of a tile are taken against the maximum of the tiles before it, in one pass over the
// scores; only where one comes out 2^8 or more too large (weights are kept times 2^7, so 2^15 in f16)
// are the row's maximum raised, the accumulator rescaled and the tile's weights taken again.
//
// Measured: one prompt of 15504 tokens, 16 heads on 4 of 128 channels: 830 us, 1.19 PFLOP/s (the 16-bit
// products alone would take 517).  Bound by the handshakes of a key tile (with the exponentials,
// conversions and most products left out 8192 tokens still took 245 of 264 us) and by the converting
// warps' loads (fetched one tile ahead instead of two: 919 us).  What was slower: tiles of 128 keys
// (974, no room for scores and weights apart), two threads a row (1070), 8 converting warps (1044,
// fewer registers for each).
#pragma once
#include <type_traits>

#include "lm_attention.cuh"

namespace voc {

constexpr int kPrThreads = 512;
constexpr int kPrStages = 4;       // key tiles in shared memory
// Registers: 256 softmax threads, 128 converting, 128 others: 256 x 184 + 128 x 104 + 128 x 40 =
// 65536, the block's registers at launch (512 x 128).
constexpr int kPrSoftRegs = 184, kPrConvRegs = 104, kPrRestRegs = 40;
static_assert(256 * kPrSoftRegs + 128 * kPrConvRegs + 128 * kPrRestRegs <= 512 * 128, "registers");

template <int D>
struct PromptSmem {
  static constexpr int kSlab = kBlockTokens * 128;      // 64 keys of 64 f16 values
  static constexpr int kK = D / 64 * kSlab;             // one key tile
  static constexpr int kV = D * 128;                    // D rows of 64 keys
  static constexpr int kQ = D == 64 ? 0 : 2 * 128 * 128;  // the second row tile's queries
  static constexpr size_t kBytes = kPrStages * (kK + kV) + kQ + 1024;
};

// The 16-byte unit `u` of a 128-byte row `r` in the 128-byte swizzle.
__device__ __forceinline__ uint32_t sw128(int r, int u) { return r * 128 + ((u ^ (r & 7)) << 4); }

// 16 codes to 16 halves, stored as units u and u + 1 of a swizzled row.
__device__ __forceinline__ void store_codes(uint32_t tile, int row, int u, const uint4 &c) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t h[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[2 * i] = e4m3x2_to_f16x2(w[i] & 0xffff);
    h[2 * i + 1] = e4m3x2_to_f16x2(w[i] >> 16);
  }
  sts128(tile + sw128(row, u), make_uint4(h[0], h[1], h[2], h[3]));
  sts128(tile + sw128(row, u + 1), make_uint4(h[4], h[5], h[6], h[7]));
}

template <typename T, int D>
__global__ void __launch_bounds__(kPrThreads, 1) attn_prompt_kernel(const LmAttnArgs p) {
  using S = PromptSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base_ptr = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sk = smem_u32(base_ptr), sv = sk + kPrStages * S::kK, sq = sv + kPrStages * S::kV;
  // [row tile][stage]: s_full -- the scores of a key tile are there and its K stage is free again;
  // p_empty -- its weights and its V stage are
  __shared__ __align__(8) uint64_t q_full, k_full[kPrStages], v_full[kPrStages],
      s_full[2][kPrStages], p_empty[2][kPrStages], s_empty[2], p_full[2], sc_full[2], sc_empty[2],
      o_full[2], drain[2];
  __shared__ float4 scales[2][32];  // key scale, log2 and reciprocal of the value scale, by tile
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, wg = warp / 4;
  volatile int *abort = &abort_flag;
  const int never = 0;

  const int hk = blockIdx.y;
  int b = blockIdx.z, split = 0, nth = blockIdx.x;  // nth: which of the sequence's tiles
  pdl_wait();
  if (p.flat) {
    split = blockIdx.z;
    b = find_tile(p, blockIdx.x, lane, nth);  // no CTAs for tiles that short chunks do not have
    if (b < 0) return;  // the whole block, before any barrier or allocation
  }
  const SeqSpan span = seq_span(p.cu, b, p.n_seq, p.n_tokens, p.max_q);
  const int rows = span.count * p.group;
  // the latest rows see the most keys: they start first
  const int r0 = (prompt_tiles(p, span) - 1 - nth) * kPrRows;
  if (r0 < 0) return;  // likewise
  const int r_last = min(rows, r0 + kPrRows) - 1;
  const bool two = r_last - r0 >= 128;  // the second row tile has rows
  if (tid == 0) {
    mbar_init(smem_u32(&q_full), 8);  // one arrival per warp, here and below
    for (int i = 0; i < kPrStages; ++i) {
      mbar_init(smem_u32(k_full + i), 4);
      mbar_init(smem_u32(v_full + i), 4);
      for (int t = 0; t < 2; ++t) {
        mbar_init(smem_u32(&s_full[t][i]), 1);
        mbar_init(smem_u32(&p_empty[t][i]), 1);
      }
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(s_empty + i), 4);
      mbar_init(smem_u32(p_full + i), 4);
      mbar_init(smem_u32(sc_full + i), 1);
      mbar_init(smem_u32(sc_empty + i), two ? 8 : 4);
      mbar_init(smem_u32(o_full + i), 1);
      mbar_init(smem_u32(drain + i), 1);
    }
    abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 12) {
    tmem_alloc(smem_u32(&tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // Only now: a later kernel's CTA that came before this allocation and took columns on this SM would
  // wait for this grid while this grid waited for its columns.
  pdl_launch_dependents();
  const uint32_t tmem = tmem_slot;  // columns: two outputs, two scores, two weights, queries
  constexpr uint32_t kColS = 2 * D, kColP = kColS + 2 * kBlockTokens, kColQ = kColP + kBlockTokens;
  const long long len = max(0ll, min(static_cast<long long>(p.lens[b]),
                                     static_cast<long long>(p.table_cols) * kBlockTokens));
  const long long p0 = static_cast<long long>(p.lens[b]) - span.count;
  const long long key_lo = visible(p, p0 + r0 / p.group, len).lo;
  const long long key_hi = visible(p, p0 + r_last / p.group, len).hi;
  const long long tile0 = key_lo / kBlockTokens;
  const long long n_all = key_hi > key_lo ? (key_hi - 1) / kBlockTokens + 1 - tile0 : 0;
  const long long per = (n_all + p.splits - 1) / p.splits;
  const long long first = tile0 + min(n_all, split * per);
  const int n = static_cast<int>(min(n_all, (split + 1) * per) - min(n_all, split * per));
  // page of key tile kt (not yet checked: a use right behind the load would wait for it)
  const int *table = p.table + b * p.ldt + first;
  auto page_of = [&](int kt) { return kt < n ? table[kt] : -1; };
  // A wait that runs out raises the flag, and everybody goes on without waiting: the loops keep their
  // shape (their warps stay together) and end, with a result that the caller is told not to use.
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    if (!mbar_wait(smem_u32(bar), parity, p.budget, abort)) *abort = 1;
    __syncwarp();
  };
  // one arrival for the warp: 32 of them on one barrier would queue up in shared memory
  auto arrive = [&](uint64_t *bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(bar));
  };
  auto known = [&](int page) { return page >= 0 && page < p.n_pages; };

  if (wg < 2) {
    regs_inc<kPrSoftRegs>();
    const int local = tid % 128;                 // row of the tile, lane of the accumulator
    const int r = min(r0 + wg * 128 + local, r_last);
    const bool live = r0 + wg * 128 + local <= r_last;
    const int tok = r / p.group, head = hk * p.group + r % p.group;
    const KeySpan see = visible(p, p0 + tok, len);
    const float flip = p.scale_log2 < 0.f ? -1.f : 1.f;  // scores are scaled by a value >= 0
    float qc;
    {
      const T *src = static_cast<const T *>(p.q) + (span.first + tok) * p.ldq + head * p.hsq;
      const bool vec = (reinterpret_cast<uintptr_t>(src) & 15) == 0;
      uint4 raw[D / 8];
      uint32_t a = 0;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        if (!live) {
          raw[i] = make_uint4(0, 0, 0, 0);
        } else if (vec) {
          raw[i] = reinterpret_cast<const uint4 *>(src)[i];
        } else {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint16_t *s16 = reinterpret_cast<const uint16_t *>(src) + 8 * i + 2 * j;
            w[j] = s16[0] | static_cast<uint32_t>(s16[1]) << 16;
          }
          raw[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        float f[8];
        Vec16<T>::unpack(raw[i], f);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (abs_bits(f[j]) < kInfBits) a = max(a, abs_bits(f[j]));
      }
      const int e = query_exponent(a);
      const float up = pow2(e) * flip;
      qc = fabsf(p.scale_log2) * pow2(-e);
      uint32_t h[D / 2];
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        float f[8];
        Vec16<T>::unpack(raw[i], f);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[4 * i + j] = f16x2(f[2 * j] * up, f[2 * j + 1] * up);
      }
      if (D == 64 || wg == 0) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
          tmem_st32(tmem + (static_cast<uint32_t>((warp % 4) * 32) << 16) + kColQ + wg * (D / 2) +
                        32 * i, h + 32 * i);
        tmem_st_wait();
      } else {
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
          sts128(sq + i / 8 * (128 * 128) + sw128(local, i % 8),
                 make_uint4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]));
        fence_proxy_async_smem();
      }
    }
    tc_fence_before();
    arrive(&q_full);

    const uint32_t lane_base = static_cast<uint32_t>((warp % 4) * 32) << 16;
    const uint32_t s_addr = tmem + lane_base + kColS + wg * kBlockTokens;
    const uint32_t p_addr = tmem + lane_base + kColP + wg * (kBlockTokens / 2);
    const uint32_t o_addr = tmem + lane_base + wg * D;
    float m = -INFINITY, l = 0.f;
    if (wg == 0 || two) {
      // key tiles that every row of the warp sees whole: [whole0, whole1)
      const int whole0 = __reduce_max_sync(
          0xffffffffu, static_cast<int>(min(static_cast<long long>(n),
                                            max(0ll, (see.lo + kBlockTokens - 1) / kBlockTokens - first))));
      const int whole1 = __reduce_min_sync(
          0xffffffffu, static_cast<int>(min(static_cast<long long>(n),
                                            max(0ll, see.hi / kBlockTokens - first))));
      for (int kt = 0; kt < n; ++kt) {
        const uint32_t st = static_cast<uint32_t>(kt) % kPrStages;
        const uint32_t ph = static_cast<uint32_t>(kt) / kPrStages & 1;
        if (kt % 32 == 0) wait(sc_full + (kt >> 5 & 1), kt >> 6 & 1);
        const float4 block = scales[kt >> 5 & 1][kt & 31];
        const float c = fmaxf(qc * block.x, 1e-37f);  // above 0: masked scores stay -inf
        const float lvs = block.y, ivs = block.z;
        wait(&s_full[wg][st], ph);
        tc_fence_after();
        uint32_t sc[kBlockTokens];
        tmem_ld32_issue(s_addr, sc);
        tmem_ld32_issue(s_addr + 32, sc + 32);
        tmem_ld_wait_all();
        tmem_ld32_after_wait(sc);
        tmem_ld32_after_wait(sc + 32);
        tc_fence_before();
        arrive(s_empty + wg);
        if (kt < whole0 || kt >= whole1) {  // the row's keys of this tile
          const long long base = (first + kt) * kBlockTokens;
          const int from = static_cast<int>(max(-1ll, min(see.lo - base, 64ll)));
          const int upto = static_cast<int>(max(-1ll, min(see.hi - base, 64ll)));
#pragma unroll
          for (int i = 0; i < kBlockTokens; ++i)
            if (i < from || i >= upto) sc[i] = 0xff800000u;
        }
        uint32_t w[kBlockTokens / 2];
        bool raise = kt == 0, mine = raise;  // for some row of the warp, for this row
        while (true) {
          if (raise) {  // a look at the maximum, and the row's weights taken against it from here on
            float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < kBlockTokens; ++i) t[i % 4] = fmaxf(t[i % 4], __uint_as_float(sc[i]));
            // (a row that did not ask for it stays as it is, whoever its neighbours are)
            const float nm =
                mine ? fmaxf(m, fmaf(fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])), c, lvs)) : m;
            const float alpha = nm == m ? 1.f : ex2(m - nm);
            m = nm;
            l *= alpha;
            if (kt > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
              wait(&p_empty[wg][(kt - 1) % kPrStages], (kt - 1) / kPrStages & 1);  // O is at rest
              tc_fence_after();
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                uint32_t o[16];
                tmem_ld16_issue(o_addr + 16 * i, o);
                tmem_ld16_wait(o);
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
                tmem_st16(o_addr + 16 * i, o);
              }
            }
          }
          const float d = lvs - ((m == -INFINITY ? 0.f : m) - kPShift);
          const float2 cc = make_float2(c, c), dd = make_float2(d, d);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int i = 0; i < kBlockTokens / 2; ++i) {
            float2 u = fma2(make_float2(__uint_as_float(sc[2 * i]), __uint_as_float(sc[2 * i + 1])),
                            cc, dd);
            u.x = ex2(u.x), u.y = ex2(u.y);
            sum[i % 2] = add2(sum[i % 2], u);
            w[i] = f16x2(u.x, u.y);
          }
          // the weights' sum bounds them: below 2^15 (and not NaN) all fit in f16; a row that has
          // seen no key yet needs its first maximum
          const float all = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          if (!raise) {
            mine = !(all < 32768.f) || m == -INFINITY;
            raise = __any_sync(0xffffffffu, mine);
            if (raise) continue;
          }
          l = fmaf(all, ivs, l);
          break;
        }
        // the last weights are used up
        if (kt > 0) wait(&p_empty[wg][(kt - 1) % kPrStages], (kt - 1) / kPrStages & 1);
        tc_fence_after();
        tmem_st32(p_addr, w);
        tmem_st_wait();
        tc_fence_before();
        arrive(p_full + wg);
        if (kt % 32 == 31) arrive(sc_empty + (kt >> 5 & 1));
      }
    }
    // outputs
    if (n > 0 && (wg == 0 || two)) {
      const bool done = mbar_wait(smem_u32(o_full + wg), 0, 4 * p.budget, &never);
      if (!__all_sync(0xffffffffu, done)) *abort = 1;
      tc_fence_after();
    }
    if (wg == 0 || two) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      T *dst = static_cast<T *>(p.out) + (span.first + tok) * p.ldo + head * p.hso;
      const bool vec = (reinterpret_cast<uintptr_t>(dst) & 15) == 0;
      // the parts of a tile: [tile, its sequence's first one first][head][split][row]
      const long long tile = static_cast<long long>(blockIdx.x) - nth + r0 / kPrRows;
      const long long at = ((tile * p.kv_heads + hk) * p.splits + split) * kPrRows + r - r0;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        uint32_t o[32];
        if (n > 0) {
          tmem_ld32_issue(o_addr + 32 * i, o);
          tmem_ld_wait_all();
          tmem_ld32_after_wait(o);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = 0;
        }
        if (live && p.splits > 1) {
          float *po = p.part_o + at * D + 32 * i;
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            *reinterpret_cast<uint4 *>(po + j) = make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
        } else if (live) {
          float f[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) f[j] = l == 0.f ? 0.f : __uint_as_float(o[j]) * inv;
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            float f8[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) f8[k] = f[j + k];
            if (vec) {
              *reinterpret_cast<uint4 *>(dst + 32 * i + j) = Vec16<T>::pack(f8);
            } else {
#pragma unroll
              for (int k = 0; k < 8; ++k) dst[32 * i + j + k] = from_f32<T>(f8[k]);
            }
          }
        }
      }
      if (live && p.splits > 1) p.part_ml[at] = make_float2(m, l);
    }
  } else if (wg == 2) {
    regs_dec<kPrConvRegs>();
    const int ct = tid - 256, quarter = ct % 4, row0 = ct / 4;
    constexpr int kPerK = 2 * (D / 64), kPerV = D / 32;  // 16-code pieces of a thread
    uint4 kr[2][kPerK], vr[2][kPerV];  // codes of two key tiles under way
    const uint4 zero = make_uint4(0, 0, 0, 0);
    auto load_k = [&](uint4 (&kr)[kPerK], int page) {
#pragma unroll
      for (int i = 0; i < kPerK; ++i) {
        const int row = row0 + 32 * (i % 2), slab = i / 2;
        kr[i] = !known(page) ? zero
                             : *reinterpret_cast<const uint4 *>(
                                   p.kc + ((static_cast<long long>(page) * p.kv_heads + hk) *
                                               kBlockTokens + row) * D + 64 * slab + 16 * quarter);
      }
    };
    auto load_v = [&](uint4 (&vr)[kPerV], int page, int kt) {
#pragma unroll
      for (int i = 0; i < kPerV; ++i)
        vr[i] = !known(page) ? zero
                             : *reinterpret_cast<const uint4 *>(
                                   p.vc + ((static_cast<long long>(page) * p.kv_heads + hk) * D +
                                           row0 + 32 * i) * kBlockTokens + 16 * quarter);
      // values of keys that no row of the CTA sees count as zero, whatever their codes
      const long long base = (first + kt) * kBlockTokens;
      if (base < key_lo || base + kBlockTokens > key_hi) {
        uint32_t keep[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const long long key = base + 16 * quarter + j;
          if (key < key_lo || key >= key_hi) keep[j / 4] &= ~(0xffu << 8 * (j % 4));
        }
#pragma unroll
        for (int i = 0; i < kPerV; ++i)
          vr[i] = make_uint4(vr[i].x & keep[0], vr[i].y & keep[1], vr[i].z & keep[2],
                             vr[i].w & keep[3]);
      }
    };
    // the stage of key tile kt is free when both row tiles are done with its last use
    auto freed = [&](uint64_t (*bars)[kPrStages], int kt) {
      const uint32_t st = static_cast<uint32_t>(kt) % kPrStages;
      const uint32_t ph = (static_cast<uint32_t>(kt) / kPrStages & 1) ^ 1;
      if (kt < kPrStages) return;
      wait(&bars[0][st], ph);
      if (two) wait(&bars[1][st], ph);
    };
    // warp 8 hands the softmax threads the scales of 32 key tiles at a time, a lane each, and loads
    // the next 32 then
    float ks = 1.f, vs = 0.f;
    auto fetch_scales = [&](int i0) {  // no page: no weight
      ks = 1.f, vs = 0.f;
      const int page = page_of(i0 + lane);
      if (known(page)) {
        const long long slot = static_cast<long long>(page) * p.kv_heads + hk;
        ks = p.ks[slot], vs = fmaxf(p.vs[slot], kScaleMin);
      }
    };
    auto put_scales = [&](int i0) {
      const int half = i0 / 32 & 1;
      if (i0 >= 64) wait(sc_empty + half, (i0 / 64 - 1) & 1);
      scales[half][lane] =
          make_float4(ks, vs == 0.f ? -INFINITY : log2f(vs), vs == 0.f ? 0.f : 1.f / vs, 0.f);
      arrive(sc_full + half);
      fetch_scales(i0 + 32);
    };
    if (warp == 8) fetch_scales(0);
    int pages[2] = {page_of(2), page_of(3)};  // of the tiles to load next
    if (n > 0) {
      const int page0 = page_of(0), page1 = page_of(1);
      load_k(kr[0], page0);
      load_v(vr[0], page0, 0);
      if (n > 1) load_k(kr[1], page1);
      if (n > 1) load_v(vr[1], page1, 1);
    }
    // A tile's loads are issued two tiles ahead: one tile is not enough to cover them.
    auto step = [&](int kt, auto which) {
      constexpr int w = decltype(which)::value;
      const uint32_t st = static_cast<uint32_t>(kt) % kPrStages;
      const int page = pages[w];
      pages[w] = page_of(kt + 4);
      if (warp == 8 && kt % 32 == 0) put_scales(kt);
      freed(s_full, kt);
      const uint32_t kd = sk + st * S::kK, vd = sv + st * S::kV;
#pragma unroll
      for (int i = 0; i < kPerK; ++i)
        store_codes(kd + i / 2 * S::kSlab, row0 + 32 * (i % 2), 2 * quarter, kr[w][i]);
      fence_proxy_async_smem();
      arrive(k_full + st);
      if (kt + 2 < n) load_k(kr[w], page);
      freed(p_empty, kt);
#pragma unroll
      for (int i = 0; i < kPerV; ++i) store_codes(vd, row0 + 32 * i, 2 * quarter, vr[w][i]);
      fence_proxy_async_smem();
      arrive(v_full + st);
      if (kt + 2 < n) load_v(vr[w], page, kt + 2);
    };
    for (int kt = 0; kt < n; kt += 2) {
      step(kt, std::integral_constant<int, 0>());
      if (kt + 1 < n) step(kt + 1, std::integral_constant<int, 1>());
    }
  } else {
    regs_dec<kPrRestRegs>();
    // The row tile is a compile-time number here: operands that the compiler does not see to be the
    // same for the warp are moved into place for every MMA, which then waits for that (measured: 8 MMAs
    // of 32 cycles each took 1400 to issue with the tile taken from the warp's number).
    auto issue = [&](auto tile, auto what) {
      constexpr int t = decltype(tile)::value, kind = decltype(what)::value;
      constexpr uint32_t kIdS = idesc_f16_f32(128, kBlockTokens), kIdO = idesc_f16_f32(128, D);
      if (kind == 0) {  // S over one key tile after the other
        const uint32_t q = sw128_desc_lo(sq), d = tmem + kColS + t * kBlockTokens;
        const uint32_t a = tmem + kColQ + t * (D / 2);
        if (n > 0) wait(&q_full, 0);
        for (int kt = 0; kt < n; ++kt) {
          const uint32_t st = static_cast<uint32_t>(kt) % kPrStages;
          wait(k_full + st, static_cast<uint32_t>(kt) / kPrStages & 1);
          if (kt > 0) wait(s_empty + t, (kt - 1) & 1);
          tc_fence_after();
          const uint32_t k = sw128_desc_lo(sk + st * S::kK);
#pragma unroll
          for (int s = 0; s < D / 16; ++s) {
            const uint32_t b = k + s / 4 * (S::kSlab >> 4) + s % 4 * 2;
            if constexpr (D == 64 || t == 0)
              mma_f16_warp_ts(d, a + 8 * s, b, kSw128DescHi, kIdS, s > 0 ? 1u : 0u);
            else
              mma_f16_warp_ss(d, q + s / 4 * (128 * 128 >> 4) + s % 4 * 2, b, kSw128DescHi, kIdS,
                              s > 0 ? 1u : 0u);
          }
          mma_commit_warp(smem_u32(&s_full[t][st]));
        }
      } else {  // O += P V
        for (int kt = 0; kt < n; ++kt) {
          const uint32_t st = static_cast<uint32_t>(kt) % kPrStages;
          wait(v_full + st, static_cast<uint32_t>(kt) / kPrStages & 1);
          wait(p_full + t, kt & 1);
          tc_fence_after();
          const uint32_t v = sw128_desc_lo(sv + st * S::kV);
#pragma unroll
          for (int s = 0; s < kBlockTokens / 16; ++s)
            mma_f16_warp_ts(tmem + t * D, tmem + kColP + t * (kBlockTokens / 2) + 8 * s, v + 2 * s,
                            kSw128DescHi, kIdO, kt > 0 || s > 0 ? 1u : 0u);
          mma_commit_warp(smem_u32(&p_empty[t][st]));
        }
      }
      // after a give-up too: everything issued is done before tensor memory is freed
      uint64_t *end = kind == 0 ? drain + t : o_full + t;
      mma_commit_warp(smem_u32(end));
      if (!mbar_wait(smem_u32(end), 0, 4 * p.budget, &never)) *abort = 1;
      __syncwarp();
      if (*abort && lane == 0 && p.timeout) *p.timeout = 1;
    };
    using Zero = std::integral_constant<int, 0>;
    using One = std::integral_constant<int, 1>;
    if (warp == 12) issue(Zero(), Zero());
    if (warp == 13 && two) issue(One(), Zero());
    if (warp == 14) issue(Zero(), One());
    if (warp == 15 && two) issue(One(), One());
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) tmem_dealloc(tmem, 512);
}

}  // namespace voc
