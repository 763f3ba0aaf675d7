// lm_prompt.cuh -- the attention of lm_attention.cuh for many queries of a sequence at once, on
// the 5th-generation tensor cores.
//
// A CTA takes 256 rows (queries that share a key head) as two tiles of 128 and walks over its keys
// in tiles of 128 (two cache blocks):
//   warps 0..3, 4..7   one thread per row of the first / second row tile: softmax of the scores
//   warps 8..11        convert K and V codes to f16 (exact) in shared memory
//   warp 12            issues the products: S = Q K^T from shared memory, O += P V with P in
//                      tensor memory, in the place of the scores it was made from
// The two row tiles take turns: while one's scores go through its softmax, the tensor cores work
// on the other's products.  Both operands are 16-bit: the codes are exact in f16 and the weights
// keep 11 bits, where an e4m3 product would round queries and weights to 4.
//
// The running maximum that the weights are taken against (see lm_attention.cuh) is raised only
// when a row's new maximum is more than 8 above it, so the accumulator is rarely rescaled; weights
// are kept times 2^7 and stay below 2^15, inside f16.
#pragma once
#include "lm_attention.cuh"

namespace voc {

constexpr int kPrThreads = 512;
constexpr int kPrRows = 256;       // rows of a CTA
constexpr int kPrKeys = 128;       // keys of a tile
constexpr int kPartRows = 16;      // rows of a tile of partial outputs
// Registers: 256 softmax threads, 128 converting, 128 others: 256 x 184 + 128 x 104 + 128 x 40 =
// 65536, the block's registers at launch (512 x 128).
constexpr int kPrSoftRegs = 184, kPrConvRegs = 104, kPrRestRegs = 40;
static_assert(256 * kPrSoftRegs + 128 * kPrConvRegs + 128 * kPrRestRegs <= 512 * 128, "registers");

template <int D>
struct PromptSmem {
  static constexpr int kSlab = 128 * 128;               // 128 rows of 64 f16 values
  static constexpr int kQ = D / 64 * kSlab;             // one row tile
  static constexpr int kK = D / 64 * kSlab;             // one key tile
  static constexpr int kV = 2 * D * 128;                // two blocks of D rows of 64 keys
  static constexpr size_t kBytes = 2 * kQ + 2 * kK + 2 * kV + 1024;
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
  const uint32_t sq = smem_u32(base_ptr), sk = sq + 2 * S::kQ, sv = sk + 2 * S::kK;
  __shared__ __align__(8) uint64_t q_full, k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2],
      p_full[2], o_full;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, wg = warp / 4;
  volatile int *abort = &abort_flag;
  const int never = 0;

  const int b = blockIdx.z / p.splits, split = blockIdx.z % p.splits, hk = blockIdx.y;
  const SeqSpan span = seq_span(p.cu, b, p.n_seq, p.n_tokens, p.max_q);
  const int rows = span.count * p.group;
  if (tid == 0) {
    mbar_init(smem_u32(&q_full), 256);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(k_full + i), 128);
      mbar_init(smem_u32(v_full + i), 128);
      mbar_init(smem_u32(k_empty + i), 1);
      mbar_init(smem_u32(v_empty + i), 1);
      mbar_init(smem_u32(s_full + i), 1);
      mbar_init(smem_u32(p_full + i), 128);
    }
    mbar_init(smem_u32(&o_full), 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  pdl_wait();
  pdl_launch_dependents();
  // the latest rows see the most keys: they start first
  const int tile_max = static_cast<int>(gridDim.x) - 1 - static_cast<int>(blockIdx.x);
  const int r0 = tile_max * kPrRows;
  if (r0 >= span.count * p.group) return;  // the whole block, before any barrier or allocation
  if (warp == 12) {
    tmem_alloc(smem_u32(&tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;  // scores 0..127 and 128..255, outputs from 256
  const int r_last = min(rows, r0 + kPrRows) - 1;
  const bool two = r_last - r0 >= 128;  // the second row tile has rows
  const long long len = max(0ll, min(static_cast<long long>(p.lens[b]),
                                     static_cast<long long>(p.table_cols) * kBlockTokens));
  const long long p0 = static_cast<long long>(p.lens[b]) - span.count;
  const long long key_lo = visible(p, p0 + r0 / p.group, len).lo;
  const long long key_hi = visible(p, p0 + r_last / p.group, len).hi;
  const long long tile0 = key_lo / kPrKeys;
  const long long n_all = key_hi > key_lo ? (key_hi - 1) / kPrKeys + 1 - tile0 : 0;
  const long long per = (n_all + p.splits - 1) / p.splits;
  const long long first = tile0 + min(n_all, split * per);
  const int n = static_cast<int>(min(n_all, (split + 1) * per) - min(n_all, split * per));
  const int *table = p.table + b * p.ldt;
  // page of a block, or -1 where the CTA sees none of its keys
  auto page_of = [&](long long blk) {
    if (blk * kBlockTokens >= key_hi || (blk + 1) * kBlockTokens <= key_lo) return -1;
    const int page = table[blk];
    return page >= 0 && page < p.n_pages ? page : -1;
  };

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
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        float f[8];
        Vec16<T>::unpack(raw[i], f);
        uint32_t h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = f16x2(f[2 * j] * up, f[2 * j + 1] * up);
        sts128(sq + wg * S::kQ + i / 8 * S::kSlab + sw128(local, i % 8),
               make_uint4(h[0], h[1], h[2], h[3]));
      }
    }
    fence_proxy_async_smem();
    mbar_arrive(smem_u32(&q_full));

    const uint32_t lane_base = static_cast<uint32_t>((warp % 4) * 32) << 16;
    const uint32_t s_addr = tmem + lane_base + wg * 128, o_addr = tmem + lane_base + 256 + wg * D;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    if (wg == 0 || two) {
      // scales of the tile's two blocks, one tile ahead of their use; pages two ahead
      int pg[2] = {page_of(2 * first), page_of(2 * first + 1)};
      float ks[2], vs[2];
      auto load_scales = [&]() {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const long long slot = static_cast<long long>(pg[h]) * p.kv_heads + hk;
          ks[h] = pg[h] >= 0 ? p.ks[slot] : 1.f;
          vs[h] = pg[h] >= 0 ? p.vs[slot] : 0.f;
        }
      };
      if (n > 0) load_scales();
      if (n > 1) pg[0] = page_of(2 * (first + 1)), pg[1] = page_of(2 * (first + 1) + 1);
      for (int kt = 0; kt < n; ++kt) {
        float c[2], lvs[2], ivs[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float v = fmaxf(vs[h], kScaleMin);
          c[h] = fmaxf(qc * ks[h], 1e-37f);  // above 0: masked scores stay -inf
          lvs[h] = vs[h] == 0.f ? -INFINITY : log2f(v);  // no page: no weight
          ivs[h] = vs[h] == 0.f ? 0.f : 1.f / v;
        }
        if (kt + 1 < n) {
          load_scales();
          if (kt + 2 < n) {
            pg[0] = page_of(2 * (first + kt + 2));
            pg[1] = page_of(2 * (first + kt + 2) + 1);
          }
        }
        ok = mbar_wait(smem_u32(s_full + wg), kt & 1, p.budget, abort);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          *abort = 1;
          break;
        }
        tc_fence_after();
        uint32_t sc[128];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32_issue(s_addr + 32 * i, sc + 32 * i);
        tmem_ld_wait_all();
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32_after_wait(sc + 32 * i);
        const long long base = (first + kt) * kPrKeys;
        if (__any_sync(0xffffffffu, base < see.lo || base + kPrKeys > see.hi)) {
          const int a = static_cast<int>(max(-1ll, min(see.lo - base, 128ll)));
          const int z = static_cast<int>(max(-1ll, min(see.hi - base, 128ll)));
#pragma unroll
          for (int i = 0; i < 128; ++i)
            if (i < a || i >= z) sc[i] = 0xff800000u;
        }
        float top[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
          for (int i = 0; i < 64; i += 2) {
            t0 = fmaxf(t0, __uint_as_float(sc[64 * h + i]));
            t1 = fmaxf(t1, __uint_as_float(sc[64 * h + i + 1]));
          }
          top[h] = fmaf(fmaxf(t0, t1), c[h], lvs[h]);
        }
        const float nm = fmaxf(top[0], top[1]);
        float alpha = 1.f;
        if (nm > m + kLazy || (m == -INFINITY && nm > m)) {
          alpha = ex2(m - nm);
          m = nm;
        }
        const float off = (m == -INFINITY ? 0.f : m) - kPShift;
        l *= alpha;
        if (kt > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
          // the products that this tile's scores were issued behind are done: O is at rest
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            uint32_t o[32];
            tmem_ld32_issue(o_addr + 32 * i, o);
            tmem_ld_wait_all();
            tmem_ld32_after_wait(o);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
            tmem_st32(o_addr + 32 * i, o);
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float2 cc = make_float2(c[h], c[h]);
          const float d = lvs[h] - off;
          const float2 dd = make_float2(d, d);
          float2 sum = make_float2(0.f, 0.f);
          uint32_t w[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float2 u = fma2(make_float2(__uint_as_float(sc[64 * h + 2 * i]),
                                        __uint_as_float(sc[64 * h + 2 * i + 1])),
                            cc, dd);
            u.x = ex2(u.x), u.y = ex2(u.y);
            sum = add2(sum, u);
            w[i] = f16x2(u.x, u.y);
          }
          tmem_st32(s_addr + 32 * h, w);
          l = fmaf(sum.x + sum.y, ivs[h], l);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(smem_u32(p_full + wg));
      }
    }
    // outputs
    if (n > 0 && (wg == 0 || two)) {
      const bool done = mbar_wait(smem_u32(&o_full), 0, 4 * p.budget, &never);
      if (!__all_sync(0xffffffffu, done)) *abort = 1;
      tc_fence_after();
    }
    if (wg == 0 || two) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      T *dst = static_cast<T *>(p.out) + (span.first + tok) * p.ldo + head * p.hso;
      const bool vec = (reinterpret_cast<uintptr_t>(dst) & 15) == 0;
      const long long tile16 =
          (static_cast<long long>(b) * p.kv_heads + hk) * p.row_tiles + r / kPartRows;
      const long long at = (tile16 * p.splits + split) * kPartRows + r % kPartRows;
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
    constexpr int kSlabs = D / 64;
    uint4 kr[4 * kSlabs], vr[2 * (D / 32)];
    int pg[2], next[2];
    auto pages = [&](int kt, int (&to)[2]) {
      to[0] = kt < n ? page_of(2 * (first + kt)) : -1;
      to[1] = kt < n ? page_of(2 * (first + kt) + 1) : -1;
    };
    const uint4 zero = make_uint4(0, 0, 0, 0);
    auto load_k = [&](const int (&from)[2]) {
#pragma unroll
      for (int i = 0; i < 4 * kSlabs; ++i) {
        const int row = row0 + 32 * (i % 4), slab = i / 4, page = from[i % 4 / 2];
        kr[i] = page < 0 ? zero
                         : *reinterpret_cast<const uint4 *>(
                               p.kc + ((static_cast<long long>(page) * p.kv_heads + hk) *
                                           kBlockTokens + row % kBlockTokens) * D +
                               64 * slab + 16 * quarter);
      }
    };
    auto load_v = [&](const int (&from)[2], int kt) {
#pragma unroll
      for (int i = 0; i < 2 * (D / 32); ++i) {
        const int blk = i / (D / 32), row = row0 + 32 * (i % (D / 32)), page = from[blk];
        vr[i] = page < 0 ? zero
                         : *reinterpret_cast<const uint4 *>(
                               p.vc + ((static_cast<long long>(page) * p.kv_heads + hk) * D + row) *
                                          kBlockTokens + 16 * quarter);
      }
      // values of keys that no row of the CTA sees count as zero, whatever their codes
      const long long base = (first + kt) * kPrKeys;
      if (base < key_lo || base + kPrKeys > key_hi) {
#pragma unroll
        for (int i = 0; i < 2 * (D / 32); ++i) {
          const long long key = base + i / (D / 32) * kBlockTokens + 16 * quarter;
          uint32_t w[4] = {vr[i].x, vr[i].y, vr[i].z, vr[i].w};
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (key + j < key_lo || key + j >= key_hi) w[j / 4] &= ~(0xffu << 8 * (j % 4));
          vr[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    };
    pages(0, pg);
    pages(1, next);
    if (n > 0) {
      load_k(pg);
      load_v(pg, 0);
    }
    for (int kt = 0; kt < n; ++kt) {
      const int st = kt & 1, ph = kt >> 1 & 1;
      if (kt >= 2 && !mbar_wait(smem_u32(k_empty + st), ph ^ 1, p.budget, abort)) {
        *abort = 1;
        break;
      }
      const uint32_t kd = sk + st * S::kK, vd = sv + st * S::kV;
#pragma unroll
      for (int i = 0; i < 4 * kSlabs; ++i)
        store_codes(kd + i / 4 * S::kSlab, row0 + 32 * (i % 4), 2 * quarter, kr[i]);
      fence_proxy_async_smem();
      mbar_arrive(smem_u32(k_full + st));
      if (kt + 1 < n) load_k(next);
      if (kt >= 2 && !mbar_wait(smem_u32(v_empty + st), ph ^ 1, p.budget, abort)) {
        *abort = 1;
        break;
      }
#pragma unroll
      for (int i = 0; i < 2 * (D / 32); ++i)
        store_codes(vd + i / (D / 32) * (D * 128), row0 + 32 * (i % (D / 32)), 2 * quarter, vr[i]);
      fence_proxy_async_smem();
      mbar_arrive(smem_u32(v_full + st));
      if (kt + 1 < n) {
        load_v(next, kt + 1);
        pages(kt + 2, next);
      }
    }
  } else {
    regs_dec<kPrRestRegs>();
    if (warp == 12) {
      constexpr uint32_t kIdS = idesc_f16_f32(128, kPrKeys), kIdO = idesc_f16_f32(128, D);
      bool ok = true;
      auto wait = [&](uint64_t *bar, int parity) {
        const bool landed = mbar_wait(smem_u32(bar), parity, p.budget, abort);
        if (!__all_sync(0xffffffffu, landed)) {
          *abort = 1;
          ok = false;
        }
        tc_fence_after();
        return ok;
      };
      auto scores = [&](int t, int kt) {  // S of row tile t over key tile kt
        const uint32_t a = sw128_desc_lo(sq + t * S::kQ), k = sw128_desc_lo(sk + (kt & 1) * S::kK);
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          const uint32_t step = s / 4 * (S::kSlab >> 4) + s % 4 * 2;
          mma_f16_warp_ss(tmem + t * 128, a + step, k + step, kSw128DescHi, kIdS, s > 0 ? 1u : 0u);
        }
        mma_commit_warp(smem_u32(s_full + t));
      };
      auto values = [&](int t, int kt) {  // O of row tile t += P V
        const uint32_t v = sw128_desc_lo(sv + (kt & 1) * S::kV);
#pragma unroll
        for (int s = 0; s < kPrKeys / 16; ++s)
          mma_f16_warp_ts(tmem + 256 + t * D, tmem + t * 128 + 8 * s,
                          v + s / 4 * (D * 128 >> 4) + s % 4 * 2, kSw128DescHi, kIdO,
                          kt > 0 || s > 0 ? 1u : 0u);
      };
      if (n > 0 && wait(&q_full, 0) && wait(k_full, 0)) {
        scores(0, 0);
        if (two) scores(1, 0);
        mma_commit_warp(smem_u32(k_empty));
        for (int kt = 0; kt < n && ok; ++kt) {
          const int st = kt & 1, ph = kt >> 1 & 1;
          if (!wait(v_full + st, ph) || !wait(p_full, kt & 1)) break;
          values(0, kt);
          if (kt + 1 < n) {
            if (!wait(k_full + (st ^ 1), (kt + 1) >> 1 & 1)) break;
            scores(0, kt + 1);
          }
          if (two) {
            if (!wait(p_full + 1, kt & 1)) break;
            values(1, kt);
          }
          mma_commit_warp(smem_u32(v_empty + st));
          if (kt + 1 < n) {
            if (two) scores(1, kt + 1);
            mma_commit_warp(smem_u32(k_empty + (st ^ 1)));
          }
        }
      }
      // after a give-up too: everything issued is done before tensor memory is freed
      mma_commit_warp(smem_u32(&o_full));
      if (!mbar_wait(smem_u32(&o_full), 0, 4 * p.budget, &never)) *abort = 1;
      __syncwarp();
      if (*abort && lane == 0 && p.timeout) *p.timeout = 1;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) tmem_dealloc(tmem, 512);
}

}  // namespace voc
