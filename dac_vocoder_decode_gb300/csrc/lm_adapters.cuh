// lm_adapters.cuh -- low-rank adapters of many requests at once beside a shared projection.
//
//   out[m] = y[m] + scale[a] * xs[m] * B_a (A_a x[m]),   a = ids[m]   (no adapter: out[m] = y[m])
//
// x in e4m3 with a scale per row, as the projection takes it; A_a [rank][K] and B_a [N][rank] in 16 bits;
// sums in 32 bits.  The low-rank values between the two products go on as two 16-bit parts, of 16 (bf16) or
// 22 (f16, of the token's largest) bits together: they lose 2^-8 of half a step of a 16-bit output, or less.
// Beside 32-bit outputs bf16 takes three, 24 bits together.
#pragma once
#include <type_traits>

#include "lm_common.cuh"
#include "lm_rows.cuh"

namespace voc {

struct LmAdaptersArgs {
  const uint8_t *x;
  const float *xs;
  const void *y, *a, *b;
  const float *scale;
  const int *ids, *ranks;
  void *out;
  long long ldx, ldy, ldo, lda, sa, ldb, sb;  // sa, sb: from one adapter to the next
  int M, N, K, rank, pool;
};

constexpr int kAdThreads = 256;
constexpr int kAdTokens = 64;  // tokens of a tile
constexpr int kAdK = 256;      // channels of x of a stage, 8 segments of 32
constexpr int kAdSeg = 32;

// 16-bit parts of a low-rank value.
template <typename W, typename Y>
constexpr int kAdParts = sizeof(Y) == 4 && std::is_same<W, __nv_bfloat16>::value ? 3 : 2;

template <int R, int PARTS>
struct AdapterSmem {
  static constexpr int kX = kAdTokens * kAdK, kA = R * kAdK * 2;
  static constexpr int kStage = kX + kA;
  static constexpr int kStages = R <= 32 ? 3 : 2;
  // after the first product, in the ring's place: sums of the warps, of the CTA, and the parts
  static constexpr int kWarpSums = 8 * 16 * R * 4;
  static constexpr int kSums = kAdTokens * R * 4;
  static constexpr int kRow = R * 2 + (R >= 64 ? 64 : 0);  // bytes of a row of a part, rows on other banks
  static constexpr int kPart = kAdTokens * kRow;
  static constexpr int kAfter = kWarpSums + kSums + PARTS * kPart;
  static constexpr int kBytes = kStages * kStage > kAfter ? kStages * kStage : kAfter;
};

__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                      __half) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                      __nv_bfloat16) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two e4m3 codes to two 16-bit values (exact in both types).
__device__ __forceinline__ uint32_t e4m3x2_to(uint32_t two, __half) {
  return e4m3x2_to_f16x2(static_cast<uint16_t>(two));
}
__device__ __forceinline__ uint32_t e4m3x2_to(uint32_t two, __nv_bfloat16) {
  const float2 f = e4m3x2_to_f32(static_cast<uint16_t>(two));
  return pack2<__nv_bfloat16>(f.x, f.y);
}

// 16 bytes to shared memory, of which the first `bytes` (0 to 16) are read and the others zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The exponent e, from -126 to 126, for which 2^-e brings the finite value of magnitude bits `amax` to [1, 2)
// (0 for zeros; beyond those exponents as near as they go).
__device__ __forceinline__ int binade(uint32_t amax) {
  return amax == 0 ? 0 : max(-126, min(126, static_cast<int>(amax >> 23) - 127));
}

// The words of 8 (4) values of which the first `left` (any number) count, zeros for the others.
template <int WORDS>
__device__ __forceinline__ void cut_words(uint32_t (&w)[WORDS], int left) {
#pragma unroll
  for (int i = 0; i < WORDS; ++i)
    w[i] = left >= 2 * i + 2 ? w[i] : left == 2 * i + 1 ? w[i] & 0xffffu : 0u;
}

// Eight values of a row of y or out, at `p`, of which `left` lie in the row, in the widest accesses that
// `start` (what all rows of both start on, in bytes) allows.
template <typename Y>
struct Eight {
  static constexpr int kWords = 2 * static_cast<int>(sizeof(Y));
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const Y *p, int left, int start) {
    if (left < 8) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (sizeof(Y) == 4) {
          w[i] = i < left ? reinterpret_cast<const uint32_t *>(p)[i] : 0u;
        } else {
          const uint32_t h = i < left ? reinterpret_cast<const uint16_t *>(p)[i] : 0u;
          w[i / 2] = i % 2 ? w[i / 2] | h << 16 : h;
        }
      }
    } else if (start % 16 == 0) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 v = *reinterpret_cast<const uint4 *>(reinterpret_cast<const uint32_t *>(p) + i);
        w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
      }
    } else if (start % 8 == 0) {
#pragma unroll
      for (int i = 0; i < kWords; i += 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(reinterpret_cast<const uint32_t *>(p) + i);
        w[i] = v.x, w[i + 1] = v.y;
      }
    } else if (sizeof(Y) == 4 || start % 4 == 0) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const uint32_t *>(p)[i];
    } else if constexpr (sizeof(Y) == 2) {
      RowVec<Y, 16>::load_any(p, w);
    }
  }
  __device__ __forceinline__ void store(Y *p, int left, int start) const {
    if (left < 8) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) {
          if constexpr (sizeof(Y) == 4)
            reinterpret_cast<uint32_t *>(p)[i] = w[i];
          else
            reinterpret_cast<uint16_t *>(p)[i] = static_cast<uint16_t>(w[i / 2] >> 16 * (i % 2));
        }
    } else if (start % 16 == 0) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4)
        *reinterpret_cast<uint4 *>(reinterpret_cast<uint32_t *>(p) + i) =
            make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    } else if (start % 8 == 0) {
#pragma unroll
      for (int i = 0; i < kWords; i += 2)
        *reinterpret_cast<uint2 *>(reinterpret_cast<uint32_t *>(p) + i) = make_uint2(w[i], w[i + 1]);
    } else if (sizeof(Y) == 4 || start % 4 == 0) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) reinterpret_cast<uint32_t *>(p)[i] = w[i];
    } else if constexpr (sizeof(Y) == 2) {
      RowVec<Y, 16>::store_any(p, w);
    }
  }
  __device__ __forceinline__ void unpack(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (sizeof(Y) == 4)
        f[i] = __uint_as_float(w[i]);
      else
        unpack2<Y>(w[i], f[2 * i], f[2 * i + 1]);
    }
  }
  __device__ __forceinline__ void pack(const float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (sizeof(Y) == 4)
        w[i] = __float_as_uint(f[i]);
      else
        w[i] = pack2<Y>(f[2 * i], f[2 * i + 1]);
    }
  }
};

// A cluster of CTAs (along z) takes those of the adapters that the 64 tokens of tile blockIdx.x use whose
// turn it is (every gridDim.y-th, in the order in which they first occur), one after the other, with all
// of their tokens gathered from the tile.  First product: each CTA a part of K, its 8 warps the tokens in
// sixteens and, with fewer than 128 tokens, shares of K; the CTAs' sums are read through distributed shared
// memory by all of them, in a fixed order.  Second product: each CTA a part of the output channels, added to
// y on the way.  So a few tokens keep 8 CTAs busy, and many tokens read every adapter once a tile, from
// cache.
// Measured: 8 tokens with a voice each, 1024 -> 1536, rank 16: 5.2 us, two barriers of the cluster in a chain of
// five reads; 33 x 4096 -> 12288, rank 16: 11.0 us; 15423 tokens x 1001 -> 1540, rank 32: 53 us, 2.1 TB/s (rows
// of y start on 8 bytes); 15504 x 4096 -> 4096, rank 64: 124 us, 2.6 TB/s.  Bound by latencies: 16 warps an SM,
// what 128 registers leave (3 CTAs of 80: prompts 76 us), issue in 44 % of the cycles, the matrix pipe a third.
// Skipping the eights of ranks that an adapter lacks cost the full ones more (136 us) than it spares.
// Other ranks and outputs, 15504 x 4096 -> 4096, bf16 / f16 pools: rank 16 81 / 77 us, with f32 y 114 / 109; rank 64
// 124 / 121, with f32 y 159 / 146 (bf16 with two parts 148); rank 128 (one CTA an SM, 242 registers) 257 / 255, with f32
// y 315 / 278 (280).  Ids in no order cost a turn of a tile for each adapter in it, 1024 -> 1536, rank 16: 15504
// tokens of 8 adapters 93 us, 4000 of 64 214 us, 2000 of an adapter each 316 us.
template <typename W, typename Y, int R>
__global__ void __launch_bounds__(kAdThreads, R <= 64 ? 2 : 1) adapters_kernel(const LmAdaptersArgs p) {
  constexpr int kParts = kAdParts<W, Y>;
  using Smem = AdapterSmem<R, kParts>;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ int rows[kAdTokens];
  __shared__ float factor[kAdTokens];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int g = lane / 4, t = lane % 4;
  const int split = gridDim.z, part = blockIdx.z;
  const long long m0 = static_cast<long long>(blockIdx.x) * kAdTokens;
  pdl_wait();
  pdl_launch_dependents();

  // The tile's tokens by adapter; every warp for itself.  -1: none, -2: beyond the last token.
  int id[2];
  uint32_t same[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const long long m = m0 + 32 * h + lane;
    int v = -2;
    if (m < p.M) {
      v = p.ids[m];
      if (v < 0 || v >= p.pool) v = -1;
    }
    id[h] = v;
    same[h] = __match_any_sync(0xffffffffu, v);
  }
  bool repeated = false;  // the second half's id occurs in the first
  if (m0 + 32 < p.M)
    for (int i = 0; i < 32; ++i) repeated |= __shfl_sync(0xffffffffu, id[0], i) == id[1];
  const uint32_t below = (1u << lane) - 1u;
  const bool leads0 = id[0] != -2 && __ffs(same[0]) - 1 == lane;
  const bool leads1 = id[1] != -2 && __ffs(same[1]) - 1 == lane && !repeated;
  const uint32_t first0 = __ballot_sync(0xffffffffu, leads0), first1 = __ballot_sync(0xffffffffu, leads1);
  const int here = __popc(first0), distinct = here + __popc(first1);

  for (int turn = blockIdx.y; turn < distinct; turn += gridDim.y) {
    const uint32_t at0 = __ballot_sync(0xffffffffu, leads0 && __popc(first0 & below) == turn);
    const uint32_t at1 = __ballot_sync(0xffffffffu, leads1 && here + __popc(first1 & below) == turn);
    const int which = __shfl_sync(0xffffffffu, at0 ? id[0] : id[1], __ffs(at0 | at1) - 1);
    const uint32_t use0 = __ballot_sync(0xffffffffu, id[0] == which);
    const uint32_t use1 = __ballot_sync(0xffffffffu, id[1] == which);
    const int count = __popc(use0) + __popc(use1);
    if (warp == 0) {
      if (use0 >> lane & 1) rows[__popc(use0 & below)] = lane;
      if (use1 >> lane & 1) rows[__popc(use0) + __popc(use1 & below)] = 32 + lane;
    }
    __syncthreads();
    int rank = 0;
    if (which >= 0) rank = p.ranks ? max(0, min(p.ranks[which], p.rank)) : p.rank;
    // output channels of this CTA, in groups of 32
    const int groups = (p.N + 31) / 32;
    const int g0 = static_cast<int>(static_cast<long long>(groups) * part / split);
    const int g1 = static_cast<int>(static_cast<long long>(groups) * (part + 1) / split);
    const Y *y = static_cast<const Y *>(p.y);
    Y *out = static_cast<Y *>(p.out);
    const int start = static_cast<int>((reinterpret_cast<uintptr_t>(y) | reinterpret_cast<uintptr_t>(out) |
                                        (p.ldy * sizeof(Y)) | (p.ldo * sizeof(Y))) & 15);
    if (rank == 0) {  // uniform in the cluster
      if (p.out != p.y)
        for (int i = tid; i < count * (g1 - g0) * 4; i += kAdThreads) {
          const int r = i / ((g1 - g0) * 4), n = 32 * g0 + i % ((g1 - g0) * 4) * 8;
          const long long m = m0 + rows[r];
          Eight<Y> v;
          v.load(y + m * p.ldy + n, p.N - n, start);
          v.store(out + m * p.ldo + n, p.N - n, start);
        }
      __syncthreads();  // rows are read
      continue;
    }

    const W *b = static_cast<const W *>(p.b) + which * p.sb;
    if (count <= 16 && tid == 0 && g0 < g1 && p.ldb <= 2 * p.rank) {  // the second product's rows meanwhile to L2
      const int n0 = 32 * g0, n1 = min(p.N, 32 * g1);
      bulk_prefetch_l2(b + n0 * p.ldb, static_cast<uint32_t>(((n1 - 1 - n0) * p.ldb + p.rank) * 2));
    }
    // ---------------------------------------------------------------- A x, this CTA's part of K
    const W *a = static_cast<const W *>(p.a) + which * p.sa;
    const int segs = (p.K + kAdSeg - 1) / kAdSeg;
    const int s0 = static_cast<int>(static_cast<long long>(segs) * part / split);
    const int s1 = static_cast<int>(static_cast<long long>(segs) * (part + 1) / split);
    const int chunks = (s1 - s0 + 7) / 8;
    const int k_end = min(p.K, s1 * kAdSeg);
    const uint32_t base = smem_u32(ring);
    auto load = [&](int c) {
      const uint32_t xs = base + (c % Smem::kStages) * Smem::kStage, as = xs + Smem::kX;
      const int k0 = (s0 + 8 * c) * kAdSeg;
      {
        const int chunk = tid % 16, k = k0 + 16 * chunk;
        const int bytes = max(0, min(16, k_end - k));
        for (int r = tid / 16; r < count; r += kAdThreads / 16)
          copy16(xs + r * kAdK + ((chunk ^ (r & 3) << 1) << 4),
                 bytes ? p.x + (m0 + rows[r]) * p.ldx + k : p.x, bytes);
      }
      {
        const int chunk = lane, k = k0 + 8 * chunk;
        const int bytes = max(0, min(16, 2 * (k_end - k)));
        for (int r = warp; r < R; r += kAdThreads / 32) {  // zeros behind the rank
          const int some = r < rank ? bytes : 0;
          copy16(as + r * (2 * kAdK) + ((chunk ^ (r & 1) << 2) << 4),
                 some ? static_cast<const void *>(a + r * p.lda + k) : p.a, some);
        }
      }
    };
    const int m_tiles = count > 32 ? 4 : count > 16 ? 2 : 1;
    const int mt = warp % m_tiles, share = warp / m_tiles, shares = 8 / m_tiles;
    float acc[R / 8][4];
#pragma unroll
    for (int j = 0; j < R / 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
    for (int c = 0; c < Smem::kStages - 1; ++c) {
      if (c < chunks) load(c);
      copy_commit();
    }
    for (int c = 0; c < chunks; ++c) {
      copy_wait<Smem::kStages - 2>();
      __syncthreads();  // stage c has landed for all, and the stage before it has been read
      if (c + Smem::kStages - 1 < chunks) load(c + Smem::kStages - 1);
      copy_commit();
      const uint8_t *xs = ring + (c % Smem::kStages) * Smem::kStage + (mt * 16 + g) * kAdK + 8 * (t & 1);
      const uint8_t *as = ring + (c % Smem::kStages) * Smem::kStage + Smem::kX + g * (2 * kAdK);
      for (int seg = share; seg < 8; seg += shares) {
        // lane t takes channels 8t to 8t + 7 of the segment in both operands
        uint32_t xa[2][4];
        const int x_at = ((2 * seg + t / 2) ^ (g & 3) << 1) << 4, a_at = ((4 * seg + t) ^ (g & 1) << 2) << 4;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint2 v = *reinterpret_cast<const uint2 *>(xs + 8 * h * kAdK + x_at);
          xa[0][h] = e4m3x2_to(v.x & 0xffffu, W());
          xa[0][2 + h] = e4m3x2_to(v.x >> 16, W());
          xa[1][h] = e4m3x2_to(v.y & 0xffffu, W());
          xa[1][2 + h] = e4m3x2_to(v.y >> 16, W());
        }
#pragma unroll
        for (int j = 0; j < R / 8; ++j) {
          const uint4 w = *reinterpret_cast<const uint4 *>(as + 8 * j * (2 * kAdK) + a_at);
          mma16(acc[j], xa[0], w.x, w.y, W());
          mma16(acc[j], xa[1], w.z, w.w, W());
        }
      }
    }
    copy_wait<0>();
    __syncthreads();  // the ring has been read
    float *warp_sums = reinterpret_cast<float *>(ring);
    float *sums = reinterpret_cast<float *>(ring + Smem::kWarpSums);
    uint8_t *parts = ring + Smem::kWarpSums + Smem::kSums;
#pragma unroll
    for (int j = 0; j < R / 8; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<float2 *>(warp_sums + (warp * 16 + g + 8 * h) * R + 8 * j + 2 * t) =
            make_float2(acc[j][2 * h], acc[j][2 * h + 1]);
    __syncthreads();
    constexpr int kQuads = R / 4;  // a token's sums, four to a thread
    const int col = tid % kQuads * 4;
    for (int r = tid / kQuads; r < count; r += kAdThreads / kQuads) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int s = 0; s < shares; ++s) {
        const float4 o = *reinterpret_cast<const float4 *>(
            warp_sums + ((s * m_tiles + r / 16) * 16 + r % 16) * R + col);
        v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
      }
      *reinterpret_cast<float4 *>(sums + r * R + col) = v;
    }
    if (split > 1)
      cluster_sync();
    else
      __syncthreads();

    // ------------------------------------------- all of K, relative to the token's largest, in parts
    const uint32_t sums_at = smem_u32(sums + col);
    const float scale = p.scale[which];
    for (int r0 = 0; r0 < count; r0 += kAdThreads / kQuads) {  // whole warps: they exchange maxima
      const int r = r0 + tid / kQuads;
      float4 all[8];  // read together, added in the CTAs' order
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        all[q] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < count && q < split) all[q] = ld_cluster_f32x4(mapa_shared(sums_at + r * (R * 4), q));
      }
      float v[4] = {all[0].x, all[0].y, all[0].z, all[0].w};
#pragma unroll
      for (int q = 1; q < 8; ++q) v[0] += all[q].x, v[1] += all[q].y, v[2] += all[q].z, v[3] += all[q].w;
      uint32_t top = 0;  // of the finite ones, which stay finite in 16 bits beside an infinity
#pragma unroll
      for (int i = 0; i < 4; ++i) top = max(top, abs_bits(v[i]) < kInfBits ? abs_bits(v[i]) : 0u);
#pragma unroll
      for (int o = 1; o < kQuads; o *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int e = binade(top);
      const float down = pow2(-e);
      uint2 words[kParts];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] *= down;
#pragma unroll
      for (int i = 0; i < kParts; ++i) {
        words[i] = make_uint2(pack2<W>(v[0], v[1]), pack2<W>(v[2], v[3]));
#pragma unroll
        for (int j = 0; j < 4; ++j)  // an infinity is whole in the first part (infinity less itself would be NaN)
          v[j] = abs_bits(v[j]) == kInfBits ? 0.f : v[j] - to_f32(from_f32<W>(v[j]));
      }
      if (r < count) {
#pragma unroll
        for (int i = 0; i < kParts; ++i)
          *reinterpret_cast<uint2 *>(parts + i * Smem::kPart + r * Smem::kRow + col * 2) = words[i];
        if (col == 0) factor[r] = p.xs[m0 + rows[r]] * pow2(e) * scale;
      }
    }
    if (split > 1) cluster_arrive();  // has read the others' sums
    __syncthreads();

    // ---------------------------------------------------------------- B v, this CTA's channels
    const Y *y_tile = y + m0 * p.ldy;
    Y *out_tile = out + m0 * p.ldo;
    const int ldy = static_cast<int>(p.ldy), ldo = static_cast<int>(p.ldo), ldb = static_cast<int>(p.ldb);
    constexpr int kWords = R >= 32 ? 4 : 2;  // a lane's words of a row of B: 8 (4) ranks in a row
    constexpr int kBlocks = R >= 32 ? R / 32 : 1;
    for (int gr = g0 + warp; gr < g1; gr += 8) {
      uint32_t bw[4][kBlocks][kWords];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = 32 * gr + 8 * (g / 2) + 2 * j + g % 2;
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {
          const int k = 32 * i + 2 * kWords * t, left = n < p.N ? rank - k : 0;
#pragma unroll
          for (int w = 0; w < kWords; ++w) bw[j][i][w] = 0;
          if (left > 0) {
            const W *from = b + static_cast<long long>(n) * ldb + k;
            if constexpr (kWords == 4) {
              const uint4 v = *reinterpret_cast<const uint4 *>(from);
              bw[j][i][0] = v.x, bw[j][i][1] = v.y, bw[j][i][2] = v.z, bw[j][i][3] = v.w;
            } else {
              const uint2 v = *reinterpret_cast<const uint2 *>(from);
              bw[j][i][0] = v.x, bw[j][i][1] = v.y;
            }
          }
        }
      }
      if (rank % (2 * kWords)) {  // behind all loads: a look at one value would wait for it
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < kBlocks; ++i) cut_words(bw[j][i], rank - 32 * i - 2 * kWords * t);
      }
      const int n = 32 * gr + 8 * t, left = p.N - n;
      constexpr int kTogether = sizeof(Y) == 4 ? 2 : 4;  // sixteens of tokens whose y is under way together
      const int sixteens = (count + 15) / 16;
      for (int first16 = 0; first16 < sixteens; first16 += kTogether) {
        Eight<Y> yw[kTogether][2];
#pragma unroll
        for (int m = 0; m < kTogether; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = (first16 + m) * 16 + g + 8 * h;
            if (r < count && left > 0) yw[m][h].load(y_tile + static_cast<long long>(rows[r]) * ldy + n, left, start);
          }
#pragma unroll
        for (int m = 0; m < kTogether; ++m) {
          if (first16 + m >= sixteens) break;
          float o[4][4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[j][i] = 0.f;
#pragma unroll
          for (int part_of = 0; part_of < kParts; ++part_of) {
            const uint8_t *from = parts + part_of * Smem::kPart + ((first16 + m) * 16 + g) * Smem::kRow +
                                  4 * kWords * t;
#pragma unroll
            for (int i = 0; i < kBlocks; ++i) {
              uint32_t va[kWords / 2][4];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint8_t *at = from + h * 8 * Smem::kRow + 64 * i;
                if constexpr (kWords == 4) {
                  const uint4 v = *reinterpret_cast<const uint4 *>(at);
                  va[0][h] = v.x, va[0][2 + h] = v.y, va[1][h] = v.z, va[1][2 + h] = v.w;
                } else {
                  const uint2 v = *reinterpret_cast<const uint2 *>(at);
                  va[0][h] = v.x, va[0][2 + h] = v.y;
                }
              }
#pragma unroll
              for (int s = 0; s < kWords / 2; ++s)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  mma16(o[j], va[s], bw[j][i][2 * s], bw[j][i][2 * s + 1], W());
            }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = (first16 + m) * 16 + g + 8 * h;
            if (r >= count || left <= 0) continue;
            const float by = factor[r];
            float f[8];
            yw[m][h].unpack(f);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              f[2 * j] = fmaf(o[j][2 * h], by, f[2 * j]);
              f[2 * j + 1] = fmaf(o[j][2 * h + 1], by, f[2 * j + 1]);
            }
            yw[m][h].pack(f);
            yw[m][h].store(out_tile + static_cast<long long>(rows[r]) * ldo + n, left, start);
          }
        }
      }
    }
    if (split > 1) cluster_wait();  // nobody leaves or writes its sums' place while they are being read
    __syncthreads();                // rows, factors and parts are read
  }
}

}  // namespace voc
