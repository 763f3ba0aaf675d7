// lm_linear.cuh -- product of e4m3 rows with e4m3 weights,
//
//   y[m][n] = xs[m] * ws[n] * sum_k x[m][k] w[n][k] (+ bias[n]),
//
// on the 5th-generation tensor cores (e4m3 products, fp32 accumulation).
#pragma once
#include <cuda.h>

#include "lm_common.cuh"

namespace voc {

struct LmLinearArgs {
  const float *xs, *ws, *bias;
  void *out;
  long long ldo;
  int M, N, K;
  int nt;        // tokens of a tile (a multiple of 16, at most 256)
  int stages, chunks, tmem_cols;
  long long budget;
  int *timeout;
};

constexpr int kLinThreads = 192;     // 4 epilogue warps, 1 copy warp, 1 MMA warp
constexpr int kLinRows = 128;        // weight rows (output channels) of a tile
constexpr int kLinK = 128;           // bytes of K per stage: one 128-byte swizzle row

// Few tokens: the weights take the MMA's M side (128 output channels) and the tokens its N side
// (16 to 256), so that a handful of tokens does not leave the tile's rows empty; the accumulator's
// lanes are output channels.  K is split over the CTAs of a cluster, which add their parts up
// through distributed shared memory in a fixed order.
// Bound by the weights' bytes: 33 tokens, N x K = 12288 x 4096 (51 MB): 12.4 us, 4.1 TB/s, of which about
// 4 us are the launch, the first loads' way and the epilogue; 8 tokens, 1536 x 1024: 3.4 us, these alone.
template <typename T>
__global__ void __launch_bounds__(kLinThreads, 2)
    linear_few_kernel(const __grid_constant__ CUtensorMap xmap,
                      const __grid_constant__ CUtensorMap wmap, const LmLinearArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *ring = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ __align__(8) uint64_t full[16], empty[16], done;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int split = gridDim.z, rank = blockIdx.z;
  const int n0 = blockIdx.x * kLinRows, m0 = blockIdx.y * p.nt;
  const int c0 = static_cast<int>(static_cast<long long>(p.chunks) * rank / split);
  const int c1 = static_cast<int>(static_cast<long long>(p.chunks) * (rank + 1) / split);
  const uint32_t stage_bytes = (kLinRows + p.nt) * kLinK;
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(smem_u32(full + i), 1);
      mbar_init(smem_u32(empty + i), 1);
    }
    mbar_init(smem_u32(&done), 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 5) {
    tmem_alloc(smem_u32(&tmem_slot), p.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const int never = 0;
  volatile int *abort = &abort_flag;
  // Every thread, ahead of its first wait with a limit: the kernel before this one may take longer than
  // the limit, and only from here on does a wait depend on this grid alone.
  pdl_wait();

  int issued = c0;  // copies up to here are under way or done
  if (warp == 4) {
    if (lane == 0) {
      pdl_launch_dependents();  // one thread's call stands for the CTA; by all of them it took 0.2 us more
      for (int c = c0; c < c1; ++c) {
        const int i = c - c0, st = i % p.stages;
        if (i >= p.stages &&
            !mbar_wait(smem_u32(empty + st), (i / p.stages - 1) & 1, p.budget, abort)) {
          *abort = 1;
          break;
        }
        const uint32_t bar = smem_u32(full + st), dst = smem_u32(ring) + st * stage_bytes;
        mbar_arrive_expect_tx(bar, stage_bytes);
        tma_load_2d(dst, &wmap, bar, c * kLinK, n0);
        tma_load_2d(dst + kLinRows * kLinK, &xmap, bar, c * kLinK, m0);
        issued = c + 1;
      }
    }
  } else if (warp == 5) {
    const uint32_t idesc = idesc_e4m3_f32(kLinRows, p.nt);
    for (int c = c0; c < c1; ++c) {
      const int i = c - c0, st = i % p.stages;
      const bool landed = mbar_wait(smem_u32(full + st), (i / p.stages) & 1, p.budget, abort);
      if (!__all_sync(0xffffffffu, landed)) {
        *abort = 1;
        if (p.timeout) *p.timeout = 1;
        break;
      }
      tc_fence_after();
      const uint32_t a = sw128_desc_lo(smem_u32(ring) + st * stage_bytes);
      const uint32_t b = sw128_desc_lo(smem_u32(ring) + st * stage_bytes + kLinRows * kLinK);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        mma_e4m3_warp_lo<false>(tmem, a + 2 * k, b + 2 * k, kSw128DescHi, idesc,
                                i > 0 || k > 0 ? 1u : 0u);
      mma_commit_warp(smem_u32(empty + st));
    }
    mma_commit_warp(smem_u32(&done));
  }
  // every thread waits for the products (after a give-up: for those that were issued)
  if (!mbar_wait(smem_u32(&done), 0, 4 * p.budget, &never)) {
    *abort = 1;
    if (p.timeout) *p.timeout = 1;
  }
  __syncwarp();
  tc_fence_after();

  // The accumulator's lanes are channels: it goes through shared memory as [token][128] so that a
  // warp writes a token's 128 channels in a row.  CTA `rank` adds up every split-th token.
  const int tokens = min(p.nt, p.M - m0);
  float *part = reinterpret_cast<float *>(ring);
  if (warp < 4) {
    for (int t0 = 0; t0 < tokens; t0 += 16) {
      uint32_t r[16];
      tmem_ld16_issue(tmem + (static_cast<uint32_t>(warp * 32) << 16) + t0, r);
      tmem_ld16_wait(r);
#pragma unroll
      for (int j = 0; j < 16; ++j)
        part[(t0 + j) * kLinRows + warp * 32 + lane] = __uint_as_float(r[j]);
    }
  }
  tc_fence_before();
  __syncwarp();
  if (split > 1)
    cluster_sync();
  else
    __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, p.tmem_cols);
  }
  T *out = static_cast<T *>(p.out);
  const int n = n0 + 4 * lane;  // this lane's four channels
  float ws[4], bias[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    ws[j] = n + j < p.N ? p.ws[n + j] : 0.f;
    bias[j] = p.bias && n + j < p.N ? p.bias[n + j] : 0.f;
  }
  // the reads of 4 tokens are in flight together
  constexpr int kWarps = kLinThreads / 32, kTogether = 4;
  for (int t0 = rank + split * warp; t0 < tokens; t0 += kTogether * kWarps * split) {
    float4 v[kTogether];
    float xs[kTogether];
#pragma unroll
    for (int j = 0; j < kTogether; ++j) {
      const int t = t0 + j * kWarps * split;
      v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      xs[j] = t < tokens ? p.xs[m0 + t] : 0.f;
    }
    for (int s = 0; s < split; ++s) {
      const uint32_t from = mapa_shared(smem_u32(part + 4 * lane), s);
      float4 r[kTogether];
#pragma unroll
      for (int j = 0; j < kTogether; ++j) {
        const int t = t0 + j * kWarps * split;
        r[j] = t < tokens ? ld_cluster_f32x4(from + t * (kLinRows * 4))
                          : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int j = 0; j < kTogether; ++j)
        v[j].x += r[j].x, v[j].y += r[j].y, v[j].z += r[j].z, v[j].w += r[j].w;
    }
#pragma unroll
    for (int j = 0; j < kTogether; ++j) {
      const int t = t0 + j * kWarps * split;
      if (t >= tokens) continue;
      T *dst = out + static_cast<long long>(m0 + t) * p.ldo + n;
      const float f[4] = {fmaf(v[j].x * xs[j], ws[0], bias[0]), fmaf(v[j].y * xs[j], ws[1], bias[1]),
                          fmaf(v[j].z * xs[j], ws[2], bias[2]), fmaf(v[j].w * xs[j], ws[3], bias[3])};
      if (n + 4 <= p.N && reinterpret_cast<uintptr_t>(dst) % (4 * sizeof(T)) == 0) {
        if constexpr (sizeof(T) == 4)
          *reinterpret_cast<float4 *>(dst) = make_float4(f[0], f[1], f[2], f[3]);
        else
          *reinterpret_cast<uint2 *>(dst) = make_uint2(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]));
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (n + k < p.N) dst[k] = from_f32<T>(f[k]);
      }
    }
  }
  // Leave with no copy in flight.  Without a give-up (a barrier has been passed since the flag was last
  // raised) the products have waited for every copy.
  if (warp == 4 && lane == 0 && *abort) {
    if (p.timeout) *p.timeout = 1;
    for (int c = max(c0, issued - p.stages); c < issued; ++c)
      if (!mbar_wait(smem_u32(full + (c - c0) % p.stages), ((c - c0) / p.stages) & 1, p.budget, &never))
        break;
  }
  if (split > 1) {
    __syncwarp();
    cluster_sync();  // nobody leaves while its part is being read
  }
}

// Many tokens: 256 tokens x 256 channels by a pair of CTAs that share one MMA (cta_group::2).  Each
// CTA stages its 128 token rows and half of the channels, so the tensor core reads 64 bytes a clock
// from each SM's shared memory where a 128 x 256 tile of one CTA would read 96 beside the copies'
// writes.  Persistent; two accumulators, so a tile's output runs beside the next tile's products.
// Bound by the tensor cores: 15504 tokens, N x K = 4096 x 4096: 139 us, 3.74 PFLOP/s (twice the 16-bit
// peak measured with a library product is 3.81); called back to back for seconds the power limit makes
// it about 166 us.  With a warp that relays the second CTA's loads to the first, in place of copies that
// count on the first one's barrier, it ran at a third of that.
constexpr int kManyTile = 256;
constexpr int kManyStage = 2 * 128 * kLinK;  // bytes of a stage in each CTA
constexpr int kManyStages = 6;
constexpr int kManyOut = 8 * 32 * 64;        // output staging: 32 rows of 64 bytes for each warp
constexpr size_t kManySmem = static_cast<size_t>(kManyStages) * kManyStage + kManyOut + 1024;

// A staged piece, 32 rows of 64 bytes of which `left` values are of the row, to rows that start on
// sizeof(U) bytes, in U: lanes next to each other write what lies next to each other.
template <typename T, typename U>
__device__ __forceinline__ void store_piece(T *dst, long long ldo, const uint8_t *stage, int rows,
                                            int left, int lane) {
  constexpr int kUnits = 64 / static_cast<int>(sizeof(U)), kRows = 32 / kUnits;
  constexpr int kVals = static_cast<int>(sizeof(U) / sizeof(T));
  const int u = lane % kUnits, c = u * kVals;
#pragma unroll
  for (int i = 0; i < 32 / kRows; ++i) {
    const int r = i * kRows + lane / kUnits, at = u * static_cast<int>(sizeof(U));
    const U v = *reinterpret_cast<const U *>(stage + r * 64 + ((at / 16 ^ (r >> 1 & 3)) << 4) + at % 16);
    if (r >= rows) continue;
    T *to = dst + r * ldo + c;
    if (c + kVals <= left) {
      *reinterpret_cast<U *>(to) = v;
    } else if constexpr (kVals > 1) {
      T e[kVals];
      memcpy(e, &v, sizeof(U));
#pragma unroll
      for (int j = 0; j < kVals; ++j)
        if (c + j < left) to[j] = e[j];
    }
  }
}

constexpr int kManyEpi = 8;                          // epilogue warps, two for each 32 token rows
constexpr int kManyThreads = 32 * (kManyEpi + 2);    // and a copy warp and an MMA warp

template <typename T>
__global__ void __launch_bounds__(kManyThreads, 1) __cluster_dims__(2, 1, 1)
    linear_many_kernel(const __grid_constant__ CUtensorMap xmap,
                       const __grid_constant__ CUtensorMap wmap, const LmLinearArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *ring = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  // full: both halves of a stage have landed (the even CTA's barriers count both CTAs' copies)
  __shared__ __align__(8) uint64_t full[kManyStages], empty[kManyStages], acc_full[2],
      acc_empty[2], drain, unused;
  __shared__ __align__(16) float col_scale[2][kManyTile], col_bias[2][kManyTile];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();
  const int m_tiles = (p.M + kManyTile - 1) / kManyTile, n_tiles = (p.N + kManyTile - 1) / kManyTile;
  const long long jobs = static_cast<long long>(m_tiles) * n_tiles;
  const long long job0 = cluster_id_x(), step = cluster_count_x();
  volatile int *abort = &abort_flag;
  const int never = 0;
  auto raise = [&]() {
    *abort = 1;
    st_cluster_u32(mapa_shared(smem_u32(&abort_flag), rank ^ 1u), 1u);
    if (p.timeout) *p.timeout = 1;
  };
  if (threadIdx.x == 0) {
    for (int i = 0; i < kManyStages; ++i) {
      mbar_init(smem_u32(full + i), 1);
      mbar_init(smem_u32(empty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(acc_full + i), 1);
      mbar_init(smem_u32(acc_empty + i), 2 * kManyEpi);  // the epilogue warps of both CTAs
    }
    mbar_init(smem_u32(&drain), 1);
    mbar_init(smem_u32(&unused), 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kManyEpi + 1) {
    tmem_alloc_pair(smem_u32(&tmem_slot), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();  // the other CTA's barriers stand before anything arrives there
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  pdl_wait();  // every thread, ahead of its first wait with a limit (as in linear_few_kernel)
  pdl_launch_dependents();

  if (warp == kManyEpi) {
    if (lane == 0) {
      const uint32_t full0 = mapa_shared(smem_u32(full), 0u);
      int it = 0;
      bool ok = true;
      for (long long job = job0; job < jobs && ok; job += step) {
        const int m0 = static_cast<int>(job / n_tiles) * kManyTile + 128 * static_cast<int>(rank);
        const int n0 = static_cast<int>(job % n_tiles) * kManyTile + 128 * static_cast<int>(rank);
        for (int c = 0; c < p.chunks; ++c, ++it) {
          const int st = it % kManyStages;
          if (it >= kManyStages &&
              !mbar_wait_cluster(smem_u32(empty + st), (it / kManyStages - 1) & 1, p.budget, abort)) {
            ok = false;
            break;
          }
          const uint32_t dst = smem_u32(ring) + st * kManyStage;
          if (rank == 0) mbar_arrive_expect_tx(smem_u32(full + st), 2 * kManyStage);
          tma_load_2d_pair(dst, &xmap, full0 + st * 8, c * kLinK, m0);
          tma_load_2d_pair(dst + kManyStage / 2, &wmap, full0 + st * 8, c * kLinK, n0);
        }
      }
      // Leave with no copy in flight, also where the products give up after the last copy was issued: the
      // even CTA's barriers count both CTAs' copies, and neither leaves without the other.
      if (rank == 0)
        for (int i = max(0, it - kManyStages); i < it && ok; ++i)
          ok = mbar_wait_cluster(smem_u32(full + i % kManyStages), (i / kManyStages) & 1, p.budget,
                                 &never);
      if (!ok) {
        raise();
        // the odd CTA may have issued more: that lands well within this wait, which nothing ends early
        mbar_wait(smem_u32(&unused), 0, p.budget, &never);
      }
    }
  } else if (warp == kManyEpi + 1 && rank == 0) {
    constexpr uint32_t kId = idesc_e4m3_f32(256, kManyTile);
    auto wait = [&](uint64_t *bar, int parity) {
      const bool got = mbar_wait_cluster(smem_u32(bar), parity, p.budget, abort);
      return __all_sync(0xffffffffu, got) != 0;
    };
    int it = 0, k = 0;
    bool ok = true;
    for (long long job = job0; job < jobs && ok; job += step, ++k) {
      const int acc = k & 1;
      if (k >= 2 && !wait(acc_empty + acc, (k / 2 - 1) & 1)) {
        ok = false;
        break;
      }
      tc_fence_after();
      for (int c = 0; c < p.chunks; ++c, ++it) {
        const int st = it % kManyStages, ph = (it / kManyStages) & 1;
        if (!wait(full + st, ph)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t a = sw128_desc_lo(smem_u32(ring) + st * kManyStage);
        const uint32_t b = sw128_desc_lo(smem_u32(ring) + st * kManyStage + kManyStage / 2);
#pragma unroll
        for (int s = 0; s < 4; ++s)
          mma_e4m3_warp_lo<true>(tmem + acc * kManyTile, a + 2 * s, b + 2 * s, kSw128DescHi, kId,
                                 c > 0 || s > 0 ? 1u : 0u);
        mma_commit_pair_warp(smem_u32(empty + st), 3);
      }
      if (ok) mma_commit_pair_warp(smem_u32(acc_full + acc), 3);
    }
    if (!ok) raise();
    mma_commit_pair_warp(smem_u32(&drain), 1);
    mbar_wait_cluster(smem_u32(&drain), 0, 4 * p.budget, &never);
    __syncwarp();
  } else if (warp < kManyEpi) {
    // The accumulator's lanes are token rows.  A warp takes 32 rows of half of the columns and turns
    // pieces of 32 rows x 64 bytes around in shared memory, so that its stores fill whole sectors.
    constexpr int kCols = 64 / static_cast<int>(sizeof(T));  // columns of a staged piece
    constexpr int kPer = 16 / static_cast<int>(sizeof(T));
    const int quad = warp % 4, c_first = warp / 4 * (kManyTile / 2);
    T *out = static_cast<T *>(p.out);
    // what every output row (and so every piece of one, 64 bytes apart) starts on
    const uint32_t start = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(out)) |
                           static_cast<uint32_t>(p.ldo * sizeof(T));
    const uint32_t empty0 = mapa_shared(smem_u32(acc_empty), 0u);
    const uint32_t stage = smem_u32(ring) + kManyStages * kManyStage + warp * (32 * 64);
    int k = 0;
    bool ok = true;  // after a give-up the warps go on without work: all meet at every barrier
    for (long long job = job0; job < jobs; job += step, ++k) {
      const int acc = k & 1;
      const int row0 = static_cast<int>(job / n_tiles) * kManyTile + 128 * static_cast<int>(rank) +
                       quad * 32;
      const int n0 = static_cast<int>(job % n_tiles) * kManyTile;
      const int cols = min(kManyTile, p.N - n0);
      for (int c = threadIdx.x; c < kManyTile; c += 32 * kManyEpi) {
        col_scale[acc][c] = c < cols ? p.ws[n0 + c] : 0.f;
        col_bias[acc][c] = p.bias && c < cols ? p.bias[n0 + c] : 0.f;
      }
      const float xs = row0 + lane < p.M ? p.xs[row0 + lane] : 0.f;
      asm volatile("bar.sync 1, 256;" ::: "memory");  // the epilogue warps
      const bool got =
          ok && mbar_wait_cluster(smem_u32(acc_full + acc), (k / 2) & 1, 4 * p.budget, abort);
      if (!__all_sync(0xffffffffu, got)) {
        if (ok && lane == 0) raise();
        ok = false;
        continue;
      }
      tc_fence_after();
      const int c_end = min(cols, c_first + kManyTile / 2);
      for (int c0 = c_first; c0 < c_end; c0 += kCols) {
        uint32_t r[kCols];
        const uint32_t from =
            tmem + (static_cast<uint32_t>(quad * 32) << 16) + acc * kManyTile + c0;
        if constexpr (kCols == 32) {
          tmem_ld32_issue(from, r);
          tmem_ld_wait_all();
          tmem_ld32_after_wait(r);
        } else {
          tmem_ld16_issue(from, r);
          tmem_ld16_wait(r);
        }
        __syncwarp();  // the previous piece has been read
#pragma unroll
        for (int i = 0; i < kCols; i += kPer) {
          T e[kPer];
#pragma unroll
          for (int j = 0; j < kPer; j += 4) {
            const float4 w = *reinterpret_cast<const float4 *>(&col_scale[acc][c0 + i + j]);
            const float4 z = *reinterpret_cast<const float4 *>(&col_bias[acc][c0 + i + j]);
            e[j] = from_f32<T>(fmaf(__uint_as_float(r[i + j]) * xs, w.x, z.x));
            e[j + 1] = from_f32<T>(fmaf(__uint_as_float(r[i + j + 1]) * xs, w.y, z.y));
            e[j + 2] = from_f32<T>(fmaf(__uint_as_float(r[i + j + 2]) * xs, w.z, z.z));
            e[j + 3] = from_f32<T>(fmaf(__uint_as_float(r[i + j + 3]) * xs, w.w, z.w));
          }
          uint4 v;
          memcpy(&v, e, 16);
          sts128(stage + lane * 64 + (((i / kPer) ^ (lane >> 1 & 3)) << 4), v);
        }
        __syncwarp();
        T *dst = out + static_cast<long long>(row0) * p.ldo + n0 + c0;
        const uint8_t *piece = ring + kManyStages * kManyStage + warp * (32 * 64);
        if (start % 16 == 0)
          store_piece<T, uint4>(dst, p.ldo, piece, p.M - row0, cols - c0, lane);
        else if (start % 4 == 0)
          store_piece<T, uint32_t>(dst, p.ldo, piece, p.M - row0, cols - c0, lane);
        else
          store_piece<T, T>(dst, p.ldo, piece, p.M - row0, cols - c0, lane);
      }
      __syncwarp();
      tc_fence_before();
      if (lane == 0) mbar_arrive_cluster(empty0 + acc * 8);
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // neither CTA leaves while the other may reach its barriers
  if (warp == kManyEpi + 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

}  // namespace voc
