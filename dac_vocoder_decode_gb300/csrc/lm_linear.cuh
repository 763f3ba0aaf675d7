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
template <typename T>
__global__ void __launch_bounds__(kLinThreads, 1)
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

  if (warp == 4) {
    if (lane == 0) {
      pdl_wait();
      int issued = c0;
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
      if (*abort) {  // leave with no copy in flight
        for (int c = max(c0, issued - p.stages); c < issued; ++c)
          mbar_wait(smem_u32(full + (c - c0) % p.stages), ((c - c0) / p.stages) & 1, p.budget,
                    &never);
        if (p.timeout) *p.timeout = 1;
      }
    }
  } else if (warp == 5) {
    const uint32_t idesc = idesc_e4m3_f32(kLinRows, p.nt);
    for (int c = c0; c < c1; ++c) {
      const int i = c - c0, st = i % p.stages;
      const bool landed = mbar_wait(smem_u32(full + st), (i / p.stages) & 1, p.budget, abort);
      if (!__all_sync(0xffffffffu, landed)) {
        *abort = 1;
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

  T *out = static_cast<T *>(p.out);
  const int tokens = min(p.nt, p.M - m0);
  const int feat = n0 + warp * 32 + lane;
  float *part = reinterpret_cast<float *>(ring);  // [token][128], split > 1
  if (warp < 4) {
    pdl_wait();
    const float ws = feat < p.N ? p.ws[feat] : 0.f;
    const float bias = p.bias && feat < p.N ? p.bias[feat] : 0.f;
    for (int t0 = 0; t0 < tokens; t0 += 16) {
      uint32_t r[16];
      tmem_ld16_issue(tmem + (static_cast<uint32_t>(warp * 32) << 16) + t0, r);
      tmem_ld16_wait(r);
      if (split > 1) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          part[(t0 + j) * kLinRows + warp * 32 + lane] = __uint_as_float(r[j]);
      } else if (feat < p.N) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (t0 + j < tokens) {
            const long long row = m0 + t0 + j;
            out[row * p.ldo + feat] = from_f32<T>(__uint_as_float(r[j]) * p.xs[row] * ws + bias);
          }
      }
    }
    if (split > 1) {
      __syncwarp();
      cluster_sync();
      if (feat < p.N)
        for (int t = rank; t < tokens; t += split) {
          float v = 0.f;
          const uint32_t at = smem_u32(part + t * kLinRows + warp * 32 + lane);
          for (int s = 0; s < split; ++s) v += ld_cluster_f32(mapa_shared(at, s));
          const long long row = m0 + t;
          out[row * p.ldo + feat] = from_f32<T>(v * p.xs[row] * ws + bias);
        }
      __syncwarp();
      cluster_sync();  // nobody leaves while its part is being read
    }
  } else if (split > 1) {
    __syncwarp();
    cluster_sync();
    cluster_sync();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 5) tmem_dealloc(tmem, p.tmem_cols);
}

}  // namespace voc
