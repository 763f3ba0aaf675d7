// lm_rows.cuh -- rows of a token model to e4m3 with one 32-bit scale per row.
//
//   h = x (+ residual, in 32 bits; the sum also goes out, rounded once to x's type)
//   n = h * (1 / sqrt(mean(h^2) + eps)) * weight      VOC_LM_RMS
//   n = h                                             VOC_LM_NONE
//   n = g / (1 + e^-g) * u, x = [g | u]               VOC_LM_GATED
//   scale = max(max|n|, 2^-96) / 448,  q = e4m3(n / scale)
//
// The norm is taken of the 32-bit sum, not of the rounded one: the sum is at hand and one
// rounding less reaches q.
#pragma once
#include <type_traits>

#include "lm_common.cuh"

namespace voc {

struct LmRowsArgs {
  const void *x, *res, *w;
  void *sum;
  uint8_t *out;
  float *scale;
  long long rows, ldx, ldr, lds, ldo;
  int d;
  float eps;
};

enum { kRowsRms = 0, kRowsNone = 1, kRowsGated = 2 };

// Factors of a row's norm: n = (h * pre) * rs * weight.  Squares of the usual magnitudes are
// summed as they are (pre = 1); rows of very large or very small values are summed again with
// their largest magnitude brought near 1, so that no square overflows or vanishes.
struct RowNorm {
  float pre, rs;
};
__device__ __forceinline__ bool rms_needs_scaling(uint32_t amax) {
  const float a = __uint_as_float(amax);
  return amax < kInfBits && a != 0.f && (a > 0x1p50f || a < 0x1p-50f);
}
__device__ __forceinline__ float rms_prescale(uint32_t amax) {
  const int e = static_cast<int>(amax >> 23) - 127;  // -127 for subnormals
  return pow2(min(100, -e));
}
__device__ __forceinline__ float rms_factor(float sumsq, int d, float eps, float pre) {
  const float ms = sumsq / static_cast<float>(d);
  const float e = eps * pre * pre;
  if (e > 0x1p100f) return 1.f / (sqrtf(eps) * pre);  // the squares count for nothing beside eps
  const float v = ms + e;
  return v > 0.f ? 1.f / sqrtf(v) : (v == 0.f ? 0.f : v);  // a row of zeros without eps: zeros
}

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.f + expf(-g)) * u; }

// scale and 1/scale of a row whose largest |n| has the bits `amax` (NaN kept).
__device__ __forceinline__ float2 row_scale(uint32_t amax) {
  const float a = amax > kInfBits ? __uint_as_float(amax) : fmaxf(__uint_as_float(amax), kScaleMin);
  return make_float2(a / kE4m3Max, kE4m3Max / a);
}

// Any width, stride and alignment: one CTA per row, the row read once per pass (the later passes
// from cache).
template <typename T, int MODE>
__global__ void __launch_bounds__(256) rows_any_kernel(const LmRowsArgs p) {
  __shared__ float red[32];
  pdl_wait();
  pdl_launch_dependents();
  const long long row = blockIdx.x;
  const T *x = static_cast<const T *>(p.x) + row * p.ldx;
  const T *r = p.res ? static_cast<const T *>(p.res) + row * p.ldr : nullptr;
  const T *w = static_cast<const T *>(p.w);
  T *s = p.sum ? static_cast<T *>(p.sum) + row * p.lds : nullptr;
  auto load = [&](int i) {
    if (MODE == kRowsGated) return silu_mul(to_f32(x[i]), to_f32(x[p.d + i]));
    const float h = to_f32(x[i]);
    return r ? h + to_f32(r[i]) : h;
  };
  float pre = 1.f, rs = 1.f;
  if (MODE == kRowsRms) {
    float ss = 0.f;
    uint32_t m = 0;
    for (int i = threadIdx.x; i < p.d; i += 256) {
      const float h = load(i);
      ss += h * h;
      m = max(m, abs_bits(h));
    }
    ss = group_sum<256>(ss, red);
    m = group_max<256>(m, red);
    if (rms_needs_scaling(m)) {
      pre = rms_prescale(m);
      ss = 0.f;
      for (int i = threadIdx.x; i < p.d; i += 256) {
        const float h = load(i) * pre;
        ss += h * h;
      }
      ss = group_sum<256>(ss, red);
    }
    rs = rms_factor(ss, p.d, p.eps, pre);
  }
  auto norm = [&](float h, int i) {
    return MODE == kRowsRms ? h * pre * rs * to_f32(w[i]) : h;
  };
  uint32_t m = 0;
  for (int i = threadIdx.x; i < p.d; i += 256) m = max(m, abs_bits(norm(load(i), i)));
  m = group_max<256>(m, red);
  const float2 sc = row_scale(m);
  if (threadIdx.x == 0) p.scale[row] = sc.x;
  for (int i = threadIdx.x; i < p.d; i += 256) {
    const float h = load(i);  // read before the sum's store: the sum may take x's or r's place
    if (s) s[i] = from_f32<T>(h);
    p.out[row * p.ldo + i] = e4m3(norm(h, i) * sc.y);
  }
}

// Loads and stores of VB bytes of T (N values).
template <typename T, int VB>
struct RowVec {
  static constexpr int N = VB / static_cast<int>(sizeof(T));
  using Raw = typename std::conditional<
      VB == 16, uint4,
      typename std::conditional<VB == 8, uint2,
                                typename std::conditional<VB == 4, uint32_t,
                                                          uint16_t>::type>::type>::type;
  union U {
    Raw raw;
    T v[N];
    __device__ U() {}
  };
  static __device__ __forceinline__ void load(const T *p, float (&f)[N]) {
    U u;
    u.raw = *reinterpret_cast<const Raw *>(p);
#pragma unroll
    for (int j = 0; j < N; ++j) f[j] = to_f32(u.v[j]);
  }
  static __device__ __forceinline__ void store(T *p, const float *f) {
    U u;
#pragma unroll
    for (int j = 0; j < N; ++j) u.v[j] = from_f32<T>(f[j]);
    *reinterpret_cast<Raw *>(p) = u.raw;
  }
};

constexpr int kRowValues = 32;    // values of a row that a thread keeps in registers
constexpr int kRowThreads = 512;  // most threads of a row: rows of up to 16384 values

// Sum or maximum over a row's `tpr` threads (a power of two from 32 on); `red` has a float per
// warp.  The order is fixed.
template <bool MAX>
__device__ __forceinline__ uint32_t row_reduce(uint32_t v, int tpr, float *red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const uint32_t w = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? max(v, w) : __float_as_uint(__uint_as_float(v) + __uint_as_float(w));
  }
  if (tpr > 32) {
    __syncthreads();
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = __uint_as_float(v);
    __syncthreads();
    const int base = threadIdx.x / tpr * (tpr / 32);
    v = __float_as_uint(red[base]);
    for (int i = 1; i < tpr / 32; ++i) {
      const uint32_t w = __float_as_uint(red[base + i]);
      v = MAX ? max(v, w) : __float_as_uint(__uint_as_float(v) + __uint_as_float(w));
    }
  }
  return v;
}

// Rows of up to 16384 values, each read once and kept in registers by its `tpr` threads.  VB is the
// widest access that the row's buffers and strides allow.
template <typename T, int MODE, int VB>
__global__ void __launch_bounds__(kRowThreads) rows_kernel(const LmRowsArgs p, const int tpr) {
  using Vec = RowVec<T, VB>;
  constexpr int N = Vec::N, kChunks = kRowValues / N;
  __shared__ float red[kRowThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x % tpr;
  const long long row =
      static_cast<long long>(blockIdx.x) * (blockDim.x / tpr) + threadIdx.x / tpr;
  const bool live = row < p.rows;  // spare threads of the last block keep to the barriers
  const int chunks = live ? p.d / N : 0;
  const T *x = static_cast<const T *>(p.x) + row * p.ldx;
  const T *r = static_cast<const T *>(p.res) + row * p.ldr;
  const T *w = static_cast<const T *>(p.w);
  float h[kChunks][N];
  uint32_t m = 0;
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int c = lane + i * tpr;
    if (c < chunks) {
      Vec::load(x + c * N, h[i]);
      if (MODE == kRowsGated) {
        float u[N];
        Vec::load(x + p.d + c * N, u);
#pragma unroll
        for (int j = 0; j < N; ++j) h[i][j] = silu_mul(h[i][j], u[j]);
      } else if (p.res) {
        float u[N];
        Vec::load(r + c * N, u);
#pragma unroll
        for (int j = 0; j < N; ++j) h[i][j] += u[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) h[i][j] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      m = max(m, abs_bits(h[i][j]));
      if (MODE == kRowsRms) ss = fmaf(h[i][j], h[i][j], ss);
    }
  }
  if (p.sum) {
    T *s = static_cast<T *>(p.sum) + row * p.lds;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int c = lane + i * tpr;
      if (c < chunks) Vec::store(s + c * N, h[i]);
    }
  }
  if (MODE == kRowsRms) {
    ss = __uint_as_float(row_reduce<false>(__float_as_uint(ss), tpr, red));
    m = row_reduce<true>(m, tpr, red);
    float pre = 1.f;
    if (tpr > 32 ? __syncthreads_or(rms_needs_scaling(m)) : rms_needs_scaling(m)) {
      if (rms_needs_scaling(m)) pre = rms_prescale(m);
      float again = 0.f;
#pragma unroll
      for (int i = 0; i < kChunks; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) {
          h[i][j] *= pre;
          again = fmaf(h[i][j], h[i][j], again);
        }
      ss = __uint_as_float(row_reduce<false>(__float_as_uint(again), tpr, red));
    }
    const float rs = rms_factor(ss, p.d, p.eps, pre);
    m = 0;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int c = lane + i * tpr;
      if (c < chunks) {
        float u[N];
        Vec::load(w + c * N, u);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          h[i][j] = h[i][j] * rs * u[j];
          m = max(m, abs_bits(h[i][j]));
        }
      }
    }
  }
  m = row_reduce<true>(m, tpr, red);
  const float2 sc = row_scale(m);
  if (live && lane == 0) p.scale[row] = sc.x;
  uint8_t *out = p.out + row * p.ldo;
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int c = lane + i * tpr;
    if (c < chunks) {
      if constexpr (N == 1) {
        out[c] = e4m3(h[i][0] * sc.y);
      } else {
        uint32_t q[(N + 3) / 4];
#pragma unroll
        for (int j = 0; j < N; j += 2) {
          const uint32_t two = e4m3x2(h[i][j] * sc.y, h[i][j + 1] * sc.y);
          q[j / 4] = j % 4 ? q[j / 4] | two << 16 : two;
        }
        if constexpr (N == 8)
          *reinterpret_cast<uint2 *>(out + c * N) = make_uint2(q[0], q[1]);
        else if constexpr (N == 4)
          *reinterpret_cast<uint32_t *>(out + c * N) = q[0];
        else
          *reinterpret_cast<uint16_t *>(out + c * N) = static_cast<uint16_t>(q[0]);
      }
    }
  }
}

}  // namespace voc
