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

}  // namespace voc
