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
  const int e = static_cast<int>(amax >> 23) - 127;  // -127 for subnormals, 127 at most
  return pow2(max(-126, min(100, -e)));              // 2^-127 would not be a normal number
}
__device__ __forceinline__ float rms_factor(float sumsq, int d, float eps, float pre) {
  const float ms = sumsq / static_cast<float>(d);
  const float e = eps * pre * pre;
  if (e > 0x1p100f) return 1.f / (sqrtf(eps) * pre);  // the squares count for nothing beside eps
  const float v = ms + e;
  return v > 0.f ? 1.f / sqrtf(v) : (v == 0.f ? 0.f : v);  // a row of zeros without eps: zeros
}

// The exponential's and the reciprocal's approximations are good to a few 2^-23 (far below zero the
// rounding of the exponent's argument makes it 2^-17), far inside half an e4m3 step.  For gates from
// kGateLow on, where the reciprocal still is a normal number.  (Six instructions a value; with a full
// division 4001 x 4100 took 0.8 us more.)
constexpr float kGateLow = -80.f;
__device__ __forceinline__ float silu_mul(float g, float u) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2(-1.44269504f * g)));
  return g * r * u;
}
// The same for any gate.  Below kGateLow 1 / (1 + e^-g) is e^g, which u may bring back into range: a half
// of it goes to either factor.  (NaN takes the first way, and stays.)
__device__ __forceinline__ float silu_mul_any(float g, float u) {
  if (!(g < kGateLow)) return silu_mul(g, u);
  const float t = expf(0.5f * g);
  return (g * t) * (u * t);
}

// Whether a row's sum of squares lost nothing: no overflow, and squares that vanished count for less
// than 2^-24 of it.
__device__ __forceinline__ bool rms_sum_holds(float ss) { return ss >= 0x1p-60f && ss < INFINITY; }

// scale and 1/scale of a row whose largest |n| has the bits `amax` (NaN kept).
__device__ __forceinline__ float2 row_scale(uint32_t amax) {
  const float a = amax > kInfBits ? __uint_as_float(amax) : fmaxf(__uint_as_float(amax), kScaleMin);
  return make_float2(a / kE4m3Max, kE4m3Max / a);
}

constexpr int kRowValues = 32;    // values of a row that a thread keeps in registers
constexpr int kAnyThreads = 256;  // threads of a row of any width
constexpr int kRowThreads = 512;  // most threads of a row that is kept in registers: 16384 values

// Sum, or maximum of magnitudes as bits (NaN kept), over a row's `tpr` threads (a power of two from 32 on);
// `red` has a float per warp.  The order is fixed.
__device__ __forceinline__ float row_sum(float v, int tpr, float *red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (tpr > 32) {
    __syncthreads();
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    const int base = threadIdx.x / tpr * (tpr / 32);
    v = red[base];
    for (int i = 1; i < tpr / 32; ++i) v += red[base + i];
  }
  return v;
}
__device__ __forceinline__ uint32_t row_max(uint32_t bits, int tpr, float *red) {
  uint32_t v = __reduce_max_sync(0xffffffffu, bits);
  if (tpr > 32) {
    __syncthreads();
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = __uint_as_float(v);
    __syncthreads();
    const int base = threadIdx.x / tpr * (tpr / 32);
    v = __float_as_uint(red[base]);
    for (int i = 1; i < tpr / 32; ++i) v = max(v, __float_as_uint(red[base + i]));
  }
  return v;
}

// Rows of more than 16384 values (unaligned: less a vector), any stride and alignment: one CTA per row,
// the row read once per pass (the later passes from cache), a value at a time.  Bound by its dependent loads: 512 x 20000
// bf16 with norm and residual 65 us (1.1 TB/s), gated 31 us.
template <typename T, int MODE>
__global__ void __launch_bounds__(kAnyThreads) rows_any_kernel(const LmRowsArgs p) {
  __shared__ float red[kAnyThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  const long long row = blockIdx.x;
  const T *x = static_cast<const T *>(p.x) + row * p.ldx;
  const T *r = p.res ? static_cast<const T *>(p.res) + row * p.ldr : nullptr;
  const T *w = static_cast<const T *>(p.w);
  T *s = p.sum ? static_cast<T *>(p.sum) + row * p.lds : nullptr;
  auto load = [&](int i) {
    if (MODE == kRowsGated) return silu_mul_any(to_f32(x[i]), to_f32(x[p.d + i]));
    const float h = to_f32(x[i]);
    return r ? h + to_f32(r[i]) : h;
  };
  float pre = 1.f, rs = 1.f;
  if (MODE == kRowsRms) {
    float ss = 0.f;
    uint32_t m = 0;
    for (int i = threadIdx.x; i < p.d; i += kAnyThreads) {
      const float h = load(i);
      ss += h * h;
      m = max(m, abs_bits(h));
    }
    ss = row_sum(ss, kAnyThreads, red);
    m = row_max(m, kAnyThreads, red);
    if (rms_needs_scaling(m)) {
      pre = rms_prescale(m);
      ss = 0.f;
      for (int i = threadIdx.x; i < p.d; i += kAnyThreads) {
        const float h = load(i) * pre;
        ss += h * h;
      }
      ss = row_sum(ss, kAnyThreads, red);
    }
    rs = rms_factor(ss, p.d, p.eps, pre);
  }
  auto norm = [&](float h, int i) {
    return MODE == kRowsRms ? h * pre * rs * to_f32(w[i]) : h;
  };
  uint32_t m = 0;
  for (int i = threadIdx.x; i < p.d; i += kAnyThreads) m = max(m, abs_bits(norm(load(i), i)));
  m = row_max(m, kAnyThreads, red);
  const float2 sc = row_scale(m);
  if (threadIdx.x == 0) p.scale[row] = sc.x;
  for (int i = threadIdx.x; i < p.d; i += kAnyThreads) {
    const float h = load(i);  // read before the sum's store: the sum may take x's or r's place
    if (s) s[i] = from_f32<T>(h);
    p.out[row * p.ldo + i] = e4m3(norm(h, i) * sc.y);
  }
}

// Loads and stores of VB bytes of T (N values), 16 or 8.
template <typename T, int VB>
struct RowVec {
  static constexpr int N = VB / static_cast<int>(sizeof(T));
  static constexpr int kWords = VB / 4;
  using Words = uint32_t[kWords];
  static __device__ __forceinline__ void load(const T *p, Words &w) {
    if constexpr (VB == 16) {
      const uint4 u = *reinterpret_cast<const uint4 *>(p);
      w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    } else {
      const uint2 u = *reinterpret_cast<const uint2 *>(p);
      w[0] = u.x, w[1] = u.y;
    }
  }
  static __device__ __forceinline__ void store(T *p, const Words &w) {
    if constexpr (VB == 16)
      *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else
      *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
  }
  static __device__ __forceinline__ void unpack(const Words &w, float (&f)[N]) {
#pragma unroll
    for (int j = 0; j < kWords; ++j) {
      if constexpr (sizeof(T) == 4)
        f[j] = __uint_as_float(w[j]);
      else
        unpack2<T>(w[j], f[2 * j], f[2 * j + 1]);
    }
  }
  static __device__ __forceinline__ void pack(const float (&f)[N], Words &w) {
#pragma unroll
    for (int j = 0; j < kWords; ++j) {
      if constexpr (sizeof(T) == 4)
        w[j] = __float_as_uint(f[j]);
      else
        w[j] = pack2<T>(f[2 * j], f[2 * j + 1]);
    }
  }
  // Whether one of the values is below `bound` (NaN is not).
  template <int CH>
  static __device__ __forceinline__ bool any_below(const Words (&w)[CH], float bound) {
    float lo[2] = {INFINITY, INFINITY};
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int j = 0; j < kWords; ++j) lo[j % 2] = fminf(lo[j % 2], __uint_as_float(w[i][j]));
    } else {
      uint32_t m = w[0][0];
#pragma unroll
      for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int j = 0; j < kWords; ++j) m = min2<T>(m, w[i][j]);
      unpack2<T>(m, lo[0], lo[1]);
    }
    return fminf(lo[0], lo[1]) < bound;
  }
  // The same from and to any place of T's alignment: whole words where they are, and 16-bit values at
  // the ends of a stretch that starts between two.
  static __device__ __forceinline__ void load_any(const T *p, Words &w) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    if (at % VB == 0) {
      load(p, w);
    } else if (at % 4 == 0) {
#pragma unroll
      for (int j = 0; j < kWords; ++j) w[j] = reinterpret_cast<const uint32_t *>(p)[j];
    } else {
      const uint16_t *h = reinterpret_cast<const uint16_t *>(p);
      uint32_t mid[kWords - 1];
#pragma unroll
      for (int j = 0; j < kWords - 1; ++j) mid[j] = *reinterpret_cast<const uint32_t *>(h + 1 + 2 * j);
      const uint32_t first = h[0], last = h[2 * kWords - 1];
      w[0] = first | mid[0] << 16;
#pragma unroll
      for (int j = 1; j < kWords - 1; ++j) w[j] = __funnelshift_r(mid[j - 1], mid[j], 16);
      w[kWords - 1] = mid[kWords - 2] >> 16 | last << 16;
    }
  }
  static __device__ __forceinline__ void store_any(T *p, const Words &w) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    if (at % VB == 0) {
      store(p, w);
    } else if (at % 4 == 0) {
#pragma unroll
      for (int j = 0; j < kWords; ++j) reinterpret_cast<uint32_t *>(p)[j] = w[j];
    } else {
      uint16_t *h = reinterpret_cast<uint16_t *>(p);
      h[0] = static_cast<uint16_t>(w[0]);
#pragma unroll
      for (int j = 0; j < kWords - 1; ++j)
        *reinterpret_cast<uint32_t *>(h + 1 + 2 * j) = __funnelshift_r(w[j], w[j + 1], 16);
      h[2 * kWords - 1] = static_cast<uint16_t>(w[kWords - 1] >> 16);
    }
  }
  // Those of the values that lie in [0, d), the first of them at row[e0]; zeros for the others.
  static __device__ __forceinline__ void load_part(const T *row, int e0, int d, Words &w) {
    constexpr int kPer = 4 / static_cast<int>(sizeof(T));
#pragma unroll
    for (int j = 0; j < N; ++j) {
      uint32_t v = 0;
      if (e0 + j >= 0 && e0 + j < d) {
        if constexpr (kPer == 1)
          v = reinterpret_cast<const uint32_t *>(row)[e0 + j];
        else
          v = reinterpret_cast<const uint16_t *>(row)[e0 + j];
      }
      w[j / kPer] = j % kPer ? w[j / kPer] | v << 16 : v;
    }
  }
};

// Rows of up to 16384 values, each read once and kept in registers by its `tpr` threads, CH
// vectors of VB bytes each.  VB is the widest access that the row's buffers and strides allow, 16 or 8.
// With d values a row moves 7 d bytes (16-bit, residual), and the kernel has to spend few
// instructions on a value to keep up with that: conversions two at a time, and magnitudes before
// the norm are looked at only where the sum of squares says that squares overflowed or vanished.
// ANY: rows of any alignment (odd widths).  The vectors lie on the codes' 8-byte grid (4 for f32), each
// buffer is read and written at them in the widest accesses of its own alignment, and the first and
// the last vector, where the row covers them only in part, value by value.
// Measured (bf16, residual): 15504 x 1536 27.8 us, 6.0 TB/s, where a plain copy reaches 6.8 (one value
// at a time it was 46.5 us); 15504 x 1537 57 us (in the accesses that every row allows, 2 bytes, 137),
// 1538 40 (4 bytes: 51); 2000 x 16384 40 us, 5.7 TB/s; 8 x 1024 2.2 us, a launch and a chain of two
// loads and two reductions.  Gated 4001 x 4100 f16: 19.1 us, 4.3 TB/s: 8-byte accesses (the rows'
// second halves start on 8 bytes), 4 rows in flight on an SM, each read, reduced and written in turn.
template <typename T, int MODE, int VB, int CH, bool ANY>
__global__ void __launch_bounds__(kRowThreads) rows_kernel(const LmRowsArgs p, const int tpr) {
  using Vec = RowVec<T, VB>;
  constexpr int N = Vec::N;
  __shared__ float red[kRowThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x % tpr;
  const long long row =
      static_cast<long long>(blockIdx.x) * (blockDim.x / tpr) + threadIdx.x / tpr;
  const bool live = row < p.rows;  // spare threads of the last block keep to the barriers
  const T *x = static_cast<const T *>(p.x) + row * p.ldx;
  const T *w = static_cast<const T *>(p.w);
  uint8_t *out = p.out + row * p.ldo;
  const int lead = ANY ? static_cast<int>(reinterpret_cast<uintptr_t>(out) % N) : 0;
  const int chunks = live ? (p.d + lead + (ANY ? N - 1 : 0)) / N : 0;
  auto whole = [&](int c) { return !ANY || (c * N >= lead && (c + 1) * N <= p.d + lead); };
  auto load = [&](const T *from, int c, typename Vec::Words &v) {  // vector c of a row
    const int e0 = c * N - lead;
    if (!whole(c))
      Vec::load_part(from, e0, p.d, v);
    else if (ANY)
      Vec::load_any(from + e0, v);
    else
      Vec::load(from + e0, v);
  };
  float h[CH][N];
  if (MODE == kRowsGated || p.res) {
    const T *r = MODE == kRowsGated ? x + p.d : static_cast<const T *>(p.res) + row * p.ldr;
    typename Vec::Words a[CH], b[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = lane + i * tpr;
#pragma unroll
      for (int j = 0; j < Vec::kWords; ++j) a[i][j] = b[i][j] = 0;
      if (c < chunks) {
        load(x, c, a[i]);
        load(r, c, b[i]);
      }
    }
    const bool low = MODE == kRowsGated && Vec::any_below(a, kGateLow);  // rare
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      float u[N];
      Vec::unpack(a[i], h[i]);
      Vec::unpack(b[i], u);
      if (MODE != kRowsGated) {
#pragma unroll
        for (int j = 0; j < N; ++j) h[i][j] += u[j];
      } else if (lane + i * tpr < chunks) {  // nothing for the places beyond the row (their h is 0)
#pragma unroll
        for (int j = 0; j < N; ++j) h[i][j] = silu_mul(h[i][j], u[j]);
      }
    }
    if (low) {  // once more, from the row: a look per thread costs less than one per value
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = lane + i * tpr;
        if (c >= chunks) continue;
        typename Vec::Words v;
        float g[N], u[N];
        load(x, c, v);
        Vec::unpack(v, g);
        load(r, c, v);
        Vec::unpack(v, u);
#pragma unroll
        for (int j = 0; j < N; ++j) h[i][j] = silu_mul_any(g[j], u[j]);
      }
    }
    if (MODE != kRowsGated && p.sum) {
      T *s = static_cast<T *>(p.sum) + row * p.lds;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = lane + i * tpr, e0 = c * N - lead;
        if (c >= chunks) continue;
        if (whole(c)) {
          typename Vec::Words v;
          Vec::pack(h[i], v);
          if (ANY)
            Vec::store_any(s + e0, v);
          else
            Vec::store(s + e0, v);
        } else {
#pragma unroll
          for (int j = 0; j < N; ++j)
            if (e0 + j >= 0 && e0 + j < p.d) s[e0 + j] = from_f32<T>(h[i][j]);
        }
      }
    }
  } else {
    typename Vec::Words a[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = lane + i * tpr;
#pragma unroll
      for (int j = 0; j < Vec::kWords; ++j) a[i][j] = 0;
      if (c < chunks) load(x, c, a[i]);
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) Vec::unpack(a[i], h[i]);
  }
  float rs = 1.f;
  if (MODE == kRowsRms) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) ss = fmaf(h[i][j], h[i][j], ss);
    ss = row_sum(ss, tpr, red);
    float pre = 1.f;
    const bool holds = rms_sum_holds(ss);
    if (tpr > 32 ? __syncthreads_or(!holds) : !holds) {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) m = max_abs(m, h[i][j]);
      const uint32_t top = row_max(abs_bits(m), tpr, red);
      if (!holds && rms_needs_scaling(top)) pre = rms_prescale(top);
      float again = 0.f;
#pragma unroll
      for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) {
          h[i][j] *= pre;
          again = fmaf(h[i][j], h[i][j], again);
        }
      ss = row_sum(again, tpr, red);
    }
    rs = rms_factor(ss, p.d, p.eps, pre);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = lane + i * tpr;
      if (c < chunks) {
        typename Vec::Words v;
        float u[N];
        load(w, c, v);
        Vec::unpack(v, u);
#pragma unroll
        for (int j = 0; j < N; ++j) h[i][j] = h[i][j] * rs * u[j];
      }
    }
  }
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) m = max_abs(m, h[i][j]);
  const float2 sc = row_scale(row_max(abs_bits(m), tpr, red));
  if (live && lane == 0) p.scale[row] = sc.x;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = lane + i * tpr, e0 = c * N - lead;
    if (c >= chunks) continue;
    uint32_t q[(N + 3) / 4];
#pragma unroll
    for (int j = 0; j < N; j += 2) {
      const uint32_t two = e4m3x2(h[i][j] * sc.y, h[i][j + 1] * sc.y);
      q[j / 4] = j % 4 ? q[j / 4] | two << 16 : two;
    }
    if (!whole(c)) {
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (e0 + j >= 0 && e0 + j < p.d) out[e0 + j] = static_cast<uint8_t>(q[j / 4] >> 8 * (j % 4));
    } else if constexpr (N == 8) {
      *reinterpret_cast<uint2 *>(out + e0) = make_uint2(q[0], q[1]);
    } else if constexpr (N == 4) {
      *reinterpret_cast<uint32_t *>(out + e0) = q[0];
    } else {
      *reinterpret_cast<uint16_t *>(out + e0) = static_cast<uint16_t>(q[0]);
    }
  }
}

}  // namespace voc
