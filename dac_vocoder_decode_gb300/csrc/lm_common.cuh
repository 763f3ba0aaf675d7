// lm_common.cuh -- pieces shared by the 8-bit operators of a token model (lm_*.cuh): element
// types and e4m3 conversions.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"

namespace voc {

constexpr float kE4m3Max = 448.f;       // largest finite e4m3
constexpr int kScaleMinExp = -96;       // scales never fall below 2^-96 (rows: 2^-96 / 448)
constexpr float kScaleMin = 0x1p-96f;
constexpr int kBlockTokens = 64;        // tokens of one cache block (VOC_LM_BLOCK)
constexpr uint32_t kInfBits = 0x7f800000u;

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// 16 bytes of a 16-bit type <-> floats.
template <typename T>
struct Vec16;
template <>
struct Vec16<__half> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4 &u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __half2 h;
      memcpy(&h, &w[i], 4);
      const float2 v = __half22float2(h);
      f[2 * i] = v.x, f[2 * i + 1] = v.y;
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      memcpy(&w[i], &h, 4);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec16<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4 &u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      memcpy(&w[i], &h, 4);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// A 32-bit word of two 16-bit values <-> floats.
template <typename T>
__device__ __forceinline__ void unpack2(uint32_t w, float &a, float &b);
template <>
__device__ __forceinline__ void unpack2<__half>(uint32_t w, float &a, float &b) {
  __half2 h;
  memcpy(&h, &w, 4);
  const float2 v = __half22float2(h);
  a = v.x, b = v.y;
}
template <>
__device__ __forceinline__ void unpack2<__nv_bfloat16>(uint32_t w, float &a, float &b) {
  a = __uint_as_float(w << 16), b = __uint_as_float(w & 0xffff0000u);
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  uint32_t w;
  memcpy(&w, &h, 4);
  return w;
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  uint32_t w;
  memcpy(&w, &h, 4);
  return w;
}

// The smaller ones of two pairs of 16-bit values (a number before NaN).
template <typename T>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b);
template <>
__device__ __forceinline__ uint32_t min2<__half>(uint32_t a, uint32_t b) {
  __half2 x, y;
  memcpy(&x, &a, 4), memcpy(&y, &b, 4);
  x = __hmin2(x, y);
  memcpy(&a, &x, 4);
  return a;
}
template <>
__device__ __forceinline__ uint32_t min2<__nv_bfloat16>(uint32_t a, uint32_t b) {
  __nv_bfloat162 x, y;
  memcpy(&x, &a, 4), memcpy(&y, &b, 4);
  x = __hmin2(x, y);
  memcpy(&a, &x, 4);
  return a;
}

// Two floats to two e4m3 codes, `lo` in the low byte: round to nearest even, magnitudes over 448
// (infinities too) to 448, NaN to 0x7f.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}
__device__ __forceinline__ uint8_t e4m3(float v) { return static_cast<uint8_t>(e4m3x2(v, 0.f)); }
// Two e4m3 codes to two halves (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_to_f32(uint16_t v) {
  const uint32_t u = e4m3x2_to_f16x2(v);
  __half2 h;
  memcpy(&h, &u, 4);
  return __half22float2(h);
}

// |v| as an integer: its maximum orders magnitudes like the float's and keeps a NaN, which a
// floating maximum would drop.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// max(m, |v|) that keeps a NaN.
__device__ __forceinline__ float max_abs(float m, float v) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(v)));
  return r;
}

// 2^e for e in [-126, 127].
__device__ __forceinline__ float pow2(int e) {
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

}  // namespace voc
