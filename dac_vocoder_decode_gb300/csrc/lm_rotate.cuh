// lm_rotate.cuh -- queries and keys between the product that makes them and the cache: RMS norm of each
// head and rotation by position in one pass.
//
//   n = x * (1 / sqrt(mean(x^2) + eps)) * weight                of a head's d channels (without weight: x)
//   turn = position[axis[p]] * turns[p], in units of 2^-64 of a turn, modulo a turn
//   (a, b) -> (a cos - b sin, a sin + b cos)                    for the two channels of pair p
//
// Pairs are channels (p, p + pairs) or neighbours (2p, 2p + 1); channels behind the 2 * pairs first ones
// keep n.
#pragma once
#include "lm_common.cuh"
#include "lm_rows.cuh"

namespace voc {

struct LmRotateArgs {
  const void *x[2], *w[2];  // queries and keys
  void *out[2];
  long long ldx[2], hsx[2], ldo[2], hso[2];
  int heads[2], groups[2];  // heads, and turns of a warp that they take
  const int *pos, *axis;
  const unsigned long long *turns;
  long long ldp, tokens;
  int axes, pairs, d;
  int per, parts;  // turns of a warp, warps of a token
  float eps;
};

constexpr int kRotThreads = 128;

// cos and sin of position * turn.  The product modulo 2^64 is exact, so a far position loses nothing; the
// upper half, a signed fraction of a turn good to 2^-33, goes through the hardware's approximations
// (2^-20 absolute, inside half a step of the 16-bit result by 2^8).
__device__ __forceinline__ float2 turn_cos_sin(int pos, unsigned long long turn) {
  const unsigned long long t = static_cast<unsigned long long>(static_cast<long long>(pos)) * turn;
  const float a = static_cast<float>(static_cast<int>(t >> 32)) * (6.28318531f * 0x1p-32f);
  float2 r;
  asm("cos.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(a));
  asm("sin.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(a));
  return r;
}

// A head belongs to L lanes, 16 channels each: two vectors that hold both channels of 8 pairs, so that
// nothing is exchanged but the sum of squares, and a warp takes 32 / L heads of a token at a time.  The
// 8 angles of a lane are the same for all heads of the token and are computed once.
template <typename T, int L, bool NEAR>
__global__ void __launch_bounds__(kRotThreads) rotate_kernel(const LmRotateArgs p) {
  constexpr int kAtOnce = 32 / L;
  const long long task =
      static_cast<long long>(blockIdx.x) * (kRotThreads / 32) + threadIdx.x / 32;
  const int lane = threadIdx.x % 32, unit = lane % L;
  pdl_wait();
  pdl_launch_dependents();
  const long long token = task / p.parts;
  if (token >= p.tokens) return;
  const int first = static_cast<int>(task % p.parts) * p.per;
  const int last = min(first + p.per, p.groups[0] + p.groups[1]);
  const int blocks = p.pairs / 8;  // lanes that turn pairs
  const bool turns = unit < blocks, channels = unit < p.d / 16;
  const int c0 = 8 * (turns && !NEAR ? unit : 2 * unit);
  const int c1 = turns && !NEAR ? c0 + p.pairs : c0 + 8;
  float co[8], si[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) co[i] = 1.f, si[i] = 0.f;
  if (turns) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int pair = 8 * unit + i;
      const int axis = p.axis ? p.axis[pair] : 0;
      if (axis >= 0 && axis < p.axes) {
        const float2 cs = turn_cos_sin(p.pos[axis * p.ldp + token], p.turns[pair]);
        co[i] = cs.x, si[i] = cs.y;
      }
    }
  }
  int of = -1;  // whose weights are at hand
  uint4 w0 = {}, w1 = {};
  for (int g = first; g < last; ++g) {
    const int which = g >= p.groups[0];
    const int head = (g - (which ? p.groups[0] : 0)) * kAtOnce + lane / L;
    const bool live = channels && head < p.heads[which];
    const T *w = static_cast<const T *>(p.w[which]);
    if (which != of && w && channels) {
      w0 = *reinterpret_cast<const uint4 *>(w + c0);
      w1 = *reinterpret_cast<const uint4 *>(w + c1);
    }
    of = which;
    uint4 a = {}, b = {};
    if (live) {
      const T *x = static_cast<const T *>(p.x[which]) + token * p.ldx[which] + head * p.hsx[which];
      a = *reinterpret_cast<const uint4 *>(x + c0);
      b = *reinterpret_cast<const uint4 *>(x + c1);
    }
    float h[16];
    {
      float f[8];
      Vec16<T>::unpack(a, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = f[i];
      Vec16<T>::unpack(b, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[8 + i] = f[i];
    }
    if (w) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) ss = fmaf(h[i], h[i], ss);
#pragma unroll
      for (int o = 1; o < L; o *= 2) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      float pre = 1.f;
      const bool holds = rms_sum_holds(ss) || head >= p.heads[which];
      if (__any_sync(0xffffffffu, !holds)) {  // rare: squares that overflowed or vanished
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) m = max_abs(m, h[i]);
        uint32_t top = abs_bits(m);
#pragma unroll
        for (int o = 1; o < L; o *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (!holds && rms_needs_scaling(top)) pre = rms_prescale(top);
        float again = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          h[i] *= pre;
          again = fmaf(h[i], h[i], again);
        }
#pragma unroll
        for (int o = 1; o < L; o *= 2) again += __shfl_xor_sync(0xffffffffu, again, o);
        ss = again;
      }
      const float rs = rms_factor(ss, p.d, p.eps, pre);
      float f[8];
      Vec16<T>::unpack(w0, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = h[i] * rs * f[i];
      Vec16<T>::unpack(w1, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[8 + i] = h[8 + i] * rs * f[i];
    }
    if (turns) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int ia = NEAR ? 2 * i : i, ib = NEAR ? 2 * i + 1 : 8 + i;
        const float u = h[ia], v = h[ib];
        h[ia] = u * co[i] - v * si[i];
        h[ib] = u * si[i] + v * co[i];
      }
    }
    if (live) {
      float f[8];
      T *o = static_cast<T *>(p.out[which]) + token * p.ldo[which] + head * p.hso[which];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = h[i];
      *reinterpret_cast<uint4 *>(o + c0) = Vec16<T>::pack(f);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = h[8 + i];
      *reinterpret_cast<uint4 *>(o + c1) = Vec16<T>::pack(f);
    }
  }
}

}  // namespace voc
