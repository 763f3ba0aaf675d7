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
  auto unpack8 = [](const uint4 &u, float2 *f) {
    unpack2<T>(u.x, f[0].x, f[0].y), unpack2<T>(u.y, f[1].x, f[1].y);
    unpack2<T>(u.z, f[2].x, f[2].y), unpack2<T>(u.w, f[3].x, f[3].y);
  };
  auto pack8 = [](const float2 *f) {
    return make_uint4(pack2<T>(f[0].x, f[0].y), pack2<T>(f[1].x, f[1].y), pack2<T>(f[2].x, f[2].y),
                      pack2<T>(f[3].x, f[3].y));
  };
  const bool turns = unit < blocks, channels = unit < p.d / 16;
  const int c0 = 8 * (turns && !NEAR ? unit : 2 * unit);
  const int c1 = turns && !NEAR ? c0 + p.pairs : c0 + 8;
  float2 co[4], si[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) co[i] = {1.f, 1.f}, si[i] = {0.f, 0.f};
  if (turns) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int pair = 8 * unit + i;
      const int axis = p.axis ? p.axis[pair] : 0;
      if (axis >= 0 && axis < p.axes) {
        const float2 cs = turn_cos_sin(p.pos[axis * p.ldp + token], p.turns[pair]);
        if (i % 2)
          co[i / 2].y = cs.x, si[i / 2].y = cs.y;
        else
          co[i / 2].x = cs.x, si[i / 2].x = cs.y;
      }
    }
  }
  const float inv_d = 1.f / static_cast<float>(p.d);
  // A turn of the warp: its head, whether this lane has channels of it, and where they are.
  auto head_of = [&](int g, int which) {
    return (g - (which ? p.groups[0] : 0)) * kAtOnce + lane / L;
  };
  auto load = [&](int g, uint4 &a, uint4 &b) {
    const int which = g >= p.groups[0], head = head_of(g, which);
    a = b = make_uint4(0, 0, 0, 0);
    if (channels && g < last && head < p.heads[which]) {
      const T *x = static_cast<const T *>(p.x[which]) + token * p.ldx[which] + head * p.hsx[which];
      a = *reinterpret_cast<const uint4 *>(x + c0);
      b = *reinterpret_cast<const uint4 *>(x + c1);
    }
  };
  int of = -1;  // whose weights are at hand
  uint4 w0 = {}, w1 = {}, a, b;
  load(first, a, b);
  for (int g = first; g < last; ++g) {
    const int which = g >= p.groups[0];
    const int head = head_of(g, which);
    const bool live = channels && head < p.heads[which];
    const T *w = static_cast<const T *>(p.w[which]);
    if (which != of && w && channels) {
      w0 = *reinterpret_cast<const uint4 *>(w + c0);
      w1 = *reinterpret_cast<const uint4 *>(w + c1);
    }
    of = which;
    float2 h[8];
    unpack8(a, h), unpack8(b, h + 4);
    load(g + 1, a, b);  // in flight meanwhile; an output in the input's place is another head's
    if (w) {
      float2 sq = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 8; ++i) sq = fma2(h[i], h[i], sq);
      float ss = sq.x + sq.y;
#pragma unroll
      for (int o = 1; o < L; o *= 2) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const bool holds = rms_sum_holds(ss) || head >= p.heads[which];
      float rs = rsqrtf(fmaf(ss, inv_d, p.eps));
      if (__any_sync(0xffffffffu, !holds)) {  // rare: squares that overflowed or vanished
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max_abs(max_abs(m, h[i].x), h[i].y);
        uint32_t top = abs_bits(m);
#pragma unroll
        for (int o = 1; o < L; o *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float pre = !holds && rms_needs_scaling(top) ? rms_prescale(top) : 1.f;
        float again = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          h[i].x *= pre, h[i].y *= pre;
          again = fmaf(h[i].x, h[i].x, fmaf(h[i].y, h[i].y, again));
        }
#pragma unroll
        for (int o = 1; o < L; o *= 2) again += __shfl_xor_sync(0xffffffffu, again, o);
        if (!holds) rs = rms_factor(again, p.d, p.eps, pre);
      }
      float2 f[8];
      unpack8(w0, f), unpack8(w1, f + 4);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = mul2(mul2(h[i], {rs, rs}), f[i]);
    }
    if (turns) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (NEAR) {
          const float2 u = h[2 * i], v = h[2 * i + 1];
          h[2 * i] = {u.x * co[i].x - u.y * si[i].x, u.x * si[i].x + u.y * co[i].x};
          h[2 * i + 1] = {v.x * co[i].y - v.y * si[i].y, v.x * si[i].y + v.y * co[i].y};
        } else {
          const float2 u = h[i], v = h[4 + i], less = {-v.x, -v.y};
          h[i] = fma2(less, si[i], mul2(u, co[i]));
          h[4 + i] = fma2(u, si[i], mul2(v, co[i]));
        }
      }
    }
    if (live) {
      T *o = static_cast<T *>(p.out[which]) + token * p.ldo[which] + head * p.hso[which];
      *reinterpret_cast<uint4 *>(o + c0) = pack8(h);
      *reinterpret_cast<uint4 *>(o + c1) = pack8(h + 4);
    }
  }
}

}  // namespace voc
