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
  int per;  // turns of a warp
  float eps;
};

constexpr int kRotThreads = 128;

// cos and sin of position * turn.  The product modulo 2^64 is exact, so a far position loses nothing; the
// upper half, a signed fraction of a turn good to 2^-33, goes through the hardware's approximations
// (2^-20.5 absolute over [-pi, pi], beside 2^-21 of the 32-bit angle).  With the norm's sums a result is off by
// 2^-18 of |a| + |b| at most before it is rounded: 2^-7 of half a step of f16 and 2^-9 of bf16's where it is of
// their size, and more than half a step where a cos and b sin cancel or the larger one's sine is near 0 (a slow
// pair near its start: a = 1, b = 0, angle 1e-4, 20 times half a step of f16).
__device__ __forceinline__ void turn_cos_sin(int pos, unsigned long long turn, float &co, float &si) {
  const uint32_t lo = static_cast<uint32_t>(turn), hi = static_cast<uint32_t>(turn >> 32);
  const uint32_t upper = __umulhi(static_cast<uint32_t>(pos), lo) + static_cast<uint32_t>(pos) * hi -
                         (pos < 0 ? lo : 0u);
  const float a = static_cast<float>(static_cast<int>(upper)) * (6.28318531f * 0x1p-32f);
  asm("cos.approx.ftz.f32 %0, %1;" : "=f"(co) : "f"(a));
  asm("sin.approx.ftz.f32 %0, %1;" : "=f"(si) : "f"(a));
}

// A head belongs to L lanes, 16 channels each: two vectors that hold both channels of 8 pairs, so that
// nothing is exchanged but the sum of squares, and a warp takes 32 / L heads of a token at a time.  The
// 8 angles of a lane are the same for all heads of the token and are computed once.
// Bound by DRAM and by its instructions: 15504 tokens x 20 heads of 128 bf16 channels (159 MB) 29.3 us, 5.4
// TB/s; 4001 x 32 f16, three axes (66 MB) 13.9 us, 4.7 TB/s (11.4 us with the input in L2); 8 x 20 heads of 64
// 1.9 us.  Next to 72 registers a thread (7 CTAs an SM) and the next head's loads ahead, 15504 tokens took with 80
// registers and the weights unpacked 31.7 us, 64 registers 30.2, without loads ahead 32.8.
template <typename T, int L, bool NEAR>
__global__ void __launch_bounds__(kRotThreads, 7) rotate_kernel(const LmRotateArgs p) {
  constexpr int kAtOnce = 32 / L;
  const long long token =
      static_cast<long long>(blockIdx.x) * (kRotThreads / 32) + threadIdx.x / 32;
  const int lane = threadIdx.x % 32, unit = lane % L;
  pdl_wait();
  pdl_launch_dependents();
  if (token >= p.tokens) return;
  const int first = static_cast<int>(blockIdx.y) * p.per;
  const int last = min(first + p.per, p.groups[0] + p.groups[1]);
  auto unpack8 = [](const uint4 &u, float2 *f) {
    unpack2<T>(u.x, f[0].x, f[0].y), unpack2<T>(u.y, f[1].x, f[1].y);
    unpack2<T>(u.z, f[2].x, f[2].y), unpack2<T>(u.w, f[3].x, f[3].y);
  };
  auto pack8 = [](const float2 *f) {
    return make_uint4(pack2<T>(f[0].x, f[0].y), pack2<T>(f[1].x, f[1].y), pack2<T>(f[2].x, f[2].y),
                      pack2<T>(f[3].x, f[3].y));
  };
  const bool turns = unit < p.pairs / 8, channels = unit < p.d / 16;
  const int c0 = 8 * (turns && !NEAR ? unit : 2 * unit);
  const int behind = turns && !NEAR ? p.pairs : 8;  // from the first vector to the second
  float2 co[4], si[4];
  const float inv_d = 1.f / static_cast<float>(p.d);
  bool turned = false;  // whether the angles are at hand
  for (int which = 0; which < 2; ++which) {
    const int base = which ? p.groups[0] : 0;
    const int lo = max(first, base) - base, hi = min(last, base + p.groups[which]) - base;
    if (lo >= hi) continue;
    const int heads = p.heads[which];
    int head = lo * kAtOnce + lane / L;
    const long long step = kAtOnce * p.hsx[which], out_step = kAtOnce * p.hso[which];
    const T *x = static_cast<const T *>(p.x[which]) + token * p.ldx[which] + head * p.hsx[which] + c0;
    T *out = static_cast<T *>(p.out[which]) + token * p.ldo[which] + head * p.hso[which] + c0;
    uint4 a = {}, b = {};
    if (channels && head < heads) {
      a = *reinterpret_cast<const uint4 *>(x);
      b = *reinterpret_cast<const uint4 *>(x + behind);
    }
    const T *w = static_cast<const T *>(p.w[which]);
    uint4 w0 = {}, w1 = {};
    if (w && channels) {
      w0 = *reinterpret_cast<const uint4 *>(w + c0);
      w1 = *reinterpret_cast<const uint4 *>(w + c0 + behind);
    }
    if (turns && !turned) {
      const ulonglong2 *at = reinterpret_cast<const ulonglong2 *>(p.turns + 8 * unit);
      const int pos = p.pos[token];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const ulonglong2 two = at[i];
        int pa = pos, pb = pos;
        if (p.axis) {  // on no axis: position 0
          const int2 axis = reinterpret_cast<const int2 *>(p.axis + 8 * unit)[i];
          pa = axis.x >= 0 && axis.x < p.axes ? p.pos[axis.x * p.ldp + token] : 0;
          pb = axis.y >= 0 && axis.y < p.axes ? p.pos[axis.y * p.ldp + token] : 0;
        }
        turn_cos_sin(pa, two.x, co[i].x, si[i].x);
        turn_cos_sin(pb, two.y, co[i].y, si[i].y);
      }
    }
    turned = true;
    for (int turn = lo; turn < hi; ++turn) {
      const bool some = head < heads, live = channels && some;
      float2 h[8];
      unpack8(a, h), unpack8(b, h + 4);
      head += kAtOnce;
      x += step;
      if (channels && head < heads && turn + 1 < hi) {
        // in flight meanwhile; an output in the input's place is another head's
        a = *reinterpret_cast<const uint4 *>(x);
        b = *reinterpret_cast<const uint4 *>(x + behind);
      }
      if (w) {
        float2 sq = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 8; ++i) sq = fma2(h[i], h[i], sq);
        float ss = sq.x + sq.y;
#pragma unroll
        for (int o = 1; o < L; o *= 2) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const bool holds = rms_sum_holds(ss) || !some;
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
        *reinterpret_cast<uint4 *>(out) = pack8(h);
        *reinterpret_cast<uint4 *>(out + behind) = pack8(h + 4);
      }
      out += out_step;
    }
  }
}

}  // namespace voc
