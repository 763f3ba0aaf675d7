// lm_logprobs.cuh -- rows of logits: log probabilities of given tokens, entropy, top alternatives.
//
//   z = x / temperature,  lse = log sum_i e^z_i
//   logprob = z_token - lse,  entropy = lse - sum_i e^(z_i - lse) z_i
//   top: the k largest x, the lowest index first among equal ones, and their log probabilities
//
// One pass over the row with a running maximum m and the sums s = sum e^((x - m) c), t = sum (x - m) c
// e^((x - m) c), c = log2(e) / temperature and powers of two: logprob = (x - m) / temperature - ln2 log2 s,
// entropy = ln2 (log2 s - t / s).  In the sums x - m is taken before the factor and may leave 32 bits: the weight is
// 0 all the same, and the type's lowest value as a mask in every place gives equal weights, as the formula
// does.  In the results it is taken by halves and without log2(e), so that one that 32 bits hold does not
// overflow on the way (a token of the type's lowest value beside ordinary ones).
#pragma once
#include "lm_common.cuh"

namespace voc {

struct LmLogprobsArgs {
  const void *x;
  const long long *tokens;
  float *logprob, *entropy, *top;
  long long *top_tokens;
  long long rows, ldx;
  int vocab, k;
  float c, twice;  // log2(e) / temperature, 2 / temperature
};

constexpr int kLpMaxTop = 32;

// A value and its index as one number: larger values first, then lower indices; never 0.
__device__ __forceinline__ uint32_t order_bits(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);  // -0 counts as 0
  return v != v ? 0xffffffffu : b ^ (static_cast<uint32_t>(static_cast<int>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ unsigned long long order_key(float v, int index) {
  return static_cast<unsigned long long>(order_bits(v)) << 32 | ~static_cast<uint32_t>(index);
}
__device__ __forceinline__ float key_value(unsigned long long key) {
  const uint32_t b = static_cast<uint32_t>(key >> 32);
  return __uint_as_float(b >> 31 ? b ^ 0x80000000u : ~b);
}
__device__ __forceinline__ int key_index(unsigned long long key) {
  return static_cast<int>(~static_cast<uint32_t>(key));
}

// Maximum and sums of a part of a row, relative to its maximum.
struct LpPart {
  float m, s, t;
};
// The parts of a warp's lanes, in a fixed order, to all of them.  A part without weight (nothing but
// -infinity) stays out, and one too far below for its weight to count adds 0, not 0 times a difference that
// left 32 bits; NaN stays.
__device__ __forceinline__ LpPart lp_join_warp(const LpPart &a, float c) {
  LpPart r;
  r.m = a.m;
#pragma unroll
  for (int o = 16; o; o >>= 1) r.m = fmaxf(r.m, __shfl_xor_sync(0xffffffffu, r.m, o));
  const float d = a.m == -INFINITY ? 0.f : (a.m - r.m) * c, f = ex2(d);
  r.s = a.s * f;
  r.t = f > 0.f ? f * fmaf(a.s, d, a.t) : a.s * 0.f;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    r.s += __shfl_xor_sync(0xffffffffu, r.s, o);
    r.t += __shfl_xor_sync(0xffffffffu, r.t, o);
  }
  return r;
}

// The larger ones of two pairs of 16-bit values (a number before NaN).
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b, __half) {
  __half2 x, y;
  memcpy(&x, &a, 4), memcpy(&y, &b, 4);
  x = __hmax2(x, y);
  memcpy(&a, &x, 4);
  return a;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b, __nv_bfloat16) {
  __nv_bfloat162 x, y;
  memcpy(&x, &a, 4), memcpy(&y, &b, 4);
  x = __hmax2(x, y);
  memcpy(&a, &x, 4);
  return a;
}

// A row in 16-byte vectors that lie on the 16-byte grid, whatever the row starts on: those at its ends
// that it covers only in part are read value by value, with -infinity in the places outside of it.
template <int N>
struct LpCount {
  static constexpr int value = N;
};

template <typename T>
struct LpRow {
  static constexpr int N = 16 / static_cast<int>(sizeof(T));
  static constexpr int kBatch = 32 / N;  // vectors of 32 values
  const T *row;
  int lead, vocab, lo, hi;  // vectors [lo, hi) are whole

  __device__ __forceinline__ LpRow(const T *r, int v) : row(r), vocab(v) {
    lead = static_cast<int>(reinterpret_cast<uintptr_t>(r) % 16) / static_cast<int>(sizeof(T));
    lo = lead > 0;
    hi = (lead + vocab) / N;
  }
  __device__ __forceinline__ int vectors() const { return (lead + vocab + N - 1) / N; }
  __device__ __forceinline__ int index(int v, int j) const { return v * N + j - lead; }
  static __device__ __forceinline__ uint4 nothing() {
    const uint32_t w = sizeof(T) == 4 ? 0xff800000u : pack_inf(T());
    return make_uint4(w, w, w, w);
  }
  static __device__ __forceinline__ uint32_t pack_inf(float) { return 0xff800000u; }
  static __device__ __forceinline__ uint32_t pack_inf(__half) { return 0xfc00fc00u; }
  static __device__ __forceinline__ uint32_t pack_inf(__nv_bfloat16) { return 0xff80ff80u; }
  __device__ __forceinline__ uint4 load(int v) const {
    if (v >= lo && v < hi) return *reinterpret_cast<const uint4 *>(row + index(v, 0));
    const uint4 none = nothing();
    uint32_t w[4] = {none.x, none.y, none.z, none.w};
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int i = index(v, j);
      if (i < 0 || i >= vocab) continue;
      if constexpr (sizeof(T) == 4) {
        w[j] = reinterpret_cast<const uint32_t *>(row)[i];
      } else {
        const uint32_t h = reinterpret_cast<const uint16_t *>(row)[i];
        w[j / 2] = j % 2 ? (w[j / 2] & 0xffffu) | h << 16 : (w[j / 2] & 0xffff0000u) | h;
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // Vectors v, v + step, ..., all of them whole.
  __device__ __forceinline__ void load_batch(int v, int step, uint4 (&u)[kBatch]) const {
    const uint4 *at = reinterpret_cast<const uint4 *>(row + index(v, 0));
#pragma unroll
    for (int b = 0; b < kBatch; ++b) u[b] = at[b * step];
  }
  // Values 2i and 2i + 1 of a vector.
  static __device__ __forceinline__ float2 pair(const uint4 &u, int i) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    float2 f;
    if constexpr (sizeof(T) == 4)
      f = make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    else
      unpack2<T>(w[i], f.x, f.y);
    return f;
  }
  static __device__ __forceinline__ float value(const uint4 &u, int j) {
    const float2 f = pair(u, j / 2);
    return j % 2 ? f.y : f.x;
  }
  // Largest of V vectors (of NaN only: NaN or -infinity).
  template <int V>
  static __device__ __forceinline__ float largest(const uint4 *u) {
    if constexpr (sizeof(T) == 4) {
      float m[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int b = 0; b < V; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) m[i % 2] = fmaxf(m[i % 2], value(u[b], i));
      return fmaxf(m[0], m[1]);
    } else {
      uint32_t m[2] = {max2(u[0].x, u[0].z, T()), max2(u[0].y, u[0].w, T())};
#pragma unroll
      for (int b = 1; b < V; ++b) {
        m[0] = max2(max2(m[0], u[b].x, T()), u[b].z, T());
        m[1] = max2(max2(m[1], u[b].y, T()), u[b].w, T());
      }
      float a, b;
      unpack2<T>(max2(m[0], m[1], T()), a, b);
      return fmaxf(a, b);
    }
  }
};

// max(v, lo) that keeps a NaN.
__device__ __forceinline__ float max_nan(float v, float lo) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "f"(lo));
  return r;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t cluster_addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr) : "memory");
  return v;
}
__device__ __forceinline__ unsigned long long ld_cluster_u64(uint32_t cluster_addr) {
  unsigned long long v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(cluster_addr) : "memory");
  return v;
}

constexpr int kLpWide = 256;  // threads of a row that has a CTA, or several, for itself
constexpr int kLpWarps = 4;   // warps of a CTA whose warps have a row each

template <int TPR>
struct LpShared {
  static constexpr int kSubs = TPR == 32 ? 32 : 128;  // parts of a row, for its alternatives
  static constexpr int kRoom = TPR == 32 ? 256 : 1024;
  unsigned long long sub[kSubs], cand[kRoom], top[kLpMaxTop], bound;
  int reach[kSubs];  // subsets that reach the bound
  int reached, count;
};

// The n numbers of `cand` (n <= room; all different but for zeros, which do not count): the k largest, in
// order, to `top`.
template <int TPR>
__device__ __forceinline__ void lp_rank(const unsigned long long *cand, int n, int k,
                                        unsigned long long *top, int tid) {
  for (int i = tid; i < n; i += TPR) {
    const unsigned long long mine = cand[i];
    int above = 0;
    for (int j = 0; j < n; ++j) above += cand[j] > mine;
    if (mine && above < k) top[above] = mine;
  }
}

// One warp: a lower bound of the k-th largest number of a row from the largest of each subset (0: nothing in
// it), and the subsets that reach it.  The lanes' heads are compared k times, by their 32 - log2(kSubs) first
// bits; the smallest of the k winners' whole numbers is the bound.  (What those bits do not tell apart may
// pass a larger one over; that makes the bound lower, and the subsets that reach it are looked up anew.)
template <int TPR>
__device__ __forceinline__ void lp_bound(LpShared<TPR> &sh, int k, int lane) {
  constexpr int kSubs = LpShared<TPR>::kSubs, kOwn = kSubs / 32;
  uint32_t own[kOwn];
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    const uint32_t v = static_cast<uint32_t>(sh.sub[lane + 32 * i] >> 32);
    own[i] = v ? (v & ~(kSubs - 1u)) | (lane + 32 * i) : 0;
  }
  auto order = [&](int i, int j) {
    const uint32_t hi = max(own[i], own[j]), lo = min(own[i], own[j]);
    own[i] = hi, own[j] = lo;
  };
  if constexpr (kOwn == 4) {
    order(0, 1), order(2, 3), order(0, 2), order(1, 3), order(1, 2);
  }
  uint32_t mine = 0;  // the k-th turn's winner in lane k
  for (int i = 0; i < k; ++i) {
    const uint32_t top = __reduce_max_sync(0xffffffffu, own[0]);
    if (lane == i) mine = top;
    if (own[0] == top) {
#pragma unroll
      for (int n = 0; n + 1 < kOwn; ++n) own[n] = own[n + 1];
      own[kOwn - 1] = 0;
    }
  }
  unsigned long long key = ~0ull;
  if (lane < k) key = mine ? sh.sub[mine & (kSubs - 1)] : 0;  // fewer subsets than k hold anything: all of them
  const uint32_t hi = __reduce_min_sync(0xffffffffu, static_cast<uint32_t>(key >> 32));
  const uint32_t lo = __reduce_min_sync(
      0xffffffffu, static_cast<uint32_t>(key >> 32) == hi ? static_cast<uint32_t>(key) : 0xffffffffu);
  const unsigned long long bound = static_cast<unsigned long long>(hi) << 32 | lo;
  int reached = 0;
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    const unsigned long long s = sh.sub[lane + 32 * i];
    const bool in = s && s >= bound;
    const uint32_t all = __ballot_sync(0xffffffffu, in);
    if (in) sh.reach[reached + __popc(all & ((1u << lane) - 1u))] = lane + 32 * i;
    reached += __popc(all);
  }
  if (lane == 0) sh.bound = bound, sh.reached = reached, sh.count = 0;
}

// TPR threads take a row, or with a cluster of several CTAs (along z) a part of it each.
//
// Top: the row falls into subsets (of a lane or a pair of lanes).  The k-th largest of their maxima is a
// lower bound of the k-th largest value, and few subsets reach it: these are read again (from cache), what
// reaches the bound is gathered, some k to 2k numbers for logits in no order, and ranked by counting.  Where
// more of them come together than there is room for, the k-th largest of those at hand is a higher bound,
// and they are gathered again.
// Bound by instructions beside DRAM: 4001 rows of 50001 f16 values, 5 alternatives: 82 us, 4.9 TB/s (six
// instructions a value in the stream, as many again for a row's way in and out; 5 CTAs on an SM, with 4 87 us,
// with 6 or 3 101; rows of 128 threads 83); 15504 x 2048 bf16, none: 15.1 us, 4.2 TB/s (a warp a row, 36 on an
// SM; with 48 19.9, with 32 15.9).  Few rows by latency: 128 x 2048, 20 alternatives 4.7 us, 8 x 131072 f32, 20
// alternatives 9.8 (8 CTAs a row; rows of 128 threads 12.2).
template <typename T, int TPR, bool TOP>
__global__ void __launch_bounds__(TPR == 32 ? 32 * kLpWarps : kLpWide,
                                  TPR == 32 ? (sizeof(T) == 2 ? 9 : 5) : (sizeof(T) == 2 ? 5 : 3))
    logprobs_kernel(const LmLogprobsArgs p) {
  using Row = LpRow<T>;
  constexpr int B = Row::kBatch, N = Row::N;
  constexpr int kWarps = TPR / 32;
  using Shared = LpShared<TPR>;
  __shared__ Shared shared[TOP ? (TPR == 32 ? kLpWarps : 1) : 1];
  __shared__ LpPart parts[kWarps + 1];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int tid = TPR == 32 ? lane : threadIdx.x;
  Shared &sh = shared[TOP && TPR == 32 ? warp : 0];
  const long long at = TPR == 32 ? static_cast<long long>(blockIdx.x) * kLpWarps + warp : blockIdx.x;
  const int split = gridDim.z, rank = blockIdx.z;
  auto sync = [] {
    if (TPR == 32)
      __syncwarp();
    else
      __syncthreads();
  };
  pdl_wait();
  pdl_launch_dependents();
  if (at >= p.rows) return;  // TPR = 32 only
  const Row row(static_cast<const T *>(p.x) + at * p.ldx, p.vocab);
  const int all = row.vectors();
  const int v0 = static_cast<int>(static_cast<long long>(all) * rank / split);
  const int v1 = static_cast<int>(static_cast<long long>(all) * (rank + 1) / split);
  const float c = p.c;

  LpPart mine{-INFINITY, 0.f, 0.f};
  int best = v0 + tid;  // first vector of the batch that holds this thread's maximum first
  {
    float2 s = {0.f, 0.f}, t = {0.f, 0.f};
    // Adds V vectors, the first of them number v.
    auto add = [&](const uint4 *u, auto count, int v) {
      constexpr int kVectors = decltype(count)::value;
      const float m = Row::template largest<kVectors>(u);
      if (m > mine.m) {
        const float d = (mine.m - m) * c, f = mine.m == -INFINITY ? 0.f : ex2(d);
        if (f > 0.f)
          t.x = f * fmaf(s.x, d, t.x), t.y = f * fmaf(s.y, d, t.y);
        else
          t.x = s.x * 0.f, t.y = s.y * 0.f;  // 0, or NaN
        s.x *= f, s.y *= f;
        mine.m = m;
        best = v;
      }
      const float neg = mine.m == -INFINITY ? 0.f : -mine.m;
      const float2 from = {neg, neg}, by = {c, c};
#pragma unroll
      for (int b = 0; b < kVectors; ++b)
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          float2 d = mul2(add2(Row::pair(u[b], i), from), by);
          d.x = max_nan(d.x, -200.f), d.y = max_nan(d.y, -200.f);  // -infinity weighs 0, and 0 times it is 0
          const float2 e = {ex2(d.x), ex2(d.y)};
          s = add2(s, e);
          t = fma2(e, d, t);
        }
    };
    int v = v0 + tid;
    const int whole = min(v1, row.hi) - (B - 1) * TPR;  // batches that start below it are whole
    if (v < row.lo) {  // the row's first vector, covered in part
      const uint4 u = row.load(v);
      add(&u, LpCount<1>(), v);
      v += TPR;
    }
    if (v < whole) {
      uint4 u[B];
      row.load_batch(v, TPR, u);
      for (; v < whole; v += B * TPR) {
        uint4 now[B];
#pragma unroll
        for (int b = 0; b < B; ++b) now[b] = u[b];
        if (v + B * TPR < whole) row.load_batch(v + B * TPR, TPR, u);
        add(now, LpCount<B>(), v);
      }
    }
    for (; v < v1; v += TPR) {
      const uint4 u = row.load(v);
      add(&u, LpCount<1>(), v);
    }
    mine.s = s.x + s.y, mine.t = t.x + t.y;
  }
  const float top_value = mine.m;
  mine = lp_join_warp(mine, c);
  if (TPR > 32 && lane == 0) parts[warp] = mine;

  if constexpr (TOP) {
    constexpr int kEach = TPR / Shared::kSubs;  // lanes of a subset
    unsigned long long key = 0;
    if (v0 + tid < v1) {
      // the vector that holds the maximum first; its last index stands for the value's, which is no larger
      int at_vector = best;
#pragma unroll
      for (int b = B - 1; b >= 0; --b) {
        const int v = best + b * TPR;
        if (v < v1) {
          const uint4 u = row.load(v);
          if (Row::template largest<1>(&u) == top_value) at_vector = v;
        }
      }
      key = order_key(top_value, row.index(at_vector, N - 1));
    }
    if (kEach == 2) {
      const unsigned long long other = __shfl_xor_sync(0xffffffffu, key, 1);
      key = other > key ? other : key;
    }
    if (tid % kEach == 0) sh.sub[tid / kEach] = key;
    if (tid < kLpMaxTop) sh.top[tid] = 0;
    sync();
    if (tid < 32) lp_bound<TPR>(sh, p.k, lane);
    sync();
    unsigned long long bound = sh.bound;
    const int each = (v1 - v0 + TPR - 1) / TPR * kEach;  // vectors of a subset, at most
    const int items = sh.reached * each;
    while (true) {
      const float least = bound ? key_value(bound) : -INFINITY;
      for (int i = tid; i < items; i += TPR) {
        const int w = i / each, r = i % each;
        const int v = v0 + sh.reach[w] * kEach + r % kEach + r / kEach * TPR;
        if (v >= v1) continue;
        const uint4 u = row.load(v);
        if (Row::template largest<1>(&u) < least) continue;
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const float x = Row::value(u, j);
          const int at_index = row.index(v, j);
          if (x < least || at_index < 0 || at_index >= p.vocab) continue;
          const unsigned long long one = order_key(x, at_index);
          if (one < bound) continue;
          const int to = atomicAdd(&sh.count, 1);  // in any order: they are ranked
          if (to < Shared::kRoom) sh.cand[to] = one;
        }
      }
      sync();
      const int n = sh.count;
      lp_rank<TPR>(sh.cand, min(n, Shared::kRoom), p.k, sh.top, tid);
      sync();
      if (n <= Shared::kRoom) break;
      bound = sh.top[p.k - 1];
      if (tid == 0) sh.count = 0;
      sync();
    }
  } else if (TPR > 32) {
    __syncthreads();
  }
  if (TPR > 32 && warp == 0)  // the first warp's from here on
    mine = lp_join_warp(lane < kWarps ? parts[lane] : LpPart{-INFINITY, 0.f, 0.f}, c);
  if (TPR > 32 && split > 1) {
    if (tid == 0) parts[kWarps] = mine;
    cluster_sync();
    if (rank == 0) {
      if (warp == 0) {
        LpPart other{-INFINITY, 0.f, 0.f};
        if (lane < split) {
          const uint32_t from = mapa_shared(smem_u32(&parts[kWarps]), lane);
          other = {ld_cluster_f32(from), ld_cluster_f32(from + 4), ld_cluster_f32(from + 8)};
        }
        mine = lp_join_warp(other, c);
      }
      if constexpr (TOP) {
        const int n = split * p.k;  // no more than there is room for
        for (int i = tid; i < n; i += TPR)
          sh.cand[i] = ld_cluster_u64(mapa_shared(smem_u32(&sh.top[i % p.k]), i / p.k));
        __syncthreads();
        lp_rank<TPR>(sh.cand, n, p.k, sh.top, tid);
        __syncthreads();
      }
    }
  }
  if (rank == 0 && (TPR == 32 || warp == 0)) {
    constexpr float kLn2 = 0.693147181f;
    const float log2s = log2f(mine.s);
    const bool none = mine.s == 0.f;  // nothing but -infinity: no token has any weight
    auto logprob = [&](float x) {
      return none ? -INFINITY : fmaf(0.5f * x - 0.5f * mine.m, p.twice, -kLn2 * log2s);
    };
    if (tid == 0) {
      if (p.entropy) p.entropy[at] = none ? 0.f : (log2s - mine.t / mine.s) * kLn2;
      if (p.tokens) {
        const long long i = p.tokens[at];
        const float x = i >= 0 && i < p.vocab ? to_f32(row.row[i]) : -INFINITY;
        p.logprob[at] = logprob(x);
      }
    }
    if constexpr (TOP) {
      if (lane < p.k) {
        const unsigned long long key = sh.top[lane];
        p.top[at * p.k + lane] = logprob(key_value(key));
        p.top_tokens[at * p.k + lane] = key_index(key);
      }
    }
  }
  if (TPR > 32 && split > 1) cluster_sync();  // nobody leaves while its part is being read
}

}  // namespace voc
