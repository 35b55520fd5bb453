// Rows of router logits in registers and the blocks' sums, shared by the routing kernels
// (k_route.hip, k_scored.hip).
#pragma once

#include "launch.h"
#include "ops_device.h"

namespace profk {

constexpr u32 kRouteMaxBlocks = 512;
constexpr u64 kLeastRows = 8;  // that a block takes at a time
constexpr u32 kFinishExperts = 16;
constexpr u32 kTurnsInRegisters = 4;  // rows a lane sums in 32 bits
constexpr u32 kMostFinishing = kRouteMaxExperts / kFinishExperts;
constexpr size_t kRouteScratchHead = 256 + 8 * kMostFinishing;

__device__ __forceinline__ u32 max_u(u32 a, u32 b) { return a > b ? a : b; }

// e^x for x <= 0 to about one unit in the last place: the rounding of x log2(e), which
// grows with |x|, is made up for by two multiply-adds (x - t ln 2 is what the rounded t
// left).  Differences as far apart as the type reaches (and -inf) are cut to one whose
// exponential is 0, and so is NaN: rows that hold one are told apart beforehand.
__device__ __forceinline__ float exp_f(float x) {
  x = __builtin_fmaxf(x, -150.f);
  const float t = x * 1.44269502f;
  const float r = __builtin_fmaf(-t, 0.693147182f, x);
  const float e = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(e, r, e);
}

// A sigmoid and its complement, each to a few units in its own last place.
struct Sigmoid {
  float up, down;
};
__device__ __forceinline__ Sigmoid sigmoid_of(float x) {
  const float e = exp_f(-__builtin_fabsf(x)), t = 1.f + e;
  float r = __builtin_amdgcn_rcpf(t);
  r = __builtin_fmaf(__builtin_fmaf(-t, r, 1.f), r, r);
  const float far = e * r;
  Sigmoid s = {x < 0.f ? far : r, x < 0.f ? r : far};
  if (x != x) s.up = s.down = x;
  return s;
}

// Scores far below 1.  A sigmoid up to e^-21 is its exponential to 2^-30 of itself, so a row that
// has no larger one, and chosen scores whose sum is below 2^-30, share by their distances from the
// largest of them: in 32 bits the scores themselves would be 0 from 2^-126 down.  The definition's
// are 0 where 64 bits hold none, below 2^-1075 (e^-745.13).
constexpr float kFarScores = 0x1p-30f, kFarLogit = -21.f, kLeastLogit = -745.133f;
// of a softmax, relative to the row's top and sum
__device__ __forceinline__ float least_held(float top, float inverse) {
  return top + __builtin_fmaf(__builtin_amdgcn_logf(inverse), 0.693147181f, kLeastLogit);
}
__device__ __forceinline__ float far_share(float l, float largest, float least) {
  return l < least ? 0.f : exp_f(l - largest);
}

// Four neighbouring entries with one load or store.
template <class T>
struct alignas(4 * sizeof(T)) Four {
  T e[4];
};

// One row in registers: C entries per lane.  QUAD: four neighbours at a time.
template <int G, int C, bool QUAD>
struct Row {
  float v[C];
  float e[C];  // exp(v - top)
  bool live;
  bool far;  // with sigmoid scores: e is relative to the largest one's
  float top;

  static __device__ __forceinline__ u32 index(int i, u32 g) {
    return QUAD ? (u32)(i / 4 * G) * 4 + (u32)(i % 4) + g * 4 : (u32)i * G + g;
  }
  // What a lane's loads of a row bring.
  template <class T>
  struct Raw {
    Four<T> q[QUAD ? C / 4 : 1];
    T s[QUAD ? 1 : C];
  };
  // All loads go out before the first is used: places past the row's end read its start,
  // rows past the last (x of a row that exists) are read and not taken.
  template <class T>
  static __device__ __forceinline__ void fetch(const T* x, u32 E, u32 g, Raw<T>& raw) {
    if constexpr (QUAD) {
#pragma unroll
      for (int i = 0; i < C; i += 4) {  // E is a multiple of 4
        const u32 at = index(i, g);
        raw.q[i / 4] = *reinterpret_cast<const Four<T>*>(x + (at < E ? at : 0u));
      }
    } else {
#pragma unroll
      for (int i = 0; i < C; ++i) raw.s[i] = x[index(i, g) < E ? index(i, g) : 0u];
    }
  }
  template <class T>
  __device__ __forceinline__ void take(const Raw<T>& raw, u32 E, u32 g, bool in) {
    if constexpr (QUAD) {
#pragma unroll
      for (int i = 0; i < C; i += 4) {  // by words: two entries of 16 bits at a time
        Four<T> q = raw.q[i / 4];
        u32 w[sizeof(T)];
        __builtin_memcpy(w, &q, 4 * sizeof(T));
#pragma unroll
        for (u32 k = 0; k < sizeof(T); ++k) w[k] = in && index(i, g) < E ? w[k] : NoneWord<T>::value;
        __builtin_memcpy(&q, w, 4 * sizeof(T));
#pragma unroll
        for (int k = 0; k < 4; ++k) v[i + k] = to_f32(q.e[k]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < C; ++i) v[i] = in && index(i, g) < E ? to_f32(raw.s[i]) : kNone;
    }
  }
  template <class T>
  __device__ __forceinline__ void load(const T* x, u32 E, u32 g, bool in) {
    Raw<T> raw;
    fetch(x, E, g, raw);
    take(raw, E, g, in);
  }
  // The largest entry and the exponentials.  A row that holds a NaN has NaN for its top,
  // and every NaN becomes the one that the order ranks first; there, and where the top is
  // +inf, all exponentials are NaN.
  __device__ __forceinline__ void weigh(bool in) {
    static_assert(C % 2 == 0, "pairs behind the first, and one");
    float m = v[0];
    bool nan = false;
#pragma unroll
    for (int i = 1; i + 1 < C; i += 2) m = max3(m, v[i], v[i + 1]);
    m = max_f(m, v[C - 1]);
#pragma unroll
    for (int i = 0; i < C; i += 2) nan |= __builtin_isunordered(v[i], v[i + 1 < C ? i + 1 : i]);
    top = group_reduce<G>(m, max_f);
    live = in && !(top == kNone);
    const float base = live ? top : 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) e[i] = exp_f(v[i] - base);  // entries of -inf: 0
    if (__builtin_expect(__ballot(nan || top == __builtin_huge_valf()) != 0, 0)) {
      const float first = __uint_as_float(0x7FFFFFFFu);
      if (group_reduce<G>((u32)nan, max_u)) {
        top = first;
        live = true;
      }
      if (!(top < __builtin_huge_valf())) {
#pragma unroll
        for (int i = 0; i < C; ++i) {
          v[i] = v[i] != v[i] ? first : v[i];
          e[i] = first;
        }
      }
    }
  }
  // Sigmoid scores for e, and falling = 1 - e where the caller has room for it, each to 8 units of
  // 2^-24 of itself.  nan: this lane has one.  e is 0 in a row that does not take part, and beside a
  // larger score than e^-21 for logits up to -87.4 (the reciprocal's result is flushed; beyond -88
  // differences do not count, so that nothing overflows on the way); so is falling there.
  template <int N>
  __device__ __forceinline__ void score(bool in, bool& nan, float (&falling)[N]) {
    static_assert(C % 2 == 0, "pairs behind the first, and one");
    float m = v[0];
#pragma unroll
    for (int i = 1; i + 1 < C; i += 2) m = max3(m, v[i], v[i + 1]);
    m = max_f(m, v[C - 1]);
#pragma unroll
    for (int i = 0; i < C; i += 2) nan |= __builtin_isunordered(v[i], v[i + 1]);
    top = group_reduce<G>(m, max_f);
    live = in && !(top == kNone);
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const float x = __builtin_amdgcn_fmed3f(v[i], -88.f, 150.f), y = x * -1.44269502f;
      const float r = __builtin_fmaf(y, -0.693147182f, -x);  // what the rounding of y left
      const float t = __builtin_amdgcn_exp2f(y), u = __builtin_fmaf(t, r, t);
      e[i] = __builtin_amdgcn_rcpf(u + 1.f);
      if constexpr (N == C) falling[i] = u * e[i];
    }
    if (!in) {  // rows that are not live hold -inf
#pragma unroll
      for (int i = 0; i < C; ++i) e[i] = 0.f;
    }
    far = live && top < kFarLogit;
    if (__builtin_expect(__ballot(far) != 0, 0)) {
#pragma unroll
      for (int i = 0; i < C; ++i) {
        e[i] = far ? far_share(v[i], top, kLeastLogit) : e[i];
        if constexpr (N == C) falling[i] = far ? 1.f : falling[i];
      }
    }
    if (__builtin_expect(__ballot(nan) != 0, 0)) {
      if (group_reduce<G>((u32)nan, max_u)) live = in;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        e[i] = v[i] != v[i] ? v[i] : e[i];
        if constexpr (N == C) falling[i] = v[i] != v[i] ? v[i] : falling[i];
      }
    }
  }
  // 1 / the row's sum; 0 for a row that is not live.  ALL_NONE: or all of whose scores are 0, which
  // sigmoid scores may be.
  template <bool ALL_NONE = false>
  __device__ __forceinline__ float inverse() const {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) s += e[i];
    s = group_reduce<G>(s, add_f);
    if constexpr (ALL_NONE) return live && s != 0.f ? 1.f / s : 0.f;
    return live ? 1.f / s : 0.f;
  }
};

// Selection keys of 32 bits: the value's ordered code with its low bits replaced by the
// entry's complement, so that the largest key is the first entry by value, then lower
// index, wherever the bits that are left tell the values apart.
constexpr int key_bits(int entries) {
  int b = 0;
  while ((1 << b) < entries) ++b;
  return b;
}

// A launch of several blocks leaves each block's counts, sums and live rows here for the
// finishing launch; one block alone writes the outputs itself.
struct RouteScratch {
  u64* loss;     // the finishing blocks' parts of the loss, and how many there are
  double* parts; // small ones of them, a place per finishing block
  double* sums;  // blocks * E
  u32* counts;   // blocks * E
  u32* rows;     // blocks
};

__host__ __device__ inline RouteScratch route_scratch(char* s, u32 blocks, u32 E) {
  RouteScratch r;
  r.loss = (u64*)s;
  r.parts = (double*)(s + 256);
  r.sums = (double*)(s + kRouteScratchHead);
  r.counts = (u32*)(r.sums + (u64)blocks * E);
  r.rows = r.counts + (u64)blocks * E;
  return r;
}

// Sum of one double per thread over the block, in a fixed order; thread 0 has it.
template <int WAVES>
__device__ __forceinline__ double block_sum(double v, double* wave_tot) {
#pragma unroll
  for (int d = kWave / 2; d; d >>= 1) v += __shfl_down(v, d);
  if (lane_id() == 0) wave_tot[threadIdx.x / kWave] = v;
  __syncthreads();
  double s = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) s += wave_tot[w];
  return s;
}

__device__ __forceinline__ float balance_of(double total, u64 rows, u32 E, u32 k) {
  return rows ? (float)((double)E * total / ((double)rows * (double)k * (double)rows)) : 0.f;
}

// Blocks of a kernel that takes `each` rows a block at a time: no more than are resident at
// once, as what a block does before and after its rows (the sums over its lanes and
// wavefronts; the loss's factors) costs as much as a row or two a wavefront, and no more
// than share the rounds evenly.
inline u32 route_blocks(u64 T, u32 each, u32 resident) {
  const u64 rounds = (T + each - 1) / each;
  if (rounds <= resident) return rounds ? (u32)rounds : 1;
  const u64 turns = (rounds + resident - 1) / resident;
  return (u32)((rounds + turns - 1) / turns);
}

// L::launch with the lanes per row and entries per lane: the smallest that hold the row, and the fewest lanes
// that hold it in 16 entries each (16384 x 384 fp16, forward and backward: 25 us by 32 lanes
// with 12 entries, 34 by 64 with 8; x 700: 38 by 64 with 12, 43 with 16).  Up to 64 entries
// 8 lanes are better for long batches, whose blocks of 128 rows reach every CU: 131072 x 64
// bf16, forward with the loss and backward in one graph, 33 us by 8 lanes and 40 by 16; 65536
// rows 22.9 and 24.9, 32768 rows 15.4 and 18.1, 16384 rows 14.1 and 13.1 (fp32 the same way).
// The bound is a constant on the safe side of 256 CUs' 32768 rows.
template <class L, class T, bool QUAD, class A>
hipError_t route_shape(const A& a, hipStream_t s) {
  if (a.E <= 16) return L::template launch<T, 4, 4, QUAD>(a, s);
  if (a.E <= 32) return L::template launch<T, 8, 4, QUAD>(a, s);
  if (a.E <= 64 && a.T >= 65536) return L::template launch<T, 8, 8, QUAD>(a, s);
  if (a.E <= 64) return L::template launch<T, 16, 4, QUAD>(a, s);
  if (a.E <= 128) return L::template launch<T, 16, 8, QUAD>(a, s);
  if (a.E <= 192) return L::template launch<T, 16, 12, QUAD>(a, s);
  if (a.E <= 256) return L::template launch<T, 16, 16, QUAD>(a, s);
  if (a.E <= 384) return L::template launch<T, 32, 12, QUAD>(a, s);
  if (a.E <= 512) return L::template launch<T, 32, 16, QUAD>(a, s);
  if (a.E <= 768) return L::template launch<T, 64, 12, QUAD>(a, s);
  return L::template launch<T, 64, 16, QUAD>(a, s);
}

inline const void* written(const RouteArgs&) { return nullptr; }
inline const void* written(const RouteGradArgs& a) { return a.d_x; }

// Four entries at a time where every row starts at a multiple of four entries' bytes and
// ends with a whole four.
template <class L, class T, class A>
hipError_t route_rows(const A& a, hipStream_t s) {
  const uintptr_t bases = (uintptr_t)a.x | (uintptr_t)written(a);
  if (a.E % 4 == 0 && a.ld % 4 == 0 && bases % (4 * sizeof(T)) == 0) return route_shape<L, T, true>(a, s);
  return route_shape<L, T, false>(a, s);
}

template <class L, class A>
hipError_t route_type(const A& a, int dtype, hipStream_t s) {
  if (dtype == PROFK_FP32) return route_rows<L, float>(a, s);
  if (dtype == PROFK_FP16) return route_rows<L, Half16>(a, s);
  return route_rows<L, Brain16>(a, s);
}

}  // namespace profk
