// Sampling a token from each row of logits, with temperature, top-k, top-p and min-p,
// from a given uniform number per row.
//
// Mathematics.  Order a row's entries by value, descending, ties by lower index.  With
// w_i = exp((l_i - max) / T), every filter keeps a prefix of that order:
//   K = the first top_k entries;  P = the shortest prefix of K with mass >= top_p mass(K);
//   F = the entries of P with w_i >= min_p;  W = mass(F).
// The token is the first entry of the order whose cumulative mass exceeds u W.  So the
// whole operator is a few questions of one kind, "where does the running count, or the
// running mass, of the order first reach Q?", and no row is ever sorted: a histogram answers
// a question up to one bin, whose entries are then looked at.  One workgroup of 1024 threads
// takes a row, in one of three ways: 16-bit logits by a counter for every value; 32-bit
// logits by 4096 value bins; rows that overflow either by value bins split as often as it
// takes (the first part of this file, right for every row).
//
// Exactness.  Weights are integers q_i = round(w_i 2^F), with F = min(50, 62 - ceil(log2 V))
// as large as lets a row's sum fit 63 bits (50 up to 4096 entries, 45 at 2^17, 38 at 2^24),
// from 64-bit floats.  Integer sums do not depend on their order, so LDS atomics give the same
// bits on every run.  A row's V roundings move a border by at most V 2^-(F+1) of the largest
// weight: 2^-29 at 2^17 entries and 2^-27 at 2^18, below the 2^-24 steps of u, but 2^-23 at
// 2^20 and 2^-15 at 2^24, so in rows that long a draw next to a border may fall on its other
// side.  (Counted values are summed in 64-bit floats, sixteen at a time, and rounded to such
// integers.)  An entry below about 2^-F of the largest counts as absent.
#include <type_traits>

#include "block_select.h"
#include "launch.h"
#include "ops_device.h"

namespace profk {

namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / kWave;
constexpr u32 kTokBins = kThreads;  // value bins of a histogram, one per thread in the scans
constexpr u32 kListCap = 4096;      // entries collected into LDS and sorted

struct RowSettings {
  float t, p, m;
  u64 k;  // 0: all
  float u;
};

struct Prefix {  // a prefix of the order: entries, mass, and its last entry's key (0: not known)
  u64 n, mass, key;
};

struct TokLds {
  u64 mass[kTokBins];
  u32 cnt[kTokBins];
  u64 list[kListCap];
  u64 cum[kListCap];  // inclusive mass of the sorted list
  u64 wave_m[kWaves];
  u64 wave_n[kWaves];
  u64 ans_key, ans_mass, ans_n;
  u32 ans_bin, list_n;
  u32 lo, hi;
  u64 minp_mass;
  u32 minp_n;
};

// Lane exchanges of a scan over the wavefront, as DPP moves (a shuffle through LDS takes
// about ten times as long, and every answer waits for several scans): within rows of 16 by
// 1, 2, 4, 8, then each row's last lane to the rows after it.  Lanes without a partner get
// `none`.
template <int STEP>
__device__ __forceinline__ u32 scan_from(u32 v, u32 none) {
  constexpr int ctrl = STEP < 4 ? 0x110 | 1 << STEP : STEP == 4 ? 0x142 : 0x143;
  constexpr int rows = STEP < 4 ? 0xF : STEP == 4 ? 0xA : 0xC;
  return (u32)__builtin_amdgcn_update_dpp((int)none, (int)v, ctrl, rows, 0xF, false);
}
template <int STEP>
__device__ __forceinline__ u64 scan_from(u64 v, u64 none) {
  return (u64)scan_from<STEP>((u32)(v >> 32), (u32)(none >> 32)) << 32 | scan_from<STEP>((u32)v, (u32)none);
}
template <class V, class F>
__device__ __forceinline__ V wave_scan(V v, V none, F f) {  // inclusive
  v = f(v, scan_from<0>(v, none));
  v = f(v, scan_from<1>(v, none));
  v = f(v, scan_from<2>(v, none));
  v = f(v, scan_from<3>(v, none));
  v = f(v, scan_from<4>(v, none));
  return f(v, scan_from<5>(v, none));
}
__device__ __forceinline__ u32 of_lane(u32 v, u32 lane) {  // the lane is the same for all
  return (u32)__builtin_amdgcn_readlane((int)v, (int)lane);
}
__device__ __forceinline__ u64 of_lane(u64 v, u32 lane) {
  return (u64)of_lane((u32)(v >> 32), lane) << 32 | of_lane((u32)v, lane);
}
template <class V>
__device__ __forceinline__ V wave_scan(V v) {
  return wave_scan(v, (V)0, [](V x, V y) { return x + y; });
}
template <class V>
__device__ __forceinline__ V wave_sum(V v) {
  return of_lane(wave_scan(v), kWave - 1);
}
template <class V>
__device__ __forceinline__ V wave_min(V v) {
  return of_lane(wave_scan(v, (V)~(V)0, [](V x, V y) { return x < y ? x : y; }), kWave - 1);
}

// The value of the lane across in a quad: quad_perm [1,0,3,2] or [2,3,0,1].
template <int CTRL>
__device__ __forceinline__ u32 quad_xor(u32 v) {
  return (u32)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
template <int CTRL>
__device__ __forceinline__ u64 quad_xor(u64 v) {
  return (u64)quad_xor<CTRL>((u32)(v >> 32)) << 32 | quad_xor<CTRL>((u32)v);
}

// Inclusive scan over the block, one u64 per thread.
__device__ __forceinline__ u64 block_scan_u64(u64 v, u64* wave_tot) {
  v = wave_scan(v);
  const u32 wid = threadIdx.x / kWave;
  if (lane_id() == kWave - 1) wave_tot[wid] = v;
  lds_barrier();
  const u64 t = wave_scan(lane_id() < (u32)kWaves ? wave_tot[lane_id()] : 0);
  const u64 before = wid ? of_lane(t, __builtin_amdgcn_readfirstlane(wid) - 1) : 0;
  lds_barrier();
  return v + before;
}

// Both at once.
__device__ __forceinline__ void block_scan(u64& m, u32& n, u64* wave_m, u32* wave_n) {
  m = wave_scan(m);
  n = wave_scan(n);
  const u32 wid = threadIdx.x / kWave, lane = lane_id();
  if (lane == kWave - 1) {
    wave_m[wid] = m;
    wave_n[wid] = n;
  }
  lds_barrier();
  const u64 tm = wave_scan(lane < (u32)kWaves ? wave_m[lane] : 0);
  const u32 tn = wave_scan(lane < (u32)kWaves ? wave_n[lane] : 0);
  if (wid) {
    m += of_lane(tm, __builtin_amdgcn_readfirstlane(wid) - 1);
    n += of_lane(tn, __builtin_amdgcn_readfirstlane(wid) - 1);
  }
}

// Calls f(value, index) for every entry of the row, each once, over the block's threads.
// 16-byte loads between the row's first and last 16-byte boundaries.
template <class T, class F>
__device__ __forceinline__ void for_each_entry(const T* row, u32 V, F f) {
  constexpr u32 W = 16 / sizeof(T);
  u32 head = (u32)((16 - ((uintptr_t)row & 15)) & 15) / (u32)sizeof(T);
  if (head > V) head = V;
  const u32 nvec = (V - head) / W;
  for (u32 i = threadIdx.x; i < head; i += kThreads) f(to_f32(row[i]), i);
  const uint4* vec = reinterpret_cast<const uint4*>(row + head);
  for (u32 j = threadIdx.x; j < nvec; j += kThreads) {
    const uint4 v = vec[j];
    T e[W];
    __builtin_memcpy(e, &v, 16);
#pragma unroll
    for (u32 w = 0; w < W; ++w) f(to_f32(e[w]), head + j * W + w);
  }
  for (u32 i = head + nvec * W + threadIdx.x; i < V; i += kThreads) f(to_f32(row[i]), i);
}

// A constant in scalar registers: as a literal of a 64-bit instruction it would take two
// vector moves.
__device__ __forceinline__ double scalar(double v) {
  asm("" : "+s"(v));
  return v;
}

// 2^y for y <= 0: y = n + f with |f| <= 1/2, the Taylor series of e^(f ln 2) to the power
// 13 (the next term is below 2^-57), scaled by 2^n.  2^0 is exactly 1; NaN gives 0.  The
// even and the odd powers are summed apart, in half the steps.
__device__ __forceinline__ double pow2(double y, int F = 0) {  // times 2^F
  y = __builtin_fmax(y, -2000.0);
  const double n = rint(y), x = (y - n) * scalar(0.69314718055994530942), xx = x * x;
  double even = scalar(1.0 / 479001600), odd = scalar(1.0 / 6227020800.0);
  even = __builtin_fma(even, xx, scalar(1.0 / 3628800));
  odd = __builtin_fma(odd, xx, scalar(1.0 / 39916800));
  even = __builtin_fma(even, xx, scalar(1.0 / 40320));
  odd = __builtin_fma(odd, xx, scalar(1.0 / 362880));
  even = __builtin_fma(even, xx, scalar(1.0 / 720));
  odd = __builtin_fma(odd, xx, scalar(1.0 / 5040));
  even = __builtin_fma(even, xx, scalar(1.0 / 24));
  odd = __builtin_fma(odd, xx, scalar(1.0 / 120));
  even = __builtin_fma(even, xx, 0.5);
  odd = __builtin_fma(odd, xx, scalar(1.0 / 6));
  even = __builtin_fma(even, xx, 1.0);
  odd = __builtin_fma(odd, xx, 1.0);
  return __builtin_ldexp(__builtin_fma(odd, x, even), (int)n + F);
}

// The row's weights relative to its largest value.
struct Weigher {
  float top;     // the largest value
  double c;      // log2(e) / T
  double scale;  // 2^F
  double limit;  // -F: entries below are absent
  double bins;   // bins per unit of the exponent
  __device__ __forceinline__ double exponent(float v) const {
    return v == top ? 0.0 : ((double)v - (double)top) * c;  // 0 also where both are +inf
  }
  __device__ __forceinline__ bool present(double y) const { return y >= limit; }  // false for NaN
  // A weight times 2^F as an integer: adding 2^52 leaves it, rounded, in the low bits (F <= 50).
  __device__ __forceinline__ u64 whole(double p) const {
    return __builtin_bit_cast(u64, p + 0x1p52) - __builtin_bit_cast(u64, 0x1p52);
  }
  __device__ __forceinline__ u64 weight(double y) const { return (u64)rint(pow2(y) * scale); }
  __device__ __forceinline__ u32 bin(double y) const {  // monotone in the value
    const double b = -y * bins;
    return b >= (double)(kTokBins - 1) ? kTokBins - 1 : (u32)b;
  }
};

__device__ __forceinline__ float value_of_key(u64 key) { return __uint_as_float(bits_of_ord32((u32)(key >> 32))); }

// The bin where the running count (by_mass false) or mass reaches Q.  cnt and mass hold
// inclusive prefixes.  The answer is in L.ans_bin after the barrier; Q is at most the total.
__device__ __forceinline__ u32 find_bin(TokLds& L, bool by_mass, u64 Q) {
  const u32 b = threadIdx.x;
  const u64 here = by_mass ? L.mass[b] : (u64)L.cnt[b];
  const u64 before = b ? (by_mass ? L.mass[b - 1] : (u64)L.cnt[b - 1]) : 0;
  if (here >= Q && before < Q) L.ans_bin = b;
  __syncthreads();
  const u32 r = L.ans_bin;
  __syncthreads();
  return r;
}

// cnt and mass become inclusive prefixes.
__device__ __forceinline__ void scan_bins(TokLds& L) {
  const u32 b = threadIdx.x;
  const u64 m = block_scan_u64(L.mass[b], L.wave_m);
  const u64 n = block_scan_u64(L.cnt[b], L.wave_n);
  L.mass[b] = m;
  L.cnt[b] = (u32)n;
  __syncthreads();
}

// Sorts L.list[0..n) descending and fills L.cum with the inclusive masses.
__device__ __forceinline__ void sort_and_weigh(TokLds& L, u32 n, const Weigher& w) {
  u32 P = 1;
  while (P < n) P <<= 1;
  for (u32 i = n + threadIdx.x; i < P; i += kThreads) L.list[i] = 0;
  __syncthreads();
  block_bitonic_desc(L.list, P);
  u64 base = 0;
  for (u32 s = 0; s < n; s += kThreads) {
    const u32 i = s + threadIdx.x;
    const u64 q = i < n ? w.weight(w.exponent(value_of_key(L.list[i]))) : 0;
    const u64 c = base + block_scan_u64(q, L.wave_m);
    if (i < n) L.cum[i] = c;
    if (threadIdx.x == kThreads - 1) L.ans_mass = c;
    __syncthreads();
    base = L.ans_mass;
    __syncthreads();
  }
}

// The answer inside the sorted list, whose first entry comes after `n0` entries and
// `m0` mass of the order.
__device__ __forceinline__ Prefix find_in_list(TokLds& L, u32 n, u64 n0, u64 m0, bool by_mass, u64 Q) {
  if (by_mass) {
    for (u32 i = threadIdx.x; i < n; i += kThreads) {
      const u64 here = m0 + L.cum[i], before = i ? m0 + L.cum[i - 1] : m0;
      if (here >= Q && before < Q) L.ans_bin = i;
    }
    __syncthreads();
  } else {
    if (threadIdx.x == 0) L.ans_bin = (u32)(Q - n0 - 1);
    __syncthreads();
  }
  const u32 i = L.ans_bin;
  const Prefix r = {n0 + i + 1, m0 + L.cum[i], L.list[i]};
  __syncthreads();
  return r;
}

// Collects the entries accepted by `pick(value, exponent)` into L.list (at most kListCap;
// the caller knows the number).
template <class T, class F>
__device__ __forceinline__ u32 collect(TokLds& L, const T* row, u32 V, const Weigher& w, F pick) {
  if (threadIdx.x == 0) L.list_n = 0;
  __syncthreads();
  for_each_entry(row, V, [&](float v, u32 i) {
    const double y = w.exponent(v);
    if (w.present(y) && pick(v, y)) {
      const u32 at = atomicAdd(&L.list_n, 1u);
      if (at < kListCap) L.list[at] = make_key(__float_as_uint(v), i);
    }
  });
  __syncthreads();
  const u32 n = L.list_n < kListCap ? L.list_n : kListCap;
  __syncthreads();
  return n;
}

// Histogram of the row's present entries into the value bins, as prefix sums.
template <class T>
__device__ __forceinline__ void value_histogram(TokLds& L, const T* row, u32 V, const Weigher& w, float min_p) {
  L.mass[threadIdx.x] = 0;
  L.cnt[threadIdx.x] = 0;
  if (threadIdx.x == 0) {
    L.minp_mass = 0;
    L.minp_n = 0;
  }
  __syncthreads();
  u64 mm = 0;
  u32 mn = 0;
  for_each_entry(row, V, [&](float v, u32) {
    const double y = w.exponent(v);
    if (!w.present(y)) return;
    const double e = pow2(y);
    const u64 q = (u64)rint(e * w.scale);
    const u32 b = w.bin(y);
    atomicAdd(&L.mass[b], q);
    atomicAdd(&L.cnt[b], 1u);
    if (e >= (double)min_p) {
      mm += q;
      ++mn;
    }
  });
  if (min_p > 0.f && mn) {
    atomicAdd(&L.minp_mass, mm);
    atomicAdd(&L.minp_n, mn);
  }
  __syncthreads();
  scan_bins(L);
}

// Position in the order of the first prefix whose count / mass reaches Q.  The value
// histogram (prefix sums) is in L; hist_lost is set where a bin had to be split in its place.
template <class T>
__device__ __forceinline__ Prefix resolve(TokLds& L, const T* row, u32 V, const Weigher& w, bool by_mass, u64 Q, bool want_key,
                          bool& hist_lost) {
  const u32 b = find_bin(L, by_mass, Q);
  u64 n0 = b ? L.cnt[b - 1] : 0, m0 = b ? L.mass[b - 1] : 0;
  const u32 n = L.cnt[b] - (u32)n0;
  if (n <= kListCap) {
    const u32 got = collect(L, row, V, w, [&](float, double y) { return w.bin(y) == b; });
    sort_and_weigh(L, got, w);
    return find_in_list(L, got, n0, m0, by_mass, Q);
  }
  // A bin too full for the list: split its key range, at most four times (2^32 codes, 2^10
  // bins a level).
  hist_lost = true;
  if (threadIdx.x == 0) {
    L.lo = ~0u;
    L.hi = 0;
  }
  __syncthreads();
  u32 lo = ~0u, hi = 0;
  for_each_entry(row, V, [&](float v, u32) {
    const double y = w.exponent(v);
    if (w.present(y) && w.bin(y) == b) {
      const u32 o = ord32(__float_as_uint(v));
      lo = o < lo ? o : lo;
      hi = o > hi ? o : hi;
    }
  });
  atomicMin(&L.lo, lo);
  atomicMax(&L.hi, hi);
  __syncthreads();
  lo = L.lo;
  hi = L.hi;
  __syncthreads();
  for (;;) {
    u32 shift = 0;
    while (((hi - lo) >> shift) >= kTokBins) ++shift;
    L.mass[threadIdx.x] = 0;
    L.cnt[threadIdx.x] = 0;
    __syncthreads();
    for_each_entry(row, V, [&](float v, u32) {
      const u32 o = ord32(__float_as_uint(v));
      if (o < lo || o > hi) return;
      const u32 s = (hi - o) >> shift;
      atomicAdd(&L.mass[s], w.weight(w.exponent(v)));
      atomicAdd(&L.cnt[s], 1u);
    });
    __syncthreads();
    scan_bins(L);
    const u32 s = find_bin(L, by_mass, Q - (by_mass ? m0 : n0));
    const u32 in_bin = L.cnt[s] - (s ? L.cnt[s - 1] : 0);
    const u64 bin_mass = L.mass[s] - (s ? L.mass[s - 1] : 0);
    n0 += s ? L.cnt[s - 1] : 0;
    m0 += s ? L.mass[s - 1] : 0;
    hi -= s << shift;
    lo = (hi - lo) >> shift ? hi - ((1u << shift) - 1) : lo;
    __syncthreads();
    if (in_bin <= kListCap) {
      const u32 got = collect(L, row, V, w, [&](float v, double) {
        const u32 o = ord32(__float_as_uint(v));
        return o >= lo && o <= hi;
      });
      sort_and_weigh(L, got, w);
      return find_in_list(L, got, n0, m0, by_mass, Q);
    }
    if (shift == 0) {  // one value, more often than the list holds: equal weights
      const u64 q = bin_mass / in_bin;
      const u64 j = by_mass ? (Q - m0 + q - 1) / q : Q - n0;
      Prefix r = {n0 + j, m0 + j * q, 0};
      if (!want_key) return r;
      // the j-th of them by index: counts per contiguous stretch of the row, then one stretch
      const u32 per = (V + kThreads - 1) / kThreads;
      const u32 i0 = threadIdx.x * per, i1 = i0 + per < V ? i0 + per : V;
      u32 c = 0;
      for (u32 i = i0; i < i1; ++i) c += ord32(__float_as_uint(to_f32(row[i]))) == hi;
      const u64 upto = block_scan_u64(c, L.wave_n);
      if (upto >= j && upto - c < j) {
        u64 left = j - (upto - c);
        for (u32 i = i0; i < i1; ++i)
          if (ord32(__float_as_uint(to_f32(row[i]))) == hi && --left == 0) {
            L.ans_key = ((u64)hi << 32) | (u64)(~i);
            break;
          }
      }
      __syncthreads();
      r.key = L.ans_key;
      __syncthreads();
      return r;
    }
  }
}

__device__ __forceinline__ RowSettings row_settings(const TokenArgs& a, u64 r) {
  RowSettings s;
  s.t = a.t_row ? a.t_row[r] : a.t;
  s.p = a.p_row ? a.p_row[r] : a.p;
  s.m = a.m_row ? a.m_row[r] : a.m;
  const int64_t k = a.k_row ? a.k_row[r] : a.k;
  s.k = k <= 0 || (u64)k >= a.V ? 0 : (u64)k;
  const float u = a.u[r];
  s.u = u >= 0.f ? (u < 0x1.fffffep-1f ? u : 0x1.fffffep-1f) : 0.f;  // NaN: 0
  if (!(s.t > 0.f)) s.t = 0.f;             // greedy
  if (!(s.p < 1.f)) s.p = 1.f;             // off
  if (!(s.m > 0.f)) s.m = 0.f;             // off
  if (s.m > 1.f) s.m = 1.f;
  return s;
}

// One row by value bins: any type, any length.
template <class T>
__device__ __forceinline__ void sample_row_by_value(TokLds& L, const TokenArgs& a, u64 r) {
  const T* row = reinterpret_cast<const T*>(a.x) + r * a.ld;
  const u32 V = (u32)a.V;
  const RowSettings s = row_settings(a, r);
  // 1. the largest value and its lowest index (NaN ranks above everything)
  if (threadIdx.x == 0) {
    L.ans_key = 0;
    L.ans_bin = 0;
  }
  __syncthreads();
  u64 best = 0;
  for_each_entry(row, V, [&](float v, u32 i) {
    const u64 key = make_key(__float_as_uint(v), i);
    best = key > best ? key : best;
  });
  atomicMax(&L.ans_key, best);
  __syncthreads();
  best = L.ans_key;
  __syncthreads();
  const u32 top = (u32)(best >> 32);
  if (top >= ord32(0x7F800001u) || top <= ord32(0xFF800000u) || s.t == 0.f) {
    if (threadIdx.x == 0) {
      const bool nan = top >= ord32(0x7F800001u), none = top <= ord32(0xFF800000u);
      a.tokens[r] = nan || none ? -1 : (int64_t)key_index(best);
      a.logprobs[r] = nan ? __uint_as_float(0x7FC00000u) : none ? -__builtin_huge_valf() : 0.f;
    }
    return;
  }
  Weigher w;
  w.top = value_of_key(best);
  w.c = 1.4426950408889634074 / (double)s.t;
  u32 lg = 0;
  while ((1ull << lg) < a.V) ++lg;
  const int F = 62 - (int)lg < 50 ? 62 - (int)lg : 50;
  w.scale = (double)(1ull << F);
  w.limit = -(double)F;
  w.bins = (double)kTokBins / (double)(F + 1);
  // 2. histogram, and the questions in their order
  value_histogram(L, row, V, w, s.m);
  const u64 N = L.cnt[kTokBins - 1], Z = L.mass[kTokBins - 1];
  const u64 mn = L.minp_n, mm = L.minp_mass;
  __syncthreads();
  u64 kn = N, km = Z;  // what is kept: entries and mass
  bool lost = false;
  for (int step = 0; step < 4; ++step) {  // one place where the search is inlined
    bool by_mass = true;
    u64 Q;
    if (step == 0) {
      if (!s.k || s.k >= kn) continue;
      by_mass = false;
      Q = s.k;
    } else if (step == 1) {
      Q = (u64)ceil((double)s.p * (double)km);
      if (Q < 1 || !(s.p > 0.f)) Q = 1;
      if (s.p >= 1.f || Q >= km) continue;
    } else if (step == 2) {
      if (s.m > 0.f && mn < kn) {
        kn = mn;
        km = mm;
      }
      continue;
    } else {
      Q = (u64)((double)s.u * (double)km) + 1;
      if (Q > km) Q = km;
    }
    if (lost) {
      value_histogram(L, row, V, w, 0.f);
      lost = false;
    }
    const Prefix at = resolve(L, row, V, w, by_mass, Q, step == 3, lost);
    if (step < 3) {
      kn = at.n;
      km = at.mass;
    } else if (threadIdx.x == 0) {
      const double y = w.exponent(value_of_key(at.key));
      a.tokens[r] = (int64_t)key_index(at.key);
      a.logprobs[r] = (float)(y * 0.69314718055994530942 - log((double)km / w.scale));
    }
  }
}

// ---------------------------------------------------------------------------------------
// Rows of 16-bit logits: a counter for every value.
//
// A row of such logits has few different values, so it is enough to count them: 65536
// counters of 16 bits fill 128 KB of LDS, an entry costs one LDS addition and no
// exponential, and the weights are worked out once per value that occurs, not once per
// entry.  512 rows of 131072: 58 us, 2.3 TB/s (by value bins, two passes with an exponential
// and two additions per entry: 356 us).  Of a row's 28 us the counting takes 14 to 16, the
// weights 6, the questions 2, the chosen value's entries 3; over the kernel the vector units
// are at work 67 % of the cycles and the LDS 30 %, two thirds of that for bank conflicts of
// the additions.  Codes go down with the value: code(h) = h ^ 0x7FFF for
// h >= 0, else h, so -0 comes right after +0; a positive value's counter is the low half of
// word code, a negative one's the high half of word code - 0x8000.  A counter that
// overflows makes the counters' sum differ from the number of entries counted, since each
// carry takes 65536 or 65535 from it; such a row (it holds 65536 equal entries) goes by
// value bins, as a last part of the same kernel (a second launch for it took 4 us).
//
// Sixteen neighbouring codes (a cell) lie within one binade, so their weights are a geometric
// series: two exponentials give all of them, and equal largest entries weigh exactly 2^F.  Cells are summed in 64-bit
// floats and rounded to integers; sums of cells are exact, so the answer depends on the
// counters alone.
constexpr u32 kCodeWords = 32768;
constexpr u32 kCellCodes = 16;
constexpr u32 kGroupCodes = kCellCodes * kWave;  // one wavefront's step: 1024 codes
constexpr u32 kGroups = 65536 / kGroupCodes;
constexpr u32 kUnitCodes = kWave;  // what a question is answered to before it looks at codes
constexpr u32 kUnits = 65536 / kUnitCodes;
static_assert(kUnits == (u32)kThreads, "a thread per unit in the scans");
constexpr u32 kMatchCap = 1024;

struct CodeLds {
  u32 cnt[kCodeWords];
  u64 mass[kUnits];  // inclusive prefixes
  u32 n[kUnits];
  u32 match[kMatchCap];
  u64 scan[kWaves];
  u32 scan_n[kWaves];
  u32 top, end, counted, matches;  // the first and the last code; the entries counted
  u32 code, j;
};


typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef short i16x2 __attribute__((ext_vector_type(2)));

// The counters' words, permuted so that 16 lanes that read four words each of 16
// neighbouring cells use all banks.
__device__ __forceinline__ u32 counter_word(u32 code) {
  const u32 w = code & 0x7FFFu;
  return w ^ (w >> 4 & 0xCu);
}

__device__ __forceinline__ u32 pk_counter_words(u32 codes) {
  const u32 w = codes & 0x7FFF7FFFu;
  return w ^ (__builtin_bit_cast(u32, __builtin_bit_cast(u16x2, w) >> 4) & 0x000C000Cu);
}

// Four times the low or the high 16 bits, as one instruction.
template <int HIGH>
__device__ __forceinline__ u32 word_bytes(u32 v) {
  const u32 two = 2;
  u32 r;
  if constexpr (HIGH)
    asm("v_lshlrev_b32_sdwa %0, %1, %2 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:DWORD src1_sel:WORD_1"
        : "=v"(r) : "v"(two), "v"(v));
  else
    asm("v_lshlrev_b32_sdwa %0, %1, %2 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:DWORD src1_sel:WORD_0"
        : "=v"(r) : "v"(two), "v"(v));
  return r;
}
__device__ __forceinline__ u32* counter_at(CodeLds& L, u32 bytes) {
  return reinterpret_cast<u32*>(reinterpret_cast<char*>(L.cnt) + bytes);
}

template <class T> struct CodeOf;
template <> struct CodeOf<Half16> { static constexpr u32 inf = 0x7C00; };
template <> struct CodeOf<Brain16> { static constexpr u32 inf = 0x7F80; };

template <class T>
__device__ __forceinline__ float value_of_code(u32 c) {
  T h;
  h.bits = (unsigned short)(c < 0x8000u ? c ^ 0x7FFFu : c);
  return to_f32(h);
}

__device__ __forceinline__ u32 code_of_bits(u32 h) { return h < 0x8000u ? h ^ 0x7FFFu : h; }

// A code at or past that of every value >= lim, and of a number.
template <class T>
__device__ __forceinline__ u32 code_past(float lim) {
  constexpr u32 lowest = 0x8000u | (CodeOf<T>::inf - 1);
  if (!(lim > -3.4e38f)) return lowest;
  T h;
  from_f32(lim, h);
  const u32 c = code_of_bits(h.bits) + 1;
  return c < lowest ? c : lowest;
}

// The last code that counts, below a largest value of code `top`: entries under 2^-F of it
// are absent.
template <class T>
__device__ __forceinline__ u32 last_code(u32 top, float t, float F) {
  const float v = value_of_code<T>(top);
  if (!(v < __builtin_huge_valf())) return top;
  return code_past<T>(v - F * 0.69314718f * t);
}


__device__ __forceinline__ u32 pk_signs(u32 w) {  // 0 or 0xFFFF each
  return __builtin_bit_cast(u32, __builtin_bit_cast(i16x2, w) >> 15);
}
__device__ __forceinline__ u32 pk_codes(u32 w) {  // two codes
  return w ^ (0x7FFF7FFFu & ~pk_signs(w));
}
__device__ __forceinline__ u32 pk_min(u32 a, u32 b) {
  const u16x2 x = __builtin_bit_cast(u16x2, a), y = __builtin_bit_cast(u16x2, b);
  return __builtin_bit_cast(u32, __builtin_elementwise_min(x, y));
}
__device__ __forceinline__ u32 pk_max(u32 a, u32 b) {
  const u16x2 x = __builtin_bit_cast(u16x2, a), y = __builtin_bit_cast(u16x2, b);
  return __builtin_bit_cast(u32, __builtin_elementwise_max(x, y));
}
// The 16-byte vectors of a row, a thread's kBatch in flight while others are dealt with (all
// loaded at once, the first waits until the last is on its way: 83 us in place of 64 for 512
// rows of 131072).  NV > 0: a thread's NV vectors stay in registers for later passes.  Places
// past the row's end hold `fill`: put there once (FILL_ONCE), or in each pass, where the longer
// lives of the changed registers would make the compiler spill others.
typedef u32 u32x4 __attribute__((ext_vector_type(4)));
constexpr int kBatch = 4;
template <int NV, bool FILL_ONCE>
struct RowVectors {
  static constexpr int kHeld = NV ? NV : kBatch;
  const u32x4* vec;
  u32 nvec, fill, tid;
  u32x4 held[kHeld];

  __device__ __forceinline__ u32x4 at(u32 j) const {  // 32-bit offsets from a scalar base
    return *reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(vec) + (j < nvec ? j : nvec - 1) * 16u);
  }
  __device__ __forceinline__ u32x4 filled(u32x4 v, u32 j) const {
    return j < nvec ? v : (u32x4){fill, fill, fill, fill};
  }
  // Each pass works out its own places and loads: kept for the next pass, they would take
  // more registers than there are.
  __device__ __forceinline__ void begin() {
    tid = threadIdx.x;
    asm volatile("" : "+v"(tid)::"memory");
  }
  __device__ __forceinline__ void load() {  // of a row of at least one vector
    begin();
#pragma unroll
    for (int i = 0; i < kBatch; ++i) held[i] = at(tid + (u32)i * kThreads);
  }
  // What is worked out of the vectors in one pass is not kept for the next.
  __device__ __forceinline__ void forget() {
    begin();
#pragma unroll
    for (int i = 0; i < kHeld; ++i) asm volatile("" : "+v"(held[i]));
  }
  template <class F>
  __device__ __forceinline__ void first_batch(F f) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) f(filled(held[i], tid + (u32)i * kThreads));
  }
  // f(the vector, its place).  LOAD: the pass after load().
  template <bool LOAD, class F>
  __device__ __forceinline__ void for_each(F f) {
    if constexpr (NV > 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const u32 j = tid + (u32)i * kThreads;
        if (LOAD && i + kBatch < NV) held[i + kBatch < NV ? i + kBatch : 0] = at(j + kBatch * kThreads);
        if constexpr (FILL_ONCE) {
          if (LOAD && (u32)(i + 1) * kThreads > nvec) held[i] = filled(held[i], j);
          if ((u32)i * kThreads < nvec) f(held[i], j);
        } else if ((u32)i * kThreads < nvec) {
          f(filled(held[i], j), j);
        }
        __builtin_amdgcn_sched_barrier(0);  // one vector's work at a time: registers
      }
    } else {
      u32 j = tid;
      for (; j - tid + kBatch * kThreads <= nvec; j += kBatch * kThreads) {
        u32x4 next[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) next[i] = at(j + (u32)(kBatch + i) * kThreads);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          f(held[i], j + (u32)i * kThreads);
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) held[i] = next[i];
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i, j += kThreads)
        if (j - tid < nvec) f(filled(held[i], j), j);
    }
  }
};

// How often each code of the cell of code c0 (a multiple of 16) occurs, and their number.
// EDGE: the group holds the largest value's code `top` or the last that counts.
template <bool EDGE>
__device__ __forceinline__ u32 cell_counters(const CodeLds& L, u32 c0, u32 last, u32 (&n)[kCellCodes]) {
  const u32 shift = c0 >> 15 << 4;
  u32 sum = 0;
#pragma unroll
  for (u32 i = 0; i < kCellCodes; i += 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(&L.cnt[counter_word(c0 + i)]);
    const u32 w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (u32 k = 0; k < 4; ++k) {
      n[i + k] = w[k] >> shift & 0xFFFFu;
      if (EDGE && c0 + i + k > last) n[i + k] = 0;
      sum += n[i + k];
    }
  }
  return sum;
}
// Their mass.  The largest value's cell begins at that value: the codes before it do not
// occur.
template <class T, bool EDGE>
__device__ __forceinline__ u64 cell_mass(const Weigher& w, u32 top, u32 c0, const u32 (&n)[kCellCodes]) {
  const double v0 = (double)value_of_code<T>(c0), v1 = (double)value_of_code<T>(c0 + 1);
  const double rho = pow2((v1 - v0) * w.c);
  double p = EDGE && c0 <= top ? w.scale : pow2((v0 - (double)w.top) * w.c) * w.scale;
  if constexpr (EDGE) {
    double s = 0;
#pragma unroll
    for (u32 i = 0; i < kCellCodes; ++i) {
      s = __builtin_fma((double)n[i], p, s);
      if (c0 + i >= top) p *= rho;
    }
    return (u64)rint(s);
  } else {  // the polynomial in rho by halves
    double s[kCellCodes], power = rho;
#pragma unroll
    for (u32 i = 0; i < kCellCodes; ++i) s[i] = (double)n[i];
#pragma unroll
    for (u32 h = kCellCodes / 2; h; h /= 2) {
#pragma unroll
      for (u32 i = 0; i < h; ++i) s[i] = __builtin_fma(s[2 * i + 1], power, s[2 * i]);
      power *= power;
    }
    return (u64)rint(s[0] * p);
  }
}
__device__ __forceinline__ bool edge_group(u32 g, u32 top, u32 last) { return g == top / kGroupCodes || g == last / kGroupCodes; }

// A code, the prefix of the order before it and through it, and one entry's weight.
struct CodePlace {
  u32 code;
  u32 n0, n1;
  u64 m0, m1, q;
  // entries of this code up to the first whose prefix's mass reaches Q
  __device__ __forceinline__ u32 entries(u64 Q) const {
    const u32 cnt = n1 - n0;
    if (Q <= m0 || cnt <= 1 || q == 0) return 1;
    const u64 X = Q - m0;
    double e = ceil((double)X / (double)q);
    u64 j = e >= (double)cnt ? cnt : (u64)e;  // off by at most one
    if (j * q < X) ++j;
    if (j > 1 && (j - 1) * q >= X) --j;
    return j < 1 ? 1 : j > cnt ? cnt : (u32)j;
  }
  __device__ __forceinline__ u64 mass_through(u32 j) const {
    const u64 m = m0 + j * q;
    return n0 + j == n1 || m > m1 ? m1 : m;
  }
};

enum class Ask { kCount, kMass, kCode };

// Where the running count or mass reaches Q, or the place of code Q, in one wavefront: the
// unit in two steps of LDS reads (64 sixteens of units, then the sixteen), then its codes, a
// lane each.  A step that scanned a thousand codes' masses instead took three times as long.
template <class T>
__device__ __forceinline__ CodePlace find_code(const CodeLds& L, const Weigher& w, u32 top, u32 last, Ask ask, u64 Q) {
  const u32 lane = lane_id();
  u32 unit = __builtin_amdgcn_readfirstlane((u32)Q) / kUnitCodes;
  if (ask != Ask::kCode) {
    constexpr u32 kStep = kUnits / kWave;
    auto reaches = [&](u32 u) { return ask == Ask::kMass ? L.mass[u] >= Q : (u64)L.n[u] >= Q; };
    const u64 far = __builtin_amdgcn_ballot_w64(reaches(lane * kStep + kStep - 1));
    unit = (far ? (u32)__builtin_ctzll(far) : (u32)kWave - 1) * kStep;
    const u64 near = __builtin_amdgcn_ballot_w64(lane >= kStep - 1 || reaches(unit + lane));
    unit += (u32)__builtin_ctzll(near);
  }
  const u64 ms = unit ? L.mass[unit - 1] : 0;
  const u32 ns = unit ? L.n[unit - 1] : 0;
  const u32 code = unit * kUnitCodes + lane;
  const bool mine = code >= top && code <= last;
  const u32 nc = mine ? L.cnt[counter_word(code)] >> (code >> 15 << 4) & 0xFFFFu : 0u;
  const double q = mine ? pow2(w.exponent(value_of_code<T>(code))) * w.scale : 0.0;
  const u64 mc = (u64)rint((double)nc * q), mi = ms + wave_scan(mc);
  const u32 ni = ns + wave_scan(nc);
  u32 i = __builtin_amdgcn_readfirstlane((u32)Q) % kUnitCodes;
  if (ask != Ask::kCode) {
    const u64 some = __builtin_amdgcn_ballot_w64(nc != 0);
    const u64 reach = some & __builtin_amdgcn_ballot_w64(ask == Ask::kMass ? mi >= Q : (u64)ni >= Q);
    i = reach ? (u32)__builtin_ctzll(reach) : some ? 63u - (u32)__builtin_clzll(some) : 0u;
  }
  return {unit * kUnitCodes + i, of_lane(ni - nc, i),       of_lane(ni, i),
          of_lane(mi - mc, i),   of_lane(mi, i), of_lane((u64)rint(q), i)};
}

// The last code whose weight is at least m: each of three steps tries 64 codes at a time.
template <class T>
__device__ u32 last_code_of_weight(const Weigher& w, u32 top, u32 last, float m) {
  u32 lo = top, len = last - top + 1;  // code lo has it
  while (len > 1) {
    const u32 step = (len + kWave - 1) / kWave;
    const u32 c = lo + lane_id() * step;
    const u64 has = __ballot(c < lo + len && pow2(w.exponent(value_of_code<T>(c))) >= (double)m);
    const u32 at = has ? 63u - (u32)__builtin_clzll(has) : 0u;
    const u32 end = lo + len;
    lo += at * step;
    len = end - lo < step ? end - lo : step;
  }
  return lo;
}

// The three filters and the draw, in one wavefront.
template <class T>
__device__ __forceinline__ void answer_codes(CodeLds& L, const TokenArgs& a, u64 r, const RowSettings& s,
                                             const Weigher& w, u32 top, u32 last) {
  const u32 lane = lane_id();
  u64 kn = L.n[kUnits - 1], km = L.mass[kUnits - 1];  // what is kept: entries and mass
  for (int step = 0; step < 4; ++step) {  // one place where the search is inlined
    Ask ask = Ask::kMass;
    u64 Q;
    if (step == 0) {
      if (!s.k || s.k >= kn) continue;
      ask = Ask::kCount;
      Q = s.k;
    } else if (step == 1) {
      Q = (u64)ceil((double)s.p * (double)km);
      if (Q < 1 || !(s.p > 0.f)) Q = 1;
      if (s.p >= 1.f || Q >= km) continue;
    } else if (step == 2) {
      if (!(s.m > 0.f)) continue;
      ask = Ask::kCode;
      Q = last_code_of_weight<T>(w, top, last, s.m);
    } else {
      Q = (u64)((double)s.u * (double)km) + 1;
      if (Q > km) Q = km;
    }
    const CodePlace c = find_code<T>(L, w, top, last, ask, Q);
    if (step == 2 && c.n1 >= kn) continue;
    const u32 j = step == 0 ? (u32)Q - c.n0 : step == 2 ? c.n1 - c.n0 : c.entries(Q);
    if (step < 3) {
      kn = c.n0 + j;
      km = c.mass_through(j);
    } else if (lane == 0) {
      L.code = c.code;
      L.j = j;
      const double y = w.exponent(value_of_code<T>(c.code));
      a.logprobs[r] = (float)(y * 0.69314718055994530942 - log((double)km / w.scale));
    }
  }
}

template <class T, int NV>
__device__ __forceinline__ bool sample_row_by_code(CodeLds& L, const TokenArgs& a, u64 r) {
  constexpr u32 kInf = CodeOf<T>::inf;
  constexpr u32 kLowest = 0x8000u | (kInf - 1);  // the lowest number's code
  constexpr u32 kFill = (0x8000u | kInf) * 0x10001u;  // two entries of -inf
  const unsigned short* row = reinterpret_cast<const unsigned short*>(a.x) + r * a.ld;
  const u32 V = (u32)a.V;
  const RowSettings s = row_settings(a, r);
  u32 lg = 0;
  while ((1ull << lg) < a.V) ++lg;
  const int F = 62 - (int)lg < 50 ? 62 - (int)lg : 50;
  u32 head = (u32)((16 - ((uintptr_t)row & 15)) & 15) / 2;
  if (head > V) head = V;
  const u32 nvec = (V - head) / 8, tail = head + nvec * 8;
  RowVectors<NV, true> vectors;
  vectors.vec = reinterpret_cast<const u32x4*>(row + head);
  vectors.nvec = nvec;
  vectors.fill = kFill;
  if (nvec) vectors.load();
  for (u32 i = threadIdx.x; i < kCodeWords / 4; i += kThreads)
    reinterpret_cast<uint4*>(L.cnt)[i] = make_uint4(0, 0, 0, 0);
  if (threadIdx.x == 0) {
    L.top = 0xFFFFu;
    L.end = L.counted = L.matches = 0;
  }
  lds_barrier();  // the row's loads stay in flight
  // 1. count every entry that may be present: of the largest value so far, or less than
  // 2^-(F+1) below it, so that a masked row's lowest values do not queue for one counter
  u32 tops = 0xFFFFFFFFu, ends = 0, thr = 0, counted = 0;
  auto count = [&](u32 w) {  // two entries, in packed 16-bit operations as far as they go
    const u32 sign = pk_signs(w), c = w ^ (0x7FFF7FFFu & ~sign);
    tops = pk_min(tops, c);
    ends = pk_max(ends, c);
    const u32 at = pk_counter_words(c);
    const bool lo = (c & 0xFFFFu) <= thr, hi = c >> 16 <= thr;
    if (lo) atomicAdd(counter_at(L, word_bytes<0>(at)), (sign & 0xFFFFu) + 1);  // 1 or 2^16
    if (hi) atomicAdd(counter_at(L, word_bytes<1>(at)), (sign >> 16) + 1);
    counted += (u32)__builtin_popcountll(__builtin_amdgcn_ballot_w64(lo)) +
               (u32)__builtin_popcountll(__builtin_amdgcn_ballot_w64(hi));
  };
  u32 edge = kFill;  // the entries before and after the vectors: at most 7 and 7
  if (threadIdx.x < head) edge = row[threadIdx.x] | (kFill & 0xFFFF0000u);
  if (threadIdx.x < V - tail) edge = (edge & 0xFFFFu) | (u32)row[tail + threadIdx.x] << 16;
  tops = pk_codes(edge);
  if (nvec)
    vectors.first_batch([&](u32x4 v) {
      tops = pk_min(tops, pk_min(pk_min(pk_codes(v.x), pk_codes(v.y)), pk_min(pk_codes(v.z), pk_codes(v.w))));
    });
  {
    const u32 t2 = tops & 0xFFFFu, t1 = tops >> 16;
    const u32 top = wave_min(t1 < t2 ? t1 : t2);
    thr = top > kLowest ? kLowest : s.t > 0.f ? last_code<T>(top, s.t, (float)(F + 1)) : top;
  }
  if (nvec)
    vectors.template for_each<true>([&](u32x4 v, u32) {
      count(v.x);
      count(v.y);
      count(v.z);
      count(v.w);
    });
  count(edge);
  {
    const u32 t2 = tops & 0xFFFFu, t1 = tops >> 16, e2 = ends & 0xFFFFu, e1 = ends >> 16;
    const u32 t = wave_min(t1 < t2 ? t1 : t2), e = ~wave_min(~(e1 > e2 ? e1 : e2));
    if (lane_id() == 0) {
      atomicMin(&L.top, t);
      atomicMax(&L.end, e);
      atomicAdd(&L.counted, counted);  // the wavefront's
    }
  }
  lds_barrier();
  const u32 top = L.top;
  const bool nan = top < (0x7FFFu ^ kInf) || L.end > (0x8000u | kInf);
  if (nan || top > kLowest) {
    if (threadIdx.x == 0) {
      a.tokens[r] = -1;
      a.logprobs[r] = nan ? __uint_as_float(0x7FC00000u) : -__builtin_huge_valf();
    }
    return true;
  }
  if constexpr (NV == 0) {  // the last pass's first vectors, on their way meanwhile
    if (nvec) vectors.load();
  } else {
    vectors.forget();
  }
  // 2. the groups' counts and masses, then the questions
  if (s.t > 0.f) {
    Weigher w;
    w.top = value_of_code<T>(top);
    w.c = 1.4426950408889634074 / (double)s.t;
    w.scale = (double)(1ull << F);
    const u32 last = last_code<T>(top, s.t, (float)F);
    for (u32 g = threadIdx.x / kWave; g < kGroups; g += kWaves) {
      u64 m = 0;
      u32 n = 0;
      if (g >= top / kGroupCodes && g <= last / kGroupCodes) {
        const u32 c0 = g * kGroupCodes + lane_id() * kCellCodes;
        u32 cnt[kCellCodes];
        if (edge_group(g, top, last)) {
          n = cell_counters<true>(L, c0, last, cnt);
          if (__builtin_amdgcn_ballot_w64(n != 0)) m = cell_mass<T, true>(w, top, c0, cnt);
        } else {
          n = cell_counters<false>(L, c0, last, cnt);
          if (__builtin_amdgcn_ballot_w64(n != 0)) m = cell_mass<T, false>(w, top, c0, cnt);
        }
        static_assert(kUnitCodes == 4 * kCellCodes, "four lanes' cells are a unit");
        m += quad_xor<0xB1>(m);
        n += quad_xor<0xB1>(n);
        m += quad_xor<0x4E>(m);
        n += quad_xor<0x4E>(n);
      }
      if (lane_id() % 4 == 0) {
        const u32 unit = (g * kGroupCodes + lane_id() * kCellCodes) / kUnitCodes;
        L.mass[unit] = m;
        L.n[unit] = n;
      }
    }
    lds_barrier();
    {
      u64 m = L.mass[threadIdx.x];
      u32 n = L.n[threadIdx.x];
      block_scan(m, n, L.scan, L.scan_n);
      L.mass[threadIdx.x] = m;
      L.n[threadIdx.x] = n;
    }
    lds_barrier();
    // A counter may have overflowed, or entries been counted that are absent.
    if (NV != 4 && __builtin_expect(V > 0xFFFFu && L.n[kUnits - 1] != L.counted, 0)) {
      u32 n = 0;
      for (u32 i = threadIdx.x; i < kCodeWords / 4; i += kThreads) {
        const uint4 c = reinterpret_cast<const uint4*>(L.cnt)[i];
        n = __builtin_amdgcn_sad_u16(c.x, 0, n);
        n = __builtin_amdgcn_sad_u16(c.y, 0, n);
        n = __builtin_amdgcn_sad_u16(c.z, 0, n);
        n = __builtin_amdgcn_sad_u16(c.w, 0, n);
      }
      n = wave_sum(n);
      if (lane_id() == 0) L.scan[threadIdx.x / kWave] = n;
      lds_barrier();
      u32 total = 0;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) total += (u32)L.scan[i];
      const bool lost = total != L.counted;
      lds_barrier();
      if (lost) {
        return false;
      }
    }
    if (threadIdx.x < kWave) answer_codes<T>(L, a, r, s, w, top, last);
  } else if (threadIdx.x == 0) {
    L.code = top;
    L.j = 1;
    a.logprobs[r] = 0.f;
  }
  lds_barrier();
  // 3. the j-th entry of that code, by index
  const u32 code = L.code;
  const bool zero = code == 0x7FFFu || code == 0x8000u;
  const u32 j = L.j + (code == 0x8000u ? L.cnt[counter_word(0x7FFFu)] & 0xFFFFu : 0u);
  const u32 want = zero ? 0u : (code < 0x8000u ? code ^ 0x7FFFu : code) * 0x10001u;
  const u32 mask = zero ? 0x7FFF7FFFu : 0xFFFFFFFFu;
  auto match = [&](u32 i) {
    const u32 at = atomicAdd(&L.matches, 1u);
    if (at < kMatchCap) L.match[at] = i;
  };
  auto look = [&](u32 x, u32 i) {  // x: two entries, equal ones 0
    if ((x & 0xFFFFu) == 0) match(i);
    if (x < 0x10000u) match(i + 1);
  };
  if (threadIdx.x < head && (((edge ^ want) & mask) & 0xFFFFu) == 0) match(threadIdx.x);
  if (threadIdx.x < V - tail && ((edge ^ want) & mask) < 0x10000u) match(tail + threadIdx.x);
  if (nvec) {
    vectors.template for_each<NV == 0>([&](u32x4 v, u32 at) {
      const u32 x[4] = {(v.x ^ want) & mask, (v.y ^ want) & mask, (v.z ^ want) & mask, (v.w ^ want) & mask};
      const u32 least = pk_min(pk_min(x[0], x[1]), pk_min(x[2], x[3]));
      if (least < 0x10000u || (least & 0xFFFFu) == 0) {
        const u32 e = head + at * 8;
#pragma unroll
        for (u32 k = 0; k < 4; ++k) look(x[k], e + 2 * k);
      }
    });
  }
  lds_barrier();
  const u32 n = L.matches;
  if (n <= kMatchCap) {
    if (threadIdx.x < n) {
      const u32 mine = L.match[threadIdx.x];
      u32 rank = 0;
      for (u32 i = 0; i < n; ++i) rank += L.match[i] < mine;
      if (rank == j - 1) a.tokens[r] = mine;
    }
    return true;
  }
  // many of them: counts per stretch of the row, then one stretch
  const u32 per = (V + kThreads - 1) / kThreads;
  const u32 i0 = threadIdx.x * per, i1 = i0 + per < V ? i0 + per : V;
  u32 c = 0;
  for (u32 i = i0; i < i1; ++i) c += (((u32)row[i] ^ want) & mask & 0xFFFFu) == 0;
  const u64 upto = block_scan_u64(c, L.scan);
  if (upto >= j && upto - c < j) {
    u64 left = j - (upto - c);
    for (u32 i = i0; i < i1; ++i)
      if ((((u32)row[i] ^ want) & mask & 0xFFFFu) == 0 && --left == 0) {
        a.tokens[r] = i;
        break;
      }
  }
  return true;
}

// ---------------------------------------------------------------------------------------
// Rows of 32-bit logits.
//
// Almost every value differs, so each entry has its weight worked out, once: an LDS
// histogram of 4096 value bins takes the integer weights (and the entries' number where a
// top-k asks for it), and a question is answered to one bin by the bins' prefix sums and
// inside it by ranks: each of the bin's entries adds up the weights of those before it.
// Bins are cut from the 32-bit difference to the largest value, which rounds monotonously.
// Rows of up to 65536 entries stay in registers between the passes.  A row with a bin of
// more than kListed entries, with +inf, or of a temperature next to the type's largest, goes
// by the passes above that split bins.
// 256 rows of 65536: 39 us a call, 1.7 TB/s (all passes over memory, each entry's weight in
// 26 vector instructions of 64 bits and its mass and number in two additions: 82 us); of a
// workgroup's 38 us the first pass takes 8, the histogram 15, a question 4 to 5.
constexpr u32 kFloatBins = 4096;
constexpr u32 kListed = 1024;
constexpr u32 kPowers = 1024;

struct FloatLds {
  u64 mass[kFloatBins];
  u32 n[kFloatBins];
  u64 key[kListed], weight[kListed], before[kListed];
  u32 rank[kListed];
  u64 scan[kWaves];
  u32 scan_n[kWaves];
  double power[kPowers];  // 2^(F + j / kPowers)
  u64 far_mass[kWave];  // every 64th of the prefixes
  u32 far_n[kWave];
  u32 top, nan, listed[4];
  u64 minp;
  u64 ans_mass, ans_key;
};

template <int NV>
__device__ __forceinline__ bool sample_row_of_floats(FloatLds& L, const TokenArgs& a, u64 r) {
  const float* row = reinterpret_cast<const float*>(a.x) + r * a.ld;
  const u32 V = (u32)a.V;
  const RowSettings s = row_settings(a, r);
  u32 lg = 0;
  while ((1ull << lg) < a.V) ++lg;
  const int F = 62 - (int)lg < 50 ? 62 - (int)lg : 50;
  constexpr float kNone = -__builtin_huge_valf();
  u32 head = (u32)((16 - ((uintptr_t)row & 15)) & 15) / 4;
  if (head > V) head = V;
  const u32 nvec = (V - head) / 4, tail = head + nvec * 4;
  RowVectors<NV, false> vectors;
  vectors.vec = reinterpret_cast<const u32x4*>(row + head);
  vectors.nvec = nvec;
  vectors.fill = __float_as_uint(kNone);
  if (nvec) vectors.load();
  // the entries before and after the vectors, at most 3 and 3: a thread each
  u32 edge_at = threadIdx.x < head ? threadIdx.x : ~0u;
  if (threadIdx.x >= 64 && threadIdx.x - 64 < V - tail) edge_at = tail + threadIdx.x - 64;
  const float edge = edge_at != ~0u ? row[edge_at] : kNone;
  auto for_each = [&](auto load, auto f) {  // f(four values, the first one's index), each entry once
    const float e[4] = {edge, kNone, kNone, kNone};
    f(e, edge_at);
    if (nvec)
      vectors.template for_each<decltype(load)::value>([&](u32x4 v, u32 j) {
        const float x[4] = {__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w)};
        f(x, head + 4 * j);
      });
  };
  for (u32 i = threadIdx.x; i < kFloatBins; i += kThreads) {
    L.mass[i] = 0;
    L.n[i] = 0;
  }
  if (threadIdx.x == 0) {
    L.top = L.nan = 0;
    L.minp = 0;
  }
  if (threadIdx.x < 4) L.listed[threadIdx.x] = 0;
  static_assert(kPowers == (u32)kThreads, "a power each");
  L.power[threadIdx.x] = pow2((double)threadIdx.x / kPowers - 1.0, F + 1);
  lds_barrier();
  // 1. the largest value
  {
    float m = kNone;
    bool nan = false;
    for_each(std::true_type(), [&](const float (&v)[4], u32) {
      m = __builtin_fmaxf(m, __builtin_fmaxf(__builtin_fmaxf(v[0], v[1]), __builtin_fmaxf(v[2], v[3])));
      nan |= __builtin_isunordered(v[0], v[1]) || __builtin_isunordered(v[2], v[3]);
    });
    const u32 t = ~wave_min(~ord32(__float_as_uint(m)));
    if (lane_id() == 0) atomicMax(&L.top, t);
    if (nan) L.nan = 1;
  }
  if constexpr (NV == 0)
    if (nvec) vectors.load();
  lds_barrier();
  const float top = __uint_as_float(bits_of_ord32(L.top));
  if (L.nan || top == kNone) {
    if (threadIdx.x == 0) {
      a.tokens[r] = -1;
      a.logprobs[r] = L.nan ? __uint_as_float(0x7FC00000u) : kNone;
    }
    return true;
  }
  if (__builtin_expect(top == -kNone, 0)) return false;  // entries of +inf share everything
  const bool greedy = s.t == 0.f;  // the first of the entries equal to the largest
  Weigher w;
  w.top = top;
  w.c = 1.4426950408889634074 / (double)s.t;
  w.scale = (double)(1ull << F);
  const float reach_f = (float)F * 0.69314718f * s.t;  // of what is present
  // From temperatures of about 1e37 on, differences that are still present pass 32-bit floats.
  if (__builtin_expect(!(reach_f <= 3.4e38f), 0)) return false;
  const float bins = greedy ? 0.f : (float)(kFloatBins - 1) / reach_f;
  // An entry's bin; absent from kFloatBins on.  The conversion saturates and makes 0 of NaN
  // (the largest value's 0 times infinity, where the temperature is next to 0).
  auto bin_of = [&](float v, float top) -> u32 {
    u32 b;
    asm("v_cvt_u32_f32 %0, %1" : "=v"(b) : "v"((top - v) * bins));
    return b;
  };
  // An entry's weight times 2^F: y = n + j / 1024 + f, 2^(j / 1024) from the table and 2^f by
  // its series to the power 3 (|f ln 2| < 2^-11.5: the next term is below 2^-50).  The
  // histogram is bound by the vector instructions, of which 64-bit ones take twice the time
  // (65536 entries a CU: 25 us with pow2, 11 us with no weights at all).
  const double units = greedy ? 0.0 : w.c * kPowers;
  auto weight_of = [&](float v) -> double {
    const double y = ((double)v - (double)top) * units;
    const double t = y + scalar(0x1.8p52);  // the nearest integer in the low bits
    const u32 i = (u32)__builtin_bit_cast(u64, t);
    const double x = y - (t - scalar(0x1.8p52)), T = L.power[i % kPowers];
    constexpr double k = 0.69314718055994530942 / kPowers;
    const double e = __builtin_fma(x, __builtin_fma(x, scalar(k * k * k / 6), scalar(k * k / 2)), scalar(k));
    const u64 bits = __builtin_bit_cast(u64, __builtin_fma(T, x * e, T));
    const u32 high = (u32)(bits >> 32) + ((i & ~(kPowers - 1)) << 10);  // 2^n
    return __builtin_bit_cast(double, (u64)high << 32 | (u32)bits);
  };
  static_assert(kPowers == 1024, "n is i >> 10, the exponent begins at bit 20");
  // 2. the histogram: several weights at a time, for the 64-bit instructions' latency
  if (!greedy) {
    constexpr int kTogether = NV == 16 ? 2 : 4;
    if (NV) vectors.forget();
    const bool counts = s.k != 0;
    const bool has_least = s.m > 0.f;
    const double least = (double)s.m * w.scale;
    u64 minp = 0;
    for_each(std::bool_constant<NV == 0>(), [&](const float (&v)[4], u32) {
#pragma unroll
      for (int at = 0; at < 4; at += kTogether) {
        u32 b[kTogether];
        u64 q[kTogether];
        bool kept[kTogether];
#pragma unroll
        for (int k = 0; k < kTogether; ++k) {
          b[k] = bin_of(v[at + k], top);
          const double p = weight_of(v[at + k]);
          q[k] = w.whole(p);
          kept[k] = has_least && p >= least;
        }
        // all of them before the first addition, behind which a table read would queue
#pragma unroll
        for (int k = 0; k < kTogether; ++k) asm volatile("" : "+v"(q[k]));
#pragma unroll
        for (int k = 0; k < kTogether; ++k)
          if (b[k] < kFloatBins) {
            atomicAdd(&L.mass[b[k]], q[k]);
            if (counts) atomicAdd(&L.n[b[k]], 1u);
            if (has_least) minp += kept[k] ? q[k] : 0;
          }
        __builtin_amdgcn_sched_barrier(0);
      }
    });
    if (s.m > 0.f) {
      minp = wave_sum(minp);
      if (lane_id() == 0) atomicAdd(&L.minp, minp);
    }
  }
  lds_barrier();
  u64 km = 0;  // the mass that is kept
  if (!greedy) {
    constexpr u32 kEach = kFloatBins / kThreads;
    u64 m[kEach], sm = 0;
    u32 n[kEach], sn = 0;
#pragma unroll
    for (u32 i = 0; i < kEach; ++i) {
      m[i] = sm += L.mass[threadIdx.x * kEach + i];
      n[i] = sn += L.n[threadIdx.x * kEach + i];
    }
    const u64 tm = sm;
    const u32 tn = sn;
    block_scan(sm, sn, L.scan, L.scan_n);
#pragma unroll
    for (u32 i = 0; i < kEach; ++i) {
      L.mass[threadIdx.x * kEach + i] = sm - tm + m[i];
      L.n[threadIdx.x * kEach + i] = sn - tn + n[i];
    }
    if (threadIdx.x % 16 == 15) {
      L.far_mass[threadIdx.x / 16] = sm;
      L.far_n[threadIdx.x / 16] = sn;
    }
    lds_barrier();
    km = L.far_mass[kWave - 1];
  }
  // 3. the questions
  const u64 minp = L.minp, kn = greedy ? 0 : L.far_n[kWave - 1];
  for (int step = greedy ? 3 : 0; step < 4; ++step) {
    bool by_mass = !greedy;
    u64 Q;
    if (greedy) {
      Q = 1;
    } else if (step == 0) {
      if (!s.k || s.k >= kn) continue;
      by_mass = false;
      Q = s.k;
    } else if (step == 1) {
      Q = (u64)ceil((double)s.p * (double)km);
      if (Q < 1 || !(s.p > 0.f)) Q = 1;
      if (s.p >= 1.f || Q >= km) continue;
    } else if (step == 2) {
      if (s.m > 0.f && minp < km) km = minp;
      continue;
    } else {
      Q = (u64)((double)s.u * (double)km) + 1;
      if (Q > km) Q = km;
    }
    static_assert(kFloatBins == kWave * kWave, "two steps of 64");
    const u32 lane = lane_id();
    u32 b = 0;
    u64 m0 = 0, n0 = 0;
    if (!greedy) {  // the bin, by every wavefront: first 64 sixty-fourths of the bins, then one of them
      u64 reach = __builtin_amdgcn_ballot_w64(by_mass ? L.far_mass[lane] >= Q : L.far_n[lane] >= Q);
      b = reach ? (u32)__builtin_ctzll(reach) * kWave : kFloatBins - kWave;
      reach = __builtin_amdgcn_ballot_w64(lane == kWave - 1 ||
                                          (by_mass ? L.mass[b + lane] >= Q : L.n[b + lane] >= Q));
      b += (u32)__builtin_ctzll(reach);
      m0 = b ? L.mass[b - 1] : 0;
      n0 = b ? L.n[b - 1] : 0;
    }
    float here = top;  // another for the compiler, which would keep every entry's bin over the loop
    asm volatile("" : "+v"(here));
    // its entries: near its middle (more than the bin where rounding may tell), then in it
    const float middle = greedy ? top : top - ((float)b + 0.5f) / bins;
    const float near = greedy ? 0.f : 0.51f / bins + (__builtin_fabsf(top) + reach_f) * 0x1p-21f;
    vectors.begin();
    if (NV == 0 && nvec) vectors.load();
    for_each(std::bool_constant<NV == 0>(), [&](const float (&v)[4], u32 i) {
#pragma unroll
      for (u32 k = 0; k < 4; ++k)
        if (!(__builtin_fabsf(v[k] - middle) > near) && bin_of(v[k], here) == b) {
          const u32 at = atomicAdd(&L.listed[step], 1u);
          if (at < kListed) L.key[at] = make_key(__float_as_uint(v[k]), i + k);
        }
    });
    lds_barrier();
    const u32 n = L.listed[step];
    if (n > kListed) {
      return false;
    }
    if (threadIdx.x < n) {
      L.weight[threadIdx.x] = w.whole(weight_of(value_of_key(L.key[threadIdx.x])));
      L.before[threadIdx.x] = 0;
      L.rank[threadIdx.x] = 0;
    }
    lds_barrier();
    // entry i's rank and the mass before it: by 1024 / P threads each, P >= n a power of 2
    u32 P = 1;
    while (P < n) P <<= 1;
    const u32 i = threadIdx.x & (P - 1);
    if (i < n) {
      const u64 mine = L.key[i];
      u64 before = 0;
      u32 rank = 0;
      for (u32 j = threadIdx.x / P; j < n; j += kThreads / P)
        if (L.key[j] > mine) {
          before += L.weight[j];
          ++rank;
        }
      if (P == kThreads) {
        L.before[i] = before;
        L.rank[i] = rank;
      } else if (rank) {
        atomicAdd(&L.before[i], before);
        atomicAdd(&L.rank[i], rank);
      }
    }
    lds_barrier();
    if (threadIdx.x < n) {
      const u64 before = m0 + L.before[threadIdx.x], through = before + L.weight[threadIdx.x];
      if (by_mass ? through >= Q && before < Q : n0 + L.rank[threadIdx.x] + 1 == Q) {
        L.ans_mass = through;
        L.ans_key = L.key[threadIdx.x];
      }
    }
    lds_barrier();
    if (step < 3) {
      km = L.ans_mass;
      lds_barrier();
    } else if (threadIdx.x == 0) {
      const u64 key = L.ans_key;
      a.tokens[r] = (int64_t)key_index(key);
      a.logprobs[r] = greedy ? 0.f
                             : (float)(w.exponent(value_of_key(key)) * 0.69314718055994530942 -
                                       log((double)km / w.scale));
    }
  }
  return true;
}

}  // namespace

template <class T, int NV>
__global__ __launch_bounds__(kThreads) void sample_codes_kernel(TokenArgs a) {
  __shared__ union {
    CodeLds code;
    TokLds value;
  } S;
  if (__builtin_expect(sample_row_by_code<T, NV>(S.code, a, blockIdx.x), 1)) return;
  if constexpr (NV != 4) {
    __syncthreads();
    sample_row_by_value<T>(S.value, a, blockIdx.x);
  }
}

template <int NV>
__global__ __launch_bounds__(kThreads) void sample_floats_kernel(TokenArgs a) {
  __shared__ union {
    FloatLds bins;
    TokLds value;
  } S;
  if (__builtin_expect(sample_row_of_floats<NV>(S.bins, a, blockIdx.x), 1)) return;
  __syncthreads();
  sample_row_by_value<float>(S.value, a, blockIdx.x);
}

static void launch_floats(const TokenArgs& a, hipStream_t s) {
  const u32 B = (u32)a.B;
  const u64 vectors = (a.V + 3) / 4;
  if (vectors <= 4 * kThreads)
    sample_floats_kernel<4><<<B, kThreads, 0, s>>>(a);
  else if (vectors <= 8 * kThreads)
    sample_floats_kernel<8><<<B, kThreads, 0, s>>>(a);
  else if (vectors <= 16 * kThreads)
    sample_floats_kernel<16><<<B, kThreads, 0, s>>>(a);
  else
    sample_floats_kernel<0><<<B, kThreads, 0, s>>>(a);
}

template <class T>
static void launch_codes(const TokenArgs& a, hipStream_t s) {
  const u32 B = (u32)a.B;
  const u64 vectors = (a.V + 7) / 8;
  if (vectors <= 4 * kThreads)
    sample_codes_kernel<T, 4><<<B, kThreads, 0, s>>>(a);
  else if (vectors <= 8 * kThreads)
    sample_codes_kernel<T, 8><<<B, kThreads, 0, s>>>(a);
  else if (vectors <= 16 * kThreads)
    sample_codes_kernel<T, 16><<<B, kThreads, 0, s>>>(a);
  else
    sample_codes_kernel<T, 0><<<B, kThreads, 0, s>>>(a);
}

// A workgroup a row, and a grid has fewer than 2^32 threads: longer batches go in parts.
hipError_t launch_sample_tokens(const TokenArgs& a, int dtype, hipStream_t s) {
  constexpr u64 kMostRows = (1ull << 32) / kThreads - 1;
  const u64 size = dtype == PROFK_FP32 ? 4 : 2;
  for (u64 r = 0; r < a.B; r += kMostRows) {
    TokenArgs part = a;
    part.B = a.B - r < kMostRows ? a.B - r : kMostRows;
    part.x = reinterpret_cast<const char*>(a.x) + r * a.ld * size;
    part.u += r;
    if (a.t_row) part.t_row += r;
    if (a.p_row) part.p_row += r;
    if (a.m_row) part.m_row += r;
    if (a.k_row) part.k_row += r;
    part.tokens += r;
    part.logprobs += r;
    if (dtype == PROFK_FP32)
      launch_floats(part, s);
    else if (dtype == PROFK_FP16)
      launch_codes<Half16>(part, s);
    else
      launch_codes<Brain16>(part, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace profk
