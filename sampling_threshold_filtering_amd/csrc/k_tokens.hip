// Sampling a token from each row of logits, with temperature, top-k, top-p and min-p,
// from a given uniform number per row.
//
// Mathematics.  Order a row's entries by value, descending, ties by lower index.  With
// w_i = exp((l_i - max) / T), every filter keeps a prefix of that order:
//   K = the first top_k entries;  P = the shortest prefix of K with mass >= top_p mass(K);
//   F = the entries of P with w_i >= min_p;  W = mass(F).
// The token is the first entry of the order whose cumulative mass exceeds u W.  So the
// whole operator is a few questions of one kind, "where does the running count, or the
// running mass, of the order first reach Q?", and no row is ever sorted: a histogram over
// value bins answers a question up to one bin, whose entries are then collected and
// sorted in LDS (a bin too full for that is split into finer bins by key first).
//
// Exactness.  Weights are integers q_i = round(w_i 2^F), with F as large as lets a row's
// sum fit 63 bits (F = 46 at 2^17 entries), from exp2 in 64 bits.  Integer sums do not
// depend on their order, so LDS atomics and any split of the row give the same bits, and
// the rounding of a weight (2^-(F+1) of the largest) is far below what a 24-bit u can
// tell apart.  An entry below 2^-F of the largest counts as absent.
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

// Inclusive scan over the block, one u64 per thread.
__device__ __forceinline__ u64 block_scan_u64(u64 v, u64* wave_tot) {
  const u32 lane = lane_id(), wid = threadIdx.x / kWave;
#pragma unroll
  for (u32 d = 1; d < (u32)kWave; d <<= 1) {
    const u64 o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  if (lane == kWave - 1) wave_tot[wid] = v;
  __syncthreads();
  u64 before = 0;
  for (u32 w = 0; w < wid; ++w) before += wave_tot[w];
  __syncthreads();
  return v + before;
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
  __device__ __forceinline__ u64 weight(double y) const { return (u64)rint(exp2(y) * scale); }
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
__device__ inline void sort_and_weigh(TokLds& L, u32 n, const Weigher& w) {
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
__device__ inline Prefix find_in_list(TokLds& L, u32 n, u64 n0, u64 m0, bool by_mass, u64 Q) {
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
__device__ inline u32 collect(TokLds& L, const T* row, u32 V, const Weigher& w, F pick) {
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
__device__ inline void value_histogram(TokLds& L, const T* row, u32 V, const Weigher& w, float min_p) {
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
    const double e = exp2(y);
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
__device__ Prefix resolve(TokLds& L, const T* row, u32 V, const Weigher& w, bool by_mass, u64 Q, bool want_key,
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

}  // namespace

template <class T>
__global__ __launch_bounds__(kThreads) void sample_tokens_kernel(TokenArgs a) {
  __shared__ TokLds L;
  const u64 r = blockIdx.x;
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
  bool lost = false;
  auto ask = [&](bool by_mass, u64 Q, bool want_key) {
    if (lost) {
      value_histogram(L, row, V, w, 0.f);
      lost = false;
    }
    return resolve(L, row, V, w, by_mass, Q, want_key, lost);
  };
  Prefix keep = {N, Z, 0};
  if (s.k && s.k < N) keep = ask(false, s.k, false);
  if (s.p < 1.f) {
    u64 Q = (u64)ceil((double)s.p * (double)keep.mass);
    if (Q < 1 || !(s.p > 0.f)) Q = 1;
    if (Q < keep.mass) keep = ask(true, Q, false);
  }
  if (s.m > 0.f && mn < keep.n) keep = {mn, mm, 0};
  u64 Q = (u64)((double)s.u * (double)keep.mass) + 1;
  if (Q > keep.mass) Q = keep.mass;
  const Prefix at = ask(true, Q, true);
  if (threadIdx.x == 0) {
    const double y = w.exponent(value_of_key(at.key));
    a.tokens[r] = (int64_t)key_index(at.key);
    a.logprobs[r] = (float)(y * 0.69314718055994530942 - log((double)keep.mass / w.scale));
  }
}

size_t sample_tokens_scratch_bytes(u64, u64) { return 0; }

hipError_t launch_sample_tokens(const TokenArgs& a, int dtype, hipStream_t s) {
  if (dtype == PROFK_FP32)
    sample_tokens_kernel<float><<<(u32)a.B, kThreads, 0, s>>>(a);
  else if (dtype == PROFK_FP16)
    sample_tokens_kernel<Half16><<<(u32)a.B, kThreads, 0, s>>>(a);
  else
    sample_tokens_kernel<Brain16><<<(u32)a.B, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace profk
