// Routing tokens to experts by scores: softmax or sigmoid, a bias per expert, groups, a scale.
//
// Mathematics, for logits l[T, E] (rows: the live ones, as in k_route.hip):
//   s_t = softmax(l_t), or s_te = 1 / (1 + exp(-l_te));  choice score c_te = s_te + b_e
//   (experts of a logit or a bias of -inf: none);  a group's score is the sum of its one or
//   two largest c;  of the top_groups best groups, ties by lower index, the first k experts by
//   c, ties by lower index;  gate weights: scale times s, or s over the chosen ones' sum
//   p_t = s_t / sum_e s_te;  counts and loss from the choice and p as in k_route.hip
// The choice is that of c in 64 bits.  The gradient is k_route.hip's.
//
// The choice goes by keys of 32 bits, as in k_route.hip: c in units of (its possible range) /
// 2^24, from the lowest bias up, above the entry's complement.  c in 32 bits is off by up to
// some units, so where two neighbours among the first k + 1 keys are within that error of each
// other, the wavefront ranks those that may be among the first k in 64 bits, a lane each; where
// the worst group kept and the best left out are, it scores the groups that near in 64 bits; and
// rows with NaN, or with more near ties than lanes, it chooses again whole.  A fixed point rather
// than the float's own bits: beside the index a float keeps 15 of its 24 at 256 experts.
//
// Bound by vector instructions: 65536 x 256 bf16, sigmoid, bias, 4 of 8 groups, k = 8 with the loss
// takes 54 us (74 % of the busy cycles; 33 MB of logits) and 5 for the joining launch, and the
// gradient 23 (78 %); the plain routing of that size 24, 5 and 21.  What it has on top: the keys'
// bias from LDS and groups' two best through LDS, a third of the cycles (half of those bank
// conflicts), and the 64-bit paths, some 9 us: less by the rows that take them, one in a thousand
// there, than by standing in the rows' loop.  They take 108 to 142 vector registers, so four
// wavefronts a SIMD fit, and 68 to 87 scalar registers live in lanes of vector ones; 16 entries a
// lane spill up to 9 vector registers.  8 x 256 fp32 11.3 us, one row's chain.
#include "route_device.h"

namespace profk {

namespace {

constexpr int kScoredThreads = 512;
constexpr int kScoredWaves = kScoredThreads / kWave;
static_assert(kScoredWaves >= (int)kLeastRows, "the scratch holds a block's sums for each of so many rows");

// Ordered codes of 64-bit floats: NaN above all, -0 as +0; 0: none.
__device__ __forceinline__ u64 code_of(double c) {
  if (c != c) return ~0ull;
  const u64 b = __builtin_bit_cast(u64, c + 0.0);
  return b ^ ((u64)((int64_t)b >> 63) | 1ull << 63);
}
__device__ __forceinline__ double of_code(u64 u) {
  if (u == ~0ull) return __builtin_nan("");
  return __builtin_bit_cast(double, u >> 63 ? u ^ 1ull << 63 : ~u);
}
__device__ __forceinline__ u32 wave_max(u32 v) { return wave_reduce_u32(v, max_u); }
__device__ __forceinline__ u64 wave_max(u64 v) {  // the upper halves, then the lower ones of those that have it
  const u32 high = wave_max((u32)(v >> 32));
  return (u64)high << 32 | wave_max((u32)(v >> 32) == high ? (u32)v : 0u);
}
__device__ __forceinline__ u32 wave_min(u32 v) {
  return ~wave_max(~v);
}

// A constant in scalar registers, made where it is used: held in vector registers over the rows'
// loop, the few dozen of the 64-bit choice took a third of the loop's.
__device__ __forceinline__ double in_scalar(double v) {
  asm volatile("" : "+s"(v));
  return v;
}

// e^x: x = n ln 2 + f with |f| <= ln 2 / 2, the Taylor series of e^f to the power 13 (the next
// term is below 2^-57), scaled by 2^n.  NaN stays.
__device__ __forceinline__ double exp_64(double x) {
  const double y = __builtin_fmin(__builtin_fmax(x, in_scalar(-800.0)), in_scalar(800.0));
  const double n = rint(y * in_scalar(1.4426950408889634));
  // ln 2 in two parts, the first with room for n's bits
  double f = __builtin_fma(-n, in_scalar(0x1.62e42fefap-1), y);
  f = __builtin_fma(-n, in_scalar(0x1.cf79abc9e3b3ap-40), f);
  double p = in_scalar(1.0 / 6227020800.0);
  p = __builtin_fma(p, f, in_scalar(1.0 / 479001600));
  p = __builtin_fma(p, f, in_scalar(1.0 / 39916800));
  p = __builtin_fma(p, f, in_scalar(1.0 / 3628800));
  p = __builtin_fma(p, f, in_scalar(1.0 / 362880));
  p = __builtin_fma(p, f, in_scalar(1.0 / 40320));
  p = __builtin_fma(p, f, in_scalar(1.0 / 5040));
  p = __builtin_fma(p, f, in_scalar(1.0 / 720));
  p = __builtin_fma(p, f, in_scalar(1.0 / 120));
  p = __builtin_fma(p, f, in_scalar(1.0 / 24));
  p = __builtin_fma(p, f, in_scalar(1.0 / 6));
  p = __builtin_fma(p, f, 0.5);
  p = __builtin_fma(p, f, 1.0);
  p = __builtin_fma(p, f, 1.0);
  return x != x ? x : __builtin_ldexp(p, (int)n);
}

// What the wavefront's rows need of the choice: the keys in LDS, row by row.
template <int G, int C>
struct Choice {
  static constexpr int kBits = key_bits(G * C);
  static constexpr u32 kLow = (1u << kBits) - 1;
  static constexpr int kUnits = 32 - kBits < 24 ? 32 - kBits : 24;  // bits of c
  static constexpr u32 kMostGroups = G * C < (int)kRouteMaxGroups ? G * C : kRouteMaxGroups;
};

// A row's values in LDS, by entry.
template <bool QUAD, int G, int C, class V>
__device__ __forceinline__ void to_lds(V* row, u32 g, const V (&v)[C]) {
  if constexpr (QUAD) {
#pragma unroll
    for (int i = 0; i < C; i += 4)
      *reinterpret_cast<Four<V>*>(row + Row<G, C, QUAD>::index(i, g)) = Four<V>{{v[i], v[i + 1], v[i + 2], v[i + 3]}};
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i) row[Row<G, C, QUAD>::index(i, g)] = v[i];
  }
}
template <bool QUAD, int G, int C, class V>
__device__ __forceinline__ void from_lds(const V* row, u32 g, V (&v)[C]) {
  if constexpr (QUAD) {
#pragma unroll
    for (int i = 0; i < C; i += 4) {
      const Four<V> q = *reinterpret_cast<const Four<V>*>(row + Row<G, C, QUAD>::index(i, g));
#pragma unroll
      for (int k = 0; k < 4; ++k) v[i + k] = q.e[k];
    }
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = row[Row<G, C, QUAD>::index(i, g)];
  }
}

}  // namespace

// The kernel's arguments, read again: held in scalar registers over the rows' loop, those that
// only the 64-bit choice needs would drive others out of them.
__device__ __forceinline__ const RouteArgs& arguments_again() {
  typedef const __attribute__((address_space(4))) RouteArgs* Constant;
  Constant p = (Constant)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const RouteArgs*)p;
}

// The sum of a row's softmax in 64 bits, by the whole wavefront; top is the row's largest logit
// (NaN or +inf make every score NaN).
template <class T>
__device__ __forceinline__ double softmax_sum(const RouteArgs& a, const T* x, float top) {
  double sum = 0;
#pragma unroll 1
  for (u32 e = lane_id(); e < a.E; e += kWave) sum += exp_64((double)to_f32(x[e]) - (double)top);
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) sum += __shfl_xor(sum, d);
  return sum;
}

// The code of the choice score of an entry of logit l and bias b; 0: none.  (A bias of -inf is asked
// for by itself: beside a score of NaN the sum does not show it.)
__device__ __forceinline__ u64 choice_code(const RouteArgs& a, float l, float b, float top, double sum) {
  const double s = a.sigmoid ? 1.0 / (1.0 + exp_64(-(double)l)) : exp_64((double)l - (double)top) / sum;
  const double c = a.bias ? s + (double)b : s;
  return l == kNone || b == kNone ? 0 : code_of(c);
}

// The first keys of a row, `n` of them and among them its k experts, in the order of 64 bits:
// lane j has the j-th key's expert and gets its rank.
template <class T>
__device__ __forceinline__ u32 rank_exactly(const RouteArgs& a, u64 row, u32 n, u32 e, float top) {
  const T* x = reinterpret_cast<const T*>(a.x) + row * a.ld;
  const bool mine = lane_id() < n;
  const float l = mine ? to_f32(x[e]) : kNone, b = mine && a.bias ? a.bias[e] : 0.f;
  const u64 code = choice_code(a, l, b, top, a.sigmoid ? 1.0 : softmax_sum(a, x, top));
  u32 rank = 0;
#pragma unroll 1
  for (u32 j = 0; j < n; ++j) {
    const u64 o = (u64)(u32)__builtin_amdgcn_readlane((int)(code >> 32), (int)j) << 32 |
                  (u32)__builtin_amdgcn_readlane((int)code, (int)j);
    const u32 f = (u32)__builtin_amdgcn_readlane((int)e, (int)j);
    rank += o > code || (o == code && f < e);
  }
  return rank;
}

// The code of group q's score, by the whole wavefront.
template <class T>
__device__ __forceinline__ u64 group_code(const RouteArgs& a, const T* x, u32 q, u32 size, float top, double sum) {
  u64 first = 0, second = 0;
#pragma unroll 1
  for (u32 j = lane_id(); j < size; j += kWave) {
    const u32 e = q * size + j;
    const u64 c = choice_code(a, to_f32(x[e]), a.bias ? a.bias[e] : 0.f, top, sum), low = c < first ? c : first;
    second = low > second ? low : second;
    first = c > first ? c : first;
  }
  const u64 best = wave_max(first);
  if (a.group_best != 2) return best;
  const u64 holders = __ballot(first == best);
  second = holders & (holders - 1) ? best : wave_max(first == best ? second : first);
  return second ? code_of(of_code(best) + of_code(second)) : best;
}

// One row by the whole wavefront in 64 bits: lane j gets slot j's expert, or ~0.  `codes` has
// room for E.  No array of it lives in registers: the rows that come here are few, and the
// others' loop keeps its registers.
template <class T>
__device__ __forceinline__ u32 choose_exactly(const RouteArgs& a, u64 row, float top, u64* codes) {
  const T* x = reinterpret_cast<const T*>(a.x) + row * a.ld;
  const u32 lane = lane_id(), E = a.E;
  const double sum = a.sigmoid ? 1.0 : softmax_sum(a, x, top);
#pragma unroll 1
  for (u32 e = lane; e < E; e += kWave) codes[e] = choice_code(a, to_f32(x[e]), a.bias ? a.bias[e] : 0.f, top, sum);
  wave_lds_sync();
  if (a.top_groups < a.groups) {
    const u32 size = E / a.groups;
    u64 mine = 0;  // lane g: group g's score
#pragma unroll 1
    for (u32 g = 0; g < a.groups; ++g) {
      const u64 c = group_code(a, x, g, size, top, sum);
      if (lane == g) mine = c;
    }
    u32 before = 0;
#pragma unroll 1
    for (u32 g = 0; g < a.groups; ++g) {
      const u64 o = __shfl(mine, (int)g);
      before += o > mine || (o == mine && g < lane);
    }
    const u64 kept = __ballot(lane < a.groups && before < a.top_groups);
#pragma unroll 1
    for (u32 e = lane; e < E; e += kWave)
      if (!(kept >> (e / size) & 1)) codes[e] = 0;
    wave_lds_sync();
  }
  u32 slot = ~0u;
  static_assert(kRouteMaxK <= kWave, "a lane per slot");
#pragma unroll 1
  for (u32 j = 0; j < a.k; ++j) {
    u64 first = 0;
    u32 at = ~0u;
#pragma unroll 1
    for (u32 e = lane; e < E; e += kWave) {
      const u64 c = codes[e];
      if (c > first) {
        first = c;
        at = e;
      }
    }
    const u64 top = wave_max(first);
    if (!top) break;
    at = wave_min(first == top ? at : ~0u);
    if (lane == j) slot = at;
    if (lane == at % kWave) codes[at] = 0;
    wave_lds_sync();
  }
  return slot;
}

template <class T, int G, int C, bool QUAD, bool SIGMOID>
__global__ __launch_bounds__(kScoredThreads, 4) void scored_kernel(RouteArgs args) {
  const RouteArgs& a = args;  // up to the rows' loop
  using R = Row<G, C, QUAD>;
  using K = Choice<G, C>;
  constexpr int kGroups = kScoredThreads / G, kRows = kWave / G;  // rows of a block, of a wavefront
  // the rows' keys and, for the rows chosen in 64 bits, one row's codes
  __shared__ alignas(16) u32 s_key[kScoredWaves][kRows > 1 ? kRows : 2][G * C];
  __shared__ u32 s_group[kScoredWaves][kRows][K::kMostGroups];
  __shared__ u32 s_cnt[G * C];
  __shared__ alignas(16) float s_base[G * C];  // the biases in units from the lowest; -inf: none
  // each lane's sums of probabilities, four experts together; while they are joined, the wavefront's
  __shared__ alignas(16) float s_sum[kScoredWaves][kWave * C];
  __shared__ u32 s_rows;
  __shared__ double s_part[kScoredWaves];
  static_assert(G * C <= 2 * kScoredThreads, "two experts a thread");
  const u32 g = threadIdx.x % G, grp = threadIdx.x / G, wave = threadIdx.x / kWave, row_of_wave = lane_id() / G;
  for (u32 e = threadIdx.x; e < G * C; e += kScoredThreads) s_cnt[e] = 0;
  if (threadIdx.x == 0) s_rows = 0;
  u32* key_row = s_key[wave][row_of_wave];
  u32* group_row = s_group[wave][row_of_wave];
  const T* x = reinterpret_cast<const T*>(a.x);
  const u64 step = (u64)gridDim.x * kGroups;
  // A row's loads go out a turn ahead: with four wavefronts a SIMD the others do not cover them.
  typename R::template Raw<T> raw;
  bool masked = true;
  auto fetch = [&](u64 t0) {
    const RouteArgs& a = arguments_again();
    const u64 t = t0 + grp, tr = t < a.T ? t : a.T - 1;
    masked = a.mask && !a.mask[tr];
    R::fetch(reinterpret_cast<const T*>(a.x) + tr * a.ld, a.E, g, raw);
  };
  u64 t0 = (u64)blockIdx.x * kGroups;
  if (t0 < a.T) fetch(t0);
  float low = a.bias ? __builtin_huge_valf() : 0.f, high = a.bias ? -__builtin_huge_valf() : 0.f;
  bool odd = false;  // a bias that the keys cannot hold
#pragma unroll 1
  for (u32 e = lane_id(); e < a.E; e += kWave) {
    const float b = a.bias ? a.bias[e] : 0.f;
    odd |= b != b || b == __builtin_huge_valf();
    if (b > kNone && b < __builtin_huge_valf()) {
      low = __builtin_fminf(low, b);
      high = __builtin_fmaxf(high, b);
    }
  }
  low = -group_reduce<kWave>(-low, max_f);
  high = group_reduce<kWave>(high, max_f);
  if (!(low <= high)) low = high = 0.f;
  odd = __ballot(odd) != 0;
  // a unit: the range of c over 2^kUnits, less room for roundings at both ends
  const float unit = (float)(((double)(1u << K::kUnits) - 64.0) / ((double)high - (double)low + 1.0));
  for (u32 e = threadIdx.x; e < G * C; e += kScoredThreads) {
    const float b = e >= a.E ? kNone : a.bias ? a.bias[e] : 0.f;
    s_base[e] = b == kNone ? kNone : (float)(((double)b - (double)low) * (double)unit + 32.0);
  }
  __syncthreads();
  const u32 size = a.E / a.groups;
  const bool grouped = a.top_groups < a.groups;
  const u32 best = a.group_best < size ? a.group_best : size;
  u32 lanes_log = 0;  // lanes per group of experts
  while ((2u << lanes_log) * a.groups <= (u32)G) ++lanes_log;
  const u32 lanes = 1u << lanes_log, part = g & (lanes - 1);

  u32 rows = 0;
  // The lane's sums live in LDS: in registers they would take 16 of 128, and the row's choice spill.
  Four<float>* sums = reinterpret_cast<Four<float>*>(s_sum[wave]) + lane_id();
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < C / 4; ++i) sums[i * kWave] = Four<float>{{0.f, 0.f, 0.f, 0.f}};
  };
  clear();
  double total[2] = {0, 0};  // of experts threadIdx.x and threadIdx.x + kScoredThreads
  auto join = [&]() {
    float v[C];
#pragma unroll
    for (int i = 0; i < C; i += 4) {
      const Four<float> q = sums[i / 4 * kWave];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[i + k] = q.e[k];
    }
    wave_lds_sync();
#pragma unroll
    for (int i = 0; i < C; ++i) {
#pragma unroll
      for (int d = G; d < kWave; d <<= 1) v[i] += __shfl_xor(v[i], d);
      if (lane_id() < G) s_sum[wave][R::index(i, g)] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u32 e = threadIdx.x + h * kScoredThreads;
      if (e < arguments_again().E)
#pragma unroll
        for (int w = 0; w < kScoredWaves; ++w) total[h] += (double)s_sum[w][e];
    }
  };
  u32 turn = 0;
  for (; t0 < arguments_again().T; t0 += step) {
    const RouteArgs& a = arguments_again();
    const u64 t = t0 + grp;
    const bool here = t < a.T, in = here && !masked;
    const T* xt = x + (here ? t : a.T - 1) * a.ld;
    R row;
    row.take(raw, a.E, g, in);
    if (t0 + step < a.T) fetch(t0 + step);
    // entries of -inf, a bit each: the logits themselves do not stay in registers
    u32 none = 0;
    float least_logit = row.v[0];
#pragma unroll
    for (int i = 1; i < C; ++i) least_logit = __builtin_fminf(least_logit, row.v[i]);
    const bool nones = __ballot(least_logit == kNone) != 0;
    if (nones) {
#pragma unroll
      for (int i = 0; i < C; ++i) none |= (u32)(row.v[i] == kNone) << i;
    }
    bool nan = false;
    if constexpr (SIGMOID) {
      float unused[1];
      row.score(in, nan, unused);
    } else {
      row.weigh(in);
      nan = !(row.top < __builtin_huge_valf());
    }
    const float inv = row.template inverse<SIGMOID>();
    if (a.loss) {
#pragma unroll
      for (int i = 0; i < C; i += 4) {
        Four<float> q = sums[i / 4 * kWave];
#pragma unroll
        for (int k = 0; k < 4; ++k) q.e[k] = __builtin_fmaf(row.e[i + k], inv, q.e[k]);
        sums[i / 4 * kWave] = q;
      }
    }
    rows += row.live && g == 0;
    // keys
    u32 key[C];
    // (beside a bias a row of far scores has none: 2^-30 of it, 1/64 of a unit)
    const float per = !SIGMOID ? unit * inv : row.far ? 0.f : unit;
    float base[C];
    const u32 low = opaque_u32(K::kLow - R::index(0, g));  // of entry 0; here, so that 16 of them do not stay in registers
    from_lds<QUAD, G, C>(s_base, g, base);
    if (nones) {
#pragma unroll
      for (int i = 0; i < C; ++i) base[i] = none >> i & 1 ? kNone : base[i];
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const float u = __builtin_fmaf(row.e[i], per, base[i]);  // of an entry that is none -inf: converts to 0
      key[i] = (u32)__builtin_fmaxf(u, 0.f) << K::kBits | (low - R::index(i, 0));
    }
    auto same = [&](u32 m, u32 n) {  // the entries of two keys
      const RouteArgs& a = arguments_again();
      const u32 e = K::kLow - (m & K::kLow), f = K::kLow - (n & K::kLow);
      return to_f32(xt[e]) == to_f32(xt[f]) && (!a.bias || a.bias[e] == a.bias[f]);
    };
    // How far two keys may be off each other, in units.  A sigmoid is off by 5 h of 1 at most (h =
    // 2^-24: half of its exponential's 4 h, the sum's h, the reciprocal's 2 h), which is 5 units at
    // most; a probability by (32 + 2 |d|) h of itself, below 64 h of the row's largest; the product's
    // and the bias's rounding by half a unit each, the cut by one.
    const u32 near = SIGMOID ? 15 : 5 + (u32)(__builtin_fminf(unit * inv, 0x1p24f) * 0x1p-17f);
    const u32 close = near << K::kBits | K::kLow;  // in keys
    bool unsure = odd || group_reduce<G>((u32)nan, max_u) != 0;
    if (grouped) {
      const RouteArgs& a = arguments_again();
      to_lds<QUAD, G, C>(key_row, g, key);
      wave_lds_sync();
      // A lane's groups: their two largest keys, then their scores: one key, or a sum of two values.
      for (u32 q = g >> lanes_log; q < a.groups; q += (u32)G >> lanes_log) {
        u32 first = 0, second = 0;
        auto take = [&](u32 u) {
          second = max_u(second, first < u ? first : u);
          first = max_u(first, u);
        };
        if (QUAD && size % 4 == 0) {
          for (u32 j = part * 4; j < size; j += lanes * 4) {
            const uint4 u = *reinterpret_cast<const uint4*>(key_row + q * size + j);
            take(u.x);
            take(u.y);
            take(u.z);
            take(u.w);
          }
        } else {
#pragma unroll 4
          for (u32 j = part; j < size; j += lanes) take(key_row[q * size + j]);
        }
        for (u32 d = 1; d < lanes; d <<= 1) {
          const u32 f = __shfl_xor(first, (int)d), s = __shfl_xor(second, (int)d);
          second = max_u(max_u(second, s), first < f ? first : f);
          first = max_u(first, f);
        }
        if (first <= K::kLow) first = 0;
        if (best == 2) {
          unsure |= first && second <= K::kLow;  // one score against sums of two
          first = (first >> K::kBits) + (second >> K::kBits);
        }
        if (part == 0) group_row[q] = first;
      }
      wave_lds_sync();
      u32 least = ~0u, most = 0;  // of the groups kept, of those left out
      u32 kept = 0, turn_of = 1;  // a bit for each of the lane's groups
      for (u32 q = g >> lanes_log; q < a.groups; q += (u32)G >> lanes_log, turn_of <<= 1) {
        const u32 own = group_row[q];
        u32 before = 0;
#pragma unroll 4
        for (u32 h = 0; h < a.groups; ++h) {
          const u32 o = group_row[h];
          before += o > own || (o == own && h < q);
        }
        if (before < a.top_groups) {
          least = least < own ? least : own;
          kept |= turn_of;
        } else {
          most = max_u(most, own);
        }
      }
      least = ~group_reduce<G>(~least, max_u);
      most = group_reduce<G>(most, max_u);
      // Groups whose order against the border rounding may have changed.
      const u32 margin = best == 2 ? 2 * near : close;
      bool border = most && least - most <= margin && row.live && !unsure;
      if (best == 1 && border) {
        // Of the same best logit and bias they are told apart by their index in any arithmetic: so are
        // these if whatever may be the best of one of them is the same.
        border = false;
        turn_of = 1;
        for (u32 q = g >> lanes_log; q < a.groups; q += (u32)G >> lanes_log, turn_of <<= 1) {
          const u32 own = group_row[q];
          if (!own || (kept & turn_of ? own - most : least - own) > margin) continue;
          for (u32 j = part; j < size; j += lanes) {
            const u32 u = key_row[q * size + j];
            border |= u > K::kLow && (u > most || most - u <= 2 * margin) && !same(u, most);
          }
        }
      }
      border = group_reduce<G>((u32)border, max_u) != 0;
      for (u64 left = __ballot(border && g == 0); left; left &= left - 1) {
        // as many of them are kept as were, by their scores in 64 bits; lane f has the f-th of them
        const RouteArgs& b = arguments_again();
        const u32 from = (u32)__builtin_ctzll(left), lane = lane_id(), per = (u32)G >> lanes_log;
        const bool own_row = lane / G == from / G;
        const T* xr = reinterpret_cast<const T*>(b.x) + (t0 + wave * kRows + from / G) * b.ld;
        const float top = __shfl(row.top, (int)from);
        const double sum = b.sigmoid ? 1.0 : softmax_sum(b, xr, top);
        u64 code = 0;
        u32 group = 0, count = 0, keep = 0;
        turn_of = 1;
        for (u32 q0 = 0; q0 < b.groups; q0 += per, turn_of <<= 1) {
          const u32 q = q0 + (g >> lanes_log), own = q < b.groups ? group_row[q] : 0;
          const bool was = kept & turn_of;
          for (u64 near_ones = __ballot(own_row && part == 0 && own && (was ? own - most : least - own) <= margin); near_ones;
               near_ones &= near_ones - 1) {
            const u32 l = (u32)__builtin_ctzll(near_ones), it = q0 + ((l - from) >> lanes_log);
            const u64 c = group_code(b, xr, it, size, top, sum);
            if (lane == count) {
              code = c;
              group = it;
            }
            ++count;
            keep += (u32)__builtin_amdgcn_readlane((int)was, (int)l) != 0;
          }
        }
        u32 rank = 0;
        for (u32 f = 0; f < count; ++f) {
          const u64 o = (u64)(u32)__builtin_amdgcn_readlane((int)(code >> 32), (int)f) << 32 |
                        (u32)__builtin_amdgcn_readlane((int)code, (int)f);
          rank += o > code || (o == code && f < lane);  // (lane f's group comes before lane f + 1's)
        }
        for (u32 f = 0; f < count; ++f) {
          const u32 it = (u32)__builtin_amdgcn_readlane((int)group, (int)f);
          const u32 bit = 1u << it / per;
          if (own_row && it % per == g >> lanes_log)
            kept = (u32)__builtin_amdgcn_readlane((int)rank, (int)f) < keep ? kept | bit : kept & ~bit;
        }
      }
      turn_of = 1;
      for (u32 q = g >> lanes_log; q < a.groups; q += (u32)G >> lanes_log, turn_of <<= 1)
        if (!(kept & turn_of))
          for (u32 j = part; j < size; j += lanes) key_row[q * size + j] = K::kLow - (q * size + j);
      wave_lds_sync();
      from_lds<QUAD, G, C>(key_row, g, key);
      wave_lds_sync();
    }
    // the first k keys, and the next: lane g holds slots g, g + G, ... of them
    bool closes = false;
    u32 m = key[0], mine = 0;
#pragma unroll
    for (int i = 1; i < C; ++i) m = max_u(m, key[i]);
    m = group_reduce<G>(m, max_u);
    const u32 slots = arguments_again().k, last_slot = slots - 1, experts = arguments_again().E;
    for (u32 j = 0;; ++j) {
      if (g == j % G) mine = m;
      if (j % G == G - 1 || j == last_slot) {
        if (slots > (u32)G && g <= j % G) key_row[j / G * G + g] = mine;
      }
      if (j + 1 == experts) break;
      u32 d = 0;
#pragma unroll
      for (int i = 0; i < C; ++i) d = max_u(d, key[i] - m);
      const u32 n = m + group_reduce<G>(d, max_u);
      closes |= n > K::kLow && m - n <= close;
      if (j == last_slot) break;
      m = n;
    }
    wave_lds_sync();
    unsure = group_reduce<G>((u32)unsure, max_u) && row.live;
    closes = closes && !unsure && row.live;
    if (__builtin_expect(__ballot(closes) != 0, 0)) {
      // Whatever may be among the first k: the keys down to as far below the k-th as two may be off
      // each other.  The wavefront ranks them in 64 bits, a lane each.
      // (m is the k-th.)  Many of one logit and bias, as of a router that starts at zero, are told
      // apart by their index in any arithmetic, and are not gone through one by one.
      u32 these = 0;
      if (closes && m > K::kLow) {
#pragma unroll
        for (int i = 0; i < C; ++i) these |= (u32)(key[i] > K::kLow && (key[i] >= m || m - key[i] <= close)) << i;
      }
      if (group_reduce<G>((u32)__popc(these), [](u32 p, u32 q) { return p + q; }) > slots + 8) {
        bool others = false;
        for (; these && !others; these &= these - 1) others = !same(m, K::kLow - R::index(__builtin_ctz(these), g));
        closes = group_reduce<G>((u32)others, max_u) != 0;
      }
      u32 last = 0, border = 0, some = 0;
      bool differ = false;  // neighbours of the same logit and bias go by their index in any arithmetic
      for (u32 j = 0; j < (u32)kWave && j < experts; ++j) {
        u32 d = 0;
#pragma unroll
        for (int i = 0; i < C; ++i) d = max_u(d, key[i] - last);
        const u32 n = last + group_reduce<G>(d, max_u);
        const bool takes = closes && some == j && n > K::kLow && (j <= last_slot || border - n <= close);
        if (__ballot(takes) == 0) break;
        if (!takes) continue;
        differ |= j && last - n <= close && !same(last, n);
        if (g == 0) key_row[j] = n;
        if (j == last_slot) border = n;
        last = n;
        some = j + 1;
      }
      // Those beyond the wavefront's lanes, a bit each: with one of another logit or bias among them
      // the whole row is chosen in 64 bits.
      u32 beyond = 0;
      if (closes && some == (u32)kWave) {
#pragma unroll
        for (int i = 0; i < C; ++i) beyond |= (u32)(key[i] > K::kLow && key[i] < last && border - key[i] <= close) << i;
      }
      bool other = false;
      for (u32 left = beyond; left; left &= left - 1)
        other |= !same(last, K::kLow - R::index(__builtin_ctz(left), g));
      differ |= group_reduce<G>((u32)other, max_u) != 0;
      closes = closes && differ;
      if (group_reduce<G>((u32)(beyond != 0), max_u)) unsure = closes;
      wave_lds_sync();
      for (u64 left = __ballot(closes && !unsure && g == 0); left; left &= left - 1) {
        const RouteArgs& b = arguments_again();
        const u32 from = (u32)__builtin_ctzll(left);  // the row's first lane
        const u32 count = (u32)__builtin_amdgcn_readlane((int)some, (int)from), lane = lane_id();
        u32* keys = s_key[wave][from / G];
        const u32 n = lane < count ? keys[lane] : 0;
        const u32 rank = rank_exactly<T>(b, t0 + wave * kRows + from / G, count, K::kLow - (n & K::kLow),
                                         __shfl(row.top, (int)from));
        wave_lds_sync();
        if (lane < count && rank < b.k) keys[rank] = n;
      }
      wave_lds_sync();
      if (closes && !unsure && slots <= (u32)G && g < some && g < slots) mine = key_row[g];
    }
    auto weight_of = [](const RouteArgs& a, float v, float top, float inverse) {
      if constexpr (SIGMOID) return sigmoid_of(v).up;
      if (!(top < __builtin_huge_valf())) return top - top;  // of +inf or NaN: NaN
      const float w = exp_f(v - top);
      return a.normalize ? w : w * inverse;
    };
    auto share_of = [](const RouteArgs& a, float w, float chosen) { return chosen == 0.f ? 0.f : w / chosen * a.scale; };
    // lane g takes slots g, g + G, ...
    if (here && !unsure) {
      const RouteArgs& a = arguments_again();
      const u64 at = t * a.k;
      float chosen = 0.f, w = 0.f;
      for (u32 j = g; j < a.k; j += G) {
        const u32 n = a.k > (u32)G ? key_row[j] : mine, e = K::kLow - (n & K::kLow);
        const bool some = row.live && n > K::kLow;
        w = 0.f;
        if (some) {
          w = weight_of(a, to_f32(xt[e]), row.top, inv);
          atomicAdd(&s_cnt[e], 1u);
        }
        chosen += w;
        a.experts[at + j] = some ? (int64_t)e : -1;
        if (!a.normalize || a.k > (u32)G) a.weights[at + j] = a.normalize ? w : w * a.scale;
      }
      if (a.normalize) {
        chosen = group_reduce<G>(chosen, add_f);
        if (__builtin_expect(row.live && chosen < kFarScores, 0)) {
          float largest = kNone;
          for (u32 j = g; j < a.k; j += G) {
            const u32 n = a.k > (u32)G ? key_row[j] : mine;
            if (n > K::kLow) largest = max_f(largest, to_f32(xt[K::kLow - (n & K::kLow)]));
          }
          largest = group_reduce<G>(largest, max_f);
          const float least = SIGMOID ? kLeastLogit : least_held(row.top, inv);
          chosen = 0.f;
          for (u32 j = g; j < a.k; j += G) {
            const u32 n = a.k > (u32)G ? key_row[j] : mine;
            w = n > K::kLow ? far_share(to_f32(xt[K::kLow - (n & K::kLow)]), largest, least) : 0.f;
            chosen += w;
            if (a.k > (u32)G) a.weights[at + j] = w;
          }
          chosen = group_reduce<G>(chosen, add_f);
        }
        if (a.k <= (u32)G) {
          if (g < a.k) a.weights[at + g] = share_of(a, w, chosen);
        } else {
          for (u32 j = g; j < a.k; j += G) a.weights[at + j] = share_of(a, a.weights[at + j], chosen);
        }
      }
    }
    wave_lds_sync();
    for (u64 left = __ballot(unsure && g == 0); left; left &= left - 1) {
      const RouteArgs& b = arguments_again();
      const u32 from = (u32)__builtin_ctzll(left);  // the row's first lane
      const u64 r = t0 + wave * kRows + from / G;
      const float top = __shfl(row.top, (int)from), inverse = __shfl(inv, (int)from);
      const u32 e = choose_exactly<T>(b, r, top, reinterpret_cast<u64*>(s_key[wave][0]));
      const bool slot = lane_id() < b.k, some = slot && e < b.E;
      float w = 0.f, l = kNone;
      if (some) {
        l = to_f32(reinterpret_cast<const T*>(b.x)[r * b.ld + e]);
        w = weight_of(b, l, top, inverse);
        atomicAdd(&s_cnt[e], 1u);
      }
      float chosen = group_reduce<kWave>(w, add_f);
      if (b.normalize && chosen < kFarScores) {
        const float largest = group_reduce<kWave>(l, max_f);
        w = some ? far_share(l, largest, SIGMOID ? kLeastLogit : least_held(top, inverse)) : 0.f;
        chosen = group_reduce<kWave>(w, add_f);
      }
      if (slot) {
        b.experts[r * b.k + lane_id()] = some ? (int64_t)e : -1;
        b.weights[r * b.k + lane_id()] = b.normalize ? share_of(b, w, chosen) : w * b.scale;
      }
      wave_lds_sync();
    }
    if (arguments_again().loss && ++turn == kTurnsInRegisters && t0 + step < arguments_again().T) {  // the same for the whole block
      join();
      __syncthreads();
      turn = 0;
      clear();
    }
  }
  if (rows) atomicAdd(&s_rows, rows);
  join();
  const RouteArgs& z = arguments_again();
  if (gridDim.x == 1) {
    double part = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u32 e = threadIdx.x + h * kScoredThreads;
      if (e < z.E) {
        z.counts[e] = (int64_t)s_cnt[e];
        part += (double)s_cnt[e] * total[h];
      }
    }
    part = block_sum<kScoredWaves>(part, s_part);
    if (threadIdx.x == 0) {
      *z.rows = (int64_t)s_rows;
      if (z.loss) *z.loss = balance_of(part, s_rows, z.E, z.k);
    }
    return;
  }
  const RouteScratch sc = route_scratch(z.scratch, gridDim.x, z.E);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const u32 e = threadIdx.x + h * kScoredThreads;
    if (e < z.E) {
      sc.counts[(u64)blockIdx.x * z.E + e] = s_cnt[e];
      sc.sums[(u64)blockIdx.x * z.E + e] = total[h];
    }
  }
  if (threadIdx.x == 0) {
    sc.rows[blockIdx.x] = s_rows;
    if (blockIdx.x == 0) *sc.loss = 0;
  }
  if (blockIdx.x == 0 && threadIdx.x < kMostFinishing) sc.parts[threadIdx.x] = 0;
}

namespace {

struct Scored {
  template <class T, int G, int C, bool QUAD, bool SIGMOID>
  static hipError_t launch_one(RouteArgs a, hipStream_t s) {
    static const u32 fit = resident_blocks(scored_kernel<T, G, C, QUAD, SIGMOID>, kScoredThreads);
    a.blocks = route_blocks(a.T, kScoredThreads / G, fit < kRouteMaxBlocks ? fit : kRouteMaxBlocks);
    scored_kernel<T, G, C, QUAD, SIGMOID><<<a.blocks, kScoredThreads, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess || a.blocks == 1 ? e : launch_route_finish(a, s);
  }
  template <class T, int G, int C, bool QUAD>
  static hipError_t launch(const RouteArgs& a, hipStream_t s) {
    return a.sigmoid ? launch_one<T, G, C, QUAD, true>(a, s) : launch_one<T, G, C, QUAD, false>(a, s);
  }
};

}  // namespace

hipError_t launch_scored(const RouteArgs& a, int dtype, hipStream_t s) { return route_type<Scored>(a, dtype, s); }

}  // namespace profk
