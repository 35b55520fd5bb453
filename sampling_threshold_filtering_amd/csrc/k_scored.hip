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
// 2^24, from the lowest bias up, above the entry's complement.  A unit is a few times the
// error of c in 32 bits, so where two neighbours among the first k + 1 keys, or the worst
// group kept and the best left out, are within that error of each other, the wavefront
// chooses again in 64 bits; two entries of the same logit and bias are told apart by their
// index in any arithmetic and do not need it.  A fixed point rather than the float's own bits:
// its low bits are what the index leaves of a float's 24 (at 256 experts 15, too few for one
// row in 30; the fixed point's 24 leave one row in 600).
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
__device__ __forceinline__ u64 wave_max(u64 v) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const u64 o = __shfl_xor(v, d);
    v = o > v ? o : v;
  }
  return v;
}
__device__ __forceinline__ u32 wave_min(u32 v) {
  return ~wave_reduce_u32(~v, [](u32 a, u32 b) { return a > b ? a : b; });
}

// What the wavefront's rows need of the choice: the keys in LDS, row by row.
template <int G, int C>
struct Choice {
  static constexpr int kBits = key_bits(G * C);
  static constexpr u32 kLow = (1u << kBits) - 1;
  static constexpr int kUnits = 32 - kBits < 24 ? 32 - kBits : 24;  // bits of c
  static constexpr u32 kMostGroups = G * C < (int)kRouteMaxGroups ? G * C : kRouteMaxGroups;
};

}  // namespace

// One row by the whole wavefront in 64 bits: lane j gets slot j's expert, or ~0.
template <class T, int E64>
__device__ __forceinline__ u32 choose_exactly(const RouteArgs& a, const T* x) {
  const u32 lane = lane_id();
  double l[E64];
  double top = -__builtin_huge_val();
#pragma unroll
  for (int i = 0; i < E64; ++i) {
    const u32 e = i * kWave + lane;
    l[i] = e < a.E ? (double)to_f32(x[e]) : -__builtin_huge_val();
    top = l[i] > top || l[i] != l[i] ? l[i] : top;
  }
  u64 code[E64];
  if (!a.sigmoid) {
    // (a NaN or +inf makes every score NaN)
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const double o = __shfl_xor(top, d);
      top = o > top || o != o ? o : top;
    }
    double sum = 0;
#pragma unroll
    for (int i = 0; i < E64; ++i) sum += exp(l[i] - top);
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) sum += __shfl_xor(sum, d);
#pragma unroll
    for (int i = 0; i < E64; ++i) code[i] = __builtin_bit_cast(u64, exp(l[i] - top) / sum);
  } else {
#pragma unroll
    for (int i = 0; i < E64; ++i) code[i] = __builtin_bit_cast(u64, 1.0 / (1.0 + exp(-l[i])));
  }
#pragma unroll
  for (int i = 0; i < E64; ++i) {
    const u32 e = i * kWave + lane;
    const double b = a.bias && e < a.E ? (double)a.bias[e] : 0.0;
    const double c = __builtin_bit_cast(double, code[i]) + b;
    code[i] = e >= a.E || l[i] == -__builtin_huge_val() || c == -__builtin_huge_val() ? 0 : code_of(c);
  }
  const u32 size = a.E / a.groups;
  if (a.top_groups < a.groups) {
    u64 mine = 0;  // lane g: group g's score
    for (u32 g = 0; g < a.groups; ++g) {
      u64 first = 0;
#pragma unroll
      for (int i = 0; i < E64; ++i) {
        const u32 e = i * kWave + lane;
        if (e / size == g && code[i] > first) first = code[i];
      }
      first = wave_max(first);
      u64 score = first;
      if (a.group_best == 2 && first) {
        u32 at = ~0u;
#pragma unroll
        for (int i = 0; i < E64; ++i) {
          const u32 e = i * kWave + lane;
          if (e / size == g && code[i] == first && e < at) at = e;
        }
        at = wave_min(at);
        u64 second = 0;
#pragma unroll
        for (int i = 0; i < E64; ++i) {
          const u32 e = i * kWave + lane;
          if (e / size == g && e != at && code[i] > second) second = code[i];
        }
        second = wave_max(second);
        if (second) score = code_of(of_code(first) + of_code(second));
      }
      if (lane == g) mine = score;
    }
    u32 before = 0;
    for (u32 g = 0; g < a.groups; ++g) {
      const u64 o = __shfl(mine, (int)g);
      before += o > mine || (o == mine && g < lane);
    }
    const u64 kept = __ballot(lane < a.groups && before < a.top_groups);
#pragma unroll
    for (int i = 0; i < E64; ++i) {
      const u32 e = i * kWave + lane;
      if (e < a.E && !(kept >> (e / size) & 1)) code[i] = 0;
    }
  }
  u32 slot = ~0u;
  static_assert(kRouteMaxK <= kWave, "a lane per slot");
  for (u32 j = 0; j < a.k; ++j) {
    u64 first = 0;
#pragma unroll
    for (int i = 0; i < E64; ++i) first = code[i] > first ? code[i] : first;
    first = wave_max(first);
    u32 at = ~0u;
    if (first) {
#pragma unroll
      for (int i = 0; i < E64; ++i) {
        const u32 e = i * kWave + lane;
        if (code[i] == first && e < at) at = e;
      }
      at = wave_min(at);
#pragma unroll
      for (int i = 0; i < E64; ++i)
        if (i * kWave + lane == at) code[i] = 0;
    }
    if (lane == j) slot = at;
  }
  return slot;
}

template <class T, int G, int C, bool QUAD, bool SIGMOID>
__global__ __launch_bounds__(kScoredThreads) void scored_kernel(RouteArgs a) {
  using R = Row<G, C, QUAD>;
  using K = Choice<G, C>;
  constexpr int kGroups = kScoredThreads / G, kRows = kWave / G;  // rows of a block, of a wavefront
  __shared__ u32 s_key[kScoredWaves][kRows][G * C];
  __shared__ u32 s_group[kScoredWaves][kRows][K::kMostGroups];
  __shared__ u32 s_cnt[G * C];
  __shared__ float s_sum[kScoredWaves][G * C];
  __shared__ u32 s_rows;
  __shared__ double s_part[kScoredWaves];
  static_assert(G * C <= 2 * kScoredThreads, "two experts a thread");
  const u32 g = threadIdx.x % G, grp = threadIdx.x / G, wave = threadIdx.x / kWave, row_of_wave = lane_id() / G;
  for (u32 e = threadIdx.x; e < G * C; e += kScoredThreads) s_cnt[e] = 0;
  if (threadIdx.x == 0) s_rows = 0;
  __syncthreads();
  u32* key_row = s_key[wave][row_of_wave];
  u32* group_row = s_group[wave][row_of_wave];
  const T* x = reinterpret_cast<const T*>(a.x);
  // The biases in units from the lowest; entries without one (-inf) get none.
  float low = a.bias ? __builtin_huge_valf() : 0.f, high = a.bias ? -__builtin_huge_valf() : 0.f;
  bool odd = false;  // a bias that the keys cannot hold
  float base[C];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const u32 e = R::index(i, g);
    base[i] = e >= a.E ? kNone : a.bias ? a.bias[e] : 0.f;
    odd |= base[i] != base[i] || base[i] == __builtin_huge_valf();
    if (base[i] > kNone && base[i] < __builtin_huge_valf()) {
      low = __builtin_fminf(low, base[i]);
      high = __builtin_fmaxf(high, base[i]);
    }
  }
  low = -group_reduce<G>(-low, max_f);
  high = group_reduce<G>(high, max_f);
  if (!(low <= high)) low = high = 0.f;
  odd = group_reduce<G>((u32)odd, max_u) != 0;
  // a unit: the range of c over 2^kUnits, less room for roundings at both ends
  const float unit = (float)(((double)(1u << K::kUnits) - 64.0) / ((double)high - (double)low + 1.0));
#pragma unroll
  for (int i = 0; i < C; ++i)
    base[i] = base[i] == kNone ? kNone : (float)(((double)base[i] - (double)low) * (double)unit + 32.0);
  const u32 size = a.E / a.groups;
  const bool grouped = a.top_groups < a.groups;
  const u32 best = a.group_best < size ? a.group_best : size;
  u32 lanes = 1;  // per group of experts
  while (lanes * 2 * a.groups <= (u32)G) lanes *= 2;

  float sum[C];
#pragma unroll
  for (int i = 0; i < C; ++i) sum[i] = 0.f;
  u32 rows = 0;
  const u64 step = (u64)gridDim.x * kGroups;
  double total[2] = {0, 0};  // of experts threadIdx.x and threadIdx.x + kScoredThreads
  auto join = [&]() {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float v = sum[i];
#pragma unroll
      for (int d = G; d < kWave; d <<= 1) v += __shfl_xor(v, d);
      if (lane_id() < G) s_sum[wave][R::index(i, g)] = v;
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u32 e = threadIdx.x + h * kScoredThreads;
      if (e < a.E)
#pragma unroll
        for (int w = 0; w < kScoredWaves; ++w) total[h] += (double)s_sum[w][e];
    }
  };
  u32 turn = 0;
  for (u64 t0 = (u64)blockIdx.x * kGroups; t0 < a.T; t0 += step) {
    const u64 t = t0 + grp, tr = t < a.T ? t : a.T - 1;
    const bool in = (!a.mask || a.mask[tr]) && t < a.T, here = t < a.T;
    const T* xt = x + tr * a.ld;
    R row;
    row.load(xt, a.E, g, in);
    bool nan = false;
    if constexpr (SIGMOID) {
      float unused[1];
      row.score(in, unused);
    } else {
      row.weigh(in);
    }
#pragma unroll
    for (int i = 0; i < C; ++i) nan |= row.e[i] != row.e[i];
    const float inv = row.inverse();
    if (a.loss) {
#pragma unroll
      for (int i = 0; i < C; ++i) sum[i] = __builtin_fmaf(row.e[i], inv, sum[i]);
    }
    rows += row.live && g == 0;
    // keys
    u32 key[C];
    const float per = SIGMOID ? unit : unit * inv;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const u32 e = R::index(i, g);
      const float u = __builtin_fmaf(row.e[i], per, base[i]);
      key[i] = row.v[i] > kNone && base[i] > kNone ? (u32)u << K::kBits | (K::kLow - e) : K::kLow - e;
    }
    // How far two keys may be off each other, in units.  A sigmoid is off by 3.5 h of 1 at most (h =
    // 2^-24), which is 3.5 units at most; a probability by (32 + 2 |d|) h of itself, below 64 h of
    // the row's largest; the product's and the bias's rounding by half a unit each, the cut by one.
    const u32 near = SIGMOID ? 12 : 5 + (u32)(__builtin_fminf(unit * inv, 0x1p24f) * 0x1p-17f);
    bool unsure = odd || group_reduce<G>((u32)nan, max_u) != 0;
    if (grouped) {
#pragma unroll
      for (int i = 0; i < C; ++i)
        if (R::index(i, g) < a.E) key_row[R::index(i, g)] = key[i];
      wave_lds_sync();
      for (u32 q = g / lanes; q < a.groups; q += (u32)G / lanes) {
        u32 first = 0, second = 0;
        for (u32 j = g % lanes; j < size; j += lanes) {
          const u32 u = key_row[q * size + j] >> K::kBits;
          second = max_u(second, first < u ? first : u);
          first = max_u(first, u);
        }
        for (u32 d = 1; d < lanes; d <<= 1) {
          const u32 f = __shfl_xor(first, (int)d), s = __shfl_xor(second, (int)d);
          second = max_u(max_u(second, s), first < f ? first : f);
          first = max_u(first, f);
        }
        if (best == 2) {
          unsure |= first && !second;  // one score against sums of two
          first += second;
        }
        if (g % lanes == 0) group_row[q] = first;
      }
      wave_lds_sync();
      u32 least = ~0u, most = 0;  // of the groups kept, of those left out
      for (u32 q = g / lanes; q < a.groups; q += (u32)G / lanes) {
        const u32 own = group_row[q];
        u32 before = 0;
        for (u32 h = 0; h < a.groups; ++h) {
          const u32 o = group_row[h];
          before += o > own || (o == own && h < q);
        }
        if (before < a.top_groups) {
          least = least < own ? least : own;
        } else {
          most = max_u(most, own);
          for (u32 j = g % lanes; j < size; j += lanes) key_row[q * size + j] = K::kLow - (q * size + j);
        }
      }
      least = ~group_reduce<G>(~least, max_u);
      most = group_reduce<G>(most, max_u);
      unsure |= most && least - most <= 2 * near;
      wave_lds_sync();
#pragma unroll
      for (int i = 0; i < C; ++i)
        if (R::index(i, g) < a.E) key[i] = key_row[R::index(i, g)];
      wave_lds_sync();
    }
    // the first k keys, and the next
    u32 m = 0;
    auto next_key = [&]() {
      u32 d = 0;
#pragma unroll
      for (int i = 0; i < C; ++i) d = max_u(d, key[i] - m);
      return m + group_reduce<G>(d, max_u);
    };
    for (u32 j = 0; j <= a.k && j < a.E; ++j) {
      const u32 n = next_key();
      if (j && n > K::kLow && (m >> K::kBits) - (n >> K::kBits) <= near) {
        const u32 e = K::kLow - (m & K::kLow), f = K::kLow - (n & K::kLow);
        unsure |= to_f32(xt[e]) != to_f32(xt[f]) || (a.bias && a.bias[e] != a.bias[f]);
      }
      m = n;
      if (g == 0 && j < a.k) key_row[j] = n > K::kLow ? K::kLow - (n & K::kLow) : ~0u;
    }
    unsure = group_reduce<G>((u32)unsure, max_u) && row.live;
    wave_lds_sync();
    for (u64 left = __ballot(unsure && g == 0); left; left &= left - 1) {
      const u32 from = (u32)__builtin_ctzll(left) / G;
      const u32 slot = choose_exactly<T, (G * C + kWave - 1) / kWave>(a, x + (t0 + wave * kRows + from) * a.ld);
      if (lane_id() < a.k) s_key[wave][from][lane_id()] = slot;
      wave_lds_sync();
    }
    // lane g takes slots g, g + G, ...
    if (here) {
      const u64 at = t * a.k;
      float chosen = 0.f, w = 0.f;
      for (u32 j = g; j < a.k; j += G) {
        const u32 e = key_row[j];
        const bool some = row.live && e < a.E;
        w = 0.f;
        if (some) {
          const float v = to_f32(xt[e]);
          if constexpr (SIGMOID) {
            w = sigmoid_of(v).up;
          } else {
            w = exp_f(v - row.top);
            if (!(row.top < __builtin_huge_valf())) w = row.top - row.top;  // of +inf or NaN: NaN
            if (!a.normalize) w *= inv;
          }
          atomicAdd(&s_cnt[e], 1u);
        }
        chosen += w;
        a.experts[at + j] = some ? (int64_t)e : -1;
        if (!a.normalize || a.k > (u32)G) a.weights[at + j] = a.normalize ? w : w * a.scale;
      }
      if (a.normalize) {
        chosen = group_reduce<G>(chosen, add_f);
        const float r = chosen == 0.f ? 0.f : 1.f;
        if (a.k <= (u32)G) {
          if (g < a.k) a.weights[at + g] = r != 0.f ? w / chosen * a.scale : 0.f;
        } else {
          for (u32 j = g; j < a.k; j += G) a.weights[at + j] = r != 0.f ? a.weights[at + j] / chosen * a.scale : 0.f;
        }
      }
    }
    wave_lds_sync();
    if (a.loss && ++turn == kTurnsInRegisters && t0 + step < a.T) {  // the same for the whole block
      join();
      __syncthreads();
      turn = 0;
#pragma unroll
      for (int i = 0; i < C; ++i) sum[i] = 0.f;
    }
  }
  if (rows) atomicAdd(&s_rows, rows);
  join();
  if (gridDim.x == 1) {
    double part = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u32 e = threadIdx.x + h * kScoredThreads;
      if (e < a.E) {
        a.counts[e] = (int64_t)s_cnt[e];
        part += (double)s_cnt[e] * total[h];
      }
    }
    part = block_sum<kScoredWaves>(part, s_part);
    if (threadIdx.x == 0) {
      *a.rows = (int64_t)s_rows;
      if (a.loss) *a.loss = balance_of(part, s_rows, a.E, a.k);
    }
    return;
  }
  const RouteScratch sc = route_scratch(a.scratch, gridDim.x, a.E);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const u32 e = threadIdx.x + h * kScoredThreads;
    if (e < a.E) {
      sc.counts[(u64)blockIdx.x * a.E + e] = s_cnt[e];
      sc.sums[(u64)blockIdx.x * a.E + e] = total[h];
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
