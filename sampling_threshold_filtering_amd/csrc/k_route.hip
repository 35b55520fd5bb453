// Routing tokens to experts, and the balance loss, forward and backward.
//
// Mathematics, for logits l[T, E] (rows: the live ones, whose mask is set and which have
// an entry above -inf; n of them):
//   p_t = softmax(l_t);  the k experts of a token: the first k of its row by value,
//   descending, ties by lower index, entries of -inf never;  gate weights p, or p divided
//   by the chosen ones' sum;  counts_e = how often e was chosen
//   f_e = counts_e / (n k),  P_e = sum_t p_te / n,  loss = E sum_e f_e P_e
// Gradients (the counts are constants):
//   loss:                 dl_te = (g E / n) p_te (f_e - sum_j p_tj f_j)
//   weights:              dl_te = p_te (d_te - sum_j p_tj d_tj), d scattered to the row
//   normalised weights:   dl_te = w_te (d_te - sum_j w_tj d_tj) at the chosen, else 0
//     (they are the softmax over the chosen entries alone)
// Of sigmoid scores s (k_scored.hip), p_t = s_t / sum s_t, and w_t = s_t / sum of the chosen ones:
//   loss:                 dl_te = (g E / n) p_te (1 - s_te) (f_e - sum_j p_tj f_j)
//   weights:              dl_te = s_te (1 - s_te) d_te
//   normalised weights:   dl_te = w_te (1 - s_te) (d_te - sum_j w_tj d_tj) at the chosen, else 0
//
// Layout.  A group of G lanes takes a row and holds C entries of it per lane in registers,
// so that a row's maximum and sums are log2 G lane exchanges and 64 / G rows share every
// instruction.  A lane takes its entries four neighbours at a time where rows allow it (one
// load of 16 or 8 bytes each), else lane g takes entries g, g + G, ...  A lane keeps the
// same experts for all of its rows, so P_e is summed in its registers, in 32 bits for at
// most four rows; the wavefronts' sums of those and the blocks' are then added in 64 bits, in
// a fixed order (no floating-point atomics: the loss has the same bits on every run).  Summed
// in 32 bits to the end, the error grew with the batch: 3e-6 of P_e at 128 rows a lane.
//
// 65536 x 256 bf16, k = 8: forward 24 us and 4.8 to join the blocks, backward 21.3 us;
// 131072 x 160 bf16, loss alone: forward 17 and 4.9, backward 24 us (3.5 TB/s); backward of
// sigmoid scores, a sum and a factor more, 65536 x 256: 23 us.  The forward
// is bound by its vector instructions (90 % of the cycles in both): per entry 3 to load and
// convert, 7 for the exponential and its sum, 4 for a selection key and 2 for each of the k
// maxima; 16 lanes share a row's log2 G exchanges, which 8 lanes with twice the entries did
// not make up for (30 us: fewer wavefronts hide less).
#include "route_device.h"

namespace profk {

namespace {

constexpr int kRouteThreads = 1024;
constexpr int kRouteWaves = kRouteThreads / kWave;
constexpr int kGradThreads = 256;
constexpr int kFinishThreads = 1024;

template <int G>
__device__ __forceinline__ u64 group_reduce64(u64 v) {  // the maximum
#pragma unroll
  for (int d = 1; d < G; d <<= 1) {
    const u64 o = __shfl_xor(v, d);
    v = o > v ? o : v;
  }
  return v;
}

// Ordered code of a value as a Row holds it.
__device__ __forceinline__ u32 ord_of(float v) {
  const u32 b = __float_as_uint(v + 0.f);  // -0 as +0
  return b ^ ((u32)((int)b >> 31) | 0x80000000u);
}

}  // namespace

// The row's k experts, their weights and counts.  All keys are distinct, so the next one
// below m is the largest of (key - m) modulo 2^32: those from m up wrap to the bottom, and
// nothing has to be struck out.  In 32-bit types two neighbours among the first k + 1 keys
// can agree in all of the value's bits that they hold; then the wavefront chooses again by
// 64-bit keys.
template <class T, int G, int C, bool QUAD>
__device__ __forceinline__ void choose(const RouteArgs& a, const Row<G, C, QUAD>& row, const T* x, u64 t, u32 g,
                                       float inv, u32* s_cnt) {
  using R = Row<G, C, QUAD>;
  constexpr int kBits = key_bits(G * C);
  constexpr bool kExact = sizeof(T) == 2;  // the codes of fp16 end in 13 constant bits, of bf16 in 16
  constexpr u32 kLow = (1u << kBits) - 1;
  constexpr u32 kNoneTop = 0x007FFFFFu | kLow;  // the largest key of an entry of -inf
  u32 key[C];
#pragma unroll
  for (int i = 0; i < C; ++i) key[i] = (ord_of(row.v[i]) & ~kLow) | (kLow - R::index(i, g));
  const u64 at = t * a.k;
  const bool here = t < a.T;
  float chosen = 0.f, w = 0.f;
  // lane g's slot j0 + g holds entry e, of value v
  auto emit = [&](u32 j0, u32 nj, bool some, u32 e, float v) {
    if (g >= nj || !here) return;
    w = 0.f;
    if (some) {
      w = exp_f(v - row.top);
      if (!(row.top < __builtin_huge_valf())) w = row.top - row.top;  // of +inf or NaN: NaN
      if (!a.normalize) w *= inv;
      atomicAdd(&s_cnt[e], 1u);
    }
    chosen += w;
    a.experts[at + j0 + g] = some ? (int64_t)e : -1;
    if (!a.normalize || a.k > (u32)G) a.weights[at + j0 + g] = w;
  };
  u32 m = 0;
  auto next_key = [&]() {
    u32 d = 0;
#pragma unroll
    for (int i = 0; i < C; ++i) d = max_u(d, key[i] - m);
    return m + group_reduce<G>(d, max_u);
  };
  bool unsure = false;
  for (u32 j0 = 0; j0 < a.k; j0 += G) {
    const u32 nj = a.k - j0 < (u32)G ? a.k - j0 : (u32)G;
    u32 mine = 0;
    for (u32 j = 0; j < nj; ++j) {
      const u32 n = next_key();
      if constexpr (!kExact) unsure |= j && !((m ^ n) & ~kLow) && n > kNoneTop;
      m = n;
      if (g == j) mine = m;
    }
    const u32 e = kLow - (mine & kLow);
    const bool some = row.live && mine > kNoneTop;
    if constexpr (kExact) {
      emit(j0, nj, some, e, __uint_as_float(bits_of_ord32(mine & 0x80000000u ? mine & ~kLow : mine | kLow)));
    } else {
      if (j0 + nj < a.E) {  // the first one left out
        const u32 n = next_key();
        unsure |= !((m ^ n) & ~kLow) && n > kNoneTop;
      }
      if (__ballot(unsure && row.live) == 0) {
        emit(j0, nj, some, e, some && g < nj ? to_f32(x[e]) : 0.f);
        continue;
      }
      u64 last = ~0ull, own = 0;
      for (u32 j = 0; j < a.k; ++j) {  // again from the first: slots before j0 have been given out
        u64 n = 0;
#pragma unroll
        for (int i = 0; i < C; ++i) {
          const u64 c = ((u64)ord_of(row.v[i]) << 32) | (u32)~R::index(i, g);
          n = c < last && c > n ? c : n;
        }
        last = group_reduce64<G>(n);
        if (g == j % G) own = last;
        if (j >= j0 && (j % G == G - 1 || j + 1 == a.k))
          emit(j / G * G, j % G + 1, row.live && (u32)(own >> 32) > 0x007FFFFFu, key_index(own),
               __uint_as_float(bits_of_ord32((u32)(own >> 32))));
      }
      break;
    }
  }
  if (!a.normalize) return;
  chosen = group_reduce<G>(chosen, add_f);
  const float r = row.live ? 1.f / chosen : 0.f;
  if (!here) return;
  if (a.k <= (u32)G) {
    if (g < a.k) a.weights[at + g] = w * r;
  } else {
    for (u32 j = g; j < a.k; j += G) a.weights[at + j] *= r;
  }
}

// GIVEN: the experts are a.given's (the balance loss of a choice made elsewhere).
template <class T, int G, int C, bool QUAD, bool GIVEN>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(RouteArgs a) {
  constexpr int kGroups = kRouteThreads / G;
  __shared__ u32 s_cnt[G * C];
  __shared__ float s_sum[kRouteWaves][G * C];
  __shared__ u32 s_rows;
  const u32 g = threadIdx.x % G, grp = threadIdx.x / G;
  for (u32 e = threadIdx.x; e < G * C; e += kRouteThreads) s_cnt[e] = 0;
  if (threadIdx.x == 0) s_rows = 0;
  __syncthreads();
  const T* x = reinterpret_cast<const T*>(a.x);
  float sum[C];
#pragma unroll
  for (int i = 0; i < C; ++i) sum[i] = 0.f;
  u32 rows = 0;
  const u64 step = (u64)gridDim.x * kGroups;
  const bool balance = GIVEN || a.loss;
  // The block's sums so far, of expert threadIdx.x: a wavefront's groups by lane exchanges,
  // its wavefronts in 64 bits.
  static_assert(G * C <= kRouteThreads, "a thread per expert");
  double total = 0;
  auto join = [&]() {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float v = sum[i];
#pragma unroll
      for (int d = G; d < kWave; d <<= 1) v += __shfl_xor(v, d);
      if (lane_id() < G) s_sum[threadIdx.x / kWave][Row<G, C, QUAD>::index(i, g)] = v;
    }
    __syncthreads();
    if (threadIdx.x < a.E)
#pragma unroll
      for (int w = 0; w < kRouteWaves; ++w) total += (double)s_sum[w][threadIdx.x];
  };
  u32 turn = 0;
  for (u64 t0 = (u64)blockIdx.x * kGroups; t0 < a.T; t0 += step) {
    const u64 t = t0 + grp, tr = t < a.T ? t : a.T - 1;
    const bool in = (!a.mask || a.mask[tr]) && t < a.T;
    Row<G, C, QUAD> row;
    row.load(x + tr * a.ld, a.E, g, in);
    row.weigh(in);
    float inv = 0.f;
    if (balance || !a.normalize) inv = row.inverse();
    if (balance) {
#pragma unroll
      for (int i = 0; i < C; ++i) sum[i] = __builtin_fmaf(row.e[i], inv, sum[i]);
    }
    rows += row.live && g == 0;
    if constexpr (GIVEN) {
      if (row.live)
        for (u32 j = g; j < a.k; j += G) {
          const int64_t e = a.given[t * a.k + j];
          if (e >= 0 && e < (int64_t)a.E) atomicAdd(&s_cnt[e], 1u);
        }
    } else {
      choose<T, G, C, QUAD>(a, row, x + tr * a.ld, t, g, inv, s_cnt);
    }
    if (balance && ++turn == kTurnsInRegisters && t0 + step < a.T) {  // the same for the whole block
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
    if (threadIdx.x < a.E) {
      a.counts[threadIdx.x] = (int64_t)s_cnt[threadIdx.x];
      part = (double)s_cnt[threadIdx.x] * total;
    }
    __shared__ double s_part[kRouteWaves];
    part = block_sum<kRouteWaves>(part, s_part);
    if (threadIdx.x == 0) {
      *a.rows = (int64_t)s_rows;
      if (a.loss) *a.loss = balance_of(part, s_rows, a.E, a.k);
    }
    return;
  }
  const RouteScratch sc = route_scratch(a.scratch, gridDim.x, a.E);
  if (threadIdx.x < a.E) {
    const u64 at = (u64)blockIdx.x * a.E + threadIdx.x;
    sc.counts[at] = s_cnt[threadIdx.x];
    sc.sums[at] = total;
  }
  if (threadIdx.x == 0) {
    sc.rows[blockIdx.x] = s_rows;
    if (blockIdx.x == 0) *sc.loss = 0;
  }
  if (blockIdx.x == 0 && threadIdx.x < kMostFinishing) sc.parts[threadIdx.x] = 0;
}

// The blocks' counts and sums into the outputs.  A finishing block takes 16 experts, its
// threads 64 slices of the blocks, so that a thread adds 8 of 512, all loaded at once (one
// block over all experts, 512 each: 121 us).  The last block to add its part of the loss
// writes it.
__global__ __launch_bounds__(kFinishThreads) void route_finish_kernel(RouteArgs a) {
  constexpr u32 kSlices = kFinishThreads / kFinishExperts;
  constexpr u32 kEach = kRouteMaxBlocks / kSlices;
  constexpr u32 kWaves = kFinishThreads / kWave;
  __shared__ u32 s_c[kWaves][kFinishExperts];
  __shared__ double s_p[kWaves][kFinishExperts];
  __shared__ u32 s_rows[kWaves];
  static_assert(kRouteMaxBlocks <= kFinishThreads, "a thread per block for the rows");
  const RouteScratch sc = route_scratch(a.scratch, a.blocks, a.E);
  const u32 el = threadIdx.x % kFinishExperts, sl = threadIdx.x / kFinishExperts, wid = threadIdx.x / kWave;
  const u32 e = blockIdx.x * kFinishExperts + el;
  u32 cs[kEach];
  double ps[kEach];
  u32 rows = threadIdx.x < a.blocks ? sc.rows[threadIdx.x] : 0;
#pragma unroll
  for (u32 i = 0; i < kEach; ++i) {
    const u32 b = sl + i * kSlices;
    const bool some = e < a.E && b < a.blocks;
    cs[i] = some ? sc.counts[(u64)b * a.E + e] : 0;
    ps[i] = some && a.loss ? sc.sums[(u64)b * a.E + e] : 0.0;
  }
  u32 c = 0;  // at most T k < 2^37 slots in all; a thread's and a wavefront's are of 8 and 32 blocks
  double p = 0;
#pragma unroll
  for (u32 i = 0; i < kEach; ++i) {
    c += cs[i];
    p += ps[i];
  }
#pragma unroll
  for (u32 d = kFinishExperts; d < (u32)kWave; d <<= 1) {
    c += __shfl_xor(c, d);
    p += __shfl_xor(p, d);
  }
#pragma unroll
  for (u32 d = 1; d < (u32)kWave; d <<= 1) rows += __shfl_xor(rows, d);
  if (lane_id() < kFinishExperts) {
    s_c[wid][el] = c;
    s_p[wid][el] = p;
  }
  if (lane_id() == 0) s_rows[wid] = rows;
  __syncthreads();
  if (threadIdx.x >= kWave) return;
  double part = 0;
  if (threadIdx.x < kFinishExperts && e < a.E) {
    u64 n = 0;
    p = 0;
#pragma unroll
    for (u32 w = 0; w < kWaves; ++w) {
      n += s_c[w][el];
      p += s_p[w][el];
    }
    a.counts[e] = (int64_t)n;
    part = (double)n * p;
  }
  if (!a.loss && blockIdx.x) return;
  u64 live = 0;
#pragma unroll
  for (u32 w = 0; w < kWaves; ++w) live += s_rows[w];
  if (threadIdx.x == 0 && blockIdx.x == 0) *a.rows = (int64_t)live;
  if (!a.loss) return;
#pragma unroll
  for (u32 d = 1; d < kFinishExperts; d <<= 1) part += __shfl_xor(part, d);
  if (threadIdx.x) return;
  const double share = live ? part / ((double)live * (double)a.k * (double)live) : 0.0;
  if (gridDim.x == 1) {
    *a.loss = (float)((double)a.E * share);
    return;
  }
  // sum_e f_e P_e is at most 1: a block adds its part in units of 2^-48, one to the count of
  // blocks (at most 64) and, for NaN, one to the count of those, with a single 64-bit
  // addition, whose order does not matter.  (Parts, then a ticket, then the parts read back
  // were three trips to memory: 0.7 us more.)  Those units are too coarse for a sum below
  // kSmall, as of a choice that the probabilities do not favour; all parts of such a sum are
  // below it, and such a part is stored as it is beforehand, for the last block to add up in
  // their order.
  constexpr double kSmall = 0x1p-18;  // 64 roundings to 2^-49 are 2^-25 of it
  if (share > 0 && share < kSmall) {
    __hip_atomic_store(&sc.parts[blockIdx.x], share, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __threadfence();
  }
  const u64 mine = (share == share ? (u64)rint(share * 0x1p48) << 14 : 1ull << 7) + 1;
  const u64 sum = mine + __hip_atomic_fetch_add(sc.loss, mine, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if ((sum & 127) != gridDim.x) return;
  double all = (double)(sum >> 14) * 0x1p-48;
  if (sum >> 7 & 127) {
    all = __builtin_nan("");
  } else if (all < kSmall) {
    __threadfence();
    all = 0;
    for (u32 b = 0; b < gridDim.x; ++b)
      all += __hip_atomic_load(&sc.parts[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  *a.loss = (float)((double)a.E * all);
}

// SIGMOID: of sigmoid scores; p are their shares of the row's sum.
template <class T, int G, int C, bool QUAD, bool SIGMOID>
__global__ __launch_bounds__(kGradThreads) void route_grad_kernel(RouteGradArgs a) {
  using R = Row<G, C, QUAD>;
  constexpr int kGroups = kGradThreads / G;
  __shared__ float s_d[kGroups][G * C];  // the chosen entries' part, 0 elsewhere
  const u32 g = threadIdx.x % G, grp = threadIdx.x / G;
  float* d = s_d[grp];
  if (a.d_weights)
#pragma unroll
    for (int i = 0; i < C; ++i) d[i * G + g] = 0.f;
  const T* x = reinterpret_cast<const T*>(a.x);
  T* dx = reinterpret_cast<T*>(a.d_x);
  float f[C];  // the balance loss's constant factors, scale among them
#pragma unroll
  for (int i = 0; i < C; ++i) f[i] = 0.f;
  if (a.counts) {
    const double n = (double)*a.rows;
    if (n > 0) {
      const double scale =
          (double)(a.d_loss ? *a.d_loss : 1.f) * (double)a.d_loss_scale * (double)a.E / (n * n * (double)a.k);
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const u32 e = R::index(i, g);
        if (e < a.E) f[i] = (float)(scale * (double)a.counts[e]);
      }
    }
  }
  auto slot = [&](u64 t, u32 j) {  // its expert; not below E: none
    const int64_t e = a.experts[t * a.k + j];
    return (u64)e < (u64)a.E ? (u32)e : ~0u;
  };
  const u64 step = (u64)gridDim.x * kGroups;
  for (u64 t0 = (u64)blockIdx.x * kGroups; t0 < a.T; t0 += step) {
    const u64 t = t0 + grp, tr = t < a.T ? t : a.T - 1;
    const bool in = (!a.mask || a.mask[tr]) && t < a.T;
    u32 first_e = ~0u;
    float first_d = 0.f;
    if (a.d_weights && g < a.k) {
      first_e = slot(tr, g);
      first_d = a.d_weights[tr * a.k + g] * a.scale;
    }
    R row;
    row.load(x + tr * a.ld, a.E, g, in);
    float falling[SIGMOID ? C : 1];  // 1 - score
    if constexpr (SIGMOID) {
      bool nan = false;
      row.score(in, nan, falling);
    } else {
      row.weigh(in);
    }
    const float inv = row.template inverse<SIGMOID>();
    float out[C];
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      row.e[i] *= inv;  // p
      dot = __builtin_fmaf(row.e[i], f[i], dot);
    }
    dot = group_reduce<G>(dot, add_f);
    if (a.d_weights) {
      // the chosen entries: lane g takes slots g, g + G, ...; its first one stays in registers
      const T* xt = x + tr * a.ld;
      // A normalised weight is of the exponentials themselves: the only one of its row is 1, and
      // its gradient 0, exactly.
      const float unit = a.normalize ? 1.f : inv;
      bool far = false;  // the chosen scores are relative to the largest of them
      float largest = kNone, least = kNone;
      auto weight = [&](u32 e) {
        const float l = to_f32(xt[e]);
        if (far) return far_share(l, largest, least);
        if constexpr (SIGMOID) return sigmoid_of(l).up;
        return exp_f(l - row.top) * unit;
      };
      const bool first = row.live && first_e < a.E;
      const float d0 = first ? first_d : 0.f;  // where there is no expert d_weights may hold anything
      float p0 = 0.f, wsum = 0.f, wd = 0.f;
      auto add_up = [&]() {
        p0 = first ? weight(first_e) : 0.f;
        wsum = p0;
        wd = p0 * d0;
        if (row.live)
          for (u32 j = g + G; j < a.k; j += G) {
            const u32 e = slot(tr, j);
            if (e >= a.E) continue;
            const float p = weight(e);
            wsum += p;
            wd = __builtin_fmaf(p, a.d_weights[tr * a.k + j] * a.scale, wd);
          }
        wsum = group_reduce<G>(wsum, add_f);
        wd = group_reduce<G>(wd, add_f);
      };
      add_up();
      bool lone = false;
      if (a.normalize && row.live && wsum < 1.f) {  // (of the row's top or more it is 1 or more)
        // the only one of a row has weight 1 and gradient 0, exactly, also where its exponential is not 1
        u32 slots = first;
        if (first) largest = to_f32(xt[first_e]);
        for (u32 j = g + G; j < a.k; j += G) {
          const u32 e = slot(tr, j);
          if (e >= a.E) continue;
          ++slots;
          largest = max_f(largest, to_f32(xt[e]));
        }
        lone = group_reduce<G>(slots, [](u32 p, u32 q) { return p + q; }) == 1;
        if (wsum < kFarScores) {
          largest = group_reduce<G>(largest, max_f);
          least = SIGMOID ? kLeastLogit : least_held(row.top, inv);
          far = true;
          add_up();
          if constexpr (SIGMOID) {
#pragma unroll
            for (int i = 0; i < C; ++i) falling[i] = row.e[i] == 0.f ? 1.f : falling[i];  // of scores that were flushed
          }
        }
      }
      const float r = !a.normalize ? 1.f : wsum == 0.f ? 0.f : 1.f / wsum;  // 0: no score that 64 bits hold
      const float mean = wd * r, from = a.normalize ? mean : 0.f;
      if (!a.normalize && !SIGMOID) dot += mean;
      if (first && !lone) atomicAdd(&d[first_e], p0 * r * (d0 - from));
      if (row.live)
        for (u32 j = g + G; j < a.k; j += G) {
          const u32 e = slot(tr, j);
          if (e < a.E && !lone) atomicAdd(&d[e], weight(e) * r * (a.d_weights[tr * a.k + j] * a.scale - from));
        }
      wave_lds_sync();
#pragma unroll
      for (int i = 0; i < C; ++i) {
        out[i] = __builtin_fmaf(row.e[i], f[i] - dot, d[R::index(i, g)]);
        if constexpr (SIGMOID) out[i] *= falling[i];
      }
      wave_lds_sync();
      if (first) d[first_e] = 0.f;
      if (row.live)
        for (u32 j = g + G; j < a.k; j += G) {
          const u32 e = slot(tr, j);
          if (e < a.E) d[e] = 0.f;
        }
      wave_lds_sync();
    } else {
#pragma unroll
      for (int i = 0; i < C; ++i) {
        out[i] = row.e[i] * (f[i] - dot);
        if constexpr (SIGMOID) out[i] *= falling[i];
      }
    }
    if (t >= a.T) continue;  // no lane exchange below
    T* to = dx + t * a.E;
    if constexpr (QUAD) {
#pragma unroll
      for (int i = 0; i < C; i += 4) {
        Four<T> q;
#pragma unroll
        for (int w = 0; w < 4; ++w) from_f32(row.live ? out[i + w] : 0.f, q.e[w]);
        if (R::index(i, g) < a.E) *reinterpret_cast<Four<T>*>(to + R::index(i, g)) = q;
      }
    } else {
#pragma unroll
      for (int i = 0; i < C; ++i) {
        T o;
        from_f32(row.live ? out[i] : 0.f, o);
        if (R::index(i, g) < a.E) to[R::index(i, g)] = o;
      }
    }
  }
}

hipError_t launch_route_finish(const RouteArgs& a, hipStream_t s) {
  route_finish_kernel<<<(a.E + kFinishExperts - 1) / kFinishExperts, kFinishThreads, 0, s>>>(a);
  return hipGetLastError();
}

namespace {

template <class T, int G, int C, bool QUAD, bool GIVEN>
hipError_t route_launch_one(RouteArgs a, hipStream_t s) {
  static const u32 fit = resident_blocks(route_kernel<T, G, C, QUAD, GIVEN>, kRouteThreads);
  a.blocks = route_blocks(a.T, kRouteThreads / G, fit < kRouteMaxBlocks ? fit : kRouteMaxBlocks);
  route_kernel<T, G, C, QUAD, GIVEN><<<a.blocks, kRouteThreads, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess || a.blocks == 1 ? e : launch_route_finish(a, s);
}

struct Forward {
  template <class T, int G, int C, bool QUAD>
  static hipError_t launch(const RouteArgs& a, hipStream_t s) {
    return a.balance_only ? route_launch_one<T, G, C, QUAD, true>(a, s) : route_launch_one<T, G, C, QUAD, false>(a, s);
  }
};

struct Gradient {
  template <class T, int G, int C, bool QUAD, bool SIGMOID>
  static hipError_t launch_one(const RouteGradArgs& a, hipStream_t s) {
    static const u32 fit = resident_blocks(route_grad_kernel<T, G, C, QUAD, SIGMOID>, kGradThreads);
    const u32 blocks = route_blocks(a.T, kGradThreads / G, fit);
    route_grad_kernel<T, G, C, QUAD, SIGMOID><<<blocks, kGradThreads, 0, s>>>(a);
    return hipGetLastError();
  }
  template <class T, int G, int C, bool QUAD>
  static hipError_t launch(const RouteGradArgs& a, hipStream_t s) {
    return a.sigmoid ? launch_one<T, G, C, QUAD, true>(a, s) : launch_one<T, G, C, QUAD, false>(a, s);
  }
};

}  // namespace

size_t route_scratch_bytes(u64 T, u32 E) {
  const u64 rounds = (T + kLeastRows - 1) / kLeastRows;
  const u64 b = rounds < kRouteMaxBlocks ? (rounds ? rounds : 1) : kRouteMaxBlocks;
  return kRouteScratchHead + b * (4 + 12 * (size_t)E);
}

hipError_t launch_route(const RouteArgs& a, int dtype, hipStream_t s) { return route_type<Forward>(a, dtype, s); }
hipError_t launch_route_grad(const RouteGradArgs& a, int dtype, hipStream_t s) { return route_type<Gradient>(a, dtype, s); }

}  // namespace profk
