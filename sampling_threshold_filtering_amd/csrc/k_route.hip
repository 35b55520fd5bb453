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
//
// Layout.  A group of G lanes takes a row, lane g its entries g, g + G, g + 2G, ... (C of
// them, in registers), so that the loads of a wavefront are contiguous for any E and any
// row stride, a row's maximum and sums are log2 G lane exchanges, and 64 / G rows share
// every instruction.  A lane keeps the same experts for all of its rows, so P_e is summed
// in its registers; lanes, wavefronts and blocks are then added in a fixed order (no
// floating-point atomics: the loss has the same bits on every run).
#include "launch.h"
#include "ops_device.h"

namespace profk {

namespace {

constexpr int kRouteThreads = 256;
constexpr int kRouteWaves = kRouteThreads / kWave;
constexpr u32 kRouteMaxBlocks = 512;
constexpr int kFinishThreads = 1024;
constexpr u32 kFinishExperts = 16;

// Sum / maximum over the G lanes of a group; every lane gets the result.
template <int G, class V, class F>
__device__ __forceinline__ V group_reduce(V v, F f) {
  const u32 lane = lane_id();
  if constexpr (G > 1) v = f(v, __builtin_bit_cast(V, lane_xor_u32<1>(__builtin_bit_cast(u32, v), lane)));
  if constexpr (G > 2) v = f(v, __builtin_bit_cast(V, lane_xor_u32<2>(__builtin_bit_cast(u32, v), lane)));
  if constexpr (G > 4) v = f(v, __builtin_bit_cast(V, lane_xor_u32<4>(__builtin_bit_cast(u32, v), lane)));
  if constexpr (G > 8) v = f(v, __builtin_bit_cast(V, lane_xor_u32<8>(__builtin_bit_cast(u32, v), lane)));
  if constexpr (G > 16) v = f(v, __builtin_bit_cast(V, lane_xor_u32<16>(__builtin_bit_cast(u32, v), lane)));
  if constexpr (G > 32) v = f(v, __builtin_bit_cast(V, lane_xor_u32<32>(__builtin_bit_cast(u32, v), lane)));
  return v;
}

__device__ __forceinline__ float add_f(float a, float b) { return a + b; }
// NaN wins, so that a row that holds one has NaN weights.
__device__ __forceinline__ float max_f(float a, float b) { return a != a || a > b ? a : b; }
__device__ __forceinline__ u32 max_u(u32 a, u32 b) { return a > b ? a : b; }
__device__ __forceinline__ u32 min_u(u32 a, u32 b) { return a < b ? a : b; }

// e^x for x <= 0 to about one unit in the last place: the rounding of x log2(e), which
// grows with |x|, is made up for by one more multiply-add.  Differences as far apart as the
// type reaches (and -inf) are cut to one whose exponential is 0; NaN stays NaN.
__device__ __forceinline__ float exp_f(float x) {
  x = x < -150.f ? -150.f : x;
  const float t = x * 1.44269502f;  // log2(e) = 1.44269502 + 1.925963e-8
  const float r = __builtin_fmaf(x, 1.44269502f, -t) + x * 1.925963e-8f;
  const float e = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(e, r * 0.693147182f, e);
}

// One row in registers: its C entries per lane and what the softmax needs.
template <int G, int C>
struct Row {
  float v[C];
  float p[C];
  bool live;
  float top, inv;  // the largest entry; 1 / sum of exp

  template <class T>
  __device__ __forceinline__ void load(const T* x, u32 E, u32 g, bool in) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const u32 e = (u32)i * G + g;
      v[i] = in && e < E ? to_f32(x[e]) : -__builtin_huge_valf();
    }
  }
  __device__ __forceinline__ void softmax(bool in) {
    float m = v[0];
#pragma unroll
    for (int i = 1; i < C; ++i) m = max_f(m, v[i]);
    top = group_reduce<G>(m, max_f);
    live = in && !(top == -__builtin_huge_valf());
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      p[i] = exp_f(v[i] - top);  // entries of -inf: 0
      s += p[i];
    }
    s = group_reduce<G>(s, add_f);
    inv = 1.f / s;
#pragma unroll
    for (int i = 0; i < C; ++i) p[i] = live ? p[i] * inv : 0.f;
  }
};

// A launch of several blocks leaves each block's counts, sums and live rows here for the
// finishing launch; one block alone writes the outputs itself.
struct RouteScratch {
  u32* ticket;   // finishing blocks that have left their part
  double* part;  // one per finishing block
  u32* rows;     // blocks
  u32* counts;   // blocks * E
  float* sums;   // blocks * E
};

__host__ __device__ inline RouteScratch route_scratch(char* s, u32 blocks, u32 E) {
  RouteScratch r;
  r.ticket = (u32*)s;
  r.part = (double*)(s + 256);
  r.rows = (u32*)(s + 256 + 8 * kRouteMaxExperts);
  r.counts = r.rows + blocks;
  r.sums = (float*)(r.counts + (u64)blocks * E);
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

}  // namespace

// GIVEN: the experts are a.given's (the balance loss of a choice made elsewhere).
template <class T, int G, int C, bool GIVEN>
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
  for (u64 t0 = (u64)blockIdx.x * kGroups; t0 < a.T; t0 += step) {
    const u64 t = t0 + grp;
    const bool in = t < a.T && (!a.mask || a.mask[t]);
    Row<G, C> row;
    row.load(x + t * a.ld, a.E, g, in);
    row.softmax(in);
#pragma unroll
    for (int i = 0; i < C; ++i) sum[i] += row.p[i];
    rows += row.live && g == 0;
    if (t >= a.T) continue;  // no lane exchange below crosses groups
    if constexpr (GIVEN) {
      if (row.live)
        for (u32 j = g; j < a.k; j += G) {
          const int64_t e = a.given[t * a.k + j];
          if (e >= 0 && e < (int64_t)a.E) atomicAdd(&s_cnt[e], 1u);
        }
    } else {
      u32 key[C];
#pragma unroll
      for (int i = 0; i < C; ++i) key[i] = row.live && row.v[i] != -__builtin_huge_valf() ? ord32(__float_as_uint(row.v[i])) : 0u;
      float chosen = 0.f;
      for (u32 j = 0; j < a.k; ++j) {
        u32 m = 0;
#pragma unroll
        for (int i = 0; i < C; ++i) m = max_u(m, key[i]);
        m = group_reduce<G>(m, max_u);
        u32 e = ~0u;
        float p = 0.f;
#pragma unroll
        for (int i = C - 1; i >= 0; --i)
          if (key[i] == m) e = (u32)i * G + g;
        e = group_reduce<G>(e, min_u);
        if (m == 0) e = ~0u;
#pragma unroll
        for (int i = 0; i < C; ++i)
          if (e == (u32)i * G + g) {
            key[i] = 0;
            p = row.p[i];
          }
        p = group_reduce<G>(p, add_f);
        chosen += p;
        if (g == 0) {
          a.experts[t * a.k + j] = m ? (int64_t)e : -1;
          a.weights[t * a.k + j] = p;
          if (m) atomicAdd(&s_cnt[e], 1u);
        }
      }
      if (a.normalize && g == 0 && row.live) {
        const float r = 1.f / chosen;
        for (u32 j = 0; j < a.k; ++j) a.weights[t * a.k + j] *= r;
      }
    }
  }
  // the block's sums: the wavefront's groups, then its wavefronts
#pragma unroll
  for (int i = 0; i < C; ++i) {
    float v = sum[i];
#pragma unroll
    for (int d = G; d < kWave; d <<= 1) v += __shfl_xor(v, d);
    if (lane_id() < G) s_sum[threadIdx.x / kWave][i * G + g] = v;
  }
  if (rows) atomicAdd(&s_rows, rows);
  __syncthreads();
  if (gridDim.x == 1) {
    double part = 0;
    for (u32 e = threadIdx.x; e < a.E; e += kRouteThreads) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kRouteWaves; ++w) v += s_sum[w][e];
      a.counts[e] = (int64_t)s_cnt[e];
      part += (double)s_cnt[e] * (double)v;
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
  for (u32 e = threadIdx.x; e < a.E; e += kRouteThreads) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kRouteWaves; ++w) v += s_sum[w][e];
    sc.counts[(u64)blockIdx.x * a.E + e] = s_cnt[e];
    sc.sums[(u64)blockIdx.x * a.E + e] = v;
  }
  if (threadIdx.x == 0) {
    sc.rows[blockIdx.x] = s_rows;
    if (blockIdx.x == 0) *sc.ticket = 0;
  }
}

// The blocks' counts and sums into the outputs.  A finishing block takes 16 experts, its
// threads 64 slices of the blocks, so that a thread adds 8 of 512 (one block over all
// experts, 512 each: 121 us).  The last block to leave its part of the loss adds the
// parts, in their order.
__global__ __launch_bounds__(kFinishThreads) void route_finish_kernel(RouteArgs a) {
  constexpr u32 kSlices = kFinishThreads / kFinishExperts;
  __shared__ u64 s_c[kSlices][kFinishExperts + 1];
  __shared__ double s_p[kSlices][kFinishExperts + 1];
  __shared__ double s_part[kFinishThreads / kWave];
  __shared__ u32 s_last;
  const RouteScratch sc = route_scratch(a.scratch, a.blocks, a.E);
  const u32 el = threadIdx.x % kFinishExperts, sl = threadIdx.x / kFinishExperts;
  const u32 e = blockIdx.x * kFinishExperts + el;
  u64 c = 0;
  double p = 0;
  if (e < a.E)
    for (u32 b = sl; b < a.blocks; b += kSlices) {
      c += sc.counts[(u64)b * a.E + e];
      p += (double)sc.sums[(u64)b * a.E + e];
    }
  s_c[sl][el] = c;
  s_p[sl][el] = p;
  __syncthreads();
  double part = 0;
  if (threadIdx.x < kFinishExperts && e < a.E) {
    c = 0;
    p = 0;
    for (u32 i = 0; i < kSlices; ++i) {
      c += s_c[i][el];
      p += s_p[i][el];
    }
    a.counts[e] = (int64_t)c;
    part = (double)c * p;
  }
  part = block_sum<kFinishThreads / kWave>(part, s_part);
  if (threadIdx.x == 0) {
    s_last = 1;
    if (gridDim.x > 1) {
      __hip_atomic_store(&sc.part[blockIdx.x], part, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      s_last = __hip_atomic_fetch_add(sc.ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
    }
  }
  __syncthreads();
  if (!s_last) return;
  double rows = 0;  // exact: below 2^31
  for (u32 b = threadIdx.x; b < a.blocks; b += kFinishThreads) rows += (double)sc.rows[b];
  __syncthreads();
  rows = block_sum<kFinishThreads / kWave>(rows, s_part);
  if (threadIdx.x == 0) {
    if (gridDim.x > 1) {
      part = 0;
      for (u32 b = 0; b < gridDim.x; ++b)
        part += __hip_atomic_load(&sc.part[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    *a.rows = (int64_t)rows;
    if (a.loss) *a.loss = balance_of(part, (u64)rows, a.E, a.k);
  }
}

template <class T, int G, int C>
__global__ __launch_bounds__(kRouteThreads) void route_grad_kernel(RouteGradArgs a) {
  constexpr int kGroups = kRouteThreads / G;
  __shared__ float s_d[kGroups][G * C];
  const u32 g = threadIdx.x % G, grp = threadIdx.x / G;
  float* d = s_d[grp];
#pragma unroll
  for (int i = 0; i < C; ++i) d[i * G + g] = 0.f;
  const T* x = reinterpret_cast<const T*>(a.x);
  T* dx = reinterpret_cast<T*>(a.d_x);
  float f[C];
#pragma unroll
  for (int i = 0; i < C; ++i) f[i] = 0.f;
  float scale = 0.f;
  if (a.counts) {
    const double n = (double)*a.rows;
    if (n > 0) {
      scale = (float)((double)(a.d_loss ? *a.d_loss : 1.f) * (double)a.d_loss_scale * (double)a.E / n);
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const u32 e = (u32)i * G + g;
        if (e < a.E) f[i] = (float)((double)a.counts[e] / (n * (double)a.k));
      }
    }
  }
  const u64 step = (u64)gridDim.x * kGroups;
  for (u64 t0 = (u64)blockIdx.x * kGroups; t0 < a.T; t0 += step) {
    const u64 t = t0 + grp;
    const bool in = t < a.T && (!a.mask || a.mask[t]);
    Row<G, C> row;
    row.load(x + t * a.ld, a.E, g, in);
    row.softmax(in);
    float out[C];
    // the loss's part: constant factors f
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) dot += row.p[i] * f[i];
    dot = group_reduce<G>(dot, add_f);
#pragma unroll
    for (int i = 0; i < C; ++i) out[i] = scale * row.p[i] * (f[i] - dot);
    if (a.d_weights) {
      // the chosen entries: lane g takes slots g, g + G, ...
      float wsum = 0.f, wd = 0.f;
      if (row.live)
        for (u32 j = g; j < a.k; j += G) {
          const int64_t e = a.experts[t * a.k + j];
          if (e < 0 || e >= (int64_t)a.E) continue;
          const float p = exp_f(to_f32(x[t * a.ld + e]) - row.top) * row.inv;
          wsum += p;
          wd += p * a.d_weights[t * a.k + j];
        }
      wsum = group_reduce<G>(wsum, add_f);
      wd = group_reduce<G>(wd, add_f);
      const float r = a.normalize ? 1.f / wsum : 1.f;
      const float mean = a.normalize ? wd * r : wd;
      if (row.live)
        for (u32 j = g; j < a.k; j += G) {
          const int64_t e = a.experts[t * a.k + j];
          if (e < 0 || e >= (int64_t)a.E) continue;
          const float p = exp_f(to_f32(x[t * a.ld + e]) - row.top) * row.inv * r;
          const float dw = a.d_weights[t * a.k + j];
          atomicAdd(&d[e], p * (a.normalize ? dw - mean : dw));
        }
      wave_lds_sync();
#pragma unroll
      for (int i = 0; i < C; ++i) {
        out[i] += d[i * G + g];
        if (!a.normalize) out[i] -= row.p[i] * mean;
      }
      wave_lds_sync();
#pragma unroll
      for (int i = 0; i < C; ++i) d[i * G + g] = 0.f;
      wave_lds_sync();
    }
    if (t < a.T)
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const u32 e = (u32)i * G + g;
        T o;
        from_f32(row.live ? out[i] : 0.f, o);
        if (e < a.E) dx[t * a.E + e] = o;
      }
  }
}

namespace {

u32 route_blocks(u64 T, u32 groups) {
  const u64 b = (T + groups - 1) / groups;
  return (u32)(b < kRouteMaxBlocks ? (b ? b : 1) : kRouteMaxBlocks);
}

template <class T, int G, int C>
hipError_t route_launch(const RouteArgs& a0, hipStream_t s) {
  RouteArgs a = a0;
  a.blocks = route_blocks(a.T, kRouteThreads / G);
  if (a.balance_only)
    route_kernel<T, G, C, true><<<a.blocks, kRouteThreads, 0, s>>>(a);
  else
    route_kernel<T, G, C, false><<<a.blocks, kRouteThreads, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.blocks == 1) return e;
  route_finish_kernel<<<(a.E + kFinishExperts - 1) / kFinishExperts, kFinishThreads, 0, s>>>(a);
  return hipGetLastError();
}

template <class T, int G, int C>
hipError_t route_launch(const RouteGradArgs& a, hipStream_t s) {
  const u64 b = (a.T + kRouteThreads / G - 1) / (kRouteThreads / G);
  const u64 cap = (u64)device_cu_count() * 8;
  route_grad_kernel<T, G, C><<<(u32)(b < cap ? (b ? b : 1) : cap), kRouteThreads, 0, s>>>(a);
  return hipGetLastError();
}

// Lanes per row and entries per lane: the smallest C of the list that holds the row.
template <class T, class A>
hipError_t route_shape(const A& a, hipStream_t s) {
  if (a.E <= 16) return route_launch<T, 16, 1>(a, s);
  if (a.E <= 64) return route_launch<T, 16, 4>(a, s);
  if (a.E <= 128) return route_launch<T, 16, 8>(a, s);
  if (a.E <= 256) return route_launch<T, 16, 16>(a, s);
  if (a.E <= 512) return route_launch<T, 64, 8>(a, s);
  return route_launch<T, 64, 16>(a, s);
}

template <class A>
hipError_t route_type(const A& a, int dtype, hipStream_t s) {
  if (dtype == PROFK_FP32) return route_shape<float>(a, s);
  if (dtype == PROFK_FP16) return route_shape<Half16>(a, s);
  return route_shape<Brain16>(a, s);
}

}  // namespace

size_t route_scratch_bytes(u64 T, u32 E) {
  const u64 b = T < kRouteMaxBlocks ? (T ? T : 1) : kRouteMaxBlocks;
  return 256 + 8 * (size_t)kRouteMaxExperts + b * (4 + 8 * (size_t)E);
}

hipError_t launch_route(const RouteArgs& a, int dtype, hipStream_t s) { return route_type(a, dtype, s); }
hipError_t launch_route_grad(const RouteGradArgs& a, int dtype, hipStream_t s) { return route_type(a, dtype, s); }

}  // namespace profk
