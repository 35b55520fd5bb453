// The operators that train a policy on given tokens: their log-probabilities, the clipped
// policy loss and the preference loss, forward and gradient.
//
// Mathematics, for logits x[T, V], a token a_t per row and a temperature tau.  A row is live
// when its mask is set and its token is in [0, V).
//   lp_t = x_ta / tau - ln sum_j exp(x_tj / tau);  dlp_t / dx_tj = ([j = a] - p_tj) / tau
// Held relative to the row's top M, and with the token's own term apart from the others':
//   e_j = exp((x_j - M) / tau), R = sum over j != a of e_j, s = R + e_a
//   lp = (x_a - M) / tau - ln s, and -ln(1 + R) where the token is the top
//   dlp/dx_a = R / (s tau), dlp/dx_j = -e_j / (s tau)
// so a likely token's log-probability and gradient keep their digits: neither is a difference
// of numbers near 1.  Every operator's gradient is c_t times that, with c_t = dloss / dlp_t:
//   policy: r = exp(lp - old), l = -min(r A, clip(r, 1 - lo, 1 + hi) A) + b (e^q - 1 - q),
//     q = ref - lp;  dl/dlp = -r A (0 where clipped) - b (e^q - 1);  c_t = w_t dl/dlp
//   preference: D = sum (or mean) over a sequence's live rows of lp - ref,
//     z = beta (D_chosen - D_rejected) - margin, l = (1 - h) softplus(-z) + h softplus(z),
//     dl/dz = sigmoid(z) - (1 - h);  c_t = +-beta dl/dz / pairs (/ the sequence's live rows)
#include "ops_device.h"

namespace profk {

namespace {

constexpr u32 kVocabMaxBlocks = 2048;
constexpr u32 kCountBlocks = 64;
constexpr int kCountThreads = 1024;
constexpr int kPairThreads = 256;
constexpr u32 kPairBlocks = 1024;

// What the blocks leave for the last of them.
struct BlockTerms {
  double loss, kl;
  u64 clipped;
};
struct VocabScratch {
  u32* ticket;
  u32* live;          // kCountBlocks parts of the number of live rows
  BlockTerms* terms;  // kVocabMaxBlocks
  double* lp;         // T, for the preference loss
};
constexpr size_t kVocabHead = 512;
__host__ __device__ inline VocabScratch vocab_scratch(char* s) {
  VocabScratch v;
  v.ticket = (u32*)s;
  v.live = (u32*)(s + 128);
  v.terms = (BlockTerms*)(s + kVocabHead);
  v.lp = (double*)(s + kVocabHead + kVocabMaxBlocks * sizeof(BlockTerms));
  return v;
}

constexpr float kLowest = -3.402823466e38f;

typedef u32 Words __attribute__((ext_vector_type(4)));
typedef u32 HalfAlignedWords __attribute__((ext_vector_type(4), aligned(2)));
typedef u32 WordAlignedWords __attribute__((ext_vector_type(4), aligned(4)));
template <class T> struct AnyWords { typedef HalfAlignedWords type; };  // at any multiple of the element's size
template <> struct AnyWords<float> { typedef WordAlignedWords type; };

// Entry k of a vector's words.
template <class T>
__device__ __forceinline__ float entry(const Words& w, int k) {
  if constexpr (sizeof(T) == 4) {
    return __uint_as_float(w[k]);
  } else {
    T v;
    v.bits = (unsigned short)(k & 1 ? w[k / 2] >> 16 : w[k / 2]);
    if constexpr (__is_same(T, Brain16)) return __uint_as_float(k & 1 ? w[k / 2] & 0xFFFF0000u : w[k / 2] << 16);
    return to_f32(v);
  }
}

// The same with a place known at run time, the same for the wavefront.
template <class T>
__device__ __forceinline__ void set_entry(Words& w, u32 k, T v) {
  constexpr u32 each = 4 / sizeof(T);
  u32 bits = 0;
  __builtin_memcpy(&bits, &v, sizeof(T));
  const u32 shift = k % each * 16, hold = sizeof(T) == 4 ? 0 : ~(0xFFFFu << shift);
#pragma unroll
  for (u32 i = 0; i < 4; ++i)
    if (i == k / each) w[i] = (w[i] & hold) | bits << (sizeof(T) == 4 ? 0 : shift);
}
template <class T>
__device__ __forceinline__ T get_entry(const Words& w, u32 k) {
  constexpr u32 each = 4 / sizeof(T);
  u32 bits = 0;
#pragma unroll
  for (u32 i = 0; i < 4; ++i)
    if (i == k / each) bits = w[i];
  if (sizeof(T) == 2) bits >>= k % each * 16;
  T v;
  __builtin_memcpy(&v, &bits, sizeof(T));
  return v;
}
template <class T>
__device__ __forceinline__ T none_entry() {
  const u32 w = NoneWord<T>::value;
  T v;
  __builtin_memcpy(&v, &w, sizeof(T));
  return v;
}

// exp(d / tau) for d <= 0.  32-bit rows make up for the rounding of d log2(e) / tau, which
// grows with |d|; of 16-bit ones its 1e-6 is lost in the gradient's rounding, and terms so far
// below the top do not count in the sum.
struct Exponent {
  float hi, lo;  // log2(e) / tau
  template <class T>
  __device__ __forceinline__ float of(float d) const {
    const float t = d * hi;
    const float e = __builtin_amdgcn_exp2f(t);
    if constexpr (sizeof(T) == 2) return e;
    // past -150 the result is 0, also where t is infinite (d of a masked entry)
    const float r = t > -150.f ? __builtin_fmaf(d, lo, __builtin_fmaf(d, hi, -t)) : 0.f;
    return __builtin_fmaf(e * 0.693147182f, r, e);
  }
};

// A row's sums: what the gradient and the loss need of it.
struct RowSums {
  float top, rest, token;  // M, R, x_a
};

struct RowEnd {
  double lp;
  float total;   // s
  bool absent;   // the token's weight is 0
};

__device__ __forceinline__ RowEnd end_of(const VocabArgs& a, const RowSums& r) {
  RowEnd e;
  const double d = ((double)r.token - (double)r.top) * a.inverse_temperature;
  e.total = r.rest + expf((float)d);
  e.absent = false;
  if (!(e.total < __builtin_huge_valf())) {  // the row holds a NaN or +inf
    e.lp = __builtin_nan("");
  } else if (r.token == kNone) {
    e.lp = -__builtin_huge_val();
    e.absent = true;
  } else if (r.token == r.top) {
    e.lp = -(double)log1pf(r.rest);
  } else {
    e.lp = d - (double)logf(e.total);
    e.absent = (float)e.lp == kNone;
  }
  return e;
}

// e^q - 1 - q: near 0 by its series, where the difference would lose its digits (the next
// term is below 2^-26 of the sum).
__device__ __forceinline__ float kl_of(float q) {
  if (__builtin_fabsf(q) >= 0.5f) return expm1f(q) - q;
  float p = 1.f / 362880;
  p = __builtin_fmaf(p, q, 1.f / 40320);
  p = __builtin_fmaf(p, q, 1.f / 5040);
  p = __builtin_fmaf(p, q, 1.f / 720);
  p = __builtin_fmaf(p, q, 1.f / 120);
  p = __builtin_fmaf(p, q, 1.f / 24);
  p = __builtin_fmaf(p, q, 1.f / 6);
  p = __builtin_fmaf(p, q, 0.5f);
  return p * q * q;
}

struct RowTerms {
  double loss = 0, kl = 0;
  u32 clipped = 0;
  float c = 0;  // dloss / dlp, d_loss among it
};

__device__ __forceinline__ RowTerms terms_of(const VocabArgs& a, u64 t, const RowEnd& e, double d_loss, double share) {
  RowTerms o;
  if (a.given) {
    o.c = (float)((double)a.given[t] * d_loss);
    return o;
  }
  if (!a.policy || e.absent) return o;
  const float adv = a.advantages[t];
  const float ratio = expf((float)(e.lp - (double)a.old[t]));
  const float cut = __builtin_fminf(__builtin_fmaxf(ratio, a.clip_low), a.clip_high);
  const bool clipped = cut * adv < ratio * adv;
  double loss = -(double)adv * (double)(clipped ? cut : ratio);
  double slope = clipped ? 0.0 : -(double)adv * (double)ratio;
  const double w = a.weights ? (double)a.weights[t] : share;
  if (a.ref) {
    const float q = (float)((double)a.ref[t] - e.lp);
    const double k = (double)kl_of(q);
    o.kl = w * k;
    if (a.kl_weight > 0.f) {  // with weight 0 the term may be infinite (of a token masked by the lowest value)
      loss += (double)a.kl_weight * k;
      slope -= (double)a.kl_weight * (double)expm1f(q);
    }
  }
  o.loss = w * loss;
  o.clipped = clipped;
  o.c = (float)(w * slope * d_loss);
  return o;
}

__device__ __forceinline__ bool row_live(const VocabArgs& a, u64 t) {
  const int64_t k = a.tokens[t];
  return (!a.mask || a.mask[t]) && k >= 0 && (u64)k < a.V;
}

// Sum of one value per thread over the block, in a fixed order; every thread has it.
template <int WAVES, class S>
__device__ __forceinline__ S block_total(S v, S* wave_tot) {
#pragma unroll
  for (int d = kWave / 2; d; d >>= 1) v += __shfl_xor(v, d);
  if (lane_id() == 0) wave_tot[threadIdx.x / kWave] = v;
  lds_barrier();
  S s = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) s += wave_tot[w];
  lds_barrier();
  return s;
}

__device__ __forceinline__ void st_double(double* p, double v) { st_agent((u64*)p, __builtin_bit_cast(u64, v)); }
__device__ __forceinline__ double ld_double(const double* p) { return __builtin_bit_cast(double, ld_agent((const u64*)p)); }

}  // namespace

// The live rows, in kCountBlocks parts at most, and the ticket at 0.
__global__ __launch_bounds__(kCountThreads) void vocab_count_kernel(VocabArgs a) {
  __shared__ u32 s_n[kCountThreads / kWave];
  const VocabScratch sc = vocab_scratch(a.scratch);
  u32 n = 0;
  for (u64 t = (u64)blockIdx.x * kCountThreads + threadIdx.x; t < a.T; t += (u64)gridDim.x * kCountThreads)
    n += row_live(a, t);
  n = block_total<kCountThreads / kWave>(n, s_n);
  if (threadIdx.x == 0) {
    sc.live[blockIdx.x] = n;
    if (blockIdx.x == 0) *sc.ticket = 0;
  }
}

// A team of TEAM threads takes a row, N vectors of it per thread in registers; of a longer row
// (MULTI) that many at a time, the last of them staying for the gradient.
template <class T, int TEAM, int N, bool GRAD, bool MULTI>
__global__ __launch_bounds__(TEAM < 256 ? 256 : TEAM) void vocab_kernel(VocabArgs a) {
  constexpr int kBlock = TEAM < 256 ? 256 : TEAM, kTeams = kBlock / TEAM, kTeamWaves = TEAM / kWave;
  constexpr int kBlockWaves = kBlock / kWave;
  constexpr u32 W = 16 / sizeof(T);
  __shared__ float s_top[2][kBlockWaves], s_rest[2][kBlockWaves], s_token[2][kTeams];
  __shared__ double s_d[kBlockWaves];
  __shared__ u32 s_n[kBlockWaves], s_last;
  const VocabScratch sc = vocab_scratch(a.scratch);
  const u32 wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const u32 team = wave / kTeamWaves, tid = threadIdx.x % TEAM, base = wave % kTeamWaves * kWave;
  const Exponent ex = {a.exponent_hi, a.exponent_lo};
    u32 n = 0;
  if (a.policy)
    for (u32 i = 0; i < a.count_blocks; ++i) n += sc.live[i];
  const double share = n ? 1.0 / (double)n : 0.0;
  const double d_loss = GRAD ? (double)(a.d_loss ? *a.d_loss : 1.f) * (double)a.d_loss_scale : 0.0;
  RowTerms sum;
  u32 turn = 0;
  for (u64 t = (u64)blockIdx.x * kTeams + team; t < a.T; t += (u64)gridDim.x * kTeams) {
    const T* x = reinterpret_cast<const T*>(a.x) + t * a.ld;
    T* dx = GRAD ? reinterpret_cast<T*>(a.d_x) + t * a.V : nullptr;
    // vectors between the 16-byte boundaries of what is written, or of what is read
    u32 head = (u32)(-(uintptr_t)(GRAD ? (const T*)dx : x) & 15) / (u32)sizeof(T);
    if (head > a.V) head = (u32)a.V;
    const u32 nvec = (u32)(a.V - head) / W;
    const u32 edges = (u32)a.V - nvec * W, mine = tid < head ? tid : nvec * W + tid;  // entry of this thread's edge
    const T* xv = x + head;
    T* dv = GRAD ? dx + head : nullptr;
    const u32 segments = MULTI ? (nvec + TEAM * N - 1) / (TEAM * N) : 1;
    auto store = [&](u32 j, const Words& w) {
      __builtin_nontemporal_store(w, reinterpret_cast<Words*>(dv + (u64)j * W));
    };
    auto zero_row = [&]() {
      for (u32 j = tid; j < nvec; j += TEAM) store(j, Words{0, 0, 0, 0});
      T z;
      from_f32(0.f, z);
      if (tid < edges) dx[mine] = z;
    };
    if (!row_live(a, t) || (GRAD && a.given && a.given[t] == 0.f)) {
      if (GRAD) zero_row();
      if (tid == 0) {
        if (a.logprobs) a.logprobs[t] = 0.f;
        if (a.pairs) sc.lp[t] = 0;
      }
      continue;
    }
    const u32 token = (u32)a.tokens[t];
    // the token's vector, if it is in one: slot of which thread's, and the entry in it
    const u32 in_vec = token - head;
    const bool in_vecs = token >= head && in_vec < nvec * W;
    const u32 slot = in_vec / W / TEAM, owner = in_vec / W % TEAM, place = in_vec % W;
    const bool own_wave = in_vecs && owner / kWave * kWave == base;
    float edge = kNone, x_token = kNone;
    if (tid < edges) {
      edge = to_f32(x[mine]);
      if (mine == token) {
        x_token = edge;
        edge = kNone;
      }
    }
    float top = edge > kLowest ? edge : kLowest, rest[4] = {0.f, 0.f, 0.f, 0.f};
    Words v[N];
    u32 first = 0;  // the first vector of the segment
    auto load = [&]() {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const u32 j = first + i * TEAM + tid;
        if (first + i * TEAM + base >= nvec) continue;
        v[i] = Words{NoneWord<T>::value, NoneWord<T>::value, NoneWord<T>::value, NoneWord<T>::value};
        if (j < nvec) v[i] = __builtin_nontemporal_load(reinterpret_cast<const typename AnyWords<T>::type*>(xv + (u64)j * W));
      }
    };
    auto slot_of = [&]() { return own_wave && slot >= first / TEAM && slot < first / TEAM + N ? (int)(slot - first / TEAM) : -1; };
    for (u32 seg = 0; seg < segments; ++seg) {
      first = seg * TEAM * N;
      load();
      const int at = slot_of();
      const float before = top;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (first + i * TEAM + base >= nvec) continue;
        if (i == at && tid == owner) {
          x_token = to_f32(get_entry<T>(v[i], place));
          set_entry<T>(v[i], place, none_entry<T>());
        }
#pragma unroll
        for (u32 k = 0; k < W; k += 2) top = max3(top, entry<T>(v[i], k), entry<T>(v[i], k + 1));
      }
      if (MULTI && seg) {
        const float f = ex.of<T>(before - top);
#pragma unroll
        for (int k = 0; k < 4; ++k) rest[k] *= f;
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (first + i * TEAM + base >= nvec) continue;
#pragma unroll
        for (u32 k = 0; k < W; ++k) rest[k % 4] += ex.of<T>(entry<T>(v[i], k) - top);
      }
    }
    rest[0] += ex.of<T>(edge - top);
    // over the lanes, then over the team's wavefronts
    RowSums row;
    row.top = group_reduce<kWave>(top, max_f);
    row.rest = group_reduce<kWave>((rest[0] + rest[1] + (rest[2] + rest[3])) * ex.of<T>(top - row.top), add_f);
    if constexpr (kTeamWaves == 1) {
      const u32 lane = in_vecs ? owner : (token < head ? token : token - nvec * W);
      row.token = __uint_as_float((u32)__builtin_amdgcn_readlane((int)__float_as_uint(x_token), (int)lane));
    } else {
      const u32 b = turn++ & 1;  // written again only behind the next row's barrier
      if (tid % kWave == 0) {
        s_top[b][wave] = row.top;
        s_rest[b][wave] = row.rest;
      }
      if (in_vecs ? tid == owner : (tid < edges && mine == token)) s_token[b][team] = x_token;
      lds_barrier();
      const u32 from = team * kTeamWaves + tid % kTeamWaves;
      const float m = s_top[b][from], s = s_rest[b][from];
      row.top = group_reduce<kTeamWaves>(m, max_f);
      row.rest = group_reduce<kTeamWaves>(s * ex.of<T>(m - row.top), add_f);
      row.token = s_token[b][team];
    }
    if (row.token > row.top) {
      row.rest *= ex.of<T>(row.top - row.token);
      row.top = row.token;
    }
    const RowEnd end = end_of(a, row);
    const RowTerms o = terms_of(a, t, end, d_loss, share);
    sum.loss += o.loss;
    sum.kl += o.kl;
    sum.clipped += o.clipped;
    if (tid == 0) {
      if (a.logprobs) a.logprobs[t] = (float)end.lp;
      if (a.pairs) sc.lp[t] = end.lp;
    }
    if constexpr (GRAD) {
      if (o.c == 0.f || end.absent) {
        zero_row();
        continue;
      }
      const float c = (float)((double)o.c * a.inverse_temperature);
      const float scale = -c / end.total;
      T at_token;
      from_f32(c * (row.rest / end.total), at_token);
      if (tid < edges) {
        T g;
        from_f32(scale * ex.of<T>(edge - row.top), g);
        dx[mine] = mine == token ? at_token : g;
      }
      for (u32 seg = segments; seg-- > 0;) {
        if (MULTI && (seg + 1 < segments)) {
          first = seg * TEAM * N;
          load();
        }
        const int at = slot_of();
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const u32 j = first + i * TEAM + tid;
          if (first + i * TEAM + base >= nvec) continue;
          Words w;
#pragma unroll
          for (u32 k = 0; k < 4; ++k) {
            T g[4 / sizeof(T)];
#pragma unroll
            for (u32 h = 0; h < 4 / sizeof(T); ++h)
              from_f32(scale * ex.of<T>(entry<T>(v[i], k * (4 / sizeof(T)) + h) - row.top), g[h]);
            u32 bits;
            __builtin_memcpy(&bits, g, 4);
            w[k] = bits;
          }
          if (i == at && tid == owner) set_entry<T>(w, place, at_token);
          if (j < nvec) store(j, w);
        }
      }
    }
  }
  if (!a.policy) return;
  // the block's terms, then the blocks' by the last one to end: sums in a fixed order
  if (tid) sum = RowTerms();
  sum.loss = block_total<kBlockWaves>(sum.loss, s_d);
  sum.kl = block_total<kBlockWaves>(sum.kl, s_d);
  sum.clipped = block_total<kBlockWaves>(sum.clipped, s_n);
  if (threadIdx.x == 0) {
    BlockTerms* o = sc.terms + blockIdx.x;
    st_double(&o->loss, sum.loss);
    st_double(&o->kl, sum.kl);
    st_agent(&o->clipped, (u64)sum.clipped);
    drain_memory_ops();
    s_last = __hip_atomic_fetch_add(sc.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1 == gridDim.x;
  }
  __syncthreads();
  if (!s_last) return;
  double loss = 0, kl = 0, clipped = 0;  // counts below 2^53
  for (u32 i = threadIdx.x; i < gridDim.x; i += kBlock) {
    loss += ld_double(&sc.terms[i].loss);
    kl += ld_double(&sc.terms[i].kl);
    clipped += (double)ld_agent(&sc.terms[i].clipped);
  }
  loss = block_total<kBlockWaves>(loss, s_d);
  kl = block_total<kBlockWaves>(kl, s_d);
  clipped = block_total<kBlockWaves>(clipped, s_d);
  if (threadIdx.x == 0) {
    *a.loss = (float)loss;
    *a.kl = (float)kl;
    *a.clipped = (int64_t)clipped;
    *a.rows = (int64_t)n;
  }
}

// The pairs' losses, and every row's coefficient.  A block takes a pair at a time.
__global__ __launch_bounds__(kPairThreads) void pair_kernel(PairArgs a) {
  constexpr int kWaves = kPairThreads / kWave;
  __shared__ double s_d[kWaves];
  __shared__ u64 s_n[kWaves];
  __shared__ u32 s_last;
  const VocabScratch sc = vocab_scratch(a.v.scratch);
  // offsets as far as they rise, within [0, T]: an offset below an earlier one counts as that
  auto offset = [&](u64 i) {
    int64_t m = 0;
    for (u64 k = threadIdx.x; k <= i; k += kPairThreads) m = a.offsets[k] > m ? a.offsets[k] : m;
#pragma unroll
    for (int d = kWave / 2; d; d >>= 1) {
      const int64_t o = __shfl_xor(m, d);
      m = o > m ? o : m;
    }
    if (lane_id() == 0) s_n[threadIdx.x / kWave] = (u64)m;
    lds_barrier();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) m = (int64_t)s_n[w] > m ? (int64_t)s_n[w] : m;
    lds_barrier();
    return (u64)m < a.v.T ? (u64)m : a.v.T;
  };
  double total = 0;
  u64 rows = 0;
  for (u64 p = blockIdx.x; p < a.pairs; p += gridDim.x) {
    u64 start[2], end[2], live[2];
    double ratio[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u64 s = p + h * a.pairs;
      start[h] = offset(s);
      end[h] = offset(s + 1);
      double own = 0, ref = 0;
      u64 n = 0;
      for (u64 t = start[h] + threadIdx.x; t < end[h]; t += kPairThreads) {
        if (!row_live(a.v, t)) continue;
        ++n;
        const double lp = sc.lp[t];
        if (lp == -__builtin_huge_val()) continue;  // a token of weight 0 adds nothing
        own += lp;
        if (a.v.ref) ref += (double)a.v.ref[t];
      }
      own = block_total<kWaves>(own, s_d);
      ref = block_total<kWaves>(ref, s_d);
      live[h] = block_total<kWaves>(n, s_n);
      const double mean = a.average && live[h] ? 1.0 / (double)live[h] : 1.0;
      ratio[h] = (own - ref) * mean;
      if (threadIdx.x == 0) a.sequence_logprobs[s] = (float)(own * mean);
      rows += live[h];
    }
    const double z = a.beta * (ratio[0] - ratio[1]) - a.margin;
    const double e = exp(-fabs(z)), tail = log1p(e);  // softplus(z) = max(z, 0) + tail
    const double up = (z < 0 ? -z : 0.0) + tail, down = (z > 0 ? z : 0.0) + tail;
    const double sigmoid = (z < 0 ? e : 1.0) / (1.0 + e), other = (z < 0 ? 1.0 : e) / (1.0 + e);
    const double keep = 1.0 - a.smoothing;
    total += z == z ? keep * up + a.smoothing * down : z;
    if (threadIdx.x == 0) a.margins[p] = (float)z;
    const double slope = a.beta / (double)a.pairs * (a.smoothing * sigmoid - keep * other);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const double mean = a.average && live[h] ? 1.0 / (double)live[h] : 1.0;
      const float c = (float)((h ? -slope : slope) * mean);
      for (u64 t = start[h] + threadIdx.x; t < end[h]; t += kPairThreads)
        a.coefficients[t] = row_live(a.v, t) ? c : 0.f;
    }
    if (p == 0)
      for (u64 t = threadIdx.x; t < start[0]; t += kPairThreads) a.coefficients[t] = 0.f;
    if (p == a.pairs - 1)
      for (u64 t = end[1] + threadIdx.x; t < a.v.T; t += kPairThreads) a.coefficients[t] = 0.f;
  }
  if (threadIdx.x == 0) {
    st_double(&sc.terms[blockIdx.x].loss, total);
    st_agent(&sc.terms[blockIdx.x].clipped, rows);
    drain_memory_ops();
    s_last = __hip_atomic_fetch_add(sc.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1 == gridDim.x;
  }
  __syncthreads();
  if (!s_last) return;
  double loss = 0;
  u64 n = 0;
  for (u32 i = threadIdx.x; i < gridDim.x; i += kPairThreads) {
    loss += ld_double(&sc.terms[i].loss);
    n += ld_agent(&sc.terms[i].clipped);
  }
  loss = block_total<kWaves>(loss, s_d);
  n = block_total<kWaves>(n, s_n);
  if (threadIdx.x == 0) {
    *a.v.loss = (float)(loss / (double)a.pairs);
    *a.v.rows = (int64_t)n;
  }
}

namespace {

template <class T, int TEAM, int N, bool GRAD, bool MULTI>
hipError_t vocab_launch(const VocabArgs& a, hipStream_t s) {
  constexpr int kBlock = TEAM < 256 ? 256 : TEAM, kTeams = kBlock / TEAM;
  static const u32 fit = resident_blocks(vocab_kernel<T, TEAM, N, GRAD, MULTI>, kBlock);
  const u64 rounds = (a.T + kTeams - 1) / kTeams;
  u64 blocks = rounds < fit ? rounds : fit;
  if (blocks > kVocabMaxBlocks) blocks = kVocabMaxBlocks;
  if (!blocks) blocks = 1;
  vocab_kernel<T, TEAM, N, GRAD, MULTI><<<(u32)blocks, kBlock, 0, s>>>(a);
  return hipGetLastError();
}

template <class T, bool GRAD>
hipError_t vocab_shape(const VocabArgs& a, hipStream_t s) {
  const u64 bytes = a.V * sizeof(T);
  if (bytes <= 64 * 16 * 4) return vocab_launch<T, 64, 4, GRAD, false>(a, s);
  if (bytes <= 64 * 16 * 16) return vocab_launch<T, 64, 16, GRAD, false>(a, s);
  if (bytes <= 256 * 16 * 16) return vocab_launch<T, 256, 16, GRAD, false>(a, s);
  if (bytes <= 512 * 16 * 16) return vocab_launch<T, 512, 16, GRAD, false>(a, s);
  if (bytes <= 1024 * 16 * 16) return vocab_launch<T, 1024, 16, GRAD, false>(a, s);
  return vocab_launch<T, 1024, 16, GRAD, true>(a, s);
}

template <class T>
hipError_t vocab_grad(const VocabArgs& a, hipStream_t s) {
  return a.d_x ? vocab_shape<T, true>(a, s) : vocab_shape<T, false>(a, s);
}

}  // namespace

size_t vocab_scratch_bytes(u64 T) { return kVocabHead + kVocabMaxBlocks * sizeof(BlockTerms) + 8 * T; }

hipError_t launch_vocab(VocabArgs a, int dtype, hipStream_t s) {
  if (a.policy || a.pairs) {
    const u64 rounds = (a.T + kCountThreads * 4 - 1) / (kCountThreads * 4);
    a.count_blocks = rounds < 1 ? 1 : rounds < kCountBlocks ? (u32)rounds : kCountBlocks;
    vocab_count_kernel<<<a.count_blocks, kCountThreads, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!a.T && !a.policy) return hipSuccess;
  if (dtype == PROFK_FP32) return vocab_grad<float>(a, s);
  if (dtype == PROFK_FP16) return vocab_grad<Half16>(a, s);
  return vocab_grad<Brain16>(a, s);
}

hipError_t launch_pairs(const PairArgs& a, hipStream_t s) {
  pair_kernel<<<a.pairs < kPairBlocks ? (u32)a.pairs : kPairBlocks, kPairThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace profk
