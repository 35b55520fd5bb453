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
//
// Bound by HBM: a row is read once into registers, where its top, its sum and its gradient are
// taken from, and the gradient written; each row's end is one thread's, in 64 bits.  Kernels'
// times (MI355X, whose copy reaches 5.0 TB/s and whose reads alone up to 6.5):
//   log-probabilities  4096 x 131072 bf16 217 us (4.9 TB/s), 4099 x 50257 fp32 with 30 % of the rows
//                      masked, which are not read, 111 (5.2), 12000 x 65536 bf16 with 40 % masked 167
//                      (5.7), one row of 32000 6.8
//   gradient           4096 x 131072 bf16 478 to 518 (4.1 to 4.5 TB/s read and written), the 12000 x 65536
//                      463 (5.4)
//   policy loss and gradient  8192 x 131072 bf16 890 to 980 (4.4 to 4.8) and 6 for the sum of the terms,
//                      3001 x 50257 fp16 with 40 % masked 105 (4.6) and 5.7, 48 x 32000 bf16 in slices 4.7
//                      and 6.6
//   pairs              10.8 us for 16 pairs of 12000 rows
// Beside that exponentials and sums take 45 % (32 bits) to 84 % of the vector units' cycles, and all of
// them in the 12000 x 65536 log-probabilities.
#include "ops_device.h"

namespace profk {

namespace {

constexpr int kCountThreads = 1024;
constexpr u32 kCountBlocks = 64;  // a lane per part of the count
constexpr int kTermThreads = 256;
constexpr u32 kTermBlocks = 512;
constexpr int kPairThreads = 512;
constexpr u32 kPairBlocks = 1024;
constexpr u32 kSlices = 64;       // most parts of a row: a lane each
constexpr u64 kSplitRows = 512;   // most rows that are split

// A row's terms of the policy loss (times its weight, where there are weights), or a block's sums
// of them or of its pairs.
struct Terms {
  double loss, kl;
  u32 clipped, rows;
};
// Of a slice of a row that is split.
struct Part {
  double rest;
  float top;
};

// All of it is written before it is read within a call.
struct VocabScratch {
  u32* last;      // a ticket for the blocks that add up
  u32* live;      // kCountBlocks parts of the number of live rows
  Terms* blocks;  // of each block that adds up: kTermBlocks or kPairBlocks at most
  Terms* rows;    // T, with the policy loss
  double* lp;     // T, with the preference loss
  Part* parts;    // T * kSlices, where rows are split
};
__host__ __device__ inline VocabScratch vocab_scratch(char* s, u64 T) {
  VocabScratch v;
  v.last = (u32*)s;
  v.live = (u32*)(s + 128);
  v.blocks = (Terms*)(s + 512);
  s += 512 + sizeof(Terms) * (kTermBlocks > kPairBlocks ? kTermBlocks : kPairBlocks);
  v.rows = (Terms*)s;
  v.lp = (double*)s;
  v.parts = (Part*)(s + sizeof(Terms) * T);
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

// exp((x - top) / tau).  log2(e) / tau is taken to 48 bits, hi + lo: the rounding of its upper half
// alone would make every sum too large or too small by some 1e-7, and a sequence's with its length.
struct Exponent {
  float hi, lo;
  __device__ __forceinline__ float of(float d) const {  // of a difference, for all of them: -inf too
    return __builtin_amdgcn_exp2f(__builtin_fmaf(d, lo, d * hi));
  }
  // In 64 bits, where a likely token's whole R takes the factor; a part of a row joins the others by
  // `of`, whose rounding, d 2^-24 of a part of weight e^-d, is below 3e-8 of the sum.
  __device__ __forceinline__ double exactly(float d) const { return exp2((double)d * ((double)hi + (double)lo)); }
};

// The same from x itself: x hi + (-top hi), each in one rounding, is as exact as x - top and a
// product, in one instruction less; what the second product's rounding left is a factor of all
// terms, `left`.  Where a top's product passes 2^31 that factor
// would leave 32 bits' range (half a unit is 64 there), and any other value is at least 64 below it:
// the terms are 1 or, as 2^-64 of it or less, 0, which a power of two in place of the factors gives,
// whose products are exact; one that puts the top's at 2^40 puts the next one 2^15 below.
struct Shifted {
  float hi, lo, from;
  __device__ __forceinline__ Shifted(const Exponent& ex, float top, bool both) {
    from = -top * ex.hi;
    const bool fits = __builtin_fabsf(from) < 0x1p31f || !(__builtin_fabsf(top) < __builtin_huge_valf());
    const float power = __builtin_ldexpf(1.f, 40 - __builtin_amdgcn_frexp_expf(top));
    hi = fits ? ex.hi : both ? 0.5f * power : power;
    lo = fits ? ex.lo : 0.5f * power;
    from = fits ? from : -top * power;
  }
  // sum * left.  Rounded to 32 bits, left would put its own error on the whole row; 1 and the rest
  // apart keep it where |top| / tau is below 2^14.
  __device__ __forceinline__ double whole(double sum, float top, bool both) const {
    if (__builtin_fabsf(from) >= 0x1p31f) return sum;  // a power of two
    const float part = __builtin_fmaf(-top, hi, -from), rest = both ? __builtin_fmaf(-top, lo, part) : part;
    const float z = rest * 0.693147181f;
    const bool small = __builtin_fabsf(rest) < 0x1p-10f;
    const float most = small ? 1.f : __builtin_amdgcn_exp2f(rest), more = small ? __builtin_fmaf(0.5f * z, z, z) : 0.f;
    return __builtin_fma(sum, (double)more, sum * (double)most);
  }
  // BOTH: with lo.  A 16-bit gradient's rounding hides what it adds.  It counts where x is large:
  // below half a unit of t it changes nothing, which leaves a row's sum off by 1e-8 to 3e-8.
  template <bool BOTH>
  __device__ __forceinline__ float of(float x) const {
    const float t = __builtin_fmaf(x, hi, from);
    return __builtin_amdgcn_exp2f(BOTH ? __builtin_fmaf(x, lo, t) : t);
  }
};

// Sum over groups of G lanes in 64 bits.
template <int G>
__device__ __forceinline__ double lanes_sum(double v) {
#pragma unroll
  for (int d = 1; d < G; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

// A row's sums: what the gradient and the loss need of it.
struct RowSums {
  float top, token;  // M, x_a
  double rest;       // R
};

struct RowEnd {
  double lp, total;  // total: s
  bool absent;       // the token's weight is 0
};

__device__ __forceinline__ RowEnd end_of(const VocabArgs& a, const RowSums& r) {
  RowEnd e;
  const double d = ((double)r.token - (double)r.top) * a.inverse_temperature;
  e.total = r.rest + exp(d);
  e.absent = false;
  if (!(e.total < __builtin_huge_val())) {  // the row holds a NaN or +inf
    e.lp = __builtin_nan("");
  } else if (r.token == kNone) {
    e.lp = -__builtin_huge_val();
    e.absent = true;
  } else if (r.token == r.top) {
    e.lp = -log1p(r.rest);
  } else {
    e.lp = d - log(e.total);
    e.absent = (float)e.lp == kNone;
  }
  return e;
}

struct RowTerms {
  double loss = 0, kl = 0;
  bool clipped = false;
  float c = 0;  // dloss / dlp, d_loss and the share among it
};

// What a row's terms need from memory, on its way before the row itself.
struct RowInputs {
  float given = 0, old = 0, advantage = 0, ref = 0, weight = 0;
  __device__ __forceinline__ RowInputs(const VocabArgs& a, u64 t) {
    if (a.given) given = a.given[t];
    if (!a.policy) return;
    old = a.old[t];
    advantage = a.advantages[t];
    if (a.ref) ref = a.ref[t];
    if (a.weights) weight = a.weights[t];
  }
};

// share: a row's weight in the gradient where none are given (the sums are scaled when added up)
__device__ __forceinline__ RowTerms terms_of(const VocabArgs& a, const RowInputs& in, const RowEnd& e, double d_loss,
                                             double share) {
  RowTerms o;
  if (a.given) {
    o.c = (float)((double)in.given * d_loss);
    return o;
  }
  if (!a.policy || e.absent) return o;
  const double adv = (double)in.advantage;
  const double ratio = exp(e.lp - (double)in.old);
  const double cut = __builtin_fmin(__builtin_fmax(ratio, a.clip_low), a.clip_high);
  const bool clipped = cut * adv < ratio * adv;
  const double w = a.weights ? (double)in.weight : 1.0;
  double loss = -adv * (clipped ? cut : ratio);
  double slope = clipped ? 0.0 : -adv * ratio;
  double rise = 0, k = 0;
  // with weight 0 the term may be infinite (of a token masked by the lowest value)
  const double kl_weight = a.ref ? a.kl_weight : 0.0;
  if (a.ref) {
    const double q = (double)in.ref - e.lp;
    rise = expm1(q);
    k = rise - q;
  }
  auto with_kl = [&]() {
    if (kl_weight > 0) {
      loss += kl_weight * k;
      slope -= kl_weight * rise;
    }
  };
  with_kl();
  o.kl = w * k;
  o.loss = w * loss;
  if (__builtin_expect(!(__builtin_fabs(o.loss + o.kl) < __builtin_huge_val()), 0)) {
    // A ratio and an e^q that 64 bits do not hold are finite numbers all the same: a weight or an
    // advantage of 0 makes 0 of them.
    const bool numbers = e.lp == e.lp && in.old == in.old && in.advantage - in.advantage == 0 && in.ref == in.ref;
    if (w == 0 && numbers) {
      o.loss = o.kl = slope = 0;
    } else if (adv == 0 && ratio == __builtin_huge_val()) {
      loss = slope = 0;
      with_kl();
      o.loss = w * loss;
    }
  }
  o.clipped = clipped;
  o.c = (float)((a.weights ? w : share) * slope * d_loss);
  return o;
}

__device__ __forceinline__ bool row_live(const VocabArgs& a, u64 t) {
  const int64_t k = a.tokens[t];
  const unsigned char m = a.mask ? a.mask[t] : 1;  // both loads at once
  return (u32)(m != 0) & (u32)((u64)k < a.V);
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

// The live rows, in kCountBlocks parts at most.
__global__ __launch_bounds__(kCountThreads) void vocab_count_kernel(VocabArgs a) {
  __shared__ u32 s_n[kCountThreads / kWave];
  const VocabScratch sc = vocab_scratch(a.scratch, a.T);
  u32 n = 0;
  for (u64 t = (u64)blockIdx.x * kCountThreads + threadIdx.x; t < a.T; t += (u64)gridDim.x * kCountThreads)
    n += row_live(a, t);
  n = block_total<kCountThreads / kWave>(n, s_n);
  if (threadIdx.x == 0) sc.live[blockIdx.x] = n;
}

// The sums of a row that is split, from its parts, by one thread.
template <class T>
__device__ __forceinline__ RowSums sums_of(const VocabArgs& a, const Part* parts, u64 t) {
  const Exponent ex = {a.exponent_hi, a.exponent_lo};
  RowSums row = {kLowest, to_f32(reinterpret_cast<const T*>(a.x)[t * a.ld + (u64)a.tokens[t]]), 0};
  const Part* p = parts + t * a.slices;
#pragma unroll 4
  for (u32 i = 0; i < a.slices; ++i) row.top = max_f(row.top, p[i].top);
#pragma unroll 4
  for (u32 i = 0; i < a.slices; ++i) row.rest += p[i].rest * (double)ex.of(p[i].top - row.top);
  if (row.token > row.top) {
    row.rest *= ex.exactly(row.top - row.token);
    row.top = row.token;
  }
  return row;
}

// Block `block` of `blocks` adds up its rows' terms of the policy loss; the last one to end, the
// blocks' (sums in a fixed order).  Of rows that are split it works the terms out, a thread a row,
// and the log-probabilities.  (A ticket per 1024 rows, drawn by every row when its terms were
// written, was one launch less and took 8 ns a row: 131072 x 512 1080 us in place of 110; and a
// workgroup alone on its CU waited for it.)
template <class T>
__device__ __forceinline__ void add_terms(const VocabArgs& a, u32 block, u32 blocks) {
  constexpr int kWaves = kTermThreads / kWave;
  __shared__ double s_loss[kWaves], s_kl[kWaves];
  __shared__ u32 s_clipped[kWaves], s_rows[kWaves], s_last;
  const VocabScratch sc = vocab_scratch(a.scratch, a.T);
  Terms sum = {0, 0, 0, 0};
  for (u64 t = (u64)block * kTermThreads + threadIdx.x; t < a.T; t += (u64)blocks * kTermThreads) {
    const bool live = row_live(a, t);
    if (a.slices) {
      RowEnd end = {0, 1, false};
      if (live) {
        const RowInputs in(a, t);
        end = end_of(a, sums_of<T>(a, sc.parts, t));
        const RowTerms o = terms_of(a, in, end, 0, 0);
        sum.loss += o.loss;
        sum.kl += o.kl;
        sum.clipped += o.clipped;
      }
      if (a.logprobs) a.logprobs[t] = (float)end.lp;
    } else {
      const Terms o = sc.rows[t];
      sum.loss += o.loss;
      sum.kl += o.kl;
      sum.clipped += o.clipped;
    }
    sum.rows += live;
  }
  if (!a.policy) return;
  auto total = [&](double& loss, double& kl, u64& clipped, u64& rows) {
    loss = block_total<kWaves>(loss, s_loss);
    kl = block_total<kWaves>(kl, s_kl);
    clipped = block_total<kWaves>((u32)clipped, s_clipped);  // T < 2^31
    rows = block_total<kWaves>((u32)rows, s_rows);
  };
  double loss = sum.loss, kl = sum.kl;
  u64 clipped = sum.clipped, rows = sum.rows;
  total(loss, kl, clipped, rows);
  if (blocks > 1) {
    if (threadIdx.x == 0) {
      Terms* o = sc.blocks + block;
      st_double(&o->loss, loss);
      st_double(&o->kl, kl);
      st_agent((u64*)&o->clipped, rows << 32 | clipped);
      drain_memory_ops();
      s_last = __hip_atomic_fetch_add(sc.last, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1 == blocks;
    }
    __syncthreads();
    if (!s_last) return;
    loss = kl = 0;
    clipped = rows = 0;
    for (u32 i = threadIdx.x; i < blocks; i += kTermThreads) {
      loss += ld_double(&sc.blocks[i].loss);
      kl += ld_double(&sc.blocks[i].kl);
      const u64 both = ld_agent((const u64*)&sc.blocks[i].clipped);
      clipped += (u32)both;
      rows += both >> 32;
    }
    total(loss, kl, clipped, rows);
  }
  if (threadIdx.x == 0) {
    const double share = a.weights ? 1.0 : rows ? 1.0 / (double)rows : 0.0;
    *a.loss = (float)(loss * share);
    *a.kl = (float)(kl * share);
    *a.clipped = (int64_t)clipped;
    *a.rows = (int64_t)rows;
  }
}

template <class T>
__global__ __launch_bounds__(kTermThreads) void vocab_terms_kernel(VocabArgs a) {
  add_terms<T>(a, blockIdx.x, gridDim.x);
}

// WHOLE: a team takes a row.  PART: a block takes a slice of a row, and leaves its sums; one block
// more counts the live rows.  JOIN: a block takes a slice of a row again for its gradient, with the
// row's sums from all its parts; with the policy loss, blocks behind those add up the terms.
enum { kWhole, kPart, kJoin };

// A team of TEAM threads with N vectors per thread in registers; of more (MULTI) that many at a
// time, the last of them staying for the gradient.
// Wavefronts a SIMD: with 4 a gradient's 512 threads come twice to a CU, one's loads beside the
// other's sums; a forward pass holds fewer registers, and of 512 threads at 6 wavefronts there are
// three workgroups (12000 x 65536 bf16, 40 % masked, 189 us a call; at 5, with two, 212).  Of 256
// threads there are as many workgroups as wavefronts; at 6 rows in segments spill 19 to 25 vector
// registers (8192 x 131072 bf16 410 us at 5 and 666 at 6, 8192 x 30001 fp16 88 and 94, 40000 x 9001 bf16 183
// and 178).  What spills at these bounds: two vector registers of 16-bit forward rows of 512
// threads and in segments, 35 of gradients in segments; scalar ones, into lanes of a vector one: 42
// to 44 of the gradients, 24 of joins and forward segments.
constexpr int waves_of(int team, int n, bool grad, bool multi) { return team < 256 || n < 16 ? 1 : grad ? 4 : team == 256 ? 5 : 6; }

template <class T, int TEAM, int N, bool GRAD, bool MULTI, int MODE>
__global__ __launch_bounds__(TEAM < 256 ? 256 : TEAM, waves_of(TEAM, N, GRAD, MULTI)) void vocab_kernel(VocabArgs a) {
  constexpr int kBlock = TEAM < 256 ? 256 : TEAM, kTeams = kBlock / TEAM, kTeamWaves = TEAM / kWave;
  constexpr u32 W = 16 / sizeof(T);
  __shared__ float s_top[kBlock / kWave], s_token[kTeams];
  __shared__ double s_rest[kBlock / kWave];
  __shared__ u32 s_n[kBlock / kWave];
  const VocabScratch sc = vocab_scratch(a.scratch, a.T);
  const u32 wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const u32 team = wave / kTeamWaves, tid = threadIdx.x % TEAM, base = wave % kTeamWaves * kWave, lane = lane_id();
  const Exponent ex = {a.exponent_hi, a.exponent_lo};
  constexpr bool kSliced = MODE != kWhole;
  if constexpr (MODE == kJoin) {
    const u32 slices = (u32)a.T * a.slices;
    if (blockIdx.x >= slices) return add_terms<T>(a, blockIdx.x - slices, gridDim.x - slices);
  }
  const u32 slice = kSliced ? blockIdx.x % a.slices : 0;
  const u64 t = kSliced ? blockIdx.x / a.slices : a.row0 + (u64)blockIdx.x * kTeams + team;
  if constexpr (MODE == kPart) {
    if (t == a.T) {
      u32 n = 0;
      for (u64 r = tid; r < a.T; r += kBlock) n += row_live(a, r);
      n = block_total<kBlock / kWave>(n, s_n);
      if (tid == 0) {
        *sc.live = n;
        *sc.last = 0;
      }
    }
  }
  if (MODE == kWhole && t == 0 && tid == 0 && (a.policy || a.pairs)) *sc.last = 0;  // for the kernel behind this one
  if (t >= a.T) return;  // no barrier below joins teams of a wavefront each
  const T* x = reinterpret_cast<const T*>(a.x) + t * a.ld;
  T* dx = GRAD ? reinterpret_cast<T*>(a.d_x) + t * a.V : nullptr;
  // vectors between the 16-byte boundaries of what is written, or of what is read
  u32 head = (u32)(-(uintptr_t)(GRAD ? (const T*)dx : x) & 15) / (u32)sizeof(T);
  if (head > a.V) head = (u32)a.V;
  const u32 all = (u32)(a.V - head) / W;
  // this slice's vectors; the entries outside all vectors are the first slice's
  const u32 each = kSliced ? (all + a.slices - 1) / a.slices : all;
  const u32 from = slice * each < all ? slice * each : all, nvec = each < all - from ? each : all - from;
  const u32 edges = slice ? 0 : (u32)a.V - all * W, mine = tid < head ? tid : all * W + tid;  // this thread's edge
  const char* xv = reinterpret_cast<const char*>(x + head) + (u64)from * 16;
  char* dv = GRAD ? reinterpret_cast<char*>(dx + head) + (u64)from * 16 : nullptr;
  const u32 off = tid * 16;
  u32 first = 0;  // the segment's first vector
  // Vectors of this wavefront in the segment that begins at f; of the last of them, whether this
  // lane has one.
  auto count = [&](u32 f) {
    const u32 left = nvec > f + base ? (nvec - f - base + TEAM - 1) / TEAM : 0;
    return (int)(left < N ? left : N);
  };
  auto has = [&](u32 f, int i) { return f + i * TEAM + tid < nvec; };
  auto store = [&](int i, const Words& w) {
    __builtin_nontemporal_store(w, reinterpret_cast<Words*>(dv + (u64)(first + i * TEAM) * 16 + off));
  };
  auto zero_row = [&]() {
    for (u32 j = tid; j < nvec; j += TEAM) __builtin_nontemporal_store(Words{0, 0, 0, 0}, reinterpret_cast<Words*>(dv + (u64)j * 16));
    T z;
    from_f32(0.f, z);
    if (tid < edges) dx[mine] = z;
  };
  const u32 live_part = GRAD && a.policy && !a.weights && lane < a.count_blocks ? sc.live[lane] : 0;
  const RowInputs in(a, t);
  const double d_loss = GRAD ? (double)(a.d_loss ? *a.d_loss : 1.f) * (double)a.d_loss_scale : 0.0;
  const bool live = row_live(a, t);
  if (!live || (GRAD && a.given && in.given == 0.f)) {
    if (GRAD) zero_row();
    if (MODE == kWhole && tid == 0) {
      if (a.logprobs) a.logprobs[t] = 0.f;
      if (a.policy) sc.rows[t] = Terms{0, 0, 0, 0};
      if (a.pairs) sc.lp[t] = 0;
    }
    return;
  }
  const u32 token = (u32)a.tokens[t];
  // the token's vector, if it is in one of this slice: slot of which thread's, and the entry in it
  const u32 in_vec = token - head - from * W;
  const bool in_vecs = token >= head + from * W && in_vec < nvec * W;
  const u32 slot = in_vec / W / TEAM, owner = in_vec / W % TEAM, place = in_vec % W;
  const bool own_wave = in_vecs && owner / kWave * kWave == base;
  Words v[N];
  auto load_one = [&](u32 f, int i, int n) {
    if (i + 1 == n) v[i] = Words{NoneWord<T>::value, NoneWord<T>::value, NoneWord<T>::value, NoneWord<T>::value};
    if (i + 1 < n || has(f, i))
      v[i] = __builtin_nontemporal_load(
          reinterpret_cast<const typename AnyWords<T>::type*>(xv + (u64)(f + i * TEAM) * 16 + off));
  };
  auto load = [&]() {
    const int n = count(first);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) load_one(first, i, n);
  };
  auto slot_of = [&]() { return own_wave && slot >= first / TEAM && slot < first / TEAM + N ? (int)(slot - first / TEAM) : -1; };
  const u32 segments = MULTI && nvec > TEAM * N ? (nvec + TEAM * N - 1) / (TEAM * N) : 1;
  float edge = kNone;
  RowSums row;
  if constexpr (MODE == kJoin) {
    first = (segments - 1) * (TEAM * N);
    load();
    if (tid < edges && mine != token) edge = to_f32(x[mine]);
    const Part p = lane < a.slices ? sc.parts[t * a.slices + lane] : Part{0, kLowest};
    row.top = group_reduce<kWave>(p.top, max_f);
    row.rest = lanes_sum<kWave>(p.rest * (double)ex.of(p.top - row.top));
    row.token = to_f32(x[token]);
    const int at = slot_of();
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i == at && tid == owner) set_entry<T>(v[i], place, none_entry<T>());
  } else {
    float x_token = kNone;
    if (tid < edges) {
      edge = to_f32(x[mine]);
      if (mine == token) {
        x_token = edge;
        edge = kNone;
      }
    }
    float top = kLowest;  // of the wavefront
    double rest = 0;
    load();
    for (u32 seg = 0; seg < segments; ++seg) {
      first = seg * TEAM * N;
      const int at = slot_of(), n = count(first), next = seg + 1 < segments ? count(first + TEAM * N) : 0;
      const float before = top;
      float m = seg == 0 && edge > kLowest ? edge : kLowest;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (i >= n) continue;
        if (i == at && tid == owner) {
          x_token = to_f32(get_entry<T>(v[i], place));
          set_entry<T>(v[i], place, none_entry<T>());
        }
#pragma unroll
        for (u32 k = 0; k < W; k += 2) m = max3(m, entry<T>(v[i], k), entry<T>(v[i], k + 1));
      }
      top = max_f(top, __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(group_reduce<kWave>(m, max_f)))));
      if (MULTI && seg) rest *= (double)ex.of(before - top);
      const Shifted sh(ex, top, true);
      double sum = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (i >= n) continue;
        // a vector's terms by pairs, the vectors in 64 bits: one after the other in 32, those beside
        // the largest would lose 2e-7 of it
        float e[W];
#pragma unroll
        for (u32 k = 0; k < W; ++k) e[k] = sh.of<true>(entry<T>(v[i], k));
#pragma unroll
        for (u32 d = 1; d < W; d <<= 1)
#pragma unroll
          for (u32 k = 0; k < W; k += 2 * d) e[k] += e[k + d];
        sum += (double)e[0];
        // its place for the next segment's, on its way while the others are dealt with
        if (MULTI && i < next) load_one(first + TEAM * N, i, next);
      }
      rest += sh.whole(sum, top, true);
    }
    rest += (double)ex.of(edge - top);
    // over the lanes, then over the team's wavefronts
    row.top = top;
    row.rest = lanes_sum<kWave>(rest);
    if constexpr (kTeamWaves == 1) {
      const u32 l = in_vecs ? owner : (token < head ? token : token - all * W);
      row.token = __uint_as_float((u32)__builtin_amdgcn_readlane((int)__float_as_uint(x_token), (int)l));
    } else {
      if (lane == 0) {
        s_top[wave] = row.top;
        s_rest[wave] = row.rest;
      }
      if (in_vecs ? tid == owner : (tid < edges && mine == token)) s_token[team] = x_token;
      lds_barrier();
      const float m = s_top[tid % kTeamWaves];
      row.top = group_reduce<kTeamWaves>(m, max_f);
      row.rest = lanes_sum<kTeamWaves>(s_rest[tid % kTeamWaves] * (double)ex.of(m - row.top));
      row.token = s_token[team];  // (nobody's, in a slice that does not hold it)
    }
    if constexpr (MODE == kPart) {
      if (tid == 0) sc.parts[t * a.slices + slice] = Part{row.rest, row.top};
      return;
    }
  }
  if (row.token > row.top) {
    row.rest *= ex.exactly(row.top - row.token);
    row.top = row.token;
  }
  const u32 n = wave_reduce_u32(live_part, [](u32 p, u32 q) { return p + q; });  // the live rows of all
  const RowEnd end = end_of(a, row);
  const RowTerms o = terms_of(a, in, end, d_loss, n ? 1.0 / (double)n : 0.0);
  if (MODE == kWhole && tid == 0) {
    if (a.logprobs) a.logprobs[t] = (float)end.lp;
    if (a.policy) sc.rows[t] = Terms{o.loss, o.kl, o.clipped, 0};
    if (a.pairs) sc.lp[t] = end.lp;
  }
  if constexpr (GRAD) {
    if (o.c == 0.f || end.absent) {
      zero_row();
    } else {
      const float c = (float)((double)o.c * a.inverse_temperature);
      const float scale = (float)(-(double)c / end.total);
      T at_token;
      from_f32((float)((double)c * (row.rest / end.total)), at_token);
      if (tid < edges) {
        T g;
        from_f32(scale * ex.of(edge - row.top), g);
        dx[mine] = mine == token ? at_token : g;
      }
      constexpr bool kBoth = sizeof(T) == 4;
      const Shifted sh(ex, row.top, kBoth);
      const float scaled = (float)sh.whole((double)scale, row.top, kBoth);
      for (u32 seg = segments; seg-- > 0;) {
        if (MULTI && (seg + 1 < segments)) {
          first = seg * TEAM * N;
          load();
        }
        const int at = slot_of(), cnt = count(first);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if (i >= cnt) continue;
          Words w;
#pragma unroll
          for (u32 k = 0; k < 4; ++k) {
            T g[4 / sizeof(T)];
#pragma unroll
            for (u32 h = 0; h < 4 / sizeof(T); ++h)
              from_f32(scaled * sh.of<kBoth>(entry<T>(v[i], k * (4 / sizeof(T)) + h)), g[h]);
            u32 bits;
            __builtin_memcpy(&bits, g, 4);
            w[k] = bits;
          }
          if (i == at && tid == owner) set_entry<T>(w, place, at_token);
          if (i + 1 < cnt || has(first, i)) store(i, w);
        }
      }
    }
  }
}

// No rows at all.
__global__ void vocab_empty_kernel(VocabArgs a) {
  *vocab_scratch(a.scratch, 0).last = 0;
  if (!a.policy) return;
  *a.loss = *a.kl = 0.f;
  *a.clipped = *a.rows = 0;
}

// The pairs' losses, and every row's coefficient.  A block takes a run of neighbouring pairs, one at a
// time with all of its threads: few pairs of long sequences leave the other CUs idle (131072 rows in
// one pair 299 us with their log-probabilities, in 64 pairs 87).
template <class T>
__global__ __launch_bounds__(kPairThreads) void pair_kernel(PairArgs a) {
  constexpr int kWaves = kPairThreads / kWave;
  __shared__ double s_d[kWaves], s_own[2][kWaves], s_ref[2][kWaves];
  __shared__ u64 s_n[kWaves], s_live[2][kWaves];
  __shared__ u32 s_rise[2][kWaves];
  __shared__ u32 s_last;
  const VocabScratch sc = vocab_scratch(a.v.scratch, a.v.T);
  // A live row's log-probability; of rows that are split, from their parts.
  auto lp_of = [&](u64 t, bool here) {
    if (!a.v.slices) return sc.lp[t];
    return here ? end_of(a.v, sums_of<T>(a.v, sc.parts, t)).lp : 0.0;
  };
  // Rows that no sequence takes.
  auto outside = [&](u64 t) {
    a.coefficients[t] = 0.f;
    if (a.v.slices) a.v.logprobs[t] = (float)lp_of(t, row_live(a.v, t));
  };
  double total = 0;
  u64 rows = 0;
  // Offsets as far as they rise, within [0, T] (T < 2^31): one below an earlier one counts as that.
  // A block takes neighbouring pairs, so it looks at all that come before once.
  const u64 chunk = (a.pairs + gridDim.x - 1) / gridDim.x, p0 = blockIdx.x * chunk;
  const u64 p1 = p0 + chunk < a.pairs ? p0 + chunk : a.pairs;
  auto within = [&](u64 k) {
    const int64_t o = a.offsets[k];
    return o < 0 ? 0u : (u64)o < a.v.T ? (u32)o : (u32)a.v.T;
  };
  u32 risen[2] = {0, 0};  // up to offsets p and p + pairs
  if (p0 < p1) {
    for (u64 k = threadIdx.x; k <= p0 + a.pairs; k += kPairThreads) {
      const u32 o = within(k);
      risen[1] = o > risen[1] ? o : risen[1];
      if (k <= p0) risen[0] = risen[1];
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      risen[h] = wave_reduce_u32(risen[h], [](u32 x, u32 y) { return x > y ? x : y; });
      if (lane_id() == 0) s_rise[h][threadIdx.x / kWave] = risen[h];
    }
    lds_barrier();
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int w = 0; w < kWaves; ++w) risen[h] = s_rise[h][w] > risen[h] ? s_rise[h][w] : risen[h];
  }
  for (u64 p = p0; p < p1; ++p) {
    lds_barrier();  // the last pair's sums have been read
    u64 start[2], end[2], live[2] = {0, 0};
    double own[2] = {0, 0}, ref[2] = {0, 0}, ratio[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u32 o = within(p + h * a.pairs + 1);
      start[h] = risen[h];
      end[h] = risen[h] = o > risen[h] ? o : risen[h];
    }
    // the rows of both, all of a row's loads at once
    const u64 first = end[0] - start[0], both = first + (end[1] - start[1]);
    auto row_of = [&](u64 i) { return i < first ? start[0] + i : start[1] + (i - first); };
    for (u64 i = threadIdx.x; i < both; i += kPairThreads) {
      const u64 t = row_of(i);
      const int h = i >= first;
      const bool here = row_live(a.v, t);
      const float r = a.v.ref ? a.v.ref[t] : 0.f;
      const double lp = lp_of(t, here);
      if (a.v.slices) a.v.logprobs[t] = here ? (float)lp : 0.f;
      const bool counts = here && lp != -__builtin_huge_val();  // a token of weight 0 adds nothing
      live[0] += here && !h;
      live[1] += here && h;
      own[0] += counts && !h ? lp : 0.0;
      own[1] += counts && h ? lp : 0.0;
      ref[0] += counts && !h ? (double)r : 0.0;
      ref[1] += counts && h ? (double)r : 0.0;
    }
#pragma unroll
    for (int d = kWave / 2; d; d >>= 1)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        own[h] += __shfl_xor(own[h], d);
        ref[h] += __shfl_xor(ref[h], d);
        live[h] += __shfl_xor(live[h], d);
      }
    if (lane_id() == 0)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        s_own[h][threadIdx.x / kWave] = own[h];
        s_ref[h][threadIdx.x / kWave] = ref[h];
        s_live[h][threadIdx.x / kWave] = live[h];
      }
    lds_barrier();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      own[h] = ref[h] = 0;
      live[h] = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        own[h] += s_own[h][w];
        ref[h] += s_ref[h][w];
        live[h] += s_live[h][w];
      }
      const double mean = a.average && live[h] ? 1.0 / (double)live[h] : 1.0;
      ratio[h] = (own[h] - ref[h]) * mean;
      if (threadIdx.x == 0) a.sequence_logprobs[p + h * a.pairs] = (float)(own[h] * mean);
      rows += live[h];
    }
    const double z = a.beta * (ratio[0] - ratio[1]) - a.margin;
    const double e = exp(-fabs(z)), tail = log1p(e);  // softplus(z) = max(z, 0) + tail
    const double up = (z < 0 ? -z : 0.0) + tail, down = (z > 0 ? z : 0.0) + tail;
    const double sigmoid = (z < 0 ? e : 1.0) / (1.0 + e), other = (z < 0 ? 1.0 : e) / (1.0 + e);
    const double keep = 1.0 - a.smoothing;
    // up and down may be infinite, where the reference gives a token nothing: 0 of that is 0
    total += z == z ? (keep != 0 ? keep * up : 0.0) + (a.smoothing != 0 ? a.smoothing * down : 0.0) : z;
    if (threadIdx.x == 0) a.margins[p] = (float)z;
    const double slope = a.beta / (double)a.pairs * (a.smoothing * sigmoid - keep * other);
    float c[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      c[h] = (float)((h ? -slope : slope) * (a.average && live[h] ? 1.0 / (double)live[h] : 1.0));
    for (u64 i = threadIdx.x; i < both; i += kPairThreads) {
      const u64 t = row_of(i);
      a.coefficients[t] = row_live(a.v, t) ? c[i >= first] : 0.f;
    }
    if (p == 0)
      for (u64 t = threadIdx.x; t < start[0]; t += kPairThreads) outside(t);
    if (p == a.pairs - 1)
      for (u64 t = end[1] + threadIdx.x; t < a.v.T; t += kPairThreads) outside(t);
  }
  if (threadIdx.x == 0) {
    st_double(&sc.blocks[blockIdx.x].loss, total);
    st_agent((u64*)&sc.blocks[blockIdx.x].clipped, rows);
    drain_memory_ops();
    s_last = __hip_atomic_fetch_add(sc.last, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1 == gridDim.x;
  }
  __syncthreads();
  if (!s_last) return;
  double loss = 0;
  u64 n = 0;
  for (u32 i = threadIdx.x; i < gridDim.x; i += kPairThreads) {
    loss += ld_double(&sc.blocks[i].loss);
    n += ld_agent((const u64*)&sc.blocks[i].clipped);
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
hipError_t vocab_launch(VocabArgs a, hipStream_t s) {
  constexpr int kBlock = TEAM < 256 ? 256 : TEAM, kTeams = kBlock / TEAM;
  constexpr u64 kMost = ((1ull << 32) / kBlock - 1) * kTeams;  // rows of a launch, which has fewer than 2^32 threads
  for (a.row0 = 0; a.row0 < a.T; a.row0 += kMost) {
    const u64 rows = a.T - a.row0 < kMost ? a.T - a.row0 : kMost;
    vocab_kernel<T, TEAM, N, GRAD, MULTI, kWhole><<<(u32)((rows + kTeams - 1) / kTeams), kBlock, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// The fewest threads whose registers hold the row in 16 vectors each (one wavefront: in 4, where
// those do).  Few threads wait little for one another, and many rows a CU cover each other's loads.
// With the next more threads (64 with 16 vectors in place of 4), bf16, 8192 rows, log-probabilities
// and policy loss with gradient, us: 500 entries 7 -> 9 and 17 -> 21, 2048: 10 -> 11 and 22 -> 26,
// 8192: 26 -> 34 and 59 -> 68, 32768: 97 -> 94 and 206 -> 202 (the gradient alone 187 -> 214),
// 65536: 170 -> 260 and 383 -> 453.
// Longer rows go in segments, twice where there is a gradient: without one 256 threads, five
// workgroups a CU (8192 x 131072 bf16 410 us; 512 threads in segments, which spill 25 registers at
// their bound, 637; 1024, which hold the row, 450).  One workgroup of 1024 holds the longest gradient rows, one a
// CU: 512 in segments read the row twice, and took 590 us in place of 450 for 4096 x 131072 bf16.
template <class T, bool GRAD>
hipError_t vocab_shape(const VocabArgs& a, hipStream_t s) {
  const u64 bytes = a.V * sizeof(T);
  if (bytes <= 64 * 16 * 4) return vocab_launch<T, 64, 4, GRAD, false>(a, s);
  if (bytes <= 64 * 16 * 16) return vocab_launch<T, 64, 16, GRAD, false>(a, s);
  if (bytes <= 256 * 16 * 16) return vocab_launch<T, 256, 16, GRAD, false>(a, s);
  if (bytes <= 512 * 16 * 16) return vocab_launch<T, 512, 16, GRAD, false>(a, s);
  if constexpr (GRAD) {
    if (bytes <= 1024 * 16 * 16) return vocab_launch<T, 1024, 16, true, false>(a, s);
    return vocab_launch<T, 1024, 16, true, true>(a, s);
  } else {
    return vocab_launch<T, 256, 16, false, true>(a, s);
  }
}

constexpr int kSliceThreads = 256, kSliceVectors = 8;

u32 term_blocks(const VocabArgs& a) {
  const u64 b = (a.T + kTermThreads - 1) / kTermThreads;
  return b < 1 ? 1 : b < kTermBlocks ? (u32)b : kTermBlocks;
}

template <class T>
hipError_t vocab_split(const VocabArgs& a, hipStream_t s) {
  vocab_kernel<T, kSliceThreads, kSliceVectors, false, true, kPart>
      <<<(u32)a.T * a.slices + 1, kSliceThreads, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.pairs) return e;
  static_assert(kSliceThreads == kTermThreads, "blocks of one launch");
  const u32 terms = term_blocks(a);
  if (a.d_x)
    vocab_kernel<T, kSliceThreads, kSliceVectors, true, true, kJoin>
        <<<(u32)a.T * a.slices + (a.policy ? terms : 0), kSliceThreads, 0, s>>>(a);
  else
    vocab_terms_kernel<T><<<terms, kTermThreads, 0, s>>>(a);
  return hipGetLastError();
}

template <class T>
hipError_t vocab_type(VocabArgs a, hipStream_t s) {
  if (a.slices) return vocab_split<T>(a, s);
  hipError_t e;
  if (a.policy && a.d_x && !a.weights) {  // each row's share
    const u64 rounds = (a.T + kCountThreads - 1) / kCountThreads;
    a.count_blocks = rounds < kCountBlocks ? (u32)rounds : kCountBlocks;
    vocab_count_kernel<<<a.count_blocks, kCountThreads, 0, s>>>(a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  e = a.d_x ? vocab_shape<T, true>(a, s) : vocab_shape<T, false>(a, s);
  if (e != hipSuccess || !a.policy) return e;
  vocab_terms_kernel<T><<<term_blocks(a), kTermThreads, 0, s>>>(a);
  return hipGetLastError();
}

template <class T>
hipError_t pairs_type(const PairArgs& a, hipStream_t s) {
  pair_kernel<T><<<a.pairs < kPairBlocks ? (u32)a.pairs : kPairBlocks, kPairThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

size_t vocab_scratch_bytes(u64 T) {
  const VocabScratch v = vocab_scratch(nullptr, T);
  return (size_t)(uintptr_t)v.parts + sizeof(Part) * kSlices * (T < kSplitRows ? T : kSplitRows);
}

// Few rows leave most of the 256 CUs idle, so they go in slices of 16 KB that a second launch
// joins: for the losses, a launch that follows anyway.  A gradient reads its slices again then,
// where a workgroup with the whole row in registers does not.  bf16, split / whole, us:
//   log-probabilities  1 x 131072 9.4 / 18, 512 x 131072 32 / 41, 768 x 131072 48 / 48;
//                      64 x 65536 8.6 / 9.2, 256 x 65536 13 / 9.9, 1 x 32768 8.4 / 7.2
//   their gradient     64 x 131072 14 / 21, 256 x 131072 44 / 28, 64 x 32768 9.8 / 11, 64 x 16384 9.4 / 7.7
//   policy loss        64 x 65536 9.9 / 12, 512 x 65536 22 / 21, 512 x 16384 13 / 13, 512 x 8192 11 / 13
//     with gradient    64 x 131072 15 / 24, 256 x 131072 44 / 32, 64 x 32768 11 / 15, 512 x 16384 18 / 16,
//                      256 x 16384 12 / 12, 512 x 8192 13 / 17
//   preference loss    512 x 131072 43 / 49, 512 x 65536 27 / 23, 64 x 65536 13 / 16, 512 x 8192 13 / 15
u32 vocab_slices(const VocabArgs& a, int dtype) {
  const u64 bytes = a.V * (dtype == PROFK_FP32 ? 4 : 2), whole = a.d_x ? 262144 : 131072;  // what registers hold
  const bool loss = a.policy || a.pairs;
  if (bytes < (loss ? 16384 : a.d_x ? 65536 : 131072)) return 0;
  u64 most = kSplitRows;
  if (bytes <= whole) most = a.d_x && !loss ? 64 : (1 << 24) / bytes < most ? (1 << 24) / bytes : most;
  if (a.T > most) return 0;
  const u64 s = (bytes + 16383) / 16384;
  return (u32)(s < kSlices ? s : kSlices);
}

hipError_t launch_vocab(VocabArgs a, int dtype, hipStream_t s) {
  if (!a.T) {  // the policy loss of no rows; the pairs' ticket
    if (a.policy || a.pairs) vocab_empty_kernel<<<1, 1, 0, s>>>(a);
    return hipGetLastError();
  }
  a.slices = vocab_slices(a, dtype);
  a.count_blocks = 1;
  if (dtype == PROFK_FP32) return vocab_type<float>(a, s);
  if (dtype == PROFK_FP16) return vocab_type<Half16>(a, s);
  return vocab_type<Brain16>(a, s);
}

hipError_t launch_pairs(PairArgs a, int dtype, hipStream_t s) {
  a.v.slices = a.v.T ? vocab_slices(a.v, dtype) : 0;
  if (dtype == PROFK_FP32) return pairs_type<float>(a, s);
  if (dtype == PROFK_FP16) return pairs_type<Half16>(a, s);
  return pairs_type<Brain16>(a, s);
}

}  // namespace profk
