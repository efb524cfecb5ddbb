// A token per row of logits: temperature, top-k, top-p and min-p, drawn by one given number per row.
//
// With x the row's logits, top the largest, and tokens in the order of falling x (ties by index):
//   w_i = rint(2^40 * exp((x_i - top) / temperature))    a whole number, so that sums of weights are exact and do
//                                                        not depend on their order
//   S_k = the first top_k weights, S_p = the shortest prefix of at least top_p * S_k, S_m = the weights of at
//   least min_p * 2^40;  S = min(S_k, S_p, S_m), all of them sums of prefixes of the same order
//   token = the first one at which the running sum passes floor(u * S)
// Every question about the order (where does the k-th weight end, where does a running sum pass a goal) needs
// the sums up to a bin of close values, and the order inside one bin alone:
//   max    blocks find largest and least logit of a chunk of a row
//   hist   blocks count a chunk's tokens and sum their weights by bins of (x - top) / temperature
//   pick   one block per row adds the chunks' bins up and answers the questions.  The tokens of the bins it needs
//          are gathered into LDS: where those up to the last bin in question are kList at most (top-k and top-p as
//          they are used), once for all questions, from the groups of 64 logits that hold any.  There the bin
//          in question is split further by place (value, then index) until a wave can sort what is left.  A bin
//          of more than kList tokens is split by passes over the row first.
// Weights take an exp in fp64; 2^-41 of the largest and less are zero and leave early.
#include <algorithm>

#include "block_ops.hpp"
#include "device_common.hpp"
#include "step_ops.hpp"
#include "wave_ops.hpp"

namespace bl {

namespace {

typedef unsigned long long u64;

constexpr int kBins = kSampleBins;
constexpr int kList = kSampleList;       // tokens that are gathered
constexpr int kThreads = 512;            // of every block
constexpr int kWaves = kThreads / 64;
constexpr int kStep = kThreads * 8;      // logits that a block loads at a time
static_assert(kThreads == kBins, "a thread per bin");
constexpr double kOne = 1099511627776.0; // 2^40, the weight of the largest logit

struct Row {                             // what is known of a row once its largest logit is
  double top;
  double c;                              // log2(e) / temperature
  float per_fine;                        // fine bins per unit of top - x
  bool inf;                              // the largest is infinite: its equals weigh 2^40, the others nothing
};

// x as an unsigned number that falls as x rises; both zeros are one.
__device__ __forceinline__ uint32_t falling(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? u : ~u & 0x7FFFFFFFu;
}
__device__ __forceinline__ float from_falling(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k : ~k & 0x7FFFFFFFu);
}

constexpr float kNegInf = -__builtin_inff();

struct Add {
  template <class T>
  __device__ T operator()(T x, T y) const { return x + y; }
};
struct Least {
  __device__ u64 operator()(u64 x, u64 y) const { return min(x, y); }
  __device__ float operator()(float x, float y) const { return fminf(x, y); }
};

// Elements i .. i + 8 of a row without a branch around a load, so that many can be in flight: vector loads of whole
// eights (what is past them is loaded as the last one and left out below), else element by element.
template <bool BF, bool VEC>
__device__ __forceinline__ void load8_raw(const void* row, int64_t i, int64_t V, float v[8]) {
  if constexpr (VEC) {
    load_f8<BF>(row, max(min(i, V / 8 * 8 - 8), (int64_t)0), v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t k = min(i + j, V - 1);
      v[j] = BF ? __uint_as_float((uint32_t)((const uint16_t*)row)[k] << 16) : ((const float*)row)[k];
    }
  }
}
// Makes what load8_raw read the row's elements, -inf past its end; its last V % 8 are read again.
template <bool BF, bool VEC>
__device__ __forceinline__ void finish8(const void* row, int64_t i, int64_t V, float v[8]) {
  if (i + 8 <= V) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (i + j >= V) v[j] = kNegInf;
    else if (VEC)
      v[j] = BF ? __uint_as_float((uint32_t)((const uint16_t*)row)[i + j] << 16) : ((const float*)row)[i + j];
  }
}
// The same with -inf for NaN.
template <bool BF, bool VEC>
__device__ __forceinline__ void finish8_masked(const void* row, int64_t i, int64_t V, float v[8]) {
  finish8<BF, VEC>(row, i, V, v);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = v[j] == v[j] ? v[j] : kNegInf;
}
template <bool BF>
__device__ __forceinline__ const void* row_of(const SampleArgs& a, int64_t b) {
  return (const char*)a.x + b * a.stride * (BF ? 2 : 4);
}

// (x - top) / temperature / ln 2, at most 0; -inf for what weighs nothing.
__device__ __forceinline__ double scaled(const Row& r, float x) {
  if (r.inf) return x == (float)r.top ? 0.0 : -__builtin_inf();
  return x == kNegInf ? -__builtin_inf() : ((double)x - r.top) * r.c;
}
// The logit's place among kBins^2 fine bins of the row's range, kBins of them to a bin: any steps that rise as x falls
// will do, so fp32 is enough.  NaN (equals of an infinite top) counts as 0.
__device__ __forceinline__ int fine_of(const Row& r, float x) {
  return (int)__builtin_amdgcn_fmed3f(((float)r.top - x) * r.per_fine, 0.f, (float)(kBins * kBins - 1));
}

// 2^40 * 2^t rounded to a whole number, t <= 0 (NaN: 0).  2^f for |f| <= 1/2 is a polynomial through the eleven
// Chebyshev points, 2.4e-16 off at most, its coefficients times 2^40.  Adding 1.5 * 2^52 rounds to a whole number, half
// to even, in a double's low bits; 2^n goes straight into the exponent.
__device__ __forceinline__ u64 weight(double t) {
  const double magic = 6755399441055744.0;
  t = __builtin_fmax(t, -60.0);
  const double m = t + magic, f = t - (m - magic);
  double p = 0x1.e6063f7217bc6p+12;
  p = __builtin_fma(p, f, 0x1.b675bca4eeebbp+16);
  p = __builtin_fma(p, f, 0x1.62bfd47773353p+20);
  p = __builtin_fma(p, f, 0x1.ffcb54062e698p+23);
  p = __builtin_fma(p, f, 0x1.430913096fd9fp+27);
  p = __builtin_fma(p, f, 0x1.5d87fe9d7a584p+30);
  p = __builtin_fma(p, f, 0x1.3b2ab6fba1ddap+33);
  p = __builtin_fma(p, f, 0x1.c6b08d703ce49p+35);
  p = __builtin_fma(p, f, 0x1.ebfbdff82c598p+37);
  p = __builtin_fma(p, f, 0x1.62e42fefa3a19p+39);
  p = __builtin_fma(p, f, 0x1.0p+40);
  uint2 bits = __builtin_bit_cast(uint2, p);
  bits.y += __builtin_bit_cast(uint2, m).x << 20;
  bits = __builtin_bit_cast(uint2, __builtin_bit_cast(double, bits) + magic);
  return (u64)(bits.y & 0x7FFFFu) << 32 | bits.x;
}
__device__ __forceinline__ u64 weight_of(const Row& r, float x) { return weight(scaled(r, x)); }

struct Settings {
  double temp, p;
  u64 min_w;                             // what min-p keeps, in weights; 0: off
  int64_t k;                             // 0: off
  bool greedy;
};
__device__ __forceinline__ Settings settings_of(const SampleArgs& a, int64_t b) {
  Settings s;
  const float t = a.temperature ? a.temperature[b] : 1.f, p = a.top_p ? a.top_p[b] : 1.f,
              m = a.min_p ? a.min_p[b] : 0.f;
  const int32_t k = a.top_k ? a.top_k[b] : 0;
  s.greedy = !(t > 0.f);
  s.temp = t;
  s.p = p < 1.f ? max((double)p, 0.0) : 1.0;               // NaN: off
  s.min_w = m > 0.f ? (u64)ceil(fmin((double)m, 2.0) * kOne) : 0;
  s.k = k > 0 && k < a.V ? k : 0;
  return s;
}

// The chunks' largest logits (as places) and least finite ones, joined by every wave.
struct Extremes {
  u64 top;
  float least;
};
__device__ __forceinline__ Extremes row_extremes(const SampleArgs& a, int64_t b) {
  static_assert(kSampleChunks <= 64, "a lane per chunk");
  const int lane = threadIdx.x & 63;
  const int64_t at = b * a.chunks + min<int64_t>(lane, a.chunks - 1);
  return {a.top[at], a.least[at]};
}
__device__ __forceinline__ Row row_of_extremes(const Extremes& e, const Settings& s, u64* best) {
  *best = wave_all(e.top, (u64)~0ull, Least());
  const float least = wave_all(e.least, __builtin_inff(), Least());
  const float x = from_falling((uint32_t)(*best >> 32));
  Row r;
  r.top = x;
  r.inf = x == __builtin_inff();
  r.c = 1.4426950408889634 / s.temp;
  // over what weighs anything, or what there is; too narrow to be told apart: one bin
  const float per_fine = (float)(kBins * kBins / fmin((double)x - least, 41.0 / r.c));
  r.per_fine = per_fine < 1e30f && !r.inf ? per_fine : 0.f;
  return r;
}

// ---------------------------------------------------------------------------------------------
// questions about the order
// ---------------------------------------------------------------------------------------------

struct Pair {
  u64 w, n;
};

enum Question { kCount, kGoal, kPass };  // the k-th token; first sum >= goal (as doubles); first sum > r

struct Asked {
  Question q;
  u64 k;
  double goal;
  u64 r;
};
// Whether tokens up to one with these running sums answer the question.
__device__ __forceinline__ bool met(const Asked& a, const Pair& p) {
  return a.q == kCount ? p.n >= a.k : a.q == kGoal ? (double)p.w >= a.goal : p.w > a.r;
}
__device__ __forceinline__ Pair operator+(const Pair& a, const Pair& b) { return {a.w + b.w, a.n + b.n}; }

// First bin whose running sums, behind `before`, answer the question (the last one that adds anything, if none
// does).  Every wave finds it by itself: 64 ends of eight bins, then the eight.
__device__ __forceinline__ int first_bin(const Asked& q, const Pair* bins, const Pair& before) {
  static_assert(kBins == 512, "64 eights");
  const int lane = threadIdx.x & 63;
  const u64 all = bins[kBins - 1].n;
  auto yes = [&](int i) {
    const Pair p = bins[i];
    return __ballot(met(q, before + p) || p.n == all);       // rising: once it is so it stays so
  };
  const int eight = __ffsll((unsigned long long)yes(lane * 8 + 7)) - 1;
  return eight * 8 + __ffsll((unsigned long long)yes(eight * 8 + (lane & 7))) - 1;
}

// A token's place in the order: its logit as a falling number, then its index.
__device__ __forceinline__ u64 place(float x, int64_t i) { return ((u64)falling(x) << 32) | (uint32_t)i; }
__device__ __forceinline__ float logit_at(u64 place) { return from_falling((uint32_t)(place >> 32)); }

struct Range {                           // of places, both ends included
  u64 lo, hi;
};

// Largest falling() value whose logit weighs something and lies in a bin up to `bin`; the row's largest logit
// always does.  The lanes of a wave try 64 values at a time.
__device__ __forceinline__ u64 key_end(const Row& r, int bin) {
  const int lane = threadIdx.x & 63;
  uint64_t lo = falling((float)r.top), hi = (uint64_t)1 << 32;   // lo does, hi does not
  while (hi - lo > 1) {
    const uint64_t step = (hi - lo + 63) >> 6, at = lo + lane * step;
    const float x = from_falling((uint32_t)at);
    const uint64_t mask = __ballot(at < hi && x == x && weight_of(r, x) > 0 && fine_of(r, x) / kBins <= bin);
    const int last = 63 - __clzll((long long)mask);
    hi = min(hi, lo + (last + 1) * step);
    lo += last * step;
  }
  return lo;
}
__device__ __forceinline__ Range places_of(const Row& r, int bin) {
  const u64 first = bin ? key_end(r, bin - 1) + 1 : falling((float)r.top);
  return {first << 32, key_end(r, bin) << 32 | 0xFFFFFFFFu};
}

template <bool BF, bool VEC>
__global__ __launch_bounds__(kThreads) void sample_max_kernel(SampleArgs a) {
  __shared__ u64 s_top[kWaves];
  __shared__ float s_least[kWaves];
  const int64_t b = blockIdx.y;
  const void* row = row_of<BF>(a, b);
  const int64_t i0 = (int64_t)blockIdx.x * a.chunk, i1 = min(i0 + a.chunk, a.V);
  u64 top = ~0ull;
  float least = __builtin_inff();
  for (int64_t at = i0; at < i1; at += 2 * kStep) {
    const int64_t i = at + threadIdx.x * 8;
    float v[2][8];
#pragma unroll
    for (int k = 0; k < 2; ++k) load8_raw<BF, VEC>(row, i + k * kStep, a.V, v[k]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (at + k * kStep >= i1) break;
      finish8_masked<BF, VEC>(row, i + k * kStep, a.V, v[k]);
      float most = kNegInf;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        least = fminf(least, v[k][j] == kNegInf ? __builtin_inff() : v[k][j]);
        most = fmaxf(most, v[k][j]);
      }
      if (falling(most) < (uint32_t)(top >> 32)) {           // the first of its equals
        int j = 7;
#pragma unroll
        for (int e = 6; e >= 0; --e) j = v[k][e] == most ? e : j;
        top = place(most, i + k * kStep + j);
      }
      most = fmaxf(most, lane_move<0xB1, 0xF>(most, most));  // lanes 1, 2 and 7 - i of eight apart
      most = fmaxf(most, lane_move<0x4E, 0xF>(most, most));
      most = fmaxf(most, lane_move<0x141, 0xF>(most, most));
      const int64_t group = (i + k * kStep) / 64;
      if ((threadIdx.x & 7) == 0 && group < a.groups) a.most[b * a.groups + group] = most;
    }
  }
  top = wave_all(top, (u64)~0ull, Least());
  least = wave_all(least, __builtin_inff(), Least());
  if ((threadIdx.x & 63) == 0) {
    s_top[threadIdx.x >> 6] = top;
    s_least[threadIdx.x >> 6] = least;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < kWaves; ++w) {
      top = min(top, s_top[w]);
      least = fminf(least, s_least[w]);
    }
    a.top[b * a.chunks + blockIdx.x] = top;
    a.least[b * a.chunks + blockIdx.x] = least;
    if (blockIdx.x == 0) a.plan[b].arrived = 0;
  }
}

// Device-scope accesses of what blocks of one launch hand to each other, past the caches that the XCDs do not
// share.
template <class T>
__device__ __forceinline__ void put(T* p, T v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <class T>
__device__ __forceinline__ T get(const T* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Whether this block is the last of `blocks` to arrive.  Every wave waits for its own accesses first; what the others
// stored before they arrived is there for get().
__device__ __forceinline__ bool last_to_arrive(uint32_t* arrived, uint32_t blocks, bool* shared) {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
  __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
  __syncthreads();
  if (threadIdx.x == 0)
    *shared = __hip_atomic_fetch_add(arrived, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == blocks - 1;
  __syncthreads();
  return *shared;
}

// Which tokens of a row the questions need: bins, at most kList tokens in all, or none if they are more.  With k or
// top-p the sums that the later questions start from are known to within a bin only, so theirs may lie in one of
// a few bins.
__device__ __forceinline__ void make_plan(SamplePlan* plan, const Settings& st, u64 sum_m, double u,
                                          const Pair* bins) {
  const Pair none = {0, 0};
  const Pair all = bins[kBins - 1];
  const u64 k = st.k && (u64)st.k < all.n ? (u64)st.k : 0;
  auto upto = [&](int bin) { return bin < 0 ? none : bins[bin]; };
  u64 lo = all.w, hi = all.w;                                // of the sum that is left
  int b0[3], b1[3], n = 0;
  if (k) {
    const int bin = first_bin({kCount, k, 0.0, 0}, bins, none);
    lo = upto(bin - 1).w;
    hi = upto(bin).w;
    b0[0] = b1[0] = bin;
    n = 1;
  }
  if (st.p < 1.0 && !(n && upto(b1[0]).n <= kList)) {
    const int bin0 = first_bin({kGoal, 0, st.p * (double)lo, 0}, bins, none);
    const int bin1 = first_bin({kGoal, 0, st.p * (double)hi, 0}, bins, none);
    lo = min(lo, upto(bin0 - 1).w);
    hi = min(hi, upto(bin1).w);
    b0[n] = bin0;
    b1[n++] = bin1;
  }
  if (st.min_w) {
    lo = min(lo, max(sum_m, (u64)kOne));
    hi = min(hi, max(sum_m, (u64)kOne));
  }
  // everything down to the first question's bin, which is the last, if it is not too much; else each for itself
  if (n && upto(b1[0]).n <= kList) {
    b0[0] = 0;
    n = 1;
  } else {
    const double part = u > 0.0 ? fmin(u, 1.0) : 0.0;
    b0[n] = first_bin({kPass, 0, 0.0, min((u64)(part * (double)lo), max(lo, (u64)1) - 1)}, bins, none);
    b1[n++] = first_bin({kPass, 0, 0.0, min((u64)(part * (double)hi), hi - 1)}, bins, none);
  }
  const int last = b1[0];
  // one that meets the one before it joins it
  int m = 0;
  for (int i = 1; i < n; ++i) {
    if (b1[i] >= b0[m]) {
      b0[m] = min(b0[m], b0[i]);
    } else {
      b0[++m] = b0[i];
      b1[m] = b1[i];
    }
  }
  u64 tokens = 0;
  for (int i = 0; i <= m; ++i) tokens += upto(b1[i]).n - upto(b0[i] - 1).n;
  n = tokens <= kList ? m + 1 : 0;
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      plan->bin0[i] = i < n ? b0[i] : 1;                     // none
      plan->bin1[i] = i < n ? b1[i] : 0;
    }
    plan->ranges = n;
    plan->upto = (uint32_t)min(upto(last).n, (u64)0xFFFFFFFFu);
    plan->count = 0;
    plan->arrived = 0;
  }
}

// Inclusive sums over the block, thread by thread.
__device__ __forceinline__ Pair scan(Pair v, Pair* waves) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  v = {wave_scan(v.w, (u64)0, Add()), wave_scan(v.n, (u64)0, Add())};
  if (lane == 63) waves[wave] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves - 1; ++w)
    if (w < wave) v = v + waves[w];
  return v;
}

template <bool BF, bool VEC>
__global__ __launch_bounds__(kThreads) void sample_hist_kernel(SampleArgs a) {
  __shared__ u64 w_bin[kBins];
  __shared__ uint32_t n_bin[kBins];
  __shared__ Pair bins[kBins], waves[kWaves];
  __shared__ double s_exp[kWaves];
  __shared__ u64 s_min[kWaves];
  __shared__ bool s_last;
  const int tid = threadIdx.x;
  const int64_t b = blockIdx.y;
  const Settings st = settings_of(a, b);
  const double u = a.u[b];
  u64 best;
  const Row r = row_of_extremes(row_extremes(a, b), st, &best);
  if (st.greedy && !a.logprob) return;
  if (r.top == -__builtin_inf()) return;                   // nothing to draw from
  w_bin[tid] = 0;
  n_bin[tid] = 0;
  __syncthreads();
  const void* row = row_of<BF>(a, b);
  const int64_t i0 = (int64_t)blockIdx.x * a.chunk, i1 = min(i0 + a.chunk, a.V);
  const float top = (float)r.top, per_bin = r.per_fine / kBins;
  double e = 0.0;                                          // sum of exp(x - top)
  u64 least_sum = 0;                                       // of the weights that min_p keeps
  for (int64_t at = i0; at < i1; at += 2 * kStep) {
    const int64_t i = at + tid * 8;
    float v[2][8];
#pragma unroll
    for (int k = 0; k < 2; ++k) load8_raw<BF, VEC>(row, i + k * kStep, a.V, v[k]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (at + k * kStep >= i1) break;
      finish8<BF, VEC>(row, i + k * kStep, a.V, v[k]);
      float d[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = top - v[k][j];
      if (a.logprob) {
        // eight at a time in fp32, unless one of them is 1, next to which small ones were lost, or NaN
        float some = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) some += __builtin_amdgcn_exp2f(d[j] * -1.44269504f);
        if (some < 1.f) {
          e += some;
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            e += v[k][j] == top ? 1.0 : d[j] > 0.f && !r.inf ? (double)__builtin_amdgcn_exp2f(d[j] * -1.44269504f) : 0.0;
        }
      }
      if (st.greedy) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const u64 w = r.inf ? weight_of(r, v[k][j]) : weight(((double)v[k][j] - r.top) * r.c);
        if (w) {
          const int bin = (int)__builtin_amdgcn_fmed3f(d[j] * per_bin, 0.f, (float)(kBins - 1));   // as in fine_of
          atomicAdd(&w_bin[bin], w);
          atomicAdd(&n_bin[bin], 1u);
          if (st.min_w && w >= st.min_w) least_sum += w;
        }
      }
    }
  }
  e = wave_all(e, 0.0, Add());
  least_sum = wave_all(least_sum, (u64)0, Add());
  if ((tid & 63) == 0) {
    s_exp[tid >> 6] = e;
    s_min[tid >> 6] = least_sum;
  }
  __syncthreads();
  const int64_t at = b * a.chunks + blockIdx.x;
  if (tid == 0) {
    double sum = s_exp[0];
    u64 kept = s_min[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) {
      sum += s_exp[w];
      kept += s_min[w];
    }
    a.exps[at] = sum;
    put(a.kept + at, kept);
  }
  if (st.greedy) return;
  put(a.w_bins + at * kBins + tid, w_bin[tid]);
  put(a.n_bins + at * kBins + tid, n_bin[tid]);
  if (!last_to_arrive(&a.plan[b].arrived, (uint32_t)a.chunks, &s_last)) return;
  // the row's bins, all chunks' sums asked for at once: running sums; and the plan
  u64 sum_m = get(a.kept + b * a.chunks + min<int64_t>(tid & 63, a.chunks - 1));
  u64 w[kSampleChunks];
  uint32_t n[kSampleChunks];
#pragma unroll
  for (int c = 0; c < kSampleChunks; ++c) {
    const int64_t from = (b * a.chunks + min<int64_t>(c, a.chunks - 1)) * kBins + tid;
    w[c] = get(a.w_bins + from);
    n[c] = get(a.n_bins + from);
  }
  Pair sum = {0, 0};
#pragma unroll
  for (int c = 0; c < kSampleChunks; ++c) sum = sum + (c < a.chunks ? Pair{w[c], n[c]} : Pair{0, 0});
  sum_m = wave_all((tid & 63) < a.chunks ? sum_m : 0, (u64)0, Add());
  sum = scan(sum, waves);
  bins[tid] = sum;
  ((ulonglong2*)a.sums)[b * kBins + tid] = make_ulonglong2(sum.w, sum.n);
  __syncthreads();
  if (tid < 64) make_plan(a.plan + b, st, sum_m, u, bins);
}

// ---------------------------------------------------------------------------------------------
// draw
// ---------------------------------------------------------------------------------------------

constexpr int kSmall = 64;               // tokens that a wave sorts

struct Found {                           // the answer to a question
  u64 sum;                               // of the weights up to and with the token found
  int64_t token;
};

struct Shared {                          // a block's memory
  u64 list[kList];                       // places of gathered tokens, in no order
  u64 few[kSmall];                       // those the answer lies among
  Pair bins[kBins], split[kBins];        // running sums by bin: of the row, of a part of it
  Pair waves[kWaves];
  uint32_t count, at, few_n;
  bool last;
};

struct Head {                            // of a plan
  int bin0[3], bin1[3];
  uint32_t ranges, upto;
};

// Appends to the list the logits of eight per lane, from index i on, that ok(x) says yes to.
template <class F>
__device__ __forceinline__ void append(Shared& s, const float v[8], int64_t i, F&& ok) {
  const int lane = threadIdx.x & 63;
  uint64_t mask[8];
  uint32_t all = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    mask[j] = __ballot(ok(v[j]));
    all += __popcll(mask[j]);
  }
  if (!all) return;
  uint32_t at = 0;
  if (lane == 0) at = atomicAdd(&s.count, all);
  at = __builtin_amdgcn_readfirstlane(at);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (!mask[j]) continue;
    const uint32_t k = at + __popcll(mask[j] & (((uint64_t)1 << lane) - 1));
    if (((mask[j] >> lane) & 1) && k < kList) s.list[k] = place(v[j], i + j);
    at += __popcll(mask[j]);
  }
}

// The plan's bins as bounds on (top - x) * per_fine, which is no number where there is one bin alone and x or top
// infinite, and the least logit that weighs anything.
struct Named {
  float lo[3], hi[3], least;
};
__device__ __forceinline__ Named named_by(const Row& r, const Head& plan) {
  Named n;
  bool light = r.per_fine == 0.f;        // what weighs nothing is in the last bin, or in the only one
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const bool last = plan.bin1[i] == kBins - 1;
    light |= last;
    n.lo[i] = (float)(plan.bin0[i] * kBins);
    // the largest number below the next bin; of no range: below its first
    n.hi[i] = last ? __builtin_inff() : __uint_as_float(__float_as_uint((float)((plan.bin1[i] + 1) * kBins)) - 1);
  }
  n.least = light ? from_falling((uint32_t)key_end(r, kBins - 1)) : kNegInf;
  return n;
}
__device__ __forceinline__ bool is_named(const Row& r, const Named& n, float x) {   // a NaN is not
  const float y = ((float)r.top - x) * r.per_fine;
  bool out = true;
#pragma unroll
  for (int i = 0; i < 3; ++i) out &= y < n.lo[i] || y > n.hi[i];
  return !out && x >= n.least;
}

// Whether one block reads a row's tokens, looking for them only in groups of 64 logits whose largest is in their bins,
// in place of all blocks reading all logits.  That takes it 14 ns a group more, and saves the launch's blocks a second
// reading, of little cost while all of them are there at once.  131072 logits, calls with one block and with all: one
// row, 100 tokens 25.0 and 25.3 us, 300 29.3 and 26.1; 16 rows, 100 27.8 and 29.5, 600 38.6 and 31.7; 64 rows, 300 53.7
// and 75.6, 1500 73 and 85.
__device__ __forceinline__ bool few_groups(const SampleArgs& a, const Head& plan) {
  const int64_t more = max(a.B * a.V - ((int64_t)1 << 21), (int64_t)0) >> 12;
  return plan.ranges == 1 && min((int64_t)plan.upto, a.groups) <= 128 + more;
}
// The list: the plan's tokens from such groups, eight lanes to each.
template <bool BF, bool VEC>
__device__ __forceinline__ void gather_groups(const SampleArgs& a, int64_t b, const Row& r, const Head& plan, Shared& s) {
  const int tid = threadIdx.x;
  const void* row = row_of<BF>(a, b);
  const Named named = named_by(r, plan);
  uint32_t* groups = (uint32_t*)s.split;
  constexpr int kAll = 4 * kThreads, kAhead = 2, kTeams = kThreads / 8;
  static_assert(sizeof(s.split) >= kAll * 4, "a round's groups fit");
  const float* most = a.most + b * a.groups;
  for (int64_t g0 = 0; g0 < a.groups; g0 += kAll) {
    if (tid == 0) s.at = 0;
    float m[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) m[k] = most[min(g0 + k * kThreads + tid, a.groups - 1)];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t i = g0 + k * kThreads + tid;
      if (i < a.groups && !(((float)r.top - m[k]) * r.per_fine > named.hi[0])) groups[atomicAdd(&s.at, 1u)] = (uint32_t)i;
    }
    __syncthreads();
    const int n = s.at;
    for (int k0 = 0; k0 < n; k0 += kAhead * kTeams) {
      float v[kAhead][8];
      int64_t i[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int at = k0 + k * kTeams + (tid >> 3);
        i[k] = at < n ? (int64_t)groups[at] * 64 + (tid & 7) * 8 : a.V;
        load8_raw<BF, VEC>(row, i[k], a.V, v[k]);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (k0 + k * kTeams >= n) break;
        finish8<BF, VEC>(row, i[k], a.V, v[k]);
        append(s, v[k], i[k], [&](float x) { return is_named(r, named, x); });
      }
    }
    __syncthreads();
  }
}

// The list: the plan's tokens of one chunk.
template <bool BF, bool VEC>
__device__ __forceinline__ void gather_chunk(const SampleArgs& a, int64_t b, int64_t part, const Row& r, const Head& plan,
                                             Shared& s) {
  const void* row = row_of<BF>(a, b);
  const Named named = named_by(r, plan);
  const int64_t i0 = part * a.chunk, i1 = min(i0 + a.chunk, a.V);
  for (int64_t at = i0; at < i1; at += 2 * kStep) {
    const int64_t i = at + threadIdx.x * 8;
    float v[2][8];
#pragma unroll
    for (int k = 0; k < 2; ++k) load8_raw<BF, VEC>(row, i + k * kStep, a.V, v[k]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (at + k * kStep >= i1) break;
      finish8<BF, VEC>(row, i + k * kStep, i1, v[k]);        // a chunk is a multiple of eight, but for the row's end
      append(s, v[k], i + k * kStep, [&](float x) { return is_named(r, named, x); });
    }
  }
  __syncthreads();
}

// Calls f(in, place) for the lanes' logits where any lane's is in the range: the whole row, by one block.  A NaN's
// place is outside of what weighs anything.
template <bool BF, class F>
__device__ __forceinline__ void each(const SampleArgs& a, int64_t b, const Range& g, F&& f) {
  constexpr int kAhead = 4;
  const void* row = row_of<BF>(a, b);
  for (int64_t at = 0; at < a.V; at += kAhead * kThreads) {
    float v[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int64_t i = min(at + k * kThreads + threadIdx.x, a.V - 1);
      v[k] = BF ? __uint_as_float((uint32_t)((const uint16_t*)row)[i] << 16) : ((const float*)row)[i];
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int64_t i = at + k * kThreads + threadIdx.x;
      const u64 p = place(v[k], i);
      const bool in = i < a.V && p >= g.lo && p <= g.hi;
      if (__any(in)) f(in, p);
    }
  }
}

// n <= 64 tokens in order, one to a lane: running sums of their weights, and their indices.  Every wave has them all.
struct Few {
  u64 upto;
  uint32_t token;
  int n;
};
__device__ __forceinline__ Few sort_few(const Row& r, const u64* places, int n) {
  const int lane = threadIdx.x & 63;
  const u64 p = lane < n ? places[lane] : ~0ull;
  const u64 w = lane < n ? weight_of(r, logit_at(p)) : 0;
  int rank = 0;
  for (int j0 = 0; j0 < n; j0 += 8) {                        // reads at places past n find anything, and do not count
    u64 other[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) other[j] = places[j0 + j];
#pragma unroll
    for (int j = 0; j < 8; ++j) rank += j0 + j < n && other[j] < p;
  }
  if (lane >= n) rank = lane;
  const uint32_t token = __builtin_amdgcn_ds_permute(rank * 4, (int)(uint32_t)p);
  const uint32_t w0 = __builtin_amdgcn_ds_permute(rank * 4, (int)(uint32_t)w);
  const uint32_t w1 = __builtin_amdgcn_ds_permute(rank * 4, (int)(uint32_t)(w >> 32));
  return {wave_scan((u64)w1 << 32 | w0, (u64)0, Add()), token, n};
}
// The answer among them, `before` which come others; the last one if none answers.
__device__ __forceinline__ Found among_few(const Asked& q, const Few& f, const Pair& before) {
  const int lane = threadIdx.x & 63;
  const uint64_t yes = __ballot(lane < f.n && met(q, before + Pair{f.upto, (u64)lane + 1}));
  const int at = yes ? __ffsll((unsigned long long)yes) - 1 : f.n - 1;
  return {before.w + lane_value(f.upto, at), (int64_t)lane_value(f.token, at)};
}

// The answer among the list's tokens that in(place) says yes to, n <= 64 of them.
template <class F>
__device__ __forceinline__ Found among_some(const Row& r, const Asked& q, int n, const Pair& before, Shared& s, F&& in) {
  __syncthreads();
  if (threadIdx.x == 0) s.few_n = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < (int)s.count; i += kThreads) {
    const u64 p = s.list[i];
    if (in(p)) s.few[atomicAdd(&s.few_n, 1u)] = p;
  }
  __syncthreads();
  return among_few(q, sort_few(r, s.few, n), before);
}

// Adds a lane's token to its part of a split; equal logits of a wave in one addition.
__device__ __forceinline__ void split_add(const Row& r, Shared& s, bool in, u64 p, uint32_t part) {
  const uint64_t mask = __ballot(in);
  if (!mask) return;
  const u64 w = weight_of(r, logit_at(p));
  const int first = __ffsll((unsigned long long)mask) - 1;
  const uint32_t part1 = lane_value(part, first), key1 = lane_value((uint32_t)(p >> 32), first);
  if (__ballot(in && part == part1 && (uint32_t)(p >> 32) == key1) == mask) {
    if ((int)(threadIdx.x & 63) == first) {
      atomicAdd(&s.split[part].w, w * __popcll(mask));
      atomicAdd(&s.split[part].n, (u64)__popcll(mask));
    }
  } else if (in) {
    atomicAdd(&s.split[part].w, w);
    atomicAdd(&s.split[part].n, 1ull);
  }
}
// After the additions: the part that holds the answer, and its tokens' number; what comes before it joins `before`.
__device__ __forceinline__ int split_choose(const Asked& q, Shared& s, Pair* before, u64* n) {
  __syncthreads();
  const Pair mine = s.split[threadIdx.x], upto = scan(mine, s.waves);
  s.split[threadIdx.x] = upto;
  __syncthreads();
  const int k = first_bin(q, s.split, *before);
  const Pair skip = k ? s.split[k - 1] : Pair{0, 0};
  *n = s.split[k].n - skip.n;
  *before = *before + skip;
  return k;
}

// The plan's tokens, a few to a thread: their places, fine bins (-1: none) and weights.
constexpr int kEach = kList / kThreads;
struct Mine {
  u64 p[kEach], w[kEach];
  int fine[kEach];
};

// The answer from the plan's tokens: those of the bin, by its fine bins if they are many.  False if too many share a
// fine bin.
__device__ __forceinline__ bool answer_mine(const Row& r, const Asked& q, const Mine& t, int bin, Pair before, u64 n,
                                            Shared& s, Found* found) {
  const int tid = threadIdx.x;
  __syncthreads();
  s.split[tid] = {0, 0};
  if (tid == 0) s.few_n = 0;
  __syncthreads();
  int part = -1;                         // of the bin; -1: all of it
  if (n > kSmall) {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      if (t.fine[i] >= 0 && t.fine[i] / kBins == bin) {
        atomicAdd(&s.split[t.fine[i] % kBins].w, t.w[i]);
        atomicAdd(&s.split[t.fine[i] % kBins].n, 1ull);
      }
    }
    part = split_choose(q, s, &before, &n);
    if (n > kSmall) return false;
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    if (t.fine[i] >= 0 && (part < 0 ? t.fine[i] / kBins == bin : t.fine[i] == bin * kBins + part))
      s.few[atomicAdd(&s.few_n, 1u)] = t.p[i];
  __syncthreads();
  *found = among_few(q, sort_few(r, s.few, (int)n), before);
  return true;
}

// The answer from the row itself, read by this block: its bin by places, nine bits at a time, down to a single token
// if need be; from LDS once its tokens fit.
template <bool BF>
__device__ __forceinline__ Found answer_row(const SampleArgs& a, int64_t b, const Row& r, const Asked& q, int bin,
                                            Pair before, u64 n, Shared& s) {
  const int tid = threadIdx.x;
  Range g = places_of(r, bin);
  auto in = [&](u64 p) { return p >= g.lo && p <= g.hi; };
  auto gather = [&] {
    __syncthreads();
    if (tid == 0) s.count = 0;
    __syncthreads();
    each<BF>(a, b, g, [&](bool is, u64 p) {
      if (is) {
        const uint32_t at = atomicAdd(&s.count, 1u);
        if (at < kList) s.list[at] = p;
      }
    });
    __syncthreads();
  };
  bool listed = false;
  while (n > kSmall) {
    if (!listed && n <= kList) {
      gather();
      listed = true;
    }
    const int bits = 64 - __clzll((long long)(g.hi - g.lo)), shift = max(bits - 9, 0);
    static_assert(kBins == 512, "nine bits");
    __syncthreads();
    s.split[tid] = {0, 0};
    __syncthreads();
    auto part_at = [&](u64 p) { return (uint32_t)((p - g.lo) >> shift); };
    if (listed) {
      for (int i0 = 0; i0 < (int)s.count; i0 += kThreads) {
        const u64 p = s.list[min(i0 + tid, (int)s.count - 1)];
        const bool is = i0 + tid < (int)s.count && in(p);
        split_add(r, s, is, p, is ? part_at(p) : 0);
      }
    } else {
      each<BF>(a, b, g, [&](bool is, u64 p) { split_add(r, s, is, p, is ? part_at(p) : 0); });
    }
    const int k = split_choose(q, s, &before, &n);
    g.lo += (u64)k << shift;
    g.hi = min(g.hi, g.lo + (((u64)1 << shift) - 1));
  }
  if (!listed) gather();
  return among_some(r, q, (int)n, before, s, in);
}

template <bool BF, bool VEC>
__global__ __launch_bounds__(kThreads) void sample_draw_kernel(SampleArgs a) {
  __shared__ Shared s;
  const int tid = threadIdx.x;
  const int64_t b = blockIdx.y;
  // workgroups are dealt to the XCDs in turn, so a row's first chunk is on another one than the last row's
  const int64_t part = (blockIdx.x + blockIdx.y) % a.chunks;
  const int chunk = min<int64_t>(tid & 63, a.chunks - 1);
  const Settings st = settings_of(a, b);
  const Extremes ex = row_extremes(a, b);
  SamplePlan* const plan_at = a.plan + b;
  Head plan;                             // a greedy row has none, and does not look at it
  plan.ranges = plan_at->ranges;
  plan.upto = plan_at->upto;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    plan.bin0[i] = plan_at->bin0[i];
    plan.bin1[i] = plan_at->bin1[i];
  }
  double exps = a.exps[b * a.chunks + chunk];
  u64 sum_m = a.kept[b * a.chunks + chunk];
  const ulonglong2 mine = ((const ulonglong2*)a.sums)[b * kBins + tid];
  u64 best;
  const Row r = row_of_extremes(ex, st, &best);
  const bool masked = r.top == -__builtin_inf();
  int64_t token = masked ? -1 : (int64_t)(uint32_t)best;
  const bool draws = !st.greedy && !masked;
  const bool alone = !draws || plan.ranges == 0 || few_groups(a, plan);   // one block does it all
  if (alone && part > 0) return;
  if (draws) {
    if (tid == 0) s.count = 0;
    s.bins[tid] = {mine.x, mine.y};
    __syncthreads();
    const u64* elsewhere = nullptr;
    uint32_t tokens = 0;
    if (plan.ranges) {
      if (alone) gather_groups<BF, VEC>(a, b, r, plan, s);
      else gather_chunk<BF, VEC>(a, b, part, r, plan, s);
      tokens = s.count;
      if (!alone && a.chunks > 1) {      // the row's list, by whichever block is last
        u64* const lists = a.lists + b * kList;
        if (tid == 0 && tokens)
          s.at = __hip_atomic_fetch_add(&plan_at->count, tokens, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        for (uint32_t i = tid; i < tokens; i += kThreads)
          if (s.at + i < kList) put(lists + s.at + i, s.list[i]);
        if (!last_to_arrive(&plan_at->arrived, (uint32_t)a.chunks, &s.last)) return;
        tokens = get(&plan_at->count);
        elsewhere = lists;
      }
      tokens = min(tokens, (uint32_t)kList);
    }
    Mine t;
    if (elsewhere) {
#pragma unroll
      for (int i = 0; i < kEach; ++i)
        if (i * kThreads < tokens) t.p[i] = get(elsewhere + min(i * kThreads + tid, (int)tokens - 1));
    } else {
#pragma unroll
      for (int i = 0; i < kEach; ++i)
        if (i * kThreads < tokens) t.p[i] = s.list[min(i * kThreads + tid, (int)tokens - 1)];
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      t.fine[i] = -1;
      if (i * kThreads >= tokens) continue;
      const float x = logit_at(t.p[i]);
      t.w[i] = weight_of(r, x);
      t.fine[i] = i * kThreads + tid < tokens ? fine_of(r, x) : -1;
    }
    const bool small = plan.ranges == 1 && tokens <= kSmall;     // one order answers all questions
    Few few = {0, 0, 0};
    if (small) {
      if (tid < (int)tokens) s.few[tid] = t.p[0];
      __syncthreads();
      few = sort_few(r, s.few, (int)tokens);
    }
    sum_m = wave_all((tid & 63) < a.chunks ? sum_m : 0, (u64)0, Add());
    const Pair all = s.bins[kBins - 1];
    const u64 k = st.k && (u64)st.k < all.n ? (u64)st.k : 0;
    const double u = a.u[b];
    u64 sum = all.w;
    // the questions in turn by the same code, which is fetched once
#pragma unroll 1
    for (int question = k ? kCount : st.p < 1.0 ? kGoal : kPass; question <= kPass; ++question) {
      Asked q = {(Question)question, k, st.p * (double)sum, 0};
      if (question == kGoal && !(st.p < 1.0)) continue;
      if (question == kPass) {
        if (st.min_w) sum = min(sum, max(sum_m, (u64)kOne));
        const double at = u > 0.0 ? fmin(u, 1.0) * (double)sum : 0.0;   // NaN: 0
        q.r = min((u64)at, sum - 1);
      }
      const int bin = small ? plan.bin0[0] : first_bin(q, s.bins, {0, 0});
      const Pair before = bin ? s.bins[bin - 1] : Pair{0, 0};
      const u64 n = s.bins[bin].n - before.n;
      Found f;
      bool held = plan.ranges > 0;
      if (small) {
        f = among_few(q, few, before);
      } else {
        bool named = false;
#pragma unroll
        for (int i = 0; i < 3; ++i) named |= plan.bin0[i] <= bin && bin <= plan.bin1[i];
        held = held && named && answer_mine(r, q, t, bin, before, n, s, &f);
        if (!held) f = answer_row<BF>(a, b, r, q, bin, before, n, s);
      }
      sum = min(sum, f.sum);
      token = f.token;
    }
    token = min(token, a.V - 1);         // within the row whatever a workspace that two calls write at once may hold
  }
  if (tid >= 64) return;
  exps = wave_all(tid < a.chunks ? exps : 0.0, 0.0, Add());
  if (tid == 0) {
    a.token[b] = (int32_t)token;
    if (a.logprob) {
      float lp = kNegInf;
      if (!masked) {
        const void* row = row_of<BF>(a, b);
        const float x = BF ? __uint_as_float((uint32_t)((const uint16_t*)row)[token] << 16) : ((const float*)row)[token];
        lp = (float)((r.inf ? 0.0 : (double)x - r.top) - log(exps));
      }
      a.logprob[b] = lp;
    }
  }
}

template <bool BF, bool VEC>
hipError_t run(const SampleArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)a.chunks, (unsigned)a.B);
  sample_max_kernel<BF, VEC><<<grid, kThreads, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  sample_hist_kernel<BF, VEC><<<grid, kThreads, 0, s>>>(a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  sample_draw_kernel<BF, VEC><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_sample(const SampleArgs& a, bool bf16, bool vec, hipStream_t s) {
  if (bf16) return vec ? run<true, true>(a, s) : run<true, false>(a, s);
  return vec ? run<false, true>(a, s) : run<false, false>(a, s);
}

}  // namespace bl
