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
  double per_bin;                        // bins per unit of (x - top) * c
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

// v of the lane that a DPP control names, `id` where there is none or the row mask leaves the lane out.
template <int CTRL, int ROWS, class T>
__device__ __forceinline__ T lane_move(T v, T id) {
  if constexpr (sizeof(T) == 8) {
    const uint2 x = __builtin_bit_cast(uint2, v), y = __builtin_bit_cast(uint2, id);
    const uint2 z = {(uint32_t)__builtin_amdgcn_update_dpp((int)y.x, (int)x.x, CTRL, ROWS, 0xF, false),
                     (uint32_t)__builtin_amdgcn_update_dpp((int)y.y, (int)x.y, CTRL, ROWS, 0xF, false)};
    return __builtin_bit_cast(T, z);
  } else {
    return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, id), __builtin_bit_cast(int, v),
                                                             CTRL, ROWS, 0xF, false));
  }
}
// op over the lanes up to each one (id: what changes nothing), in registers: within rows of 16 lanes, then over
// them.  The order is fixed.
template <class T, class Op>
__device__ __forceinline__ T wave_scan(T v, T id, Op op) {
  v = op(lane_move<0x111, 0xF>(v, id), v);   // 1, 2, 4, 8 lanes up the row
  v = op(lane_move<0x112, 0xF>(v, id), v);
  v = op(lane_move<0x114, 0xF>(v, id), v);
  v = op(lane_move<0x118, 0xF>(v, id), v);
  v = op(lane_move<0x142, 0xA>(v, id), v);   // last lane of a row to the next one
  v = op(lane_move<0x143, 0xC>(v, id), v);   // of the lower half to the upper
  return v;
}
template <class T>
__device__ __forceinline__ T lane_value(T v, int lane) {
  if constexpr (sizeof(T) == 8) {
    const uint2 x = __builtin_bit_cast(uint2, v);
    const uint2 z = {(uint32_t)__builtin_amdgcn_readlane((int)x.x, lane), (uint32_t)__builtin_amdgcn_readlane((int)x.y, lane)};
    return __builtin_bit_cast(T, z);
  } else {
    return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
  }
}
template <class T, class Op>
__device__ __forceinline__ T wave_all(T v, T id, Op op) {
  return lane_value(wave_scan(v, id, op), 63);
}
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
__device__ __forceinline__ int bin_of(const Row& r, double t) { return min((int)(-t * r.per_bin), kBins - 1); }

// 2^40 * 2^t rounded to a whole number, t <= 0.  2^f for |f| <= 1/2 by its Taylor sum: the first term left out
// is below 2^-57.  Adding 2^52 rounds to a whole number, half to even.
__device__ __forceinline__ u64 weight(double t) {
  if (!(t > -41.0)) return 0;
  const double n = rint(t), f = t - n;
  double p = 2.5678435993488196e-11;                       // (ln 2)^12 / 12!
  p = __builtin_fma(p, f, 4.4455382718708102e-10);
  p = __builtin_fma(p, f, 7.0549116208011211e-09);
  p = __builtin_fma(p, f, 1.0178086009239696e-07);
  p = __builtin_fma(p, f, 1.3215486790144305e-06);
  p = __builtin_fma(p, f, 1.5252733804059838e-05);
  p = __builtin_fma(p, f, 1.5403530393381606e-04);
  p = __builtin_fma(p, f, 1.3333558146428441e-03);
  p = __builtin_fma(p, f, 9.6181291076284771e-03);
  p = __builtin_fma(p, f, 5.5504108664821576e-02);
  p = __builtin_fma(p, f, 2.4022650695910070e-01);
  p = __builtin_fma(p, f, 6.9314718055994531e-01);
  p = __builtin_fma(p, f, 1.0);
  const double w = ldexp(p, 40 + (int)n) + 4503599627370496.0;
  return (u64)__double_as_longlong(w) & 0xFFFFFFFFFFFFFull;
}

struct Settings {
  double temp, p, min_p;
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
  s.min_p = m > 0.f ? (double)m : 0.0;
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
  const double range = r.inf ? 0.0 : fmin(((double)x - least) * r.c, 41.0);
  r.per_bin = range > 0.0 ? kBins / range : 0.0;
  if (!(r.per_bin < 1e30)) r.per_bin = 0.0;                // too narrow to be told apart: one bin
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

// Whether a falling() value's logit weighs something and lies in a bin up to `bin`.
__device__ __forceinline__ bool reaches(const Row& r, uint64_t key, int bin) {
  const float x = from_falling((uint32_t)key);
  const double t = scaled(r, x);
  return x == x && weight(t) > 0 && bin_of(r, t) <= bin;
}
// Largest falling() value that reaches up to a bin; the row's largest logit always does.  The lanes of a wave try 64
// values at a time.
__device__ __forceinline__ u64 key_end(const Row& r, int bin) {
  const int lane = threadIdx.x & 63;
  uint64_t lo = falling((float)r.top), hi = (uint64_t)1 << 32;   // lo does, hi does not
  while (hi - lo > 1) {
    const uint64_t step = (hi - lo + 63) >> 6, at = lo + lane * step;
    const uint64_t mask = __ballot(at < hi && reaches(r, at, bin));
    const int last = 63 - __clzll((long long)mask);
    hi = min(hi, lo + (last + 1) * step);
    lo += last * step;
  }
  return lo;
}
// Places of the tokens of bins bin0 to bin1.  Half of the lanes try the 32 values around where each end should be.
__device__ __forceinline__ Range places_of(const Row& r, int bin0, int bin1) {
  const int lane = threadIdx.x & 63;
  const bool upper = lane >= 32;
  const int bin = upper ? bin1 : max(bin0 - 1, 0);
  const uint64_t top = falling((float)r.top);
  const double t = r.per_bin > 0.0 && bin < kBins - 1 ? fmin((bin + 1) / r.per_bin, 41.0) : 41.0;
  const uint64_t guess = r.inf ? top : falling((float)(r.top - t / r.c));
  const uint64_t at = min(max(guess, top + 16) - 16, ((uint64_t)1 << 32) - 32) + (lane & 31);
  const uint64_t mask = __ballot(reaches(r, at, bin));
  const uint32_t m0 = (uint32_t)mask, m1 = (uint32_t)(mask >> 32);
  const u64 end0 = (m0 & 1) && !(m0 >> 31) ? lane_value((u64)at, 31 - __clz((int)m0)) : key_end(r, max(bin0 - 1, 0));
  const u64 end1 = (m1 & 1) && !(m1 >> 31) ? lane_value((u64)at, 63 - __clz((int)m1)) : key_end(r, bin1);
  return {(bin0 ? end0 + 1 : top) << 32, end1 << 32 | 0xFFFFFFFFu};
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
__device__ __forceinline__ void make_plan(SamplePlan* plan, const Row& r, const Settings& st, u64 sum_m, double u,
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
  if (st.min_p > 0.0) {
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
  for (int i = 0; i < n; ++i) {
    const Range g = places_of(r, b0[i], b1[i]);
    if (threadIdx.x == 0) {
      plan->lo[i] = g.lo;
      plan->hi[i] = g.hi;
      plan->bin0[i] = b0[i];
      plan->bin1[i] = b1[i];
    }
  }
  if (threadIdx.x == 0) {
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
  const double min_w = st.min_p * kOne;
  const float top = (float)r.top;
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
      finish8_masked<BF, VEC>(row, i + k * kStep, a.V, v[k]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = v[k][j];
        if (a.logprob) e += r.inf ? (x == top ? 1.0 : 0.0) : (double)__builtin_amdgcn_exp2f((x - top) * 1.44269504f);
        if (st.greedy) continue;
        const double t = scaled(r, x);
        const u64 w = weight(t);
        if (w) {
          const int bin = bin_of(r, t);
          atomicAdd(&w_bin[bin], w);
          atomicAdd(&n_bin[bin], 1u);
          if ((double)w >= min_w) least_sum += w;
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
  if (tid < 64) make_plan(a.plan + b, r, st, sum_m, u, bins);
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
  Range range[3];
  int bin0[3], bin1[3];
  uint32_t ranges, upto;
};

struct Bounds {                          // the logits of a range: a little wider where it ends among equals
  float lo, hi;
};
__device__ __forceinline__ Bounds bounds_of(const Range& g) {
  const uint32_t key0 = (uint32_t)(g.lo >> 32), key1 = (uint32_t)(g.hi >> 32);
  // the value of -0, which no logit has, is above +0's: a range must not reach back to it
  return {from_falling(key1), from_falling(key0 == 0x80000000u ? key0 + 1 : key0)};
}
__device__ __forceinline__ bool inside(const Bounds& b, float x) {     // a NaN equals nothing
  return __builtin_amdgcn_fmed3f(x, b.lo, b.hi) == x;
}

// Appends to the list the logits of eight per lane, from index i on, that ok(x, place) says yes to.
template <class F>
__device__ __forceinline__ void append(Shared& s, const float v[8], int64_t i, F&& ok) {
  const int lane = threadIdx.x & 63;
  uint64_t mask[8];
  uint32_t all = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    mask[j] = __ballot(ok(v[j], place(v[j], i + j)));
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

// The list: the tokens of the plan's one range, few enough for one block to read the groups of 64 logits again whose
// largest reaches it, eight lanes to each.
__device__ __forceinline__ bool few_groups(const SampleArgs& a, const Head& plan) {
  return plan.ranges == 1 && (int64_t)plan.upto * 128 <= a.V;
}
template <bool BF, bool VEC>
__device__ __forceinline__ void gather_groups(const SampleArgs& a, int64_t b, const Head& plan, Shared& s) {
  const int tid = threadIdx.x;
  const void* row = row_of<BF>(a, b);
  const Bounds bd = bounds_of(plan.range[0]);
  uint32_t* groups = (uint32_t*)s.split;                     // room for kAll
  constexpr int kAll = 4 * kThreads;
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
      if (i < a.groups && m[k] >= bd.lo) groups[atomicAdd(&s.at, 1u)] = (uint32_t)i;
    }
    __syncthreads();
    const int n = s.at;
    for (int k0 = 0; k0 < n; k0 += kThreads / 8) {
      const int k = k0 + (tid >> 3);
      const int64_t i = k < n ? (int64_t)groups[k] * 64 + (tid & 7) * 8 : a.V;
      float v[8];
      load8_raw<BF, VEC>(row, i, a.V, v);
      finish8<BF, VEC>(row, i, a.V, v);
      append(s, v, i, [&](float x, u64) { return inside(bd, x); });
    }
    __syncthreads();
  }
}

// The list: this block's chunk of the tokens that the plan names.
template <bool BF, bool VEC>
__device__ __forceinline__ void gather_chunk(const SampleArgs& a, int64_t b, const Head& plan, Shared& s) {
  const void* row = row_of<BF>(a, b);
  const int64_t i0 = (int64_t)blockIdx.x * a.chunk, i1 = min(i0 + a.chunk, a.V);
  const bool more = plan.ranges > 1, third = plan.ranges > 2;
  const Bounds b0 = bounds_of(plan.range[0]), b1 = more ? bounds_of(plan.range[1]) : b0,
               b2 = third ? bounds_of(plan.range[2]) : b0;
  for (int64_t at = i0; at < i1; at += 2 * kStep) {
    const int64_t i = at + threadIdx.x * 8;
    float v[2][8];
#pragma unroll
    for (int k = 0; k < 2; ++k) load8_raw<BF, VEC>(row, i + k * kStep, a.V, v[k]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (at + k * kStep >= i1) break;
      finish8<BF, VEC>(row, i + k * kStep, i1, v[k]);        // a chunk is a multiple of eight, but for the row's end
      append(s, v[k], i + k * kStep, [&](float x, u64) {
        return inside(b0, x) || (more && inside(b1, x)) || (third && inside(b2, x));   // ranges do not meet
      });
    }
  }
  __syncthreads();
}

// Calls f(v, i) for eight logits of a lane from index i on where any lane of the wave has one within the range's
// bounds: the whole row, by one block.
template <bool BF, bool VEC, class F>
__device__ __forceinline__ void each(const SampleArgs& a, int64_t b, const Range& g, F&& f) {
  constexpr int kRing = 4;
  const void* row = row_of<BF>(a, b);
  const Bounds bd = bounds_of(g);
  float v[kRing][8];
  const int64_t first = threadIdx.x * 8;
#pragma unroll
  for (int u = 0; u < kRing; ++u) load8_raw<BF, VEC>(row, first + u * kStep, a.V, v[u]);
  for (int64_t at = 0; at < a.V; at += kRing * kStep) {
#pragma unroll
    for (int u = 0; u < kRing; ++u) {
      const int64_t i = at + u * kStep + first;
      finish8<BF, VEC>(row, i, a.V, v[u]);
      bool any = false;
#pragma unroll
      for (int j = 0; j < 8; ++j) any |= inside(bd, v[u][j]);
      if (__any(any)) f(v[u], i);
      load8_raw<BF, VEC>(row, i + kRing * kStep, a.V, v[u]);
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
  const u64 w = lane < n ? weight(scaled(r, logit_at(p))) : 0;
  int rank = lane < n ? 0 : lane;
  for (int j = 0; j < n; ++j) rank += lane_value(p, j) < p && lane < n;
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
  const u64 w = weight(scaled(r, logit_at(p)));
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

// The answer wherever it lies.  The list holds the tokens of the plan's ranges.
template <bool BF, bool VEC>
__device__ __forceinline__ Found answer(const SampleArgs& a, int64_t b, const Row& r, const Asked& q,
                                        Head& plan, Shared& s) {
  const int tid = threadIdx.x;
  const Pair none = {0, 0};
  const int bin = first_bin(q, s.bins, none);
  bool listed = false;
#pragma unroll
  for (int i = 0; i < 3; ++i) listed |= i < (int)plan.ranges && plan.bin0[i] <= bin && bin <= plan.bin1[i];
  Pair before = bin ? s.bins[bin - 1] : none;
  u64 n = s.bins[bin].n - before.n;
  if (listed) {
    // the list's tokens of the bin, by bins within the bin if they are many
    auto bin_at = [&](u64 p) { return bin_of(r, scaled(r, logit_at(p))); };
    if (n <= kSmall) return among_some(r, q, (int)n, before, s, [&](u64 p) { return bin_at(p) == bin; });
    auto part_at = [&](u64 p) {
      const double y = -scaled(r, logit_at(p)) * r.per_bin;
      return min(max((int)((y - bin) * kBins), 0), kBins - 1);   // the last bin's may lie past it
    };
    const Pair outside = before;
    u64 few = n;
    __syncthreads();
    s.split[tid] = none;
    __syncthreads();
    for (int i0 = 0; i0 < (int)s.count; i0 += kThreads) {
      const u64 p = s.list[min(i0 + tid, (int)s.count - 1)];
      const bool in = i0 + tid < (int)s.count && bin_at(p) == bin;
      split_add(r, s, in, p, in ? part_at(p) : 0);
    }
    const int part = split_choose(q, s, &before, &few);
    if (few <= kSmall)
      return among_some(r, q, (int)few, before, s, [&](u64 p) { return bin_at(p) == bin && part_at(p) == part; });
    before = outside;
  }
  // by places, nine bits at a time, down to a single token if need be
  if (!listed) plan.ranges = 0;          // the list is written over
  Range g = places_of(r, bin, bin);
  while (n > kSmall) {
    if (!listed && n <= kList) {
      __syncthreads();
      if (tid == 0) s.count = 0;
      __syncthreads();
      each<BF, VEC>(a, b, g, [&](const float* v, int64_t i) {
        append(s, v, i, [&](float, u64 p) { return p >= g.lo && p <= g.hi; });
      });
      listed = true;
    }
    const int bits = 64 - __clzll((long long)(g.hi - g.lo)), shift = max(bits - 9, 0);
    static_assert(kBins == 512, "nine bits");
    __syncthreads();
    s.split[tid] = none;
    __syncthreads();
    auto part_at = [&](u64 p) { return (uint32_t)((p - g.lo) >> shift); };
    if (listed) {
      for (int i0 = 0; i0 < (int)s.count; i0 += kThreads) {
        const u64 p = s.list[min(i0 + tid, (int)s.count - 1)];
        const bool in = i0 + tid < (int)s.count && p >= g.lo && p <= g.hi;
        split_add(r, s, in, p, in ? part_at(p) : 0);
      }
    } else {
      each<BF, VEC>(a, b, g, [&](const float* v, int64_t i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const u64 p = place(v[j], i + j);
          const bool in = p >= g.lo && p <= g.hi;
          split_add(r, s, in, p, in ? part_at(p) : 0);
        }
      });
    }
    const int k = split_choose(q, s, &before, &n);
    g.lo += (u64)k << shift;
    g.hi = min(g.hi, g.lo + (((u64)1 << shift) - 1));
  }
  auto in = [&](u64 p) { return p >= g.lo && p <= g.hi; };
  if (!listed) {
    __syncthreads();
    if (tid == 0) s.count = 0;
    __syncthreads();
    each<BF, VEC>(a, b, g, [&](const float* v, int64_t i) { append(s, v, i, [&](float, u64 p) { return in(p); }); });
  }
  return among_some(r, q, (int)n, before, s, in);
}

template <bool BF, bool VEC>
__global__ __launch_bounds__(kThreads) void sample_draw_kernel(SampleArgs a) {
  __shared__ Shared s;
  const int tid = threadIdx.x;
  const int64_t b = blockIdx.y;
  const int chunk = min<int64_t>(tid & 63, a.chunks - 1);
  const Settings st = settings_of(a, b);
  const Extremes ex = row_extremes(a, b);
  SamplePlan* const plan_at = a.plan + b;
  Head plan;                             // a greedy row has none, and does not look at it
  plan.ranges = plan_at->ranges;
  plan.upto = plan_at->upto;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    plan.range[i] = {plan_at->lo[i], plan_at->hi[i]};
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
  if (alone && blockIdx.x > 0) return;
  if (draws) {
    if (tid == 0) s.count = 0;
    s.bins[tid] = {mine.x, mine.y};
    __syncthreads();
    if (plan.ranges && alone) gather_groups<BF, VEC>(a, b, plan, s);
    if (!alone) {
      gather_chunk<BF, VEC>(a, b, plan, s);
      if (a.chunks > 1) {                // the row's list, by whichever block is last
        u64* const lists = a.lists + b * kList;
        const uint32_t n = s.count;
        if (tid == 0 && n)
          s.at = __hip_atomic_fetch_add(&plan_at->count, n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        for (uint32_t i = tid; i < n; i += kThreads)
          if (s.at + i < kList) put(lists + s.at + i, s.list[i]);
        if (!last_to_arrive(&plan_at->arrived, (uint32_t)a.chunks, &s.last)) return;
        const uint32_t all = min(get(&plan_at->count), (uint32_t)kList);
        for (uint32_t i = tid; i < all; i += kThreads) s.list[i] = get(lists + i);
        if (tid == 0) s.count = all;
        __syncthreads();
      }
    }
    sum_m = wave_all((tid & 63) < a.chunks ? sum_m : 0, (u64)0, Add());
    const Pair all = s.bins[kBins - 1];
    const u64 k = st.k && (u64)st.k < all.n ? (u64)st.k : 0;
    const bool small = plan.ranges == 1 && s.count <= kSmall;    // one order answers all questions
    Few few = {0, 0, 0};
    if (small) few = sort_few(r, s.list, s.count);
    const Pair above = small && plan.bin0[0] ? s.bins[plan.bin0[0] - 1] : Pair{0, 0};
    auto ask = [&](const Asked& q) { return small ? among_few(q, few, above) : answer<BF, VEC>(a, b, r, q, plan, s); };
    u64 sum = all.w;
    if (k) sum = ask({kCount, k, 0.0, 0}).sum;
    if (st.p < 1.0) sum = min(sum, ask({kGoal, 0, st.p * (double)sum, 0}).sum);
    if (st.min_p > 0.0) sum = min(sum, max(sum_m, (u64)kOne));
    const double u = a.u[b];
    const double at = u > 0.0 ? fmin(u, 1.0) * (double)sum : 0.0;     // NaN: 0
    token = ask({kPass, 0, 0.0, min((u64)at, sum - 1)}).token;
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
