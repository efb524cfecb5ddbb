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
//   max    blocks find largest and least logit of a chunk of a row, and the largest of each 64
//   hist   blocks count a chunk's tokens and sum their weights by 1024 bins of top - x.  The last block of a row adds the
//          chunks' bins up, finds the bins that the questions' answers lie in, and plans which tokens to gather: where
//          those up to the first question's bin are kList at most (top-k and top-p as they are used) all of them, once
//          for all questions, else those of each question's bin or few bins
//   draw   tokens are gathered by one block, from the groups of 64 whose largest reaches them, or by all blocks from all
//          logits, for the last of them.  The one that has them answers the questions: a bin by its fine bins, equal
//          logits (bf16 ones above all) by place (value, then index), until a wave can sort what is left.  If more than
//          kList tokens are planned for, one block reads the row and splits its bins by place
// Largest and least logit bound the bins (what weighs nothing aside), so that they are as fine as the row allows: 1024
// leave 420 tokens in the fullest of 131072 normal logits.  The questions' bins hold more than kList tokens where a wide
// top-k (a quarter of the row or more) meets top-p, each question known to within a few bins of the one before: on flat rows
// from about 200000 logits on (262144 with a deviation of 1/2, top-k of half and top-p 0.98: one row that fits 50 us, 16 some
// of which do not 200), and where many finite masks widen the bins (131072 logits, half of them -10000, top-k of 32768 and
// top-p 0.9: 124 us, 38 with -inf in their place); and for top-p alone where one far logit does (16 rows of 131072 with one
// at -60 93 us, 38 without).
//
// Latency bounds one row: 131072 logits take 3.8, 14 and 9 us in the three launches, each a chain of dependent loads, a
// hand-over between blocks (past the caches, that the XCDs do not share) and steps in LDS.  64 rows of mixed settings take
// 8.4 (4 TB/s), 25.5 and 26 us: 28 vector instructions a weight and 15 for the log probability, and rows that wait for their
// last block.
#include <algorithm>

#include "block_ops.hpp"
#include "device_common.hpp"
#include "step_ops.hpp"
#include "wave_ops.hpp"

namespace bl {

namespace {

typedef unsigned long long u64;

constexpr int kBins = kSampleBins;
constexpr int kParts = 512;              // fine bins of a bin, and parts that one is split into otherwise
constexpr int kList = kSampleList;       // tokens that are gathered
constexpr int kThreads = 512;            // of every block
constexpr int kWaves = kThreads / 64;
constexpr int kStep = kThreads * 8;      // logits that a block loads at a time
static_assert(2 * kThreads == kBins && kThreads == kParts, "two bins, and one part, to a thread");
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

// Eight elements from anywhere: the loads of 16 bytes need no more than the elements' own alignment.
typedef uint32_t v4u_of_bf16 __attribute__((ext_vector_type(4), aligned(2)));
typedef float v4f_of_f32 __attribute__((ext_vector_type(4), aligned(4)));
template <bool BF>
__device__ __forceinline__ void load8_any(const void* row, int64_t i, float v[8]) {
  if constexpr (BF) {
    const v4u_of_bf16 w = *(const v4u_of_bf16*)((const uint16_t*)row + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = bf16_lo(w[j]);
      v[2 * j + 1] = bf16_hi(w[j]);
    }
  } else {
    const v4f_of_f32 x = *(const v4f_of_f32*)((const float*)row + i), y = *(const v4f_of_f32*)((const float*)row + i + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = x[j];
      v[4 + j] = y[j];
    }
  }
}
// Elements i .. i + 8 of a row without a branch around a load, so that many can be in flight: vector loads of whole
// eights (what is past them is loaded as the last one and left out below), and where a row has no eight, element by
// element.
template <bool BF, bool VEC>
__device__ __forceinline__ void load8_raw(const void* row, int64_t i, int64_t V, float v[8]) {
  if constexpr (VEC) {
    load8_any<BF>(row, max(min(i, V / 8 * 8 - 8), (int64_t)0), v);
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
// The largest and least of three numbers, none of them NaN: one instruction, where fmaxf quiets its operands first.
__device__ __forceinline__ float max3(float x, float y, float z) {
  float m;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(m) : "v"(x), "v"(y), "v"(z));
  return m;
}
__device__ __forceinline__ float min3(float x, float y, float z) {
  float m;
  asm("v_min3_f32 %0, %1, %2, %3" : "=v"(m) : "v"(x), "v"(y), "v"(z));
  return m;
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
// The logit's place among the fine bins of the row's range, kParts of them to a bin: any steps that rise as x falls
// will do, so fp32 is enough.  NaN (equals of an infinite top) counts as 0.
__device__ __forceinline__ int fine_of(const Row& r, float x) {
  return (int)__builtin_amdgcn_fmed3f(((float)r.top - x) * r.per_fine, 0.f, (float)(kBins * kParts - 1));
}

// a * b + c in fp64 with c from scalar registers: a multiply-add that ends where c was would copy it there first.
__device__ __forceinline__ double fma_const(double a, double b, double c) {
  double d;
  asm("v_fma_f64 %0, %1, %2, %3" : "=v"(d) : "v"(a), "v"(b), "s"(c));
  return d;
}
// 2^40 * 2^t rounded to a whole number, t <= 0 (NaN: 0).  2^f for |f| <= 1/2 is a polynomial through the eleven
// Chebyshev points, 2.4e-16 off at most, its coefficients times 2^40.  Adding 1.5 * 2^52 rounds to a whole number, half
// to even, in a double's low bits.
__device__ __forceinline__ u64 weight(double t) {
  const double magic = 6755399441055744.0;
  t = __builtin_fmax(t, -60.0);
  const double m = t + magic, f = t - (m - magic);
  double p = fma_const(f, 0x1.e6063f7217bc6p+12, 0x1.b675bca4eeebbp+16);
  p = fma_const(p, f, 0x1.62bfd47773353p+20);
  p = fma_const(p, f, 0x1.ffcb54062e698p+23);
  p = fma_const(p, f, 0x1.430913096fd9fp+27);
  p = fma_const(p, f, 0x1.5d87fe9d7a584p+30);
  p = fma_const(p, f, 0x1.3b2ab6fba1ddap+33);
  p = fma_const(p, f, 0x1.c6b08d703ce49p+35);
  p = fma_const(p, f, 0x1.ebfbdff82c598p+37);
  p = fma_const(p, f, 0x1.62e42fefa3a19p+39);
  p = fma_const(p, f, 0x1.0p+40);
  const uint2 bits = __builtin_bit_cast(uint2, __builtin_ldexp(p, (int)__builtin_bit_cast(uint2, m).x) + magic);
  return (u64)(bits.y & 0x7FFFFu) << 32 | bits.x;
}
// 2^t, t <= 0 (NaN, and what is below 2^-1000: nothing that counts), for sums of exp(x - top): a polynomial of (2^f - 1) / f
// through the seven Chebyshev points, the result within 2^-33 of itself; exp2 in fp32 was off by the rounding of t, 10^-6 of
// a term 13 below the largest, which showed where one token holds most of the probability (64 rows of 131072, mixed
// settings: 25.5 us in the second launch, 22 by exp2).
__device__ __forceinline__ double power(double t) {
  const double magic = 6755399441055744.0;
  t = __builtin_fmax(t, -1000.0);
  const double m = t + magic, f = t - (m - magic);
  double p = fma_const(f, 0x1.00a5814a072d8p-16, 0x1.443fffcad88f1p-13);
  p = fma_const(p, f, 0x1.5d879ead1ff74p-10);
  p = fma_const(p, f, 0x1.3b2a1b71506d0p-7);
  p = fma_const(p, f, 0x1.c6b08d883db6cp-5);
  p = fma_const(p, f, 0x1.ebfbe045f4d65p-3);
  p = fma_const(p, f, 0x1.62e42fefa39efp-1);
  p = fma_const(p, f, 1.0);
  return __builtin_ldexp(p, (int)__builtin_bit_cast(uint2, m).x);
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
  const float per_fine = (float)(kBins * kParts / fmin((double)x - least, 41.0 / r.c));
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

// First of N bins whose running sums, behind `before`, answer the question (the last one that adds anything, if none
// does).  Every wave finds it by itself: 64 ends of a few bins, then the few.
template <int N>
__device__ __forceinline__ int first_bin(const Asked& q, const Pair* bins, const Pair& before) {
  constexpr int kFew = N / 64;
  const int lane = threadIdx.x & 63;
  const u64 all = bins[N - 1].n;
  auto yes = [&](int i) {
    const Pair p = bins[i];
    return __ballot(met(q, before + p) || p.n == all);       // rising: once it is so it stays so
  };
  const int few = __ffsll((unsigned long long)yes(lane * kFew + kFew - 1)) - 1;
  return few * kFew + __ffsll((unsigned long long)yes(few * kFew + lane % kFew)) - 1;
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
    const uint64_t mask = __ballot(at < hi && x == x && weight_of(r, x) > 0 && fine_of(r, x) / kParts <= bin);
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
      finish8<BF, VEC>(row, i + k * kStep, a.V, v[k]);
      float most = kNegInf;
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const bool is0 = v[k][j] > kNegInf, is1 = v[k][j + 1] > kNegInf;   // neither -inf nor NaN
        least = min3(least, is0 ? v[k][j] : __builtin_inff(), is1 ? v[k][j + 1] : __builtin_inff());
        v[k][j] = is0 ? v[k][j] : kNegInf;
        v[k][j + 1] = is1 ? v[k][j + 1] : kNegInf;
        most = max3(most, v[k][j], v[k][j + 1]);
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
    const int bin = first_bin<kBins>({kCount, k, 0.0, 0}, bins, none);
    lo = upto(bin - 1).w;
    hi = upto(bin).w;
    b0[0] = b1[0] = bin;
    n = 1;
  }
  if (st.p < 1.0 && !(n && upto(b1[0]).n <= kList)) {
    const int bin0 = first_bin<kBins>({kGoal, 0, st.p * (double)lo, 0}, bins, none);
    const int bin1 = first_bin<kBins>({kGoal, 0, st.p * (double)hi, 0}, bins, none);
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
    b0[n] = first_bin<kBins>({kPass, 0, 0.0, min((u64)(part * (double)lo), max(lo, (u64)1) - 1)}, bins, none);
    b1[n++] = first_bin<kBins>({kPass, 0, 0.0, min((u64)(part * (double)hi), hi - 1)}, bins, none);
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
  // Bins of what two waves add in a turn: a sum of weights and, from bit 52 on, their number, in one addition.  2048 weights
  // of at most 2^40 stay below.
  constexpr int kTables = kWaves / 2, kCountAt = 52;
  static_assert(2 * kStep / kTables <= 1 << 11 && 2 * kStep == 8192, "a turn's sums and numbers fit");
  __shared__ __attribute__((aligned(16))) u64 tables[kTables][kBins];
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
#pragma unroll
  for (int t = 0; t < kTables; ++t) *(ulonglong2*)(tables[t] + 2 * tid) = make_ulonglong2(0, 0);
  __syncthreads();
  const void* row = row_of<BF>(a, b);
  const int64_t i0 = (int64_t)blockIdx.x * a.chunk, i1 = min(i0 + a.chunk, a.V);
  const double dtop = r.inf ? 0.0 : r.top;
  const float top = (float)dtop, per_bin = r.per_fine / kParts;
  double e = 0.0;                                          // sum of exp(x - top)
  u64 least_sum = 0;                                       // of the weights that min_p keeps
  u64* const table = tables[tid / 128];
  Pair mine[2] = {};                                       // of bins 2 tid and the next
  float next[8];
  load8_raw<BF, VEC>(row, i0 + tid * 8, a.V, next);
  int turn = 1;
  for (int64_t at = i0; at < i1; at += kStep, turn ^= 1) {
    const int64_t i = at + tid * 8;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = next[j];
    load8_raw<BF, VEC>(row, i + kStep, a.V, next);         // of the next turn; past the chunk they are not used
    finish8<BF, VEC>(row, i, a.V, v);
    if (r.inf) {                                           // its equals as 0 below a largest of 0
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = v[j] == __builtin_inff() ? 0.f : kNegInf;
    }
    float d[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) d[j] = top - v[j];
    if (a.logprob) {
#pragma unroll
      for (int j = 0; j < 8; ++j) e += power(((double)v[j] - dtop) * 1.4426950408889634);
    }
    if (st.greedy) continue;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const u64 w = weight(((double)v[j] - dtop) * r.c);
      if (w) {
        const int bin = (int)__builtin_amdgcn_fmed3f(d[j] * per_bin, 0.f, (float)(kBins - 1));   // as in fine_of
        atomicAdd(&table[bin], w | (u64)1 << kCountAt);
      }
      if (st.min_w && w >= st.min_w) least_sum += w;
    }
    const bool last = at + kStep >= i1;
    if (turn && !last) continue;
    __syncthreads();
#pragma unroll
    for (int t = 0; t < kTables; ++t) {
      const ulonglong2 x = *(const ulonglong2*)(tables[t] + 2 * tid);
      mine[0] = mine[0] + Pair{x.x & (((u64)1 << kCountAt) - 1), x.x >> kCountAt};
      mine[1] = mine[1] + Pair{x.y & (((u64)1 << kCountAt) - 1), x.y >> kCountAt};
    }
    if (!last) {
      __syncthreads();
#pragma unroll
      for (int t = 0; t < kTables; ++t) *(ulonglong2*)(tables[t] + 2 * tid) = make_ulonglong2(0, 0);
      __syncthreads();
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
  put(a.w_bins + at * kBins + 2 * tid, mine[0].w);
  put(a.w_bins + at * kBins + 2 * tid + 1, mine[1].w);
  put((u64*)(a.n_bins + at * kBins) + tid, mine[0].n | mine[1].n << 32);
  if (!last_to_arrive(&a.plan[b].arrived, (uint32_t)a.chunks, &s_last)) return;
  // the row's bins, all chunks' sums asked for at once: running sums; and the plan
  u64 sum_m = get(a.kept + b * a.chunks + min<int64_t>(tid & 63, a.chunks - 1));
  Pair sum[2] = {};
  constexpr int kJoin = 8;                                 // of the chunks at a time
#pragma unroll 1
  for (int c0 = 0; c0 < a.chunks; c0 += kJoin) {
    u64 w[kJoin][2], n[kJoin];
#pragma unroll
    for (int c = 0; c < kJoin; ++c) {
      const int64_t from = (b * a.chunks + min<int64_t>(c0 + c, a.chunks - 1)) * kBins;
      w[c][0] = get(a.w_bins + from + 2 * tid);
      w[c][1] = get(a.w_bins + from + 2 * tid + 1);
      n[c] = get((const u64*)(a.n_bins + from) + tid);
    }
#pragma unroll
    for (int c = 0; c < kJoin; ++c) {
      if (c0 + c >= a.chunks) break;
      sum[0] = sum[0] + Pair{w[c][0], n[c] & 0xFFFFFFFFu};
      sum[1] = sum[1] + Pair{w[c][1], n[c] >> 32};
    }
  }
  sum_m = wave_all((tid & 63) < a.chunks ? sum_m : 0, (u64)0, Add());
  const Pair upto = scan(sum[0] + sum[1], waves), first = {upto.w - sum[1].w, upto.n - sum[1].n};
  bins[2 * tid] = first;
  bins[2 * tid + 1] = upto;
  ((ulonglong2*)a.sums)[b * kBins + 2 * tid] = make_ulonglong2(first.w, first.n);
  ((ulonglong2*)a.sums)[b * kBins + 2 * tid + 1] = make_ulonglong2(upto.w, upto.n);
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
  Pair bins[kBins], split[kParts];       // running sums by bin: of the row, of a part of it
  Pair waves[kWaves];
  Range range;                           // of the places in question
  uint32_t count, at, few_n;
  bool last;
};

struct Head {                            // of a plan
  int bin0[3], bin1[3];
  uint32_t ranges, upto;
};

// Appends to the list the logits of N eights per lane, from index i[k] on, that ok(x, index) says yes to: a lane's own one after
// another, behind those of the lanes before it.  The eights from `live` on hold none.
template <int N, class F>
__device__ __forceinline__ void append(Shared& s, const float v[N][8], const int i[N], int live, F&& ok) {
  uint32_t mine = 0;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    if (k >= live) break;
#pragma unroll
    for (int j = 0; j < 8; ++j) mine |= ok(v[k][j], i[k] + j) ? 1u << (8 * k + j) : 0u;
  }
  if (!__any(mine != 0)) return;
  const uint32_t n = __popc(mine), upto = wave_scan(n, 0u, Add()), all = lane_value(upto, 63);
  uint32_t at = 0;
  if ((threadIdx.x & 63) == 0) at = atomicAdd(&s.count, all);
  at = __builtin_amdgcn_readfirstlane(at) + upto - n;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    if (k >= live) break;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool is = mine >> (8 * k + j) & 1;
      if (is && at < kList) s.list[at] = place(v[k][j], i[k] + j);
      at += is;
    }
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
    n.lo[i] = (float)(plan.bin0[i] * kParts);
    // the largest number below the next bin; of no range: below its first
    n.hi[i] = last ? __builtin_inff() : __uint_as_float(__float_as_uint((float)((plan.bin1[i] + 1) * kParts)) - 1);
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
// in place of all blocks reading all logits.  That takes it 10 ns a group more, and saves the launch's blocks a second
// reading, of little cost while all of them are there at once.  131072 logits, calls with one block and with all: one
// row, 20 tokens 22.7 and 24.4 us, 100 26.7 and 27.7, 300 29.3 and 27.9; 16 rows, 100 31.2 and 32.3, 300 33.9 and 32.4; 64
// rows, 20 39.4 and 44.2, 300 47.9 and 48.6, 600 52.6 and 49.5.
__device__ __forceinline__ bool few_groups(const SampleArgs& a, const Head& plan) {
  const int64_t more = max(a.B * a.V - ((int64_t)1 << 21), (int64_t)0) >> 15;
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
    float next[kAhead][8];
    int at[kAhead];
    auto load = [&](int k0) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int g = k0 + k * kTeams + (tid >> 3);
        at[k] = g < n ? (int)groups[g] * 64 + (tid & 7) * 8 : (int)a.V;
        load8_raw<BF, VEC>(row, at[k], a.V, next[k]);
      }
    };
    load(0);
    for (int k0 = 0; k0 < n; k0 += kAhead * kTeams) {
      float v[kAhead][8];
      int i[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        i[k] = at[k];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[k][j] = next[k][j];
      }
      if (k0 + kAhead * kTeams < n) load(k0 + kAhead * kTeams);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) finish8<BF, VEC>(row, i[k], a.V, v[k]);
      // the one range; of a lone bin, whose bounds may be compared with no number, all that weighs anything
      append<kAhead>(s, v, i, (n - k0 + kTeams - 1) / kTeams, [&](float x, int) {
        const float y = ((float)r.top - x) * r.per_fine;
        return !(y < named.lo[0]) & !(y > named.hi[0]) & (x >= named.least);
      });
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
    for (int k = 0; k < 2; ++k) finish8<BF, VEC>(row, i + k * kStep, i1, v[k]);          // a chunk is a multiple of eight, but for the row's end
    const int is[2] = {(int)i, (int)i + kStep};
    append<2>(s, v, is, at + kStep < i1 ? 2 : 1, [&](float x, int) { return is_named(r, named, x); });
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
  const int k = first_bin<kParts>(q, s.split, *before);
  const Pair skip = k ? s.split[k - 1] : Pair{0, 0};
  *n = s.split[k].n - skip.n;
  *before = *before + skip;
  return k;
}

// The plan's tokens, a few to a thread: their places.  What follows from them is computed again where it is asked for: kept,
// it is more registers than leave room for two blocks on a CU (64 rows of wide settings 66 us, 54 with two).
constexpr int kEach = kList / kThreads;
struct Mine {
  u64 p[kEach];
  int n;                                 // of all threads
  __device__ float logit(int i) const {
    uint32_t key = (uint32_t)(p[i] >> 32);
    asm volatile("" : "+v"(key));                            // what follows stays where it is, and out of registers
    return from_falling(key);
  }
  __device__ int fine(const Row& r, int i) const {           // bin; -1: no token
    return i * kThreads + (int)threadIdx.x < n ? fine_of(r, logit(i)) : -1;
  }
};

// The answer from the plan's tokens: those of the bin, by its fine bins if they are many, and where many share a fine bin
// (equal logits) by place, until a wave can sort them.
__device__ __forceinline__ Found answer_mine(const Row& r, const Asked& q, const Mine& t, int bin, Pair before, u64 n, Shared& s) {
  const int tid = threadIdx.x;
  int part = -1;                         // of the bin; -1: all of it
  Range g = {0, ~0ull};
  auto clear = [&] {
    __syncthreads();
    s.split[tid] = {0, 0};
    if (tid == 0) {
      s.few_n = 0;
      s.range = {~0ull, 0};
    }
    __syncthreads();
  };
  auto add = [&](int i, int to) {
    atomicAdd(&s.split[to].w, weight_of(r, t.logit(i)));
    atomicAdd(&s.split[to].n, 1ull);
  };
  auto in = [&](int i) {
    const int fine = t.fine(r, i);
    return fine >= 0 && (part < 0 ? fine / kParts == bin : fine == bin * kParts + part) && t.p[i] >= g.lo && t.p[i] <= g.hi;
  };
  clear();
  if (n > kSmall) {
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (in(i)) add(i, t.fine(r, i) % kParts);
    part = split_choose(q, s, &before, &n);
  }
  if (n > kSmall) {
    u64 lo = ~0ull, hi = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const bool is = in(i);
      lo = is ? min(lo, t.p[i]) : lo;
      hi = is ? max(hi, t.p[i]) : hi;
    }
    lo = wave_all(lo, (u64)~0ull, Least());
    hi = ~wave_all(~hi, (u64)~0ull, Least());
    if ((tid & 63) == 0) {
      atomicMin(&s.range.lo, lo);
      atomicMax(&s.range.hi, hi);
    }
    __syncthreads();
    g = s.range;
#pragma unroll 1
    while (n > kSmall) {
      const int shift = max(64 - __clzll((long long)(g.hi - g.lo)) - 9, 0);
      static_assert(kParts == 512, "nine bits");
      clear();
#pragma unroll
      for (int i = 0; i < kEach; ++i)
        if (in(i)) add(i, (int)((t.p[i] - g.lo) >> shift));
      const int k = split_choose(q, s, &before, &n);
      g.lo += (u64)k << shift;
      g.hi = min(g.hi, g.lo + (((u64)1 << shift) - 1));
    }
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    if (in(i)) s.few[atomicAdd(&s.few_n, 1u)] = t.p[i];
  __syncthreads();
  return among_few(q, sort_few(r, s.few, (int)n), before);
}

// The answer from the row itself, read by this block: its bin by places, nine bits at a time, down to a single token
// if need be; from LDS once its tokens fit.
template <bool BF, bool VEC>
__device__ __forceinline__ Found answer_row(const SampleArgs& a, int64_t b, const Row& r, const Asked& q, int bin,
                                            Pair before, u64 n, Shared& s) {
  const int tid = threadIdx.x;
  Range g = places_of(r, bin);
  auto in = [&](u64 p) { return p >= g.lo && p <= g.hi; };
  auto gather = [&] {
    __syncthreads();
    if (tid == 0) s.count = 0;
    __syncthreads();
    const void* row = row_of<BF>(a, b);
#pragma unroll 1
    for (int64_t at = 0; at < a.V; at += kStep) {
      const int i[1] = {(int)at + tid * 8};
      float v[1][8];
      load8_raw<BF, VEC>(row, i[0], a.V, v[0]);
      finish8<BF, VEC>(row, i[0], a.V, v[0]);
      append<1>(s, v, i, 1, [&](float x, int at) { return in(place(x, at)); });
    }
    __syncthreads();
  };
  bool listed = false;
  while (n > kSmall) {
    if (!listed && n <= kList) {
      gather();
      listed = true;
    }
    const int bits = 64 - __clzll((long long)(g.hi - g.lo)), shift = max(bits - 9, 0);
    static_assert(kParts == 512, "nine bits");
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
__global__ __launch_bounds__(kThreads, 4) void sample_draw_kernel(SampleArgs a) {
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
  const ulonglong2* sums = (const ulonglong2*)a.sums + b * kBins;
  const ulonglong2 mine0 = sums[tid], mine1 = sums[kThreads + tid];
  u64 best;
  const Row r = row_of_extremes(ex, st, &best);
  const bool masked = r.top == -__builtin_inf();
  int64_t token = masked ? -1 : (int64_t)(uint32_t)best;
  const bool draws = !st.greedy && !masked;
  const bool alone = !draws || plan.ranges == 0 || few_groups(a, plan);   // one block does it all
  if (alone && part > 0) return;
  exps = wave_all((tid & 63) < a.chunks ? exps : 0.0, 0.0, Add());
  sum_m = wave_all((tid & 63) < a.chunks ? sum_m : 0, (u64)0, Add());
  if (draws) {
    if (tid == 0) s.count = 0;
    s.bins[tid] = {mine0.x, mine0.y};
    s.bins[kThreads + tid] = {mine1.x, mine1.y};
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
    t.n = (int)tokens;
    const bool small = plan.ranges == 1 && tokens <= kSmall;     // one order answers all questions
    Few few = {0, 0, 0};
    if (small) {
      if (tid < (int)tokens) s.few[tid] = t.p[0];
      __syncthreads();
      few = sort_few(r, s.few, (int)tokens);
    }
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
      const int bin = small ? plan.bin0[0] : first_bin<kBins>(q, s.bins, {0, 0});
      const Pair before = bin ? s.bins[bin - 1] : Pair{0, 0};
      const u64 n = s.bins[bin].n - before.n;
      Found f;
      const bool held = plan.ranges > 0;
      if (small) {
        f = among_few(q, few, before);
      } else {
        bool named = false;
#pragma unroll
        for (int i = 0; i < 3; ++i) named |= plan.bin0[i] <= bin && bin <= plan.bin1[i];
        if (held && named) f = answer_mine(r, q, t, bin, before, n, s);
        else f = answer_row<BF, VEC>(a, b, r, q, bin, before, n, s);
      }
      sum = min(sum, f.sum);
      token = f.token;
    }
    token = min(token, a.V - 1);         // within the row whatever a workspace that two calls write at once may hold
  }
  if (tid >= 64) return;
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
