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
//   pick   one block per row adds the chunks' bins up and answers the questions: the tokens of the bins it needs
//          are gathered into LDS, sorted and summed.  Where the bins up to the last one in question hold at most
//          kList tokens (top-k and top-p as they are used), they are gathered once.  A bin of more than kList
//          tokens is split by further passes over the row, down to tokens of one value if need be, which
//          are told apart by counting.
// Weights take an exp in fp64; 2^-41 of the largest and less are zero and leave early.
#include <algorithm>

#include "block_ops.hpp"
#include "device_common.hpp"
#include "step_ops.hpp"

namespace bl {

namespace {

typedef unsigned long long u64;

constexpr int kBins = kSampleBins;
constexpr int kList = 4096;              // tokens that a row's block sorts
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

// Elements i .. i + 8 of a row; NaN and what is past the end count as -inf.
template <bool BF, bool VEC>
__device__ __forceinline__ void load8(const void* row, int64_t i, int64_t V, float v[8]) {
  if (VEC && i + 8 <= V) {
    load_f8<BF>(row, i, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = kNegInf;
      if (i + j < V)
        v[j] = BF ? __uint_as_float((uint32_t)((const uint16_t*)row)[i + j] << 16) : ((const float*)row)[i + j];
    }
  }
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

// The chunks' largest logits (as falling() and index) and least finite ones, joined by a wave.
__device__ __forceinline__ Row row_stats(const SampleArgs& a, int64_t b, const Settings& s, u64* best) {
  const int lane = threadIdx.x & 63;
  u64 top = ~0ull;
  float least = __builtin_inff();
  for (int c = lane; c < a.chunks; c += 64) {
    top = min(top, a.top[b * a.chunks + c]);
    least = fminf(least, a.least[b * a.chunks + c]);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    top = min(top, (u64)__shfl_xor((long long)top, o, 64));
    least = fminf(least, __shfl_xor(least, o, 64));
  }
  const float x = from_falling((uint32_t)(top >> 32));
  *best = top;
  Row r;
  r.top = x;
  r.inf = x == __builtin_inff();
  r.c = 1.4426950408889634 / s.temp;
  double range = r.inf ? 0.0 : fmin(((double)x - least) * r.c, 41.0);
  r.per_bin = range > 0.0 ? kBins / range : 0.0;
  if (!(r.per_bin < 1e30)) r.per_bin = 0.0;                // too narrow to be told apart: one bin
  return r;
}

template <bool BF, bool VEC>
__global__ __launch_bounds__(256) void sample_max_kernel(SampleArgs a) {
  __shared__ u64 s_top[4];
  __shared__ float s_least[4];
  const int64_t b = blockIdx.y;
  const void* row = row_of<BF>(a, b);
  const int64_t i0 = (int64_t)blockIdx.x * a.chunk, i1 = min(i0 + a.chunk, a.V);
  u64 top = ~0ull;
  float least = __builtin_inff();
  for (int64_t i = i0 + threadIdx.x * 8; i < i1; i += 4 * 2048) {
    float v[4][8];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i + u * 2048 < i1) load8<BF, VEC>(row, i + u * 2048, a.V, v[u]);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (i + u * 2048 >= i1) break;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        top = min(top, ((u64)falling(v[u][j]) << 32) | (uint32_t)(i + u * 2048 + j));
        least = fminf(least, v[u][j] == kNegInf ? __builtin_inff() : v[u][j]);
      }
    }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    top = min(top, (u64)__shfl_xor((long long)top, o, 64));
    least = fminf(least, __shfl_xor(least, o, 64));
  }
  if ((threadIdx.x & 63) == 0) {
    s_top[threadIdx.x >> 6] = top;
    s_least[threadIdx.x >> 6] = least;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    a.top[b * a.chunks + blockIdx.x] = min(min(s_top[0], s_top[1]), min(s_top[2], s_top[3]));
    a.least[b * a.chunks + blockIdx.x] = fminf(fminf(s_least[0], s_least[1]), fminf(s_least[2], s_least[3]));
  }
}

template <bool BF, bool VEC>
__global__ __launch_bounds__(256) void sample_hist_kernel(SampleArgs a) {
  __shared__ u64 w_bin[kBins];
  __shared__ uint32_t n_bin[kBins];
  __shared__ double s_exp[4];
  __shared__ u64 s_min[4];
  const int tid = threadIdx.x;
  const int64_t b = blockIdx.y;
  const Settings st = settings_of(a, b);
  u64 best;
  const Row r = row_stats(a, b, st, &best);
  if (st.greedy && !a.logprob) return;
  if (r.top == -__builtin_inf()) return;                   // nothing to draw from
  for (int i = tid; i < kBins; i += 256) {
    w_bin[i] = 0;
    n_bin[i] = 0;
  }
  __syncthreads();
  const void* row = row_of<BF>(a, b);
  const int64_t i0 = (int64_t)blockIdx.x * a.chunk, i1 = min(i0 + a.chunk, a.V);
  const double min_w = st.min_p * kOne;
  const float top = (float)r.top;
  double e = 0.0;                                          // sum of exp(x - top)
  u64 least_sum = 0;                                       // of the weights that min_p keeps
  for (int64_t i = i0 + tid * 8; i < i1; i += 2 * 2048) {
    float v[2][8];
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (i + u * 2048 < i1) load8<BF, VEC>(row, i + u * 2048, a.V, v[u]);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (i + u * 2048 >= i1) break;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = v[u][j];
        if (a.logprob) e += r.inf ? (x == top ? 1.0 : 0.0) : (double)__builtin_amdgcn_exp2f((x - top) * 1.44269504f);
        if (st.greedy) continue;
        const double t = scaled(r, x);
        const u64 w = weight(t);
        if (w) {
          const int k = bin_of(r, t);
          atomicAdd(&w_bin[k], w);
          atomicAdd(&n_bin[k], 1u);
          if ((double)w >= min_w) least_sum += w;
        }
      }
    }
  }
  e = wave_sum_f64(e);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) least_sum += (u64)__shfl_xor((long long)least_sum, o, 64);
  if ((tid & 63) == 0) {
    s_exp[tid >> 6] = e;
    s_min[tid >> 6] = least_sum;
  }
  __syncthreads();
  const int64_t at = b * a.chunks + blockIdx.x;
  if (tid == 0) {
    a.exps[at] = (s_exp[0] + s_exp[1]) + (s_exp[2] + s_exp[3]);
    a.kept[at] = s_min[0] + s_min[1] + s_min[2] + s_min[3];
  }
  if (st.greedy) return;
  for (int i = tid; i < kBins; i += 256) {
    a.w_bins[at * kBins + i] = w_bin[i];
    a.n_bins[at * kBins + i] = n_bin[i];
  }
}

// ---------------------------------------------------------------------------------------------
// pick
// ---------------------------------------------------------------------------------------------

constexpr int kPick = 1024;              // threads

struct Found {                           // the answer to a question about the order
  u64 sum;                               // of the weights up to and with the token found
  int64_t token;
};

struct Pick {                            // a block's shared memory
  u64 list[kList];                       // falling() and index of gathered tokens, sorted
  u64 w[kBins], w2[kBins];               // running sums of weights by bin: of the row, of a bin's split
  uint32_t n[kBins], n2[kBins];          // and of counts
  u64 waves[kPick / 64];
  uint32_t count;
  Found found;
};

enum Question { kCount, kGoal, kPass };  // the k-th token; first sum >= goal (as doubles); first sum > r

struct Asked {
  Question q;
  int64_t k;
  double goal;
  u64 r;
};
// Whether tokens up to one with these running sums answer the question.
__device__ __forceinline__ bool met(const Asked& a, uint64_t n, u64 w) {
  return a.q == kCount ? (int64_t)n >= a.k : a.q == kGoal ? (double)w >= a.goal : w > a.r;
}

// Inclusive sums over the block.
__device__ __forceinline__ u64 scan(u64 v, Pick& s) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const u64 x = (u64)__shfl_up((long long)v, o, 64);
    if (lane >= o) v += x;
  }
  if (lane == 63) s.waves[wave] = v;
  __syncthreads();
  u64 before = 0;
#pragma unroll
  for (int w = 0; w < kPick / 64; ++w) before += w < wave ? s.waves[w] : 0;
  __syncthreads();
  return v + before;
}

// Running sums of kBins counts and weights, in place.
__device__ __forceinline__ void scan_bins(u64* w, uint32_t* n, Pick& s) {
  const int tid = threadIdx.x;
  const u64 x = scan(tid < kBins ? w[tid] : 0, s);
  const u64 y = scan(tid < kBins ? n[tid] : 0, s);
  if (tid < kBins) {
    w[tid] = x;
    n[tid] = (uint32_t)y;
  }
  __syncthreads();
}

// First bin whose running sums answer the question (the last one that adds anything, if none does).
__device__ __forceinline__ int first_bin(const Asked& a, const u64* w, const uint32_t* n, uint64_t n0, u64 w0) {
  int lo = 0, hi = kBins - 1;
  while (lo < hi) {
    const int m = (lo + hi) >> 1;
    if (met(a, n0 + n[m], w0 + w[m]) || n[m] == n[kBins - 1]) hi = m;
    else lo = m + 1;
  }
  return lo;
}

struct Range {                           // bins and falling() values, both ends included
  int bin0, bin1;
  uint32_t key0, key1;
};

// Calls f(x, i, t) for the row's tokens in a range that weigh something.
template <bool BF, bool VEC, class F>
__device__ __forceinline__ void each(const SampleArgs& a, int64_t b, const Row& r, const Range& g, F&& f) {
  const void* row = row_of<BF>(a, b);
  // bounds on x a little wider than the bins, to be tested by one comparison each
  float lo = from_falling(g.key1), hi = from_falling(g.key0);
  if (!(lo == lo)) lo = kNegInf;         // ends past the infinities are no numbers
  if (!(hi == hi)) hi = __builtin_inff();
  if (!r.inf && r.per_bin > 0.0) {
    const double unit = 1.0 / (r.per_bin * r.c);
    auto edge = [&](double bin, double way) {
      const double x = r.top - bin * unit;
      return (float)(x + way * 1e-6 * (fabs(x) + fabs(r.top) + 1e-30));
    };
    if (g.bin1 < kBins - 1) lo = fmaxf(lo, edge(g.bin1 + 1, -1.0));
    if (g.bin0 > 0) hi = fminf(hi, edge(g.bin0, 1.0));
  }
  for (int64_t i = threadIdx.x * 8; i < a.V; i += 4 * 8 * kPick) {
    float v[4][8];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i + u * 8 * kPick < a.V) load8<BF, VEC>(row, i + u * 8 * kPick, a.V, v[u]);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t at = i + u * 8 * kPick;
      if (at >= a.V) break;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = v[u][j];
        if (!(x >= lo && x <= hi)) continue;
        const uint32_t key = falling(x);
        if (key < g.key0 || key > g.key1) continue;
        const double t = scaled(r, x);
        if (!(t > -41.0) || weight(t) == 0) continue;
        const int bin = bin_of(r, t);
        if (bin >= g.bin0 && bin <= g.bin1) f(x, at + j, t);
      }
    }
  }
}

// The list, in order; n <= kList tokens.
template <bool BF, bool VEC>
__device__ __forceinline__ void gather(const SampleArgs& a, int64_t b, const Row& r, const Range& g, Pick& s) {
  const int tid = threadIdx.x;
  __syncthreads();
  if (tid == 0) s.count = 0;
  __syncthreads();
  each<BF, VEC>(a, b, r, g, [&](float x, int64_t i, double) {
    const uint32_t at = atomicAdd(&s.count, 1u);
    if (at < kList) s.list[at] = ((u64)falling(x) << 32) | (uint32_t)i;
  });
  __syncthreads();
  int size = 64;
  while (size < (int)s.count) size <<= 1;
  for (int i = s.count + tid; i < size; i += kPick) s.list[i] = ~0ull;
  __syncthreads();
  for (int n = 2; n <= size; n <<= 1) {
    for (int d = n >> 1; d > 0; d >>= 1) {
      for (int i = tid; i < size / 2; i += kPick) {
        const int lo = ((i & ~(d - 1)) << 1) | (i & (d - 1)), hi = lo | d;
        const u64 x = s.list[lo], y = s.list[hi];
        if ((x > y) == ((lo & n) == 0)) {
          s.list[lo] = y;
          s.list[hi] = x;
        }
      }
      __syncthreads();
    }
  }
}

// The answer within the sorted list, n0 and w0 of which come before it; the last token if none answers.
__device__ __forceinline__ Found locate(const Row& r, const Asked& q, uint64_t n0, u64 w0, Pick& s) {
  const int tid = threadIdx.x, n = s.count;
  constexpr int E = kList / kPick;
  u64 w[E], sum = 0;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int i = tid * E + e;
    w[e] = i < n ? weight(scaled(r, from_falling((uint32_t)(s.list[i] >> 32)))) : 0;
    sum += w[e];
  }
  u64 at = scan(sum, s) - sum + w0;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int i = tid * E + e;
    const bool before = i > 0 && met(q, n0 + i, at);
    at += w[e];
    if (i < n && !before && (met(q, n0 + i + 1, at) || i == n - 1)) s.found = {at, (int64_t)(uint32_t)s.list[i]};
  }
  __syncthreads();
  const Found f = s.found;
  __syncthreads();
  return f;
}

// Tokens of one value, whose order is that of their indices: n of them, each of weight w.
template <bool BF, bool VEC>
__device__ __forceinline__ Found among_equals(const SampleArgs& a, int64_t b, const Row& r, uint32_t key,
                                              const Asked& q, uint64_t n, uint64_t n0, u64 w0, Pick& s) {
  const u64 w = weight(scaled(r, from_falling(key)));
  uint64_t lo = 1, hi = n;               // how many of them it takes
  while (lo < hi) {
    const uint64_t m = (lo + hi) >> 1;
    if (met(q, n0 + m, w0 + m * w)) hi = m;
    else lo = m + 1;
  }
  if (q.q == kPass) {                    // which token that is
    const void* row = row_of<BF>(a, b);
    uint64_t seen = 0;
    for (int64_t i0 = 0; i0 < a.V && seen < lo; i0 += 8 * kPick) {
      const int64_t i = i0 + threadIdx.x * 8;
      float v[8];
      load8<BF, VEC>(row, i, a.V, v);
      uint32_t mine = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) mine |= (uint32_t)(i + j < a.V && falling(v[j]) == key) << j;
      const uint64_t upto = seen + scan((u64)__popc(mine), s), before = upto - __popc(mine);
      if (before < lo && lo <= upto) {
        for (uint64_t skip = lo - 1 - before; skip; --skip) mine &= mine - 1;
        s.found.token = i + __ffs(mine) - 1;
      }
      if (threadIdx.x == kPick - 1) s.waves[0] = upto;
      __syncthreads();
      seen = s.waves[0];
      __syncthreads();
    }
  }
  return {w0 + lo * w, s.found.token};
}

// The answer wherever it lies; `held` says which bins the list has.
template <bool BF, bool VEC>
__device__ __forceinline__ Found answer(const SampleArgs& a, int64_t b, const Row& r, const Asked& q, Range* held, Pick& s) {
  int bin = first_bin(q, s.w, s.n, 0, 0);
  if (held->bin0 <= bin && bin <= held->bin1) {
    bin = held->bin0;
    return locate(r, q, bin ? s.n[bin - 1] : 0, bin ? s.w[bin - 1] : 0, s);
  }
  Range g = {bin, bin, 0, 0xFFFFFFFFu};
  uint64_t n0 = bin ? s.n[bin - 1] : 0, n = s.n[bin] - n0;
  u64 w0 = bin ? s.w[bin - 1] : 0;
  while (n > kList && g.key0 < g.key1) {                   // split the range into kBins
    int shift = 0;
    while ((g.key1 - g.key0) >> shift >= kBins) ++shift;
    for (int i = threadIdx.x; i < kBins; i += kPick) {
      s.w2[i] = 0;
      s.n2[i] = 0;
    }
    __syncthreads();
    each<BF, VEC>(a, b, r, g, [&](float x, int64_t, double t) {
      const uint32_t k = (falling(x) - g.key0) >> shift;
      atomicAdd(&s.w2[k], weight(t));
      atomicAdd(&s.n2[k], 1u);
    });
    __syncthreads();
    scan_bins(s.w2, s.n2, s);
    const int k = first_bin(q, s.w2, s.n2, n0, w0);
    n = s.n2[k] - (k ? s.n2[k - 1] : 0);
    n0 += k ? s.n2[k - 1] : 0;
    w0 += k ? s.w2[k - 1] : 0;
    g.key0 += (uint32_t)k << shift;
    g.key1 = min(g.key1, g.key0 + ((1u << shift) - 1));
    __syncthreads();
  }
  held->bin0 = 0;
  held->bin1 = -1;                       // the list has no whole bins, or will not
  if (n > kList) return among_equals<BF, VEC>(a, b, r, g.key0, q, n, n0, w0, s);
  gather<BF, VEC>(a, b, r, g, s);
  if (g.key0 == 0 && g.key1 == 0xFFFFFFFFu) *held = g;
  return locate(r, q, n0, w0, s);
}

template <bool BF, bool VEC>
__global__ __launch_bounds__(kPick) void sample_pick_kernel(SampleArgs a) {
  __shared__ Pick s;
  __shared__ double s_exp;
  const int tid = threadIdx.x;
  const int64_t b = blockIdx.x;
  const Settings st = settings_of(a, b);
  u64 best;
  const Row r = row_stats(a, b, st, &best);
  if (r.top == -__builtin_inf()) {
    if (tid == 0) {
      a.token[b] = -1;
      if (a.logprob) a.logprob[b] = kNegInf;
    }
    return;
  }
  if (a.logprob && tid == 0) {
    double e = 0.0;
    for (int c = 0; c < a.chunks; ++c) e += a.exps[b * a.chunks + c];
    s_exp = e;
  }
  int64_t token = (uint32_t)best;
  if (!st.greedy) {
    if (tid < kBins) {
      u64 w = 0;
      uint32_t n = 0;
      for (int c = 0; c < a.chunks; ++c) {
        const int64_t at = (b * a.chunks + c) * kBins + tid;
        w += a.w_bins[at];
        n += a.n_bins[at];
      }
      s.w[tid] = w;
      s.n[tid] = n;
    }
    u64 sum_m = 0;
    for (int c = 0; c < a.chunks; ++c) sum_m += a.kept[b * a.chunks + c];
    __syncthreads();
    scan_bins(s.w, s.n, s);
    const u64 all = s.w[kBins - 1];
    const int64_t k = st.k && st.k < s.n[kBins - 1] ? st.k : 0;
    Range held = {0, -1, 0, 0xFFFFFFFFu};
    // everything up to the last bin in question at once, if it is not too much
    Asked q = {kCount, k, 0.0, 0};
    if (k || st.p < 1.0) {
      if (!k) q = {kGoal, 0, st.p * (double)all, 0};
      const int cut = first_bin(q, s.w, s.n, 0, 0);
      if (s.n[cut] <= kList) {
        held.bin1 = cut;
        gather<BF, VEC>(a, b, r, held, s);
      }
    }
    u64 sum = all;
    if (k) sum = answer<BF, VEC>(a, b, r, {kCount, k, 0.0, 0}, &held, s).sum;
    if (st.p < 1.0) {
      const u64 sum_p = answer<BF, VEC>(a, b, r, {kGoal, 0, st.p * (double)sum, 0}, &held, s).sum;
      sum = min(sum, sum_p);
    }
    if (st.min_p > 0.0) sum = min(sum, max(sum_m, (u64)kOne));
    const double u = a.u[b];
    const double at = u > 0.0 ? fmin(u, 1.0) * (double)sum : 0.0;     // NaN: 0
    const u64 pass = min((u64)at, sum - 1);
    token = answer<BF, VEC>(a, b, r, {kPass, 0, 0.0, pass}, &held, s).token;
  }
  __syncthreads();
  if (tid == 0) {
    a.token[b] = (int32_t)token;
    if (a.logprob) {
      float x;
      const void* row = row_of<BF>(a, b);
      if constexpr (BF) x = __uint_as_float((uint32_t)((const uint16_t*)row)[token] << 16);
      else x = ((const float*)row)[token];
      a.logprob[b] = (float)((r.inf ? 0.0 : (double)x - r.top) - log(s_exp));
    }
  }
}

template <bool BF, bool VEC>
hipError_t run(const SampleArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)a.chunks, (unsigned)a.B);
  sample_max_kernel<BF, VEC><<<grid, 256, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  sample_hist_kernel<BF, VEC><<<grid, 256, 0, s>>>(a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  sample_pick_kernel<BF, VEC><<<(unsigned)a.B, kPick, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_sample(const SampleArgs& a, bool bf16, bool vec, hipStream_t s) {
  if (bf16) return vec ? run<true, true>(a, s) : run<true, false>(a, s);
  return vec ? run<false, true>(a, s) : run<false, false>(a, s);
}

}  // namespace bl
