// Pages and slots of a step, from request lengths that are on the device.
//
// With have = ceil(cached / page), need = ceil((cached + fresh) / page) and extra = need - have:
// ended requests push their pages on the stack of free pages, the others take their extra pages from
// its top in the order of requests, and each new token gets its request, position and slot.  All of it
// is prefix sums over the requests: one block of 1024 threads takes 1024 requests at a time, so that a
// step of a serving batch is one launch.  What the prefix sums assign (pages to table entries, tokens to
// rows) is spread evenly over the threads, each of which finds its request by bisection in LDS: a
// request with many pages or tokens costs no more than many with one.
//
// Bound by latency: a chain of loads, scans and dependent stores, 8.3 us for 64 requests.  Above kRowsHere token rows a
// second launch writes them, four to a thread (65536 rows of 500 requests, 64 blocks: 8.3 us).
#include "device_common.hpp"
#include "step_ops.hpp"
#include "wave_ops.hpp"

namespace bl {

namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
// Rows that the one block writes itself.  64 requests, with and without a second launch: 64 rows 7.6 and 6.2 us, 4096
// 12.1 and 8.7, 8192 12.3 and 11.4, 16384 12.3 and 17.1; 512 requests and 65536 rows 15.6 and 52.
constexpr int kRowsHere = 8192;
constexpr int kStartsLds = 8192;     // request starts that a block of the second launch holds

struct Pair {
  int64_t a, b;
};

// Inclusive prefix sums of v over the block; *total: over all threads.  Starts and ends with every
// thread past its use of `waves`.
__device__ __forceinline__ Pair block_scan(Pair v, Pair* waves, Pair* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  auto add = [](int64_t x, int64_t y) { return x + y; };
  v = {wave_scan(v.a, (int64_t)0, add), wave_scan(v.b, (int64_t)0, add)};
  if (lane == 63) waves[wave] = v;
  __syncthreads();
  Pair all = {0, 0};
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const Pair p = waves[w];
    if (w == wave) { v.a += all.a; v.b += all.b; }
    all.a += p.a; all.b += p.b;
  }
  *total = all;
  __syncthreads();
  return v;
}

// Largest i with first[i] <= j, of kThreads rising values with first[0] = 0.
__device__ __forceinline__ int owner(const uint32_t* first, uint32_t j) {
  int i = 0;
#pragma unroll
  for (int step = kThreads / 2; step > 0; step >>= 1)
    if (first[i + step] <= j) i += step;
  return i;
}

__device__ __forceinline__ uint32_t ceil_div(uint32_t x, uint32_t d) { return x / d + (x % d != 0); }

__device__ __forceinline__ void put_row(const KvStepArgs& a, int64_t t, int64_t b, uint32_t p) {
  a.seq[t] = (int32_t)b;
  a.pos[t] = (int32_t)p;
  if (a.slot) {
    const uint32_t i = p / a.page;
    a.slot[t] = (int64_t)a.blocks[b * a.per + i] * a.page + (p - i * a.page);
  }
}
__device__ __forceinline__ void pad_row(const KvStepArgs& a, int64_t t) {
  a.seq[t] = -1;
  a.pos[t] = -1;
  if (a.slot) a.slot[t] = -1;
}

__global__ __launch_bounds__(kThreads) void kv_step_kernel(KvStepArgs a, int rows) {
  __shared__ Pair waves[kWaves];
  __shared__ uint32_t page0[kThreads], tok0[kThreads], old_pages[kThreads], old_len[kThreads];
  const int tid = threadIdx.x;
  int64_t count = min(max((int64_t)*a.count, (int64_t)0), a.cap);
  Pair total;

  // ended requests give their pages back
  int64_t back = 0;
  for (int64_t b0 = 0; b0 < a.B; b0 += kThreads) {
    const int64_t b = b0 + tid;
    const bool ended = b < a.B && a.fresh[b] < 0;
    if (!__syncthreads_or(ended)) continue;
    const int64_t n = ended ? min((int64_t)ceil_div((uint32_t)max(a.cached[b], 0), a.page), a.per) : 0;
    const Pair in = block_scan({n, 0}, waves, &total);
    const int64_t base = count + back;
    // pages past the stack's end are dropped
    page0[tid] = (uint32_t)min(in.a - n, a.cap);
    __syncthreads();
    const int64_t fit = min(total.a, a.cap - base);
    for (int64_t j = tid; j < fit; j += kThreads) {
      const int i = owner(page0, (uint32_t)j);
      a.free_pages[base + j] = a.blocks[(b0 + i) * a.per + (j - page0[i])];
    }
    back += max(fit, (int64_t)0);
    __syncthreads();
  }
  count += back;

  Pair want_sum = {0, 0}, got_sum = {0, 0};      // of the requests before this chunk
  for (int64_t b0 = 0; b0 < a.B; b0 += kThreads) {
    const int64_t b = b0 + tid;
    const bool in_batch = b < a.B;
    const uint32_t len = in_batch ? (uint32_t)max(a.cached[b], 0) : 0u;
    const int32_t fresh = in_batch ? a.fresh[b] : 0;
    const uint32_t want = (uint32_t)max(fresh, 0);
    const uint32_t have = ceil_div(len, a.page), need = ceil_div(len + want, a.page);
    const uint32_t extra = need - have;
    Pair in = block_scan({(int64_t)extra, (int64_t)want}, waves, &total);
    in.a += want_sum.a;
    in.b += want_sum.b;
    want_sum.a += total.a;
    want_sum.b += total.b;
    const bool served = in_batch && fresh >= 0 && need <= a.per && (extra == 0 || in.a <= count) &&
                        in.b <= a.T && len + want <= 0x7FFFFFFFu;
    const Pair mine = {served ? (int64_t)extra : 0, served ? (int64_t)want : 0};
    in = block_scan(mine, waves, &total);
    page0[tid] = (uint32_t)(in.a - mine.a);
    tok0[tid] = (uint32_t)(in.b - mine.b);
    old_pages[tid] = have;
    old_len[tid] = len;
    if (in_batch) {
      a.lens[b] = fresh < 0 ? 0 : (int32_t)(len + (uint32_t)mine.b);
      a.starts[b] = (int32_t)(got_sum.b + in.b - mine.b);
    }
    __syncthreads();
    for (int64_t j = tid; j < total.a; j += kThreads) {
      const int i = owner(page0, (uint32_t)j);
      a.blocks[(b0 + i) * a.per + old_pages[i] + (j - page0[i])] =
          a.free_pages[count - 1 - got_sum.a - j];
    }
    __syncthreads();                             // the table's entries, before rows read them
    if (rows) {
      for (int64_t j = tid; j < total.b; j += kThreads) {
        const int i = owner(tok0, (uint32_t)j);
        put_row(a, got_sum.b + j, b0 + i, old_len[i] + (uint32_t)j - tok0[i]);
      }
    }
    got_sum.a += total.a;
    got_sum.b += total.b;
    __syncthreads();
  }
  if (tid == 0) {
    a.starts[a.B] = (int32_t)got_sum.b;
    *a.count_out = (int32_t)(count - got_sum.a);
  }
  if (rows)
    for (int64_t t = got_sum.b + tid; t < a.T; t += kThreads) pad_row(a, t);
}

// The rows alone, from the starts, lengths and table of the launch before.
__global__ __launch_bounds__(256) void kv_rows_kernel(KvStepArgs a) {
  __shared__ int32_t held[kStartsLds];
  const bool lds = a.B + 1 <= kStartsLds;
  if (lds) {
    for (int i = threadIdx.x; i <= a.B; i += 256) held[i] = a.starts[i];
    __syncthreads();
  }
  const int32_t* starts = lds ? held : a.starts;
  const int32_t all = starts[a.B];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int64_t t = ((int64_t)blockIdx.x * 4 + r) * 256 + threadIdx.x;
    if (t >= a.T) return;
    if (t >= all) {
      pad_row(a, t);
      continue;
    }
    int64_t lo = 0, hi = a.B;                    // starts[lo] <= t < starts[hi]
    while (hi - lo > 1) {
      const int64_t m = (lo + hi) >> 1;
      if (starts[m] <= t) lo = m;
      else hi = m;
    }
    put_row(a, t, lo, (uint32_t)(a.lens[lo] - starts[lo + 1] + (int32_t)t));
  }
}

}  // namespace

hipError_t launch_kv_step(const KvStepArgs& a, hipStream_t s) {
  const bool here = a.T <= kRowsHere;
  kv_step_kernel<<<1, kThreads, 0, s>>>(a, here);
  const hipError_t e = hipGetLastError();
  if (here || e != hipSuccess) return e;
  kv_rows_kernel<<<(unsigned)((a.T + 1023) / 1024), 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace bl
