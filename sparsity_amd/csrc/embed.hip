// Embedding rows by token id, and the gradient of the table.
//
//   y[t] = round(scale * table[ids[t]])
//   dtable[v] (+)= scale * sum over the tokens t with ids[t] = v of dy[t]
//
// Forward: a wave takes up to 2048 columns of one token, all of its loads before the first store.
//
// Gradient: tokens are sorted by id, so that a row's tokens are a run of sorted positions, and each run
// is summed in the order of its tokens: results do not vary from run to run, and nothing is added by
// atomics.  Launches:
//   sort   blocks sort a chunk of tokens each in LDS; where the gradient is overwritten, the other blocks
//          of the launch clear it meanwhile (most of the bytes of a large table)
//   rank   (several chunks) an element's place is its place in its chunk plus, by bisection, what the
//          other chunks hold before it
//   sum    a wave takes 16 sorted positions and 512 columns; it sums every run that starts there, up to
//          32 positions of it, and writes the row; of a longer run, what lies inside its 16 goes to the
//          workspace
//   join   the pieces of long runs, in order
#include <algorithm>

#include "block_ops.hpp"
#include "device_common.hpp"
#include "step_ops.hpp"

namespace bl {

namespace {

// ---------------------------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------------------------

template <bool TBF, bool YBF>
__global__ __launch_bounds__(256) void embed_kernel(EmbedArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= a.T) return;
  const int64_t id = a.ids[t];
  const int c0 = blockIdx.y * 2048 + lane * 8;
  const size_t from = (size_t)id * a.K, to = (size_t)t * a.K;
  float v[4][8];
  if (id >= 0 && id < a.V) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c0 + 512 * i < a.K) load_f8<TBF>(a.table, from + c0 + 512 * i, v[i]);
  } else {
    const float fill = id < 0 ? 0.f : __uint_as_float(0x7FC00000u);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = fill;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (c0 + 512 * i >= a.K) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] *= a.scale;
    store_f8<YBF>(a.y, to + c0 + 512 * i, v[i]);
  }
}

// ---------------------------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------------------------

constexpr uint32_t kNone = 0xFFFFFFFFu;      // an id outside the table: sorted last, never summed
constexpr int kFillBlocks = 2048;

struct Sorted {                              // the workspace's arrays
  uint32_t *chunk_id, *chunk_tok, *id, *tok;
  uint32_t* runs;                            // [0]: number of long runs; then {first position, id} each
  float* part;
  int32_t chunks;
};

// Chunk blockIdx.x of CH tokens by id, then token; the blocks behind clear the gradient.
template <int CH, int THREADS>
__global__ __launch_bounds__(THREADS) void embed_sort_kernel(EmbedBwdArgs a, Sorted s) {
  __shared__ uint64_t key[CH];
  const int tid = threadIdx.x;
  if ((int)blockIdx.x >= s.chunks) {
    const int64_t n = a.V * a.K / 4;
    const int64_t step = (int64_t)(gridDim.x - s.chunks) * THREADS;
    float4* out = (float4*)a.dtable;
    for (int64_t i = (int64_t)(blockIdx.x - s.chunks) * THREADS + tid; i < n; i += step)
      out[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    return;
  }
  const int64_t t0 = (int64_t)blockIdx.x * CH;
  if (blockIdx.x == 0 && tid == 0) s.runs[0] = 0;
  for (int i = tid; i < CH; i += THREADS) {
    const int64_t t = t0 + i;
    uint32_t id = kNone;
    if (t < a.T) {
      const int32_t v = a.ids[t];
      if (v >= 0 && v < a.V) id = (uint32_t)v;
    }
    key[i] = ((uint64_t)id << 32) | (uint32_t)i;
  }
  __syncthreads();
  // bitonic network: after the step of size n, runs of n are in order, every other one reversed
  for (int n = 2; n <= CH; n <<= 1) {
    for (int d = n >> 1; d > 0; d >>= 1) {
      for (int i = tid; i < CH / 2; i += THREADS) {
        const int lo = ((i & ~(d - 1)) << 1) | (i & (d - 1)), hi = lo | d;
        const uint64_t x = key[lo], y = key[hi];
        if ((x > y) == ((lo & n) == 0)) {
          key[lo] = y;
          key[hi] = x;
        }
      }
      __syncthreads();
    }
  }
  for (int i = tid; i < CH; i += THREADS) {
    s.chunk_id[t0 + i] = (uint32_t)(key[i] >> 32);
    s.chunk_tok[t0 + i] = (uint32_t)t0 + (uint32_t)key[i];
  }
}

// Places of the sorted chunks' elements among all of them: chunks before count what is not above, the
// ones behind what is below, so equal ids stay in the order of their tokens.
template <int CH>
__global__ __launch_bounds__(256) void embed_rank_kernel(int64_t T, Sorted s) {
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int mine = (int)(e / CH);
  const uint32_t id = s.chunk_id[e], tok = s.chunk_tok[e];
  int64_t place = e - (int64_t)mine * CH;
#pragma unroll 4
  for (int c = 0; c < s.chunks; ++c) {
    if (c == mine) continue;
    const uint32_t* k = s.chunk_id + (int64_t)c * CH;
    const uint64_t bar = (uint64_t)id + (c < mine);   // what is below this comes first
    int n = 0;
#pragma unroll
    for (int d = CH / 2; d > 0; d >>= 1)
      if (k[n + d - 1] < bar) n += d;
    if (k[n] < bar) ++n;
    place += n;
  }
  if (tok < T && place < T) {
    s.id[place] = id;
    s.tok[place] = tok;
  }
}

// One wave: kEmbedTile sorted positions, 512 columns.
template <bool DBF, bool ACC>
__global__ __launch_bounds__(256) void embed_sum_kernel(EmbedBwdArgs a, Sorted s) {
  constexpr int U = ACC ? 4 : 8;             // rows in flight
  const int lane = threadIdx.x & 63;
  const int64_t tile = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t p0 = tile * kEmbedTile;
  if (p0 >= a.T) return;
  const int col = blockIdx.y * 512 + lane * 8;
  const bool live = col < a.K;
  // ids and tokens of the 64 positions from p0 on, ids of the 64 before
  const uint32_t id = p0 + lane < a.T ? s.id[p0 + lane] : kNone;
  const uint32_t tok = p0 + lane < a.T ? s.tok[p0 + lane] : 0;
  const uint32_t before = p0 - 64 + lane >= 0 ? s.id[p0 - 64 + lane] : kNone;
  const uint64_t valid = __ballot(id != kNone);
  if (!(valid & 1)) return;
  const uint32_t next = __shfl_down(id, 1, 64);
  // position i ends its run (that of lane 63, which is never asked for, may not)
  const uint64_t last = __ballot(next != id) & valid;
  const uint32_t id0 = __shfl(id, 0, 64);
  const uint64_t same = __ballot(before == id0);
  const int back = same == ~0ull ? 64 : __clzll((long long)~same);
  const int ahead = __ffsll((unsigned long long)(last | (1ull << 63)));   // positions of the first run
  const bool head_long = back > 0 && back + ahead > kEmbedLong;
  int i0 = 0, end = 0;
  bool piece = false;                        // the last run goes on: its part is a piece
  if (back > 0 && !head_long) i0 = ahead;    // summed by the wave where it starts
  if (i0 >= kEmbedTile) return;
  if (head_long && ahead >= kEmbedTile) {
    end = kEmbedTile;
    piece = true;
  } else {
    // the run that holds the tile's last valid position
    const uint64_t inside = valid & ((1ull << kEmbedTile) - 1);
    const int at = 63 - __clzll((long long)inside);
    if (at < i0) return;
    const uint64_t ends_before = last & ((1ull << at) - 1);
    const int start = ends_before ? 64 - __clzll((long long)ends_before) : 0;
    const int stop = __ffsll((unsigned long long)((last >> at) | (1ull << 63))) + at;
    const bool is_head = start == 0 && back > 0;
    if (!is_head && stop - start > kEmbedLong) {
      end = kEmbedTile;
      piece = true;
      if (lane == 0 && blockIdx.y == 0) {    // the list's order is irrelevant: its runs are independent
        const uint32_t k = atomicAdd(s.runs, 1u);
        s.runs[1 + 2 * k] = (uint32_t)(p0 + start);
        s.runs[2 + 2 * k] = (uint32_t)__builtin_amdgcn_readlane((int)id, at);
      }
    } else {
      end = stop;
    }
  }
  float acc[8] = {};
  bool first = true;                         // the run in hand is the one at p0
  for (int i = i0; i < end; i += U) {
    float v[U][8], old[ACC ? U : 1][8];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int p = min(i + j, end - 1);
      const size_t row = (uint32_t)__builtin_amdgcn_readlane((int)tok, p);
      if (live) load_f8<DBF>(a.dy, row * a.K + col, v[j]);
      if constexpr (ACC) {
        if ((last >> p) & 1) {
          const size_t to = (uint32_t)__builtin_amdgcn_readlane((int)id, p);
          if (live) load_f8<false>(a.dtable, to * a.K + col, old[j]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int p = i + j;
      if (p >= end) break;
#pragma unroll
      for (int c = 0; c < 8; ++c) acc[c] += v[j][c];
      const bool ends = (last >> p) & 1;
      if (!ends && p + 1 < end) continue;
      float* to;
      if (first && head_long) to = s.part + (size_t)tile * 2 * a.K;
      else if (piece && p + 1 == end) to = s.part + ((size_t)tile * 2 + 1) * a.K;
      else {
        to = a.dtable + (size_t)(uint32_t)__builtin_amdgcn_readlane((int)id, p) * a.K;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          acc[c] *= a.scale;
          if constexpr (ACC) acc[c] += old[j][c];
        }
      }
      if (live) store_f8<false>(to, col, acc);
#pragma unroll
      for (int c = 0; c < 8; ++c) acc[c] = 0.f;
      first = false;
    }
  }
}

// Long runs: the pieces of one run and 512 columns at a time, by 16 waves, each of which sums every
// sixteenth piece in order.
template <bool ACC>
__global__ __launch_bounds__(1024) void embed_join_kernel(EmbedBwdArgs a, Sorted s) {
  __shared__ float sums[16][512];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = blockIdx.y * 512 + lane * 8;
  const bool live = col < a.K;
  const uint32_t n = s.runs[0];
  for (uint32_t k = blockIdx.x; k < n; k += gridDim.x) {
    const int64_t start = s.runs[1 + 2 * k];
    const uint32_t id = s.runs[2 + 2 * k];
    int64_t lo = start, hi = a.T;            // s.id[lo] is the run's, s.id[hi] is not
    while (hi - lo > 1) {
      const int64_t m = (lo + hi) >> 1;
      if (s.id[m] == id) lo = m;
      else hi = m;
    }
    const int64_t t0 = start / kEmbedTile, t1 = lo / kEmbedTile;   // tiles of its first and last piece
    float acc[8] = {};
    for (int64_t t = t0 + wave; t <= t1; t += 16) {
      float v[8];
      if (live) {
        load_f8<false>(s.part, ((size_t)t * 2 + (t == t0)) * a.K + col, v);
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[c] += v[c];
      }
    }
    store_f8<false>(sums[wave], lane * 8, acc);
    __syncthreads();
    if (threadIdx.x < 512 && blockIdx.y * 512 + (int)threadIdx.x < a.K) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < 16; ++w) sum += sums[w][threadIdx.x];
      float* to = a.dtable + (size_t)id * a.K + blockIdx.y * 512 + threadIdx.x;
      sum *= a.scale;
      if constexpr (ACC) sum += *to;
      *to = sum;
    }
    __syncthreads();
  }
}

}  // namespace

hipError_t launch_embed(const EmbedArgs& a, bool table_bf16, bool y_bf16, hipStream_t s) {
  const dim3 grid((unsigned)((a.T + 3) / 4), (unsigned)((a.K + 2047) / 2048));
  if (table_bf16) {
    if (y_bf16) embed_kernel<true, true><<<grid, 256, 0, s>>>(a);
    else embed_kernel<true, false><<<grid, 256, 0, s>>>(a);
  } else {
    if (y_bf16) embed_kernel<false, true><<<grid, 256, 0, s>>>(a);
    else embed_kernel<false, false><<<grid, 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

hipError_t launch_embed_bwd(const EmbedBwdArgs& a, bool dy_bf16, hipStream_t s) {
  const EmbedBwdWs w = embed_bwd_ws(a.T, a.K);
  Sorted so;
  so.chunk_id = (uint32_t*)(a.ws + w.chunk_id);
  so.chunk_tok = (uint32_t*)(a.ws + w.chunk_tok);
  so.id = (uint32_t*)(a.ws + w.id);
  so.tok = (uint32_t*)(a.ws + w.tok);
  so.runs = (uint32_t*)(a.ws + w.runs);
  so.part = (float*)(a.ws + w.part);
  so.chunks = (int32_t)w.chunks;
  const int64_t n = a.V * a.K / 4;
  const bool wide = w.chunk == 4096;
  const int threads = wide ? 1024 : 256;
  const unsigned fill = a.accumulate ? 0 : (unsigned)std::min<int64_t>(kFillBlocks, (n + threads - 1) / threads);
  const unsigned blocks = (unsigned)w.chunks + fill;
  if (blocks == 0) return hipSuccess;
  if (wide) embed_sort_kernel<4096, 1024><<<blocks, 1024, 0, s>>>(a, so);
  else embed_sort_kernel<1024, 256><<<blocks, 256, 0, s>>>(a, so);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.T == 0) return e;
  if (w.chunks > 1) {
    const unsigned grid = (unsigned)(w.chunks * w.chunk / 256);
    if (wide) embed_rank_kernel<4096><<<grid, 256, 0, s>>>(a.T, so);
    else embed_rank_kernel<1024><<<grid, 256, 0, s>>>(a.T, so);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  const unsigned slices = (unsigned)((a.K + 511) / 512);
  const dim3 grid((unsigned)((w.tiles + 3) / 4), slices);
  if (dy_bf16) {
    if (a.accumulate) embed_sum_kernel<true, true><<<grid, 256, 0, s>>>(a, so);
    else embed_sum_kernel<true, false><<<grid, 256, 0, s>>>(a, so);
  } else {
    if (a.accumulate) embed_sum_kernel<false, true><<<grid, 256, 0, s>>>(a, so);
    else embed_sum_kernel<false, false><<<grid, 256, 0, s>>>(a, so);
  }
  if ((e = hipGetLastError()) != hipSuccess || a.T <= kEmbedLong) return e;
  const dim3 jgrid((unsigned)std::min<int64_t>(64, a.T / (kEmbedLong + 1)), slices);
  if (a.accumulate) embed_join_kernel<true><<<jgrid, 1024, 0, s>>>(a, so);
  else embed_join_kernel<false><<<jgrid, 1024, 0, s>>>(a, so);
  return hipGetLastError();
}

}  // namespace bl
