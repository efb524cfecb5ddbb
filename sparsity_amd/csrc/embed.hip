// Embedding rows by token id, and the gradient of the table.
//
//   y[t] = round(scale * table[ids[t]])
//   dtable[v] (+)= scale * sum over the tokens t with ids[t] = v of dy[t]
//
// Forward: a wave takes up to 2048 columns of one token, all of its loads before the first store.  Bound by memory: 8192
// tokens of 3200, fp32 to bf16, 18.7 us (7.8 TB/s, part of it from the last cache); 16 tokens of 2560 2 to 5 us, latency.
//
// Gradient: tokens are sorted by id, so that a row's tokens are a run of sorted positions, and each run
// is summed in the order of its tokens: results do not vary from run to run, and nothing is added by
// atomics.  Launches:
//   sort   blocks sort a chunk of tokens each, in registers and LDS; where the gradient is overwritten, others clear its
//          first rows
//   rank   (several chunks) an element's place is its place in its chunk plus, by bisection, what the
//          other chunks of its span of 65536 tokens hold before it; where there are several spans, once more
//   sum    a wave takes 16 sorted positions and 512 columns; it sums every run that starts there, up to
//          32 positions of it, and writes the row; of a longer run, what lies inside its 16 goes to the
//          workspace.  Where the gradient is overwritten, the other blocks of the launch clear those of the remaining
//          rows that no token names
//   join   the pieces of long runs, in order
// Bound by memory in the sums: 8192 bf16 tokens of 3200 written over 32000 rows, 457 MB, take 16 (84 MB cleared), 5, 64 and 5
// us; 32749 fp32 tokens of 2560 added to a table of 131072 rows, 579 MB, 11, 11, 130 (4.5 TB/s, the rate of a copy) and 11.
// The other launches are latency: chains of dependent loads, LDS steps and barriers.
#include <algorithm>

#include "block_ops.hpp"
#include "device_common.hpp"
#include "step_ops.hpp"
#include "wave_ops.hpp"

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
constexpr int kChunk = kEmbedChunk;
constexpr int kSortThreads = kChunk / 2;
constexpr int kFillRows = 8;                 // rows that a wave of a fill block looks up
// Bytes of the gradient that are cleared beside the sort, whose few blocks leave most of the chip idle.  Whole calls with
// none, 40, 80 and 160 MB: 8192 tokens of 3200 onto 32000 rows 112, 107, 102 and 104 us, 64 of 2560 67, 64, 62 and 65,
// 32749 of 2560 onto 131072 rows 335, 332, 329 and 332.
constexpr int64_t kFillSort = 80 << 20;
constexpr unsigned kFillBlocks = 512;
// Where tokens can name an eighth of the rows at most, all is cleared there but for as much as hides the sums, and without
// looking rows up: named ones are written twice, little of the whole.  Blocks of 256 threads with one store each write 6.6
// TB/s (1.26 GB; blocks of 1024 6.1, pieces of 64 KB and more, as those of a row's block, 5.0).  Whole calls with 80 MB in
// 512 blocks, and with all but 128, 64 and 0 MB: 64 tokens of 2400 onto 131072 rows 247, 198, 196 and 198 us (zeros and an
// addition by index 204), 8192 of 2400 254, 217, 221 and 227, 4000 of 2560 onto 32000 67, 63, 68 and 74.
constexpr int kPieceThreads = 256;
constexpr int64_t kFillSum = 128 << 20;

struct Sorted {                              // the workspace's arrays
  uint32_t *chunk_id, *chunk_tok, *span_id, *span_tok, *id, *tok;
  uint32_t* runs;                            // [0]: number of long runs; then {first position, id} each
  float* part;
  int32_t chunks;
};

// One step of a bitonic network inside a wave: the lane's key against the one at distance d.
template <class Key>
__device__ __forceinline__ Key exchange(Key v, int d, bool up) {
  Key w;
  if constexpr (sizeof(Key) == 8) w = (Key)__shfl_xor((long long)v, d, 64);
  else if (d == 1) w = lane_move<0xB1, 0xF>(v, v);           // within rows of lanes in registers
  else if (d == 2) w = lane_move<0x4E, 0xF>(v, v);
  else if (d == 8) w = lane_move<0x128, 0xF>(v, v);
  else w = (Key)__shfl_xor((int)v, d, 64);
  const bool low = (threadIdx.x & d) == 0;
  return (v < w) == (low == up) ? v : w;
}

// Past the caches: 1024 tokens of 2560 onto 32000 rows 78 -> 66 us a call, 8192 of 512 onto 131072 77 -> 63 (32749 of 2560
// 329 -> 335).
__device__ __forceinline__ void clear4(float4* p) { __builtin_nontemporal_store((v4f){0.f, 0.f, 0.f, 0.f}, (v4f*)p); }

// Clears the gradient's first rows, whatever comes to stand there: block `at` of `blocks`.
__device__ __forceinline__ void fill_first(const EmbedBwdArgs& a, int64_t rows, int64_t at, int64_t blocks) {
  float4* out = (float4*)a.dtable;
  const int64_t i1 = rows * a.K / 4;
  for (int64_t i = at * blockDim.x + threadIdx.x; i < i1; i += blocks * blockDim.x)
    clear4(out + i);
}

// Chunk blockIdx.x of the tokens by id, then token.  A key is the id over the bits of the token's place in the
// chunk: 32 bits in all for tables of less than 2^21 rows.  A few keys to a thread; distances below 64 inside a wave.  The
// first `top` places, a power of two, hold all tokens that there are.
template <class Key, int kThreads>
__global__ __launch_bounds__(kThreads) void embed_sort_kernel(EmbedBwdArgs a, Sorted s, int64_t fill, int top) {
  constexpr int kKeys = kChunk / kThreads;
  __shared__ Key key[kChunk];
  if ((int)blockIdx.x >= s.chunks) {
    fill_first(a, fill, blockIdx.x - s.chunks, gridDim.x - s.chunks);
    return;
  }
  constexpr int kBits = kEmbedChunkBits;
  const int tid = threadIdx.x;
  const int64_t t0 = (int64_t)blockIdx.x * kChunk;
  const Key none = (Key)~(Key)0 >> kBits;
  if (blockIdx.x == 0 && tid == 0) s.runs[0] = 0;
  Key v[kKeys];
#pragma unroll
  for (int h = 0; h < kKeys; ++h) {
    const int i = h * kThreads + tid;
    const int32_t id = t0 + i < a.T ? a.ids[t0 + i] : -1;
    v[h] = (id >= 0 && id < a.V ? (Key)id : none) << kBits | (Key)i;
  }
  for (int n = 2; n <= top; n <<= 1) {       // runs of n in order, every other one reversed
    if (n > 64) {
      __syncthreads();
#pragma unroll
      for (int h = 0; h < kKeys; ++h) key[h * kThreads + tid] = v[h];
      __syncthreads();
      for (int d = n >> 1; d >= 64; d >>= 1) {
#pragma unroll
        for (int h = 0; h < kKeys / 2; ++h) {
          const int i = h * kThreads + tid, lo = ((i & ~(d - 1)) << 1) | (i & (d - 1)), hi = lo | d;
          const Key x = key[lo], y = key[hi];
          if ((x > y) == ((lo & n) == 0)) {
            key[lo] = y;
            key[hi] = x;
          }
        }
        __syncthreads();
      }
#pragma unroll
      for (int h = 0; h < kKeys; ++h) v[h] = key[h * kThreads + tid];
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
      if (d >= n) continue;
#pragma unroll
      for (int h = 0; h < kKeys; ++h) v[h] = exchange(v[h], d, ((h * kThreads + tid) & n) == 0);
    }
  }
#pragma unroll
  for (int h = 0; h < kKeys; ++h) {
    const int i = h * kThreads + tid;
    s.chunk_id[t0 + i] = v[h] >> kBits == none ? kNone : (uint32_t)(v[h] >> kBits);
    s.chunk_tok[t0 + i] = (uint32_t)t0 + (uint32_t)(v[h] & (kChunk - 1));
  }
}

// Places of the sorted chunks' elements among those of their span: chunks before count what is not above, the
// ones behind what is below, so equal ids stay in the order of their tokens.  The chunks' ids are searched in
// LDS, four chunks at a time.
constexpr int kRankChunks = 16;              // in LDS at a time
constexpr int kRankThreads = 512;
constexpr int kTogether = 4;                 // searches in flight
__global__ __launch_bounds__(kRankThreads) void embed_rank_kernel(int64_t T, Sorted s) {
  __shared__ __attribute__((aligned(16))) uint32_t k[kRankChunks * kChunk];
  const int64_t e = (int64_t)blockIdx.x * kRankThreads + threadIdx.x;
  const int mine = (int)(e / kChunk);
  const uint32_t id = s.chunk_id[e], tok = s.chunk_tok[e];
  const int first = mine / kEmbedSpan * kEmbedSpan, end = min(first + kEmbedSpan, s.chunks);
  int64_t place = e - (int64_t)(mine - first) * kChunk;
  for (int c0 = first; c0 < end; c0 += kRankChunks) {
    const int n = min(kRankChunks, end - c0);
    __syncthreads();
    static_assert(kRankThreads * 4 == kChunk, "a chunk at a time");
    uint4 all[kRankChunks];
#pragma unroll
    for (int c = 0; c < kRankChunks; ++c)
      all[c] = ((const uint4*)s.chunk_id)[(int64_t)min(c0 + c, end - 1) * kRankThreads + threadIdx.x];
#pragma unroll
    for (int c = 0; c < kRankChunks; ++c) ((uint4*)k)[c * kRankThreads + threadIdx.x] = all[c];
    __syncthreads();
    for (int c = 0; c < n; c += kTogether) {
      int at[kTogether] = {};
      uint64_t bar[kTogether];
      const uint32_t* in[kTogether];
#pragma unroll
      for (int j = 0; j < kTogether; ++j) {
        bar[j] = (uint64_t)id + (c0 + c + j < mine);         // what is below this comes first
        in[j] = k + min(c + j, n - 1) * kChunk;
      }
#pragma unroll
      for (int d = kChunk / 2; d > 0; d >>= 1)
#pragma unroll
        for (int j = 0; j < kTogether; ++j) at[j] += in[j][at[j] + d - 1] < bar[j] ? d : 0;
#pragma unroll
      for (int j = 0; j < kTogether; ++j) {
        at[j] += in[j][at[j]] < bar[j];
        if (c + j < n && c0 + c + j != mine) place += at[j];
      }
    }
  }
  if (tok < T) {
    s.span_id[place] = id;
    s.span_tok[place] = tok;
  }
}

// The same of the spans' elements, among all: four spans at a time, from the L2.  Without spans the time of the ranks
// grows with the square of the tokens: 2^20 tokens 3.2 ms and 2^22 45 ms, of 64 columns.
__global__ __launch_bounds__(256) void embed_spans_kernel(int64_t T, Sorted s) {
  constexpr int kSpan = kEmbedSpan * kChunk;
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= T) return;
  const int mine = (int)(e / kSpan), spans = (int)((T + kSpan - 1) / kSpan);
  const uint32_t id = s.span_id[e];
  int64_t place = e - (int64_t)mine * kSpan;
  for (int c = 0; c < spans; c += 4) {
    int at[4] = {}, n[4];
    uint64_t bar[4];
    const uint32_t* in[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int span = min(c + j, spans - 1);
      bar[j] = (uint64_t)id + (span < mine);
      in[j] = s.span_id + (int64_t)span * kSpan;
      n[j] = c + j < spans && span != mine ? (int)min(T - (int64_t)span * kSpan, (int64_t)kSpan) : 0;
    }
    for (int d = kSpan; d > 0; d >>= 1)
#pragma unroll
      for (int j = 0; j < 4; ++j) at[j] += at[j] + d <= n[j] && in[j][at[j] + d - 1] < bar[j] ? d : 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) place += at[j];
  }
  s.id[place] = id;
  s.tok[place] = s.span_tok[e];
}

// Rows of a fill block: a few waves' where they are short.
__host__ __device__ inline int fill_rows_of_block(int K) { return K <= 1024 ? 4 * kFillRows : kFillRows; }

// Clears the rows from r0 on that no token names.  Eight lanes look one row up among the sorted ids, eight places at a time.
__device__ __forceinline__ void fill_rows(const EmbedBwdArgs& a, const Sorted& s, int64_t r0, int rows) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  __shared__ uint8_t named[4 * kFillRows];
  const int mine = wave * kFillRows + (lane >> 3);
  if (mine < rows) {
    const uint32_t row = (uint32_t)(r0 + mine);
    int64_t lo = 0, hi = a.T;                // the first place whose id is not below the row's
    while (hi > lo) {
      const int64_t step = (hi - lo + 7) >> 3, at = lo + (lane & 7) * step;
      const bool below = at < hi && s.id[at] < row;
      const uint32_t mask = (uint32_t)(__ballot(below) >> (lane & 56)) & 0xFF;
      if (mask == 0) break;                  // s.id[lo] is not
      const int last = 31 - __clz((int)mask);
      hi = min(hi, lo + (last + 1) * step);
      lo += last * step + 1;
    }
    if ((lane & 7) == 0) named[mine] = lo < a.T && s.id[lo] == row;
  }
  __syncthreads();
  const int k4 = a.K / 4;
  int w = 256;                               // threads to a row
  while (w / 2 >= k4) w >>= 1;
  for (int r = tid / w; r < rows; r += 256 / w) {
    if (r0 + r >= a.V || named[r]) continue;
    float4* out = (float4*)(a.dtable + (size_t)(r0 + r) * a.K);
    for (int c = tid & (w - 1); c < k4; c += w) clear4(out + c);
  }
}

// One wave: kEmbedTile sorted positions, 512 columns.  The blocks behind the sums' clear the other rows.
template <bool DBF, bool ACC>
__global__ __launch_bounds__(256) void embed_sum_kernel(EmbedBwdArgs a, Sorted s, int64_t sum_blocks, int slices,
                                                        int64_t filled) {
  constexpr int U = ACC ? 4 : 8;             // rows in flight
  if constexpr (!ACC) {
    if ((int64_t)blockIdx.x >= sum_blocks) {
      const int rows = fill_rows_of_block(a.K);
      const int64_t step = gridDim.x - sum_blocks;
      for (int64_t b = blockIdx.x - sum_blocks; filled + b * rows < a.V; b += step) {
        fill_rows(a, s, filled + b * rows, rows);
        __syncthreads();
      }
      return;
    }
  }
  const int lane = threadIdx.x & 63;
  const int slice = blockIdx.x % slices;
  const int64_t tile = (int64_t)(blockIdx.x / slices) * 4 + (threadIdx.x >> 6);
  const int64_t p0 = tile * kEmbedTile;
  if (p0 >= a.T) return;
  const int col = slice * 512 + lane * 8;
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
      if (lane == 0 && slice == 0) {         // the list's order is irrelevant: its runs are independent
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
    int64_t lo = start, hi = a.T;            // s.id[lo] is the run's, s.id[hi] is not: 64 places at a time
    while (hi - lo > 1) {
      const int64_t step = (hi - lo + 63) >> 6, at = lo + lane * step;
      const uint64_t same = __ballot(at < hi && s.id[at] == id);
      const int last = 63 - __clzll((long long)same);
      hi = min(hi, lo + (last + 1) * step);
      lo += last * step;
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
  so.span_id = (uint32_t*)(a.ws + w.span_id);
  so.span_tok = (uint32_t*)(a.ws + w.span_tok);
  so.id = (uint32_t*)(a.ws + w.id);
  so.tok = (uint32_t*)(a.ws + w.tok);
  so.runs = (uint32_t*)(a.ws + w.runs);
  so.part = (float*)(a.ws + w.part);
  so.chunks = (int32_t)w.chunks;
  hipError_t e = hipSuccess;
  int64_t filled = 0;
  if (a.T > 0) {
    const unsigned sorts = (unsigned)w.chunks;
    const int64_t row = (int64_t)a.K * 4, rest = a.V * row - kFillSum;
    const bool pieces = !a.accumulate && a.T <= a.V / 8 && rest > kFillSort;
    unsigned some = 0;                       // blocks that clear
    if (pieces) {
      filled = rest / row;
      some = (unsigned)std::min<int64_t>((filled * row / 16 + kPieceThreads - 1) / kPieceThreads, 1 << 22);
    } else if (!a.accumulate) {
      filled = std::min<int64_t>(a.V, kFillSort / row);
      some = kFillBlocks;
    }
    int top = 64;
    while (top < kChunk && top < a.T) top *= 2;
    const bool small = a.V < ((int64_t)1 << (32 - kEmbedChunkBits));
    if (pieces) {
      if (small) embed_sort_kernel<uint32_t, kPieceThreads><<<sorts + some, kPieceThreads, 0, s>>>(a, so, filled, top);
      else embed_sort_kernel<uint64_t, kPieceThreads><<<sorts + some, kPieceThreads, 0, s>>>(a, so, filled, top);
    } else {
      if (small) embed_sort_kernel<uint32_t, kSortThreads><<<sorts + some, kSortThreads, 0, s>>>(a, so, filled, top);
      else embed_sort_kernel<uint64_t, kSortThreads><<<sorts + some, kSortThreads, 0, s>>>(a, so, filled, top);
    }
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (w.chunks > 1) {
      embed_rank_kernel<<<(unsigned)w.chunks * (kChunk / kRankThreads), kRankThreads, 0, s>>>(a.T, so);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (w.chunks > kEmbedSpan) {
      embed_spans_kernel<<<(unsigned)((a.T + 255) / 256), 256, 0, s>>>(a.T, so);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
  }
  const int slices = (a.K + 511) / 512;
  const int64_t sums = (w.tiles + 3) / 4 * slices;
  const int fill = fill_rows_of_block(a.K);
  const int64_t blocks = sums + (a.accumulate ? 0 : std::min<int64_t>((a.V - filled + fill - 1) / fill, 1 << 20));
  if (blocks == 0) return hipSuccess;
  if (dy_bf16) {
    if (a.accumulate) embed_sum_kernel<true, true><<<(unsigned)blocks, 256, 0, s>>>(a, so, sums, slices, filled);
    else embed_sum_kernel<true, false><<<(unsigned)blocks, 256, 0, s>>>(a, so, sums, slices, filled);
  } else {
    if (a.accumulate) embed_sum_kernel<false, true><<<(unsigned)blocks, 256, 0, s>>>(a, so, sums, slices, filled);
    else embed_sum_kernel<false, false><<<(unsigned)blocks, 256, 0, s>>>(a, so, sums, slices, filled);
  }
  if ((e = hipGetLastError()) != hipSuccess || a.T <= kEmbedLong) return e;
  const dim3 jgrid((unsigned)std::min<int64_t>(256, a.T / (kEmbedLong + 1)), (unsigned)slices);
  if (a.accumulate) embed_join_kernel<true><<<jgrid, 1024, 0, s>>>(a, so);
  else embed_join_kernel<false><<<jgrid, 1024, 0, s>>>(a, so);
  return hipGetLastError();
}

}  // namespace bl
