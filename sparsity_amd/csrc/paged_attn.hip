// Attention of one new token per sequence over a paged key-value cache, split over the cache's
// length and joined.
//
//   s_j = scale * (q . k_j)      p_j = exp(s_j - m)      out = sum p_j v_j / sum p_j      lse = m + log sum p_j
//
// over the sequence's live positions j (its last `window` ones where a window is given).  The keys
// and values are read once, 4 bytes per element pair in bf16, for 4 G flops (G query heads share a
// key head), so the kernel is bound by memory: the work is to keep loads in flight and to spend
// little on each byte.
//
// A wave takes 32 keys at a time (64 of an int8 cache) for up to 16 query heads of one key head (32 in
// two tiles, see paged_attn_split), the running maximum and sum of the softmax in registers:
//   S^T = K Q^T   16x16x32 MFMAs with 16 keys as rows.  A lane's operand is 16 contiguous bytes of
//                 its key's row, straight from memory.  Lane (g, n) (g = lane / 16, n = lane % 16)
//                 receives the scores of query n and keys 4g..4g+3 of each 16-key tile.
//   O^T = V^T P^T the contraction runs over keys, whose order is free: lane (g, n) supplies for the
//                 B operand exactly the eight probabilities it already holds (4g..4g+3 of both
//                 tiles), so P never leaves its registers, and for the A operand the value rows of
//                 the same eight keys.  It loads VE contiguous elements of each (16 lanes cover a
//                 whole row), and one byte permute per two elements turns eight row pieces into
//                 VE operands (operand j: element VE n + j of the eight keys).  No LDS, no shuffle.
// A lane's accumulators all belong to query n, so a new maximum rescales them by one lane-local
// factor.  Probabilities enter the product as three bf16 terms (the value, and what the terms so far
// leave of it), an fp32 query as three as well: both keep their 24 bits.  (Two terms of a probability,
// good to 2^-17, would be 2 to 3e-6 off before a bf16 output's rounding, ten times the error of 32-bit
// operations; the third costs nothing over a bf16 cache, 1 to 2% over an int8 one at D = 128 and up to
// 5% at D = 64: 16 x 8000 tokens 39.7 -> 41.6 us.)
//
// The launch is one block per resident place of the chip (two per CU, one where registers ask for it: a
// wave then has 16 KB of keys and values in flight while the matrix cores work on the last 16; three waves
// per SIMD spill, one leaves int8 caches at half the rate).  The blocks share all keys of all sequences evenly (see Work), the
// four waves of a block take quarters of its run and join in LDS; a run that is not its group's whole
// goes to the workspace as partial sums, and the last block of the group to finish joins the runs, in
// their order, so the result does not depend on which block that is.
//
// Measured: 64 x 8192 tokens, 8 key heads, 32 query heads of 128, bf16: 362 us, 5.9 TB/s; the same in
// int8 210 us, 5.3 TB/s; one sequence of 262144 tokens, 5 key heads: 131 us, 5.1 TB/s; 48 ragged
// sequences up to 6001 tokens, int8: 71 us, 4.2 TB/s; 700 tokens: 12 us, ten dependent round trips to
// memory; 24 heads on one key head of 256, read twice, 64 x 8000 tokens: 175 us, 3.0 TB/s.  What is lost: 7 us to the first keys (lengths, then pages, then rows), blocks that end up to
// 12% apart under equal shares (memory serves the CUs unevenly), about 3 us for a join.
#include <algorithm>

#include "block_ops.hpp"
#include "device_common.hpp"

namespace bl {

namespace {

constexpr int kWaves = 4;
constexpr int kQ = 16;                      // query heads of an MFMA
constexpr int64_t kTile = 32 * kWaves;      // keys of a tile: one group of 32 per wave
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ v4f mfma_bf16(const bf16x8& a, const bf16x8& b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ bf16x8 frag(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint4 u = make_uint4(a, b, c, d);
  return __builtin_bit_cast(bf16x8, u);
}
// Signed byte j of a dword as fp32; exact in bf16, so its upper half is the bf16 value.
__device__ __forceinline__ uint32_t i8_f32(uint32_t w, int j) {
  return __float_as_uint((float)(int8_t)(w >> (8 * j)));
}
__device__ __forceinline__ uint32_t upper_halves(uint32_t lo, uint32_t hi) {
  return __builtin_amdgcn_perm(hi, lo, 0x07060302u);
}
// Four bytes of a dword as four bf16 in two dwords.
__device__ __forceinline__ void i8x4_bf16(uint32_t w, uint32_t& a, uint32_t& b) {
  a = upper_halves(i8_f32(w, 0), i8_f32(w, 1));
  b = upper_halves(i8_f32(w, 2), i8_f32(w, 3));
}

// Weight of a partial sum with running maximum m and sum l under the joint maximum.  One without live
// keys has sums of zero and weighs nothing; any other one counts even at a weight of 0 or NaN, so that
// a sum that is not finite is not hidden.
__device__ __forceinline__ float weight(float m, float l, float top) {
  if (m == -INFINITY) return l == 0.f ? 0.f : __builtin_nanf("");
  return __builtin_amdgcn_exp2f(m - top);
}

// Device-scope accesses of the partial sums, past the caches that the XCDs do not share.
__device__ __forceinline__ void put(float* p, float v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float get(const float* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ v4f get4(const float* p) {   // 8-byte aligned
  const uint64_t lo = __hip_atomic_load((const uint64_t*)p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const uint64_t hi = __hip_atomic_load((const uint64_t*)p + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return v4f{__uint_as_float((uint32_t)lo), __uint_as_float((uint32_t)(lo >> 32)),
             __uint_as_float((uint32_t)hi), __uint_as_float((uint32_t)(hi >> 32))};
}

// VE contiguous elements of VE * BYTES bytes as dwords.
template <int N>
__device__ __forceinline__ void load_dw(const void* p, uint32_t* r) {
  if constexpr (N == 1) {
    r[0] = *(const uint32_t*)p;
  } else if constexpr (N == 2) {
    const uint2 u = *(const uint2*)p;
    r[0] = u.x; r[1] = u.y;
  } else {
    const uint4 u = *(const uint4*)p;
    r[0] = u.x; r[1] = u.y; r[2] = u.z; r[3] = u.w;
  }
}

// Resident blocks per CU (one wave of each per SIMD) that the registers allow without spilling (but for 20
// bytes with two query tiles of fp32 queries over int8 keys of 64).
constexpr int resident(int DT, int QT) { return DT * QT <= 128 ? 2 : 1; }

// The work of a launch as one run of units: sequence after sequence, group (key head and query tile)
// after group, each the cost of starting and ending a group, kStart units, and then its tiles of
// kTile keys.  Every block takes an equal share, whatever the lengths; the tiles of a block fall into
// segments, one per group it meets.  (A sequence without keys counts as one tile, so that its zeros
// get written.)  kStart: a group costs a block about the time of 96 KB of keys and values; without it,
// the blocks that drew the short sequences of a ragged batch ran twice as long as the others.
constexpr int64_t start_units(int DT, int EB) {
  const int64_t tile = kTile * 2 * DT * EB;
  return (98304 + tile - 1) / tile;
}

struct Work {
  int64_t total;      // units
  int64_t blocks;     // blocks that take part
  __device__ int64_t first(int64_t block) const { return block * total / blocks; }
  __device__ int64_t owner(int64_t unit) const { return ((unit + 1) * blocks - 1) / total; }
};

// A value that is the same in every lane, for the compiler to know it is.
__device__ __forceinline__ int64_t uniform(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)v >> 32));
  return (int64_t)((uint64_t)hi << 32 | lo);
}

// The same value, which the compiler may not compute ahead of this place: what the end of a segment
// derives from the thread's index would otherwise sit in registers all through the loop over keys
// (256 of them and 112 bytes of spills at D = 128, against 232 and none).
__device__ __forceinline__ int here(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// Live positions of a sequence: [first, len).
struct Span {
  int64_t first, len;
  __device__ int64_t tiles() const { return max((int64_t)1, (len - first + kTile - 1) / kTile); }
};
__device__ __forceinline__ Span span_of(const AttnArgs& a, int64_t b) {
  const int64_t cap = a.blocks_per_seq * a.kv.page_size;
  Span s;
  s.len = max((int64_t)0, min((int64_t)a.lens[b], cap));
  s.first = a.window > 0 ? max((int64_t)0, s.len - a.window) : 0;
  return s;
}

// DT: 64, 128 or 256, the head dimension's room.  I8: int8 cache.  QF: fp32 queries.  QT: query tiles.
template <int DT, bool I8, bool QF, int QT>
__global__ __launch_bounds__(64 * kWaves, resident(DT, QT)) void paged_attn_kernel(AttnArgs a) {
  constexpr int R = kQ * QT;                // query heads of a block
  constexpr int EB = I8 ? 1 : 2;            // bytes per cache element
  constexpr int VE = DT / 16;               // value elements per lane and key
  constexpr int VW = VE * EB / 4;           // their dwords
  constexpr int VL = VW > 4 ? 2 : 1;        // 16-byte loads (or one narrower)
  constexpr int KC = DT / 32;               // 32-element steps of the q . k contraction
  constexpr int KW = DT * EB / 16;          // key dwords per lane and key tile
  constexpr int QS = QF ? 3 : 1;            // bf16 terms of a query element
  constexpr int PS = 3;                     // and of a probability
  // runs of 32 keys a wave takes at a time: 16 KB at D = 128 (fp32 queries at D = 256 leave no registers
  // for two: 64 x 8000 tokens 589 us with spills, 418 with one)
  constexpr int KG = I8 && !(DT > 128 && QF) ? 2 : 1;
  constexpr int GK = 32 * KG;

  __shared__ __attribute__((aligned(16))) float sm_o[kWaves][R][DT + 4];   // the waves' sums
  __shared__ float sm_m[kWaves][R], sm_l[kWaves][R];
  // per-wave rings of two groups of keys: byte offsets of the keys' rows (-1: masked), scales
  __shared__ __attribute__((aligned(16))) int64_t ring[kWaves][2][GK];
  __shared__ __attribute__((aligned(16))) float sring[I8 ? kWaves : 1][2][I8 ? GK : 1];
  __shared__ int last_sh;

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane >> 4, n = lane & 15;
  const int D = a.kv.head_dim;
  const int per_seq = a.kv.heads * a.qtiles;   // groups per sequence
  const int prows = min(R, a.G);               // rows of a partial sum

  // this block's units [u0, u1), and the sequence of the first: sums over the lengths, 64 at a time
  constexpr int64_t kStart = start_units(DT, EB);
  auto units_of = [&](int64_t b) { return b < a.B ? (span_of(a, b).tiles() + kStart) * per_seq : 0; };
  Work work;
  int64_t held = units_of(lane);               // of sequence `lane`
  int64_t mine = held;
  for (int64_t b = lane + 64; b < a.B; b += 64) mine += units_of(b);
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) mine += __shfl_xor(mine, s, 64);
  work.total = uniform(mine);
  work.blocks = min((int64_t)gridDim.x, work.total);
  if ((int64_t)blockIdx.x >= work.blocks) return;
  const int64_t u0 = work.first(blockIdx.x), u1 = work.first(blockIdx.x + 1);
  int64_t b = 0, seq0 = 0;                     // sequence, its first unit
  for (int64_t base = 0; base < a.B; base += 64) {
    int64_t end = base ? units_of(base + lane) : held;   // to inclusive sums
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const int64_t v = __shfl_up(end, s, 64);
      if (lane >= s) end += v;
    }
    const uint64_t past = __ballot(seq0 + end <= u0 && base + lane < a.B);   // a prefix of the lanes
    const int skip = __popcll(past);
    if (skip > 0) seq0 += uniform(__shfl(end, skip - 1, 64));
    b = base + skip;
    if (skip < 64) break;
  }

  for (int64_t unit = u0; unit < u1;) {
    const Span sp = span_of(a, b);
    const int64_t tiles = sp.tiles(), units = tiles + kStart;
    const int in_seq = (int)((unit - seq0) / units);      // group of the sequence
    const int64_t next_group = seq0 + (in_seq + 1) * units, g0 = next_group - tiles;   // g0: its first tile
    const int64_t tile = max(unit, g0), end = min(u1, next_group);   // the segment is [tile, end)
    const int64_t sq = b;
    unit = end;
    if (unit == seq0 + units * per_seq) { seq0 = unit; ++b; }
    if (tile >= end) continue;                            // the start of a group that the next block takes
    const int hk = in_seq / a.qtiles, qt = in_seq - hk * a.qtiles;
    const int64_t owner0 = work.owner(g0);
    const int active = (int)(work.owner(g0 + tiles - 1) - owner0) + 1;   // blocks that share the group
    const int rows = min(R, a.G - qt * R);                // live query heads
    const int hq0 = hk * a.G + qt * R;
    const int64_t k0 = sp.first + (tile - g0) * kTile, k1 = min(sp.len, sp.first + (end - g0) * kTile);
    // this wave's quarter, in whole runs of 32 keys
    const int64_t quarter = ((k1 - k0 + kWaves - 1) / kWaves + 31) / 32 * 32;
    const int64_t w0 = min(k1, k0 + wave * quarter), w1 = min(k1, w0 + quarter);
    const int groups = (int)((w1 - w0 + GK - 1) / GK);

    const int32_t* table = a.blocks + sq * a.blocks_per_seq;
    const int ps = a.kv.page_size;
    const int64_t head_off = hk * a.kv.head_stride;
    const char* kbase = (const char*)a.kv.k + head_off * EB;
    const char* vbase = (const char*)a.kv.v + head_off * EB;

    // lane j of the wave looks after key j of each group (of 32 keys, lanes 32 and up repeat the lower
    // ones): its page is read one group ahead of the row offset that needs it
    auto key_of = [&](int grpi) { return w0 + GK * (int64_t)grpi + (lane & (GK - 1)); };
    auto page_of = [&](int grpi) -> int32_t {
      const int64_t t = key_of(grpi);
      return t < w1 ? table[(uint32_t)t / (uint32_t)ps] : -1;
    };
    const int32_t page0 = page_of(0);
    int32_t next = page_of(1);

    // queries, as they lie in memory: operand c of lane (g, n), eight elements of head 16 f + n (zero past
    // the live heads and past D)
    constexpr int QL = QF ? 2 : 1;            // 16-byte loads
    uint4 qraw[QT][KC][QL];
#pragma unroll
    for (int f = 0; f < QT; ++f)
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        // the int8 cache reads 16 elements per lane, so its steps come in pairs of adjacent eights
        const int d = I8 ? 64 * (c / 2) + 16 * g + 8 * (c & 1) : 32 * c + 8 * g;
        const int h = kQ * f + n;
        const char* p = (const char*)a.q + (sq * a.q_tok + (int64_t)(hq0 + h) * a.q_head + d) * (QF ? 4 : 2);
#pragma unroll
        for (int e = 0; e < QL; ++e)
          qraw[f][c][e] = h < rows && d < D ? ((const uint4*)p)[e] : make_uint4(0, 0, 0, 0);
      }

    // scales of the lane's key and value, on their way to LDS, and whether the key is live
    float scl[2] = {0.f, 0.f};
    bool scl_ok = false;
    auto put_rows = [&](int grpi, int32_t page) {
      const int64_t t = key_of(grpi);
      const int off = (int)((uint32_t)t % (uint32_t)ps);
      const bool ok = page >= 0 && page < a.kv.pages;   // a hole in the table is a masked run of keys
      ring[wave][grpi & 1][lane & (GK - 1)] =
          ok ? ((int64_t)page * a.kv.page_stride + (int64_t)off * a.kv.tok_stride) * EB : -1;
      if constexpr (I8) {
        const int64_t sr = ok ? ((int64_t)page * a.kv.heads + hk) * ps + off : 0;
        scl[0] = a.kv.k_scale[sr];
        scl[1] = a.kv.v_scale[sr];
        scl_ok = ok;
      }
      // LDS serves a wave's accesses in order; only the compiler has to keep them so
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    };

    // A lane whose elements lie past D reads the row's first ones instead: its key elements are
    // cleared before use, its value elements reach only outputs past D.  A masked key reads row 0.
    uint32_t kr[KG][2][KW], vr[KG][8][VW];
    int live[KG];                             // which of the lane's eight keys of a run are live
    auto load_k = [&](int grpi) {
#pragma unroll
      for (int u = 0; u < KG; ++u)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int64_t r = max((int64_t)0, ring[wave][grpi & 1][32 * u + 16 * t + n]);
#pragma unroll
          for (int c = 0; c < KW / 4; ++c) {
            const int d = I8 ? 64 * c + 16 * g : 32 * c + 8 * g;
            load_dw<4>(kbase + r + (d < D ? d : 0) * EB, &kr[u][t][4 * c]);
          }
        }
    };
    auto clear_k = [&](int u) {
      if (D == DT) return;
#pragma unroll
      for (int c = 0; c < KW / 4; ++c) {
        const bool in = (I8 ? 64 * c + 16 * g : 32 * c + 8 * g) < D;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int t = 0; t < 2; ++t) kr[u][t][4 * c + j] = in ? kr[u][t][4 * c + j] : 0u;
      }
    };
    auto load_v = [&](int grpi) {
#pragma unroll
      for (int u = 0; u < KG; ++u) {
        live[u] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int64_t raw = ring[wave][grpi & 1][32 * u + 16 * (i / 4) + 4 * g + (i & 3)];
          const int64_t r = max((int64_t)0, raw);
          live[u] |= (raw >= 0 ? 1 : 0) << i;
#pragma unroll
          for (int c = 0; c < VL; ++c) {
            const int d = VE * n + (VE / VL) * c;
            load_dw<VW / VL>(vbase + r + (d < D ? d : 0) * EB, &vr[u][i][VW / VL * c]);
          }
        }
      }
    };

    v4f o[QT][VE];
    float m[QT], l[QT];
    auto clear_sums = [&]() {
#pragma unroll
      for (int f = 0; f < QT; ++f) {
        m[f] = -INFINITY;
        l[f] = 0.f;
#pragma unroll
        for (int j = 0; j < VE; ++j) o[f][j] = v4f{0.f, 0.f, 0.f, 0.f};
      }
    };
    clear_sums();

    if (groups > 0) {
      put_rows(0, page0);
      load_k(0);
      load_v(0);
    }
    // the queries as bf16 terms, each what the ones before leave
    bf16x8 qf[QT][QS][KC];
#pragma unroll
    for (int f = 0; f < QT; ++f)
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        if constexpr (QF) {
          float v[8];
          const uint4 lo = qraw[f][c][0], hi = qraw[f][c][1];
          const uint32_t bits[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(bits[j]);
          // cut off, not rounded: a rounding makes the largest infinite (a canonical NaN survives the cut)
#pragma unroll
          for (int t = 0; t < QS; ++t) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float x = t ? v[2 * j] : __builtin_canonicalizef(v[2 * j]);
              const float y = t ? v[2 * j + 1] : __builtin_canonicalizef(v[2 * j + 1]);
              w[j] = upper_halves(__float_as_uint(x), __float_as_uint(y));
              v[2 * j] -= bf16_lo(w[j]);
              v[2 * j + 1] -= bf16_hi(w[j]);
            }
            qf[f][t][c] = frag(w[0], w[1], w[2], w[3]);
          }
        } else {
          qf[f][0][c] = __builtin_bit_cast(bf16x8, qraw[f][c][0]);
        }
      }
    // An infinite value times a term of its weight that is zero would be NaN.  A wave whose sums hold a NaN
    // takes its keys again with the leading term in the place of all three: that is infinite, or NaN, where
    // the formula is, and stands for the NaNs alone.  Looking for them costs 0 to 1 us of a launch.
    uint32_t taken = 0xFFFF0000u;             // of a weight's bits, what a term takes from those after it
    for (;;) {
      for (int i = 0; i < groups; ++i) {
        const bool more = i + 1 < groups;
        if constexpr (I8) {
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
          sring[wave][0][lane & (GK - 1)] = scl[0];
          sring[wave][1][lane & (GK - 1)] = scl_ok ? scl[1] : 0.f;   // times a masked weight of 0
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
          __builtin_amdgcn_wave_barrier();
        }
        // scores
        float x[QT][KG][8];
        bool full = true;
#pragma unroll
        for (int u = 0; u < KG; ++u) {
          clear_k(u);
          full = full && __all(live[u] == 0xFF);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            v4f s[QT], rest[QT];
#pragma unroll
            for (int f = 0; f < QT; ++f) s[f] = rest[f] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < KC; ++c) {
              bf16x8 kf;
              if constexpr (I8) {
                uint32_t w[4];
                i8x4_bf16(kr[u][t][2 * c], w[0], w[1]);
                i8x4_bf16(kr[u][t][2 * c + 1], w[2], w[3]);
                kf = frag(w[0], w[1], w[2], w[3]);
              } else {
                kf = frag(kr[u][t][4 * c], kr[u][t][4 * c + 1], kr[u][t][4 * c + 2], kr[u][t][4 * c + 3]);
              }
#pragma unroll
              for (int f = 0; f < QT; ++f) {
                s[f] = mfma_bf16(kf, qf[f][0][c], s[f]);
#pragma unroll
                for (int e = 1; e < QS; ++e) rest[f] = mfma_bf16(kf, qf[f][e][c], rest[f]);
              }
            }
#pragma unroll
            for (int f = 0; f < QT; ++f)
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                float v = s[f][r];
                // an infinite key times a query's zero or negative remainder would spoil its score
                if constexpr (QF) v = __builtin_isfinite(v) ? v + rest[f][r] : v;
                x[f][u][4 * t + r] = v * a.scale_log2;
              }
          }
        }
        if (more) {
          put_rows(i + 1, next);
          load_k(i + 1);
          next = page_of(i + 2);
        }
        float mx[QT];
        bool rise = false;
#pragma unroll
        for (int f = 0; f < QT; ++f) {
          mx[f] = -INFINITY;
#pragma unroll
          for (int u = 0; u < KG; ++u)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              float& v = x[f][u][k];
              if constexpr (I8) v *= sring[wave][0][32 * u + 16 * (k / 4) + 4 * g + (k & 3)];
              if (!full && !((live[u] >> k) & 1)) v = -INFINITY;
              mx[f] = fmaxf(mx[f], v);
            }
          rise = rise || mx[f] > m[f];
        }
        if (__any(rise)) {                    // a new maximum: shared by the four lanes of a query
#pragma unroll
          for (int f = 0; f < QT; ++f) {
            float top = fmaxf(mx[f], __shfl_xor(mx[f], 16, 64));
            top = fmaxf(m[f], fmaxf(top, __shfl_xor(top, 32, 64)));
            const float fall = m[f] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m[f] - top);
            m[f] = top;
            l[f] *= fall;
#pragma unroll
            for (int j = 0; j < VE; ++j) o[f][j] *= fall;
          }
        }
#pragma unroll
        for (int u = 0; u < KG; ++u) {
          bf16x8 pf[QT][PS];
#pragma unroll
          for (int f = 0; f < QT; ++f) {
            const float base = m[f] == -INFINITY ? 0.f : m[f];
            uint32_t pw[PS][4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float p0 = __builtin_amdgcn_exp2f(x[f][u][2 * k] - base);
              float p1 = __builtin_amdgcn_exp2f(x[f][u][2 * k + 1] - base);
              l[f] += p0 + p1;
              if constexpr (I8) {
                const float* vs = &sring[wave][1][32 * u + 16 * (k / 2) + 4 * g + (2 * k & 3)];
                p0 *= vs[0];
                p1 *= vs[1];
              }
#pragma unroll
              for (int e = 0; e < PS; ++e) {    // by truncation: the terms have the weight's sign
                const uint32_t b0 = __float_as_uint(p0), b1 = __float_as_uint(p1);
                pw[e][k] = upper_halves(b0, b1);
                p0 -= __uint_as_float(b0 & taken);
                p1 -= __uint_as_float(b1 & taken);
              }
            }
#pragma unroll
            for (int e = 0; e < PS; ++e) pf[f][e] = frag(pw[e][0], pw[e][1], pw[e][2], pw[e][3]);
          }
          if (!full) {                        // a masked row may hold anything: 0 * NaN is not 0
#pragma unroll
            for (int k = 0; k < 8; ++k)
#pragma unroll
              for (int w = 0; w < VW; ++w) vr[u][k][w] = (live[u] >> k) & 1 ? vr[u][k][w] : 0u;
          }
#pragma unroll
          for (int j = 0; j < VE; ++j) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t* v0 = vr[u][2 * k];
              const uint32_t* v1 = vr[u][2 * k + 1];
              if constexpr (I8) w[k] = upper_halves(i8_f32(v0[j / 4], j & 3), i8_f32(v1[j / 4], j & 3));
              else w[k] = __builtin_amdgcn_perm(v1[j / 2], v0[j / 2], j & 1 ? 0x07060302u : 0x05040100u);
            }
            const bf16x8 vf = frag(w[0], w[1], w[2], w[3]);
#pragma unroll
            for (int f = 0; f < QT; ++f)
#pragma unroll
              for (int e = 0; e < PS; ++e) o[f][j] = mfma_bf16(vf, pf[f][e], o[f][j]);
          }
        }
        if (more) load_v(i + 1);
      }
      // the wave's sums, to be joined.  Lane (g, n) holds elements VE (4g + r) + j of head 16 f + n.
      const int wl = here(threadIdx.x) & 63, wn = wl & 15;
      auto place = [&](int f, int r, int j) -> float& {
        return sm_o[wave][kQ * f + wn][VE * (4 * (wl >> 4) + r) + j];
      };
      if (__builtin_expect(!taken, 0)) {      // only the NaNs of the first time give way
#pragma unroll
        for (int f = 0; f < QT; ++f)
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int j = 0; j < VE; ++j) {
              const float v = place(f, r, j);
              o[f][j][r] = v == v ? v : o[f][j][r];
            }
      }
      v4f all = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int f = 0; f < QT; ++f) {
        l[f] += __shfl_xor(l[f], 16, 64);
        l[f] += __shfl_xor(l[f], 32, 64);
#pragma unroll
        for (int j = 0; j < VE; ++j) all += o[f][j];
        const int h = kQ * f + wn;
        if (h >= rows) continue;
        if (wl < kQ) { sm_m[wave][h] = m[f]; sm_l[wave][h] = l[f]; }
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int j = 0; j < VE; ++j) place(f, r, j) = o[f][j][r];
      }
      const float sum = (all[0] + all[1]) + (all[2] + all[3]);   // NaN if any of them is
      if (__builtin_expect(!taken || !__any(sum != sum), 1)) break;
      taken = 0u;
      clear_sums();
      put_rows(0, page_of(0));
      load_k(0);
      load_v(0);
      next = page_of(1);
    }
    const int tid = here(threadIdx.x), tl = tid & 63, tw = tid >> 6;
    __syncthreads();
    const int64_t orow = (sq * a.Hq + hq0) * (int64_t)D;
    auto finish = [&](int h, int d, float num, float den, float top) {
      const float v = den > 0.f ? num / den : 0.f;   // NaN sums fall to 0 / 0 below
      const float r = den == den ? v : num;
      if constexpr (QF) ((float*)a.out)[orow + (int64_t)h * D + d] = r;
      else ((uint16_t*)a.out)[orow + (int64_t)h * D + d] = (uint16_t)pack_bf16(r, 0.f);
      if (d == 0 && a.lse)
        a.lse[sq * a.Hq + hq0 + h] = den > 0.f ? (top + log2f(den)) * kLn2 : den == den ? -INFINITY : den;
    };
    // a block's partial sums: place 0 for a group that an earlier block began, 1 for one it begins
    const int64_t place = 2 * (int64_t)blockIdx.x + (owner0 == (int64_t)blockIdx.x);
    float* part = a.part + place * prows * D;   // [prows][D]
    float* ml = a.ml + place * 2 * R;           // [2][R]
    for (int e = tid; e < rows * D; e += 64 * kWaves) {
      const int h = e / D, d = e - h * D;
      float top = sm_m[0][h];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) top = fmaxf(top, sm_m[w][h]);
      float num = 0.f, den = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float f = weight(sm_m[w][h], sm_l[w][h], top);
        num += f * sm_o[w][h][d];
        den += f * sm_l[w][h];
      }
      if (active == 1) {
        finish(h, d, num, den, top);
      } else {
        put(part + h * D + d, num);
        if (d == 0) { put(ml + h, top); put(ml + R + h, den); }
      }
    }
    if (active > 1) {
      // The last block of the group to arrive joins the runs.  Partial sums are stored and read by
      // device-scope atomic accesses, which pass by the caches that the XCDs do not share, and every
      // wave waits for its stores before the block counts as arrived; the block that arrives last
      // reads after that.  That is the order of a device-scope release and acquire, without their
      // write-back and invalidation of the XCD's L2 (10 us per block for the one, up to 8 us for the
      // other while the rest of the chip streams).  Arrivals are counted at the block that begins the
      // group: a block begins at most one group that goes on in the next, so no two share a count.
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
      __builtin_amdgcn_s_waitcnt(waitcnt_imm(0));
      __syncthreads();
      if (tid == 0) {
        last_sh = __hip_atomic_fetch_add(a.ticket + owner0, 1u, __ATOMIC_RELAXED,
                                         __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)active - 1;
        if (last_sh)                            // ready for the next launch
          __hip_atomic_store(a.ticket + owner0, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      __syncthreads();
      if (last_sh) {
        // The weights of the runs in LDS (sm_o is free), as many runs at a time as fit; then runs
        // s = w, w + 4, ... to wave w, a lane two fours of 512 columns, the waves' sums joined in
        // order.  The first runs' sums, maxima and columns are all asked for before any is used: a
        // round trip to memory is most of what a join of few runs costs.
        constexpr int kCols = 512;
        constexpr int kRoom = kWaves * R * (DT + 4) - kWaves * kCols;
        float* wt = &sm_o[0][0][0];               // [rows][at]
        float* sums = wt + kRoom;                 // [kWaves][kCols]
        const int at = kRoom / rows;
        const int cols = rows * D;
        auto run = [&](int s) { return 2 * (owner0 + s) + (s == 0); };
        auto column = [&](int s, int e) {
          return e < cols ? get4(a.part + run(s) * prows * D + e) : v4f{0.f, 0.f, 0.f, 0.f};
        };
        // thread (i, row): runs i, i + kSlots, ... of a row, the first kHeld of them in registers
        constexpr int kHeld = 4, kAhead = 4, kSlots = 64 * kWaves / R;
        const int hrow = tid & (R - 1), i0 = tid / R;
        float hm[kHeld], hl[kHeld];
#pragma unroll
        for (int k = 0; k < kHeld; ++k) {
          const int s = i0 + kSlots * k;
          const bool in = hrow < rows && s < active;
          const float* p = a.ml + run(in ? s : 0) * 2 * R + hrow;
          hm[k] = in ? get(p) : -INFINITY;
          hl[k] = in ? get(p + R) : 0.f;
        }
        v4f ahead[kAhead][2];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int s = min(tw + kWaves * k, active - 1);
          ahead[k][0] = column(s, 4 * tl);
          ahead[k][1] = column(s, 256 + 4 * tl);
        }
        float top = -INFINITY, den = 0.f;
#pragma unroll
        for (int k = 0; k < kHeld; ++k) top = fmaxf(top, hm[k]);
        if (hrow < rows)
          for (int s = i0 + kSlots * kHeld; s < active; s += kSlots)
            top = fmaxf(top, get(a.ml + run(s) * 2 * R + hrow));
        auto over_rows = [&](float v, auto op) {  // of the kSlots threads of each row
          if constexpr (QT == 1) v = op(v, __shfl_xor(v, 16, 64));
          v = op(v, __shfl_xor(v, 32, 64));
          __syncthreads();
          if (tl < R) sums[R * tw + tl] = v;
          __syncthreads();
#pragma unroll
          for (int w = 0; w < kWaves; ++w) v = w ? op(v, sums[R * w + hrow]) : sums[hrow];
          return v;
        };
        top = over_rows(top, [](float x, float y) { return fmaxf(x, y); });
#pragma unroll 1
        for (int j = 0; j < cols; j += kCols) {
          const int e = j + 4 * tl;
          const int h0 = min(e / D, rows - 1), h1 = min((e + 256) / D, rows - 1);   // D % 8 == 0: one row per four
          v4f num[2] = {v4f{0.f, 0.f, 0.f, 0.f}, v4f{0.f, 0.f, 0.f, 0.f}};
#pragma unroll 1
          for (int s0 = 0; s0 < active; s0 += at) {
            const int ns = min(at, active - s0);
            if (j == 0 || active > at) {
              __syncthreads();
              if (hrow < rows) {
                auto put_weight = [&](int s, float pm, float pl) {
                  const float f = weight(pm, pl, top);
                  wt[hrow * at + s] = f;
                  if (j == 0) den += f * pl;
                };
                int s = i0;
                if (s0 == 0) {
#pragma unroll
                  for (int k = 0; k < kHeld; ++k, s += kSlots)
                    if (s < ns) put_weight(s, hm[k], hl[k]);
                }
                for (; s < ns; s += kSlots) {
                  const float* p = a.ml + run(s0 + s) * 2 * R + hrow;
                  put_weight(s, get(p), get(p + R));
                }
              }
              __syncthreads();
            }
            const float* w0r = wt + h0 * at;
            const float* w1r = wt + h1 * at;
            int s = tw;
            if (j == 0 && s0 == 0) {
#pragma unroll
              for (int k = 0; k < kAhead; ++k, s += kWaves)
                if (s < ns) { num[0] += w0r[s] * ahead[k][0]; num[1] += w1r[s] * ahead[k][1]; }
            }
#pragma unroll 4
            for (; s < ns; s += kWaves) {
              const v4f v0 = column(s0 + s, e), v1 = column(s0 + s, e + 256);
              num[0] += w0r[s] * v0;
              num[1] += w1r[s] * v1;
            }
          }
          if (j == 0) {
            den = over_rows(den, [](float x, float y) { return x + y; });
            if (tid < R) { sm_l[0][hrow] = den; sm_m[0][hrow] = top; }
            __syncthreads();                      // sums is free again
          }
          *(v4f*)(sums + kCols * tw + 4 * tl) = num[0];
          *(v4f*)(sums + kCols * tw + 256 + 4 * tl) = num[1];
          __syncthreads();
#pragma unroll
          for (int u = 0; u < kCols; u += 64 * kWaves) {
            const int c = j + u + tid;
            if (c < cols) {
              const int h = c / D;
              float nsum = 0.f;
#pragma unroll
              for (int w = 0; w < kWaves; ++w) nsum += sums[kCols * w + u + tid];
              finish(h, c - h * D, nsum, sm_l[0][h], sm_m[0][h]);
            }
          }
          __syncthreads();
        }
      }
    }
    __syncthreads();                          // the next segment reuses the LDS
  }
}

template <int DT, int QT>
hipError_t launch_attn_t(const AttnArgs& a, bool q_bf16, hipStream_t s) {
  const dim3 grid((unsigned)a.nblocks), block(64 * kWaves);
  const bool i8 = a.kv.dtype == BL_DTYPE_I8;
  if (q_bf16) {
    if (i8) paged_attn_kernel<DT, true, false, QT><<<grid, block, 0, s>>>(a);
    else paged_attn_kernel<DT, false, false, QT><<<grid, block, 0, s>>>(a);
  } else {
    if (i8) paged_attn_kernel<DT, true, true, QT><<<grid, block, 0, s>>>(a);
    else paged_attn_kernel<DT, false, true, QT><<<grid, block, 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace

// A block takes two query tiles where a key head has more than 16 query heads: its keys and values are
// then read once for 32 of them (D > 128 has no registers for it).  It also doubles what is joined, by
// half the blocks, so a small batch of few groups stays at one tile.  24 query heads over one key head,
// one tile against two, us at head dimensions 64 and 128: 64 sequences of 64000 tokens 299 : 209 and
// 590 : 388, 64 of 4000 33 : 30 and 56 : 49, 16 of 16000 28 : 35 and 50 : 50, 64 of 1000 19 : 23 and 29 : 29,
// 2 of 64000 44 : 94 and 60 : 83.
void paged_attn_split(bl_attn_plan& p) {
  const int64_t G = p.q_heads / p.kv_heads, D = p.head_dim;
  const int64_t keys = p.window ? std::min<int64_t>(p.window, p.max_len) : p.max_len;
  const int64_t tiles = (keys + kTile - 1) / kTile, pairs = p.B * p.kv_heads;
  const int64_t many = std::min<int64_t>(pairs, 256);
  const bool two = G > kQ && D <= 128 && pairs * tiles >= 1024 && many * many * tiles >= 1 << 16;
  p.q_rows = two ? 2 * kQ : kQ;
  // a block per resident place of the chip, fewer where there is less work: tiles of keys, and the
  // start of a group as so many more (at most six: start_units)
  const int64_t groups = pairs * ((G + p.q_rows - 1) / p.q_rows);
  const int64_t places = kAttnBlocks / 2 * resident(D <= 64 ? 64 : D <= 128 ? 128 : 256, two ? 2 : 1);
  p.blocks = (int32_t)std::max<int64_t>(1, std::min(places, groups * (tiles + 6)));
}

hipError_t launch_paged_attn(const AttnArgs& a, bool q_bf16, hipStream_t s) {
  const int D = a.kv.head_dim;
  if (a.q_rows == 2 * kQ)
    return D <= 64 ? launch_attn_t<64, 2>(a, q_bf16, s) : launch_attn_t<128, 2>(a, q_bf16, s);
  if (D <= 64) return launch_attn_t<64, 1>(a, q_bf16, s);
  if (D <= 128) return launch_attn_t<128, 1>(a, q_bf16, s);
  return launch_attn_t<256, 1>(a, q_bf16, s);
}

}  // namespace bl
