// Products of int8 rows with weights in 4 bits, a bf16 scale for each group of 32, 64 or 128 columns of a
// row, and the packing of such weights.
//
//   y[t][o] = x_scale[t] * sum over groups g of s[o][g] * (sum over k in g of q[o][k] * xq[t][k])
//
// A group's inner sum is an int32 sum of one or two int8 MFMAs, exact; groups are joined in fp32.  The MFMA
// takes 16 weight rows and 16 tokens.  A nibble becomes int8 by moving it into the upper half of its byte,
// which is 16 times its value: one shift and two masks for eight weights, and the 16 leaves where the sum is read as a
// float.
//
// Few tokens: a wave takes a tile of 16 rows and all tokens, whose rows lie in LDS, as many columns at a time as fit.
// More: a block's waves share two LDS buffers of the tokens' rows, NT tiles of 16.  KS waves of a block share a tile's
// columns when the rows alone are too few waves, and add up their sums in LDS in a fixed order.  Codes are laid out as
// the instruction takes them: one 16-byte load per lane is 16 rows x 128 columns (the layout is in bitlinear.h).
//
// Bound by memory for few tokens: half a byte per weight and 2 / group of scales, read once, as long as one block holds
// all tokens (64).  131072 x 2560 in groups of 64, 179 MB, one token 30 us (6 TB/s); 16 tokens of 100003 x 4096 in groups of
// 128 43 us (5.1 TB/s); 64 tokens of the first 60 us: there the vector units are busy half of the time with the sums of a
// group (a subtraction and a multiply-add each), and a barrier per buffer keeps the waves from filling the other half.
// Above 64 tokens, blocks of 64 each read and unpack the weights again: 128, 512 and 2048 tokens of the first 113, 394 and
// 1700 us (760 to 870 T operations/s).
#include <algorithm>

#include "block_ops.hpp"
#include "device_common.hpp"
#include "step_ops.hpp"

namespace bl {

namespace {

constexpr int kWaves = 8;
constexpr int kAhead = 4;            // 128-column blocks asked for at a time
constexpr int kLds = 40 * 1024;      // four blocks per CU

// ---------------------------------------------------------------------------------------------
// packing
// ---------------------------------------------------------------------------------------------

// A wave takes a tile of 16 rows by 128 columns, a lane the columns of its 16 bytes of codes; the four lanes of a row
// join its groups' largest magnitudes.  Bound by memory: 131072 x 2560 fp32 in groups of 64, 1.52 GB, 332 us (4.6 TB/s; 368
// with four bytes of codes to a lane, whose lines were written 2.3 times).
template <bool BF, int G>
__global__ __launch_bounds__(256) void q4_pack_kernel(Q4PackArgs a) {
  constexpr int NG = 128 / G;
  const int lane = threadIdx.x & 63, q = lane >> 4, r = lane & 15;
  const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (unit >= a.tiles * a.blocks) return;
  const int64_t row = unit / a.blocks * 16 + r, col = unit % a.blocks * 128;
  float v[4][8] = {};
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const int64_t c = col + (G == 32 ? 32 * w + 8 * q : 64 * (w >> 1) + 16 * q + 8 * (w & 1));
    if (row < a.n && c < a.K) load_f8<BF>(a.W, (size_t)row * a.K + c, v[w]);
  }
  uint32_t top[NG] = {};                                   // of magnitudes; NaN above infinity above all else
#pragma unroll
  for (int w = 0; w < 4; ++w)
#pragma unroll
    for (int i = 0; i < 8; ++i) top[w * NG / 4] = max(top[w * NG / 4], __float_as_uint(v[w][i]) & 0x7FFFFFFFu);
  uint16_t scale[NG];
  v4i codes;
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    top[g] = max(top[g], (uint32_t)__shfl_xor((int)top[g], 16, 64));
    top[g] = max(top[g], (uint32_t)__shfl_xor((int)top[g], 32, 64));
    const bool finite = top[g] < 0x7F800000u;
    const __bf16 sb = finite ? (__bf16)(__uint_as_float(top[g]) / 7.0f) : __builtin_bit_cast(__bf16, (uint16_t)0x7FC0);
    const float s = (float)sb;
    scale[g] = __builtin_bit_cast(uint16_t, sb);
#pragma unroll
    for (int w = g * 4 / NG; w < (g + 1) * 4 / NG; ++w) {
      uint32_t word = 0;
      if (finite && s > 0.f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x = fminf(fmaxf(rintf(v[w][i] / s), -7.f), 7.f);
          word |= ((uint32_t)(int)x & 15u) << (8 * (i & 3) + 4 * (i >> 2));
        }
      }
      codes[w] = (int)word;
    }
  }
  ((v4i*)a.codes)[unit * 64 + lane] = codes;
#pragma unroll
  for (int g = 0; g < NG; ++g)
    if (q == g) a.scales[(unit * 4 + (r >> 2)) * (NG * 4) + g * 4 + (r & 3)] = scale[g];
}

// ---------------------------------------------------------------------------------------------
// product
// ---------------------------------------------------------------------------------------------

typedef int v2i __attribute__((ext_vector_type(2)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

// The MFMA's sums start from the bits of 1.5 * 2^19, a float whose last bit is 1 / 16: what comes out, 16 times the group's
// sum and below 2^22, read as a float is that number plus the sum itself, and a subtraction takes the place of a conversion.
// No factor of 16 is left to overflow in the joined sums or to cost the smallest scales of tokens their bits.
constexpr float kBias = 786432.f;
constexpr int kBiasBits = 0x49400000;

// Four rows' sums of a token, from row o on.
__device__ __forceinline__ void put_rows(const Q4Args& a, int t, int64_t o, const float sum[4]) {
  if (o >= a.n) return;
  const float s = a.x_scale[t];
  float* y = a.y + (size_t)t * a.n + o;
  if (a.n % 4 == 0) {
    *(float4*)y = make_float4(sum[0] * s, sum[1] * s, sum[2] * s, sum[3] * s);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (o + e < a.n) y[e] = sum[e] * s;
  }
}

// A few tokens (16 would fit, fwd() sends four at most): few registers and little LDS, so that many waves are there to wait for memory.
template <int G>
__global__ __launch_bounds__(64 * kWaves) void q4_narrow_kernel(Q4Args a) {
  constexpr int NG = 128 / G;
  constexpr int U = G == 32 ? 32 : 64;                     // columns of one MFMA
  extern __shared__ __attribute__((aligned(16))) int8_t sm_x[];      // [chunk / U][tokens][U]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int q = lane >> 4, r = lane & 15;
  const int tokens = a.T;
  const int ks = a.ksplit, part = wave % ks;
  const int64_t tile = (int64_t)blockIdx.x * (kWaves / ks) + wave / ks;
  const bool busy = tile < a.tiles;
  const int64_t from = min(tile, a.tiles - 1);
  const v4i* codes = (const v4i*)a.codes + from * a.blocks * 64 + lane;
  const v2u* scales = (const v2u*)a.scales + (from * a.blocks * 4 + q) * NG;
  const int8_t* x = sm_x + min(r, tokens - 1) * U + U / 4 * q;       // a spare token repeats the last one

  const v4i bias = {kBiasBits, kBiasBits, kBiasBits, kBiasBits};
  float sum[4] = {};
  for (int c0 = 0; c0 < a.blocks; c0 += a.chunk / 128) {   // blocks whose columns are in LDS
    const int cn = min(a.chunk / 128, a.blocks - c0);
    if (c0) __syncthreads();
    {
      const int cols = min(cn * 128, a.K - c0 * 128);      // what is past K meets codes of zero
      const int per = cols / 16;                           // K % 32 == 0
      for (int i = threadIdx.x; i < tokens * per; i += 64 * kWaves) {
        const int t = i / per, c = (i - t * per) * 16;
        *(v4i*)(sm_x + ((c / U) * tokens + t) * U + c % U) = *(const v4i*)(a.xq + (size_t)t * a.K + c0 * 128 + c);
      }
    }
    __syncthreads();
    if (!busy) continue;
    for (int b0 = part; b0 < cn; b0 += ks * kAhead) {
      v4i code[kAhead];
      v2u scale[kAhead][NG];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int64_t b = c0 + min(b0 + u * ks, cn - 1);
        code[u] = __builtin_nontemporal_load(codes + b * 64);
#pragma unroll
        for (int g = 0; g < NG; ++g) scale[u][g] = scales[b * 4 * NG + g];
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int b = b0 + u * ks;
        if (b >= cn) break;
        v4i av[2];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t d = (uint32_t)code[u][w];
          av[w >> 1][(w & 1) * 2] = (int)((d << 4) & 0xF0F0F0F0u);
          av[w >> 1][(w & 1) * 2 + 1] = (int)(d & 0xF0F0F0F0u);
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const int8_t* p = x + (b * 128 + g * G) * tokens;
          v4i acc;
          if constexpr (G == 32) {
            const v2i half = {av[g >> 1][(g & 1) * 2], av[g >> 1][(g & 1) * 2 + 1]};
            acc = __builtin_amdgcn_mfma_i32_16x16x32_i8(__builtin_bit_cast(long, half),
                                                        __builtin_bit_cast(long, *(const v2i*)p), bias, 0, 0, 0);
          } else if constexpr (G == 64) {
            acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(av[g], *(const v4i*)p, bias, 0, 0, 0);
          } else {
            acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(av[0], *(const v4i*)p, bias, 0, 0, 0);
            acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(av[1], *(const v4i*)(p + 64 * tokens), acc, 0, 0, 0);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t s = scale[u][g][e >> 1];
            sum[e] = __builtin_fmaf(__int_as_float(acc[e]) - kBias, (e & 1) ? bf16_hi(s) : bf16_lo(s), sum[e]);
          }
        }
      }
    }
  }

  if (ks > 1) {                                            // parts of a tile, joined by its first wave in order
    float* red = (float*)sm_x;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 4; ++e) red[wave * 256 + e * 64 + lane] = sum[e];
    __syncthreads();
    if (part) return;
    for (int p = 1; p < ks; ++p)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] += red[(wave + p) * 256 + e * 64 + lane];
  }
  if (busy && r < tokens) put_rows(a, r, tile * 16 + 4 * q, sum);
}

// More tokens: the same product with the tokens' rows in two LDS buffers of W blocks of 128 columns.  While a
// buffer is multiplied, the next one is filled past the registers and the next weights are on their way; one barrier
// and one wait per buffer.  KS waves share a tile's columns, W / KS blocks of a buffer each.
template <int G, int NT, int KS, int W>
__global__ __launch_bounds__(64 * kWaves, W <= 4 ? 4 : 2) void q4_wide_kernel(Q4Args a) {
  constexpr int NG = 128 / G, A = W / KS;
  constexpr int U = G == 32 ? 32 : 64;
  constexpr int kBuffer = 16 * NT * W * 128;
  __shared__ __attribute__((aligned(16))) int8_t sm[2][kBuffer];     // [columns / U][tokens][U]
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int q = lane >> 4, r = lane & 15;
  const int tt = a.token_tiles;
  const int64_t id = blockIdx.x;
  const int64_t rows_at = id / (8 * tt) * 8 + id % 8;
  const int token0 = (int)(id / 8 % tt) * 16 * NT;
  const int tokens = min(a.T - token0, 16 * NT);
  const int part = wave % KS;
  const int64_t tile = rows_at * (kWaves / KS) + wave / KS;
  if (rows_at * (kWaves / KS) >= a.tiles) return;          // a padding block: all of it
  const int64_t from = min(tile, a.tiles - 1);             // a spare wave repeats the last tile, stores nothing
  const v4i* codes = (const v4i*)a.codes + from * a.blocks * 64 + lane;
  const v2u* scales = (const v2u*)a.scales + (from * a.blocks * 4 + q) * NG;

  // Sixteen bytes per lane and turn, in the order in which they lie in LDS; where the tokens are fewer than the
  // buffer's, or the columns past K (which meet codes of zero), some are read twice.
  constexpr int kTurns = kBuffer / (16 * 64 * kWaves);
  auto fill = [&](int c0, int8_t* to) {
#pragma unroll
    for (int k = 0; k < kTurns; ++k) {
      const int i = (k * kWaves + wave) * 64 + lane;
      const int at = i / (U / 16), step = at / (16 * NT), t = at % (16 * NT);
      const int c = c0 * 128 + step * U + i % (U / 16) * 16;
      lds_dma16(a.xq + (size_t)(token0 + min(t, tokens - 1)) * a.K + min(c, a.K - 16),
                lds_offset(to) + (uint32_t)__builtin_amdgcn_readfirstlane((k * kWaves + wave) * 1024));
    }
  };
  v4i code[A];
  v2u scale[A][NG];
  auto load = [&](int c0) {
#pragma unroll
    for (int u = 0; u < A; ++u) {
      const int64_t b = min(c0 + part + u * KS, a.blocks - 1);
      const uint32_t live = c0 + part + u * KS < a.blocks ? ~0u : 0u;   // past the last block: scales of 0
      code[u] = __builtin_nontemporal_load(codes + b * 64);
#pragma unroll
      for (int g = 0; g < NG; ++g) scale[u][g] = scales[b * 4 * NG + g] & live;
    }
  };

  const v4i bias = {kBiasBits, kBiasBits, kBiasBits, kBiasBits};
  float sum[NT][4] = {};
  fill(0, sm[0]);
  load(0);
  for (int c0 = 0, turn = 0; c0 < a.blocks; c0 += W, turn ^= 1) {
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(0));            // this buffer and its weights
    v4i now[A];
    v2u now_scale[A][NG];
#pragma unroll
    for (int u = 0; u < A; ++u) {
      now[u] = code[u];
#pragma unroll
      for (int g = 0; g < NG; ++g) now_scale[u][g] = scale[u][g];
    }
    block_barrier_nofence();                               // and the other buffer has been read
    if (c0 + W < a.blocks) {
      fill(c0 + W, sm[turn ^ 1]);
      load(c0 + W);
    }
    const int8_t* x = sm[turn] + r * U + U / 4 * q;
#pragma unroll
    for (int u = 0; u < A; ++u) {
      const int8_t* xb = x + (part + u * KS) * 128 * 16 * NT;
      v4i av[2];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t d = (uint32_t)now[u][w];
        av[w >> 1][(w & 1) * 2] = (int)((d << 4) & 0xF0F0F0F0u);
        av[w >> 1][(w & 1) * 2 + 1] = (int)(d & 0xF0F0F0F0u);
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float sv[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sv[e] = (e & 1) ? bf16_hi(now_scale[u][g][e >> 1]) : bf16_lo(now_scale[u][g][e >> 1]);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int8_t* p = xb + (g * G * NT + j * U) * 16;
          v4i acc;
          if constexpr (G == 32) {
            const v2i half = {av[g >> 1][(g & 1) * 2], av[g >> 1][(g & 1) * 2 + 1]};
            acc = __builtin_amdgcn_mfma_i32_16x16x32_i8(__builtin_bit_cast(long, half),
                                                        __builtin_bit_cast(long, *(const v2i*)p), bias, 0, 0, 0);
          } else if constexpr (G == 64) {
            acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(av[g], *(const v4i*)p, bias, 0, 0, 0);
          } else {
            acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(av[0], *(const v4i*)p, bias, 0, 0, 0);
            acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(av[1], *(const v4i*)(p + 64 * 16 * NT), acc, 0, 0, 0);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[j][e] = __builtin_fmaf(__int_as_float(acc[e]) - kBias, sv[e], sum[j][e]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);                   // a block at a time: its weights unpacked are enough registers
    }
  }

  if constexpr (KS > 1) {                                  // parts of a tile, joined by its first wave in order
    float* red = (float*)sm;
    static_assert(sizeof(sm) >= kWaves * NT * 1024, "partial sums fit");
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) red[(wave * NT + j) * 256 + e * 64 + lane] = sum[j][e];
    __syncthreads();
    if (part) return;
    for (int p = 1; p < KS; ++p)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[j][e] += red[((wave + p) * NT + j) * 256 + e * 64 + lane];
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int t = 16 * j + r;
    if (t < tokens) put_rows(a, token0 + t, tile * 16 + 4 * q, sum[j]);
  }
}

template <int G, int NT, int KS, int W>
hipError_t wide(Q4Args a, hipStream_t s) {
  constexpr int per = kWaves / KS;
  const int64_t row_blocks = (a.tiles + per - 1) / per;
  const int64_t grid = (row_blocks + 7) / 8 * 8 * a.token_tiles;
  q4_wide_kernel<G, NT, KS, W><<<(unsigned)grid, 64 * kWaves, 0, s>>>(a);
  return hipGetLastError();
}

template <int G>
hipError_t narrow(Q4Args a, hipStream_t s) {
  // columns in LDS at a time: even parts of K
  const int most = kLds / a.T / 128 * 128;
  const int chunks = (a.blocks * 128 + most - 1) / most;
  a.chunk = (a.blocks + chunks - 1) / chunks * 128;
  // Waves on one tile's columns: as many as leave all waves there at once.  One token, by 1, 2, 4 and 8 waves to a tile:
  // 32000 x 2560 16.9, 11.9, 10.0 and 12.8 us, 16384 x 4096 -, 13.6, 9.9 and 9.0, 70001 x 2560 21.2 and 23.0.
  a.ksplit = 1;
  while (a.ksplit < kWaves && a.tiles * a.ksplit * 2 <= 8192 && a.ksplit * 2 <= a.chunk / 128) a.ksplit *= 2;
  const int64_t per = kWaves / a.ksplit;
  size_t lds = (size_t)a.T * a.chunk;
  if (a.ksplit > 1) lds = std::max(lds, (size_t)kWaves * 1024);
  q4_narrow_kernel<G><<<(unsigned)((a.tiles + per - 1) / per), 64 * kWaves, lds, s>>>(a);
  return hipGetLastError();
}

// How many waves share a tile's columns: a block's time is about 1 / KS of its columns, and there are KS times as many
// blocks.  The CU that gets the most of them is done last, one block alone is not faster than two, and each doubling costs
// a tenth or more, for the tokens' rows that each block reads.  16 tokens by 1, 2, 4 and 8 waves: 2560 x 6912 26.5, 17.4,
// 14.1 and 8.7 us, 32000 x 2560 13.9, 11.5, 12.1 and 15.3, 50000 x 2560 17.3, 19.0, 17.4 and 22.3, 100003 x 4096 47.5,
// 43.2, 47.8 and 57; 64 tokens: 2560 x 6912 37, 25, 19.5 and 15.8, 16384 x 4096 28.5, 20.1, 19.8 and 41, 131072 x 2560 64,
// 73, 103 and 223.  In groups of 32 one wave's sums and weights are more registers than there are.
template <int G, int NT>
hipError_t wide_split(Q4Args a, hipStream_t s) {
  a.token_tiles = (a.T + 16 * NT - 1) / (16 * NT);
  int ks = 0;
  double least = 0.0, tax = 1.0;
  for (int k = 1; k <= 8; k *= 2, tax *= NT == 1 ? 1.1 : 1.15) {
    if (ks && k > a.blocks) break;
    if (k == 1 && G == 32) continue;
    const int64_t blocks = (a.tiles * k + kWaves - 1) / kWaves * a.token_tiles;
    const double cost = (double)std::max<int64_t>((blocks + 255) / 256, 2) / k * tax;
    if (!ks || cost < least) {
      ks = k;
      least = cost;
    }
  }
  if constexpr (G > 32)
    if (ks == 1) return wide<G, NT, 1, 4>(a, s);
  if (ks == 2) return wide<G, NT, 2, 4>(a, s);
  if (ks == 4) return wide<G, NT, 4, 4>(a, s);
  return wide<G, NT, 8, 8>(a, s);
}

// Which kernel, in us: up to 4 tokens the narrow one (131072 x 2560, one token: 30.1, 33.0 by the other; 2560 x 6912 7.2
// and 8.6), above it the other (16 tokens of 100003 x 4096 48.1 and 43.2, 32000 x 2560 14.6 and 11.5), for as many tiles
// of 16 tokens as there are (32 of 131072 x 2560: 45 by two, 55 by four; 48: 53 by three, 59 by four).
template <int G>
hipError_t fwd(const Q4Args& a, hipStream_t s) {
  if (a.T <= 4) return narrow<G>(a, s);
  if (a.T <= 16) return wide_split<G, 1>(a, s);
  if (a.T <= 32) return wide_split<G, 2>(a, s);
  return a.T <= 48 ? wide_split<G, 3>(a, s) : wide_split<G, 4>(a, s);
}

}  // namespace

hipError_t launch_q4_pack(const Q4PackArgs& a, bool bf16, hipStream_t s) {
  const unsigned grid = (unsigned)((a.tiles * a.blocks + 3) / 4);
  auto go = [&](auto g) {
    constexpr int G = decltype(g)::value;
    if (bf16) q4_pack_kernel<true, G><<<grid, 256, 0, s>>>(a);
    else q4_pack_kernel<false, G><<<grid, 256, 0, s>>>(a);
  };
  if (a.group == 32) go(std::integral_constant<int, 32>{});
  else if (a.group == 64) go(std::integral_constant<int, 64>{});
  else go(std::integral_constant<int, 128>{});
  return hipGetLastError();
}

hipError_t launch_q4_fwd(const Q4Args& a, int group, hipStream_t s) {
  if (group == 32) return fwd<32>(a, s);
  if (group == 64) return fwd<64>(a, s);
  return fwd<128>(a, s);
}

}  // namespace bl
