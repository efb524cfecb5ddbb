// Products of int8 rows with weights in 4 bits, a bf16 scale for each group of 32, 64 or 128 columns of a
// row, and the packing of such weights.
//
//   y[t][o] = x_scale[t] * sum over groups g of s[o][g] * (sum over k in g of q[o][k] * xq[t][k])
//
// A group's inner sum is an int32 sum of one or two int8 MFMAs, exact; groups are joined in fp32.  The MFMA
// takes 16 weight rows and 16 tokens.  A nibble becomes int8 by moving it into the upper half of its byte,
// which is 16 times its value: one shift and two masks for eight weights, and the 16 leaves with the token's
// scale.
//
// A wave takes RT tiles of 16 rows and NT tiles of 16 tokens; KS waves of a block share a tile's columns when
// the rows alone are too few waves, and add up their sums in LDS in a fixed order.  The tokens' rows lie in LDS,
// as many columns at a time as fit.  Codes are laid out as the instruction takes them: one 16-byte load per lane
// is 16 rows x 128 columns (the layout is in bitlinear.h).
//
// Bound by memory: half a byte per weight and 2 / group of scales, read once, as long as one block holds all
// tokens (64).
#include <algorithm>

#include "block_ops.hpp"
#include "device_common.hpp"
#include "step_ops.hpp"

namespace bl {

namespace {

constexpr int kWaves = 8;
constexpr int kAhead = 4;            // 128-column blocks asked for at a time
constexpr int kLds = 78 * 1024;      // two blocks per CU

// ---------------------------------------------------------------------------------------------
// packing
// ---------------------------------------------------------------------------------------------

// A lane takes eight columns of a row; G / 8 neighbouring lanes hold a group.
template <bool BF, int G>
__global__ __launch_bounds__(256) void q4_pack_kernel(Q4PackArgs a) {
  const int64_t units = a.blocks * 16;                     // eights of columns of a row
  const int64_t u0 = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = u0 / units;
  const int u = (int)(u0 - row * units);
  if (row >= a.tiles * 16) return;                         // whole groups of lanes: 16 divides 256
  const int64_t col = (int64_t)u * 8;
  float v[8] = {};
  if (row < a.n && col < a.K) load_f8<BF>(a.W, (size_t)row * a.K + col, v);
  uint32_t top = 0;                                        // of magnitudes; NaN above infinity above all else
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
#pragma unroll
  for (int o = 1; o < G / 8; o <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o, 64));
  const bool finite = top < 0x7F800000u;
  const __bf16 sb = finite ? (__bf16)(__uint_as_float(top) / 7.0f) : __builtin_bit_cast(__bf16, (uint16_t)0x7FC0);
  const float s = (float)sb;
  uint32_t word = 0;
  if (finite && s > 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float r = fminf(fmaxf(rintf(v[i] / s), -7.f), 7.f);
      word |= ((uint32_t)(int)r & 15u) << (8 * (i & 3) + 4 * (i >> 2));
    }
  }
  const int64_t tile = row >> 4, r = row & 15, block = u >> 4;
  const int c = (u & 15) * 8;                              // within the block of 128
  const int w = G == 32 ? c >> 5 : ((c >> 6) << 1) | ((c >> 3) & 1);
  const int q = G == 32 ? (c >> 3) & 3 : (c >> 4) & 3;
  a.codes[((tile * a.blocks + block) * 64 + q * 16 + r) * 4 + w] = word;
  if ((c & (G - 1)) == 0)
    a.scales[((tile * a.blocks + block) * 4 + (r >> 2)) * (128 / G * 4) + c / G * 4 + (r & 3)] =
        __builtin_bit_cast(uint16_t, sb);
}

// ---------------------------------------------------------------------------------------------
// product
// ---------------------------------------------------------------------------------------------

template <int G>
struct Q4Scales {                                          // of a lane's four rows in a block
  uint32_t w[128 / G * 2];
};

template <int G, int NT, int RT>
__global__ __launch_bounds__(64 * kWaves) void q4_fwd_kernel(Q4Args a) {
  constexpr int NG = 128 / G;
  extern __shared__ __attribute__((aligned(16))) int8_t sm_x[];      // [tokens][chunk + 16]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int q = lane >> 4, r = lane & 15;
  // token tiles of the same rows run side by side on one XCD (workgroups are dealt round-robin)
  const int tt = a.token_tiles;
  const int64_t id = blockIdx.x;
  const int64_t rows_at = id / (8 * tt) * 8 + id % 8;
  const int token0 = (int)(id / 8 % tt) * 16 * NT;
  const int tokens = min(a.T - token0, 16 * NT);
  const int ks = a.ksplit, part = wave % ks;
  const int64_t tile0 = (rows_at * (kWaves / ks) + wave / ks) * RT;
  if (rows_at * (kWaves / ks) * RT >= a.tiles) return;     // a padding block: all of it
  const bool busy = tile0 < a.tiles;
  const int stride = a.chunk + 16;

  const v4i* codes[RT];
  const uint32_t* scales[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {                           // a spare tile repeats the last one, stores nothing
    const int64_t t = min(tile0 + i, a.tiles - 1);
    codes[i] = (const v4i*)a.codes + t * a.blocks * 64 + lane;
    scales[i] = (const uint32_t*)a.scales + (t * a.blocks * 4 + q) * (NG * 2);
  }
  const int8_t* x[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j)                             // a spare token repeats the last one
    x[j] = sm_x + min(16 * j + r, tokens - 1) * stride + (G == 32 ? 8 : 16) * q;

  float sum[RT][NT][4] = {};
  for (int c0 = 0; c0 < a.blocks; c0 += a.chunk / 128) {   // blocks whose columns are in LDS
    const int cn = min(a.chunk / 128, a.blocks - c0);
    if (c0) __syncthreads();
    {
      const int cols = min(cn * 128, a.K - c0 * 128);      // what is past K meets codes of zero
      const int per = cols / 16;                           // K % 32 == 0
      for (int i = threadIdx.x; i < tokens * per; i += 64 * kWaves) {
        const int t = i / per, c = (i - t * per) * 16;
        *(int4*)(sm_x + t * stride + c) = *(const int4*)(a.xq + (size_t)(token0 + t) * a.K + c0 * 128 + c);
      }
    }
    __syncthreads();
    if (!busy) continue;
    for (int b0 = part; b0 < cn; b0 += ks * kAhead) {
      v4i code[kAhead][RT];
      Q4Scales<G> sc[kAhead][RT];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int64_t b = c0 + min(b0 + u * ks, cn - 1);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          code[u][i] = __builtin_nontemporal_load(codes[i] + b * 64);
          const uint32_t* p = scales[i] + b * 4 * (NG * 2);
          if constexpr (G == 128) {
            *(uint2*)sc[u][i].w = *(const uint2*)p;
          } else {
            *(uint4*)sc[u][i].w = *(const uint4*)p;
            if constexpr (G == 32) *(uint4*)(sc[u][i].w + 4) = *(const uint4*)(p + 4);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int b = b0 + u * ks;
        if (b >= cn) break;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const int8_t* xb = x[j] + b * 128 + g * G;
            if constexpr (G == 32) {
              const int2 xv = *(const int2*)xb;
#pragma unroll
              for (int i = 0; i < RT; ++i) {
                const uint32_t d = (uint32_t)code[u][i][g];
                const uint2 lo_hi = {(d << 4) & 0xF0F0F0F0u, d & 0xF0F0F0F0u};
                const v4i acc = __builtin_amdgcn_mfma_i32_16x16x32_i8(__builtin_bit_cast(long, lo_hi),
                                                                      __builtin_bit_cast(long, xv), v4i{}, 0, 0, 0);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const uint32_t w = sc[u][i].w[g * 2 + (e >> 1)];
                  sum[i][j][e] = __builtin_fmaf((float)acc[e], (e & 1) ? bf16_hi(w) : bf16_lo(w), sum[i][j][e]);
                }
              }
            } else {
              v4i xv[G / 64];
#pragma unroll
              for (int h = 0; h < G / 64; ++h) xv[h] = *(const v4i*)(xb + 64 * h);
#pragma unroll
              for (int i = 0; i < RT; ++i) {
                v4i acc = {};
#pragma unroll
                for (int h = 0; h < G / 64; ++h) {
                  const int w0 = (G == 64 ? 2 * g : 2 * h);
                  const uint32_t d0 = (uint32_t)code[u][i][w0], d1 = (uint32_t)code[u][i][w0 + 1];
                  const v4i av = {(int)((d0 << 4) & 0xF0F0F0F0u), (int)(d0 & 0xF0F0F0F0u),
                                  (int)((d1 << 4) & 0xF0F0F0F0u), (int)(d1 & 0xF0F0F0F0u)};
                  acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(av, xv[h], acc, 0, 0, 0);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const uint32_t w = sc[u][i].w[g * 2 + (e >> 1)];
                  sum[i][j][e] = __builtin_fmaf((float)acc[e], (e & 1) ? bf16_hi(w) : bf16_lo(w), sum[i][j][e]);
                }
              }
            }
          }
        }
      }
    }
  }

  if (ks > 1) {                                            // parts of a tile, joined by its first wave in order
    float* red = (float*)sm_x;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) red[((wave * RT + i) * NT + j) * 256 + e * 64 + lane] = sum[i][j][e];
    __syncthreads();
    if (part) return;
    for (int p = 1; p < ks; ++p)
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[i][j][e] += red[(((wave + p) * RT + i) * NT + j) * 256 + e * 64 + lane];
  }
  if (!busy) return;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int t = token0 + 16 * j + r;
    if (16 * j + r >= tokens) continue;
    const float s = a.x_scale[t] * 0.0625f;
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int64_t o = (tile0 + i) * 16 + 4 * q;
      if (o >= a.n) continue;
      float* y = a.y + (size_t)t * a.n + o;
      if (a.n % 4 == 0) {
        *(float4*)y = make_float4(sum[i][j][0] * s, sum[i][j][1] * s, sum[i][j][2] * s, sum[i][j][3] * s);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (o + e < a.n) y[e] = sum[i][j][e] * s;
      }
    }
  }
}

template <int G, int NT, int RT>
hipError_t fwd(Q4Args a, hipStream_t s) {
  const int tokens = std::min(a.T, 16 * NT);
  // columns in LDS at a time: even parts of K
  const int most = (kLds / tokens - 16) / 128 * 128;
  const int chunks = (a.blocks * 128 + most - 1) / most;
  a.chunk = (a.blocks + chunks - 1) / chunks * 128;
  // waves on one tile's columns: until there are two waves per SIMD, or no columns to share
  a.token_tiles = (a.T + 16 * NT - 1) / (16 * NT);
  a.ksplit = 1;
  while (a.ksplit < kWaves && a.tiles / RT * a.token_tiles * a.ksplit < 2048 && a.ksplit * 2 <= a.chunk / 128)
    a.ksplit *= 2;
  const int64_t per = kWaves / a.ksplit * RT;
  const int64_t row_blocks = (a.tiles + per - 1) / per;
  const int64_t grid = (row_blocks + 7) / 8 * 8 * a.token_tiles;
  size_t lds = (size_t)tokens * (a.chunk + 16);
  if (a.ksplit > 1) lds = std::max(lds, (size_t)kWaves * RT * NT * 1024);
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute((const void*)q4_fwd_kernel<G, NT, RT>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
    if (e != hipSuccess) return e;
  }
  q4_fwd_kernel<G, NT, RT><<<(unsigned)grid, 64 * kWaves, lds, s>>>(a);
  return hipGetLastError();
}

template <int G>
hipError_t fwd_tokens(const Q4Args& a, hipStream_t s) {
  if (a.T <= 16) return fwd<G, 1, 1>(a, s);
  if (a.T <= 32) return fwd<G, 2, 1>(a, s);
  return fwd<G, 4, 1>(a, s);
}

}  // namespace

hipError_t launch_q4_pack(const Q4PackArgs& a, bool bf16, hipStream_t s) {
  const unsigned grid = (unsigned)(a.tiles * a.blocks);    // 16 rows x 16 eights of columns each
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
  if (group == 32) return fwd_tokens<32>(a, s);
  if (group == 64) return fwd_tokens<64>(a, s);
  return fwd_tokens<128>(a, s);
}

}  // namespace bl
