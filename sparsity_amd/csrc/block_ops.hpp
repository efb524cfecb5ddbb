// Launchers and argument records of the operators between a decoder block's projections: residual
// + RMS norm + int8 quantization and its gradient, rotary positions, the paged key-value cache and
// the decode attention over it.  Arguments are validated by block_api.hip.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bitlinear.h"

namespace bl {

// 16-bit float pairs: the hardware conversion rounds to nearest even and keeps NaN a NaN.
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const bf16x2 p = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, p);
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Eight consecutive elements of a 16-byte aligned row piece (F32: two 16-byte accesses, BF16: one).
template <bool BF16>
__device__ __forceinline__ void load_f8(const void* p, size_t off, float v[8]) {
  if constexpr (BF16) {
    const uint4 u = *(const uint4*)((const uint16_t*)p + off);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) { v[2 * j] = bf16_lo(w[j]); v[2 * j + 1] = bf16_hi(w[j]); }
  } else {
    const float4 a = *(const float4*)((const float*)p + off);
    const float4 b = *(const float4*)((const float*)p + off + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}

template <bool BF16>
__device__ __forceinline__ void store_f8(void* p, size_t off, const float v[8]) {
  if constexpr (BF16) {
    *(uint4*)((uint16_t*)p + off) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                               pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  } else {
    *(float4*)((float*)p + off) = make_float4(v[0], v[1], v[2], v[3]);
    *(float4*)((float*)p + off + 4) = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// ---- residual + RMS norm + int8 quantization ----
constexpr int64_t kNormMaxK = 32768;   // 16 waves of four eight-element pieces per lane

struct NormArgs {
  const void* x;
  const void* res;       // nullptr: no residual
  const float* w;        // nullptr: all ones
  void* h;
  int8_t* xq;
  float* scale;
  float* rstd;           // nullptr: not wanted
  double eps;
  int32_t T, K, lift_M;
};
hipError_t launch_norm_quant(const NormArgs& a, bool x_bf16, bool res_bf16, hipStream_t s);

struct NormBwdArgs {
  const void* dn;
  const void* h;
  const float* rstd;
  const float* w;
  const void* dres;
  void* dh;
  float* dw;             // nullptr: not wanted
  float* part;           // [blocks][K] column sums of each block; nullptr: dw by columns
  int32_t T, K, blocks;
};
int norm_bwd_blocks(int64_t T, int64_t K);      // blocks of the rows
bool norm_bwd_columns(int64_t T, int64_t K);    // whether dw is summed by columns, without a workspace
hipError_t launch_norm_bwd(const NormBwdArgs& a, bool dn_bf16, bool h_bf16, bool grad_bf16,
                           hipStream_t s);

// ---- rotary positions and the cache append ----
constexpr int kRopeMax = 4;            // tensors per launch

struct RopeTensor {
  const void* x;
  void* y;
  int64_t x_tok, x_head, y_tok, y_head;   // strides in elements
  int32_t head0, heads;                   // heads [head0, head0 + heads) of the launch
};
struct RopeArgs {
  RopeTensor t[kRopeMax];
  const int32_t* pos;
  const float* table;
  int64_t positions;
  int64_t T;
  int32_t count, heads, D, R;
  int32_t interleaved, inverse;
  // append: tensor 0 = q, 1 = k (rotated into the cache), 2 = v (copied into the cache)
  bl_kv_cache kv;
  const int32_t* blocks;
  const int32_t* seq;
  int64_t seqs, blocks_per_seq;
};
hipError_t launch_rope(const RopeArgs& a, bool x_bf16, bool y_bf16, bool vec, hipStream_t s);
hipError_t launch_rope_append(const RopeArgs& a, bool x_bf16, bool y_bf16, bool vec, hipStream_t s);
hipError_t launch_rope_table(const double* freq, int64_t half, int64_t positions, double mscale,
                             float* table, hipStream_t s);

// ---- decode attention over the paged cache ----
constexpr int kAttnBlocks = 512;       // blocks of a launch at most: two per CU

struct AttnArgs {
  bl_kv_cache kv;
  const void* q;
  int64_t q_tok, q_head;
  float scale_log2;      // softmax scale times log2(e)
  const int32_t* blocks;
  const int32_t* lens;
  int64_t blocks_per_seq;
  void* out;             // [B][Hq][D]
  float* lse;            // [B][Hq] or nullptr
  float* part;           // [2 * nblocks][min(G, q_rows)][D] sums of runs of keys
  float* ml;             // [2 * nblocks][2][q_rows] their running maximum and sum
  uint32_t* ticket;      // [kAttnBlocks] arrivals, zero between launches
  int64_t B;
  int32_t Hq, G, q_rows, qtiles, nblocks, window;
};
// Fills q_rows and blocks of a plan whose other sizes are set.
void paged_attn_split(bl_attn_plan& p);
hipError_t launch_paged_attn(const AttnArgs& a, bool q_bf16, hipStream_t s);

}  // namespace bl
