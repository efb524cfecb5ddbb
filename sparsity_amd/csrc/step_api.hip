// C ABI of the operators around a model's blocks: host-side validation, then launches on the caller's
// stream.  Every check runs before anything is enqueued.
#include <math.h>
#include <stdint.h>

#include "api_checks.hpp"
#include "bitlinear.h"
#include "step_ops.hpp"

using namespace bl::api;

namespace {

// Whether an output overlaps an input or another output; outs[i] may be ins[same[i]] itself (-1: none).
template <int NI, int NO>
bool clash(const Span (&in)[NI], const Span (&out)[NO], const int (&same)[NO]) {
  for (int i = 0; i < NO; ++i) {
    for (int j = 0; j < NI; ++j)
      if (!(same[i] == j && out[i].p == in[j].p) && overlap(out[i], in[j])) return true;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return true;
  }
  return false;
}

constexpr int64_t kQ4MaxN = (int64_t)1 << 27, kQ4MaxK = (int64_t)1 << 16;
constexpr int64_t kSampleMaxB = 65535, kSampleMaxV = ((int64_t)1 << 24) - 1;   // sums of weights stay below 2^64

}  // namespace

extern "C" {

int bitlinear_kv_step(const int32_t* cached, const int32_t* fresh, int64_t B, int32_t* blocks,
                      int64_t blocks_per_seq, int64_t page_size, int32_t* free_pages,
                      int64_t free_cap, const int32_t* free_count, int32_t* free_count_out, int64_t T,
                      int32_t* seq, int32_t* pos, int64_t* slot_opt, int32_t* lens, int32_t* starts,
                      void* stream) {
  if (B < 0 || B > (1 << 20) || T < 0 || T > kMaxTokens || blocks_per_seq < 1 || blocks_per_seq > INT32_MAX ||
      page_size < 1 || page_size > INT32_MAX || free_cap < 0 || free_cap > INT32_MAX)
    return BL_EINVAL;
  if (B * blocks_per_seq >= ((int64_t)1 << 40)) return BL_EINVAL;
  if (!aligned(free_count, 4) || !aligned(free_count_out, 4) || !aligned(starts, 4)) return BL_EINVAL;
  if (B > 0 && (!aligned(cached, 4) || !aligned(fresh, 4) || !aligned(blocks, 4) || !aligned(lens, 4)))
    return BL_EINVAL;
  if (free_cap > 0 && !aligned(free_pages, 4)) return BL_EINVAL;
  if (T > 0 && (!aligned(seq, 4) || !aligned(pos, 4) || (slot_opt && !aligned(slot_opt, 8)))) return BL_EINVAL;
  const Span in[3] = {{cached, (uint64_t)B * 4}, {fresh, (uint64_t)B * 4}, {free_count, 4}};
  const Span out[8] = {{lens, (uint64_t)B * 4},
                       {free_count_out, 4},
                       {blocks, (uint64_t)(B * blocks_per_seq) * 4},
                       {free_pages, (uint64_t)free_cap * 4},
                       {seq, (uint64_t)T * 4},
                       {pos, (uint64_t)T * 4},
                       {slot_opt, (uint64_t)T * 8},
                       {starts, (uint64_t)(B + 1) * 4}};
  if (clash(in, out, {0, 2, -1, -1, -1, -1, -1, -1})) return BL_EINVAL;
  const bl::KvStepArgs a = {cached, fresh, blocks, free_pages, free_count, free_count_out, seq, pos, slot_opt,
                            lens, starts, B, blocks_per_seq, free_cap, T, (uint32_t)page_size};
  return status_of(bl::launch_kv_step(a, (hipStream_t)stream));
}

int bitlinear_embed(const void* table, int table_dtype, int64_t V, int64_t K, const int32_t* ids,
                    int64_t T, float scale, void* y, int y_dtype, void* stream) {
  if (!float_dtype(table_dtype) || !float_dtype(y_dtype)) return BL_ENOTSUP;
  if (!rows_ok(T, K) || V < 1 || V > INT32_MAX || !isfinite(scale)) return BL_EINVAL;
  if (K > bl::kEmbedMaxK) return BL_ENOTSUP;
  if (T == 0) return BL_OK;
  if (!aligned(table, 16) || !aligned(ids, 4) || !aligned(y, 16)) return BL_EINVAL;
  const Span in[2] = {{table, (uint64_t)(V * K * esize(table_dtype))}, {ids, (uint64_t)T * 4}};
  const Span out[1] = {{y, (uint64_t)(T * K * esize(y_dtype))}};
  if (clash(in, out, {-1})) return BL_EINVAL;
  const bl::EmbedArgs a = {table, ids, y, scale, V, (int32_t)T, (int32_t)K};
  return status_of(bl::launch_embed(a, table_dtype == BL_DTYPE_BF16, y_dtype == BL_DTYPE_BF16,
                                    (hipStream_t)stream));
}

int bitlinear_embed_bwd_workspace_bytes(int64_t T, int64_t K, size_t* ws_bytes) {
  if (!rows_ok(T, K) || !ws_bytes) return BL_EINVAL;
  if (K > bl::kEmbedMaxK) return BL_ENOTSUP;
  *ws_bytes = T ? bl::embed_bwd_ws(T, K).total : 0;
  return BL_OK;
}

int bitlinear_embed_bwd(const void* dy, int dy_dtype, const int32_t* ids, int64_t T, int64_t V,
                        int64_t K, float scale, float* dtable, int flags, void* ws, size_t ws_bytes,
                        void* stream) {
  if (!float_dtype(dy_dtype)) return BL_ENOTSUP;
  size_t need = 0;
  const int st = bitlinear_embed_bwd_workspace_bytes(T, K, &need);
  if (st != BL_OK) return st;
  if (V < 1 || V > INT32_MAX || !isfinite(scale) || (flags & ~BL_EMBED_ACCUM)) return BL_EINVAL;
  if (T == 0 && (flags & BL_EMBED_ACCUM)) return BL_OK;
  if (!aligned(dtable, 16)) return BL_EINVAL;
  if (T > 0 && (!aligned(dy, 16) || !aligned(ids, 4) || !aligned(ws, 256))) return BL_EINVAL;
  if (ws_bytes < need) return BL_ENOSPC;
  const Span in[2] = {{dy, (uint64_t)(T * K * esize(dy_dtype))}, {ids, (uint64_t)T * 4}};
  const Span out[2] = {{dtable, (uint64_t)(V * K) * 4}, {ws, need}};
  if (clash(in, out, {-1, -1})) return BL_EINVAL;
  const bl::EmbedBwdArgs a = {dy, ids, dtable, scale, flags & BL_EMBED_ACCUM, V, T, (int32_t)K, (char*)ws};
  return status_of(bl::launch_embed_bwd(a, dy_dtype == BL_DTYPE_BF16, (hipStream_t)stream));
}

int bitlinear_q4_bytes(int64_t n, int64_t K, int group, size_t* code_bytes, size_t* scale_bytes) {
  if (group != 32 && group != 64 && group != 128) return BL_ENOTSUP;
  if (n < 1 || n > kQ4MaxN || K < group || K > kQ4MaxK || K % group || !code_bytes || !scale_bytes) return BL_EINVAL;
  const size_t blocks = (size_t)((n + 15) / 16) * (size_t)((K + 127) / 128);
  if (blocks >= (size_t)1 << 24) return BL_EINVAL;         // as many waves as a launch may have, nearly
  *code_bytes = blocks * 1024;
  *scale_bytes = blocks * (size_t)(2048 / group) * 2;
  return BL_OK;
}

int bitlinear_q4_pack(const void* W, int w_dtype, int64_t n, int64_t K, int group, uint8_t* codes,
                      uint16_t* scales, void* stream) {
  if (!float_dtype(w_dtype)) return BL_ENOTSUP;
  size_t cb = 0, sb = 0;
  const int st = bitlinear_q4_bytes(n, K, group, &cb, &sb);
  if (st != BL_OK) return st;
  if (!aligned(W, 16) || !aligned(codes, 16) || !aligned(scales, 16)) return BL_EINVAL;
  const Span in[1] = {{W, (uint64_t)(n * K * esize(w_dtype))}};
  const Span out[2] = {{codes, cb}, {scales, sb}};
  if (clash(in, out, {-1, -1})) return BL_EINVAL;
  const bl::Q4PackArgs a = {W, (uint32_t*)codes, scales, n, K, (n + 15) / 16, (K + 127) / 128, group};
  return status_of(bl::launch_q4_pack(a, w_dtype == BL_DTYPE_BF16, (hipStream_t)stream));
}

int bitlinear_q4_fwd(const int8_t* xq, const float* x_scale, int64_t T, int64_t K, const uint8_t* codes,
                     const uint16_t* scales, int group, int64_t n, float* y, void* stream) {
  size_t cb = 0, sb = 0;
  const int st = bitlinear_q4_bytes(n, K, group, &cb, &sb);
  if (st != BL_OK) return st;
  if (T < 0 || T > kMaxTokens || (n + 127) / 128 * ((T + 63) / 64) >= ((int64_t)1 << 21)) return BL_EINVAL;
  if (T == 0) return BL_OK;
  if (!aligned(xq, 16) || !aligned(x_scale, 4) || !aligned(codes, 16) || !aligned(scales, 16) || !aligned(y, 16))
    return BL_EINVAL;
  const Span in[4] = {{xq, (uint64_t)(T * K)}, {x_scale, (uint64_t)T * 4}, {codes, cb}, {scales, sb}};
  const Span out[1] = {{y, (uint64_t)(T * n) * 4}};
  if (clash(in, out, {-1})) return BL_EINVAL;
  const bl::Q4Args a = {xq, x_scale, codes, scales, y, n, (n + 15) / 16, (int32_t)T, (int32_t)K,
                        (int32_t)((K + 127) / 128), 0, 0, 0};
  return status_of(bl::launch_q4_fwd(a, group, (hipStream_t)stream));
}

int bitlinear_sample_workspace_bytes(int64_t B, int64_t V, size_t* ws_bytes) {
  if (B < 0 || B > kSampleMaxB || V < 1 || V > kSampleMaxV || !ws_bytes) return BL_EINVAL;
  bl::SampleArgs a = {};
  a.B = B;
  a.V = V;
  *ws_bytes = B ? bl::sample_split(a, nullptr) : 0;
  return BL_OK;
}

int bitlinear_sample(const void* x, int x_dtype, int64_t B, int64_t V, int64_t row_stride,
                     const float* temperature_opt, const int32_t* top_k_opt, const float* top_p_opt,
                     const float* min_p_opt, const double* u, int32_t* token, float* logprob_opt,
                     void* ws, size_t ws_bytes, void* stream) {
  if (!float_dtype(x_dtype)) return BL_ENOTSUP;
  size_t need = 0;
  const int st = bitlinear_sample_workspace_bytes(B, V, &need);
  if (st != BL_OK) return st;
  if (B > 1 && (row_stride < V || row_stride > ((int64_t)1 << 40))) return BL_EINVAL;
  if (B == 0) return BL_OK;
  if (B == 1) row_stride = V;              // never a step
  const int64_t e = esize(x_dtype);
  if (!aligned(x, e) || !aligned(u, 8) || !aligned(token, 4) || !aligned(ws, 256)) return BL_EINVAL;
  if ((temperature_opt && !aligned(temperature_opt, 4)) || (top_k_opt && !aligned(top_k_opt, 4)) ||
      (top_p_opt && !aligned(top_p_opt, 4)) || (min_p_opt && !aligned(min_p_opt, 4)) ||
      (logprob_opt && !aligned(logprob_opt, 4)))
    return BL_EINVAL;
  if (ws_bytes < need) return BL_ENOSPC;
  const uint64_t b4 = (uint64_t)B * 4;
  const Span in[6] = {{x, (uint64_t)((B - 1) * row_stride + V) * e}, {temperature_opt, b4}, {top_k_opt, b4},
                      {top_p_opt, b4}, {min_p_opt, b4}, {u, b4 * 2}};
  const Span out[3] = {{token, b4}, {logprob_opt, b4}, {ws, need}};
  if (clash(in, out, {-1, -1, -1})) return BL_EINVAL;
  bl::SampleArgs a = {};
  a.x = x;
  a.stride = row_stride;
  a.B = B;
  a.V = V;
  a.temperature = temperature_opt;
  a.top_k = top_k_opt;
  a.top_p = top_p_opt;
  a.min_p = min_p_opt;
  a.u = u;
  a.token = token;
  a.logprob = logprob_opt;
  bl::sample_split(a, (char*)ws);
  return status_of(bl::launch_sample(a, x_dtype == BL_DTYPE_BF16, V >= 8, (hipStream_t)stream));   // whole eights are loaded
}

}  // extern "C"
