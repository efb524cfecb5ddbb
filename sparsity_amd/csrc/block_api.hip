// C ABI of the operators between a decoder block's projections: host-side validation, then launches
// on the caller's stream.  Every check runs before anything is enqueued.
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "api_checks.hpp"
#include "bitlinear.h"
#include "block_ops.hpp"
#include "device_common.hpp"

using namespace bl::api;

extern "C" {

int bitlinear_norm_quant(const void* x, int x_dtype, const void* res, int res_dtype,
                         const float* w, double eps, int64_t T, int64_t K, int lift_M, void* h,
                         int8_t* xq, float* x_scale, float* rstd_opt, void* stream) {
  if (!float_dtype(x_dtype) || (res && !float_dtype(res_dtype))) return BL_ENOTSUP;
  if (lift_M != 0) {
    if (lift_M < 6 || lift_M > 16 || lift_M % 2) return BL_EINVAL;
    if (K % bl::lcm_i(lift_M, 8) != 0) return BL_EINVAL;
  }
  if (!rows_ok(T, K) || !(eps > 0.0) || !isfinite(eps)) return BL_EINVAL;
  if (K > bl::kNormMaxK) return BL_ENOTSUP;
  if (T == 0) return BL_OK;
  if (!aligned(x, 16) || !aligned(xq, 16) || !aligned(x_scale, 4)) return BL_EINVAL;
  if ((res != nullptr) != (h != nullptr)) return BL_EINVAL;
  if (res && (!aligned(res, 16) || !aligned(h, 16))) return BL_EINVAL;
  if ((w && !aligned(w, 16)) || (rstd_opt && !aligned(rstd_opt, 4))) return BL_EINVAL;
  const uint64_t n = (uint64_t)T * (uint64_t)K;
  const uint64_t keff = lift_M ? (uint64_t)K / lift_M * (2 * lift_M - 4) : (uint64_t)K;
  const Span in[3] = {{x, n * esize(x_dtype)}, {res, res ? n * esize(res_dtype) : 0}, {w, (uint64_t)K * 4}};
  const Span out[4] = {{h, h ? n * esize(res_dtype) : 0}, {xq, T * keff}, {x_scale, (uint64_t)T * 4},
                       {rstd_opt, (uint64_t)T * 4}};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 3; ++j) {
      const bool in_place = i == 0 && out[i].p == in[j].p && (j == 1 || (j == 0 && x_dtype == res_dtype));
      if (!in_place && overlap(out[i], in[j])) return BL_EINVAL;
    }
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return BL_EINVAL;
  }
  const bl::NormArgs a = {x, res, w, h, xq, x_scale, rstd_opt, eps, (int32_t)T, (int32_t)K, lift_M};
  return status_of(bl::launch_norm_quant(a, x_dtype == BL_DTYPE_BF16, res_dtype == BL_DTYPE_BF16,
                                         (hipStream_t)stream));
}

int bitlinear_norm_quant_bwd_workspace_bytes(int64_t T, int64_t K, size_t* ws_bytes) {
  if (!rows_ok(T, K) || !ws_bytes) return BL_EINVAL;
  if (K > bl::kNormMaxK) return BL_ENOTSUP;
  *ws_bytes = bl::norm_bwd_columns(T, K) ? 0 : (size_t)bl::norm_bwd_blocks(T, K) * (size_t)K * 4;
  return BL_OK;
}

int bitlinear_norm_quant_bwd(const void* dn, int dn_dtype, const void* h, int h_dtype,
                             const float* rstd, const float* w, const void* dres, void* dh,
                             int grad_dtype, float* dw, int64_t T, int64_t K, void* ws,
                             size_t ws_bytes, void* stream) {
  if (!float_dtype(dn_dtype) || !float_dtype(h_dtype) || !float_dtype(grad_dtype)) return BL_ENOTSUP;
  size_t need = 0;
  const int st = bitlinear_norm_quant_bwd_workspace_bytes(T, K, &need);
  if (st != BL_OK) return st;
  if (T == 0 && !dw) return BL_OK;
  if (T > 0 && (!aligned(dn, 16) || !aligned(h, 16) || !aligned(rstd, 4) || !aligned(dh, 16)))
    return BL_EINVAL;
  if ((w && !aligned(w, 16)) || (dres && !aligned(dres, 16)) || (dw && !aligned(dw, 16))) return BL_EINVAL;
  if (!dw) need = 0;
  if (need && !aligned(ws, 16)) return BL_EINVAL;
  if (ws_bytes < need) return BL_ENOSPC;
  if (!need) ws = nullptr;
  const uint64_t n = (uint64_t)T * (uint64_t)K;
  const Span in[5] = {{dn, n * esize(dn_dtype)}, {dres, n * esize(grad_dtype)}, {h, n * esize(h_dtype)},
                      {rstd, (uint64_t)T * 4}, {w, (uint64_t)K * 4}};
  const Span out[3] = {{dh, n * esize(grad_dtype)}, {dw, (uint64_t)K * 4}, {ws, need}};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 5; ++j) {
      const bool in_place = i == 0 && out[i].p == in[j].p && (j == 1 || (j == 0 && dn_dtype == grad_dtype));
      if (!in_place && overlap(out[i], in[j])) return BL_EINVAL;
    }
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return BL_EINVAL;
  }
  const bl::NormBwdArgs a = {dn, h, rstd, w, dres, dh, dw, (float*)ws, (int32_t)T, (int32_t)K,
                             bl::norm_bwd_blocks(T, K)};
  return status_of(bl::launch_norm_bwd(a, dn_dtype == BL_DTYPE_BF16, h_dtype == BL_DTYPE_BF16,
                                       grad_dtype == BL_DTYPE_BF16, (hipStream_t)stream));
}

int bitlinear_rope_table(const double* freq, int64_t half, int64_t positions, double mscale,
                         float* table, void* stream) {
  if (half < 1 || half > 128 || positions < 0 || positions > ((int64_t)1 << 31) / half) return BL_EINVAL;
  if (!isfinite(mscale)) return BL_EINVAL;
  if (positions == 0) return BL_OK;
  if (!aligned(freq, 8) || !aligned(table, 16)) return BL_EINVAL;
  if (overlap({freq, (uint64_t)half * 8}, {table, (uint64_t)half * positions * 8})) return BL_EINVAL;
  return status_of(bl::launch_rope_table(freq, half, positions, mscale, table, (hipStream_t)stream));
}

}  // extern "C"

namespace {

// The stride of an axis of one element is never a step and may be anything: it counts as 0.
int64_t step(int64_t stride, int64_t count) { return count > 1 ? stride : 0; }

// Whether a strided [T][heads][D] tensor can be read (strides, alignment to one element), and
// whether its rows are aligned to four.
bool strided_ok(const void* p, int64_t tok, int64_t head, int dtype) {
  const int64_t lim = (int64_t)1 << 46;
  return aligned(p, esize(dtype)) && tok >= 0 && head >= 0 && tok < lim && head < lim;
}
bool vec4(const void* p, int64_t tok, int64_t head, int dtype) {
  return aligned(p, 4 * esize(dtype)) && tok % 4 == 0 && head % 4 == 0;
}
// Rows of an output lie apart: heads inside a token, or tokens inside a head.
bool apart(int64_t T, int64_t heads, int64_t D, int64_t tok, int64_t head) {
  if (T > 1 && tok < D) return false;
  if (heads > 1 && head < D) return false;
  if (T > 1 && heads > 1) return tok <= head ? head / tok >= T - 1 && head >= (T - 1) * tok + D
                                             : tok / head >= heads - 1 && tok >= (heads - 1) * head + D;
  return true;
}

// Rows of a strided buffer, in bytes: `len` each, at p plus any multiple below `count` of each axis' stride.
typedef __int128 wide;
struct Axis {
  int64_t stride, count;
};
struct Rows {
  const void* p;
  wide len, end;             // end: of the last row
  Axis ax[3];
  Rows(const void* ptr, wide n, Axis x = {0, 1}, Axis y = {0, 1}, Axis z = {0, 1}) : p(ptr), len(n), ax{x, y, z} {
    end = (wide)(uintptr_t)p + len;
    for (auto& a : ax) {
      if (a.count <= 1) a.stride = 0;
      end += (wide)a.stride * (a.count - 1);
    }
  }
};

struct Steps {
  wide stride, lo, hi;       // multiples of the stride from lo to hi
};
wide floor_div(wide a, wide b) { return a / b - (a % b != 0 && (a < 0) != (b < 0)); }
// Whether at + some multiple of each of n strides, in falling order, lies in [lo, hi].
bool reaches(const Steps* s, int n, wide at, wide lo, wide hi, int* budget) {
  if (n == 0) return lo <= at && at <= hi;
  wide least = 0, most = 0;  // what the smaller strides can add
  for (int i = 1; i < n; ++i) {
    least += s[i].stride * s[i].lo;
    most += s[i].stride * s[i].hi;
  }
  const wide first = std::max(s[0].lo, -floor_div(at + most - lo, s[0].stride));
  const wide last = std::min(s[0].hi, floor_div(hi - least - at, s[0].stride));
  for (wide k = first; k <= last; ++k) {
    if (--*budget < 0) return false;
    if (reaches(s + 1, n - 1, at + k * s[0].stride, lo, hi, budget)) return true;
  }
  return false;
}
// Whether a row of a meets a row of b.  Axes of one stride in both count by their difference, so slices of
// one buffer beside each other take a few trials; buffers that interleave with unlike strides are looked
// at for 2^16 of them, and then taken to be apart.
bool rows_meet(const Rows& a, const Rows& b) {
  const wide at = (wide)(uintptr_t)a.p - (wide)(uintptr_t)b.p;
  if (!a.p || !b.p || a.len <= 0 || b.len <= 0) return false;
  if (a.end <= (wide)(uintptr_t)b.p || b.end <= (wide)(uintptr_t)a.p) return false;
  Steps s[6];
  int n = 0;
  for (const auto& x : a.ax)
    if (x.stride) s[n++] = {x.stride, 0, x.count - 1};
  const int na = n;
  for (const auto& x : b.ax) {
    if (!x.stride) continue;
    int i = 0;
    while (i < na && !(s[i].stride == x.stride && s[i].lo == 0)) ++i;
    if (i < na) s[i].lo = 1 - x.count;
    else s[n++] = {x.stride, 1 - x.count, 0};
  }
  std::sort(s, s + n, [](const Steps& x, const Steps& y) { return x.stride > y.stride; });
  int budget = 1 << 16;
  return reaches(s, n, at, 1 - a.len, b.len - 1, &budget);
}

// Checks common to both rope calls; fills the tensors.
int rope_tensors(const bl_rope_desc* d, int64_t count, int64_t T, int64_t D, int64_t R, int x_dtype,
                 int y_dtype, const int32_t* pos, const float* table, int64_t positions, int writes,
                 bl::RopeArgs* a, bool* vec) {
  int64_t heads = 0;
  *vec = D % 8 == 0 && R % 8 == 0;
  for (int64_t i = 0; i < count; ++i) {
    const int64_t n = d[i].heads;
    if (n < 1 || heads + n > (1 << 20)) return BL_EINVAL;
    bl::RopeTensor& t = a->t[i];
    t = {d[i].x, i < writes ? d[i].y : nullptr, step(d[i].x_tok, T), step(d[i].x_head, n),
         step(d[i].y_tok, T), step(d[i].y_head, n), (int32_t)heads, (int32_t)n};
    heads += n;
    if (T == 0) continue;
    if (!strided_ok(t.x, t.x_tok, t.x_head, x_dtype)) return BL_EINVAL;
    *vec = *vec && vec4(t.x, t.x_tok, t.x_head, x_dtype);
    if (i >= writes) continue;
    if (!strided_ok(t.y, t.y_tok, t.y_head, y_dtype)) return BL_EINVAL;
    if (!apart(T, n, D, t.y_tok, t.y_head)) return BL_EINVAL;
    if (t.x == t.y && (x_dtype != y_dtype || t.x_tok != t.y_tok || t.x_head != t.y_head)) return BL_EINVAL;
    *vec = *vec && vec4(t.y, t.y_tok, t.y_head, y_dtype);
  }
  if (T > 0 && (!aligned(pos, 4) || !aligned(table, 16))) return BL_EINVAL;
  a->pos = pos;
  a->table = table;
  a->positions = positions;
  a->T = T;
  a->count = (int32_t)count;
  a->heads = (int32_t)heads;
  a->D = (int32_t)D;
  a->R = (int32_t)R;
  return BL_OK;
}

// Checks a cache; *extent: elements from the start of k (and of v) to the end of its last row.
int check_cache(const bl_kv_cache* kv, int64_t* extent) {
  if (!kv) return BL_EINVAL;
  if (kv->dtype != BL_DTYPE_BF16 && kv->dtype != BL_DTYPE_I8) return BL_ENOTSUP;
  const int64_t q = kv->dtype == BL_DTYPE_I8 ? 16 : 8;
  if (kv->pages < 1 || kv->pages > INT32_MAX || kv->page_size < 1 || kv->heads < 1 ||
      kv->heads > (1 << 16) || kv->head_dim < 1 || kv->head_dim > 256 || kv->head_dim % q)
    return BL_EINVAL;
  // rows apart: in the order of their strides, each axis steps over all of the one before
  Axis ax[3] = {{kv->page_stride, kv->pages}, {kv->head_stride, kv->heads}, {kv->tok_stride, kv->page_size}};
  for (auto& x : ax) {
    x.stride = step(x.stride, x.count);
    if (x.stride < 0 || x.stride % q || x.stride > ((int64_t)1 << 46)) return BL_EINVAL;
  }
  std::sort(ax, ax + 3, [](const Axis& p, const Axis& r) { return p.stride < r.stride; });
  int64_t span = kv->head_dim;   // elements one step of the axes so far covers
  for (auto& x : ax) {
    if (x.count == 1) continue;
    if (x.stride < span) return BL_EINVAL;
    if (x.stride > ((int64_t)1 << 60) / x.count) return BL_EINVAL;
    span += (x.count - 1) * x.stride;
  }
  if (!aligned(kv->k, 16) || !aligned(kv->v, 16)) return BL_EINVAL;
  if (kv->dtype == BL_DTYPE_I8 && (!aligned(kv->k_scale, 4) || !aligned(kv->v_scale, 4))) return BL_EINVAL;
  *extent = span;
  return BL_OK;
}

}  // namespace

extern "C" {

int bitlinear_rope(const bl_rope_desc* descs, int64_t count, int64_t T, int64_t D, int64_t R,
                   int interleaved, int inverse, int x_dtype, int y_dtype, const int32_t* pos,
                   const float* table, int64_t positions, void* stream) {
  if (!float_dtype(x_dtype) || !float_dtype(y_dtype)) return BL_ENOTSUP;
  if (!descs || count < 1 || count > bl::kRopeMax) return BL_EINVAL;
  if (T < 0 || T > kMaxTokens || D < 1 || D > 256 || R < 2 || R > D || R % 2 || positions < 0 ||
      positions > INT32_MAX)
    return BL_EINVAL;
  bl::RopeArgs a = {};
  bool vec = false;
  const int st = rope_tensors(descs, count, T, D, R, x_dtype, y_dtype, pos, table, positions,
                              (int)count, &a, &vec);
  if (st != BL_OK) return st;
  if (T == 0) return BL_OK;
  auto rows = [&](int i, bool y) {
    const bl::RopeTensor& t = a.t[i];
    const int64_t e = esize(y ? y_dtype : x_dtype);
    return y ? Rows(t.y, D * e, {t.y_tok * e, T}, {t.y_head * e, t.heads})
             : Rows(t.x, D * e, {t.x_tok * e, T}, {t.x_head * e, t.heads});
  };
  const Rows p(pos, T * 4), tab(table, positions * R * 4);
  for (int i = 0; i < count; ++i) {
    const Rows y = rows(i, true);
    if (rows_meet(y, p) || rows_meet(y, tab)) return BL_EINVAL;
    for (int j = 0; j < count; ++j) {
      if (!(i == j && a.t[i].x == a.t[i].y) && rows_meet(y, rows(j, false))) return BL_EINVAL;
      if (j < i && rows_meet(y, rows(j, true))) return BL_EINVAL;
    }
  }
  a.interleaved = interleaved != 0;
  a.inverse = inverse != 0;
  return status_of(bl::launch_rope(a, x_dtype == BL_DTYPE_BF16, y_dtype == BL_DTYPE_BF16, vec,
                                   (hipStream_t)stream));
}

int bitlinear_rope_append(const bl_rope_desc* qkv, int64_t T, int64_t R, int interleaved,
                          int x_dtype, int q_dtype, const int32_t* pos, const int32_t* seq,
                          const int32_t* blocks, int64_t seqs, int64_t blocks_per_seq,
                          const float* table, int64_t positions, const bl_kv_cache* kv,
                          void* stream) {
  if (!float_dtype(x_dtype) || !float_dtype(q_dtype)) return BL_ENOTSUP;
  int64_t extent = 0;
  const int cs = check_cache(kv, &extent);
  if (cs != BL_OK) return cs;
  const int64_t D = kv->head_dim;
  if (!qkv || T < 0 || T > kMaxTokens || R < 2 || R > D || R % 2 || positions < 0 ||
      positions > INT32_MAX || seqs < 1 || blocks_per_seq < 1 || seqs > INT32_MAX ||
      blocks_per_seq > INT32_MAX)
    return BL_EINVAL;
  if (qkv[1].heads != kv->heads || qkv[2].heads != kv->heads) return BL_EINVAL;
  bl::RopeArgs a = {};
  bool vec = false;
  const int st = rope_tensors(qkv, 3, T, D, R, x_dtype, q_dtype, pos, table, positions, 1, &a, &vec);
  if (st != BL_OK) return st;
  if (T == 0) return BL_OK;
  if (!aligned(blocks, 4) || (seq && !aligned(seq, 4))) return BL_EINVAL;
  const bool i8 = kv->dtype == BL_DTYPE_I8;
  const int64_t ce = esize(kv->dtype), xe = esize(x_dtype), qe = esize(q_dtype);
  auto cache = [&](const void* p) {
    return Rows(p, D * ce, {step(kv->page_stride, kv->pages) * ce, kv->pages},
                {step(kv->head_stride, kv->heads) * ce, kv->heads},
                {step(kv->tok_stride, kv->page_size) * ce, kv->page_size});
  };
  auto rows = [&](const bl::RopeTensor& t) {
    return Rows(t.x, D * xe, {t.x_tok * xe, T}, {t.x_head * xe, t.heads});
  };
  const wide scales = i8 ? (wide)kv->pages * kv->heads * kv->page_size * 4 : 0;
  const bl::RopeTensor& q = a.t[0];
  const Rows out[5] = {Rows(q.y, D * qe, {q.y_tok * qe, T}, {q.y_head * qe, q.heads}), cache(kv->k),
                       cache(kv->v), Rows(kv->k_scale, scales), Rows(kv->v_scale, scales)};
  const Rows in[7] = {rows(q), rows(a.t[1]), rows(a.t[2]), Rows(pos, T * 4), Rows(seq, T * 4),
                      Rows(blocks, (wide)seqs * blocks_per_seq * 4), Rows(table, positions * R * 4)};
  for (int i = 0; i < 5; ++i) {
    for (int j = 0; j < 7; ++j)
      if (!(i == 0 && j == 0 && q.x == q.y) && rows_meet(out[i], in[j])) return BL_EINVAL;
    for (int j = 0; j < i; ++j)
      if (rows_meet(out[i], out[j])) return BL_EINVAL;
  }
  a.interleaved = interleaved != 0;
  a.kv = *kv;
  a.blocks = blocks;
  a.seq = seq;
  a.seqs = seqs;
  a.blocks_per_seq = blocks_per_seq;
  return status_of(bl::launch_rope_append(a, x_dtype == BL_DTYPE_BF16, q_dtype == BL_DTYPE_BF16, vec,
                                          (hipStream_t)stream));
}

}  // extern "C"

namespace {

constexpr int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

// The arrival counts first, as many for every plan: no plan's partial sums lie where another one's counts
// have to be zero, so plans can take turns on a workspace.
struct AttnWs {
  int64_t ticket, ml, part, total;
};
AttnWs attn_ws(const bl_attn_plan& p) {
  const int64_t G = p.q_heads / p.kv_heads, rows = p.q_rows;
  AttnWs w;
  w.ticket = 0;
  w.ml = up256(bl::kAttnBlocks * 4);
  w.part = w.ml + up256((int64_t)p.blocks * 2 * 2 * rows * 4);
  w.total = w.part + up256((int64_t)p.blocks * 2 * std::min(G, rows) * p.head_dim * 4);
  return w;
}

}  // namespace

extern "C" {

int bitlinear_paged_attn_plan(int64_t B, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                              int64_t max_len, int64_t window, bl_attn_plan* plan) {
  if (!plan || B < 0 || B > (1 << 20) || kv_heads < 1 || kv_heads > (1 << 16) || q_heads < kv_heads ||
      q_heads > (1 << 20) || q_heads % kv_heads || head_dim < 8 || head_dim > 256 || head_dim % 8 ||
      max_len < 1 || max_len > INT32_MAX || window < 0 || window > INT32_MAX)
    return BL_EINVAL;
  const int64_t G = q_heads / kv_heads;
  if (B * kv_heads * ((G + 15) / 16) > ((int64_t)1 << 22)) return BL_EINVAL;
  *plan = {B, max_len, (int32_t)q_heads, (int32_t)kv_heads, (int32_t)head_dim, (int32_t)window, 0, 0, 0};
  bl::paged_attn_split(*plan);
  plan->ws_bytes = (size_t)attn_ws(*plan).total;
  return BL_OK;
}

int bitlinear_paged_attn(const bl_attn_plan* plan, const void* q, int q_dtype, int64_t q_tok,
                         int64_t q_head, float scale, const bl_kv_cache* kv, const int32_t* blocks,
                         int64_t blocks_per_seq, const int32_t* lens, void* out, float* lse_opt,
                         void* ws, size_t ws_bytes, void* stream) {
  if (!plan) return BL_EINVAL;
  if (!float_dtype(q_dtype)) return BL_ENOTSUP;
  bl_attn_plan p;
  const int st = bitlinear_paged_attn_plan(plan->B, plan->q_heads, plan->kv_heads, plan->head_dim,
                                           plan->max_len, plan->window, &p);
  if (st != BL_OK) return st;
  if (p.blocks != plan->blocks || p.q_rows != plan->q_rows) return BL_EINVAL;   // not this build's plan
  int64_t extent = 0;
  const int cs = check_cache(kv, &extent);
  if (cs != BL_OK) return cs;
  if (kv->heads != p.kv_heads || kv->head_dim != p.head_dim) return BL_EINVAL;
  if (!isfinite(scale) || blocks_per_seq < 0 || blocks_per_seq > INT32_MAX) return BL_EINVAL;
  if (p.B == 0) return BL_OK;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lens, 4) || (lse_opt && !aligned(lse_opt, 4)) ||
      (blocks_per_seq > 0 && !aligned(blocks, 4)))
    return BL_EINVAL;
  q_tok = step(q_tok, p.B);
  q_head = step(q_head, p.q_heads);
  if (!strided_ok(q, q_tok, q_head, q_dtype) || q_tok % 8 || q_head % 8) return BL_EINVAL;
  if (!aligned(ws, 256)) return BL_EINVAL;
  if (ws_bytes < p.ws_bytes) return BL_ENOSPC;
  const AttnWs w = attn_ws(p);
  const int64_t rows = p.B * p.q_heads;
  const Span o = {out, (uint64_t)(rows * p.head_dim * esize(q_dtype))}, l = {lse_opt, (uint64_t)rows * 4},
             s = {ws, p.ws_bytes};
  if (overlap(o, l) || overlap(o, s) || overlap(l, s)) return BL_EINVAL;
  const uint64_t kvb = (uint64_t)extent * esize(kv->dtype);
  const uint64_t scb = kv->dtype == BL_DTYPE_I8 ? (uint64_t)kv->pages * kv->heads * kv->page_size * 4 : 0;
  const Span in[7] = {{q, (uint64_t)((p.B - 1) * q_tok + (p.q_heads - 1) * q_head + p.head_dim) * esize(q_dtype)},
                      {kv->k, kvb}, {kv->v, kvb}, {kv->k_scale, scb}, {kv->v_scale, scb},
                      {blocks, (uint64_t)p.B * blocks_per_seq * 4}, {lens, (uint64_t)p.B * 4}};
  for (const Span& i : in)
    if (overlap(i, o) || overlap(i, l) || overlap(i, s)) return BL_EINVAL;
  bl::AttnArgs a = {};
  a.kv = *kv;
  a.q = q;
  a.q_tok = q_tok;
  a.q_head = q_head;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.blocks = blocks;
  a.lens = lens;
  a.blocks_per_seq = blocks_per_seq;
  a.out = out;
  a.lse = lse_opt;
  a.ticket = (uint32_t*)((char*)ws + w.ticket);
  a.ml = (float*)((char*)ws + w.ml);
  a.part = (float*)((char*)ws + w.part);
  a.B = p.B;
  a.Hq = p.q_heads;
  a.G = p.q_heads / p.kv_heads;
  a.q_rows = p.q_rows;
  a.qtiles = (a.G + a.q_rows - 1) / a.q_rows;
  a.nblocks = p.blocks;
  a.window = p.window;
  return status_of(bl::launch_paged_attn(a, q_dtype == BL_DTYPE_BF16, (hipStream_t)stream));
}

}  // extern "C"
