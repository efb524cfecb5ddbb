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
// A wave takes 32 keys at a time for up to 16 query heads of one key head, the running maximum and
// sum of the softmax in registers:
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
// factor.  Probabilities enter the product as two bf16 terms (the value and its rounding error),
// and fp32 queries as three, so the products are good to 2^-17 and better; the matrix cores are
// idle enough that this costs nothing.
//
// The four waves of a block take quarters of the block's run of keys and join in LDS; a run's
// partial sums go to the workspace and the last block of a (sequence, head group) to finish joins
// them, in the order of the runs, so the result does not depend on which block that is.
#include <algorithm>

#include "block_ops.hpp"
#include "device_common.hpp"

namespace bl {

namespace {

constexpr int kWaves = 4;
constexpr int kQ = 16;                      // query heads of a block
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

// DT: 64, 128 or 256, the head dimension's room.  I8: int8 cache.  QF: fp32 queries.
template <int DT, bool I8, bool QF>
__global__ __launch_bounds__(64 * kWaves) void paged_attn_kernel(AttnArgs a) {
  constexpr int EB = I8 ? 1 : 2;            // bytes per cache element
  constexpr int VE = DT / 16;               // value elements per lane and key
  constexpr int VW = VE * EB / 4;           // their dwords
  constexpr int VL = VW > 4 ? 2 : 1;        // 16-byte loads (or one narrower)
  constexpr int KC = DT / 32;               // 32-element steps of the q . k contraction
  constexpr int KW = DT * EB / 16;          // key dwords per lane and key tile
  constexpr int QS = QF ? 3 : 1;            // bf16 terms of a query element

  // union: per-wave rings of two 32-key groups' row offsets, then the waves' sums
  __shared__ __attribute__((aligned(16))) float sm_o[kWaves][kQ][DT + 4];
  __shared__ float sm_m[kWaves][kQ], sm_l[kWaves][kQ];
  __shared__ __attribute__((aligned(16))) int64_t ring[kWaves][2][32];
  __shared__ __attribute__((aligned(16))) int64_t sring[I8 ? kWaves : 1][I8 ? 2 : 1][I8 ? 32 : 1];

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane >> 4, n = lane & 15;
  const int64_t grp = blockIdx.x / a.splits;          // (sequence, key head, query tile)
  const int split = (int)(blockIdx.x - grp * a.splits);
  const int qt = (int)(grp % a.qtiles);
  const int64_t bh = grp / a.qtiles;
  const int hk = (int)(bh % a.kv.heads);
  const int64_t b = bh / a.kv.heads;
  const int D = a.kv.head_dim;
  const int rows = min(kQ, a.G - qt * kQ);            // live query heads
  const int hq0 = hk * a.G + qt * kQ;

  // live positions [first, len), this block's [k0, k1)
  const int64_t cap = a.blocks_per_seq * a.kv.page_size;
  const int64_t len = max((int64_t)0, min((int64_t)a.lens[b], cap));
  const int64_t first = a.window > 0 ? max((int64_t)0, len - a.window) : 0;
  const int64_t keys = len - first;
  // a sequence longer than the plan's bound takes longer runs, in whole groups per wave
  const int64_t per = (keys + a.splits - 1) / a.splits;
  const int64_t chunk = max((int64_t)a.chunk, (per + 32 * kWaves - 1) / (32 * kWaves) * (32 * kWaves));
  const int active = (int)max((int64_t)1, (keys + chunk - 1) / chunk);
  if (split >= active) return;
  const int64_t k0 = first + split * chunk, k1 = min(len, k0 + chunk);
  // this wave's quarter, in whole 32-key groups
  const int64_t quarter = ((k1 - k0 + kWaves - 1) / kWaves + 31) / 32 * 32;
  const int64_t w0 = min(k1, k0 + wave * quarter), w1 = min(k1, w0 + quarter);
  const int groups = (int)((w1 - w0 + 31) / 32);

  // queries: operand c, lane (g, n): elements of head n (zero past the live heads and past D)
  bf16x8 qf[QS][KC];
#pragma unroll
  for (int c = 0; c < KC; ++c) {
    // the int8 cache reads 16 elements per lane, so its steps come in pairs of adjacent eights
    const int d = I8 ? 64 * (c / 2) + 16 * g + 8 * (c & 1) : 32 * c + 8 * g;
    float v[8] = {};
    if (n < rows && d < D) {
      const int64_t o = b * a.q_tok + (int64_t)(hq0 + n) * a.q_head + d;
      load_f8<!QF>(a.q, o, v);
    }
#pragma unroll
    for (int t = 0; t < QS; ++t) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = pack_bf16(v[2 * j], v[2 * j + 1]);
        v[2 * j] -= bf16_lo(w[j]);
        v[2 * j + 1] -= bf16_hi(w[j]);
      }
      qf[t][c] = frag(w[0], w[1], w[2], w[3]);
    }
  }

  const int32_t* table = a.blocks + b * a.blocks_per_seq;
  const int ps = a.kv.page_size;
  const int64_t head_off = hk * a.kv.head_stride;
  const char* kbase = (const char*)a.kv.k + head_off * EB;
  const char* vbase = (const char*)a.kv.v + head_off * EB;

  // lane j < 32 of the wave looks after key j of each group: its page is read one group ahead of
  // the row offset that needs it
  auto key_of = [&](int grpi) { return w0 + 32 * (int64_t)grpi + (lane & 31); };
  auto page_of = [&](int grpi) -> int32_t {
    const int64_t t = key_of(grpi);
    return t < w1 ? table[(uint32_t)t / (uint32_t)ps] : -1;
  };
  auto put_rows = [&](int grpi, int32_t page) {
    const int64_t t = key_of(grpi);
    const int off = (int)((uint32_t)t % (uint32_t)ps);
    const bool ok = page >= 0 && page < a.kv.pages;   // a hole in the table is a masked run of keys
    if (lane < 32) {
      ring[wave][grpi & 1][lane] =
          ok ? ((int64_t)page * a.kv.page_stride + (int64_t)off * a.kv.tok_stride) * EB : -1;
      if constexpr (I8)
        sring[wave][grpi & 1][lane] = ok ? ((int64_t)page * a.kv.heads + hk) * ps + off : 0;
    }
    // LDS serves a wave's accesses in order; only the compiler has to keep them so
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  };

  uint32_t kr[2][KW], vr[8][VW];
  float ksc[I8 ? 8 : 1], vsc[I8 ? 8 : 1];
  int live = 0;                             // which of the lane's eight keys are live
  auto load_k = [&](int grpi) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int64_t r = max((int64_t)0, ring[wave][grpi & 1][16 * t + n]);   // masked: any row will do
#pragma unroll
      for (int c = 0; c < KW / 4; ++c) {
        const int d = I8 ? 64 * c + 16 * g : 32 * c + 8 * g;
        if (d < D) load_dw<4>(kbase + r + d * EB, &kr[t][4 * c]);
        else kr[t][4 * c] = kr[t][4 * c + 1] = kr[t][4 * c + 2] = kr[t][4 * c + 3] = 0;
      }
    }
  };
  auto load_v = [&](int grpi) {
    live = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int key = 16 * (i / 4) + 4 * g + (i & 3);
      const int64_t raw = ring[wave][grpi & 1][key];
      const int64_t r = max((int64_t)0, raw);
      live |= (raw >= 0 ? 1 : 0) << i;
      if constexpr (I8) {
        const int64_t sr = sring[wave][grpi & 1][key];
        ksc[i] = a.kv.k_scale[sr];
        vsc[i] = raw >= 0 ? a.kv.v_scale[sr] : 0.f;   // times a masked weight of 0
      }
#pragma unroll
      for (int c = 0; c < VL; ++c) {
        const int d = VE * n + (VE / VL) * c;
        if (d < D) load_dw<VW / VL>(vbase + r + d * EB, &vr[i][VW / VL * c]);
        else
#pragma unroll
          for (int j = 0; j < VW / VL; ++j) vr[i][VW / VL * c + j] = 0;
      }
    }
  };

  v4f o[VE];
#pragma unroll
  for (int j = 0; j < VE; ++j) o[j] = v4f{0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f;

  if (groups > 0) {
    put_rows(0, page_of(0));
    int32_t next = page_of(1);
    load_k(0);
    load_v(0);
    for (int i = 0; i < groups; ++i) {
      const bool more = i + 1 < groups;
      if (more) put_rows(i + 1, next);
      if (i + 2 < groups) next = page_of(i + 2);
      // scores
      v4f s[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        s[t] = v4f{0.f, 0.f, 0.f, 0.f};
        v4f rest = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < KC; ++c) {
          bf16x8 kf;
          if constexpr (I8) {
            uint32_t w[4];
            i8x4_bf16(kr[t][2 * c], w[0], w[1]);
            i8x4_bf16(kr[t][2 * c + 1], w[2], w[3]);
            kf = frag(w[0], w[1], w[2], w[3]);
          } else {
            kf = frag(kr[t][4 * c], kr[t][4 * c + 1], kr[t][4 * c + 2], kr[t][4 * c + 3]);
          }
          s[t] = mfma_bf16(kf, qf[0][c], s[t]);
#pragma unroll
          for (int u = 1; u < QS; ++u) rest = mfma_bf16(kf, qf[u][c], rest);
        }
        // an infinite key times a query's zero or negative remainder would spoil its score
        if constexpr (QF)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            s[t][r] = __builtin_isfinite(s[t][r]) ? s[t][r] + rest[r] : s[t][r];
      }
      if (more) load_k(i + 1);
      const bool full = __all(live == 0xFF);
      float x[8], mx = -INFINITY;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        x[k] = s[k / 4][k & 3] * a.scale_log2;
        if constexpr (I8) x[k] *= ksc[k];
        if (!full && !((live >> k) & 1)) x[k] = -INFINITY;
        mx = fmaxf(mx, x[k]);
      }
      if (__any(mx > m)) {                  // a new maximum: shared by the four lanes of a query
        mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
        mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
        const float top = fmaxf(m, mx);
        const float f = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - top);
        m = top;
        l *= f;
#pragma unroll
        for (int j = 0; j < VE; ++j) o[j] *= f;
      }
      const float base = m == -INFINITY ? 0.f : m;
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float p0 = __builtin_amdgcn_exp2f(x[2 * k] - base), p1 = __builtin_amdgcn_exp2f(x[2 * k + 1] - base);
        l += p0 + p1;
        if constexpr (I8) { p0 *= vsc[2 * k]; p1 *= vsc[2 * k + 1]; }
        hi[k] = pack_bf16(p0, p1);
        lo[k] = pack_bf16(p0 - bf16_lo(hi[k]), p1 - bf16_hi(hi[k]));
      }
      const bf16x8 ph = frag(hi[0], hi[1], hi[2], hi[3]), pl = frag(lo[0], lo[1], lo[2], lo[3]);
      if (!full) {                          // a masked row may hold anything: 0 * NaN is not 0
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int w = 0; w < VW; ++w) vr[k][w] = (live >> k) & 1 ? vr[k][w] : 0u;
      }
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if constexpr (I8)
            w[k] = upper_halves(i8_f32(vr[2 * k][j / 4], j & 3), i8_f32(vr[2 * k + 1][j / 4], j & 3));
          else
            w[k] = __builtin_amdgcn_perm(vr[2 * k + 1][j / 2], vr[2 * k][j / 2],
                                         j & 1 ? 0x07060302u : 0x05040100u);
        }
        const bf16x8 vf = frag(w[0], w[1], w[2], w[3]);
        o[j] = mfma_bf16(vf, ph, o[j]);
        o[j] = mfma_bf16(vf, pl, o[j]);
      }
      if (more) load_v(i + 1);
    }
  }
  l += __shfl_xor(l, 16, 64);
  l += __shfl_xor(l, 32, 64);

  // join the waves.  Lane (g, n) holds elements VE (4g + r) + j of head n.
  if (n < rows) {
    if (g == 0) { sm_m[wave][n] = m; sm_l[wave][n] = l; }
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int j = 0; j < VE; ++j) sm_o[wave][n][VE * (4 * g + r) + j] = o[j][r];
  }
  __syncthreads();
  const int64_t orow = (b * a.Hq + hq0) * (int64_t)D;
  auto finish = [&](int h, int d, float num, float den, float top) {
    const float v = den > 0.f ? num / den : 0.f;   // NaN sums fall to 0 / 0 below
    const float r = den == den ? v : num;
    if constexpr (QF) ((float*)a.out)[orow + (int64_t)h * D + d] = r;
    else ((uint16_t*)a.out)[orow + (int64_t)h * D + d] = (uint16_t)pack_bf16(r, 0.f);
    if (d == 0 && a.lse)
      a.lse[b * a.Hq + hq0 + h] = den > 0.f ? (top + log2f(den)) * kLn2 : den == den ? -INFINITY : den;
  };
  float* part = a.part + (grp * a.splits + split) * (int64_t)min(kQ, a.G) * D;
  float* ml = a.ml + (grp * a.splits + split) * 2 * kQ;
  for (int e = threadIdx.x; e < rows * D; e += 64 * kWaves) {
    const int h = e / D, d = e - h * D;
    float top = sm_m[0][h];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) top = fmaxf(top, sm_m[w][h]);
    float num = 0.f, den = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float f = sm_m[w][h] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(sm_m[w][h] - top);
      // a wave without live keys adds nothing; a NaN sum must not be hidden by f = 0
      if (sm_m[w][h] != -INFINITY || sm_l[w][h] != 0.f) {
        num += f * sm_o[w][h][d];
        den += f * sm_l[w][h];
      }
    }
    if (active == 1) {
      finish(h, d, num, den, top);
    } else {
      part[h * D + d] = num;
      if (d == 0) { ml[h] = top; ml[kQ + h] = den; }
    }
  }
}

// Joins the runs' partial sums: one block per (sequence, key head, query tile).
template <bool QF>
__global__ __launch_bounds__(256) void paged_attn_join_kernel(AttnArgs a) {
  const int64_t grp = blockIdx.x;
  const int qt = (int)(grp % a.qtiles);
  const int64_t bh = grp / a.qtiles;
  const int hk = (int)(bh % a.kv.heads);
  const int64_t b = bh / a.kv.heads;
  const int D = a.kv.head_dim, rows = min(kQ, a.G - qt * kQ), hq0 = hk * a.G + qt * kQ;
  const int64_t cap = a.blocks_per_seq * a.kv.page_size;
  const int64_t len = max((int64_t)0, min((int64_t)a.lens[b], cap));
  const int64_t keys = a.window > 0 ? min(len, (int64_t)a.window) : len;
  const int64_t per = (keys + a.splits - 1) / a.splits;
  const int64_t chunk = max((int64_t)a.chunk, (per + 32 * kWaves - 1) / (32 * kWaves) * (32 * kWaves));
  const int active = (int)max((int64_t)1, (keys + chunk - 1) / chunk);
  if (active == 1) return;
  for (int e = threadIdx.x; e < rows * D; e += 256) {
    const int h = e / D, d = e - h * D;
    const float* ml = a.ml + grp * a.splits * 2 * kQ;
    const float* part = a.part + grp * a.splits * (int64_t)min(kQ, a.G) * D + h * D + d;
    float top = -INFINITY;
    for (int s = 0; s < active; ++s) top = fmaxf(top, ml[s * 2 * kQ + h]);
    float num = 0.f, den = 0.f;
    for (int s = 0; s < active; ++s) {
      const float ms = ml[s * 2 * kQ + h], ls = ml[s * 2 * kQ + kQ + h];
      if (ms == -INFINITY && ls == 0.f) continue;
      const float f = ms == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(ms - top);
      num += f * part[s * (int64_t)min(kQ, a.G) * D];
      den += f * ls;
    }
    const float v = den > 0.f ? num / den : 0.f;
    const float r = den == den ? v : num;
    const int64_t o = (b * a.Hq + hq0 + h) * (int64_t)D + d;
    if constexpr (QF) ((float*)a.out)[o] = r;
    else ((uint16_t*)a.out)[o] = (uint16_t)pack_bf16(r, 0.f);
    if (d == 0 && a.lse)
      a.lse[b * a.Hq + hq0 + h] = den > 0.f ? (top + log2f(den)) * kLn2 : den == den ? -INFINITY : den;
  }
}

template <int DT>
hipError_t launch_attn_t(const AttnArgs& a, bool q_bf16, hipStream_t s) {
  const int64_t groups = a.B * a.kv.heads * a.qtiles;
  const dim3 grid((unsigned)(groups * a.splits));
  const bool i8 = a.kv.dtype == BL_DTYPE_I8;
  if (q_bf16) {
    if (i8) paged_attn_kernel<DT, true, false><<<grid, 64 * kWaves, 0, s>>>(a);
    else paged_attn_kernel<DT, false, false><<<grid, 64 * kWaves, 0, s>>>(a);
  } else {
    if (i8) paged_attn_kernel<DT, true, true><<<grid, 64 * kWaves, 0, s>>>(a);
    else paged_attn_kernel<DT, false, true><<<grid, 64 * kWaves, 0, s>>>(a);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  if (q_bf16) paged_attn_join_kernel<false><<<dim3((unsigned)groups), 256, 0, s>>>(a);
  else paged_attn_join_kernel<true><<<dim3((unsigned)groups), 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_paged_attn(const AttnArgs& a, bool q_bf16, hipStream_t s) {
  if (a.kv.head_dim <= 64) return launch_attn_t<64>(a, q_bf16, s);
  if (a.kv.head_dim <= 128) return launch_attn_t<128>(a, q_bf16, s);
  return launch_attn_t<256>(a, q_bf16, s);
}

}  // namespace bl
