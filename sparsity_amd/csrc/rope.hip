// Rotary positions on the heads of several tensors, and the same fused with the write of a step's
// keys and values into a paged cache.
//
// The first R elements of a head are R/2 pairs, (i, i + R/2) in the half layout and (2i, 2i + 1) in
// the interleaved one; with (c, s) the cosine and sine of pos * freq[i],
//   y_a = x_a c - x_b s        y_b = x_b c + x_a s         (s negated for the inverse, the gradient)
// and the elements from R on pass through.  Products and sums are separate fp32 operations, so a
// result does not depend on the layout or the kernel variant.  cos and sin come from a table by
// position that is computed once in fp64: an angle of a long context, rounded to fp32 before its
// sine, would be off by pos * 2^-24 radians.
//
// One pass over the data, bound by memory: a block takes a token, a group of lanes a head at a
// time, and a lane the same pairs of every head it visits, so cos and sin are read once per lane.
// Measured (kernel time): 8192 tokens of 50 heads of 128, fp32 to bf16: 60.5 us, 5.3 TB/s (a large
// device copy: 5.2); asking for one head ahead is worth 3.4%, two or four heads at a time lose 1 to 5%.
// 1021 tokens of 40 bf16 heads of 80: 7.0 us, of which 2.6 us would be the bytes (a token of more than 512
// is one block, so its three rounds of heads follow one another).  Append of 4096
// tokens (48 heads of 128) to an int8 cache: 27 us, 5.4 TB/s; of 16 tokens: 4.2 us of latency.
//
// The int8 cache holds act_quant_i8's expressions per token and head (absmax / 127, round half to
// even) on the rotated key and on the value.
#include <algorithm>

#include "block_ops.hpp"
#include "device_common.hpp"

namespace bl {

namespace {

template <bool BF16>
__device__ __forceinline__ float load1(const void* p, int64_t off) {
  if constexpr (BF16) return __uint_as_float((uint32_t)((const uint16_t*)p)[off] << 16);
  else return ((const float*)p)[off];
}
template <bool BF16>
__device__ __forceinline__ void store1(void* p, int64_t off, float v) {
  if constexpr (BF16) ((uint16_t*)p)[off] = (uint16_t)pack_bf16(v, 0.f);
  else ((float*)p)[off] = v;
}

// Four consecutive elements, 4-element aligned.
template <bool BF16>
__device__ __forceinline__ void load4(const void* p, int64_t off, float v[4]) {
  if constexpr (BF16) {
    const uint2 u = *(const uint2*)((const uint16_t*)p + off);
    v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x); v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
  } else {
    const float4 u = *(const float4*)((const float*)p + off);
    v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
  }
}
template <bool BF16>
__device__ __forceinline__ void store4(void* p, int64_t off, const float v[4]) {
  if constexpr (BF16)
    *(uint2*)((uint16_t*)p + off) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
  else *(float4*)((float*)p + off) = make_float4(v[0], v[1], v[2], v[3]);
}

// A lane's eight elements of a head: two runs of four, at e0 and e1.  Rotated runs are four pairs:
// element k of run 0 with element k of run 1 (half layout), or consecutive elements of the eight
// (interleaved).
struct Item {
  int e0, e1;
  int pair0;      // first pair, or -1: elements that pass through
};
__device__ __forceinline__ Item item_of(int i, int R, bool inter) {
  Item it;
  if (8 * i < R) {
    it.pair0 = 4 * i;
    it.e0 = inter ? 8 * i : 4 * i;
    it.e1 = inter ? 8 * i + 4 : R / 2 + 4 * i;
  } else {
    it.pair0 = -1;
    it.e0 = 8 * i;
    it.e1 = 8 * i + 4;
  }
  return it;
}

__device__ __forceinline__ void rotate(float u[4], float w[4], const float (&c)[4],
                                       const float (&s)[4], bool inter) {
  if (inter) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float a = u[2 * k], b = u[2 * k + 1], d = w[2 * k], e = w[2 * k + 1];
      u[2 * k] = a * c[k] - b * s[k];
      u[2 * k + 1] = b * c[k] + a * s[k];
      w[2 * k] = d * c[k + 2] - e * s[k + 2];
      w[2 * k + 1] = e * c[k + 2] + d * s[k + 2];
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float a = u[k], b = w[k];
      u[k] = a * c[k] - b * s[k];
      w[k] = b * c[k] + a * s[k];
    }
  }
}

// cos and sin of four pairs of a position.  A position below zero is padding (its rows become
// zeros); one past the table has no entry, and its rows become NaN rather than a wrong rotation.
__device__ __forceinline__ void load_cs(const RopeArgs& a, int64_t pos, int pair0, float (&c)[4],
                                        float (&s)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) { c[k] = 1.f; s[k] = 0.f; }
  if (pair0 < 0 || pos < 0 || pos >= a.positions) return;
  const float4* p = (const float4*)(a.table + (pos * (a.R / 2) + pair0) * 2);
  const float4 lo = p[0], hi = p[1];
  c[0] = lo.x; s[0] = lo.y; c[1] = lo.z; s[1] = lo.w;
  c[2] = hi.x; s[2] = hi.y; c[3] = hi.z; s[3] = hi.w;
  if (a.inverse)
#pragma unroll
    for (int k = 0; k < 4; ++k) s[k] = -s[k];
}

__device__ __forceinline__ int tensor_of(const RopeArgs& a, int head) {
  int m = 0;
#pragma unroll
  for (int i = 1; i < kRopeMax; ++i)
    if (i < a.count && head >= a.t[i].head0) m = i;
  return m;
}

// LPH lanes per head (the power of two not below D / 8), 256 / LPH heads at a time, a lane eight
// elements.  APPEND: tensors 1 and 2 go to the cache.  VEC: D and R multiples of 8, rows aligned to
// four elements.  Otherwise (APPEND only, D a multiple of 8) a lane takes elements 8 i .. 8 i + 7 of
// any alignment and reads the other half of each pair itself, an element per access: 8192 tokens of 40 + 5
// + 5 heads of 80 take 125 us at R = 20, 50 at R = 80 by the vector form.
template <bool XBF, bool YBF, bool APPEND, bool VEC, int LPH>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a) {
  constexpr int HPB = 256 / LPH;
  const int i = threadIdx.x & (LPH - 1), slot = threadIdx.x / LPH;
  const int64_t t = blockIdx.x;
  const bool on = 8 * i < a.D;
  const Item it = VEC ? item_of(i, a.R, a.interleaved) : Item{8 * i, 8 * i + 4, -1};
  // a head's elements are asked for one head ahead, the first before the position and its cosines
  auto tensor = [&](int hd) {
    return APPEND ? (hd >= a.t[1].head0) + (hd >= a.t[2].head0) : tensor_of(a, hd);
  };
  auto fetch = [&](int hd, float (&u)[4], float (&w)[4]) {
    if (!on || hd >= a.heads) return;
    const RopeTensor& x = a.t[tensor(hd)];
    const int64_t r = t * x.x_tok + (hd - x.head0) * x.x_head;
    if constexpr (VEC) {
      load4<XBF>(x.x, r + it.e0, u);
      load4<XBF>(x.x, r + it.e1, w);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        u[k] = load1<XBF>(x.x, r + it.e0 + k);
        w[k] = load1<XBF>(x.x, r + it.e1 + k);
      }
    }
  };
  const int step = gridDim.y * HPB;
  int hd = blockIdx.y * HPB + slot;
  float u[4] = {}, w[4] = {}, un[4] = {}, wn[4] = {};
  fetch(hd, un, wn);
  const int64_t pos = a.pos[t];
  float c[4], s[4];
  load_cs(a, pos, on ? it.pair0 : -1, c, s);
  // element by element: its cosine, its sine with the sign it has there, the other half of its pair
  float ec[8], es[8];
  int other[8];
  if constexpr (!VEC) {
    const int half = a.R / 2;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int e = 8 * i + k;
      ec[k] = 1.f;
      es[k] = 0.f;
      other[k] = -1;
      if (!on || e >= a.R || pos < 0 || pos >= a.positions) continue;
      const bool first = a.interleaved ? !(e & 1) : e < half;
      const float* p = a.table + (pos * half + (a.interleaved ? e / 2 : first ? e : e - half)) * 2;
      ec[k] = p[0];
      es[k] = first != (a.inverse != 0) ? -p[1] : p[1];
      other[k] = a.interleaved ? e ^ 1 : first ? e + half : e - half;
    }
  }
  const bool known = pos < a.positions, pad = pos < 0;
  int64_t page = -1;
  int off = 0;
  if constexpr (APPEND) {
    const int64_t sq = a.seq ? a.seq[t] : t;
    if (known && !pad && sq >= 0 && sq < a.seqs) {
      const int64_t b = pos / a.kv.page_size;
      off = (int)(pos - b * a.kv.page_size);
      if (b < a.blocks_per_seq) page = a.blocks[sq * a.blocks_per_seq + b];
      if (page >= a.kv.pages) page = -1;    // not a page of this cache: nothing is written
    }
  }
  for (; hd < a.heads; hd += step) {
#pragma unroll
    for (int k = 0; k < 4; ++k) { u[k] = un[k]; w[k] = wn[k]; }
    fetch(hd + step, un, wn);
    const int m = tensor(hd);
    const RopeTensor& x = a.t[m];
    const int h = hd - x.head0;
    if constexpr (VEC) {
      if ((!APPEND || m < 2) && it.pair0 >= 0) rotate(u, w, c, s, a.interleaved);
    } else if (m < 2) {
      const int64_t r = t * x.x_tok + h * x.x_head;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (other[k] >= 0) {
          float& v = k < 4 ? u[k] : w[k - 4];
          v = v * ec[k] + load1<XBF>(x.x, r + other[k]) * es[k];
        }
    }
    // In place, a lane's store overwrites what another lane reads of the same pair.  A head's lanes belong to
    // one wave and come here together: every one of them has read before any writes.
    if constexpr (!VEC) {
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
    if (!APPEND || m == 0) {
      if (!known || pad) {
        const float v = pad ? 0.f : __builtin_nanf("");
#pragma unroll
        for (int k = 0; k < 4; ++k) u[k] = w[k] = v;
      }
      if (on) {
        const int64_t r = t * x.y_tok + h * x.y_head;
        if constexpr (VEC) {
          store4<YBF>(x.y, r + it.e0, u);
          store4<YBF>(x.y, r + it.e1, w);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            store1<YBF>(x.y, r + it.e0 + k, u[k]);
            store1<YBF>(x.y, r + it.e1 + k, w[k]);
          }
        }
      }
      continue;
    }
    if constexpr (APPEND) {
      const int64_t r = page * a.kv.page_stride + h * a.kv.head_stride + off * a.kv.tok_stride;
      void* base = m == 1 ? a.kv.k : a.kv.v;
      if (a.kv.dtype == BL_DTYPE_BF16) {
        if (page >= 0 && on) {
          store4<true>(base, r + it.e0, u);
          store4<true>(base, r + it.e1, w);
        }
      } else {
        uint32_t mx = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mx = max(mx, max(__float_as_uint(u[k]) & 0x7FFFFFFFu, __float_as_uint(w[k]) & 0x7FFFFFFFu));
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) mx = max(mx, (uint32_t)__shfl_xor((int)mx, o, LPH));
        const float amax = __uint_as_float(mx);
        const float q = amax > 0.f ? 127.f / amax : 0.f;
        if (page >= 0 && on) {
          int8_t* o = (int8_t*)base + r;
          *(uint32_t*)(o + it.e0) = q8(u[0], q) | (q8(u[1], q) << 8) | (q8(u[2], q) << 16) | (q8(u[3], q) << 24);
          *(uint32_t*)(o + it.e1) = q8(w[0], q) | (q8(w[1], q) << 8) | (q8(w[2], q) << 16) | (q8(w[3], q) << 24);
          if (i == 0)
            (m == 1 ? a.kv.k_scale : a.kv.v_scale)[(page * a.kv.heads + h) * a.kv.page_size + off] = amax / 127.f;
        }
      }
    }
  }
}

// Scalar form of rope (any even R, any D, any strides): a thread takes pairs, or single elements
// that pass through.  8192 tokens of 50 heads of 80, fp32 to bf16: 165 us at R = 20, 1.2 TB/s, for an
// element per access and a division per pair (47 us at R = 80 by the vector form).
template <bool XBF, bool YBF>
__global__ __launch_bounds__(256) void rope_scalar_kernel(RopeArgs a) {
  const int64_t t = blockIdx.x;
  const int64_t pos = a.pos[t];
  const bool ok = pos >= 0 && pos < a.positions;
  const int half = a.R / 2, per = half + (a.D - a.R);
  for (int64_t n = threadIdx.x; n < (int64_t)a.heads * per; n += 256) {
    const int hd = (int)(n / per), j = (int)(n - (int64_t)hd * per);
    const RopeTensor& x = a.t[tensor_of(a, hd)];
    const int h = hd - x.head0;
    const int64_t rx = t * x.x_tok + h * x.x_head, ry = t * x.y_tok + h * x.y_head;
    const float bad = pos < 0 ? 0.f : __builtin_nanf("");
    if (j >= half) {
      const int e = a.R + j - half;
      const float v = load1<XBF>(x.x, rx + e);
      store1<YBF>(x.y, ry + e, ok ? v : bad);
      continue;
    }
    const int ea = a.interleaved ? 2 * j : j, eb = a.interleaved ? 2 * j + 1 : half + j;
    const float va = load1<XBF>(x.x, rx + ea), vb = load1<XBF>(x.x, rx + eb);
    float c = 1.f, s = 0.f;
    if (ok) {
      const float* p = a.table + (pos * half + j) * 2;
      c = p[0];
      s = a.inverse ? -p[1] : p[1];
    }
    store1<YBF>(x.y, ry + ea, ok ? va * c - vb * s : bad);
    store1<YBF>(x.y, ry + eb, ok ? vb * c + va * s : bad);
  }
}

__global__ __launch_bounds__(256) void rope_table_kernel(const double* __restrict__ freq, int64_t half,
                                                         int64_t n, double mscale,
                                                         float* __restrict__ table) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  double sn, cs;
  sincos((double)(i / half) * freq[i % half], &sn, &cs);
  *(float2*)(table + 2 * i) = make_float2((float)(cs * mscale), (float)(sn * mscale));
}

template <bool XBF, bool YBF, bool APPEND, bool VEC>
hipError_t launch_rope_t(const RopeArgs& a, hipStream_t s) {
  const int lanes = a.D / 8;
  auto go = [&](auto lph) {
    constexpr int LPH = decltype(lph)::value;
    const int hpb = 256 / LPH, rounds = (a.heads + hpb - 1) / hpb;
    // few tokens: a block per round of heads, so the heads of a token run side by side
    const int y = (int)std::min<int64_t>(rounds, std::max<int64_t>(1, 1024 / a.T));
    rope_kernel<XBF, YBF, APPEND, VEC, LPH><<<dim3((unsigned)a.T, (unsigned)y), 256, 0, s>>>(a);
  };
  if (lanes <= 8) go(std::integral_constant<int, 8>{});
  else if (lanes <= 16) go(std::integral_constant<int, 16>{});
  else go(std::integral_constant<int, 32>{});
  return hipGetLastError();
}

}  // namespace

// Calls f with the two input types as compile-time booleans.
template <class F>
static hipError_t with_types(bool x, bool y, F&& f) {
  if (x) return y ? f(std::true_type{}, std::true_type{}) : f(std::true_type{}, std::false_type{});
  return y ? f(std::false_type{}, std::true_type{}) : f(std::false_type{}, std::false_type{});
}

hipError_t launch_rope(const RopeArgs& a, bool x_bf16, bool y_bf16, bool vec, hipStream_t s) {
  return with_types(x_bf16, y_bf16, [&](auto x, auto y) {
    constexpr bool X = decltype(x)::value, Y = decltype(y)::value;
    if (vec) return launch_rope_t<X, Y, false, true>(a, s);
    rope_scalar_kernel<X, Y><<<dim3((unsigned)a.T), 256, 0, s>>>(a);
    return hipGetLastError();
  });
}

hipError_t launch_rope_append(const RopeArgs& a, bool x_bf16, bool y_bf16, bool vec, hipStream_t s) {
  return with_types(x_bf16, y_bf16, [&](auto x, auto y) {
    constexpr bool X = decltype(x)::value, Y = decltype(y)::value;
    return vec ? launch_rope_t<X, Y, true, true>(a, s) : launch_rope_t<X, Y, true, false>(a, s);
  });
}

hipError_t launch_rope_table(const double* freq, int64_t half, int64_t positions, double mscale,
                             float* table, hipStream_t s) {
  const int64_t n = half * positions;
  rope_table_kernel<<<dim3((unsigned)((n + 255) / 256)), 256, 0, s>>>(freq, half, n, mscale, table);
  return hipGetLastError();
}

}  // namespace bl
