// Residual addition, root-mean-square norm and per-token int8 quantization in one pass, and the
// gradient through them.
//
//   h    = store(x + r)                      the residual stream, rounded once to its own type
//   rstd = fl32(1 / sqrt(sum(h^2) / K + eps))  squares in fp32, their sum and the root in fp64
//   n    = fl32(fl32(h * rstd) * w)
//   xq, scale = act_quant_i8's expressions on n (absmax / 127 per token, round half to even)
//
// BitNet b1.58 puts a norm in front of every quantized projection.  The sum is held in fp64 so that
// its order cannot move rstd by an ulp and an int8 value across a rounding boundary: the int8 rows
// are those of the definition whatever the split over lanes.  At 3 bytes per element (bf16,
// no residual) to 13 (fp32 onto an fp32 stream) the kernel is bound by memory; the fp64 adds are one
// instruction per element, a few percent of the rate it could issue.
//
// A row belongs to W waves; a lane holds pieces of eight elements, p = lane, lane + 64 W, ..., in
// registers from the first load to the int8 store, so every input byte is read once.
//
// Measured (kernel time): 8192 x 3200, fp32 onto a bf16 stream with rstd: 40 us, 5.9 TB/s of the 236 MB
// it has to move (a large device copy reaches 5.2 TB/s of reads and writes); 2048 x 4096 bf16 onto an
// fp32 stream with 6:8 rows: 19 us; one token of 2560: 3.0 us, the round trips of a single load.
#include <algorithm>

#include "block_ops.hpp"
#include "device_common.hpp"

namespace bl {

namespace {

// Lifted output of one quantized row (in LDS) for (M-2):M windows: dword j = g * (M/2 - 1) + w
// holds q[M g + 2 w .. M g + 2 w + 3].  M is even, so the source is 2-byte aligned.
__device__ __forceinline__ uint32_t lifted_dword(const int8_t* row, int j, int M) {
  const int nw = M / 2 - 1;
  const int g = j / nw, w = j - g * nw;
  const uint16_t* p = (const uint16_t*)(row + M * g + 2 * w);
  return (uint32_t)p[0] | ((uint32_t)p[1] << 16);
}

// RES: 0 no residual, 1 fp32, 2 bf16.  W waves per row (1: four rows per block of four waves), P
// pieces per lane at most.
template <bool XBF, int RES, int W, int P>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void norm_quant_kernel(NormArgs a) {
  constexpr int RPB = W == 1 ? 4 : 1;       // rows per block
  extern __shared__ __attribute__((aligned(16))) int8_t sm_row[];   // lifted: RPB rows of K bytes
  __shared__ double red_s[W];
  __shared__ uint32_t red_m[W];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t_raw = (int64_t)blockIdx.x * RPB + (W == 1 ? wave : 0);
  const bool live = t_raw < a.T;
  const int64_t t = live ? t_raw : a.T - 1;  // a spare wave recomputes the last row, stores nothing
  const int K = a.K, pieces = K / 8;
  const size_t row = (size_t)t * K;
  const int p0 = W == 1 ? lane : (int)threadIdx.x;

  float h[P][8], r[RES ? P : 1][8], w[P][8];
#pragma unroll
  for (int i = 0; i < P; ++i) {            // every load of the row before the first use
    const int p = p0 + 64 * W * i;
    if (p < pieces) {
      load_f8<XBF>(a.x, row + 8 * p, h[i]);
      if constexpr (RES != 0) load_f8<RES == 2>(a.res, row + 8 * p, r[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[i][j] = 0.f;
        if constexpr (RES != 0) r[i][j] = 0.f;
      }
    }
    if (p < pieces && a.w) load_f8<false>(a.w, 8 * p, w[i]);
    else
#pragma unroll
      for (int j = 0; j < 8; ++j) w[i][j] = 1.f;
  }
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int p = p0 + 64 * W * i;
    if constexpr (RES != 0)
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] += r[i][j];
    if constexpr (RES == 2) {               // the stream's stored value is what is normed
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const uint32_t u = pack_bf16(h[i][j], h[i][j + 1]);
        h[i][j] = bf16_lo(u);
        h[i][j + 1] = bf16_hi(u);
      }
    }
    if constexpr (RES != 0)
      if (p < pieces && live) store_f8<RES == 2>(a.h, row + 8 * p, h[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += (double)(h[i][j] * h[i][j]);
  }
  sum = wave_sum_f64(sum);
  if constexpr (W > 1) {
    if (lane == 0) red_s[wave] = sum;
    __syncthreads();
    sum = 0.0;
#pragma unroll
    for (int i = 0; i < W; ++i) sum += red_s[i];
  }
  const float rstd = (float)(1.0 / sqrt(sum / K + a.eps));
  uint32_t mx = 0;
#pragma unroll
  for (int i = 0; i < P; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      h[i][j] = h[i][j] * rstd * w[i][j];
      mx = max(mx, __float_as_uint(h[i][j]) & 0x7FFFFFFFu);
    }
  mx = wave_max_u32(mx);
  if constexpr (W > 1) {
    if (lane == 0) red_m[wave] = mx;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < W; ++i) mx = max(mx, red_m[i]);
  }
  const float amax = __uint_as_float(mx);
  const float s = amax > 0.f ? 127.f / amax : 0.f;
  int8_t* lrow = sm_row + (size_t)(W == 1 ? wave : 0) * K;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int p = p0 + 64 * W * i;
    if (p >= pieces) continue;
    uint32_t q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = q8(h[i][j], s);
    const uint2 o = make_uint2(q[0] | (q[1] << 8) | (q[2] << 16) | (q[3] << 24),
                               q[4] | (q[5] << 8) | (q[6] << 16) | (q[7] << 24));
    if (a.lift_M) *(uint2*)(lrow + 8 * p) = o;
    else if (live) *(uint2*)(a.xq + row + 8 * p) = o;
  }
  if (a.lift_M) {
    __syncthreads();
    const int M = a.lift_M, n4 = K / M * (M / 2 - 1);
    uint32_t* o = (uint32_t*)(a.xq + (size_t)t * n4 * 4);
    if (live)
      for (int j = p0; j < n4; j += 64 * W) o[j] = lifted_dword(lrow, j, M);
  }
  if (live && p0 == 0) {
    a.scale[t] = amax / 127.f;
    if (a.rstd) a.rstd[t] = rstd;
  }
}

template <bool XBF, int RES, int W, int P>
void launch_norm_wp(const NormArgs& a, hipStream_t s) {
  constexpr int RPB = W == 1 ? 4 : 1;
  const dim3 grid((unsigned)((a.T + RPB - 1) / RPB)), block(W == 1 ? 256 : 64 * W);
  norm_quant_kernel<XBF, RES, W, P><<<grid, block, a.lift_M ? (size_t)RPB * a.K : 0, s>>>(a);
}

// Waves per row.  Many rows: the fewest that leave a lane two pieces (8192 x 3200: four waves 44.6 us,
// two 49.5, one 54.2, sixteen 62.1; 10922 x 1536: two 21.9, four 24.0).  Few rows, where latency counts: one piece per lane, up to eight
// waves (1 x 2560: eight 3.07 us, four 3.27, sixteen 3.60; 1 x 8192: eight 3.80, sixteen 4.13).
template <bool XBF, int RES>
hipError_t launch_norm_t(const NormArgs& a, hipStream_t s) {
  const int pieces = a.K / 8, most = a.T < 1024 ? 64 : 128;   // pieces per wave
  if (pieces <= 64) launch_norm_wp<XBF, RES, 1, 1>(a, s);
  else if (pieces <= most) launch_norm_wp<XBF, RES, 1, 2>(a, s);
  else if (pieces <= 256 && a.T >= 1024) launch_norm_wp<XBF, RES, 2, 2>(a, s);
  else if (pieces <= 256) launch_norm_wp<XBF, RES, 4, 1>(a, s);
  else if (pieces <= 4 * most) launch_norm_wp<XBF, RES, 4, 2>(a, s);
  else if (pieces <= 512) launch_norm_wp<XBF, RES, 8, 1>(a, s);
  else if (pieces <= 1024) launch_norm_wp<XBF, RES, 8, 2>(a, s);
  else if (pieces <= 2048) launch_norm_wp<XBF, RES, 16, 2>(a, s);
  else launch_norm_wp<XBF, RES, 16, 4>(a, s);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_quant(const NormArgs& a, bool x_bf16, bool res_bf16, hipStream_t s) {
  const int res = !a.res ? 0 : res_bf16 ? 2 : 1;
  if (x_bf16)
    return res == 0 ? launch_norm_t<true, 0>(a, s)
                    : res == 1 ? launch_norm_t<true, 1>(a, s) : launch_norm_t<true, 2>(a, s);
  return res == 0 ? launch_norm_t<false, 0>(a, s)
                  : res == 1 ? launch_norm_t<false, 1>(a, s) : launch_norm_t<false, 2>(a, s);
}

// ---------------------------------------------------------------------------------------------
// Gradient.  With nh = h * rstd and gw = dn * w:
//   dh = rstd * (gw - nh * mean(gw * nh)) (+ dres)        dw = sum over tokens of dn * nh
// (rounding and clipping of the quantizer pass the gradient through unchanged).  dh is the gradient
// of both addends of h.  dw is summed in a fixed order, so it does not vary from run to run, in one of
// two ways.  Many rows: each block walks rows and keeps its columns' sums in registers, and a second
// launch adds the blocks'.  Few rows: blocks of their own read dn and h once more, from the caches, and
// sum 64 columns each over all rows, in the same launch and without a workspace.
// Teams of W waves take a row each, 16 waves a block, one block per CU: two per CU read no faster and
// double the sums (6553 x 2560: 41.8 us against 39.8, 1638 x 2560: 17.7 against 14.4).  Two rows per team
// at a time gain nothing (39.6), a row asked for ahead spills and more than doubles the time.
//
// Measured: 8192 x 3200, fp32 dn, bf16 h, dres and dh: 48 us for the rows, 5.5 TB/s, 4.7 us for dw.
// More than 16384 columns: a lane's four pieces and their dw sums do not fit its 128 registers, and each
// row spills, 184 to 476 bytes a lane: 1024 x 16384 40 us, x 20480 463, x 28672 629 (bf16 dn 157), x 32768
// 717.
// ---------------------------------------------------------------------------------------------
namespace {

// dw of 64 columns: eight lanes of eight columns, 128 rows at a time, the 128 joined in LDS.
constexpr int kColumns = 64;
constexpr size_t kColumnLds = (128 + 16) * kColumns * sizeof(float);

template <bool GBF, bool HBF>
__device__ __forceinline__ void dw_columns(const NormBwdArgs& a, int block, float* lds) {
  const int c = threadIdx.x & 7, r = threadIdx.x >> 3;
  const int k = block * kColumns + 8 * c;
  float s[8] = {};
  if (k < a.K) {
#pragma unroll 4
    for (int64_t t = r; t < a.T; t += 128) {
      float g[8], h[8];
      const float rstd = a.rstd[t];
      load_f8<GBF>(a.dn, (size_t)t * a.K + k, g);
      load_f8<HBF>(a.h, (size_t)t * a.K + k, h);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] += g[j] * (h[j] * rstd);
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) lds[r * kColumns + 8 * c + j] = s[j];
  __syncthreads();
  const int col = threadIdx.x % kColumns, part = threadIdx.x / kColumns;   // 16 parts of eight rows
  float v = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) v += lds[(8 * part + i) * kColumns + col];
  float* join = lds + 128 * kColumns;
  join[part * kColumns + col] = v;
  __syncthreads();
  if (part == 0 && block * kColumns + col < a.K) {
#pragma unroll
    for (int i = 1; i < 16; ++i) v += join[i * kColumns + col];
    a.dw[block * kColumns + col] = v;
  }
}

template <bool GBF, bool HBF, bool OBF, int W, int P>
__global__ __launch_bounds__(1024) void norm_bwd_kernel(NormBwdArgs a) {
  constexpr int RPB = 16 / W;               // row teams of W waves
  __shared__ float red[2][16];
  extern __shared__ __attribute__((aligned(16))) float sm_dw[];   // [K], or dw_columns' sums
  if ((int)blockIdx.x >= a.blocks) {        // the blocks behind those of the rows
    dw_columns<GBF, HBF>(a, blockIdx.x - a.blocks, sm_dw);
    return;
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int team = wave / W;
  const int K = a.K, pieces = K / 8;
  const int p0 = threadIdx.x - team * 64 * W;
  float dw[P][8] = {};
  // weights in registers; with four pieces per lane they are read again per row (and the rest still spills)
  constexpr bool KEEP = P <= 2;
  float w[P][8];
  auto weights = [&]() {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int p = p0 + 64 * W * i;
      if (p < pieces && a.w) load_f8<false>(a.w, 8 * p, w[i]);
      else
#pragma unroll
        for (int j = 0; j < 8; ++j) w[i][j] = 1.f;
    }
  };
  if constexpr (KEEP) weights();
  const int step = a.blocks * RPB;
  int flip = 0;
  for (int t0 = blockIdx.x * RPB; t0 < a.T; t0 += step) {   // uniform over the block
    const int t = t0 + team;
    const bool live = t < a.T;
    const size_t row = (size_t)(live ? t : a.T - 1) * K;
    float g[P][8], h[P][8];
    const float rstd = a.rstd[live ? t : a.T - 1];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int p = p0 + 64 * W * i;
      if (p < pieces && live) {
        load_f8<GBF>(a.dn, row + 8 * p, g[i]);
        load_f8<HBF>(a.h, row + 8 * p, h[i]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) g[i][j] = h[i][j] = 0.f;
      }
    }
    float dot = 0.f;
    if constexpr (!KEEP) weights();
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[i][j] *= rstd;
        dw[i][j] += g[i][j] * h[i][j];
        g[i][j] *= w[i][j];
        dot += g[i][j] * h[i][j];
      }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) dot += __shfl_xor(dot, o, 64);
    if constexpr (W > 1) {
      if (lane == 0) red[flip][wave] = dot;
      __syncthreads();                      // the two slots alternate: one barrier per row
      dot = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) dot += red[flip][team * W + i];
      flip ^= 1;
    }
    const float c = dot / (float)K;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int p = p0 + 64 * W * i;
      if (p >= pieces || !live) continue;
      float o[8];
      if (a.dres) load_f8<OBF>(a.dres, row + 8 * p, o);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float v = rstd * (g[i][j] - h[i][j] * c);
        o[j] = a.dres ? v + o[j] : v;
      }
      store_f8<OBF>(a.dh, row + 8 * p, o);
    }
  }
  if (!a.part) return;
  // the teams' sums one after another into LDS, in team order
  for (int k = 0; k < RPB; ++k) {
    if (team == k) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int p = p0 + 64 * W * i;
        if (p >= pieces) continue;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float v = k ? sm_dw[8 * p + j] + dw[i][j] : dw[i][j];
          if (k == RPB - 1) a.part[(size_t)blockIdx.x * K + 8 * p + j] = v;
          else sm_dw[8 * p + j] = v;
        }
      }
    }
    __syncthreads();
  }
}

// dw[k] = sum over blocks of part[block][k]: 8 lanes of four columns, 32 row groups, joined in LDS
__global__ __launch_bounds__(256) void norm_dw_kernel(const float* __restrict__ part, int blocks,
                                                      int K, float* __restrict__ dw) {
  constexpr int C = 8, R = 32;
  __shared__ v4f red[R][C];
  const int c = threadIdx.x % C, r = threadIdx.x / C;
  const int k = (blockIdx.x * C + c) * 4;
  v4f s = v4f{0.f, 0.f, 0.f, 0.f};
  if (k < K)
#pragma unroll 8
    for (int b = r; b < blocks; b += R) s += *(const v4f*)(part + (size_t)b * K + k);
  red[r][c] = s;
  __syncthreads();
  if (r == 0 && k < K) {
#pragma unroll
    for (int i = 1; i < R; ++i) s += red[i][c];
    *(v4f*)(dw + k) = s;
  }
}

// As many waves per row as leave few lanes without a piece, up to two pieces each (4088 x 4104: 16 waves of
// one piece 47 us, eight of two 39; 31775 x 528: four waves 69 us, two 47).
template <bool GBF, bool HBF, bool OBF>
hipError_t launch_rows(const NormBwdArgs& a, int columns, hipStream_t s) {
  const int pieces = a.K / 8;
  const dim3 grid((unsigned)(a.blocks + columns)), block(1024);
  if (grid.x == 0) return hipSuccess;
  // more than 1024 pieces: one team, no sums to join
  const size_t lds = columns ? kColumnLds : a.part && pieces <= 1024 ? (size_t)a.K * 4 : 0;
  if (pieces <= 64) norm_bwd_kernel<GBF, HBF, OBF, 1, 1><<<grid, block, lds, s>>>(a);
  else if (pieces <= 128) norm_bwd_kernel<GBF, HBF, OBF, 2, 1><<<grid, block, lds, s>>>(a);
  else if (pieces <= 256) norm_bwd_kernel<GBF, HBF, OBF, 4, 1><<<grid, block, lds, s>>>(a);
  else if (pieces <= 512) norm_bwd_kernel<GBF, HBF, OBF, 4, 2><<<grid, block, lds, s>>>(a);
  else if (pieces <= 1024) norm_bwd_kernel<GBF, HBF, OBF, 8, 2><<<grid, block, lds, s>>>(a);
  else if (pieces <= 2048) norm_bwd_kernel<GBF, HBF, OBF, 16, 2><<<grid, block, lds, s>>>(a);
  else norm_bwd_kernel<GBF, HBF, OBF, 16, 4><<<grid, block, lds, s>>>(a);
  return hipGetLastError();
}

template <bool GBF, bool HBF, bool OBF>
hipError_t launch_bwd_t(NormBwdArgs a, hipStream_t s) {
  if (a.dw && !a.part) {
    const int columns = (a.K + kColumns - 1) / kColumns, rows = a.blocks;
    if (a.dh != a.dn) return launch_rows<GBF, HBF, OBF>(a, columns, s);
    // in place over dn: the columns have to be read before
    a.blocks = 0;
    const hipError_t e = launch_rows<GBF, HBF, OBF>(a, columns, s);
    a.blocks = rows;
    return e != hipSuccess ? e : launch_rows<GBF, HBF, OBF>(a, 0, s);
  }
  const hipError_t e = launch_rows<GBF, HBF, OBF>(a, 0, s);
  if (e != hipSuccess || !a.dw) return e;
  norm_dw_kernel<<<dim3((unsigned)((a.K + 31) / 32)), 256, 0, s>>>(a.part, a.blocks, a.K, a.dw);
  return hipGetLastError();
}

}  // namespace

int norm_bwd_blocks(int64_t T, int64_t K) {
  const int64_t pieces = K / 8;
  // rows a block takes at a time
  const int64_t rows = pieces <= 64 ? 16 : pieces <= 128 ? 8 : pieces <= 512 ? 4 : pieces <= 1024 ? 2 : 1;
  return (int)std::min<int64_t>(256, (T + rows - 1) / rows);
}

// By columns while a block's walk over the rows is short and the second reading comes from the caches.
// One launch against two, graph replays (calls one after another): 64 x 2560 4.3 us against 7.5 (10.8
// against 15.1), 512 x 2560 6.6 against 10.0, 512 x 8192 13.6 against 15.2; 1024 x 2560 13.2 against
// 12.0, 2048 x 512 13.3 against 8.6, 2048 x 8192 45 against 38.
bool norm_bwd_columns(int64_t T, int64_t K) { return T <= 768 && T * K <= (int64_t)1 << 22; }

hipError_t launch_norm_bwd(const NormBwdArgs& a, bool dn_bf16, bool h_bf16, bool grad_bf16,
                           hipStream_t s) {
  if (dn_bf16) {
    if (h_bf16) return grad_bf16 ? launch_bwd_t<true, true, true>(a, s) : launch_bwd_t<true, true, false>(a, s);
    return grad_bf16 ? launch_bwd_t<true, false, true>(a, s) : launch_bwd_t<true, false, false>(a, s);
  }
  if (h_bf16) return grad_bf16 ? launch_bwd_t<false, true, true>(a, s) : launch_bwd_t<false, true, false>(a, s);
  return grad_bf16 ? launch_bwd_t<false, false, true>(a, s) : launch_bwd_t<false, false, false>(a, s);
}

}  // namespace bl
