// Launchers and argument records of the operators around a model's blocks: pages and slots of a step,
// embedding rows and their gradient, products with 4-bit weights, sampling.  Arguments are validated
// by step_api.hip.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bitlinear.h"

namespace bl {

// ---- pages and slots of a step ----
struct KvStepArgs {
  const int32_t* cached;
  const int32_t* fresh;
  int32_t* blocks;
  int32_t* free_pages;
  const int32_t* count;
  int32_t* count_out;
  int32_t* seq;
  int32_t* pos;
  int64_t* slot;         // nullptr: not wanted
  int32_t* lens;
  int32_t* starts;
  int64_t B, per, cap, T;
  uint32_t page;
};
hipError_t launch_kv_step(const KvStepArgs& a, hipStream_t s);

// ---- embedding ----
constexpr int64_t kEmbedMaxK = 32768;

struct EmbedArgs {
  const void* table;
  const int32_t* ids;
  void* y;
  float scale;
  int64_t V;
  int32_t T, K;
};
hipError_t launch_embed(const EmbedArgs& a, bool table_bf16, bool y_bf16, hipStream_t s);

// Workspace of the gradient, segments 256-byte aligned:
//   chunk_id, chunk_tok  [chunks * kEmbedChunk] ids of a chunk of tokens in order, and their tokens
//   span_id, span_tok    [T] the same of spans of chunks
//   id, tok              the same of all tokens: what the last of the steps that there are wrote
//   runs                 [1 + 2 * (T / kEmbedLong + 1)] long runs: their number, then first position and id
//   part                 [tiles][2][K] sums of the pieces of long runs
constexpr int kEmbedChunkBits = 11;
constexpr int kEmbedChunk = 1 << kEmbedChunkBits;   // tokens that a block sorts
constexpr int kEmbedSpan = 32;      // chunks
constexpr int kEmbedTile = 16;      // sorted positions a wave takes
constexpr int kEmbedLong = 32;      // a run of more positions is summed in pieces

struct EmbedBwdWs {
  int64_t chunks, tiles;
  size_t chunk_id, chunk_tok, span_id, span_tok, id, tok, runs, part, total;
};
inline EmbedBwdWs embed_bwd_ws(int64_t T, int64_t K) {
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  EmbedBwdWs w = {};
  w.chunks = (T + kEmbedChunk - 1) / kEmbedChunk;
  w.tiles = (T + kEmbedTile - 1) / kEmbedTile;
  const size_t all = up((size_t)(w.chunks * kEmbedChunk) * 4);
  size_t off = 0;
  w.chunk_id = off; off += all;
  w.chunk_tok = off; off += all;
  w.id = w.chunk_id; w.tok = w.chunk_tok;
  if (w.chunks > 1) {
    w.span_id = off; off += up((size_t)T * 4);
    w.span_tok = off; off += up((size_t)T * 4);
    if (w.chunks <= kEmbedSpan) {              // else from the spans' back into the chunks'
      w.id = w.span_id; w.tok = w.span_tok;
    }
  }
  w.runs = off; off += up((size_t)(1 + 2 * (T / kEmbedLong + 1)) * 4);
  w.part = off;
  if (T > kEmbedLong) off += up((size_t)w.tiles * 2 * (size_t)K * 4);
  w.total = off;
  return w;
}

struct EmbedBwdArgs {
  const void* dy;
  const int32_t* ids;
  float* dtable;
  float scale;
  int32_t accumulate;
  int64_t V, T;
  int32_t K;
  char* ws;
};
hipError_t launch_embed_bwd(const EmbedBwdArgs& a, bool dy_bf16, hipStream_t s);

// ---- weights in 4 bits ----
struct Q4PackArgs {
  const void* W;
  uint32_t* codes;
  uint16_t* scales;
  int64_t n, K;
  int64_t tiles, blocks;   // of 16 rows, of 128 columns
  int32_t group;
};
hipError_t launch_q4_pack(const Q4PackArgs& a, bool bf16, hipStream_t s);

struct Q4Args {
  const int8_t* xq;
  const float* x_scale;
  const uint8_t* codes;
  const uint16_t* scales;
  float* y;
  int64_t n, tiles;
  int32_t T, K, blocks;
  int32_t chunk, ksplit, token_tiles;   // set by the launcher
};
hipError_t launch_q4_fwd(const Q4Args& a, int group, hipStream_t s);

// ---- sampling ----
constexpr int kSampleBins = 1024;
constexpr int kSampleChunks = 16;   // of a row, at most
constexpr int kSampleList = 4096;   // tokens that a row's questions are answered from

// What a row's questions need, and where they start from.
struct SamplePlan {
  int32_t bin0[3], bin1[3];                  // bins of the tokens to gather
  uint32_t ranges;                           // 0: too many tokens
  uint32_t upto;                             // tokens from the row's largest on to the last of them
  uint32_t count, arrived;                   // gathered tokens, blocks of the launch that are done
};

struct SampleArgs {
  const void* x;
  int64_t stride, B, V;
  const float* temperature;   // nullptr: 1
  const int32_t* top_k;       // nullptr: off, like the next two
  const float* top_p;
  const float* min_p;
  const double* u;
  int32_t* token;
  float* logprob;             // nullptr: not wanted
  int64_t chunk, chunks;      // of a row: logits each, number
  // workspace, [B][chunks] each
  unsigned long long* top;    // largest logit and its index
  unsigned long long* kept;   // weights that min-p keeps
  double* exps;               // exp(x - the row's largest)
  unsigned long long* w_bins; // [kSampleBins] weights
  uint32_t* n_bins;           // [kSampleBins] tokens
  float* least;               // least finite logit
  float* most;                // [B][groups] largest logit of each 64
  int64_t groups;
  unsigned long long* lists;  // [B][kSampleList] gathered tokens
  SamplePlan* plan;           // [B]
  unsigned long long* sums;   // [B][kSampleBins][2] running sums by bin: weights, tokens
};
// Fills chunk and chunks, and the workspace's pointers from ws; returns its bytes.
inline size_t sample_split(SampleArgs& a, char* ws) {
  // two blocks per CU from all rows together, of 4096 logits at least (64 rows of 131072, mixed settings: 61 us of
  // kernels, 66 with four, 61 with one)
  int64_t most = 512 / (a.B > 0 ? a.B : 1);
  most = most < 4 ? 4 : most > kSampleChunks ? kSampleChunks : most;
  a.chunk = ((a.V + most - 1) / most + 4095) / 4096 * 4096;
  a.chunks = (a.V + a.chunk - 1) / a.chunk;
  const size_t n = (size_t)a.B * (size_t)a.chunks;
  size_t off = 0;
  auto part = [&](size_t bytes) {
    char* p = ws + off;
    off += (bytes + 255) / 256 * 256;
    return p;
  };
  a.top = (unsigned long long*)part(n * 8);
  a.kept = (unsigned long long*)part(n * 8);
  a.exps = (double*)part(n * 8);
  a.w_bins = (unsigned long long*)part(n * kSampleBins * 8);
  a.n_bins = (uint32_t*)part(n * kSampleBins * 4);
  a.least = (float*)part(n * 4);
  a.groups = (a.V + 63) / 64;
  a.most = (float*)part((size_t)a.B * (size_t)a.groups * 4);
  a.lists = (unsigned long long*)part((size_t)a.B * kSampleList * 8);
  a.plan = (SamplePlan*)part((size_t)a.B * sizeof(SamplePlan));
  a.sums = (unsigned long long*)part((size_t)a.B * kSampleBins * 16);
  return off;
}
hipError_t launch_sample(const SampleArgs& a, bool bf16, bool vec, hipStream_t s);

}  // namespace bl
