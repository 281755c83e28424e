// Internal launch interface of the operators around the expert layer, between
// the C ABI (api.cpp) and their kernels. Not part of the public ABI.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxgg {

// --- layer norm ------------------------------------------------------------
constexpr int64_t kNormMaxCols = 16384;

struct NormFwdParams {
  const void* x;
  const void* weight;  // NULL: 1
  const void* bias;    // NULL: 0
  void* y;
  float* mean;
  float* rstd;
  int64_t rows, ldx, ldy;
  int32_t cols;
  float eps;
};
struct NormBwdParams {
  const void* dy;
  const void* x;
  const void* weight;  // NULL: 1
  const float* mean;
  const float* rstd;
  void* dx;
  float* part;         // [workgroups][2][cols] column sums
  int64_t rows, lddy, ldx, lddx;
  int32_t cols;
};
// workgroups of the backward pass at most: one partial sum of both gradients
// each
int norm_bwd_groups(int64_t rows);
hipError_t launch_layer_norm_fwd(const NormFwdParams& p, bool f32, bool wf32, hipStream_t st);
// dweight / dbias: fp32 [cols] or NULL
hipError_t launch_layer_norm_bwd(const NormBwdParams& p, bool f32, bool wf32, float* dweight, float* dbias,
                                 bool accumulate, hipStream_t st);

// --- gradient norm and clipping --------------------------------------------
// Tensors of one launch: they travel as kernel arguments, so a call needs no
// device copy of the caller's pointer list.
constexpr int kClipTensors = 192;
constexpr int kClipChunk = 8192;      // elements of one tensor that a workgroup takes at a time
constexpr int kClipGroups = 1024;     // workgroups (and partial norms) of a launch at most
struct ClipBatch {
  int32_t n;
  int32_t chunks;                     // == first[n]
  int32_t first[kClipTensors + 1];    // first chunk of each tensor
  int64_t numel[kClipTensors];
  void* data[kClipTensors];
  uint32_t f32[kClipTensors / 32];    // bit i: tensor i is fp32, else bf16
};
inline int clip_groups(int32_t chunks) { return chunks < kClipGroups ? chunks : kClipGroups; }
// one partial norm (sum of squares, or the largest magnitude) per workgroup
hipError_t launch_norm_partials(const ClipBatch& b, bool max_norm_kind, double* part, hipStream_t st);
// norm of the n partials -> *total
hipError_t launch_norm_total(const double* part, int n, bool max_norm_kind, float* total, hipStream_t st);
// data *= min(1, max_norm / (norm + 1e-6)); the norm is that of the n partials
// (written to *total too when `write`), or *total itself when n == 0
hipError_t launch_clip(const ClipBatch& b, const double* part, int n, bool max_norm_kind, float max_norm, float* total,
                       bool write, hipStream_t st);

// --- the expert layer for a few tokens ---------------------------------------
constexpr int kMoeTokens = 64;        // an expert's tokens are the bits of one 64-bit word
constexpr int kMoeTopK = 16;
constexpr int kMoeDownGroups = 256;   // workgroups that the second product is split for

// A chosen expert and some of its tokens: `tokens` rows of the inner activation
// from `base` on (an expert's rows follow each other in the order of its
// tokens).
struct MoeSegment {
  int32_t expert, base, tokens, unused;
};
// Weight and token of one row.
struct MoeRow {
  float weight;
  int32_t token;
};
// Every chosen expert has one segment that is not full at most; a segment has
// room for at least 4 tokens.
inline int64_t moe_most_segments(int64_t tokens, int64_t experts, int64_t top_k, int64_t segment = 4) {
  const int64_t rows = tokens * top_k;
  return rows / segment + (rows < experts ? rows : experts);
}
// Workspace: how many segments there are, their list, the rows,
// the second product's parts and the inner activation, bf16 (laid out as its
// reader takes it: inner_at in moe_layer.hip).
struct MoeWorkspace {
  size_t segments, rows, parts, inner, bytes;
};
inline MoeWorkspace moe_workspace(int64_t tokens, int64_t experts, int64_t top_k, int64_t inner) {
  const auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  MoeWorkspace w;
  w.segments = 256;
  w.rows = w.segments + up((size_t)moe_most_segments(tokens, experts, top_k) * sizeof(MoeSegment));
  w.parts = w.rows + up((size_t)(tokens * top_k) * sizeof(MoeRow));
  // fp32 [splits, tokens, hidden], splits * hidden <= 64 kMoeDownGroups when
  // there is more than one
  w.inner = w.parts + up((size_t)tokens * 64 * kMoeDownGroups * 4);
  // whole pieces of 128 elements: the second product reads whole ones
  w.bytes = w.inner + up((size_t)(tokens * top_k) * (size_t)((inner + 127) / 128 * 128) * 2);
  return w;
}
struct MoeParams {
  const uint16_t* x;
  const void* logits;
  const uint8_t* w13_q;
  const void* w13_s;
  const uint8_t* w2_q;
  const void* w2_s;
  uint16_t* out;
  int32_t* ids;
  float* weights;
  // workspace
  int32_t* count;                     // of the segments
  MoeSegment* segments;
  MoeRow* row_list;
  uint16_t* inner_x;
  float* parts;
  int64_t ldx, ldl;
  bool logits_f32, renormalize;
  int32_t tokens, experts, top_k, hidden, inner;
  int32_t rows;                       // of the inner activation: tokens * top_k
  // the plan of a call (moe_plan): tokens of a segment, 1 KiB loads that bring
  // a piece of them, segments at most, 16-row tiles of a wave in
  // the second product and the parts that its segments are split into
  int32_t segment, dmas, most_segments;
  int32_t down_tiles, splits;
  // byte strides of the codes: between rows, and between the 64-byte pieces of
  // a row; of the MX scales: between blocks of 32
  int64_t q13_row, q13_piece, s13_block, q2_row, q2_piece, s2_block;
};
enum MoeFormat { kMoeFp4 = 0, kMoeFp8 = 1, kMoeBlock = 2 };
// How a call is cut.
//
// Segments: one of few tokens leaves more of the LDS to weights in flight, one of
// many reads an expert's weights less often (again out of the caches). So about
// the tokens of a chosen expert and half as many more, for the spread of chance:
// with just their mean the whole layer took 91 us instead of 78 (32 tokens, 32
// experts of 4096 x 1536 in MXFP4) and 583 instead of 506 (64 tokens, 64 experts
// of 7168 x 2048, blockwise). With E2M1 codes a 1 KiB load brings 4 tokens'
// piece, with E4M3 codes 8.
//
// Second product: a wave's 16 rows of weights cost as much in loads of tokens as
// 64 do. With few tokens that is little, and 16-row tiles give four times the
// workgroups without a launch that adds parts up; hidden / 16 of them, so every CU
// has one from 4096 outputs on, and narrower layers leave some idle. Otherwise the
// tiles are 64 rows and the segments are split over workgroups, at most 8 parts,
// added up after. Both sides, whole layer in us, 32 experts of 1536, top 8, MXFP4:
//   outputs     1024         2048         4096         6144          7168
//   tokens    16   64      16   64      16   64      16   64       16   64 rows
//      1     20.7 22.1    22.8 25.2    26.8 30.3    37.0 36.9     41.3 41.5
//      4     35.8 33.7    40.7 40.3    54.3 56.8    78.4 74.8     85.6 81.6
//     16     41.2 36.4    54.2 47.2    74.3 71.3   112.9 98.4    124.2 109.6
// The rule has the better side of one token and of the wide layers; at 16 tokens
// below 6144 outputs the other would be 4 to 13 % faster. 8 tokens, 128 experts,
// 7168 outputs: 128 us, 16-row tiles 136. The split itself: 64 tokens, blockwise, 7168
// outputs 506 us, without it 570; 32 tokens, 4096 outputs 78 and 114.
inline void moe_plan(MoeParams& p, MoeFormat fmt) {
  const int each = fmt == kMoeFp4 ? 4 : 8, most = fmt == kMoeFp4 ? 3 : 2;
  const int chosen = p.rows < p.experts ? p.rows : p.experts;
  const int want = p.tokens <= each ? p.tokens : (3 * p.rows + 2 * chosen - 1) / (2 * chosen) + 1;
  p.dmas = (want + each - 1) / each;
  if (p.dmas > most) p.dmas = most;
  p.segment = p.dmas * each;
  p.most_segments = (int32_t)moe_most_segments(p.tokens, p.experts, p.top_k, p.segment);
  if (p.tokens <= 16 && p.dmas <= 2 && p.hidden < 6144) {
    p.down_tiles = 1;
    p.splits = 1;
  } else {
    p.down_tiles = 4;
    p.splits = kMoeDownGroups * 64 / p.hidden;
    p.splits = p.splits < 1 ? 1 : p.splits > 8 ? 8 : p.splits;
  }
}

// How a product's workgroup is cut: 16-row tiles that a wave holds (of W1, and as
// many of W3), waves, and pieces in a wave's ring. What the rings leave of 160 KiB
// holds the lists and sums. `xn`: the loads that bring a piece's tokens.
struct MoeCut {
  int tiles, waves, slots;
};
// First product: more tokens want more rows for each load of them (whole layer, 1
// token of 4096 x 1536: 27 us; with 32 rows of each a wave 28; 8 tokens of 7168 x
// 1024: 128 and 125. 32 tokens: 78 us; with 16 rows, and three pieces in a ring, 85;
// 64 tokens of 7168 x 2048 blockwise 506 and 499).
constexpr MoeCut moe_up_cut(int xn) { return xn == 1 ? MoeCut{1, 8, 5} : MoeCut{2, 4, xn == 2 ? 5 : 4}; }
// Second product: the waves' sums (16 rt rows of all tokens in fp32) share the LDS;
// `many`: of more than 32 tokens.
constexpr MoeCut moe_down_cut(int rt, int xn, bool many) {
  return rt == 4 ? MoeCut{4, 4, (xn == 1 ? 5 : 4) - (many ? 1 : 0)} : MoeCut{rt, 8, 4};
}
inline bool moe_down_many(const MoeParams& p) { return p.down_tiles == 4 && p.tokens > 32; }
// A piece of rt tiles: 1 KiB of codes each, their scales, the tokens.
constexpr int moe_stage_bytes(int rt, int xn) { return rt * 1024 + 256 + xn * 1024; }
// LDS of the products' workgroups, of a planned call
constexpr int kMoeLdsBytes = 160 * 1024;
inline int moe_up_lds(const MoeParams& p) {
  const MoeCut c = moe_up_cut(p.dmas);
  return c.waves * (c.slots * moe_stage_bytes(2 * c.tiles, p.dmas) + 2 * c.tiles * 1024) + p.most_segments * 8 + p.rows;
}
inline int moe_down_lds(const MoeParams& p) {
  const MoeCut c = moe_down_cut(p.down_tiles, p.dmas, moe_down_many(p));
  return c.waves * (c.slots * moe_stage_bytes(c.tiles, p.dmas) + p.tokens * c.tiles * 64) + p.most_segments * 8 +
         p.rows * 5;
}
hipError_t launch_moe_layer(MoeParams p, MoeFormat fmt, int num_cus, hipStream_t st);

}  // namespace mxgg
