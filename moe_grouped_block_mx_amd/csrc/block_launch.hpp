// Internal launch interface of the operators around the expert layer, between
// the C ABI (block_api.cpp) and their kernels. Not part of the public ABI.
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
// workgroups of the backward pass: one partial sum of both gradients each
int norm_bwd_groups(int64_t rows, int64_t cols);
hipError_t launch_layer_norm_fwd(const NormFwdParams& p, bool f32, bool wf32, hipStream_t st);
// dweight / dbias: fp32 [cols] or NULL
hipError_t launch_layer_norm_bwd(const NormBwdParams& p, bool f32, bool wf32, float* dweight, float* dbias,
                                 bool accumulate, hipStream_t st);

// --- gradient norm and clipping --------------------------------------------
// Tensors of one launch: they travel as kernel arguments, so a call needs no
// device copy of the caller's pointer list.
constexpr int kClipTensors = 128;
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

// One chosen expert: its tokens, and where their rows of the inner activation
// start (in the order of the tokens).
struct MoeExpert {
  int32_t expert, base;
  uint64_t tokens;
};
// At most 16 of its tokens (one column tile of the second product), and the
// weight and token of one row.
struct MoeSegment {
  int32_t expert, base, tokens, unused;
};
struct MoeRow {
  float weight;
  int32_t token;
};
inline int64_t moe_most_segments(int64_t tokens, int64_t experts, int64_t top_k) {
  const int64_t rows = tokens * top_k;
  return rows / 16 + (rows < experts ? rows : experts);
}
// Workspace: how many experts and segments there are, their lists, the rows
// and the inner activation, bf16 (laid out as its reader takes it: inner_at in
// moe_layer.hip).
struct MoeWorkspace {
  size_t table, segments, rows, inner, bytes;
};
inline MoeWorkspace moe_workspace(int64_t tokens, int64_t experts, int64_t top_k, int64_t inner) {
  const auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  MoeWorkspace w;
  w.table = 256;
  w.segments = w.table + up((size_t)experts * sizeof(MoeExpert));
  w.rows = w.segments + up((size_t)moe_most_segments(tokens, experts, top_k) * sizeof(MoeSegment));
  w.inner = w.rows + up((size_t)(tokens * top_k) * sizeof(MoeRow));
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
  int32_t* counts;
  MoeExpert* table;
  MoeSegment* segments;
  MoeRow* row_list;
  uint16_t* inner_x;
  int64_t ldx, ldl;
  int32_t tokens, experts, top_k, hidden, inner;
  int32_t rows;                       // of the inner activation: tokens * top_k
  int32_t most_segments;
  // byte strides of the codes: between rows, and between the 64-byte pieces of
  // a row; of the MX scales: between blocks of 32
  int64_t q13_row, q13_piece, s13_block, q2_row, q2_piece, s2_block;
};
enum MoeFormat { kMoeFp4 = 0, kMoeFp8 = 1, kMoeBlock = 2 };
hipError_t launch_moe_layer(const MoeParams& p, MoeFormat fmt, bool logits_f32, bool renormalize, hipStream_t st);

}  // namespace mxgg
