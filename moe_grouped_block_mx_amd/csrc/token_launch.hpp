// Internal launch interface of the operators that bring tokens to their experts
// and back, of the int8 products and of dropout, between the C ABI (api.cpp) and
// their kernels. Not part of the public ABI.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "device_common.hpp"

namespace mxgg {

// --- tokens to experts and back ---------------------------------------------
// Up to kSortOne choices are sorted by one workgroup in one launch. More are cut
// into chunks, a workgroup each, that meet in a table (in the workspace): one row of
// experts + 1 counts a chunk (the last: dropped choices; padded to whole 16 bytes).
// Measured, us on the card: 4096 choices in one launch 5.8 (8 experts), 7.3 (128) and
// 7.9 (511), and 4104 in two 6.7 (128), which costs the host a launch, 3.5, more; 8192
// in one 9.6 (8) and 12.6 (128), in two 6.4 and 6.8.
constexpr int kSortOne = 4096, kSortThreads = 1024;
// Choices of a chunk, 1, 2 or 4 a lane: small chunks spread over the card, large ones
// keep the table short. Measured, us, chunks of 1024, 2048 and 4096: 8192 choices of
// 128 experts 6.8 8.0 10.5; 65536 of 128 8.4 9.0 11.4, of 511 10.1 10.3 12.5; 131072
// of 128 9.8 9.9 12.0, of 511 13.2 10.8 13.4; 262144 of 128 11.9 10.8 13.0; 524288 of
// 128 16.5 14.0 14.4; 1048576 of 128 28 21 19; 4194304 of 128 90 68 58.
constexpr int64_t kSortShort = 65536, kSortLong = 1 << 20;
inline int sort_lane(int64_t choices) { return choices <= kSortShort ? 1 : choices < kSortLong ? 2 : 4; }
inline int64_t sort_chunks(int64_t choices) {
  const int64_t chunk = (int64_t)sort_lane(choices) * kSortThreads;
  return choices <= kSortOne ? 1 : (choices + chunk - 1) / chunk;
}
// Up to so many workgroups, each adds up the table's rows before its own
// itself; beyond, a launch between does it for all. Measured, us, without the launch
// and with it: 32 chunks of 32 experts 7.0 and 8.0; 64 of 128 8.3 and 8.7, of 511 10.0
// and 9.4; 128 of 128 10.9 and 11.6, of 511 13.5 and 13.4; 256 of 8 10.0 and 11.3, of
// 128 13.9 and 14.3, of 511 18.7 and 16.6. (One limit for any number of experts costs
// 0.6 us at 64 chunks of 511, 1.3 at 256 of 8, 0.4 at 256 of 128.)
constexpr int64_t kSortDirect = 128;
// A row of the table: whole 16 bytes
__host__ __device__ inline int sort_table_row(int experts) { return (experts + 4) / 4 * 4; }
inline size_t sort_workspace(int64_t choices, int64_t experts) {
  int64_t chunks = sort_chunks(choices);
  // (no less than fewer choices take, so that the space of the largest call does for all)
  if (choices > kSortShort) chunks = std::max(chunks, sort_chunks(kSortShort));
  if (choices >= kSortLong) chunks = std::max(chunks, sort_chunks(kSortLong - 1));
  return chunks <= 1 ? 0 : (size_t)((chunks + 1) * sort_table_row((int)experts)) * sizeof(int32_t);
}

struct SortParams {
  const void* ids;
  int32_t* rows;      // [choices]
  int32_t* choices;   // [choices]
  int32_t* counts;    // [experts]
  int32_t* table;     // [chunks + 1][sort_table_row(experts)]
  int64_t ldi;
  int32_t n, top_k, experts;
};
hipError_t launch_moe_sort(const SortParams& p, bool i64, hipStream_t st);

// A lane's chunk of n elements of a row of `cols` (at least n), for the columns from
// `col` on. A chunk that would pass the row's end begins earlier, to end with the row:
// its first `skip` elements are then its neighbour's.
struct RowChunk {
  int start, skip;
};
__host__ __device__ inline RowChunk row_chunk(int col, int cols, int n) {
  const int start = col < cols - n ? col : cols - n;
  return RowChunk{start, col - start};
}

struct TokenParams {
  const void* x;          // tokens' rows: dispatch's input, the gradient of combine's output
  const void* y;          // experts' rows: combine's input
  void* out;              // dispatch: experts' rows; combine: tokens' rows; its gradient: experts' rows
  const int32_t* rows;    // [tokens, top_k]
  const float* weights;   // [tokens, top_k], or NULL (1)
  float* dweights;        // [tokens, top_k]
  int64_t tokens, expert_rows, ldx, ldy, ldo;
  int32_t top_k, cols;
};
hipError_t launch_moe_dispatch(const TokenParams& p, bool f32, hipStream_t st);
hipError_t launch_moe_combine(const TokenParams& p, bool f32, hipStream_t st);
hipError_t launch_moe_combine_bwd(const TokenParams& p, bool f32, hipStream_t st);

// --- dropout ------------------------------------------------------------------
struct DropoutParams {
  const void* x;
  const void* residual;   // or NULL
  void* out;
  const int64_t* state;   // seed, step
  int64_t rows, ldx, ldr, ldo;
  int32_t cols;
  uint32_t stream;
  uint32_t limit;         // columns whose 16-bit number is below it are dropped
  float scale;            // 65536 / (65536 - limit), 0 when all are dropped
};
hipError_t launch_dropout(const DropoutParams& p, bool f32, hipStream_t st);

// --- int8 ---------------------------------------------------------------------
hipError_t launch_quant_int8(const uint16_t* x, int64_t rows, int64_t cols, int64_t ldx, int8_t* q, float* scales,
                             hipStream_t st);

// out[r, n] = a_s[r] w_s[g, n] sum_k a[r, k] w[g, n, k] for the rows r of
// expert g
struct Int8Params {
  const uint8_t* a;       // [M, K]
  const float* as;        // [M]
  const uint8_t* w;       // [G * N, K]
  const float* ws;        // [G * N]
  uint16_t* out;          // bf16 [M, N]
  int64_t n;
  int32_t k;
  SplitArgs sp;
};
// Pieces of at most `each` of an expert's m tokens (any m below 2^31: the sum is
// unsigned)
__host__ __device__ inline int32_t token_pieces(int32_t m, int each) {
  return (int32_t)(((uint32_t)m + (uint32_t)each - 1) / (uint32_t)each);
}
inline int64_t int8_pieces(const SplitArgs& sp, int each) {
  int64_t n = 0;
  for (int g = 0; g < sp.G; ++g) n += token_pieces(sp.m[g], each);
  return n;
}
// The forms of the product: tiles of 256 channels x 256 tokens, of 128 x 128, and
// for few tokens 16 i channels x 16 j tokens (kInt8Few<i><j>) with the
// contraction split over a workgroup's waves.
enum Int8Form { kInt8Big, kInt8Small, kInt8Few11, kInt8Few12, kInt8Few21, kInt8Few22, kInt8Few24, kInt8Few42, kInt8Few44 };
// Every form's time is its rounds of one workgroup a CU, times what one takes: a
// part that grows with K, in units of 16 rows of codes brought to a CU (at K = 4096
// 1.5 us), and one that does not (start, results, the wait for the first loads),
// which is less where two workgroups fit on a CU. The forms of few tokens bring the
// rows of their channels and tokens; a 128 x 128 tile's loads overlap more (11.5
// units for 16), a 256 x 256 tile's time is its MFMAs'.
// Measured, us (one expert unless said; tokens, channels, K; medians of replays, the
// weights of several layers in turn; the form that the rule takes is marked):
//                                    256    128    64 x 64  64 x 32  32 x 32  32 x 16  16 x 16
//   1, 4096, 7168                     71     31      21       20       13       12       8.4*
//   1, 8192, 1024                     18     10      6.7      6.0      5.1      4.5*     4.8
//   32, 4096, 4096                    43     20      12       10       8.3      7.2*     8.4
//   64, 4096, 4096                    44     20      13       10       9.0*     11       13
//   256, 4096, 4096                   49     21      15*      21       26       30       38
//   512, 4096, 4096                   49     22*     27       40       49       54       71
//   512, 1111, 2000                   33     16      9.9*     13       16       15       16
//   1024, 1024, 8192                  86     35      23*      32       40       51       64
//   1024, 4096, 4096                  49     24*     49       77       95       102      133
//   1024, 8192, 1024                  24     19*     40       60       95       87       141
//   2048, 4096, 4096                  52     41*     91       149
//   2048, 8192, 1024                  27*    32      77       119
//   4096, 4096, 4096                  67*    83
//   64 of 128 experts, 2048, 7168     170    127     148      141      147      126*     132
//   256 of 32, 4096, 4096             140    125     127      119*     137      110      131
//   1024 of 32, 4096, 4096            141    125*    148      151      192      191      251
//   2999 of 5, 1111, 2000             37     18*     39       49       71       71       101
//   4096 of 32, 4096, 4096            189    149*
//   8192 of 32, 4096, 4096            204*   219
//   8192 of 64, 4096, 7168            522    488*
//   16384 of 64, 4096, 7168           653*   746
//   32768 of 64, 4096, 7168           1053*  1253
// (32 x 64 and 16 x 32 are for the tokens in between, as 40 and 20.)
inline Int8Form int8_form(const SplitArgs& sp, int64_t n, int64_t k, int num_cus) {
  struct Option {
    Int8Form form;
    int channels, tokens;
    float units, fixed;   // units 0: the rows that a workgroup brings
  };
  static constexpr Option options[] = {
      {kInt8Big, 256, 256, 29.f, 8.f},     {kInt8Small, 128, 128, 11.5f, 2.2f}, {kInt8Few11, 16, 16, 0, 0.5f},
      {kInt8Few21, 32, 16, 0, 0.5f},       {kInt8Few12, 16, 32, 0, 0.5f},       {kInt8Few22, 32, 32, 0, 1.6f},
      {kInt8Few24, 32, 64, 0, 1.6f},       {kInt8Few42, 64, 32, 0, 1.6f},       {kInt8Few44, 64, 64, 0, 1.6f}};
  int64_t rows = 0;
  for (int g = 0; g < sp.G; ++g) rows += sp.m[g];
  Int8Form best = kInt8Big;
  float least = 0;
  for (const Option& o : options) {
    const int64_t pieces = int8_pieces(sp, o.tokens), groups = pieces * ((n + o.channels - 1) / o.channels);
    if (o.units == 0 && pieces > 65535) continue;      // the grid's y axis
    const float units = o.units > 0 ? o.units : (float)o.channels / 16 + (float)rows / (float)pieces / 16;
    const float cost = (float)((groups + num_cus - 1) / num_cus) * (units + o.fixed * 4096 / (float)k);
    if (o.form == kInt8Big || cost < least) {
      least = cost;
      best = o.form;
    }
  }
  return best;
}
hipError_t launch_grouped_int8(const Int8Params& p, int num_cus, hipStream_t st);

}  // namespace mxgg
