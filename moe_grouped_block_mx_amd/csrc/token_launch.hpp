// Internal launch interface of the operators that bring tokens to their experts
// and back, of the int8 products and of dropout, between the C ABI (api.cpp) and
// their kernels. Not part of the public ABI.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"

namespace mxgg {

// --- tokens to experts and back ---------------------------------------------
// Choices that one workgroup sorts; a call of more than one of them goes over
// a table of the workgroups' counts (in the workspace), one row of experts + 1
// counts each (the last: dropped choices).
constexpr int kSortChunk = 2048;
inline int64_t sort_chunks(int64_t choices) { return (choices + kSortChunk - 1) / kSortChunk; }
// Up to so many workgroups, each adds up the table's rows before its own
// itself; beyond, a launch between does it for all.
constexpr int64_t kSortDirect = 128;
inline size_t sort_workspace(int64_t choices, int64_t experts) {
  const int64_t chunks = sort_chunks(choices);
  return chunks <= 1 ? 0 : (size_t)((chunks + 1) * (experts + 1)) * sizeof(int32_t);
}

struct SortParams {
  const void* ids;
  int32_t* rows;      // [choices]
  int32_t* choices;   // [choices]
  int32_t* counts;    // [experts]
  int32_t* table;     // [chunks + 1][experts + 1]
  int64_t ldi;
  int32_t n, top_k, experts;
};
hipError_t launch_moe_sort(const SortParams& p, bool i64, hipStream_t st);

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
hipError_t launch_grouped_int8(const Int8Params& p, int num_cus, hipStream_t st);

}  // namespace mxgg
