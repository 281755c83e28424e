// Host-side argument validation of the operators that bring tokens to their
// experts and back, of the int8 products and of dropout. Pure C++ (no HIP
// calls), like validate.hpp, whose Check it returns.
#pragma once
#include <stdint.h>

#include "token_launch.hpp"
#include "validate.hpp"
#include "validate_block.hpp"

namespace mxgg {

constexpr int64_t kTokenMaxCols = (int64_t)1 << 24;

inline Check check_choices(int64_t tokens, int64_t top_k) {
  if (top_k < 1 || top_k > MXGG_MOE_MAX_TOP_K) return fail(MXGG_ERR_SHAPE, "top_k=%lld outside [1, 16]", top_k);
  // (the kernels number choices, and what lies up to a chunk behind them, in 32 bits)
  if (tokens < 0 || tokens > ((int64_t)1 << 30) / top_k)
    return fail(MXGG_ERR_SHAPE, "tokens=%lld: negative, or tokens * top_k > 2^30", tokens);
  return Check{};
}

inline Check validate_moe_sort(const void* ids, int itype, int64_t ldi, int64_t tokens, int64_t top_k, int64_t experts,
                               const void* rows, const void* choices, const void* counts) {
  if (itype != MXGG_I32 && itype != MXGG_I64) return fail(MXGG_ERR_FORMAT, "unknown integer type %lld", itype);
  MXGG_TRY(check_choices(tokens, top_k));
  if (experts < 1 || experts > MXGG_MAX_EXPERTS) return fail(MXGG_ERR_SHAPE, "experts=%lld outside [1, 512]", experts);
  if (ldi < top_k || ldi >= ((int64_t)1 << 31))
    return fail(MXGG_ERR_SHAPE, "ldi=%lld outside [top_k=%lld, 2^31)", ldi, top_k);
  MXGG_TRY(check_elem_ptr(counts, 4, "counts"));
  if (tokens == 0) return Check{};
  MXGG_TRY(check_elem_ptr(ids, itype == MXGG_I64 ? 8 : 4, "ids"));
  MXGG_TRY(check_elem_ptr(rows, 4, "rows"));
  MXGG_TRY(check_elem_ptr(choices, 4, "choices"));
  return Check{};
}

// Tokens' rows [tokens, cols] and experts' rows [expert_rows, cols]
inline Check check_token_dims(int64_t tokens, int64_t top_k, int64_t expert_rows, int64_t cols, int dtype,
                              const char* what) {
  MXGG_TRY(check_dtype(dtype, what));
  MXGG_TRY(check_choices(tokens, top_k));
  if (expert_rows < 0 || expert_rows >= ((int64_t)1 << 31))
    return fail(MXGG_ERR_SHAPE, "expert_rows=%lld outside [0, 2^31)", expert_rows);
  if (cols < 1 || cols > kTokenMaxCols) return fail(MXGG_ERR_SHAPE, "cols=%lld outside [1, 2^24]", cols);
  return Check{};
}

inline Check validate_moe_dispatch(const void* x, int64_t ldx, int dtype, int64_t tokens, int64_t cols, const void* rows,
                                   int64_t top_k, const void* out, int64_t ldo, int64_t expert_rows) {
  MXGG_TRY(check_token_dims(tokens, top_k, expert_rows, cols, dtype, "moe_dispatch x"));
  MXGG_TRY(check_ld(ldx, cols, "ldx"));
  MXGG_TRY(check_ld(ldo, cols, "ldo"));
  if (tokens == 0 || expert_rows == 0) return Check{};
  MXGG_TRY(check_elem_ptr(x, dtype_size(dtype), "x"));
  MXGG_TRY(check_elem_ptr(rows, 4, "rows"));
  MXGG_TRY(check_elem_ptr(out, dtype_size(dtype), "out"));
  return Check{};
}

inline Check validate_moe_combine(const void* y, int64_t ldy, int dtype, int64_t expert_rows, int64_t cols,
                                  const void* rows, const void* weights, int64_t tokens, int64_t top_k, const void* out,
                                  int64_t ldo) {
  MXGG_TRY(check_token_dims(tokens, top_k, expert_rows, cols, dtype, "moe_combine y"));
  MXGG_TRY(check_ld(ldy, cols, "ldy"));
  MXGG_TRY(check_ld(ldo, cols, "ldo"));
  if (tokens == 0) return Check{};
  MXGG_TRY(check_elem_ptr(y, dtype_size(dtype), "y", expert_rows == 0));
  MXGG_TRY(check_elem_ptr(rows, 4, "rows"));
  MXGG_TRY(check_elem_ptr(weights, 4, "weights", true));
  MXGG_TRY(check_elem_ptr(out, dtype_size(dtype), "out"));
  return Check{};
}

inline Check validate_moe_combine_bwd(const void* dout, int64_t lddo, const void* y, int64_t ldy, int dtype,
                                      int64_t expert_rows, int64_t cols, const void* rows, const void* weights,
                                      int64_t tokens, int64_t top_k, const void* dy, int64_t lddy, const void* dweights) {
  MXGG_TRY(check_token_dims(tokens, top_k, expert_rows, cols, dtype, "moe_combine_bwd y"));
  MXGG_TRY(check_ld(lddo, cols, "lddo"));
  MXGG_TRY(check_ld(ldy, cols, "ldy"));
  MXGG_TRY(check_ld(lddy, cols, "lddy"));
  if (tokens == 0) return Check{};
  if (dy && dy == y && lddy != ldy && expert_rows > 1)
    return fail(MXGG_ERR_SHAPE, "dy is y with another leading dimension (lddy=%lld, ldy=%lld)", lddy, ldy);
  const int size = dtype_size(dtype);
  MXGG_TRY(check_elem_ptr(dout, size, "dout"));
  MXGG_TRY(check_elem_ptr(y, size, "y", expert_rows == 0));
  MXGG_TRY(check_elem_ptr(dy, size, "dy", expert_rows == 0));
  MXGG_TRY(check_elem_ptr(rows, 4, "rows"));
  MXGG_TRY(check_elem_ptr(weights, 4, "weights"));
  MXGG_TRY(check_elem_ptr(dweights, 4, "dweights"));
  return Check{};
}

inline Check validate_dropout(const void* x, int64_t ldx, int dtype, int64_t rows, int64_t cols, float p,
                              const void* state, const void* residual, int64_t ldr, const void* out, int64_t ldo) {
  MXGG_TRY(check_dtype(dtype, "dropout x"));
  if (rows < 0 || rows >= ((int64_t)1 << 31)) return fail(MXGG_ERR_SHAPE, "rows=%lld outside [0, 2^31)", rows);
  if (cols < 1 || cols > kTokenMaxCols) return fail(MXGG_ERR_SHAPE, "cols=%lld outside [1, 2^24]", cols);
  MXGG_TRY(check_ld(ldx, cols, "ldx"));
  if (residual) MXGG_TRY(check_ld(ldr, cols, "ldr"));
  MXGG_TRY(check_ld(ldo, cols, "ldo"));
  if (!(p >= 0.f && p <= 1.f)) return fail(MXGG_ERR_SHAPE, "p is outside [0, 1]");
  if (rows == 0) return Check{};
  MXGG_TRY(check_elem_ptr(x, dtype_size(dtype), "x"));
  MXGG_TRY(check_elem_ptr(residual, dtype_size(dtype), "residual", true));
  MXGG_TRY(check_elem_ptr(out, dtype_size(dtype), "out"));
  MXGG_TRY(check_elem_ptr(state, 8, "state"));
  return Check{};
}

// int8 codes: rows of whole 16-byte pieces, and sums that 32 bits hold.
constexpr int64_t kInt8MaxK = ((int64_t)1 << 17) - 16;

inline Check check_int8_format(int f, const char* what) {
  if (f == MXGG_INT8) return Check{};
  Check r;
  r.st = MXGG_ERR_FORMAT;
  r.msg = std::string(what) + ": int8 codes have one layout (rows, one fp32 scale each): no layout or code-layout bits";
  return r;
}

inline Check check_int8_k(int64_t K, const char* name) {
  if (K > 0 && K % 16 == 0 && K <= kInt8MaxK) return Check{};
  Check r = fail(MXGG_ERR_SHAPE, "=%lld must be a multiple of 16 below 2^17", K);
  r.msg = std::string(name) + r.msg;
  return r;
}

inline Check validate_quantize_int8(const void* x, int64_t rows, int64_t cols, int64_t ldx, int fmt, const void* q,
                                    const void* scales) {
  MXGG_TRY(check_int8_format(fmt, "quantize_rowwise"));
  if (rows < 0 || rows >= ((int64_t)1 << 31)) return fail(MXGG_ERR_SHAPE, "rows=%lld outside [0, 2^31)", rows);
  MXGG_TRY(check_int8_k(cols, "cols"));
  if (ldx < cols) return fail(MXGG_ERR_SHAPE, "ldx=%lld < cols=%lld", ldx, cols);
  if (ldx % 8) return fail(MXGG_ERR_ALIGN, "ldx=%lld not a multiple of 8 elements", ldx);
  const bool nz = rows > 0;
  MXGG_TRY(check_ptr(x, nz, "x"));
  MXGG_TRY(check_ptr(q, nz, "q"));
  MXGG_TRY(check_ptr(scales, nz, "scales"));
  return Check{};
}

inline Check validate_fwd_int8(const void* a_q, const void* a_s, int a_fmt, const void* w_q, const void* w_s, int w_fmt,
                               const int64_t* m, int32_t G, int64_t M, int64_t N, int64_t K, const void* out) {
  MXGG_TRY(check_int8_format(a_fmt, "fwd A"));
  MXGG_TRY(check_int8_format(w_fmt, "fwd W"));
  if (M < 0 || M >= ((int64_t)1 << 31) || N <= 0 || N >= kMaxRowStride)
    return fail(MXGG_ERR_SHAPE, "M=%lld outside [0, 2^31) or N=%lld outside [1, 2^23)", M, N);
  MXGG_TRY(check_int8_k(K, "K"));
  MXGG_TRY(check_splits(m, G, M, "A"));
  const bool nz = M > 0;
  MXGG_TRY(check_ptr(a_q, nz, "a_q"));
  MXGG_TRY(check_ptr(a_s, nz, "a_s"));
  MXGG_TRY(check_ptr(w_q, nz, "w_q"));
  MXGG_TRY(check_ptr(w_s, nz, "w_s"));
  MXGG_TRY(check_ptr(out, nz, "out"));
  return Check{};
}

}  // namespace mxgg
