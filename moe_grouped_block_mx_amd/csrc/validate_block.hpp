// Host-side argument validation of the operators around the expert layer.
// Pure C++ (no HIP calls), like validate.hpp, whose Check it returns.
#pragma once
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <vector>

#include "block_launch.hpp"
#include "validate.hpp"

namespace mxgg {

inline int dtype_size(int dt) { return dt == MXGG_F32 ? 4 : 2; }

inline Check check_dtype(int dt, const char* what) {
  if (dt == MXGG_BF16 || dt == MXGG_F32) return Check{};
  Check r = fail(MXGG_ERR_FORMAT, "unknown element type %lld", dt);
  r.msg = std::string(what) + ": " + r.msg;
  return r;
}

// A pointer that must be non-NULL (unless `optional`) and aligned to its
// element.
inline Check check_elem_ptr(const void* p, int size, const char* name, bool optional = false) {
  if (!p) {
    if (optional) return Check{};
    Check r; r.st = MXGG_ERR_NULL; r.msg = std::string(name) + " is NULL"; return r;
  }
  if ((uintptr_t)p % (unsigned)size) {
    Check r; r.st = MXGG_ERR_ALIGN; r.msg = std::string(name) + " is not aligned to its elements"; return r;
  }
  return Check{};
}

inline Check check_norm_dims(int64_t rows, int64_t cols) {
  if (rows < 0 || rows >= ((int64_t)1 << 31)) return fail(MXGG_ERR_SHAPE, "rows=%lld outside [0, 2^31)", rows);
  if (cols < 1 || cols > kNormMaxCols)
    return fail(MXGG_ERR_SHAPE, "cols=%lld outside [1, %lld]", cols, (long long)kNormMaxCols);
  return Check{};
}

inline Check check_ld(int64_t ld, int64_t cols, const char* name) {
  if (ld >= cols && ld < ((int64_t)1 << 31)) return Check{};
  Check r = fail(MXGG_ERR_SHAPE, "=%lld outside [cols=%lld, 2^31)", ld, cols);
  r.msg = std::string(name) + r.msg;
  return r;
}

inline Check validate_layer_norm_fwd(const void* x, int64_t rows, int64_t cols, int64_t ldx, int dtype,
                                     const void* weight, const void* bias, int wdtype, float eps, const void* y,
                                     int64_t ldy, const void* mean, const void* rstd) {
  MXGG_TRY(check_dtype(dtype, "layer_norm_fwd x"));
  MXGG_TRY(check_dtype(wdtype, "layer_norm_fwd weight"));
  MXGG_TRY(check_norm_dims(rows, cols));
  MXGG_TRY(check_ld(ldx, cols, "ldx"));
  MXGG_TRY(check_ld(ldy, cols, "ldy"));
  if (!(eps >= 0.f) || std::isinf(eps)) return fail(MXGG_ERR_SHAPE, "eps is negative or not finite");
  MXGG_TRY(check_elem_ptr(weight, dtype_size(wdtype), "weight", true));
  MXGG_TRY(check_elem_ptr(bias, dtype_size(wdtype), "bias", true));
  if (rows == 0) return Check{};
  MXGG_TRY(check_elem_ptr(x, dtype_size(dtype), "x"));
  MXGG_TRY(check_elem_ptr(y, dtype_size(dtype), "y"));
  MXGG_TRY(check_elem_ptr(mean, 4, "mean"));
  MXGG_TRY(check_elem_ptr(rstd, 4, "rstd"));
  return Check{};
}

inline Check validate_layer_norm_bwd(const void* dy, int64_t lddy, const void* x, int64_t ldx, int64_t rows,
                                     int64_t cols, int dtype, const void* weight, int wdtype, const void* mean,
                                     const void* rstd, const void* dx, int64_t lddx, const void* dweight,
                                     const void* dbias, int accumulate) {
  MXGG_TRY(check_dtype(dtype, "layer_norm_bwd x"));
  MXGG_TRY(check_dtype(wdtype, "layer_norm_bwd weight"));
  MXGG_TRY(check_norm_dims(rows, cols));
  MXGG_TRY(check_ld(lddy, cols, "lddy"));
  MXGG_TRY(check_ld(ldx, cols, "ldx"));
  MXGG_TRY(check_ld(lddx, cols, "lddx"));
  if (accumulate != 0 && accumulate != 1) return fail(MXGG_ERR_FORMAT, "accumulate=%lld is not 0 or 1", accumulate);
  MXGG_TRY(check_elem_ptr(weight, dtype_size(wdtype), "weight", true));
  MXGG_TRY(check_elem_ptr(dweight, 4, "dweight", true));
  MXGG_TRY(check_elem_ptr(dbias, 4, "dbias", true));
  if (rows == 0) return Check{};
  MXGG_TRY(check_elem_ptr(dy, dtype_size(dtype), "dy"));
  MXGG_TRY(check_elem_ptr(x, dtype_size(dtype), "x"));
  MXGG_TRY(check_elem_ptr(dx, dtype_size(dtype), "dx"));
  MXGG_TRY(check_elem_ptr(mean, 4, "mean"));
  MXGG_TRY(check_elem_ptr(rstd, 4, "rstd"));
  return Check{};
}

// A launch counts the 8192-element chunks of its tensors in 32 bits.
constexpr int64_t kMaxGradElems = (int64_t)1 << 42;

// n tensors that do not overlap: each element is counted once, and scaled by
// one workgroup.
inline Check validate_grads(void* const* grads, const int64_t* numels, const int32_t* dtypes, int64_t n) {
  if (n < 0 || n >= ((int64_t)1 << 24)) return fail(MXGG_ERR_SHAPE, "n=%lld tensors outside [0, 2^24)", n);
  if (n > 0 && (!grads || !numels || !dtypes)) return fail(MXGG_ERR_NULL, "grads, numels or dtypes is NULL");
  std::vector<std::pair<uintptr_t, uintptr_t>> spans;
  spans.reserve((size_t)n);
  bool sorted = true;
  int64_t elems = 0;
  for (int64_t i = 0; i < n; ++i) {
    MXGG_TRY(check_dtype(dtypes[i], "gradient"));
    if (numels[i] < 0 || numels[i] >= kMaxGradElems || (elems += numels[i]) >= kMaxGradElems)
      return fail(MXGG_ERR_SHAPE, "numels[%lld] = %lld: negative, or over 2^42 elements together", i, numels[i]);
    if (numels[i] == 0) continue;
    MXGG_TRY(check_elem_ptr(grads[i], dtype_size(dtypes[i]), "a gradient"));
    const uintptr_t at = (uintptr_t)grads[i];
    if (!spans.empty() && at < spans.back().first) sorted = false;
    spans.emplace_back(at, at + (uintptr_t)numels[i] * (unsigned)dtype_size(dtypes[i]));
  }
  if (!sorted) std::sort(spans.begin(), spans.end());
  for (size_t i = 1; i < spans.size(); ++i)
    if (spans[i].first < spans[i - 1].second)
      return fail(MXGG_ERR_SHAPE, "two gradients overlap: each would be counted and scaled twice");
  return Check{};
}

inline Check check_norm_kind(int kind) {
  if (kind == MXGG_NORM_L2 || kind == MXGG_NORM_MAX) return Check{};
  return fail(MXGG_ERR_FORMAT, "unknown norm %lld", kind);
}

inline Check check_max_norm(float max_norm) {
  if (max_norm >= 0.f && !std::isinf(max_norm)) return Check{};
  return fail(MXGG_ERR_SHAPE, "max_norm is negative or not finite");
}

inline Check check_workspace(const void* ws, size_t bytes, size_t need) {
  if (bytes < need)
    return fail(MXGG_ERR_WORKSPACE, "workspace %lld < %lld bytes", (long long)bytes, (long long)need);
  return check_ptr(ws, need > 0, "ws");
}

inline Check validate_moe_dims(int64_t T, int64_t H, int64_t I, int64_t E, int64_t k) {
  if (T < 0 || T > MXGG_MOE_MAX_TOKENS)
    return fail(MXGG_ERR_SHAPE, "tokens=%lld outside [0, 64] (the grouped GEMMs take more)", T);
  if (E < 1 || E > MXGG_MAX_EXPERTS) return fail(MXGG_ERR_SHAPE, "experts=%lld outside [1, 512]", E);
  if (k < 1 || k > MXGG_MOE_MAX_TOP_K || k > E)
    return fail(MXGG_ERR_SHAPE, "top_k=%lld outside [1, min(16, experts=%lld)]", k, E);
  if (H < 1 || I < 1 || H > 65536 || I > 65536)
    return fail(MXGG_ERR_SHAPE, "hidden=%lld, inner=%lld outside [1, 65536]", H, I);
  return Check{};
}

inline Check validate_moe_layer(const void* x, int64_t ldx, const void* logits, int64_t ldl, int ldtype, int64_t T,
                                int64_t H, int64_t I, int64_t E, int64_t k, const void* w13_q, const void* w13_s,
                                const void* w2_q, const void* w2_s, int w_fmt, uint32_t flags, const void* out,
                                const void* ids, const void* weights) {
  MXGG_TRY(check_layout(w_fmt, "moe_layer weights", false, MXGG_KBLOCK_ROWS));
  MXGG_TRY(check_dtype(ldtype, "moe_layer logits"));
  const int f = base_format(format_bits(w_fmt));
  if (f != MXGG_MXFP4 && f != MXGG_MXFP8 && f != MXGG_FP8_128x128)
    return fail(MXGG_ERR_FORMAT, "moe_layer takes MXFP4, MXFP8 or FP8_128x128 weights (got %lld)", w_fmt);
  if (flags & ~(uint32_t)(MXGG_MOE_RENORMALIZE | MXGG_MOE_W13_KBLOCK | MXGG_MOE_W2_KBLOCK))
    return fail(MXGG_ERR_FORMAT, "unknown flags 0x%llx", flags);
  if (f == MXGG_FP8_128x128 && flags & (MXGG_MOE_W13_KBLOCK | MXGG_MOE_W2_KBLOCK))
    return fail(MXGG_ERR_FORMAT, "the K-block flags are of MX formats (got %lld)", w_fmt);
  MXGG_TRY(validate_moe_dims(T, H, I, E, k));
  const bool all = f == MXGG_FP8_128x128 || kblock_bits(w_fmt);
  const int unit_h = all || flags & MXGG_MOE_W13_KBLOCK ? 128 : 32, unit_i = all || flags & MXGG_MOE_W2_KBLOCK ? 128 : 32;
  if (H % unit_h) return fail(MXGG_ERR_SHAPE, "hidden=%lld must be a multiple of %lld", H, unit_h);
  if (I % unit_i) return fail(MXGG_ERR_SHAPE, "inner=%lld must be a multiple of %lld", I, unit_i);
  // 64 rows of x are addressed with 32-bit element offsets
  if (ldx < H || ldx >= ((int64_t)1 << 25)) return fail(MXGG_ERR_SHAPE, "ldx=%lld outside [hidden=%lld, 2^25)", ldx, H);
  if (ldx % 8) return fail(MXGG_ERR_ALIGN, "ldx=%lld not a multiple of 8 elements", ldx);
  if (ldl < E || ldl >= ((int64_t)1 << 31)) return fail(MXGG_ERR_SHAPE, "ldl=%lld outside [experts=%lld, 2^31)", ldl, E);
  if (T == 0) return Check{};
  MXGG_TRY(check_ptr(x, true, "x"));
  MXGG_TRY(check_elem_ptr(logits, dtype_size(ldtype), "logits"));
  MXGG_TRY(check_ptr(w13_q, true, "w13_q"));
  MXGG_TRY(check_ptr(w13_s, true, "w13_s"));
  MXGG_TRY(check_ptr(w2_q, true, "w2_q"));
  MXGG_TRY(check_ptr(w2_s, true, "w2_s"));
  MXGG_TRY(check_ptr(out, true, "out"));
  MXGG_TRY(check_elem_ptr(ids, 4, "ids"));
  MXGG_TRY(check_elem_ptr(weights, 4, "weights"));
  return Check{};
}

}  // namespace mxgg
