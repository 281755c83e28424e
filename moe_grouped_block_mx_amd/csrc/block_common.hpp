// Device helpers of the operators around the expert layer (layer norm,
// gradient norm and clipping, the few-token expert layer): 16-byte chunks of
// bf16 or fp32 elements at any element alignment, and wave / group sums.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

namespace mxgg {

struct bf16_t { uint16_t bits; };

typedef float v2f_b __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf_b __attribute__((ext_vector_type(2)));

// fp32 pair -> bf16 pair, round to nearest even, NaN stays NaN
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f_b{a, b}), v2bf_b));
}
__device__ __forceinline__ float bf16_low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ float load_one(const bf16_t* p) { return __uint_as_float((uint32_t)p->bits << 16); }

// 16 bytes of elements as they lie in memory: 8 bf16 or 4 fp32. Loads and
// stores go through memcpy with the element's alignment only, which on gfx950
// is still one 16-byte access, so rows at odd offsets need no path of their
// own.
template <class E>
struct Chunk {
  static constexpr int N = 16 / (int)sizeof(E);
  uint32_t w[4];

  __device__ __forceinline__ void load(const E* p) { memcpy(w, p, 16); }
  __device__ __forceinline__ void store(E* p) const { memcpy(p, w, 16); }
  // the first n < N elements, the others zero
  __device__ __forceinline__ void load_part(const E* p, int n) {
    w[0] = w[1] = w[2] = w[3] = 0;
#pragma unroll
    for (int i = 0; i < N - 1; ++i)
      if (i < n) {
        if constexpr (sizeof(E) == 2)
          w[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i % 2));
        else
          w[i] = reinterpret_cast<const uint32_t*>(p)[i];
      }
  }
  __device__ __forceinline__ void store_part(E* p, int n) const {
#pragma unroll
    for (int i = 0; i < N - 1; ++i)
      if (i < n) {
        if constexpr (sizeof(E) == 2)
          reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(w[i / 2] >> (16 * (i % 2)));
        else
          reinterpret_cast<uint32_t*>(p)[i] = w[i];
      }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(E) == 2)
      return i % 2 ? bf16_high(w[i / 2]) : bf16_low(w[i / 2]);
    else
      return __uint_as_float(w[i]);
  }
  __device__ __forceinline__ void set(const float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(E) == 2)
        w[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
      else
        w[i] = __float_as_uint(v[i]);
    }
  }
};

// A 32-bit value rotated by N within rows of 16 lanes (DPP row_ror): a few
// cycles, where a shuffle through LDS takes a hundred.
template <int N>
__device__ __forceinline__ uint32_t rotate(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x120 + N, 0xF, 0xF, false);
}
template <int N>
__device__ __forceinline__ float rotate(float v) {
  return __uint_as_float(rotate<N>(__float_as_uint(v)));
}

// Sum over W neighbouring lanes (a power of two, at most a wave), in every one
// of them. Halving steps give all lanes the same pairs, so all get the same
// bits.
template <int W>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (W >= 16) v += rotate<8>(v);
  if constexpr (W >= 8) v += rotate<4>(v);   // W < 16: of values that repeat with period W
  if constexpr (W >= 4) v += rotate<2>(v);
  if constexpr (W >= 2) v += rotate<1>(v);
  if constexpr (W >= 32) v += __shfl_xor(v, 16, 64);
  if constexpr (W >= 64) v += __shfl_xor(v, 32, 64);
  return v;
}

}  // namespace mxgg
