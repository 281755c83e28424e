// Dropout whose mask is never stored:
//
//   out = residual + (kept ? x / (1 - p') : 0),  p' = round(p 2^16) / 2^16
//
// An element's number is a function of (seed, step, stream, row, column), so the
// backward pass is the same call on the gradient, without a residual. The
// generator is Philox4x32 with 10 rounds (Salmon, Moraes, Dror, Shaw, "Parallel
// random numbers: as easy as 1, 2, 3", 2011): key = the seed, counter = (group of
// eight columns, 64 bits; stream; step).
//
// 16 bits an element, so a group of eight columns takes one call of 20 wide
// multiplications: p is rounded to 2^-16, and the scale is that of the rounded
// one, so the expectation is exact.
//
// What bounds it: the bytes. bf16 16384 x 7168: 101 us without a residual (4.7 TB/s;
// with 32 bits an element, two calls a group, 121), 138 us with one (5.1 TB/s; 142).
// A plain copy reaches 5.1 TB/s. 8 x 4096 takes 5.5 us, a launch and two latencies.
#include "block_common.hpp"
#include "token_launch.hpp"

namespace mxgg {
namespace {

constexpr int kThreads = 256;
constexpr int kGroup = 8;
constexpr int64_t kGrid = 1 << 20;

struct Words {
  uint32_t w[4];
  __device__ __forceinline__ uint32_t number(int i) const { return i % 2 ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu; }
};

__device__ __forceinline__ Words philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int round = 0; round < 10; ++round) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return Words{{c0, c1, c2, c3}};
}

// A row belongs to L lanes (a power of two, up to the workgroup), a lane to a
// group of eight columns.
template <class E, bool RESIDUAL>
__global__ __launch_bounds__(kThreads) void dropout_kernel(DropoutParams p, int lanes) {
  constexpr int N = Chunk<E>::N, CH = kGroup / N;
  const int per = kThreads / lanes, lane = threadIdx.x % lanes;
  const int group = (int)blockIdx.y * lanes + lane, col = group * kGroup;
  if (col >= p.cols) return;
  const int groups = (p.cols + kGroup - 1) / kGroup, size = min(p.cols - col, kGroup);
  const uint64_t seed = (uint64_t)p.state[0];
  const uint32_t step = (uint32_t)p.state[1];
  for (int64_t r = (int64_t)blockIdx.x * per + threadIdx.x / lanes; r < p.rows; r += (int64_t)gridDim.x * per) {
    const E* x = static_cast<const E*>(p.x) + r * p.ldx + col;
    const E* res = static_cast<const E*>(p.residual) + r * p.ldr + col;
    E* out = static_cast<E*>(p.out) + r * p.ldo + col;
    Chunk<E> c[CH], d[CH];
    const auto load = [&](Chunk<E>(&v)[CH], const E* from) {
#pragma unroll
      for (int h = 0; h < CH; ++h) {
        if (size == kGroup) v[h].load(from + h * N);
        else if (size >= (h + 1) * N) v[h].load(from + h * N);
        else v[h].load_part(from + h * N, max(size - h * N, 0));
      }
    };
    load(c, x);
    if (RESIDUAL) load(d, res);
    const uint64_t at = (uint64_t)r * (uint32_t)groups + (uint32_t)group;
    const Words w = philox((uint32_t)at, (uint32_t)(at >> 32), p.stream, step, (uint32_t)seed, (uint32_t)(seed >> 32));
#pragma unroll
    for (int h = 0; h < CH; ++h) {
      float v[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        v[i] = w.number(h * N + i) >= p.limit ? c[h].get(i) * p.scale : 0.f;
        if (RESIDUAL) v[i] += d[h].get(i);
      }
      c[h].set(v);
      if (size >= (h + 1) * N) c[h].store(out + h * N);
      else c[h].store_part(out + h * N, max(size - h * N, 0));
    }
  }
}

template <class E>
hipError_t dropout_any(const DropoutParams& p, hipStream_t st) {
  const int64_t groups = (p.cols + kGroup - 1) / kGroup;
  int lanes = 1;
  while (lanes < kThreads && lanes < groups) lanes *= 2;
  const int64_t per = kThreads / lanes, blocks = (p.rows + per - 1) / per;
  const dim3 grid((uint32_t)(blocks < kGrid ? blocks : kGrid), (uint32_t)((groups + lanes - 1) / lanes));
  if (p.residual) dropout_kernel<E, true><<<grid, kThreads, 0, st>>>(p, lanes);
  else dropout_kernel<E, false><<<grid, kThreads, 0, st>>>(p, lanes);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(const DropoutParams& p, bool f32, hipStream_t st) {
  return f32 ? dropout_any<float>(p, st) : dropout_any<bf16_t>(p, st);
}

}  // namespace mxgg
