// The norm of all gradients together, and clipping by it.
//
//   n = (sum over every tensor of x^2)^1/2, or max |x|
//   x <- x min(1, max_norm / (n + 1e-6))
//
// Two passes over the data, with the norm complete between them: the first
// leaves one partial per workgroup, and every workgroup of the second adds
// those up itself in the same order, so the norm is the same bits in each of
// them and from run to run, without atomics and without a launch in between.
// Squares are summed in fp64: a gradient of 1e30 has a norm (its fp32 square
// does not), and the memory is still what bounds the pass.
//
// A tensor is cut into chunks of 8192 elements, dealt out to the workgroups in
// turn, so many small tensors cost what one of their size does; the scaling goes
// backwards, onto what the norm pass left in the caches. 1.6 GB of fp32: 0.90 ms
// (norm 0.28 to 0.32, 5.0 to 5.7 TB/s; scaling 0.58, 5.6 TB/s read and
// written); 150 tensors of 30 million elements together, bf16 and fp32: 18 + 32 us;
// 4 tensors of 300000 elements together: 4 + 5 us, two launches.
#include "block_common.hpp"
#include "block_launch.hpp"

namespace mxgg {
namespace {

constexpr int kThreads = 256;
constexpr float kEps = 1e-6f;

// Largest magnitude that keeps NaN
__device__ __forceinline__ double max_nan(double a, double b) { return (b > a || b != b) ? b : a; }

template <bool MAX>
__device__ __forceinline__ double join(double a, double b) {
  if constexpr (MAX) return max_nan(a, b);
  return a + b;
}

// Over the workgroup, in every thread
template <bool MAX>
__device__ __forceinline__ double group_join(double v, double* lds) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = join<MAX>(v, __shfl_xor(v, d, 64));
  if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = v;
  __syncthreads();
  v = lds[0];
#pragma unroll
  for (int i = 1; i < kThreads / 64; ++i) v = join<MAX>(v, lds[i]);
  return v;
}

// The tensor that holds chunk c (first[t] <= c < first[t+1])
__device__ __forceinline__ int find_tensor(const ClipBatch& b, int c) {
  int lo = 0, hi = b.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (b.first[mid] <= c) lo = mid; else hi = mid;
  }
  return lo;
}

template <class E, bool MAX>
__device__ __forceinline__ void norm_chunk(const E* x, int64_t left, double& acc) {
  constexpr int N = Chunk<E>::N, PER = kClipChunk / (kThreads * N);
  Chunk<E> c[PER];
  if (left >= kClipChunk) {
#pragma unroll
    for (int i = 0; i < PER; ++i) c[i].load(x + (i * kThreads + threadIdx.x) * N);
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int at = (i * kThreads + threadIdx.x) * N;
      const int n = (int)left - at;
      if (n >= N) c[i].load(x + at);
      else c[i].load_part(x + at, n);
    }
  }
#pragma unroll
  for (int i = 0; i < PER; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const double v = (double)c[i].get(j);
      if constexpr (MAX) acc = max_nan(acc, fabs(v));
      else acc = fma(v, v, acc);
    }
}

template <bool MAX>
__global__ __launch_bounds__(kThreads) void grad_norm_kernel(ClipBatch b, double* part) {
  __shared__ double lds[kThreads / 64];
  double acc = 0.0;
  for (int c = blockIdx.x; c < b.chunks; c += gridDim.x) {
    const int t = find_tensor(b, c);
    const int64_t at = (int64_t)(c - b.first[t]) * kClipChunk, left = b.numel[t] - at;
    if (b.f32[t / 32] >> (t % 32) & 1)
      norm_chunk<float, MAX>(static_cast<const float*>(b.data[t]) + at, left, acc);
    else
      norm_chunk<bf16_t, MAX>(static_cast<const bf16_t*>(b.data[t]) + at, left, acc);
  }
  acc = group_join<MAX>(acc, lds);
  if (threadIdx.x == 0) part[blockIdx.x] = acc;
}

template <bool MAX>
__device__ __forceinline__ float norm_of(const double* part, int n, double* lds) {
  double v = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) v = join<MAX>(v, part[i]);
  v = group_join<MAX>(v, lds);
  return (float)(MAX ? v : sqrt(v));
}

template <bool MAX>
__global__ __launch_bounds__(kThreads) void grad_norm_total_kernel(const double* part, int n, float* total) {
  __shared__ double lds[kThreads / 64];
  const float norm = norm_of<MAX>(part, n, lds);
  if (threadIdx.x == 0) *total = norm;
}

template <class E>
__device__ __forceinline__ void scale_chunk(E* x, int64_t left, float coef) {
  constexpr int N = Chunk<E>::N, PER = kClipChunk / (kThreads * N);
  Chunk<E> c[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int at = (i * kThreads + threadIdx.x) * N;
    const int64_t n = left - at;
    if (n >= N) c[i].load(x + at);
    else c[i].load_part(x + at, n > 0 ? (int)n : 0);
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int at = (i * kThreads + threadIdx.x) * N;
    const int64_t n = left - at;
    float v[N];
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = c[i].get(j) * coef;
    c[i].set(v);
    if (n >= N) c[i].store(x + at);
    else c[i].store_part(x + at, n > 0 ? (int)n : 0);
  }
}

template <bool MAX>
__global__ __launch_bounds__(kThreads) void grad_clip_kernel(ClipBatch b, const double* part, int n, float max_norm,
                                                             float* total, int write) {
  __shared__ double lds[kThreads / 64];
  const float norm = n > 0 ? norm_of<MAX>(part, n, lds) : *total;
  if (write && blockIdx.x == 0 && threadIdx.x == 0) *total = norm;
  const float coef = max_norm / (norm + kEps);
  if (coef >= 1.f) return;   // nothing to scale: x * 1 is x (a NaN norm goes on)
  // from the end: what the norm pass read last is still in the caches
  for (int c = b.chunks - 1 - (int)blockIdx.x; c >= 0; c -= gridDim.x) {
    const int t = find_tensor(b, c);
    const int64_t at = (int64_t)(c - b.first[t]) * kClipChunk, left = b.numel[t] - at;
    if (b.f32[t / 32] >> (t % 32) & 1)
      scale_chunk<float>(static_cast<float*>(b.data[t]) + at, left, coef);
    else
      scale_chunk<bf16_t>(static_cast<bf16_t*>(b.data[t]) + at, left, coef);
  }
}

}  // namespace

hipError_t launch_norm_partials(const ClipBatch& b, bool max_norm_kind, double* part, hipStream_t st) {
  const dim3 grid((uint32_t)clip_groups(b.chunks));
  if (max_norm_kind) grad_norm_kernel<true><<<grid, kThreads, 0, st>>>(b, part);
  else grad_norm_kernel<false><<<grid, kThreads, 0, st>>>(b, part);
  return hipGetLastError();
}

hipError_t launch_norm_total(const double* part, int n, bool max_norm_kind, float* total, hipStream_t st) {
  if (max_norm_kind) grad_norm_total_kernel<true><<<1, kThreads, 0, st>>>(part, n, total);
  else grad_norm_total_kernel<false><<<1, kThreads, 0, st>>>(part, n, total);
  return hipGetLastError();
}

hipError_t launch_clip(const ClipBatch& b, const double* part, int n, bool max_norm_kind, float max_norm, float* total,
                       bool write, hipStream_t st) {
  const dim3 grid((uint32_t)clip_groups(b.chunks));
  if (max_norm_kind)
    grad_clip_kernel<true><<<grid, kThreads, 0, st>>>(b, part, n, max_norm, total, write ? 1 : 0);
  else
    grad_clip_kernel<false><<<grid, kThreads, 0, st>>>(b, part, n, max_norm, total, write ? 1 : 0);
  return hipGetLastError();
}

}  // namespace mxgg
