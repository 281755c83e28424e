// Layer norm, forward and backward.
//
//   mu = sum x / C, var = sum (x - mu)^2 / C, rstd = (var + eps)^-1/2,
//   xh = (x - mu) rstd, y = xh w + b
//   g = dy w, dx = rstd (g - mean(g) - xh mean(g xh)),
//   dw = sum_rows dy xh, db = sum_rows dy
//
// A row belongs to L lanes (L <= 1024) that keep it in registers as 16-byte
// chunks (NV of them per lane), so x and dy are read once and the variance is
// taken about the mean of the same registers. All sums are fp32.
#include "block_common.hpp"
#include "block_launch.hpp"

namespace mxgg {
namespace {

// Sums of K values over the L lanes of a row, in every lane. Rows of more than
// one wave meet in LDS; `slot` alternates between calls so that one barrier a
// call is enough (a slot is written again only after the next call's barrier).
template <int L, int THREADS, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float (*lds)[THREADS / 64][K], int slot) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = lanes_sum<(L < 64 ? L : 64)>(v[k]);
  if constexpr (L > 64) {
    const int wave = threadIdx.x / 64;
    if (threadIdx.x % 64 == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) lds[slot][wave][k] = v[k];
    __syncthreads();
    const int first = wave / (L / 64) * (L / 64);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < L / 64; ++i) s += lds[slot][first + i][k];
      v[k] = s;
    }
  }
}

template <class E>
__device__ __forceinline__ void load_chunk(Chunk<E>& c, const E* row, int col, int cols) {
  const int left = cols - col;
  if (left >= Chunk<E>::N)
    c.load(row + col);
  else if (left > 0)
    c.load_part(row + col, left);
  else
    c.w[0] = c.w[1] = c.w[2] = c.w[3] = 0;
}

template <class E>
__device__ __forceinline__ void store_chunk(const Chunk<E>& c, E* row, int col, int cols) {
  const int left = cols - col;
  if (left >= Chunk<E>::N)
    c.store(row + col);
  else if (left > 0)
    c.store_part(row + col, left);
}

// N consecutive values of a per-column vector (N = 4 or 8), as fp32
template <class W, int N>
__device__ __forceinline__ void load_cols(float (&v)[N], const W* p, int col, int cols) {
  constexpr int M = Chunk<W>::N < N ? Chunk<W>::N : N;
#pragma unroll
  for (int h = 0; h < N / M; ++h) {
    Chunk<W> c;
    if constexpr (M == Chunk<W>::N) {
      load_chunk(c, p, col + h * M, cols);
    } else {            // 4 bf16 for 4 fp32
      const int left = cols - col;
      if (left >= M) memcpy(c.w, p + col, M * sizeof(W));
      else c.load_part(p + col, left > 0 ? left : 0);
    }
#pragma unroll
    for (int i = 0; i < M; ++i) v[h * M + i] = c.get(i);
  }
}

template <class E, class W, int L, int NV, int THREADS>
__global__ __launch_bounds__(THREADS) void layer_norm_fwd_kernel(NormFwdParams p) {
  constexpr int N = Chunk<E>::N, G = THREADS / L;
  __shared__ float lds[2][THREADS / 64][1];
  const int lane = threadIdx.x % L;
  const int64_t row = (int64_t)blockIdx.x * G + threadIdx.x / L;
  const bool on = row < p.rows;
  const E* x = static_cast<const E*>(p.x) + (on ? row : 0) * p.ldx;
  Chunk<E> c[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) load_chunk(c[i], x, (i * L + lane) * N, p.cols);
  float s[1] = {0.f};
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) s[0] += c[i].get(j);
  row_sum<L, THREADS, 1>(s, lds, 0);
  const float mean = s[0] / (float)p.cols;
  // squares of (x - mu) / sqrt(C): their sum is the variance, and finite
  // wherever that is
  const float root = 1.f / sqrtf((float)p.cols);
  float q[1] = {0.f};
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float d = (c[i].get(j) - mean) * root;
      q[0] += (i * L + lane) * N + j < p.cols ? d * d : 0.f;
    }
  row_sum<L, THREADS, 1>(q, lds, 1);
  const float rstd = 1.f / sqrtf(q[0] + p.eps);
  if (!on) return;
  if (lane == 0) {
    p.mean[row] = mean;
    p.rstd[row] = rstd;
  }
  E* y = static_cast<E*>(p.y) + row * p.ldy;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * L + lane) * N;
    float v[N], t[N];
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = (c[i].get(j) - mean) * rstd;
    if (p.weight) {
      load_cols<W, N>(t, static_cast<const W*>(p.weight), col, p.cols);
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] *= t[j];
    }
    if (p.bias) {
      load_cols<W, N>(t, static_cast<const W*>(p.bias), col, p.cols);
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] += t[j];
    }
    Chunk<E> o;
    o.set(v);
    store_chunk(o, y, col, p.cols);
  }
}

// A workgroup walks rows blockIdx, + gridDim, ... (G rows at a time) and keeps
// its column sums of dy xh and dy in registers; at the end the G row groups
// meet in LDS and the workgroup writes one partial sum per column.
template <class E, class W, int L, int NV, int THREADS>
__global__ __launch_bounds__(THREADS) void layer_norm_bwd_kernel(NormBwdParams p) {
  constexpr int N = Chunk<E>::N, G = THREADS / L;
  __shared__ float lds[2][THREADS / 64][2];
  __shared__ float cross[G > 1 ? THREADS * N : 1];
  const int lane = threadIdx.x % L, grp = threadIdx.x / L;
  float dw[NV][N], db[NV][N];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) dw[i][j] = db[i][j] = 0.f;
  const float inv = 1.f / (float)p.cols;
  int slot = 0;
  for (int64_t base = (int64_t)blockIdx.x * G; base < p.rows; base += (int64_t)gridDim.x * G, slot ^= 1) {
    const int64_t row = base + grp;
    const bool on = row < p.rows;   // a group past the last row adds zeros
    const E* x = static_cast<const E*>(p.x) + (on ? row : 0) * p.ldx;
    const E* dy = static_cast<const E*>(p.dy) + (on ? row : 0) * p.lddy;
    const float mean = on ? p.mean[row] : 0.f, rstd = on ? p.rstd[row] : 0.f;
    const int cols = on ? p.cols : 0;
    Chunk<E> cx[NV], cg[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      load_chunk(cx[i], x, (i * L + lane) * N, cols);
      load_chunk(cg[i], dy, (i * L + lane) * N, cols);
    }
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * L + lane) * N;
      float w[N];
      if (p.weight) {
        load_cols<W, N>(w, static_cast<const W*>(p.weight), col, p.cols);
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) w[j] = 1.f;
      }
#pragma unroll
      for (int j = 0; j < N; ++j) {
        // past the row's end dy and w are 0, but xh is not
        const float xh = col + j < cols ? (cx[i].get(j) - mean) * rstd : 0.f, d = cg[i].get(j);
        s[0] += d * w[j];
        s[1] += d * w[j] * xh;
        dw[i][j] += d * xh;
        db[i][j] += d;
      }
    }
    row_sum<L, THREADS, 2>(s, lds, slot);
    const float c1 = s[0] * inv, c2 = s[1] * inv;
    if (on) {
      E* dx = static_cast<E*>(p.dx) + row * p.lddx;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = (i * L + lane) * N;
        float w[N], v[N];
        if (p.weight) {
          load_cols<W, N>(w, static_cast<const W*>(p.weight), col, p.cols);
        } else {
#pragma unroll
          for (int j = 0; j < N; ++j) w[j] = 1.f;
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const float xh = (cx[i].get(j) - mean) * rstd;
          v[j] = rstd * (cg[i].get(j) * w[j] - c1 - xh * c2);
        }
        Chunk<E> o;
        o.set(v);
        store_chunk(o, dx, col, p.cols);
      }
    }
  }
  float* part = p.part + (int64_t)blockIdx.x * 2 * p.cols;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float(&v)[N] = k ? db[i] : dw[i];
      if constexpr (G > 1) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < N; ++j) cross[(grp * N + j) * L + lane] = v[j];
        __syncthreads();
        for (int e = threadIdx.x; e < L * N; e += THREADS) {
          const int j = e / L, l = e % L, col = (i * L + l) * N + j;
          float t = 0.f;
          for (int g = 0; g < G; ++g) t += cross[(g * N + j) * L + l];
          if (col < p.cols) part[(int64_t)k * p.cols + col] = t;
        }
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const int col = (i * L + lane) * N + j;
          if (col < p.cols) part[(int64_t)k * p.cols + col] = v[j];
        }
      }
    }
}

// Column sums of the partials: 16 columns of dweight (blockIdx.y == 0) or
// dbias per workgroup, 16 lanes of each wave on consecutive columns.
__global__ __launch_bounds__(256) void layer_norm_grad_kernel(const float* part, int n, int cols, float* dweight,
                                                              float* dbias, int accumulate) {
  float* out = blockIdx.y ? dbias : dweight;
  if (!out) return;
  __shared__ float lds[16][17];
  const int c = threadIdx.x % 16, r = threadIdx.x / 16;
  const int col = blockIdx.x * 16 + c;
  float s = 0.f;
  if (col < cols) {
    const float* q = part + (int64_t)blockIdx.y * cols + col;
#pragma unroll 4
    for (int i = r; i < n; i += 16) s += q[(int64_t)i * 2 * cols];
  }
  lds[r][c] = s;
  __syncthreads();
  if (r == 0 && col < cols) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += lds[i][c];
    out[col] = accumulate ? out[col] + s : s;
  }
}

template <class E, class W, int L, int NV>
hipError_t fwd(const NormFwdParams& p, hipStream_t st) {
  constexpr int T = L < 256 ? 256 : L;
  const int64_t grid = (p.rows + T / L - 1) / (T / L);
  layer_norm_fwd_kernel<E, W, L, NV, T><<<dim3((uint32_t)grid), dim3(T), 0, st>>>(p);
  return hipGetLastError();
}

template <class E, class W, int L, int NV>
hipError_t bwd(const NormBwdParams& p, int grid, hipStream_t st) {
  constexpr int T = L < 512 ? 512 : L;
  layer_norm_bwd_kernel<E, W, L, NV, T><<<dim3((uint32_t)grid), dim3(T), 0, st>>>(p);
  return hipGetLastError();
}

template <class E, class W>
hipError_t fwd_any(const NormFwdParams& p, hipStream_t st) {
  const int chunks = (p.cols + Chunk<E>::N - 1) / Chunk<E>::N;
  if (chunks <= 16) return fwd<E, W, 16, 1>(p, st);
  if (chunks <= 64) return fwd<E, W, 64, 1>(p, st);
  if (chunks <= 128) return fwd<E, W, 64, 2>(p, st);
  if (chunks <= 256) return fwd<E, W, 256, 1>(p, st);
  if (chunks <= 512) return fwd<E, W, 256, 2>(p, st);
  if (chunks <= 1024) return fwd<E, W, 256, 4>(p, st);
  if (chunks <= 2048) return fwd<E, W, 1024, 2>(p, st);
  return fwd<E, W, 1024, 4>(p, st);
}

template <class E, class W>
hipError_t bwd_any(const NormBwdParams& p, int grid, hipStream_t st) {
  const int chunks = (p.cols + Chunk<E>::N - 1) / Chunk<E>::N;
  if (chunks <= 16) return bwd<E, W, 16, 1>(p, grid, st);
  if (chunks <= 64) return bwd<E, W, 64, 1>(p, grid, st);
  if (chunks <= 128) return bwd<E, W, 64, 2>(p, grid, st);
  if (chunks <= 256) return bwd<E, W, 256, 1>(p, grid, st);
  if (chunks <= 512) return bwd<E, W, 256, 2>(p, grid, st);
  if (chunks <= 1024) return bwd<E, W, 512, 2>(p, grid, st);
  if (chunks <= 2048) return bwd<E, W, 1024, 2>(p, grid, st);
  return bwd<E, W, 1024, 4>(p, grid, st);
}

}  // namespace

int norm_bwd_groups(int64_t rows, int64_t cols) {
  (void)cols;
  const int64_t most = 512;
  return (int)(rows < most ? rows : most);
}

hipError_t launch_layer_norm_fwd(const NormFwdParams& p, bool f32, bool wf32, hipStream_t st) {
  if (f32) return wf32 ? fwd_any<float, float>(p, st) : fwd_any<float, bf16_t>(p, st);
  return wf32 ? fwd_any<bf16_t, float>(p, st) : fwd_any<bf16_t, bf16_t>(p, st);
}

hipError_t launch_layer_norm_bwd(const NormBwdParams& p, bool f32, bool wf32, float* dweight, float* dbias,
                                 bool accumulate, hipStream_t st) {
  const int grid = norm_bwd_groups(p.rows, p.cols);
  hipError_t e = hipSuccess;
  if (grid > 0) {
    if (f32) e = wf32 ? bwd_any<float, float>(p, grid, st) : bwd_any<float, bf16_t>(p, grid, st);
    else e = wf32 ? bwd_any<bf16_t, float>(p, grid, st) : bwd_any<bf16_t, bf16_t>(p, grid, st);
  }
  if (e != hipSuccess || (!dweight && !dbias)) return e;
  layer_norm_grad_kernel<<<dim3((uint32_t)((p.cols + 15) / 16), 2), dim3(256), 0, st>>>(
      p.part, grid, p.cols, dweight, dbias, accumulate ? 1 : 0);
  return hipGetLastError();
}

}  // namespace mxgg
