// Layer norm, forward and backward.
//
//   mu = sum x / C, var = sum (x - mu)^2 / C, rstd = (var + eps)^-1/2,
//   xh = (x - mu) rstd, y = xh w + b
//   g = dy w, dx = rstd (g - mean(g) - xh mean(g xh)),
//   dw = sum_rows dy xh, db = sum_rows dy
//
// A row belongs to L lanes that keep it in registers as 16-byte chunks (NV of
// them per lane), so x and dy are read once and the variance is taken about the
// mean of the same registers; the next row's chunks are on their way meanwhile.
// All sums are fp32.
//
// Both passes are bound by memory (all times in this file: medians of the
// profiler's kernel times; they vary by some 4 % between runs). Forward, 16384 x
// 7168 bf16: 94 us, 5.0 TB/s (a plain 2 GiB copy: 4.9). Backward, 4096 x 4096 bf16:
// 24.5 us, 4.1 TB/s, then 4 us for the columns' partial sums (8 MB); 2500 x 5001
// fp32: 30 + 4 us, 4.4 TB/s; 16384 x 7168 bf16: 136 + 5 us, 5.0 TB/s. Narrow rows
// are not: 65536 x 96 bf16 backward takes 14 + 4 us where its bytes take 8. None is
// moved twice (26 MB read, 13 written), but a CU has two loads of 12 lanes for each
// of its 64 rows in flight (25 KB), and waits for such a step four times. 8 x 4096
// forward: 3.4 us, the time of an empty launch and one trip to memory.
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
    constexpr int W = L / 64;
    const int wave = threadIdx.x / 64;
    if (threadIdx.x % 64 == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) lds[slot][wave][k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = lanes_sum<W>(lds[slot][wave / W * W + threadIdx.x % W][k]);
  }
}

// N values of a vector over the columns, as they lie in memory
template <class W, int N>
struct ColumnValues {
  static constexpr int M = Chunk<W>::N < N ? Chunk<W>::N : N;
  Chunk<W> c[N / M];
  __device__ __forceinline__ float get(int j) const { return c[j / M].get(j % M); }
  __device__ __forceinline__ void fill(float v) {
    float all[Chunk<W>::N];
#pragma unroll
    for (int i = 0; i < Chunk<W>::N; ++i) all[i] = v;
#pragma unroll
    for (int h = 0; h < N / M; ++h) c[h].set(all);
  }
};

// A lane's N columns. A chunk that would pass the row's end is moved back to
// end there; its first `skip` elements are its neighbour's then (all N in a lane
// past the end) and count here as nothing, so every access is a whole chunk. A
// row shorter than a chunk (SHORT) is read and written by element.
template <int N, bool SHORT>
struct Columns {
  int start, skip, size;
  __device__ __forceinline__ Columns(int col, int cols) {
    start = min(col, cols - N);
    if (SHORT) start = max(start, 0);
    skip = col - start;
    size = SHORT ? min(cols, N) : N;
  }
  __device__ __forceinline__ bool has(int j) const { return j >= skip && (!SHORT || j < size); }
  __device__ __forceinline__ bool any() const { return skip < size; }

  template <class E>
  __device__ __forceinline__ void load(Chunk<E>& c, const E* row) const {
    if (SHORT && size < N) c.load_part(row + start, size);
    else c.load(row + start);
  }
  template <class E>
  __device__ __forceinline__ void store(const Chunk<E>& c, E* row) const {
    if (SHORT && size < N) c.store_part(row + start, size);
    else c.store(row + start);
  }
  // the same columns of a vector
  template <class W>
  __device__ __forceinline__ void vector(ColumnValues<W, N>& v, const W* p) const {
    constexpr int M = ColumnValues<W, N>::M;
#pragma unroll
    for (int h = 0; h < N / M; ++h) {
      const int left = size - h * M;
      if (SHORT && left < M) v.c[h].load_part(p + start + h * M, max(left, 0));
      else memcpy(v.c[h].w, p + start + h * M, M * sizeof(W));
    }
  }
};

constexpr int kThreads = 1024;

// The G = T / L rows that a workgroup has at a time. It goes through rows
// blockIdx G, + gridDim G, ... with the weights in registers and the next
// rows' loads on their way while it works on these.
template <class E, class W, int L, int NV, int T>
__global__ __launch_bounds__(T) void layer_norm_fwd_kernel(NormFwdParams p) {
  constexpr int N = Chunk<E>::N, G = T / L;
  __shared__ float lds[2][T / 64][1];
  using Cols = Columns<N, L == 16>;
  const int lane = threadIdx.x % L;
  ColumnValues<W, N> w[NV], b[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const Cols at((i * L + lane) * N, p.cols);
    w[i].fill(1.f);
    b[i].fill(0.f);
    if (p.weight) at.vector(w[i], static_cast<const W*>(p.weight));
    if (p.bias) at.vector(b[i], static_cast<const W*>(p.bias));
  }
  // squares of (x - mu) / sqrt(C): their sum is the variance, and finite
  // wherever that is
  const float root = 1.f / sqrtf((float)p.cols);
  // and x over the power of two from C up (exact): no sum is larger than the
  // largest x
  const int bits = 32 - __clz(p.cols - 1);
  const float down = __uint_as_float((uint32_t)(127 - bits) << 23), count = (float)p.cols * down;
  const int64_t step = (int64_t)gridDim.x * G;
  int64_t row = (int64_t)blockIdx.x * G + threadIdx.x / L;
  Chunk<E> next[NV];
  const auto load = [&](int64_t r) {
    const E* x = static_cast<const E*>(p.x) + (r < p.rows ? r : p.rows - 1) * p.ldx;
#pragma unroll
    for (int i = 0; i < NV; ++i) Cols((i * L + lane) * N, p.cols).load(next[i], x);
  };
  load(row);
  for (int64_t base = (int64_t)blockIdx.x * G; base < p.rows; base += step, row += step) {
    Chunk<E> c[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) c[i] = next[i];
    if (base + step < p.rows) load(row + step);
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const Cols at((i * L + lane) * N, p.cols);
#pragma unroll
      for (int j = 0; j < N; ++j) s[0] = fmaf(at.has(j) ? c[i].get(j) : 0.f, down, s[0]);
    }
    row_sum<L, T, 1>(s, lds, 0);
    const float mean = s[0] / count;
    float q[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const Cols at((i * L + lane) * N, p.cols);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float d = (c[i].get(j) - mean) * root;
        q[0] += at.has(j) ? d * d : 0.f;
      }
    }
    row_sum<L, T, 1>(q, lds, 1);
    const float rstd = 1.f / sqrtf(q[0] + p.eps);
    if (row < p.rows) {
      if (lane == 0) {
        p.mean[row] = mean;
        p.rstd[row] = rstd;
      }
      E* y = static_cast<E*>(p.y) + row * p.ldy;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float v[N];
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = (c[i].get(j) - mean) * rstd * w[i].get(j) + b[i].get(j);
        Chunk<E> o;
        o.set(v);
        const Cols at((i * L + lane) * N, p.cols);
        if (at.any()) at.store(o, y);
      }
    }
  }
}

// The same walk, AHEAD steps of loads on their way, with the column sums of dy
// xh and dy in registers; at the end the G row groups meet in LDS and the
// workgroup writes one partial sum per column.
template <class E, class W, int L, int NV, int T, int AHEAD>
__global__ __launch_bounds__(T) void layer_norm_bwd_kernel(NormBwdParams p) {
  constexpr int N = Chunk<E>::N, G = T / L;
  __shared__ float lds[2][T / 64][2];
  __shared__ float cross[G > 1 ? T * N : 1];
  using Cols = Columns<N, L == 16>;
  const int lane = threadIdx.x % L, grp = threadIdx.x / L;
  float dw[NV][N], db[NV][N];
  ColumnValues<W, N> w[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int j = 0; j < N; ++j) dw[i][j] = db[i][j] = 0.f;
    w[i].fill(1.f);
    if (p.weight) Cols((i * L + lane) * N, p.cols).vector(w[i], static_cast<const W*>(p.weight));
  }
  const float inv = 1.f / (float)p.cols;
  const int64_t step = (int64_t)gridDim.x * G;
  int64_t row = (int64_t)blockIdx.x * G + grp;
  constexpr int SLOTS = AHEAD ? AHEAD : 1;
  Chunk<E> next_x[SLOTS][NV], next_g[SLOTS][NV];
  float next_mean[SLOTS], next_rstd[SLOTS];
  const auto load = [&](int b, int64_t r) {
    // a group past the last row reads that one, and counts it as zeros
    const int64_t at = r < p.rows ? r : p.rows - 1;
    const E* x = static_cast<const E*>(p.x) + at * p.ldx;
    const E* dy = static_cast<const E*>(p.dy) + at * p.lddy;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const Cols c((i * L + lane) * N, p.cols);
      c.load(next_x[b][i], x);
      c.load(next_g[b][i], dy);
    }
    next_mean[b] = p.mean[at];
    next_rstd[b] = p.rstd[at];
  };
#pragma unroll
  for (int b = 0; b < AHEAD; ++b)
    if (b == 0 || (int64_t)blockIdx.x * G + b * step < p.rows) load(b, row + b * step);
  int slot = 0;
  for (int64_t base = (int64_t)blockIdx.x * G; base < p.rows; base += step, row += step, slot ^= 1) {
    const bool on = row < p.rows;
    Chunk<E> cx[NV], cg[NV];
    if (AHEAD == 0) load(0, row);
    float mean = next_mean[0], rstd = next_rstd[0];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      cx[i] = next_x[0][i], cg[i] = next_g[0][i];
      // of a group past the last row nothing counts: its dy below, nor its x,
      // which is another group's dx by now where dx is over x; and with x, mean
      // and rstd 0 so is xh (0 - mean of a large row, times rstd, may pass fp32)
      if constexpr (G > 1)
#pragma unroll
        for (int k = 0; k < 4; ++k) cx[i].w[k] &= on ? ~0u : 0u;
    }
    if constexpr (G > 1) {
      mean = on ? mean : 0.f;
      rstd = on ? rstd : 0.f;
    }
#pragma unroll
    for (int b = 1; b < AHEAD; ++b) {
#pragma unroll
      for (int i = 0; i < NV; ++i) next_x[b - 1][i] = next_x[b][i], next_g[b - 1][i] = next_g[b][i];
      next_mean[b - 1] = next_mean[b];
      next_rstd[b - 1] = next_rstd[b];
    }
    if (AHEAD && base + AHEAD * step < p.rows) load(AHEAD - 1, row + AHEAD * step);
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const Cols at((i * L + lane) * N, p.cols);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        // an element that does not count has dy = 0; one of the row's own is not
        // finite in xh where the row's results are not either, one past a short
        // row's end (0 - mean, times rstd) is taken as 0
        float xh = (cx[i].get(j) - mean) * rstd;
        if constexpr (L == 16) xh = at.has(j) ? xh : 0.f;
        const float d = on && at.has(j) ? cg[i].get(j) : 0.f;
        s[0] += d * w[i].get(j);
        s[1] += d * w[i].get(j) * xh;
        dw[i][j] += d * xh;
        db[i][j] += d;
      }
    }
    row_sum<L, T, 2>(s, lds, slot);
    const float c1 = s[0] * inv, c2 = s[1] * inv;
    if (on) {
      E* dx = static_cast<E*>(p.dx) + row * p.lddx;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float v[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const float xh = (cx[i].get(j) - mean) * rstd;
          v[j] = rstd * (cg[i].get(j) * w[i].get(j) - c1 - xh * c2);
        }
        Chunk<E> o;
        o.set(v);
        const Cols at((i * L + lane) * N, p.cols);
        if (at.any()) at.store(o, dx);
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
        for (int e = threadIdx.x; e < L * N; e += T) {
          const int j = e / L, l = e % L;
          const Cols at((i * L + l) * N, p.cols);
          float t = 0.f;
          for (int g = 0; g < G; ++g) t += cross[(g * N + j) * L + l];
          if (at.has(j)) part[(int64_t)k * p.cols + at.start + j] = t;
        }
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const Cols at((i * L + lane) * N, p.cols);
          if (at.has(j)) part[(int64_t)k * p.cols + at.start + j] = v[j];
        }
      }
    }
}

// Column sums of the partials: a wave's lanes take 64 neighbouring columns of
// dweight (blockIdx.y == 0) or dbias, the workgroup's waves every 16th partial.
__global__ __launch_bounds__(kThreads) void layer_norm_grad_kernel(const float* part, int n, int cols, float* dweight,
                                                                   float* dbias, int accumulate) {
  float* out = blockIdx.y ? dbias : dweight;
  if (!out) return;
  constexpr int WAVES = kThreads / 64;
  __shared__ float lds[WAVES][64];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int col = blockIdx.x * 64 + lane;
  float s = 0.f;
  if (col < cols) {
    const float* q = part + (int64_t)blockIdx.y * cols + col;
#pragma unroll 8
    for (int i = wave; i < n; i += WAVES) s += q[(int64_t)i * 2 * cols];
  }
  lds[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && col < cols) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) s += lds[i][lane];
    out[col] = accumulate ? out[col] + s : s;
  }
}

// Lanes of a row: two chunks each where the row has them, since a wave then has
// twice the bytes in flight for the same barriers (forward, 16384 rows of bf16:
// 2048 columns 25.6 us with two chunks a lane, 30.7 with one; 4096 columns 48.5 and
// 60.4; 7168 columns 90.9, with one 121, with four 95.8).
//
// The forward's grid goes up to 2^20 threads, eight 512-thread workgroups for
// each CU's two: a grid that still evens out (16384 x 7168: 90.9 us; one that just
// fills the card 98.7), and rows enough in a workgroup that the weights are not
// loaded for each (one row a workgroup: 90.6, the same). The backward has one
// workgroup a CU, because each writes a partial of both gradients (4096 x 4096, both
// launches: 28.8 us; two a CU 37.0).
constexpr int kFwdThreads = 1 << 20, kBwdGroups = 256;

template <class E, class W, int L, int NV>
hipError_t fwd(const NormFwdParams& p, hipStream_t st) {
  constexpr int T = L < 256 ? 256 : L, G = T / L, MOST = kFwdThreads / T;
  const int64_t need = (p.rows + G - 1) / G;
  layer_norm_fwd_kernel<E, W, L, NV, T><<<(uint32_t)(need < MOST ? need : MOST), T, 0, st>>>(p);
  return hipGetLastError();
}

template <class E, class W, int L, int NV>
hipError_t bwd(const NormBwdParams& p, int& grid, hipStream_t st) {
  // 512 threads leave a thread the registers for the column sums and the rows
  // on their way; rows of 16 lanes need few (65536 x 96, both launches: 18.0 us with
  // 1024 threads, 20.6 with 512; two rows ahead there 19.5). Two rows ahead rather
  // than one: 16384 x 7168 bf16 140 us and 158 (three: 141); 4096 x 4096 28.8 and
  // 31.6. With one chunk a lane four (32768 x 500: 25.4 us; two 24.7, one 32.5).
  // Where the registers would spill, none: 2048 x 16384 fp32 98 us, with one 147;
  // 4096 x 14000 bf16 91 and 100. (fp32 rows of 1024 lanes have 128 registers a
  // thread and spill 3 or 4 of them all the same; no other form spills.)
  constexpr int T = L == 16 ? 1024 : L < 512 ? 512 : L, G = T / L;
  constexpr int AHEAD = L == 16 ? 1 : NV == 1 ? 4 : NV == 4 ? 0 : 2;
  const int64_t need = (p.rows + G - 1) / G;
  grid = (int)(need < kBwdGroups ? need : kBwdGroups);
  layer_norm_bwd_kernel<E, W, L, NV, T, AHEAD><<<grid, T, 0, st>>>(p);
  return hipGetLastError();
}

template <class E, class W>
hipError_t fwd_any(const NormFwdParams& p, hipStream_t st) {
  const int chunks = (p.cols + Chunk<E>::N - 1) / Chunk<E>::N;
  if (chunks <= 16) return fwd<E, W, 16, 1>(p, st);
  if (chunks <= 64) return fwd<E, W, 64, 1>(p, st);
  if (chunks <= 128) return fwd<E, W, 64, 2>(p, st);
  if (chunks <= 256) return fwd<E, W, 128, 2>(p, st);
  if (chunks <= 512) return fwd<E, W, 256, 2>(p, st);
  if (chunks <= 1024) return fwd<E, W, 512, 2>(p, st);
  if constexpr (Chunk<E>::N == 4)   // bf16 rows have 2048 chunks at most
    if (chunks > 2048) return fwd<E, W, 1024, 4>(p, st);
  return fwd<E, W, 1024, 2>(p, st);
}

template <class E, class W>
hipError_t bwd_any(const NormBwdParams& p, int& grid, hipStream_t st) {
  const int chunks = (p.cols + Chunk<E>::N - 1) / Chunk<E>::N;
  if (chunks <= 16) return bwd<E, W, 16, 1>(p, grid, st);
  if (chunks <= 64) return bwd<E, W, 64, 1>(p, grid, st);
  if (chunks <= 128) return bwd<E, W, 64, 2>(p, grid, st);
  if (chunks <= 256) return bwd<E, W, 128, 2>(p, grid, st);
  if (chunks <= 512) return bwd<E, W, 256, 2>(p, grid, st);
  if (chunks <= 768) return bwd<E, W, 256, 3>(p, grid, st);
  if (chunks <= 1024) return bwd<E, W, 512, 2>(p, grid, st);
  if (chunks <= 1536) return bwd<E, W, 512, 3>(p, grid, st);
  if constexpr (Chunk<E>::N == 4)
    if (chunks > 2048) return bwd<E, W, 1024, 4>(p, grid, st);
  return bwd<E, W, 512, 4>(p, grid, st);
}

}  // namespace

int norm_bwd_groups(int64_t rows) { return (int)(rows < kBwdGroups ? rows : kBwdGroups); }

hipError_t launch_layer_norm_fwd(const NormFwdParams& p, bool f32, bool wf32, hipStream_t st) {
  if (f32) return wf32 ? fwd_any<float, float>(p, st) : fwd_any<float, bf16_t>(p, st);
  return wf32 ? fwd_any<bf16_t, float>(p, st) : fwd_any<bf16_t, bf16_t>(p, st);
}

hipError_t launch_layer_norm_bwd(const NormBwdParams& p, bool f32, bool wf32, float* dweight, float* dbias,
                                 bool accumulate, hipStream_t st) {
  int grid = 0;   // without rows the sums are of nothing
  hipError_t e = hipSuccess;
  if (p.rows > 0) {
    if (f32) e = wf32 ? bwd_any<float, float>(p, grid, st) : bwd_any<float, bf16_t>(p, grid, st);
    else e = wf32 ? bwd_any<bf16_t, float>(p, grid, st) : bwd_any<bf16_t, bf16_t>(p, grid, st);
  }
  if (e != hipSuccess || (!dweight && !dbias)) return e;
  layer_norm_grad_kernel<<<dim3((uint32_t)((p.cols + 63) / 64), 2), kThreads, 0, st>>>(
      p.part, grid, p.cols, dweight, dbias, accumulate ? 1 : 0);
  return hipGetLastError();
}

}  // namespace mxgg
