// Tokens to their experts and back.
//
//   sort      the choices of a router in the order of their experts (stable)
//   dispatch  out[place(t, j)] = x[t]
//   combine   out[t] = sum_j w[t, j] y[place(t, j)]
//   and its gradients: dy[place(t, j)] = w[t, j] d[t],
//             dw[t, j] = sum_c d[t, c] y[place(t, j), c]
//
// The gradient of dispatch is combine without weights. A dropped choice (its
// expert outside [0, E)) is sorted behind all others; rows holds ~place for it,
// so dispatch and the gradient know which rows to clear and combine which to
// leave out, without a second list.
#include "block_common.hpp"
#include "token_launch.hpp"

namespace mxgg {
namespace {

// ---------------------------------------------------------------------------
// Sort
//
// A wave owns a run of choices and takes them 64 at a time: the lanes that hold
// the same expert find each other with one ballot for each bit of the expert's
// number, the first of them counts all in LDS, and a lane's place among the
// wave's choices of its expert is what the counter held and the lanes of its
// kind below it. So the order is that of the choices: no atomic whose order
// matters.

constexpr int kSortBits = 10;   // experts + 1 <= 513

template <class I>
__device__ __forceinline__ int sort_key(const SortParams& p, int c) {
  int64_t at = c;
  if (p.ldi != p.top_k) {
    const int t = c / p.top_k;
    at = t * p.ldi + (c - t * p.top_k);
  }
  const I id = static_cast<const I*>(p.ids)[at];
  return id >= 0 && id < (I)p.experts ? (int)id : p.experts;
}

// Counts the `have` lanes' keys into cnt; a lane's place among them and what
// cnt held.
__device__ __forceinline__ int count_keys(int32_t* cnt, int key, bool have, int bits) {
  uint64_t same = __ballot(have);
  for (int b = 0; b < bits; ++b) {
    const uint64_t set = __ballot((key >> b) & 1);
    same &= (key >> b) & 1 ? set : ~set;
  }
  const int lane = threadIdx.x & 63;
  const int first = have ? __ffsll((unsigned long long)same) - 1 : lane;
  int before = 0;
  if (have && lane == first) before = atomicAdd(cnt + key, (int32_t)__popcll(same));
  before = __shfl(before, first, 64);
  return before + (int)__popcll(same & ((1ull << lane) - 1));
}

// Exclusive prefix sum over the block's threads.
template <int THREADS>
__device__ __forceinline__ int32_t block_exclusive(int32_t v, int32_t* part) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int32_t sum = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int32_t o = __shfl_up(sum, d, 64);
    if (lane >= d) sum += o;
  }
  if (lane == 63) part[wave] = sum;
  __syncthreads();
  int32_t base = 0;
  for (int w = 0; w < wave; ++w) base += part[w];
  return base + sum - v;
}

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kSortPer = kSortChunk / kSortThreads;   // choices of a lane
constexpr int kSortKeys = kMaxExperts + 1;
static_assert(kSortKeys <= kSortThreads && kSortKeys <= 1 << kSortBits, "a thread for each key");

// The chunk's choices: keys, and their places among those of the same key in
// the chunk; thread e < experts + 1 gets key e's count.
template <class I>
__device__ __forceinline__ int32_t sort_chunk(const SortParams& p, int first, int32_t (*cnt)[kSortKeys],
                                              int (&key)[kSortPer], int (&place)[kSortPer]) {
  const int keys = p.experts + 1, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int bits = 32 - __clz(p.experts);
  for (int e = lane; e < keys; e += 64) cnt[wave][e] = 0;
  const int run = first + wave * (64 * kSortPer) + lane;
#pragma unroll
  for (int i = 0; i < kSortPer; ++i) {
    const int c = run + i * 64;
    key[i] = c < p.n ? sort_key<I>(p, c) : p.experts;
  }
#pragma unroll
  for (int i = 0; i < kSortPer; ++i) place[i] = count_keys(cnt[wave], key[i], run + i * 64 < p.n, bits);
  __syncthreads();
  int32_t total = 0;
  if ((int)threadIdx.x < keys) {
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const int32_t v = cnt[w][threadIdx.x];
      cnt[w][threadIdx.x] = total;
      total += v;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSortPer; ++i) place[i] += cnt[wave][key[i]];
  return total;
}

__device__ __forceinline__ void store_place(const SortParams& p, int c, int key, int32_t place) {
  p.rows[c] = key < p.experts ? place : ~place;
  p.choices[place] = c;
}

// One chunk: all in one workgroup.
template <class I>
__global__ __launch_bounds__(kSortThreads) void sort_one_kernel(SortParams p) {
  __shared__ int32_t cnt[kSortWaves][kSortKeys];
  __shared__ int32_t base[kSortKeys], part[kSortWaves];
  int key[kSortPer], place[kSortPer];
  const int32_t total = sort_chunk<I>(p, 0, cnt, key, place);
  const int32_t at = block_exclusive<kSortThreads>(total, part);
  if ((int)threadIdx.x <= p.experts) base[threadIdx.x] = at;
  if ((int)threadIdx.x < p.experts) p.counts[threadIdx.x] = total;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSortPer; ++i) {
    const int c = (int)(threadIdx.x >> 6) * (64 * kSortPer) + i * 64 + (threadIdx.x & 63);
    if (c < p.n) store_place(p, c, key[i], base[key[i]] + place[i]);
  }
}

// Several: each one's counts and the places inside it, ...
template <class I>
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortParams p) {
  __shared__ int32_t cnt[kSortWaves][kSortKeys];
  int key[kSortPer], place[kSortPer];
  const int first = (int)blockIdx.x * kSortChunk;
  const int32_t total = sort_chunk<I>(p, first, cnt, key, place);
  if ((int)threadIdx.x <= p.experts) p.table[(int64_t)blockIdx.x * (p.experts + 1) + threadIdx.x] = total;
#pragma unroll
  for (int i = 0; i < kSortPer; ++i) {
    const int c = first + (int)(threadIdx.x >> 6) * (64 * kSortPer) + i * 64 + (threadIdx.x & 63);
    if (c < p.n) p.rows[c] = place[i];
  }
}

// ... the counts before each chunk (the totals behind the last), one wave a key ...
__global__ __launch_bounds__(64) void sort_scan_kernel(SortParams p, int chunks) {
  const int keys = p.experts + 1;
  int32_t* col = p.table + blockIdx.x;
  int32_t base = 0;
  for (int b0 = 0; b0 < chunks; b0 += 64) {
    const int b = b0 + (int)threadIdx.x;
    const int32_t v = b < chunks ? col[(int64_t)b * keys] : 0;
    int32_t sum = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int32_t o = __shfl_up(sum, d, 64);
      if ((int)threadIdx.x >= d) sum += o;
    }
    if (b < chunks) col[(int64_t)b * keys] = base + sum - v;
    base += __shfl(sum, 63, 64);
  }
  if (threadIdx.x == 0) col[(int64_t)chunks * keys] = base;
}

// ... and the places of all. SCANNED: the table holds what the launch above made
// of it; else every workgroup adds its columns up.
template <class I, bool SCANNED>
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(SortParams p, int chunks) {
  __shared__ int32_t base[kSortKeys], part[kSortWaves];
  const int keys = p.experts + 1, e = threadIdx.x, mine = blockIdx.x;
  const int first = mine * kSortChunk;
  int key[kSortPer], place[kSortPer];
#pragma unroll
  for (int i = 0; i < kSortPer; ++i) {
    const int c = first + i * kSortThreads + e;
    if (c < p.n) {
      key[i] = sort_key<I>(p, c);
      place[i] = p.rows[c];
    }
  }
  int32_t before = 0, total = 0;
  if (e < keys) {
    if constexpr (SCANNED) {
      before = p.table[(int64_t)mine * keys + e];
      total = p.table[(int64_t)chunks * keys + e];
    } else {
#pragma unroll 16
      for (int b = 0; b < chunks; ++b) {
        const int32_t v = p.table[(int64_t)b * keys + e];
        before += b < mine ? v : 0;
        total += v;
      }
    }
  }
  const int32_t at = block_exclusive<kSortThreads>(total, part);
  if (e < keys) base[e] = at + before;
  if (mine == 0 && e < p.experts) p.counts[e] = total;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSortPer; ++i) {
    const int c = first + i * kSortThreads + e;
    if (c < p.n) store_place(p, c, key[i], base[key[i]] + place[i]);
  }
}

template <class I>
hipError_t sort_any(const SortParams& p, hipStream_t st) {
  const int64_t chunks = sort_chunks(p.n);
  if (chunks <= 1) {
    sort_one_kernel<I><<<1, kSortThreads, 0, st>>>(p);
    return hipGetLastError();
  }
  sort_count_kernel<I><<<(uint32_t)chunks, kSortThreads, 0, st>>>(p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (chunks <= kSortDirect) {
    sort_place_kernel<I, false><<<(uint32_t)chunks, kSortThreads, 0, st>>>(p, (int)chunks);
    return hipGetLastError();
  }
  sort_scan_kernel<<<(uint32_t)p.experts + 1, 64, 0, st>>>(p, (int)chunks);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  sort_place_kernel<I, true><<<(uint32_t)chunks, kSortThreads, 0, st>>>(p, (int)chunks);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Rows
//
// A token's row belongs to L lanes (a power of two, up to the workgroup); a lane
// takes 16-byte chunks L apart.

constexpr int kRowThreads = 256;
constexpr int64_t kRowGrid = 1 << 20;   // workgroups along the tokens at most; they stay for the rest

// The chunk at `col`, moved back to end with the row (its first elements are its
// neighbour's then, and written twice with the same bits); a row shorter than a
// chunk goes by element.
template <class E>
struct RowChunk {
  static constexpr int N = Chunk<E>::N;
  int start, size;
  __device__ __forceinline__ RowChunk(int col, int cols) {
    start = max(min(col, cols - N), 0);
    size = min(cols, N);
  }
  __device__ __forceinline__ void load(Chunk<E>& c, const E* row) const {
    if (size < N) c.load_part(row, size);
    else c.load(row + start);
  }
  __device__ __forceinline__ void store(const Chunk<E>& c, E* row) const {
    if (size < N) c.store_part(row, size);
    else c.store(row + start);
  }
};

template <class E>
__global__ __launch_bounds__(kRowThreads) void dispatch_kernel(TokenParams p, int lanes) {
  constexpr int N = Chunk<E>::N;
  const int per = kRowThreads / lanes, lane = threadIdx.x % lanes;
  const int col = ((int)blockIdx.y * lanes + lane) * N;
  if (col >= p.cols) return;
  const RowChunk<E> at(col, p.cols);
  for (int64_t t = (int64_t)blockIdx.x * per + threadIdx.x / lanes; t < p.tokens; t += (int64_t)gridDim.x * per) {
    Chunk<E> c, zero{};
    at.load(c, static_cast<const E*>(p.x) + t * p.ldx);
    for (int j = 0; j < p.top_k; ++j) {
      const int32_t r = p.rows[t * p.top_k + j];
      const int32_t to = r < 0 ? ~r : r;
      if (to < p.expert_rows) at.store(r < 0 ? zero : c, static_cast<E*>(p.out) + to * p.ldo);
    }
  }
}

template <class E, bool WEIGHTED>
__global__ __launch_bounds__(kRowThreads) void combine_kernel(TokenParams p, int lanes) {
  constexpr int N = Chunk<E>::N;
  const int per = kRowThreads / lanes, lane = threadIdx.x % lanes;
  const int col = ((int)blockIdx.y * lanes + lane) * N;
  if (col >= p.cols) return;
  const RowChunk<E> at(col, p.cols);
  for (int64_t t = (int64_t)blockIdx.x * per + threadIdx.x / lanes; t < p.tokens; t += (int64_t)gridDim.x * per) {
    float sum[N] = {};
    for (int j = 0; j < p.top_k; ++j) {
      const int32_t r = p.rows[t * p.top_k + j];
      if (r < 0 || r >= p.expert_rows) continue;
      const float w = WEIGHTED ? p.weights[t * p.top_k + j] : 1.f;
      Chunk<E> c;
      at.load(c, static_cast<const E*>(p.y) + r * p.ldy);
#pragma unroll
      for (int i = 0; i < N; ++i) sum[i] += WEIGHTED ? w * c.get(i) : c.get(i);
    }
    Chunk<E> o;
    o.set(sum);
    at.store(o, static_cast<E*>(p.out) + t * p.ldo);
  }
}

// One workgroup a token: the weights' gradients are sums over the whole row.
template <class E>
__global__ __launch_bounds__(kRowThreads) void combine_bwd_kernel(TokenParams p) {
  constexpr int N = Chunk<E>::N;
  __shared__ float part[kRowThreads / 64];
  for (int64_t t = blockIdx.x; t < p.tokens; t += gridDim.x) {
    const E* d = static_cast<const E*>(p.x) + t * p.ldx;
    for (int j = 0; j < p.top_k; ++j) {
      const int32_t r = p.rows[t * p.top_k + j];
      const int32_t to = r < 0 ? ~r : r;
      const bool here = to < p.expert_rows, kept = r >= 0 && here;
      const float w = kept ? p.weights[t * p.top_k + j] : 0.f;
      float dot = 0.f;
      if (here)
        for (int col = (int)threadIdx.x * N; col < p.cols; col += kRowThreads * N) {
          const RowChunk<E> at(col, p.cols);
          Chunk<E> c, o{};
          if (kept) {
            Chunk<E> y;
            at.load(c, d);
            at.load(y, static_cast<const E*>(p.y) + r * p.ldy);
            float v[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
              // a moved chunk's first elements count in their own lane
              if (at.start + i >= col && i < at.size) dot += c.get(i) * y.get(i);
              v[i] = w * c.get(i);
            }
            o.set(v);
          }
          at.store(o, static_cast<E*>(p.out) + to * p.ldo);
        }
      dot = lanes_sum<64>(dot);
      if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = dot;
      __syncthreads();
      if (threadIdx.x == 0) p.dweights[t * p.top_k + j] = kept ? part[0] + part[1] + part[2] + part[3] : 0.f;
      __syncthreads();
    }
  }
}

// lanes of a row of `chunks` chunks
int row_lanes(int64_t chunks) {
  int l = 1;
  while (l < kRowThreads && l < chunks) l *= 2;
  return l;
}

struct RowGrid {
  int lanes;
  dim3 grid;
};
RowGrid row_grid(const TokenParams& p, int n) {
  const int64_t chunks = (p.cols + n - 1) / n;
  RowGrid g;
  g.lanes = row_lanes(chunks);
  const int64_t per = kRowThreads / g.lanes, blocks = (p.tokens + per - 1) / per;
  g.grid = dim3((uint32_t)(blocks < kRowGrid ? blocks : kRowGrid), (uint32_t)((chunks + g.lanes - 1) / g.lanes));
  return g;
}

template <class E>
hipError_t combine_any(const TokenParams& p, hipStream_t st) {
  const RowGrid g = row_grid(p, Chunk<E>::N);
  if (p.weights) combine_kernel<E, true><<<g.grid, kRowThreads, 0, st>>>(p, g.lanes);
  else combine_kernel<E, false><<<g.grid, kRowThreads, 0, st>>>(p, g.lanes);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_moe_sort(const SortParams& p, bool i64, hipStream_t st) {
  return i64 ? sort_any<int64_t>(p, st) : sort_any<int32_t>(p, st);
}

hipError_t launch_moe_dispatch(const TokenParams& p, bool f32, hipStream_t st) {
  const RowGrid g = row_grid(p, f32 ? 4 : 8);
  if (f32) dispatch_kernel<float><<<g.grid, kRowThreads, 0, st>>>(p, g.lanes);
  else dispatch_kernel<bf16_t><<<g.grid, kRowThreads, 0, st>>>(p, g.lanes);
  return hipGetLastError();
}

hipError_t launch_moe_combine(const TokenParams& p, bool f32, hipStream_t st) {
  return f32 ? combine_any<float>(p, st) : combine_any<bf16_t>(p, st);
}

hipError_t launch_moe_combine_bwd(const TokenParams& p, bool f32, hipStream_t st) {
  const uint32_t grid = (uint32_t)(p.tokens < kRowGrid ? p.tokens : kRowGrid);
  if (f32) combine_bwd_kernel<float><<<grid, kRowThreads, 0, st>>>(p);
  else combine_bwd_kernel<bf16_t><<<grid, kRowThreads, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace mxgg
