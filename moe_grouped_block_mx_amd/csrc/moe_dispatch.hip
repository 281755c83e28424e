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
//
// What bounds it: launches and latencies, not the 12 or 16 bytes a choice. 64 choices take
// 3.2 us, 4096 5.8 - 7.9 (one workgroup, whose LDS counters and ballots are its
// time), 65536 7 - 10 and 262144 9 - 13 (two launches, the second waits for the
// first), 4194304 58 (1.2 TB/s).

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

// Counts PER keys a lane into cnt (those with `have`), 64 neighbouring choices
// at a time; place: a lane's among its wave's choices of the same key. One step for
// all PER before the next, so that their latencies overlap.
template <int PER>
__device__ __forceinline__ void count_keys(int32_t* cnt, const int (&key)[PER], const bool (&have)[PER], int bits,
                                           int (&place)[PER]) {
  const int lane = threadIdx.x & 63;
  uint64_t same[PER];
  int first[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) same[i] = __ballot(have[i]);
  for (int b = 0; b < bits; ++b)
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const bool set = (key[i] >> b) & 1;
      const uint64_t with = __ballot(set);
      same[i] &= set ? with : ~with;
    }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    first[i] = have[i] ? __ffsll((unsigned long long)same[i]) - 1 : lane;
    place[i] = 0;
    if (have[i] && lane == first[i]) place[i] = atomicAdd(cnt + key[i], (int32_t)__popcll(same[i]));
  }
#pragma unroll
  for (int i = 0; i < PER; ++i)
    place[i] = __shfl(place[i], first[i], 64) + (int)__popcll(same[i] & ((1ull << lane) - 1));
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

constexpr int kSortWaves = kSortThreads / 64;
constexpr int kSortKeys = kMaxExperts + 1;
static_assert(kSortKeys <= kSortThreads && kSortKeys <= 1 << kSortBits, "a thread for each key");

// The chunk's choices: keys, and their places among those of the same key in
// the chunk; thread e < experts + 1 gets key e's count.
template <class I, int PER>
__device__ __forceinline__ int32_t sort_chunk(const SortParams& p, int first, int32_t (*cnt)[kSortKeys],
                                              int (&key)[PER], int (&place)[PER]) {
  const int keys = p.experts + 1, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int bits = 32 - __clz(p.experts);
  for (int e = lane; e < keys; e += 64) cnt[wave][e] = 0;
  const int run = first + wave * (64 * PER) + lane;
  bool have[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = run + i * 64;
    have[i] = c < p.n;
    key[i] = have[i] ? sort_key<I>(p, c) : p.experts;
  }
  count_keys<PER>(cnt[wave], key, have, bits, place);
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
  for (int i = 0; i < PER; ++i) place[i] += cnt[wave][key[i]];
  return total;
}

__device__ __forceinline__ void store_place(const SortParams& p, int c, int key, int32_t place) {
  p.rows[c] = key < p.experts ? place : ~place;
  p.choices[place] = c;
}

// One workgroup for all, PER choices a lane.
template <class I, int PER>
__global__ __launch_bounds__(kSortThreads) void sort_one_kernel(SortParams p) {
  __shared__ int32_t cnt[kSortWaves][kSortKeys];
  __shared__ int32_t base[kSortKeys], part[kSortWaves];
  int key[PER], place[PER];
  const int32_t total = sort_chunk<I, PER>(p, 0, cnt, key, place);
  const int32_t at = block_exclusive<kSortThreads>(total, part);
  if ((int)threadIdx.x <= p.experts) base[threadIdx.x] = at;
  if ((int)threadIdx.x < p.experts) p.counts[threadIdx.x] = total;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = (int)(threadIdx.x >> 6) * (64 * PER) + i * 64 + (threadIdx.x & 63);
    if (c < p.n) store_place(p, c, key[i], base[key[i]] + place[i]);
  }
}

// Several: each one's counts and the places inside it, ...
template <class I, int PER>
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortParams p) {
  __shared__ int32_t cnt[kSortWaves][kSortKeys];
  int key[PER], place[PER];
  const int first = (int)blockIdx.x * (PER * kSortThreads);
  const int32_t total = sort_chunk<I, PER>(p, first, cnt, key, place);
  const int ld = sort_table_row(p.experts);
  if ((int)threadIdx.x < ld) p.table[(int64_t)blockIdx.x * ld + threadIdx.x] = total;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = first + (int)(threadIdx.x >> 6) * (64 * PER) + i * 64 + (threadIdx.x & 63);
    if (c < p.n) p.rows[c] = place[i];
  }
}

// ... the counts before each chunk (the totals behind the last), one wave a key ...
__global__ __launch_bounds__(64) void sort_scan_kernel(SortParams p, int chunks) {
  const int ld = sort_table_row(p.experts);
  int32_t* col = p.table + blockIdx.x;
  int32_t base = 0;
  for (int b0 = 0; b0 < chunks; b0 += 64) {
    const int b = b0 + (int)threadIdx.x;
    const int32_t v = b < chunks ? col[(int64_t)b * ld] : 0;
    int32_t sum = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int32_t o = __shfl_up(sum, d, 64);
      if ((int)threadIdx.x >= d) sum += o;
    }
    if (b < chunks) col[(int64_t)b * ld] = base + sum - v;
    base += __shfl(sum, 63, 64);
  }
  if (threadIdx.x == 0) col[(int64_t)chunks * ld] = base;
}

// ... and the places of all. SCANNED: the table holds what the launch above made
// of it; else every workgroup adds its columns up, `parts` threads each four columns.
template <class I, int PER, bool SCANNED>
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(SortParams p, int chunks, int parts) {
  __shared__ int32_t base[kSortKeys], part[kSortWaves];
  __shared__ v4i sums[2][SCANNED ? 1 : kSortThreads];
  const int keys = p.experts + 1, ld = sort_table_row(p.experts), t = threadIdx.x, mine = blockIdx.x;
  const int first = mine * (PER * kSortThreads);
  int key[PER], place[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = first + i * kSortThreads + t;
    if (c < p.n) {
      key[i] = sort_key<I>(p, c);
      place[i] = p.rows[c];
    }
  }
  int32_t before = 0, total = 0;
  if constexpr (SCANNED) {
    if (t < keys) {
      before = p.table[(int64_t)mine * ld + t];
      total = p.table[(int64_t)chunks * ld + t];
    }
  } else {
    const int width = kSortThreads / parts, e = t % width * 4;
    v4i b4{}, t4{};
    if (e < ld) {
#pragma unroll 8
      for (int b = t / width; b < chunks; b += parts) {
        const v4i v = *reinterpret_cast<const v4i*>(p.table + (int64_t)b * ld + e);
        b4 += b < mine ? v : v4i{};
        t4 += v;
      }
    }
    sums[0][t] = b4;
    sums[1][t] = t4;
    __syncthreads();
    if (t < keys)
      for (int q = 0; q < parts; ++q) {
        before += reinterpret_cast<const int32_t*>(sums[0] + q * width)[t];
        total += reinterpret_cast<const int32_t*>(sums[1] + q * width)[t];
      }
  }
  const int32_t at = block_exclusive<kSortThreads>(total, part);
  if (t < keys) base[t] = at + before;
  if (mine == 0 && t < p.experts) p.counts[t] = total;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = first + i * kSortThreads + t;
    if (c < p.n) store_place(p, c, key[i], base[key[i]] + place[i]);
  }
}

template <class I, int PER>
hipError_t sort_chunked(const SortParams& p, int64_t chunks, hipStream_t st) {
  sort_count_kernel<I, PER><<<(uint32_t)chunks, kSortThreads, 0, st>>>(p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if constexpr (PER < 4)
    if (chunks <= kSortDirect) {
      int parts = 1;
      while (parts < 32 && parts * 2 * sort_table_row(p.experts) <= kSortThreads * 4) parts *= 2;
      sort_place_kernel<I, PER, false><<<(uint32_t)chunks, kSortThreads, 0, st>>>(p, (int)chunks, parts);
      return hipGetLastError();
    }
  if constexpr (PER > 1) {
    sort_scan_kernel<<<(uint32_t)p.experts + 1, 64, 0, st>>>(p, (int)chunks);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    sort_place_kernel<I, PER, true><<<(uint32_t)chunks, kSortThreads, 0, st>>>(p, (int)chunks, 1);
    e = hipGetLastError();
  }
  return e;
}

template <class I>
hipError_t sort_any(const SortParams& p, hipStream_t st) {
  static_assert(kSortShort / kSortThreads <= kSortDirect && kSortLong / (4 * kSortThreads) > kSortDirect,
                "chunks of one choice a lane take no scan, those of four always");
  const int64_t chunks = sort_chunks(p.n);
  if (chunks <= 1) {
    if (p.n <= kSortThreads) sort_one_kernel<I, 1><<<1, kSortThreads, 0, st>>>(p);
    else if (p.n <= 2 * kSortThreads) sort_one_kernel<I, 2><<<1, kSortThreads, 0, st>>>(p);
    else sort_one_kernel<I, kSortOne / kSortThreads><<<1, kSortThreads, 0, st>>>(p);
    return hipGetLastError();
  }
  switch (sort_lane(p.n)) {
    case 1: return sort_chunked<I, 1>(p, chunks, st);
    case 2: return sort_chunked<I, 2>(p, chunks, st);
    default: return sort_chunked<I, 4>(p, chunks, st);
  }
}

// ---------------------------------------------------------------------------
// Rows
//
// A token's row belongs to L lanes (a power of two, up to the workgroup); a lane
// takes 16-byte chunks L apart.
//
// Copies with places: nothing is computed that counts, so the design is about bytes in
// flight. A lane has all loads of its choices on the way before it uses the first, and
// workgroups that run at the same time have the pieces of the same rows. bf16, eight
// choices a token, 128 experts: dispatch of 4096 x 4096 49 us (6.1 TB/s, the token's
// row is read once), combine to 16384 x 7168 410 us (5.2 TB/s; with the rows in the
// tokens' order 5.3), its gradient at 4096 x 4096 110 us (5.2 TB/s). A plain copy of
// 2^30 bytes reaches 5.1, a plain read 6.4, a fill 6.9. Rows shorter than a chunk have
// kernels of their own: with a branch at every load for them combine took 450 us, and
// few tokens, whose time is much that of bringing the code, 9.8 for 5.7 (8 x 1024, the
// gradient); so have, in the gradient, rows of whole chunks (then 4.9; 64 x 7168 13.0
// and 9.1).

constexpr int kRowThreads = 256;
constexpr int64_t kRowGrid = 1 << 20;   // workgroups at most; they stay for the rest

// A thread's first token and chunk of the row: neighbouring workgroups have the
// pieces of one row, which keeps a row's reads together.
struct RowPlace {
  int64_t token, step;
  int chunk;
  __device__ __forceinline__ RowPlace(int lanes, uint32_t pieces) {
    const int per = kRowThreads / lanes;
    token = (int64_t)(blockIdx.x / pieces) * per + threadIdx.x / lanes;
    step = (int64_t)(gridDim.x / pieces) * per;
    chunk = (int)(blockIdx.x % pieces) * lanes + threadIdx.x % lanes;
  }
};

// One element, in the place of a chunk where a row is shorter than that.
template <class E>
struct Single {
  static constexpr int N = 1;
  Chunk<E> c;
  __device__ __forceinline__ void load(const E* p) { c.load_part(p, 1); }
  __device__ __forceinline__ void store(E* p) const { c.store_part(p, 1); }
  __device__ __forceinline__ float get(int) const { return c.get(0); }
  __device__ __forceinline__ void set(const float (&v)[1]) {
    float all[Chunk<E>::N] = {v[0]};
    c.set(all);
  }
};


template <class E, class C>
__global__ __launch_bounds__(kRowThreads) void dispatch_kernel(TokenParams p, int lanes, uint32_t pieces) {
  constexpr int N = C::N;
  const RowPlace pl(lanes, pieces);
  const int col = pl.chunk * N;
  if (col >= p.cols) return;
  const int at = row_chunk(col, p.cols, N).start;   // (its neighbour's elements are written twice with the same bits)
  for (int64_t t = pl.token; t < p.tokens; t += pl.step) {
    C c, zero{};
    c.load(static_cast<const E*>(p.x) + t * p.ldx + at);
    for (int j = 0; j < p.top_k; ++j) {
      const int32_t r = p.rows[t * p.top_k + j];
      const int32_t to = r < 0 ? ~r : r;
      if (to < p.expert_rows) (r < 0 ? zero : c).store(static_cast<E*>(p.out) + to * p.ldo + at);
    }
  }
}

// A token's choices j < K (at least top_k): rows and weights. A row that is not kept
// is read at place 0, and what is read there is not used: loads behind a branch
// would be waited for one after the other. A choice past top_k has no place.
template <int K>
struct Choices {
  int32_t row[K];
  float weight[K];
  uint32_t rows;
  __device__ __forceinline__ Choices(const TokenParams& p, int64_t t) : rows((uint32_t)p.expert_rows) {
#pragma unroll
    for (int j = 0; j < K; ++j) row[j] = p.rows[t * p.top_k + (j < p.top_k ? j : 0)];
#pragma unroll
    for (int j = 0; j < K; ++j) weight[j] = p.weights ? p.weights[t * p.top_k + (j < p.top_k ? j : 0)] : 1.f;
#pragma unroll
    for (int j = 0; j < K; ++j) row[j] = j < p.top_k ? row[j] : INT32_MIN;
  }
  __device__ __forceinline__ bool kept(int j) const { return (uint32_t)row[j] < rows; }
  __device__ __forceinline__ int64_t from(int j) const { return kept(j) ? row[j] : 0; }
};

template <class E, class C, int K>
__global__ __launch_bounds__(kRowThreads) void combine_kernel(TokenParams p, int lanes, uint32_t pieces) {
  constexpr int N = C::N;
  const RowPlace pl(lanes, pieces);
  const int col = pl.chunk * N;
  if (col >= p.cols) return;
  const int at = row_chunk(col, p.cols, N).start;   // (as in dispatch)
  for (int64_t t = pl.token; t < p.tokens; t += pl.step) {
    float sum[N] = {};
    if (p.expert_rows > 0) {
      const Choices<K> ch(p, t);
      C c[K], zero{};
#pragma unroll
      for (int j = 0; j < K; ++j) c[j].load(static_cast<const E*>(p.y) + ch.from(j) * p.ldy + at);
#pragma unroll
      for (int j = 0; j < K; ++j) {
        const C y = ch.kept(j) ? c[j] : zero;
        const float w = ch.kept(j) ? ch.weight[j] : 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) sum[i] = __builtin_fmaf(w, y.get(i), sum[i]);
      }
    }
    C o;
    o.set(sum);
    o.store(static_cast<E*>(p.out) + t * p.ldo + at);
  }
}

// The elements of a chunk that are the lane's own. In rows of whole chunks (or of
// single elements) all are; else the last chunk's first `skip` are its neighbour's, and
// where the gradient goes over y itself (`over`) they are not to be written: the
// neighbour may not have read them yet. (Elsewhere they get the same bits twice, as in
// dispatch, which is faster: 65536 x 125 bf16, eight choices, 76 us for 82.)
template <class C, bool RAGGED>
struct Own {
  __device__ __forceinline__ Own(int, bool) {}
  __device__ __forceinline__ C of(const C& c) const { return c; }
  template <class E>
  __device__ __forceinline__ void store(C c, E* p) const { c.store(p); }
};
template <class E>
struct Own<Chunk<E>, true> {
  static constexpr int N = Chunk<E>::N;
  int keep;            // elements that are not written
  uint32_t mask[4];
  __device__ __forceinline__ Own(int skip, bool over) : keep(over ? skip : 0) {
    constexpr int EACH = N / 4, BITS = 32 / EACH;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int before = min(max(skip - EACH * i, 0), EACH);
      mask[i] = before == EACH ? 0 : ~0u << (BITS * before);
    }
  }
  __device__ __forceinline__ Chunk<E> of(Chunk<E> c) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) c.w[i] &= mask[i];
    return c;
  }
  // the last N - keep, in 8, 4 and 2 bytes from the chunk's end on
  __device__ __forceinline__ void store(Chunk<E> c, E* p) const {
    if (keep == 0) return c.store(p);
    const int n = N - keep;
    if constexpr (N == 8) {
      const uint32_t two = n & 4 ? c.w[1] : c.w[3], one = n & 2 ? (n & 4 ? c.w[0] : c.w[2]) : two;
      if (n & 4) memcpy(p + 4, c.w + 2, 8);
      if (n & 2) memcpy(p + (n & 4 ? 2 : 6), &two, 4);
      if (n & 1) reinterpret_cast<uint16_t*>(p)[keep] = (uint16_t)(one >> 16);
    } else {
      const uint32_t one = n & 2 ? c.w[1] : c.w[3];
      if (n & 2) memcpy(p + 2, c.w + 2, 8);
      if (n & 1) memcpy(p + keep, &one, 4);
    }
  }
};

// A token belongs to L lanes that go over the whole row: the weights' gradients
// are sums over it.
template <class E, class C, int K, int L, bool RAGGED>
__global__ __launch_bounds__(kRowThreads) void combine_bwd_kernel(TokenParams p) {
  constexpr int N = C::N, PER = kRowThreads / L;
  __shared__ float part[kRowThreads / 64][K];
  const int lane = threadIdx.x % L;
  for (int64_t t0 = (int64_t)blockIdx.x * PER; t0 < p.tokens; t0 += (int64_t)gridDim.x * PER) {
    const bool here = t0 + threadIdx.x / L < p.tokens;
    const int64_t t = here ? t0 + threadIdx.x / L : p.tokens - 1;
    float dot[K] = {};
    if (here && p.expert_rows > 0) {
      const Choices<K> ch(p, t);
      const E* d = static_cast<const E*>(p.x) + t * p.ldx;
      for (int col = lane * N; col < p.cols; col += L * N) {
        const RowChunk chunk = row_chunk(col, p.cols, N);
        const int at = chunk.start;
        const Own<C, RAGGED> own(chunk.skip, p.out == p.y);
        C c, y[K], zero{};
        c.load(d + at);
#pragma unroll
        for (int j = 0; j < K; ++j) y[j].load(static_cast<const E*>(p.y) + ch.from(j) * p.ldy + at);
        const C mine = own.of(c);
#pragma unroll
        for (int j = 0; j < K; ++j) {
          const C yj = own.of(y[j]);
          float v[N];
#pragma unroll
          for (int i = 0; i < N; ++i) {
            dot[j] = __builtin_fmaf(mine.get(i), yj.get(i), dot[j]);
            v[i] = ch.weight[j] * c.get(i);
          }
          C o;
          o.set(v);
          const int32_t to = ch.row[j] < 0 ? ~ch.row[j] : ch.row[j];
          if (to < p.expert_rows) own.store(ch.kept(j) ? o : zero, static_cast<E*>(p.out) + to * p.ldo + at);
        }
      }
#pragma unroll
      for (int j = 0; j < K; ++j) dot[j] = ch.kept(j) ? dot[j] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < K; ++j) dot[j] = lanes_sum<(L < 64 ? L : 64)>(dot[j]);
    if constexpr (L > 64) {                              // (the workgroup has one token)
      if (threadIdx.x % 64 == 0)
#pragma unroll
        for (int j = 0; j < K; ++j) part[threadIdx.x / 64][j] = dot[j];
      __syncthreads();
      if (lane < p.top_k) {
        float sum = part[0][lane];
        for (int w = 1; w < L / 64; ++w) sum += part[w][lane];
        p.dweights[t * p.top_k + lane] = sum;
      }
      __syncthreads();
    } else {
      float mine = dot[0];
#pragma unroll
      for (int j = 1; j < K; ++j) mine = lane == j ? dot[j] : mine;
      if (here && lane < p.top_k) p.dweights[t * p.top_k + lane] = mine;
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
  uint32_t pieces, grid;
};
RowGrid row_grid(const TokenParams& p, int n) {
  const int64_t chunks = (p.cols + n - 1) / n;
  RowGrid g;
  g.lanes = row_lanes(chunks);
  g.pieces = (uint32_t)((chunks + g.lanes - 1) / g.lanes);
  const int64_t per = kRowThreads / g.lanes, blocks = (p.tokens + per - 1) / per, most = kRowGrid / g.pieces;
  g.grid = g.pieces * (uint32_t)(blocks < most ? blocks : most);
  return g;
}

template <class E, class C>
hipError_t dispatch(const TokenParams& p, hipStream_t st) {
  const RowGrid g = row_grid(p, C::N);
  dispatch_kernel<E, C><<<g.grid, kRowThreads, 0, st>>>(p, g.lanes, g.pieces);
  return hipGetLastError();
}
template <class E, class C, int K>
hipError_t combine(const TokenParams& p, hipStream_t st) {
  const RowGrid g = row_grid(p, C::N);
  combine_kernel<E, C, K><<<g.grid, kRowThreads, 0, st>>>(p, g.lanes, g.pieces);
  return hipGetLastError();
}
template <class E, class C, int K, int L>
hipError_t combine_bwd(const TokenParams& p, hipStream_t st) {
  constexpr int PER = kRowThreads / L;
  const int64_t blocks = (p.tokens + PER - 1) / PER;
  const uint32_t grid = (uint32_t)(blocks < kRowGrid ? blocks : kRowGrid);
  if constexpr (C::N > 1)
    if (p.cols % C::N) {
      combine_bwd_kernel<E, C, K, L, true><<<grid, kRowThreads, 0, st>>>(p);
      return hipGetLastError();
    }
  combine_bwd_kernel<E, C, K, L, false><<<grid, kRowThreads, 0, st>>>(p);
  return hipGetLastError();
}
template <class E, class C>
hipError_t combine_any(const TokenParams& p, hipStream_t st) {
  if (p.top_k <= 1) return combine<E, C, 1>(p, st);
  if (p.top_k <= 2) return combine<E, C, 2>(p, st);
  if (p.top_k <= 4) return combine<E, C, 4>(p, st);
  if (p.top_k <= 8) return combine<E, C, 8>(p, st);
  return combine<E, C, 16>(p, st);
}
constexpr int64_t kFewTokens = 256;
template <class E, int K>
hipError_t combine_bwd_wide(const TokenParams& p, hipStream_t st) {
  // Lanes that fit the row: fewer would leave few loads in flight, more would be idle;
  // but with few tokens, which leave CUs idle, a row's chunks all at once. Eight
  // choices, us with 16, 32, 64 and 256 lanes, the rule's marked: bf16 65536 x 128 60*, 85,
  // 138, 407; 65536 x 256 115, 118*, 163, 443; 32768 x 512 118, 115, 117*, 245; 16384 x 1024
  // 119, 118, 114*, 149; 16384 x 2048 291, 257, 234, 224*; 8192 x 7168 413, 407, 404, 396*;
  // fp32 65536 x 128 116, 120*, 166, 418; 16384 x 1024 293, 258, 237, 224*; 256 tokens
  // x 1024, bf16, 13, 8.8, 7.0, 5.5*, and 512 of them 13.9, 9.3, 7.1*, 7.0, 1024 15, 11, 8.4*, 11.
  if (p.cols < Chunk<E>::N) return combine_bwd<E, Single<E>, K, 16>(p, st);
  const int chunks = (p.cols + Chunk<E>::N - 1) / Chunk<E>::N;
  if (chunks <= 16) return combine_bwd<E, Chunk<E>, K, 16>(p, st);
  if (chunks <= 32) return combine_bwd<E, Chunk<E>, K, 32>(p, st);
  if (chunks > 64 && p.tokens <= kFewTokens) return combine_bwd<E, Chunk<E>, K, 256>(p, st);
  return chunks <= 128 ? combine_bwd<E, Chunk<E>, K, 64>(p, st) : combine_bwd<E, Chunk<E>, K, 256>(p, st);
}
template <class E>
hipError_t combine_bwd_any(const TokenParams& p, hipStream_t st) {
  if (p.top_k <= 1) return combine_bwd_wide<E, 1>(p, st);
  if (p.top_k <= 2) return combine_bwd_wide<E, 2>(p, st);
  if (p.top_k <= 4) return combine_bwd_wide<E, 4>(p, st);
  if (p.top_k <= 8) return combine_bwd_wide<E, 8>(p, st);
  return combine_bwd_wide<E, 16>(p, st);
}

}  // namespace

hipError_t launch_moe_sort(const SortParams& p, bool i64, hipStream_t st) {
  return i64 ? sort_any<int64_t>(p, st) : sort_any<int32_t>(p, st);
}

hipError_t launch_moe_dispatch(const TokenParams& p, bool f32, hipStream_t st) {
  if (f32) return p.cols < 4 ? dispatch<float, Single<float>>(p, st) : dispatch<float, Chunk<float>>(p, st);
  return p.cols < 8 ? dispatch<bf16_t, Single<bf16_t>>(p, st) : dispatch<bf16_t, Chunk<bf16_t>>(p, st);
}

hipError_t launch_moe_combine(const TokenParams& p, bool f32, hipStream_t st) {
  if (f32) return p.cols < 4 ? combine_any<float, Single<float>>(p, st) : combine_any<float, Chunk<float>>(p, st);
  return p.cols < 8 ? combine_any<bf16_t, Single<bf16_t>>(p, st) : combine_any<bf16_t, Chunk<bf16_t>>(p, st);
}

hipError_t launch_moe_combine_bwd(const TokenParams& p, bool f32, hipStream_t st) {
  return f32 ? combine_bwd_any<float>(p, st) : combine_bwd_any<bf16_t>(p, st);
}

}  // namespace mxgg
