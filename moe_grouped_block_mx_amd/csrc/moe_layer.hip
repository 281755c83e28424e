// A whole expert layer for a few tokens, on quantized weights.
//
//   p, e = top-k of the gate's logits (softmax over the chosen, or over all)
//   h[t, j] = silu(W1_e x[t]) * (W3_e x[t])      e = e[t, j]
//   y[t] = sum_j p[t, j] W2_e h[t, j]
//
// With at most 64 tokens every weight is used for a few columns only, so the
// layer costs what its chosen experts' weights cost to read. Activations stay
// bf16 (no quantization pass, no second rounding): the codes are converted to
// bf16, which holds every E2M1 and E4M3 value times a power of two exactly,
// and multiplied on the bf16 MFMA with fp32 accumulation. A 16x16x32 MFMA
// takes 16 weight rows against 16 tokens.
//
// Three launches (four where the second product is split): the routing takes 4
// to 7 us, the products what their weights take to read (times of a whole layer:
// medians of replays from a graph, weights of three layers in turn). 64 tokens, 64
// experts of 7168 x 2048, blockwise FP8 (2.8 GB): 506 us, 5.6 TB/s, where reading
// alone reaches 5.7; 8 tokens, 128 experts of 7168 x 1024, MXFP4 (0.6 GB): 128 us,
// 4.7 TB/s; 32 tokens, 32 experts of 4096 x 1536, MXFP4 (0.32 GB): 78 us, 4.1 TB/s.
// One token there (80 MB) takes 27 us, of which some 13 are three launches
// and the rings' filling. Routing inside the first product's workgroups took 5 us
// there, more than its launch. Where an expert has more tokens than a segment, its
// weights are read again for each: 64 tokens there read 0.62 GB for 0.32, 120 us.
//
// How a lane reads: 64 bytes of each of 16 rows are one piece; lane l owns
// bytes 16 (l/16) .. +15 of row l%16, whatever the layout (rows of codes or
// 64-byte K blocks differ in two strides only). Those 16 bytes are 32 E2M1 or
// 16 E4M3 elements, all under one scale. The contraction's order inside an
// MFMA is free as long as both operands share it, so the lane's elements feed
// 4 (2) MFMAs eight at a time, and the token's operand is the 16 bytes of x at
// the same eight positions.
#include "block_common.hpp"
#include "block_launch.hpp"
#include "device_common.hpp"
#include "launch.hpp"

namespace mxgg {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------------------
// Routing

// Order of floats as unsigned integers, NaN above all, -0 and 0 the same; 0 is
// "never chosen", which -inf is too.
__device__ __forceinline__ uint32_t order_key(float v) {
  v += 0.f;
  const uint32_t u = __float_as_uint(v);
  if (v != v) return 0xFFFFFFFFu;
  if (u == 0xFF800000u) return 0;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// The value that an order_key stands for
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k == 0xFFFFFFFFu ? 0x7FC00000u : k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// Over rows of 16 lanes, in every lane
template <class Op>
__device__ __forceinline__ uint32_t row_reduce(uint32_t v, Op op) {
  v = op(v, rotate<8>(v));
  v = op(v, rotate<4>(v));
  v = op(v, rotate<2>(v));
  return op(v, rotate<1>(v));
}

// The top-k of four tokens by a wave, 16 lanes to a token: lane l has experts
// 16 i + l. Lane j is left with choice j's expert (-1: none) and its weight.
template <int PER>
__device__ __forceinline__ void route_token(const MoeParams& p, int t, int& id, float& weight) {
  const int lane = threadIdx.x % 16;
  float v[PER];
  uint32_t key[PER];
  const int64_t at = t * p.ldl + lane;
  if (p.logits_f32) {
    const float* row = static_cast<const float*>(p.logits) + at;
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = i * 16 + lane < p.experts ? row[i * 16] : -INFINITY;
  } else {
    const bf16_t* row = static_cast<const bf16_t*>(p.logits) + at;
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = i * 16 + lane < p.experts ? load_one(row + i * 16) : -INFINITY;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) key[i] = order_key(v[i]);
  id = -1;
  float mine = 0.f, high = 0.f;
  for (int j = 0; j < p.top_k; ++j) {
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) m = max(m, key[i]);
    m = row_reduce(m, [](uint32_t a, uint32_t b) { return max(a, b); });
    uint32_t first = 0xFFFF;             // the lowest index among equal logits
#pragma unroll
    for (int i = PER - 1; i >= 0; --i)
      if (key[i] == m) first = i * 16 + lane;
    first = row_reduce(first, [](uint32_t a, uint32_t b) { return min(a, b); });
    if (j == 0) high = key_value(m);
    if (lane == j && m != 0) {           // 0: only -inf is left
      id = (int)first;
      mine = key_value(m);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i * 16 + lane == (int)first) key[i] = 0;
  }
  const float e = id >= 0 ? expf(mine - high) : 0.f;
  float total = e;
  if (!p.renormalize) {
    total = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) total += i * 16 + lane < p.experts ? expf(v[i] - high) : 0.f;
  }
  total = lanes_sum<16>(total);
  weight = id >= 0 ? e / total : 0.f;
}

// One workgroup routes all tokens (THREADS / 16 of them at most) and lists the
// segments (a chosen expert and at most p.segment of its tokens) and the
// (expert, token) rows.
template <int PER, int THREADS>
__global__ __launch_bounds__(THREADS) void moe_route_kernel(MoeParams p) {
  __shared__ unsigned long long mask[kMaxExperts];   // an expert's tokens
  __shared__ int64_t first[kMaxExperts + 1], wave_tot[THREADS / 64];
  for (int e = threadIdx.x; e < p.experts; e += THREADS) mask[e] = 0;
  __syncthreads();
  const int lane = threadIdx.x % 16, t = threadIdx.x / 16;
  int id = -1;
  float weight = 0.f;
  if (t < p.tokens) {
    route_token<PER>(p, t, id, weight);
    if (lane < p.top_k) {
      p.ids[t * p.top_k + lane] = id;
      p.weights[t * p.top_k + lane] = weight;
      if (id >= 0) atomicOr(&mask[id], 1ull << t);
    }
  }
  __syncthreads();
  // before expert e: segments, and rows in the high half
  block_prefix64<THREADS>(
      p.experts,
      [&](int e) {
        const int n = __popcll(mask[e]);
        return (int64_t)((n + p.segment - 1) / p.segment) + ((int64_t)n << 32);
      },
      first, wave_tot);
  for (int e = threadIdx.x; e < p.experts; e += THREADS) {
    MoeSegment* at = p.segments + (int32_t)first[e];
    int base = (int32_t)(first[e] >> 32);
    for (int left = __popcll(mask[e]); left > 0; left -= p.segment, base += p.segment)
      *at++ = MoeSegment{e, base, min(left, p.segment), 0};
  }
  if (id >= 0) p.row_list[(int32_t)(first[id] >> 32) + __popcll(mask[id] & ((1ull << t) - 1))] = MoeRow{weight, t};
  if (threadIdx.x == 0) *p.count = (int32_t)first[p.experts];
}

// ---------------------------------------------------------------------------
// Products

template <MoeFormat F>
struct Piece {
  static constexpr int ELEMS = F == kMoeFp4 ? 128 : 64;  // elements of 64 bytes
  static constexpr int LANE = ELEMS / 4;                 // elements of a lane
  static constexpr int MFMAS = LANE / 8;
};

// 16 bytes of codes -> MFMA operand j (eight elements), times 2^(s - 127)
template <MoeFormat F>
__device__ __forceinline__ v8bf decode(const uint4& c, int j, float scale) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t o[4];
  if constexpr (F == kMoeFp4) {
    const uint32_t u = w[j];
    o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(u, scale, 0));
    o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(u, scale, 1));
    o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(u, scale, 2));
    o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(u, scale, 3));
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t u = w[2 * j + h];
      o[2 * h] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(u, scale, false));
      o[2 * h + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(u, scale, true));
    }
  }
  return __builtin_bit_cast(v8bf, uint4{o[0], o[1], o[2], o[3]});
}

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x / 64); }

// Where element e of a row of the inner activation lies: a piece of all rows
// after the other, so the rows of a segment, which follow each other, are one
// run of each piece.
template <MoeFormat F>
__device__ __forceinline__ int64_t inner_at(int64_t row, int e, int64_t rows) {
  return (e / Piece<F>::ELEMS * rows + row) * Piece<F>::ELEMS + e % Piece<F>::ELEMS;
}

#define MXGG_LDS __attribute__((address_space(3)))

// gfx9 s_waitcnt: vmcnt in bits 3:0 and 15:14, expcnt 6:4, lgkmcnt 11:8; a
// field at its maximum does not wait.
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 0xF) | (N >> 4) << 14 | 0x7 << 4 | 0xF << 8);
  asm volatile("" ::: "memory");
}

// RT 16-row tiles of a weight operand against a segment's tokens, one piece at
// a time. The operands come to LDS by DMA, into a ring of D pieces for each
// wave (D - 1 in flight; a wave waits for its own loads only, so no barriers).
// A load to registers has to fetch 16 bytes of 16 rows at a time, which occupies
// the address unit for 30 to 60 cycles; a DMA takes its 1 KiB as it lies (rows
// of 64 bytes, tokens of ELEMS elements), and one brings the scales of all RT
// tiles. XN DMAs hold COLS tokens. A column past the segment's tokens repeats
// some token's: what the MFMA computes for it is its own and is dropped.
template <MoeFormat F, int RT, int XN, int D, bool TAIL>
struct Ring {
  static constexpr int M = Piece<F>::MFMAS, LANE = Piece<F>::LANE, ELEMS = Piece<F>::ELEMS;
  static constexpr int CHUNKS = ELEMS / 8;             // 16-byte chunks of a token's piece
  static constexpr int COLS = XN * 64 / CHUNKS;
  static constexpr int BLOCKS = F == kMoeFp4 ? 4 : 2;  // of 32, in a piece
  static constexpr int S_AT = RT * 1024, X_AT = S_AT + 256, STAGE = X_AT + XN * 1024;
  static constexpr int BYTES = D * STAGE;              // of LDS, for a wave
  static constexpr int DMAS = RT + 1 + XN, SLOTS = D;

  const uint8_t* q[RT];
  const uint8_t* s;
  const uint16_t* x;
  int64_t q_piece, s_block, x_piece;
  uint32_t q_lane, s_lane, x_lane[XN];
  uint32_t q_first, s_first, x_first[XN];   // the same at the start of the piece
  int32_t k;
  uint8_t* lds;
  v4f acc[RT];

  // Chunk c of row r lies at place c ^ swizzle: a fragment read takes one
  // chunk of 16 rows, and this spreads it over all banks.
  static __device__ __forceinline__ int q_place(int r, int c) { return c ^ (r >> 2 & 3); }
  static __device__ __forceinline__ int x_place(int t, int c) { return c ^ (CHUNKS == 16 ? t & 15 : t >> 1 & 7); }

  __device__ __forceinline__ void init(uint8_t* ring, int64_t row_stride, int64_t piece_stride, int64_t block_stride,
                                       int32_t width) {
    const int lane = threadIdx.x % 64;
    lds = ring;
    q_piece = piece_stride;
    s_block = block_stride;
    k = width;
    q_first = (uint32_t)(lane / 4 * row_stride);
    q_lane = q_first + q_place(lane / 4, lane % 4) * 16;
  }
  // which four rows (of which tile, which block) the lane's dword of scales
  // holds; tile i's scales begin at offset `at(i)`
  template <class At>
  __device__ __forceinline__ void scales(const void* base, At at) {
    const int lane = threadIdx.x % 64;
    s = static_cast<const uint8_t*>(base);
    if constexpr (F == kMoeBlock) {
      s_lane = s_first = at(lane % RT);
    } else {
      s_first = at(lane / 4 % RT) + lane % 4 * 4;
      s_lane = s_first + (uint32_t)(lane / (4 * RT) % BLOCKS * s_block);
    }
  }
  // the lane's token in each DMA, as an element offset
  template <class Row>
  __device__ __forceinline__ void columns(const uint16_t* base, int64_t piece_stride, Row row) {
    const int lane = threadIdx.x % 64;
    x = base;
    x_piece = piece_stride;
#pragma unroll
    for (int i = 0; i < XN; ++i) {
      const int t = i * (64 / CHUNKS) + lane / CHUNKS;
      x_first[i] = row(t);
      x_lane[i] = x_first[i] + x_place(t, lane % CHUNKS) * 8;
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[i] = v4f{0.f, 0.f, 0.f, 0.f};
  }

  static __device__ __forceinline__ void dma16(const void* from, uint8_t* to) {
    __builtin_amdgcn_global_load_lds(from, (MXGG_LDS void*)to, 16, 0, 0);
  }
  __device__ __forceinline__ void issue(int slot, int piece) const {
    const int lane = threadIdx.x % 64;
    uint8_t* to = lds + slot * STAGE;
    // lanes past the row's end bring the piece's first bytes once more
    const int left = k - piece * ELEMS;
    const bool q_in = !TAIL || q_place(lane / 4, lane % 4) * LANE < left;
    const bool s_in = !TAIL || lane / (4 * RT) % BLOCKS * 32 < left;
#pragma unroll
    for (int i = 0; i < RT; ++i) dma16(q[i] + piece * q_piece + (q_in ? q_lane : q_first), to + i * 1024);
    const int64_t s_at = F == kMoeBlock ? (int64_t)(piece / 2 * 4) : piece * BLOCKS * s_block;
    __builtin_amdgcn_global_load_lds(s + s_at + (s_in ? s_lane : s_first), (MXGG_LDS void*)(to + S_AT), 4, 0, 0);
#pragma unroll
    for (int i = 0; i < XN; ++i) {
      const int t = i * (64 / CHUNKS) + lane / CHUNKS;
      const bool x_in = !TAIL || x_place(t, lane % CHUNKS) * 8 < left;
      dma16(x + piece * x_piece + (x_in ? x_lane[i] : x_first[i]), to + X_AT + i * 1024);
    }
  }

  // acc += the piece in a slot. The reads are of ext_vector types and scalars:
  // through HIP's uint4 struct the compiler takes them for reads of what the DMAs
  // in flight write, and waits for those.
  __device__ __forceinline__ void compute(int slot, int piece) {
    const int lane = threadIdx.x % 64, r = lane % 16, g = lane / 16;
    const uint8_t* from = lds + slot * STAGE;
    const bool in = !TAIL || piece * ELEMS + g * LANE < k;
    const auto keep = [&](v4i v) { return v4i{in ? v[0] : 0, in ? v[1] : 0, in ? v[2] : 0, in ? v[3] : 0}; };
    v4i xs[M], c[RT];
    float scale[RT];
    const int t = r < COLS ? r : r % COLS;   // columns past the ring's tokens repeat some
#pragma unroll
    for (int j = 0; j < M; ++j)
      xs[j] = *reinterpret_cast<const v4i*>(from + X_AT + (t * CHUNKS + x_place(t, g * M + j)) * 16);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      c[i] = *reinterpret_cast<const v4i*>(from + i * 1024 + (r * 4 + q_place(r, g)) * 16);
      if constexpr (F == kMoeBlock)
        scale[i] = *reinterpret_cast<const float*>(from + S_AT + i * 4);
      else
        scale[i] = __uint_as_float((uint32_t)from[S_AT + ((F == kMoeFp4 ? g : g / 2) * RT + i) * 16 + r] << 23);
    }
    if constexpr (TAIL) {
#pragma unroll
      for (int j = 0; j < M; ++j) xs[j] = keep(xs[j]);
#pragma unroll
      for (int i = 0; i < RT; ++i) c[i] = keep(c[i]);
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      // MX: 2^(s - 127) goes into the conversion; blocks: the fp32 scale onto
      // the product, since a code times a general scale would round in bf16
      v4f v = F == kMoeBlock ? v4f{0.f, 0.f, 0.f, 0.f} : acc[i];
#pragma unroll
      for (int j = 0; j < M; ++j)
        v = __builtin_amdgcn_mfma_f32_16x16x32_bf16(decode<F>(__builtin_bit_cast(uint4, c[i]), j, F == kMoeBlock ? 1.f : scale[i]),
                                                    __builtin_bit_cast(v8bf, xs[j]), v, 0, 0, 0);
      if constexpr (F == kMoeBlock) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = fmaf(scale[i], v[e], acc[i][e]);
      }
      acc[i] = v;
    }
  }

  static __device__ __forceinline__ int next(int slot) { return slot == D - 1 ? 0 : slot + 1; }
  static __device__ __forceinline__ int before(int slot) { return slot == 0 ? D - 1 : slot - 1; }
  // the oldest piece in flight is in LDS, D - 2 are still coming
  static __device__ __forceinline__ void wait() { wait_loads<(D - 2) * DMAS>(); }
};

// Workgroup barrier that orders LDS only: loads in flight stay in flight
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_s_waitcnt(0x3 << 14 | 0xF | 0x7 << 4);   // lgkmcnt(0)
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The lists of a call to LDS: segments as expert << 8 | tokens and base, the
// rows as `put` keeps them. Returns how many segments there are. The loads of a
// thread's first elements go out together: one latency, where a loop after the
// other pays three.
template <int THREADS, class Put>
__device__ __forceinline__ int lists_to_lds(const MoeParams& p, int32_t* segments, Put put) {
  const int t = threadIdx.x;
  const int count = *p.count;
  MoeSegment sg = p.segments[min(t, p.most_segments - 1)];
  MoeRow row = p.row_list[min(t, p.rows - 1)];
  for (int i = t; i < p.most_segments; i += THREADS) {
    if (i != t) sg = p.segments[i];
    segments[2 * i] = sg.expert << 8 | sg.tokens;
    segments[2 * i + 1] = sg.base;
  }
  for (int i = t; i < p.rows; i += THREADS) {
    if (i != t) row = p.row_list[i];
    put(i, row);
  }
  return count;
}

// h, 16 TILES inner columns of one segment at a time: W1's and W3's rows
// against the segment's tokens. The grid stays: workgroup b takes units b, b +
// grid, ..., and its waves share the pieces of each, in one stream that runs on
// over the ends of units. Neighbouring units at the same time on the same XCD
// (the hardware deals workgroups out to the 8 in turn) share the lines of the
// scales, 128 rows of one block each.
template <MoeFormat F, int XN, bool TAIL>
__global__ __launch_bounds__(64 * moe_up_cut(XN).waves) void moe_up_kernel(MoeParams p) {
  constexpr MoeCut C = moe_up_cut(XN);
  constexpr int TILES = C.tiles, WAVES = C.waves, RT = 2 * TILES, THREADS = 64 * WAVES;
  using R = Ring<F, RT, XN, C.slots, TAIL>;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  v4f* sums = reinterpret_cast<v4f*>(lds + WAVES * R::BYTES);
  int32_t* segments = reinterpret_cast<int32_t*>(sums + WAVES * RT * 64);
  uint8_t* tokens = reinterpret_cast<uint8_t*>(segments + 2 * p.most_segments);
  const int lane = threadIdx.x % 64, wave = wave_id(), col = lane % 16, g = lane / 16;
  const int tiles = p.inner / (16 * TILES);
  const int units = lists_to_lds<THREADS>(p, segments, [&](int i, const MoeRow& r) { tokens[i] = (uint8_t)r.token; }) * tiles;
  const int start = blockIdx.x % 8 * (gridDim.x / 8) + blockIdx.x / 8;   // the grid is a multiple of 8
  __syncthreads();
  if (start >= units) return;
  const int pieces = (p.hidden + R::ELEMS - 1) / R::ELEMS;
  const int mine = (pieces - wave + WAVES - 1) / WAVES;   // of a unit; 0 where there are fewer pieces than waves
  const int rounds = (units - start + (int)gridDim.x - 1) / (int)gridDim.x;
  R w;
  w.init(lds + wave * R::BYTES, p.q13_row, p.q13_piece, p.s13_block, p.hidden);
  const auto aim = [&](int unit) {
    const int seg = unit / tiles, tile = unit % tiles;
    const int head = __builtin_amdgcn_readfirstlane(segments[2 * seg]),
              base = __builtin_amdgcn_readfirstlane(segments[2 * seg + 1]);
    const int n = head & 255;
    const int64_t gate = (int64_t)(head >> 8) * 2 * p.inner + tile * (16 * TILES);
#pragma unroll
    for (int i = 0; i < RT; ++i) w.q[i] = p.w13_q + (gate + i / TILES * p.inner + i % TILES * 16) * p.q13_row;
    if constexpr (F == kMoeBlock)
      // the rows of W1 in a unit share a 128-row block, those of W3 too
      w.scales(p.w13_s, [&](int i) { return (uint32_t)((gate + i / TILES * p.inner) / 128 * (p.hidden / 128) * 4); });
    else
      w.scales(static_cast<const uint8_t*>(p.w13_s) + gate,
               [&](int i) { return (uint32_t)(i / TILES * p.inner + i % TILES * 16); });
    w.columns(p.x, R::ELEMS, [&](int t) { return (uint32_t)tokens[base + min(t, n - 1)] * (uint32_t)p.ldx; });
  };
  int load_unit = start, load_piece = wave, loads = rounds * mine;
  const auto load = [&](int slot) {
    w.issue(slot, load_piece);
    if (--loads > 0 && (load_piece += WAVES) >= pieces) {   // after the last, it again
      load_piece = wave;
      load_unit += gridDim.x;
      aim(load_unit);
    }
  };
  if (mine > 0) {
    aim(start);
#pragma unroll
    for (int d = 0; d < R::SLOTS - 1; ++d) load(d);
  }
  int slot = 0;
  for (int round = 0; round < rounds; ++round) {
    w.clear();
    for (int i = 0; i < mine; ++i) {
      R::wait();
      load(R::before(slot));   // the slot whose piece went into the products last
      w.compute(slot, wave + i * WAVES);
      __builtin_amdgcn_sched_barrier(0);
      slot = R::next(slot);
    }
    if (round) lds_barrier();  // the sums before have been read
#pragma unroll
    for (int i = 0; i < RT; ++i) sums[(wave * RT + i) * 64 + lane] = w.acc[i];
    lds_barrier();
    const int tile0 = (wave - round) & (WAVES - 1);   // another wave each round
    if (tile0 < TILES) {
      v4f a = sums[tile0 * 64 + lane], u = sums[(TILES + tile0) * 64 + lane];
#pragma unroll
      for (int k = 1; k < WAVES; ++k) {
        a += sums[(k * RT + tile0) * 64 + lane];
        u += sums[(k * RT + TILES + tile0) * 64 + lane];
      }
      const int unit = start + round * (int)gridDim.x, seg = unit / tiles, tile = unit % tiles * TILES + tile0;
      if (col < (segments[2 * seg] & 255)) {
        float h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = a[k] / (1.f + expf(-a[k])) * u[k];
        // bf16, as between the two grouped products of a training step: the
        // second product reads it as its MFMA operand. It leaves the output 2.3e-3
        // off its 64-bit value (in norm), where rounding the output alone leaves
        // 1.65e-3; the rest of h in a second bf16 would double that product's token
        // loads and halve the tokens of a segment.
        uint16_t* to = p.inner_x + inner_at<F>(segments[2 * seg + 1] + col, tile * 16 + g * 4, p.rows);
        *reinterpret_cast<uint2*>(to) = uint2{bf16_pair(h[0], h[1]), bf16_pair(h[2], h[3])};
      }
    }
  }
  wait_loads<0>();
}

// The same for the second product: y for 16 RT output columns and all tokens.
// A workgroup goes through all segments, or through one of p.splits parts of
// them, so a token's sum over its experts stays here (no atomics, one order);
// the segments' pieces are dealt out to the waves in equal runs, each one
// stream. When a segment is done, its columns go, weighted, into the wave's
// sums in LDS.
template <MoeFormat F, int RT, int XN, bool TAIL, bool MANY>
__global__ __launch_bounds__(64 * moe_down_cut(RT, XN, MANY).waves) void moe_down_kernel(MoeParams p) {
  constexpr MoeCut C = moe_down_cut(RT, XN, MANY);
  constexpr int WAVES = C.waves, THREADS = 64 * WAVES;
  using R = Ring<F, RT, XN, C.slots, TAIL>;
  constexpr int ROWS = RT * 16;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  // neighbouring tiles of 128 rows on one XCD, as above
  constexpr int NEAR = 128 / ROWS;
  const int b = blockIdx.x, tile = (b / (8 * NEAR) * 8 + b % 8) * NEAR + b % (8 * NEAR) / 8, part = blockIdx.y;
  if (tile * ROWS >= p.hidden) return;
  v4f* sums = reinterpret_cast<v4f*>(lds + WAVES * R::BYTES);   // [wave][token][ROWS / 4]
  int32_t* segments = reinterpret_cast<int32_t*>(sums + WAVES * p.tokens * (ROWS / 4));
  float* weights = reinterpret_cast<float*>(segments + 2 * p.most_segments);
  uint8_t* tokens = reinterpret_cast<uint8_t*>(weights + p.rows);
  const int lane = threadIdx.x % 64, wave = wave_id(), col = lane % 16, g = lane / 16;
  const int count = lists_to_lds<THREADS>(p, segments, [&](int i, const MoeRow& r) {
    weights[i] = r.weight;
    tokens[i] = (uint8_t)r.token;
  });
  for (int i = threadIdx.x; i < WAVES * p.tokens * (ROWS / 4); i += THREADS) sums[i] = v4f{0.f, 0.f, 0.f, 0.f};
  __syncthreads();
  const int pieces = (p.inner + R::ELEMS - 1) / R::ELEMS;
  const int total = count * pieces;
  const int runs = p.splits * WAVES, run = part * WAVES + wave;
  const int begin = (int)((int64_t)total * run / runs), items = (int)((int64_t)total * (run + 1) / runs) - begin;
  R w;
  w.init(lds + wave * R::BYTES, p.q2_row, p.q2_piece, p.s2_block, p.inner);
  // rows past the last (64 need not divide them) repeat its tile, unwritten
  const int last = p.hidden - 16 - tile * ROWS;
  int load_segment = begin / pieces, load_piece = begin % pieces, loads = items;
  int segment = load_segment, piece = load_piece;
  const auto aim = [&]() {
    const int head = __builtin_amdgcn_readfirstlane(segments[2 * load_segment]),
              base = __builtin_amdgcn_readfirstlane(segments[2 * load_segment + 1]);
    const int n = head & 255;
    const int64_t row0 = (int64_t)(head >> 8) * p.hidden + tile * ROWS;
#pragma unroll
    for (int i = 0; i < RT; ++i) w.q[i] = p.w2_q + (row0 + min(i * 16, last)) * p.q2_row;
    if constexpr (F == kMoeBlock)
      w.scales(p.w2_s, [&](int) { return (uint32_t)(row0 / 128 * (p.inner / 128) * 4); });
    else
      w.scales(static_cast<const uint8_t*>(p.w2_s) + row0, [&](int i) { return (uint32_t)min(i * 16, last); });
    w.columns(p.inner_x, (int64_t)p.rows * R::ELEMS, [&](int t) { return (uint32_t)(base + min(t, n - 1)) * R::ELEMS; });
  };
  const auto load = [&](int slot) {
    w.issue(slot, load_piece);
    if (--loads > 0 && ++load_piece == pieces) {   // after the last, it again
      load_piece = 0;
      ++load_segment;
      aim();
    }
  };
  const auto finish = [&]() {
    const int n = segments[2 * segment] & 255, row = segments[2 * segment + 1] + col;
    if (col < n) {
      const float weight = weights[row];
      v4f* to = sums + (wave * p.tokens + tokens[row]) * (ROWS / 4) + g;
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        v4f v = to[i * 4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = fmaf(weight, w.acc[i][k], v[k]);
        to[i * 4] = v;
      }
    }
    w.clear();
  };
  if (items > 0) {
    w.clear();
    aim();
#pragma unroll
    for (int d = 0; d < R::SLOTS - 1; ++d) load(d);
    for (int i = 0, slot = 0; i < items; ++i) {
      R::wait();
      load(R::before(slot));
      w.compute(slot, piece);
      __builtin_amdgcn_sched_barrier(0);
      slot = R::next(slot);
      if (++piece == pieces) {
        finish();
        piece = 0;
        ++segment;
      }
    }
    if (piece > 0) finish();    // the rest of this segment is another wave's
    wait_loads<0>();
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.tokens * (ROWS / 4); i += THREADS) {
    v4f v = sums[i];
#pragma unroll
    for (int k = 1; k < WAVES; ++k) v += sums[k * p.tokens * (ROWS / 4) + i];
    const int row = tile * ROWS + i % (ROWS / 4) * 4;
    if (row >= p.hidden) continue;
    const int64_t at = (int64_t)(i / (ROWS / 4)) * p.hidden + row;
    if (p.splits == 1)
      *reinterpret_cast<uint2*>(p.out + at) = uint2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
    else
      *reinterpret_cast<v4f*>(p.parts + (int64_t)part * p.tokens * p.hidden + at) = v;
  }
}

// y from the parts
__global__ __launch_bounds__(256) void moe_sum_kernel(MoeParams p) {
  const int64_t n = (int64_t)p.tokens * p.hidden, at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (at >= n) return;
  v4f v = *reinterpret_cast<const v4f*>(p.parts + at);
  for (int k = 1; k < p.splits; ++k) v += *reinterpret_cast<const v4f*>(p.parts + k * n + at);
  *reinterpret_cast<uint2*>(p.out + at) = uint2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
}

template <int PER>
void route_per(const MoeParams& p, hipStream_t st) {
  if (p.tokens <= 16) moe_route_kernel<PER, 256><<<1, 256, 0, st>>>(p);
  else moe_route_kernel<PER, 16 * kMoeTokens><<<1, 16 * kMoeTokens, 0, st>>>(p);
}

hipError_t route(const MoeParams& p, hipStream_t st) {
  if (p.experts <= 64) route_per<4>(p, st);
  else if (p.experts <= 128) route_per<8>(p, st);
  else if (p.experts <= 256) route_per<16>(p, st);
  else route_per<32>(p, st);
  return hipGetLastError();
}

template <MoeFormat F, int XN, bool TAIL>
hipError_t up(const MoeParams& p, int num_cus, hipStream_t st) {
  constexpr MoeCut C = moe_up_cut(XN);
  static_assert(Ring<F, 2 * C.tiles, XN, C.slots, TAIL>::STAGE == moe_stage_bytes(2 * C.tiles, XN), "a piece in LDS");
  const int bytes = moe_up_lds(p);
  if (bytes > kMoeLdsBytes) return hipErrorInvalidValue;
  const hipError_t e =
      ensure_dynamic_lds(reinterpret_cast<const void*>(&moe_up_kernel<F, XN, TAIL>), kMoeLdsBytes, st);
  if (e != hipSuccess) return e;
  const int64_t units = (int64_t)p.most_segments * (p.inner / (16 * C.tiles));
  const uint32_t grid = (uint32_t)((units < num_cus ? units : num_cus) + 7) / 8 * 8;
  moe_up_kernel<F, XN, TAIL><<<grid, 64 * C.waves, bytes, st>>>(p);
  return hipGetLastError();
}

template <MoeFormat F, int RT, int XN, bool TAIL, bool MANY>
hipError_t down(const MoeParams& p, hipStream_t st) {
  constexpr MoeCut C = moe_down_cut(RT, XN, MANY);
  static_assert(Ring<F, RT, XN, C.slots, TAIL>::STAGE == moe_stage_bytes(RT, XN), "a piece in LDS");
  const int bytes = moe_down_lds(p);
  if (bytes > kMoeLdsBytes) return hipErrorInvalidValue;
  hipError_t e =
      ensure_dynamic_lds(reinterpret_cast<const void*>(&moe_down_kernel<F, RT, XN, TAIL, MANY>), kMoeLdsBytes, st);
  if (e != hipSuccess) return e;
  const uint32_t tiles = (uint32_t)((p.hidden + 1023) / 1024 * (1024 / (16 * RT)));   // whole 8 x 128-row rounds
  moe_down_kernel<F, RT, XN, TAIL, MANY><<<dim3(tiles, (uint32_t)p.splits), 64 * C.waves, bytes, st>>>(p);
  if ((e = hipGetLastError()) != hipSuccess || p.splits == 1) return e;
  moe_sum_kernel<<<(uint32_t)(((int64_t)p.tokens * p.hidden + 1023) / 1024), 256, 0, st>>>(p);
  return hipGetLastError();
}

template <MoeFormat F, int XN, bool TAIL>
hipError_t down_tiles(const MoeParams& p, hipStream_t st) {
  if constexpr (XN < 3)
    if (p.down_tiles == 1) return down<F, 1, XN, TAIL, false>(p, st);
  return moe_down_many(p) ? down<F, 4, XN, TAIL, true>(p, st) : down<F, 4, XN, TAIL, false>(p, st);
}

template <MoeFormat F, bool TAIL>
hipError_t down_any(const MoeParams& p, hipStream_t st) {
  if (p.dmas == 1) return down_tiles<F, 1, TAIL>(p, st);
  if (F != kMoeFp4 || p.dmas == 2) return down_tiles<F, 2, TAIL>(p, st);
  return down_tiles<F, F == kMoeFp4 ? 3 : 2, TAIL>(p, st);
}

template <MoeFormat F, bool TAIL>
hipError_t up_any(const MoeParams& p, int num_cus, hipStream_t st) {
  if (p.dmas == 1) return up<F, 1, TAIL>(p, num_cus, st);
  if (F != kMoeFp4 || p.dmas == 2) return up<F, 2, TAIL>(p, num_cus, st);
  return up<F, F == kMoeFp4 ? 3 : 2, TAIL>(p, num_cus, st);
}

template <MoeFormat F>
hipError_t products(const MoeParams& p, int num_cus, hipStream_t st) {
  // a row that ends inside a piece has kernels of its own (never with 128x128
  // blocks)
  hipError_t e;
  if (F != kMoeBlock && p.hidden % Piece<F>::ELEMS) e = up_any<F, F != kMoeBlock>(p, num_cus, st);
  else e = up_any<F, false>(p, num_cus, st);
  if (e != hipSuccess) return e;
  if (F != kMoeBlock && p.inner % Piece<F>::ELEMS) return down_any<F, F != kMoeBlock>(p, st);
  return down_any<F, false>(p, st);
}

}  // namespace

hipError_t launch_moe_layer(MoeParams p, MoeFormat fmt, int num_cus, hipStream_t st) {
  moe_plan(p, fmt);
  const hipError_t e = route(p, st);
  if (e != hipSuccess) return e;
  if (fmt == kMoeFp4) return products<kMoeFp4>(p, num_cus, st);
  if (fmt == kMoeFp8) return products<kMoeFp8>(p, num_cus, st);
  return products<kMoeBlock>(p, num_cus, st);
}

}  // namespace mxgg
