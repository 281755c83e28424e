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

// Reductions over the wave by DPP (rows of 16 lanes, then across rows): a few
// cycles a step, where a shuffle through LDS takes a hundred. The result is
// lane 63's, read into a scalar.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp(uint32_t old, uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)old, (int)v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, dpp<0x111, 0xF>(v, v));   // row_shr 1, 2, 4, 8
  v = max(v, dpp<0x112, 0xF>(v, v));
  v = max(v, dpp<0x114, 0xF>(v, v));
  v = max(v, dpp<0x118, 0xF>(v, v));
  v = max(v, dpp<0x142, 0xA>(v, v));   // lane 15 of a row to the next row
  v = max(v, dpp<0x143, 0xC>(v, v));   // lane 31 to the upper half
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ float wave_sum(float f) {
  const auto add = [](uint32_t a, uint32_t b) { return __float_as_uint(__uint_as_float(a) + __uint_as_float(b)); };
  uint32_t v = __float_as_uint(f);
  v = add(v, dpp<0x111, 0xF>(0, v));
  v = add(v, dpp<0x112, 0xF>(0, v));
  v = add(v, dpp<0x114, 0xF>(0, v));
  v = add(v, dpp<0x118, 0xF>(0, v));
  v = add(v, dpp<0x142, 0xA>(0, v));
  v = add(v, dpp<0x143, 0xC>(0, v));
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)v, 63));
}

// The top-k of TPW tokens by one wave (side by side: one token's steps depend
// on each other). Lane j holds choice j's expert (-1: none) and weight. Expert
// 64 i + l sits in slot i of lane l, so the lowest index among equal logits is
// the first slot's first lane.
template <class T, bool RENORM, int PER, int TPW>
__device__ __forceinline__ void route_tokens(const T* const (&row)[TPW], int experts, int top_k, int (&id)[TPW],
                                             float (&weight)[TPW]) {
  const int lane = threadIdx.x % 64;
  float v[TPW][PER], mine[TPW], high[TPW];
  uint32_t key[TPW][PER];
#pragma unroll
  for (int u = 0; u < TPW; ++u) {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      v[u][i] = i * 64 + lane < experts ? load_one(row[u] + i * 64 + lane) : -INFINITY;
    id[u] = -1;
    mine[u] = high[u] = 0.f;
  }
#pragma unroll
  for (int u = 0; u < TPW; ++u)
#pragma unroll
    for (int i = 0; i < PER; ++i) key[u][i] = order_key(v[u][i]);
  for (int j = 0; j < top_k; ++j) {
#pragma unroll
    for (int u = 0; u < TPW; ++u) {
      uint32_t m = key[u][0];
#pragma unroll
      for (int i = 1; i < PER; ++i) m = max(m, key[u][i]);
      m = wave_max(m);
      if (j == 0) high[u] = key_value(m);
      int at = -1;
#pragma unroll
      for (int i = PER - 1; i >= 0; --i) {
        const uint64_t has = __ballot(key[u][i] == m);
        if (has) at = i * 64 + __builtin_ctzll(has);
      }
      if (m == 0) at = -1;           // only -inf is left
      if (lane == j) {
        id[u] = at;
        mine[u] = key_value(m);
      }
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (i * 64 + lane == at) key[u][i] = 0;
    }
  }
#pragma unroll
  for (int u = 0; u < TPW; ++u) {
    const float e = id[u] >= 0 ? expf(mine[u] - high[u]) : 0.f;
    float total = e;
    if constexpr (!RENORM) {
      total = 0.f;
#pragma unroll
      for (int i = 0; i < PER; ++i) total += i * 64 + lane < experts ? expf(v[u][i] - high[u]) : 0.f;
    }
    total = wave_sum(total);
    weight[u] = id[u] >= 0 ? e / total : 0.f;
  }
}

// One workgroup routes all tokens and lists the chosen experts, their segments
// of at most 16 tokens, and the (expert, token) rows.
template <class T, bool RENORM, int PER, int TPW, int THREADS>
__global__ __launch_bounds__(THREADS) void moe_route_kernel(MoeParams p) {
  constexpr int WAVES = THREADS / 64;
  __shared__ unsigned long long mask[kMaxExperts];
  __shared__ int64_t first[kMaxExperts + 1], wave_tot[WAVES];
  for (int e = threadIdx.x; e < p.experts; e += THREADS) mask[e] = 0;
  __syncthreads();
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const T* row[TPW];
  int id[TPW];
  float weight[TPW];
#pragma unroll
  for (int u = 0; u < TPW; ++u) row[u] = static_cast<const T*>(p.logits) + min(wave + u * WAVES, p.tokens - 1) * p.ldl;
  route_tokens<T, RENORM, PER, TPW>(row, p.experts, p.top_k, id, weight);
#pragma unroll
  for (int u = 0; u < TPW; ++u) {
    const int t = wave + u * WAVES;
    if (t < p.tokens && lane < p.top_k) {
      p.ids[t * p.top_k + lane] = id[u];
      p.weights[t * p.top_k + lane] = weight[u];
      if (id[u] >= 0) atomicOr(&mask[id[u]], 1ull << t);
    }
  }
  __syncthreads();
  // before expert e: chosen experts, and segments << 16; rows in the high half
  block_prefix64<THREADS>(
      p.experts,
      [&](int e) {
        const int n = __popcll(mask[e]);
        return (int64_t)((n != 0) | (n + 15) / 16 << 16) + ((int64_t)n << 32);
      },
      first, wave_tot);
  for (int e = threadIdx.x; e < p.experts; e += THREADS) {
    uint64_t m = mask[e];
    if (!m) continue;
    const int32_t lists = (int32_t)first[e];
    int32_t base = (int32_t)(first[e] >> 32);
    p.table[lists & 0xFFFF] = MoeExpert{e, base, m};
    MoeSegment* seg = p.segments + (lists >> 16);
    for (int left = __popcll(m); left > 0; left -= 16, base += 16) *seg++ = MoeSegment{e, base, min(left, 16), 0};
  }
  if (threadIdx.x == 0) {
    const int32_t lists = (int32_t)first[p.experts];
    p.counts[0] = lists & 0xFFFF;
    p.counts[1] = lists >> 16;
  }
#pragma unroll
  for (int u = 0; u < TPW; ++u) {
    const int t = wave + u * WAVES;
    if (t < p.tokens && lane < p.top_k && id[u] >= 0)
      p.row_list[(int32_t)(first[id[u]] >> 32) + __popcll(mask[id[u]] & ((1ull << t) - 1))] = MoeRow{weight[u], t};
  }
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

// RT 16-row tiles of a weight operand against CT column tiles of 16 tokens.
// One stage holds one piece of each; D stages are in flight. Addresses are a
// uniform base and a 32-bit lane offset. A column without a token reads a
// token's column all the same: what the MFMA computes for it is its own and is
// dropped. So no branch surrounds a load, and each stage waits for its own
// loads only.
template <MoeFormat F, int RT, int CT, int D>
struct Products {
  static constexpr int M = Piece<F>::MFMAS, LANE = Piece<F>::LANE, ELEMS = Piece<F>::ELEMS;
  const uint8_t* q[RT];            // the tiles' codes and scales
  const uint8_t* s[RT];
  const uint16_t* x;               // the columns
  int64_t q_row, q_piece, s_block;
  int64_t x_piece;                 // elements between the pieces of a column
  uint32_t x_col[CT];              // this lane's column in each column tile
  uint32_t x_group, x_mfma;        // elements between lane groups, between MFMAs
  uint32_t q_lane, s_lane, x_lane[CT];
  v4f acc[RT][CT];

  struct Stage {
    uint4 c[RT];
    uint32_t s[RT];
    uint4 x[CT][M];
  };

  __device__ __forceinline__ void tile(int i, const uint8_t* codes, const void* scales, int64_t row0, int32_t k) {
    q[i] = codes + row0 * q_row;
    s[i] = static_cast<const uint8_t*>(scales) + (F == kMoeBlock ? row0 / 128 * (k / 128) * 4 : row0);
  }
  // the lane's place in a piece: row lane % 16, group g
  __device__ __forceinline__ void lanes(int g) {
    const int r = threadIdx.x % 16;
    q_lane = (uint32_t)(r * q_row + g * 16);
    s_lane = F == kMoeBlock ? 0 : (uint32_t)((F == kMoeFp4 ? g : g / 2) * s_block + r);
#pragma unroll
    for (int c = 0; c < CT; ++c) x_lane[c] = x_col[c] + g * x_group;
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int c = 0; c < CT; ++c) acc[i][c] = v4f{0.f, 0.f, 0.f, 0.f};
  }

  __device__ __forceinline__ void load(Stage& st, int piece) const {
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      st.c[i] = *reinterpret_cast<const uint4*>(q[i] + piece * q_piece + q_lane);
      if constexpr (F == kMoeBlock)
        st.s[i] = reinterpret_cast<const uint32_t*>(s[i])[piece / 2];
      else
        st.s[i] = (s[i] + piece * ((F == kMoeFp4 ? 4 : 2) * s_block))[s_lane];
    }
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int j = 0; j < M; ++j)
        st.x[c][j] = *reinterpret_cast<const uint4*>(x + piece * x_piece + j * x_mfma + x_lane[c]);
  }

  __device__ __forceinline__ void compute(const Stage& st) {
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      // MX: 2^(s - 127) goes into the conversion; blocks: the fp32 scale onto
      // the product, since a code times a general scale would round in bf16
      const float scale = F == kMoeBlock ? 1.f : __uint_as_float(st.s[i] << 23);
      v8bf a[M];
#pragma unroll
      for (int j = 0; j < M; ++j) a[j] = decode<F>(st.c[i], j, scale);
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        v4f t = F == kMoeBlock ? v4f{0.f, 0.f, 0.f, 0.f} : acc[i][c];
#pragma unroll
        for (int j = 0; j < M; ++j)
          t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[j], __builtin_bit_cast(v8bf, st.x[c][j]), t, 0, 0, 0);
        if constexpr (F == kMoeBlock) {
#pragma unroll
          for (int k = 0; k < 4; ++k) t[k] = fmaf(__uint_as_float(st.s[i]), t[k], acc[i][c][k]);
        }
        acc[i][c] = t;
      }
    }
  }

  // pieces first, first + step, ... (count of them, all whole)
  __device__ __forceinline__ void run(int first, int count, int step) {
    if (count <= 0) return;
    Stage st[D];
#pragma unroll
    for (int d = 0; d < D; ++d) load(st[d], first + min(d, count - 1) * step);
    int i = 0;
    for (; i + D <= count; i += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        compute(st[d]);
        // past the end the last piece again, out of the cache: cheaper than a
        // branch, after which the compiler would wait for everything. The
        // fence keeps the scheduler from moving loads to their use.
        load(st[d], first + min(i + d + D, count - 1) * step);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int d = 0; d < D - 1; ++d)
      if (i + d < count) compute(st[d]);
  }

  // zeros on both sides in lane groups that are past the row's end
  __device__ __forceinline__ void mask(Stage& st, bool in) const {
    const auto keep = [&](uint4& v) { v = uint4{in ? v.x : 0, in ? v.y : 0, in ? v.z : 0, in ? v.w : 0}; };
#pragma unroll
    for (int i = 0; i < RT; ++i) keep(st.c[i]);
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int j = 0; j < M; ++j) keep(st.x[c][j]);
  }

  // the piece that the row ends in: lane groups past the end read the first
  // group's place
  __device__ __forceinline__ void run_tail(int piece, int32_t k) {
    const int g = threadIdx.x % 64 / 16;
    const bool in = piece * ELEMS + g * LANE < k;
    lanes(in ? g : 0);
    Stage st;
    load(st, piece);
    mask(st, in);
    compute(st);
    lanes(g);
  }
};

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x / 64); }

// The n-th set bit of a word that has that many
__device__ __forceinline__ int nth_bit(uint64_t m, int n) {
  int at = 0;
  for (int i = 0; m; ++i, m &= m - 1)
    if (i == n) at = __builtin_ctzll(m);
  return at;
}

// Where element e of a row of the inner activation lies, for the second
// product: a piece's MFMAs one after the other, and in each of them all rows'
// 32 elements, so the 16 bytes of a column's four lanes are one run and the
// columns of an expert, whose rows follow each other, are too.
template <MoeFormat F>
__device__ __forceinline__ int64_t inner_at(int64_t row, int e, int64_t rows) {
  constexpr int LANE = Piece<F>::LANE, ELEMS = Piece<F>::ELEMS;
  const int piece = e / ELEMS, w = e % ELEMS, g = w / LANE, j = w % LANE / 8;
  return ((int64_t)(piece * Piece<F>::MFMAS + j) * rows + row) * 32 + g * 8 + e % 8;
}

constexpr int kUpWaves = 4;    // waves of a workgroup, sharing the contraction
constexpr int kUpTiles = 2;    // 16-row tiles of W1, and as many of W3
constexpr int kUpStages = 2;   // pieces in flight
constexpr int kDownStages = 3;
constexpr int kDownWaves = 8;
inline bool kDownTiles2(const MoeParams& p) { return p.hidden >= 6144; }

template <MoeFormat F, int CT>
__device__ __forceinline__ void up_columns(const MoeParams& p, const MoeExpert& ex, int n, int c0, int tile, v4f* lds) {
  constexpr int RT = 2 * kUpTiles;
  const int lane = threadIdx.x % 64, wave = wave_id(), col = lane % 16, g = lane / 16;
  Products<F, RT, CT, kUpStages> w;
  w.q_row = p.q13_row;
  w.q_piece = p.q13_piece;
  w.s_block = p.s13_block;
#pragma unroll
  for (int i = 0; i < RT; ++i)
    w.tile(i, p.w13_q, p.w13_s,
           ((int64_t)ex.expert * 2 + i / kUpTiles) * p.inner + (tile * kUpTiles + i % kUpTiles) * 16, p.hidden);
  w.x = p.x;
  w.x_piece = Piece<F>::ELEMS;
  w.x_group = Piece<F>::LANE;
  w.x_mfma = 8;
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    const int r = c0 + c * 16 + col;
    w.x_col[c] = (uint32_t)nth_bit(ex.tokens, r < n ? r : 0) * (uint32_t)p.ldx;
  }
  w.lanes(g);
  w.clear();
  const int whole = p.hidden / Piece<F>::ELEMS;
  w.run(wave, (whole - wave + kUpWaves - 1) / kUpWaves, kUpWaves);
  if (p.hidden % Piece<F>::ELEMS && whole % kUpWaves == wave) w.run_tail(whole, p.hidden);
  if (c0) __syncthreads();   // the sums of the columns before have been read
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int c = 0; c < CT; ++c) lds[(wave * RT * CT + i * CT + c) * 64 + lane] = w.acc[i][c];
  __syncthreads();
  for (int o = wave; o < kUpTiles * CT; o += kUpWaves) {
    const int i = o / CT, c = o % CT;
    v4f gate = lds[(i * CT + c) * 64 + lane], up = lds[((kUpTiles + i) * CT + c) * 64 + lane];
#pragma unroll
    for (int k = 1; k < kUpWaves; ++k) {
      gate += lds[((k * RT + i) * CT + c) * 64 + lane];
      up += lds[((k * RT + kUpTiles + i) * CT + c) * 64 + lane];
    }
    const int r = c0 + c * 16 + col;
    if (r < n) {
      float h[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) h[k] = gate[k] / (1.f + expf(-gate[k])) * up[k];
      // bf16, as between the two grouped products of a training step: the
      // second product reads it as its MFMA operand
      uint16_t* to = p.inner_x + inner_at<F>(ex.base + r, (tile * kUpTiles + i) * 16 + g * 4, p.rows);
      *reinterpret_cast<uint2*>(to) = uint2{bf16_pair(h[0], h[1]), bf16_pair(h[2], h[3])};
    }
  }
}

// h of one chosen expert, 32 of its inner columns: W1's and W3's rows against
// the expert's tokens.
template <MoeFormat F, int CT>
__global__ __launch_bounds__(64 * kUpWaves) void moe_up_kernel(MoeParams p) {
  __shared__ v4f lds[kUpWaves * 2 * kUpTiles * CT * 64];
  const int tiles = p.inner / (16 * kUpTiles);
  // four neighbouring tiles (128 rows: one line of every scale block) go to
  // workgroups of the same XCD, which the hardware deals out in turn
  const int b = blockIdx.x, group = b / 32 * 8 + b % 8, item = group * 4 + b % 32 / 8;
  const int slot = item / tiles, tile = item % tiles;
  if (slot >= p.experts) return;      // the grid is rounded up
  const int active = p.counts[0];
  const MoeExpert ex = p.table[slot];
  if (slot >= active) return;
  const int n = __popcll(ex.tokens);
  if (CT == 1 || n <= 16) {
    up_columns<F, 1>(p, ex, n, 0, tile, lds);
  } else if constexpr (CT > 1) {
    for (int c0 = 0; c0 < n; c0 += 16 * CT) up_columns<F, CT>(p, ex, n, c0, tile, lds);
  }
}

// y for 16 RT output columns and all tokens: the workgroup goes through every
// segment, so a token's sum over its experts stays here (no atomics, one
// order). The segments' pieces are dealt out to the waves in equal runs, and a
// wave goes through its run in one stream: while it multiplies one segment's
// last pieces, the next one's first are on their way. When a segment is done,
// its 16 columns go, weighted, into the wave's sums in LDS.
template <MoeFormat F, int RT, int WAVES, bool TAIL>
__global__ __launch_bounds__(64 * WAVES) void moe_down_kernel(MoeParams p) {
  constexpr int ROWS = RT * 16, D = kDownStages, ELEMS = Piece<F>::ELEMS;
  using P = Products<F, RT, 1, D>;
  extern __shared__ v4f lds[];
  // neighbouring tiles of 128 rows on one XCD, as above
  constexpr int NEAR = 128 / ROWS;
  const int b = blockIdx.x, tile = (b / (8 * NEAR) * 8 + b % 8) * NEAR + b % (8 * NEAR) / 8;
  if (tile * ROWS >= p.hidden) return;
  float* sums = reinterpret_cast<float*>(lds);
  int4* segments = reinterpret_cast<int4*>(sums + WAVES * p.tokens * ROWS);
  MoeRow* rows = reinterpret_cast<MoeRow*>(segments + p.most_segments);
  const int count = p.counts[1];
  for (int i = threadIdx.x; i < p.most_segments; i += 64 * WAVES)
    segments[i] = reinterpret_cast<const int4*>(p.segments)[i];
  for (int i = threadIdx.x; i < p.rows; i += 64 * WAVES) rows[i] = p.row_list[i];
  const int wave = wave_id(), lane = threadIdx.x % 64, col = lane % 16, g = lane / 16;
  sums += wave * p.tokens * ROWS;
  for (int i = lane; i < p.tokens * ROWS; i += 64) sums[i] = 0.f;
  __syncthreads();

  const int pieces = (p.inner + ELEMS - 1) / ELEMS;
  const int total = count * pieces;
  const int begin = total * wave / WAVES, items = total * (wave + 1) / WAVES - begin;
  P w;
  w.q_row = p.q2_row;
  w.q_piece = p.q2_piece;
  w.s_block = p.s2_block;
  w.x = p.inner_x;
  w.x_piece = (int64_t)p.rows * 32 * P::M;
  w.x_group = 8;
  w.x_mfma = p.rows * 32;
  // where the loads are, and where the products are
  int load_segment = begin / pieces, load_piece = begin % pieces;
  int segment = load_segment, piece = load_piece;
  const auto aim = [&]() {
    const int4 sg = segments[load_segment];
    const int expert = __builtin_amdgcn_readfirstlane(sg.x), base = __builtin_amdgcn_readfirstlane(sg.y),
              n = __builtin_amdgcn_readfirstlane(sg.z);
#pragma unroll
    for (int i = 0; i < RT; ++i) w.tile(i, p.w2_q, p.w2_s, (int64_t)expert * p.hidden + tile * ROWS + i * 16, p.inner);
    w.x_col[0] = (uint32_t)(base + min(col, n - 1)) * 32;
    w.lanes(g);
  };
  int loads = items;
  const auto load = [&](typename P::Stage& st) {
    if constexpr (TAIL) {
      // lane groups past the row's end read the first group's place
      w.lanes(load_piece * ELEMS + g * P::LANE < p.inner ? g : 0);
    }
    w.load(st, load_piece);
    if (--loads > 0 && ++load_piece == pieces) {   // after the last, it again
      load_piece = 0;
      ++load_segment;
      aim();
    }
  };
  const auto finish = [&]() {
    const int4 sg = segments[segment];
    if (col < sg.z) {
      const MoeRow r = rows[sg.y + col];
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        v4f* to = reinterpret_cast<v4f*>(sums + r.token * ROWS + i * 16 + g * 4);
        v4f v = *to;
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = fmaf(r.weight, w.acc[i][0][k], v[k]);
        *to = v;
      }
    }
    w.clear();
  };
  const auto compute = [&](typename P::Stage& st) {
    if constexpr (TAIL) w.mask(st, piece * ELEMS + g * P::LANE < p.inner);
    w.compute(st);
    if (++piece == pieces) {
      finish();
      piece = 0;
      ++segment;
    }
  };
  if (items > 0) {
    w.clear();
    aim();
    typename P::Stage st[D];
#pragma unroll
    for (int d = 0; d < D; ++d) load(st[d]);
    int i = 0;
    for (; i + D <= items; i += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        compute(st[d]);
        load(st[d]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int d = 0; d < D - 1; ++d)
      if (i + d < items) compute(st[d]);
    if (piece > 0) finish();    // the rest of this segment is another wave's
  }
  __syncthreads();
  sums = reinterpret_cast<float*>(lds);
  for (int i = threadIdx.x; i < p.tokens * ROWS / 4; i += 64 * WAVES) {
    v4f v = *reinterpret_cast<v4f*>(sums + i * 4);
#pragma unroll
    for (int k = 1; k < WAVES; ++k) v += *reinterpret_cast<v4f*>(sums + k * p.tokens * ROWS + i * 4);
    *reinterpret_cast<uint2*>(p.out + (int64_t)(i * 4 / ROWS) * p.hidden + tile * ROWS + i * 4 % ROWS) =
        uint2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
  }
}

template <class T, bool RENORM, int PER>
void route_per(const MoeParams& p, hipStream_t st) {
  if (p.tokens <= 4) moe_route_kernel<T, RENORM, PER, 1, 256><<<1, 256, 0, st>>>(p);
  else if (p.tokens <= 16) moe_route_kernel<T, RENORM, PER, 1, 1024><<<1, 1024, 0, st>>>(p);
  else moe_route_kernel<T, RENORM, PER, 4, 1024><<<1, 1024, 0, st>>>(p);
}

template <class T, bool RENORM>
hipError_t route(const MoeParams& p, hipStream_t st) {
  if (p.experts <= 64) route_per<T, RENORM, 1>(p, st);
  else if (p.experts <= 128) route_per<T, RENORM, 2>(p, st);
  else if (p.experts <= 256) route_per<T, RENORM, 4>(p, st);
  else route_per<T, RENORM, 8>(p, st);
  return hipGetLastError();
}

template <class T>
hipError_t route_any(const MoeParams& p, bool renormalize, hipStream_t st) {
  return renormalize ? route<T, true>(p, st) : route<T, false>(p, st);
}

template <MoeFormat F, int RT, int WAVES, bool TAIL>
hipError_t down(const MoeParams& p, hipStream_t st) {
  const uint32_t grid = (uint32_t)((p.hidden + 1023) / 1024 * (1024 / (16 * RT)));   // whole 8 x 128-row rounds
  const int bytes = WAVES * p.tokens * RT * 16 * 4 + p.most_segments * 16 + p.rows * (int)sizeof(MoeRow);
  const void* kernel = reinterpret_cast<const void*>(&moe_down_kernel<F, RT, WAVES, TAIL>);
  if (bytes > 65536) {
    const hipError_t e = ensure_dynamic_lds(kernel, 160 * 1024, st);
    if (e != hipSuccess) return e;
  }
  moe_down_kernel<F, RT, WAVES, TAIL><<<grid, 64 * WAVES, bytes, st>>>(p);
  return hipGetLastError();
}

template <MoeFormat F, int RT, int WAVES>
hipError_t down_any(const MoeParams& p, hipStream_t st) {
  if constexpr (F != kMoeBlock)
    if (p.inner % Piece<F>::ELEMS) return down<F, RT, WAVES, true>(p, st);
  return down<F, RT, WAVES, false>(p, st);
}

template <MoeFormat F>
hipError_t products(const MoeParams& p, hipStream_t st) {
  const int most = p.tokens * p.top_k < p.experts ? p.tokens * p.top_k : p.experts;
  const int64_t items = (int64_t)most * (p.inner / (16 * kUpTiles));
  const uint32_t grid = (uint32_t)((items + 31) / 32 * 32);
  if (p.tokens <= 16) moe_up_kernel<F, 1><<<grid, 64 * kUpWaves, 0, st>>>(p);
  else moe_up_kernel<F, 2><<<grid, 64 * kUpWaves, 0, st>>>(p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (kDownTiles2(p)) return down_any<F, 2, 8>(p, st);
  return down_any<F, 1, kDownWaves>(p, st);
}

}  // namespace

hipError_t launch_moe_layer(const MoeParams& p, MoeFormat fmt, bool logits_f32, bool renormalize, hipStream_t st) {
  const hipError_t e = logits_f32 ? route_any<float>(p, renormalize, st) : route_any<bf16_t>(p, renormalize, st);
  if (e != hipSuccess) return e;
  if (fmt == kMoeFp4) return products<kMoeFp4>(p, st);
  if (fmt == kMoeFp8) return products<kMoeFp8>(p, st);
  return products<kMoeBlock>(p, st);
}

}  // namespace mxgg
