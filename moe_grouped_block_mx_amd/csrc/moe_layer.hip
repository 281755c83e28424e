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

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = __shfl_xor(v, d, 64);
    v = o > v ? o : v;
  }
  return v;
}

template <class T>
__device__ __forceinline__ float logit_at(const T* row, int e, int experts) {
  return e < experts ? load_one(row + e) : -INFINITY;
}

// The top-k of one token by one wave; lane j holds choice j's expert (-1:
// none) and weight. Ties go to the lowest index: expert 64 i + l sits in slot
// i of lane l, so the lowest is the first slot, then the first lane.
template <class T, bool RENORM>
__device__ __forceinline__ void route_token(const T* row, int experts, int top_k, int& id, float& weight) {
  constexpr int PER = kMaxExperts / 64;
  const int lane = threadIdx.x % 64;
  float v[PER];
  uint32_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    v[i] = logit_at(row, i * 64 + lane, experts);
    key[i] = order_key(v[i]);
  }
  id = -1;
  float mine = -INFINITY, high = 0.f;
  for (int j = 0; j < top_k; ++j) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) m = key[i] > m ? key[i] : m;
    m = wave_max(m);
    if (m == 0) break;
    bool found = false;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const uint64_t has = __ballot(!found && key[i] == m);
      if (has) {
        const int l = __builtin_ctzll(has);
        const float val = __shfl(v[i], l, 64);
        if (j == 0) high = val;
        if (lane == j) {
          id = i * 64 + l;
          mine = val;
        }
        if (lane == l) key[i] = 0;
        found = true;
      }
    }
  }
  float e = id >= 0 ? expf(mine - high) : 0.f;
  float total;
  if constexpr (RENORM) {
    total = lanes_sum<64>(e);
  } else {
    total = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) total += i * 64 + lane < experts ? expf(v[i] - high) : 0.f;
    total = lanes_sum<64>(total);
  }
  weight = id >= 0 ? e / total : 0.f;
}

// One workgroup routes all tokens and lists the chosen experts.
template <class T, bool RENORM>
__global__ __launch_bounds__(1024) void moe_route_kernel(MoeParams p) {
  __shared__ unsigned long long mask[kMaxExperts];
  __shared__ int64_t first[kMaxExperts + 1], wave_tot[16];
  for (int e = threadIdx.x; e < p.experts; e += 1024) mask[e] = 0;
  __syncthreads();
  const int lane = threadIdx.x % 64;
  for (int t = threadIdx.x / 64; t < p.tokens; t += 16) {
    int id;
    float weight;
    route_token<T, RENORM>(static_cast<const T*>(p.logits) + t * p.ldl, p.experts, p.top_k, id, weight);
    if (lane < p.top_k) {
      p.ids[t * p.top_k + lane] = id;
      p.weights[t * p.top_k + lane] = weight;
      if (id >= 0) atomicOr(&mask[id], 1ull << t);
    }
  }
  __syncthreads();
  // low half: chosen experts before e, high half: their rows
  block_prefix64<1024>(
      p.experts, [&](int e) { return (int64_t)(mask[e] != 0) + ((int64_t)__popcll(mask[e]) << 32); }, first, wave_tot);
  for (int e = threadIdx.x; e < p.experts; e += 1024)
    if (mask[e]) p.table[(int32_t)first[e]] = MoeExpert{e, (int32_t)(first[e] >> 32), mask[e]};
  if (threadIdx.x == 0) *p.active = (int32_t)first[p.experts];
  __syncthreads();
  // this workgroup's own writes of ids and weights, behind the barrier
  for (int i = threadIdx.x; i < p.tokens * p.top_k; i += 1024) {
    const int e = p.ids[i], t = i / p.top_k;
    if (e >= 0) p.share[(int32_t)(first[e] >> 32) + __popcll(mask[e] & ((1ull << t) - 1))] = p.weights[i];
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

__device__ __forceinline__ uint4 zero4() { return uint4{0, 0, 0, 0}; }

// One wave's 16-row tile of a weight operand
template <MoeFormat F>
struct Tile {
  const uint8_t* q;        // this lane's codes of piece 0
  const uint8_t* s;        // MX: this lane's scale of piece 0; blocks: the row block's fp32 scales
  __device__ __forceinline__ void at(const uint8_t* codes, const void* scales, int64_t row0, int64_t row_stride,
                                     int64_t block_stride, int32_t k) {
    const int lane = threadIdx.x % 64, r = lane % 16, g = lane / 16;
    q = codes + (row0 + r) * row_stride + g * 16;
    if constexpr (F == kMoeBlock)
      s = static_cast<const uint8_t*>(scales) + row0 / 128 * (k / 128) * 4;
    else
      s = static_cast<const uint8_t*>(scales) + (F == kMoeFp4 ? g : g / 2) * block_stride + row0 + r;
  }
};

// The codes and scale of one piece; past the row's end zero codes
template <MoeFormat F>
struct Codes {
  uint4 c;
  uint32_t s;
  __device__ __forceinline__ void load(const Tile<F>& t, int piece, int64_t piece_stride, int64_t block_stride,
                                       bool in) {
    c = zero4();
    s = 0;
    if (in) {
      c = *reinterpret_cast<const uint4*>(t.q + piece * piece_stride);
      if constexpr (F == kMoeBlock)
        s = reinterpret_cast<const uint32_t*>(t.s)[piece / 2];
      else
        s = t.s[piece * (F == kMoeFp4 ? 4 : 2) * block_stride];
    }
  }
};

// acc += tile . columns over one piece
template <MoeFormat F>
__device__ __forceinline__ v4f mac(const Codes<F>& w, const v8bf (&a)[Piece<F>::MFMAS],
                                   const uint4 (&x)[Piece<F>::MFMAS], v4f acc) {
  if constexpr (F == kMoeBlock) {
    // an fp32 scale per 128x128 block: on the product, which a code in bf16
    // times a general scale would round
    v4f t = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < Piece<F>::MFMAS; ++j)
      t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[j], __builtin_bit_cast(v8bf, x[j]), t, 0, 0, 0);
    const float s = __uint_as_float(w.s);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = fmaf(s, t[i], acc[i]);
  } else {
#pragma unroll
    for (int j = 0; j < Piece<F>::MFMAS; ++j)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[j], __builtin_bit_cast(v8bf, x[j]), acc, 0, 0, 0);
  }
  return acc;
}

template <MoeFormat F>
__device__ __forceinline__ void decode_all(const Codes<F>& w, v8bf (&a)[Piece<F>::MFMAS]) {
  const float scale = F == kMoeBlock ? 1.f : __uint_as_float(w.s << 23);
#pragma unroll
  for (int j = 0; j < Piece<F>::MFMAS; ++j) a[j] = decode<F>(w.c, j, scale);
}

// The n-th set bit of a word (n < its bit count), the same word in all lanes
__device__ __forceinline__ int nth_bit(uint64_t m, int n) {
  int at = 0;
  for (int i = 0; m; ++i, m &= m - 1)
    if (i == n) at = __builtin_ctzll(m);
  return at;
}

constexpr int kUpWaves = 4;    // waves of a workgroup, sharing the contraction
constexpr int kUpTiles = 2;    // 16-row tiles of W1, and as many of W3

// h of one chosen expert, 32 of its inner columns: W1's and W3's rows against
// the expert's tokens, CT columns of 16 tokens at a time.
template <MoeFormat F, int CT>
__global__ __launch_bounds__(64 * kUpWaves) void moe_up_kernel(MoeParams p) {
  constexpr int M = Piece<F>::MFMAS, RT = 2 * kUpTiles;
  __shared__ v4f lds[kUpWaves][RT * CT][64];
  const int tiles = p.inner / (16 * kUpTiles);
  // four neighbouring tiles (128 rows: one line of every scale block) go to
  // workgroups of the same XCD, which the hardware deals out in turn
  const int b = blockIdx.x, group = b / 32 * 8 + b % 8, item = group * 4 + b % 32 / 8;
  const int slot = item / tiles, tile = item % tiles;
  if (slot >= *p.active) return;
  const MoeExpert ex = p.table[slot];
  const int n = __popcll(ex.tokens);
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, col = lane % 16, g = lane / 16;
  Tile<F> w[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
    w[i].at(p.w13_q, p.w13_s,
            ((int64_t)ex.expert * 2 + i / kUpTiles) * p.inner + (tile * kUpTiles + i % kUpTiles) * 16, p.q13_row,
            p.s13_block, p.hidden);
  const int pieces = (p.hidden + Piece<F>::ELEMS - 1) / Piece<F>::ELEMS;
  const int at = g * Piece<F>::LANE;   // the lane's first element in a piece
  for (int c0 = 0; c0 < n; c0 += 16 * CT) {
    const uint16_t* x[CT];
    bool has[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      const int r = c0 + c * 16 + col;
      has[c] = r < n;
      x[c] = p.x + (int64_t)nth_bit(ex.tokens, r) * p.ldx + at;
    }
    v4f acc[RT][CT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int c = 0; c < CT; ++c) acc[i][c] = v4f{0.f, 0.f, 0.f, 0.f};

    struct Stage {
      Codes<F> w[RT];
      uint4 x[CT][M];
    };
    const auto load = [&](Stage& s, int piece) {
      const bool in = piece * Piece<F>::ELEMS + at < p.hidden;
#pragma unroll
      for (int i = 0; i < RT; ++i) s.w[i].load(w[i], piece, p.q13_piece, p.s13_block, in);
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int j = 0; j < M; ++j)
          s.x[c][j] = in && has[c] ? *reinterpret_cast<const uint4*>(x[c] + piece * Piece<F>::ELEMS + j * 8) : zero4();
    };
    const auto compute = [&](const Stage& s) {
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        v8bf a[M];
        decode_all<F>(s.w[i], a);
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[i][c] = mac<F>(s.w[i], a, s.x[c], acc[i][c]);
      }
    };
    Stage s0, s1;
    load(s0, wave);
    for (int piece = wave; piece < pieces; piece += 2 * kUpWaves) {
      load(s1, piece + kUpWaves);
      compute(s0);
      load(s0, piece + 2 * kUpWaves);
      compute(s1);
    }
    if (c0) __syncthreads();   // the last columns' sums have been read
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int c = 0; c < CT; ++c) lds[wave][i * CT + c][lane] = acc[i][c];
    __syncthreads();
    for (int o = wave; o < kUpTiles * CT; o += kUpWaves) {
      const int i = o / CT, c = o % CT;
      v4f gate = lds[0][i * CT + c][lane], up = lds[0][(kUpTiles + i) * CT + c][lane];
#pragma unroll
      for (int k = 1; k < kUpWaves; ++k) {
        gate += lds[k][i * CT + c][lane];
        up += lds[k][(kUpTiles + i) * CT + c][lane];
      }
      const int r = c0 + c * 16 + col;
      if (r < n) {
        float h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = gate[k] / (1.f + expf(-gate[k])) * up[k];
        // bf16, as between the two grouped products of a training step: the
        // second product reads it as its MFMA operand
        uint16_t* to = p.inner_x + (int64_t)(ex.base + r) * p.inner + (tile * kUpTiles + i) * 16 + g * 4;
        *reinterpret_cast<uint2*>(to) = uint2{bf16_pair(h[0], h[1]), bf16_pair(h[2], h[3])};
      }
    }
  }
}

// y for 16 output columns and all tokens: the workgroup goes through every
// chosen expert, so the sum over a token's experts stays in its registers (no
// atomics, one order). Its waves share the experts' pieces in runs. A column
// of the MFMA is a token; a token that did not choose the expert has a zero
// column, and the share is applied when the expert is done, to its own tokens
// only.
template <MoeFormat F, int CT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void moe_down_kernel(MoeParams p) {
  constexpr int M = Piece<F>::MFMAS;
  __shared__ v4f lds[WAVES][CT][64];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, col = lane % 16, g = lane / 16;
  const int active = *p.active;
  const int pieces = (p.inner + Piece<F>::ELEMS - 1) / Piece<F>::ELEMS;
  const int at = g * Piece<F>::LANE;
  // eight neighbouring tiles (128 rows) on one XCD, as above
  const int b = blockIdx.x, tile = (b / 64 * 8 + b % 8) * 8 + b % 64 / 8;
  if (tile * 16 >= p.hidden) return;
  v4f sum[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) sum[c] = v4f{0.f, 0.f, 0.f, 0.f};
  const int total = active * pieces;
  int item = (int)((int64_t)total * wave / WAVES);
  const int end = (int)((int64_t)total * (wave + 1) / WAVES);
  while (item < end) {
    const int slot = item / pieces, first = item % pieces;
    const int last = min(pieces, first + end - item);
    item += last - first;
    const MoeExpert ex = p.table[slot];
    Tile<F> w;
    w.at(p.w2_q, p.w2_s, (int64_t)ex.expert * p.hidden + tile * 16, p.q2_row, p.s2_block, p.inner);
    const uint16_t* x[CT];
    bool has[CT];
    float share[CT];
    v4f acc[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      const int t = c * 16 + col;
      has[c] = ex.tokens >> t & 1;
      const int row = ex.base + __popcll(ex.tokens & ((1ull << t) - 1));
      x[c] = p.inner_x + (int64_t)(has[c] ? row : ex.base) * p.inner + at;
      share[c] = has[c] ? p.share[row] : 0.f;
      acc[c] = v4f{0.f, 0.f, 0.f, 0.f};
    }
    struct Stage {
      Codes<F> w;
      uint4 x[CT][M];
    };
    const auto load = [&](Stage& s, int piece) {
      const bool in = piece < last && piece * Piece<F>::ELEMS + at < p.inner;
      s.w.load(w, piece, p.q2_piece, p.s2_block, in);
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int j = 0; j < M; ++j)
          s.x[c][j] = in && has[c] ? *reinterpret_cast<const uint4*>(x[c] + piece * Piece<F>::ELEMS + j * 8) : zero4();
    };
    const auto compute = [&](const Stage& s) {
      v8bf a[M];
      decode_all<F>(s.w, a);
#pragma unroll
      for (int c = 0; c < CT; ++c)
        if (CT == 1 || (ex.tokens >> (16 * c) & 0xFFFF)) acc[c] = mac<F>(s.w, a, s.x[c], acc[c]);
    };
    Stage s0, s1;
    load(s0, first);
    for (int piece = first; piece < last; piece += 2) {
      load(s1, piece + 1);
      compute(s0);
      load(s0, piece + 2);
      compute(s1);
    }
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[c][i] = has[c] ? fmaf(share[c], acc[c][i], sum[c][i]) : sum[c][i];
  }
#pragma unroll
  for (int c = 0; c < CT; ++c) lds[wave][c][lane] = sum[c];
  __syncthreads();
  for (int c = wave; c < CT; c += WAVES) {
    v4f v = lds[0][c][lane];
#pragma unroll
    for (int k = 1; k < WAVES; ++k) v += lds[k][c][lane];
    const int t = c * 16 + col;
    if (t < p.tokens)
      *reinterpret_cast<uint2*>(p.out + (int64_t)t * p.hidden + tile * 16 + g * 4) =
          uint2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
  }
}

template <class T>
hipError_t route(const MoeParams& p, bool renormalize, hipStream_t st) {
  if (renormalize) moe_route_kernel<T, true><<<1, 1024, 0, st>>>(p);
  else moe_route_kernel<T, false><<<1, 1024, 0, st>>>(p);
  return hipGetLastError();
}

template <MoeFormat F, int CT>
void down(const MoeParams& p, hipStream_t st) {
  constexpr int WAVES = CT == 1 ? 16 : 8;   // the stages of 2 and 4 columns need over 128 registers
  const uint32_t grid = (uint32_t)((p.hidden / 16 + 63) / 64 * 64);
  moe_down_kernel<F, CT, WAVES><<<grid, 64 * WAVES, 0, st>>>(p);
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
  if (p.tokens <= 16) down<F, 1>(p, st);
  else if (p.tokens <= 32) down<F, 2>(p, st);
  else down<F, 4>(p, st);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_moe_layer(const MoeParams& p, MoeFormat fmt, bool logits_f32, bool renormalize, hipStream_t st) {
  const hipError_t e = logits_f32 ? route<float>(p, renormalize, st) : route<bf16_t>(p, renormalize, st);
  if (e != hipSuccess) return e;
  if (fmt == kMoeFp4) return products<kMoeFp4>(p, st);
  if (fmt == kMoeFp8) return products<kMoeFp8>(p, st);
  return products<kMoeBlock>(p, st);
}

}  // namespace mxgg
