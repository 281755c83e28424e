// Products of 8-bit integers, expert by expert, with a scale for each token and
// for each output channel; and the quantizer that makes codes and scales.
//
//   s[r] = amax_k |x[r, k]| / 127,  q[r, k] = the integer next to 127 x / amax
//   out[r, n] = a_s[r] w_s[g, n] sum_k a[r, k] w[g, n, k]
//
// The sum is exact: |codes| <= 128 and K < 2^17, so it fits in 32 bits. It is
// rounded to fp32 for the scales, and once more to bf16.
#include "block_common.hpp"
#include "launch.hpp"
#include "token_launch.hpp"

namespace mxgg {
namespace {

typedef int v2i __attribute__((ext_vector_type(2)));

// ---------------------------------------------------------------------------
// Quantizer
//
// A row belongs to L lanes that keep it in registers, so it is read once. The
// code of an element is exact: 127 x / amax is first approximated with the
// reciprocal and then corrected by its remainder, which leaves it about 2^-24 of itself
// off, and a quotient half way between two integers, which fp32 holds, is found as that
// and goes to the even one. No other is as near to half way: with significands X and A
// from 128 to 255, d binades apart, the quotient is q = 127 X / (A 2^d), below 253 / 2^d
// (127 for d = 0), and |q - n - 1/2| = |254 X - (2 n + 1) A 2^d| / (2 A 2^d) is 0 or at
// least 1 / (255 2^d) (the numerator is even; for d = 0 at least 1 / 510): more than
// 2^-16 q.
//
// What bounds it: the bytes. 65536 x 512 18 us (5.7 TB/s), 16384 x 7168 63 us (5.6),
// 4096 x 20480, read twice, 53 us (the second time from cache); 1 x 7168 2.6 us.

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  typedef uint16_t v2u __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(v2u, a), __builtin_bit_cast(v2u, b)));
}

struct Int8Row {
  float k;        // a power of two that keeps amax and its reciprocal normal
  float amax;     // times k
  float inv;
  bool codes;     // false: zeros (a row of zeros, or with NaN or infinity: its scale says so)
  float scale;
  // bits: the largest |element| as bf16, NaN above all
  __device__ __forceinline__ explicit Int8Row(uint32_t bits) {
    const int e = (int)(bits >> 7);
    const float top = __uint_as_float(bits << 16);
    k = e >= 191 ? 0x1p-64f : e <= 63 ? 0x1p64f : 1.f;
    codes = bits != 0 && e < 255;
    amax = codes ? top * k : 1.f;
    inv = 1.f / amax;
    scale = top / 127.f;
  }
  __device__ __forceinline__ uint32_t code(float x) const {
    const float t = x * k * 127.f, y = t * inv;
    const float q = __builtin_rintf(__builtin_fmaf(__builtin_fmaf(-y, amax, t), inv, y));
    return (uint32_t)(int)q & 0xFFu;
  }
  __device__ __forceinline__ uint64_t codes8(const Chunk<bf16_t>& c) const {
    if (!codes) return 0;
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      w[h] = code(c.get(4 * h)) | code(c.get(4 * h + 1)) << 8 | code(c.get(4 * h + 2)) << 16 | code(c.get(4 * h + 3)) << 24;
    return w[0] | (uint64_t)w[1] << 32;
  }
};

// NV chunks a lane in registers; without STAY a row is read twice.
template <int L, int NV, int THREADS, bool STAY>
__global__ __launch_bounds__(THREADS) void quant_int8_kernel(const uint16_t* x, int64_t rows, int chunks, int64_t ldx,
                                                             int8_t* q, float* scales) {
  constexpr int PER = THREADS / L, WAVES = L > 64 ? L / 64 : 1;
  __shared__ uint32_t part[THREADS / 64];
  const int lane = threadIdx.x % L;
  for (int64_t r0 = (int64_t)blockIdx.x * PER; r0 < rows; r0 += (int64_t)gridDim.x * PER) {
    const int64_t r = r0 + threadIdx.x / L;
    const bool here = r < rows;
    const bf16_t* row = reinterpret_cast<const bf16_t*>(x) + (here ? r : rows - 1) * ldx;
    Chunk<bf16_t> c[NV];
    uint32_t top = 0;
    for (int base = 0; base < chunks; base += L * NV) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int at = base + i * L + lane;
        c[i].load(row + (at < chunks ? at : chunks - 1) * 8);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int w = 0; w < 4; ++w) top = max_u16x2(top, c[i].w[w] & 0x7FFF7FFFu);
      if (STAY) break;
    }
    top = max(top & 0xFFFFu, top >> 16);
    top = max(top, rotate<8>(top));
    top = max(top, rotate<4>(top));
    top = max(top, rotate<2>(top));
    top = max(top, rotate<1>(top));
    if constexpr (L >= 32) top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
    if constexpr (L >= 64) top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
    if constexpr (L > 64) {
      if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = top;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < WAVES; ++w) top = max(top, part[threadIdx.x / L * WAVES + w]);
      __syncthreads();   // the next row's are written after this
    }
    if (!here) continue;
    const Int8Row s(top);
    if (lane == 0) scales[r] = s.scale;
    int8_t* out = q + r * (int64_t)chunks * 8;
    for (int base = 0; base < chunks; base += L * NV) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int at = base + i * L + lane;
        if (at >= chunks) continue;
        if (!STAY) c[i].load(row + at * 8);
        const uint64_t v = s.codes8(c[i]);
        memcpy(out + at * 8, &v, 8);
      }
      if (STAY) break;
    }
  }
}

template <int L, int NV, bool STAY = true>
hipError_t quant_int8(const uint16_t* x, int64_t rows, int64_t cols, int64_t ldx, int8_t* q, float* scales, hipStream_t st) {
  constexpr int THREADS = L < 256 ? 256 : L, PER = THREADS / L;
  const int64_t blocks = (rows + PER - 1) / PER, most = 1 << 20;   // a launch has 2^32 threads at most
  quant_int8_kernel<L, NV, THREADS, STAY><<<(uint32_t)(blocks < most ? blocks : most), THREADS, 0, st>>>(x, rows, (int)(cols / 8), ldx, q, scales);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Product
//
// Weights are the MFMA's first operand, tokens the second: register c of lane l of
// a 16x16 result is then channel 4 (l / 16) + c of token l % 16, four neighbouring
// channels of one row.
//
// A workgroup has 256 channels and 256 tokens at a time, and its eight waves 128 x
// 64 of them each. Stages of 64 codes of every row come to LDS by DMA, four slots in
// a ring that runs on over the workgroup's tiles. The two waves of a SIMD take
// turns: while one reads a stage's operands from LDS and issues loads, the other
// has the matrix unit to itself, and a barrier swaps them. Loads are through
// buffers that end with the tile's rows, so what lies past an end is zeros without
// a comparison.
//
// 16x16x64 MFMAs, not 32x32x32, whose results move twice the accumulators for the same
// operations: 8192 x 8192 x 8192 takes 435 - 465 us with them and took 464 - 478 with those,
// the two run in turns. (Of zeros for codes 346 - 356 and 312: without a limit by power it
// would be the other way round.)
//
// What bounds it: large products of real codes the power of the card. 8192^3 in
// 435 - 465 us is 2360 - 2530 Tops (a bf16 product reaches half of that); the same launch
// on zeros, the same instructions, takes 346 - 356, up to 3180 Tops. Issuing the loads
// between the MFMAs instead of in the other turn, and letting a tile's stores run on into
// the next tile, changed nothing. Of 64 experts with 512 rows each on average (32768 x
// 4096 x 7168, 1020 - 1060 us) a quarter of the tiles' rows are past an expert's end. A
// 128 x 128 tile brings a byte for 128 operations and is bound by that: 4096 x 4096 x
// 4096, four tiles of 1 MB on every CU, takes 83 us, 51 bytes a ns and CU.

#define MXGG_LDS __attribute__((address_space(3)))

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}
// all reads from LDS
__device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt(0xF | (3 << 14) | (0x7 << 4)); }
// Workgroup barrier without a memory fence (which would wait for every load to
// LDS in flight); nothing moves across it.
__device__ __forceinline__ void raw_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}
// Between a wave's lanes that meet in LDS (its accesses are done in order)
__device__ __forceinline__ void wave_fence() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_wave_barrier();
}
// A buffer from a wave-uniform base: reads past its end give zeros
__device__ __forceinline__ __amdgpu_buffer_rsrc_t uniform_buffer(const void* base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(((uint64_t)hi << 32) | lo), 0,
                                           (int)__builtin_amdgcn_readfirstlane(bytes), 0x00020000);
}
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
constexpr uint32_t kOutside = 0x80000000u;   // an offset past every buffer's end

constexpr int kThreads = 512, kWaves = kThreads / 64;
constexpr int kTileGroup = 4;

// FN fragments of 16 channels and FM of 16 tokens a wave; 64 KU codes of a row in a
// stage. The waves are 2 x 4 over the tile, or with SPLIT 2 x 2 twice: each half
// then multiplies every other stage.
template <int FN, int FM, int KU, int SLOTS, bool SPLIT>
struct Int8Tile {
  static constexpr int K = 64 * KU, CHUNKS = 4 * KU;
  static constexpr int WN = 16 * FN, WM = 16 * FM, TN = 2 * WN, TM = (SPLIT ? 2 : 4) * WM;
  static constexpr int W_BYTES = TN * K, STAGE = (TN + TM) * K, LDS = SLOTS * STAGE;
  // a wave's way out: 16 tokens of 64 channels, rows 16 bytes apart more
  static constexpr int OUT_PITCH = 144, OUT_BYTES = 16 * OUT_PITCH;
  static constexpr int SMEM = LDS + kWaves * OUT_BYTES;
  // 1 KiB loads of a wave and stage
  static constexpr int LW = W_BYTES / (kWaves * 1024), LA = TM * K / (kWaves * 1024);
  // loads of the stages that are on their way behind the awaited one
  static constexpr int AHEAD = (SLOTS - 2) * (LW + LA);
  // rows of a load, and of a load of all waves
  static constexpr int LOAD_ROWS = 16 / KU, ROUND_ROWS = kWaves * LOAD_ROWS;
  static constexpr int MORE = SLOTS - 1;                  // stages issued ahead
  static_assert(SMEM <= 154 * 1024 && LW >= 1 && LA >= 1 && FN % 4 == 0, "LDS: the ring beside the tables; whole loads");
};

struct Tile {
  int row0, g, col0, rows, cols;
};

// The first `left` (1 to 7) of eight bf16
__device__ __forceinline__ void store_some(uint16_t* out, uint32_t d0, uint32_t d1, uint32_t d2, uint32_t d3, int left) {
  if (left & 4) {
    const uint64_t v = d0 | (uint64_t)d1 << 32;
    memcpy(out, &v, 8);
  }
  const uint32_t a = left & 4 ? d2 : d0, b = left & 4 ? d3 : d1;
  if (left & 2) memcpy(out + (left & 4), &a, 4);
  if (left & 1) out[left & 6] = (uint16_t)(left & 2 ? b : a);
}

// Chunk c of a row lies at c ^ swizzle(row): the 16 rows of a fragment's read are
// then spread over all banks.
template <class T>
__device__ __forceinline__ int swizzle(int row) {
  return T::CHUNKS == 4 ? row / 4 % 4 : row / 2 % 8;
}

// The workgroup's tiles and the stages on their way: every wave issues its share
// of one stage after the other, from tile to tile.
template <class T>
struct Int8Stream {
  const Int8Params& p;
  uint8_t* smem;
  const int32_t *pref, *offs;       // LDS: an expert's first row, and first tile
  int w, lane, nt, total, nb, first;
  int stages;                       // of a tile; the last ones may lie behind the contraction's end
  int it, is = 0, slot = 0;         // what is issued next
  uint32_t lane_off;
  int lane_k;                       // codes of the lane's chunk begin here in a stage
  const uint8_t *base_w, *base_a;
  uint32_t size_w = 0, size_a = 0;

  __device__ __forceinline__ Int8Stream(const Int8Params& q, uint8_t* lds, int32_t* rows_at, int32_t* tiles_at,
                                        int stages_of_a_tile)
      : p(q), smem(lds), pref(rows_at), offs(tiles_at), stages(stages_of_a_tile) {
    const int G = p.sp.G;
    nt = (int)((p.n + T::TN - 1) / T::TN);
    int64_t* both = reinterpret_cast<int64_t*>(smem);     // the ring is not in use yet
    block_prefix64<kThreads>(G, [&](int g) {
      return (int64_t)token_pieces(p.sp.m[g], T::TM) << 32 | p.sp.m[g];
    }, both, both + kMaxExperts + 1);
    for (int g = threadIdx.x; g <= G; g += kThreads) {
      rows_at[g] = (int32_t)both[g];
      tiles_at[g] = (int32_t)(both[g] >> 32) * nt;
    }
    __syncthreads();
    lane = threadIdx.x & 63;
    w = uniform(threadIdx.x >> 6);
    total = uniform(offs[G]);
    nb = gridDim.x;
    // neighbouring tiles on one XCD (workgroups are dealt round the 8 of them):
    // they share operands in its L2
    const int b = blockIdx.x;
    first = it = nb % 8 == 0 ? (b % 8) * (nb / 8) + b / 8 : b;
    const int r = w * T::LOAD_ROWS + lane / T::CHUNKS;
    lane_k = ((lane % T::CHUNKS) ^ swizzle<T>(r)) * 16;
    lane_off = (uint32_t)(r * p.k + lane_k);
    base_w = p.w;
    base_a = p.a;
  }
  __device__ __forceinline__ Tile find(int t) const {
    Tile o;
    o.g = uniform(upper_bound_i32(offs, p.sp.G + 1, t) - 1);
    const int o0 = uniform(offs[o.g]), mt = (uniform(offs[o.g + 1]) - o0) / nt, local = t - o0;
    const int r0 = local / (kTileGroup * nt) * kTileGroup, hgt = min(mt - r0, kTileGroup), in = local - r0 * nt;
    const int ct = in / hgt, rt = r0 + in % hgt;
    o.row0 = uniform(pref[o.g]) + rt * T::TM;
    o.col0 = ct * T::TN;
    o.rows = min(p.sp.m[o.g] - rt * T::TM, T::TM);
    o.cols = (int)min(p.n - o.col0, (int64_t)T::TN);
    return o;
  }
  __device__ __forceinline__ void aim() {
    size_w = size_a = 0;                                  // nothing left: zeros, that the counts go on
    if (it >= total) return;
    const Tile o = find(it);
    base_w = p.w + ((int64_t)o.g * p.n + o.col0) * p.k;
    base_a = p.a + (int64_t)o.row0 * p.k;
    size_w = (uint32_t)(o.cols * p.k);
    size_a = (uint32_t)(o.rows * p.k);
  }
  __device__ __forceinline__ void issue() const {
    uint8_t* at = smem + slot * T::STAGE + w * 1024;
    const __amdgpu_buffer_rsrc_t bw = uniform_buffer(base_w, size_w), ba = uniform_buffer(base_a, size_a);
    // zeros behind the contraction's end, of the tokens (the weights may be anything)
    const uint32_t wo = lane_off + (uint32_t)(is * T::K), round = (uint32_t)(T::ROUND_ROWS * p.k);
    const uint32_t ao = is * T::K + lane_k < p.k ? wo : kOutside;
#pragma unroll
    for (int i = 0; i < T::LW; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(bw, (MXGG_LDS void*)(at + i * (kWaves * 1024)), 16,
                                               wo + (uint32_t)i * round, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < T::LA; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ba, (MXGG_LDS void*)(at + T::W_BYTES + i * (kWaves * 1024)), 16,
                                               ao + (uint32_t)i * round, 0, 0, 0);
  }
  __device__ __forceinline__ void advance() {
    slot = slot + 1 == T::MORE + 1 ? 0 : slot + 1;
    if (++is == stages) {
      is = 0;
      it += nb;
      aim();
    }
  }
  // the ring filled, its first stage landed
  __device__ __forceinline__ void start() {
    aim();
    for (int s = 0; s < T::MORE; ++s) {
      issue();
      advance();
    }
    wait_vmcnt<T::AHEAD>();
    raw_barrier();
  }
};

// Operands of a stage in a wave's registers: fragments of 16 rows, of which lane l
// holds codes 64 u + 16 (l / 16) .. of row l % 16.
template <int FN, int FM, int KU, class T>
struct Int8Operands {
  v4i w[KU][FN], a[KU][FM];
  __device__ __forceinline__ void read(const uint8_t* st, int wn, int wm, int lane) {
#pragma unroll
    for (int u = 0; u < KU; ++u) {
      const int l16 = lane % 16, piece = l16 * T::K + ((4 * u + lane / 16) ^ swizzle<T>(l16)) * 16;
#pragma unroll
      for (int i = 0; i < FN; ++i) w[u][i] = *reinterpret_cast<const v4i*>(st + wn * T::WN * T::K + piece + i * 16 * T::K);
#pragma unroll
      for (int j = 0; j < FM; ++j)
        a[u][j] = *reinterpret_cast<const v4i*>(st + T::W_BYTES + wm * T::WM * T::K + piece + j * 16 * T::K);
    }
  }
  __device__ __forceinline__ void multiply(v4i (&acc)[FN][FM]) const {
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int u = 0; u < KU; ++u)
#pragma unroll
      for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[u][i], a[u][j], acc[i][j], 0, 0, 0);
    __builtin_amdgcn_s_setprio(0);
  }
};

template <int FN, int FM>
__device__ __forceinline__ void clear(v4i (&acc)[FN][FM]) {
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[i][j] = v4i{};
}

// A wave's sums, of channels n0 .. and tokens m0 .. of the tile, scaled and stored:
// 16 tokens of 64 channels go through LDS and leave as whole lines.
template <int FN, int FM, class T>
__device__ __forceinline__ void store_sums(const Int8Params& p, const Tile& cur, const v4i (&acc)[FN][FM], int n0, int m0,
                                           uint8_t* scr, int lane) {
  const int h = lane / 16, l16 = lane % 16;
  const __amdgpu_buffer_rsrc_t scales = uniform_buffer(p.ws + (int64_t)cur.g * p.n + cur.col0, (uint32_t)cur.cols * 4);
  float sa[FM];
#pragma unroll
  for (int j = 0; j < FM; ++j) sa[j] = p.as[cur.row0 + min(m0 + j * 16 + l16, cur.rows - 1)];
  const int m_out = m0 + lane / 8, n_out = n0 + lane % 8 * 8;
  uint16_t* out = p.out + ((int64_t)cur.row0 + m_out) * p.n + cur.col0 + n_out;
#pragma unroll
  for (int c = 0; c < FN / 4; ++c) {
    v4f sw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      sw[i] = __builtin_bit_cast(
          v4f, __builtin_amdgcn_raw_buffer_load_b128(scales, (n0 + c * 64 + i * 16 + 4 * h) * 4, 0, 0));
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      wave_fence();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float o[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) o[r] = (float)acc[4 * c + i][j][r] * sa[j] * sw[i][r];
        *reinterpret_cast<v2i*>(scr + l16 * T::OUT_PITCH + (i * 16 + 4 * h) * 2) =
            v2i{(int)bf16_pair(o[0], o[1]), (int)bf16_pair(o[2], o[3])};
      }
      wave_fence();
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const v4i o = *reinterpret_cast<const v4i*>(scr + (lane / 8 + 8 * k) * T::OUT_PITCH + lane % 8 * 16);
        const int down = j * 16 + k * 8, left = cur.cols - n_out - c * 64;
        uint16_t* to = out + (int64_t)down * p.n + c * 64;
        if (m_out + down < cur.rows) {
          if (left >= 8) memcpy(to, &o, 16);
          else if (left > 0) store_some(to, o[0], o[1], o[2], o[3], left);
        }
      }
    }
  }
}

template <int FN, int FM, int KU, int SLOTS>
__global__ __launch_bounds__(kThreads, 1) void grouped_int8_kernel(const Int8Params p) {
  using T = Int8Tile<FN, FM, KU, SLOTS, false>;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ int32_t pref[kMaxExperts + 1], offs[kMaxExperts + 1];
  Int8Stream<T> in(p, smem, pref, offs, (p.k + T::K - 1) / T::K);
  const int w = in.w, lane = in.lane, turn = w / 4, wn = turn, wm = turn ? 3 - w % 4 : w % 4;
  if (in.first >= in.total) return;
  in.start();
  if (turn) raw_barrier();                                // the second four waves are one turn behind
  int slot = 0;
  for (int t = in.first; t < in.total; t += in.nb) {
    const Tile cur = in.find(t);
    const bool busy = wn * T::WN < cur.cols && wm * T::WM < cur.rows;   // else nothing of the wave's is stored
    v4i acc[FN][FM];
    clear(acc);
    for (int s = 0; s < in.stages; ++s) {
      Int8Operands<FN, FM, KU, T> f;
      if (busy) f.read(smem + slot * T::STAGE, wn, wm, lane);
      slot = slot + 1 == SLOTS ? 0 : slot + 1;
      in.issue();
      in.advance();
      wait_lds();
      if (turn) wait_vmcnt<T::AHEAD>();
      raw_barrier();
      if (busy) f.multiply(acc);
      if (!turn) wait_vmcnt<T::AHEAD>();
      raw_barrier();
    }
    if (busy) store_sums<FN, FM, T>(p, cur, acc, wn * T::WN, wm * T::WM, smem + T::LDS + w * T::OUT_BYTES, lane);
  }
  if (!turn) raw_barrier();
  wait_vmcnt<0>();
}

// The same for smaller tiles, where a turn of half the waves would have too few
// MFMAs for its reads and barriers: the halves take every other stage, all of the
// tile each, and a stage ends with every turn. At a tile's end each half has a sum of
// its own; they give each other the sums of half the tokens, through the slot of the
// last stage, which no load goes to meanwhile.
template <int FN, int FM, int KU, int SLOTS>
__global__ __launch_bounds__(kThreads, 1) void split_int8_kernel(const Int8Params p) {
  using T = Int8Tile<FN, FM, KU, SLOTS, true>;
  static_assert(FM % 2 == 0 && T::STAGE >= kWaves * FN * 1024, "exchange of 16 tokens a wave in a slot");
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ int32_t pref[kMaxExperts + 1], offs[kMaxExperts + 1];
  // an even number of stages (one may hold zeros only)
  Int8Stream<T> in(p, smem, pref, offs, (p.k + 2 * T::K - 1) / (2 * T::K) * 2);
  const int w = in.w, lane = in.lane, turn = w / 4, wn = w % 4 / 2, wm = w % 2;
  if (in.first >= in.total) return;
  in.start();
  int slot = 0;                                           // of the stage that this turn reads
  const auto turn_ends = [&](bool issued) {
    if (issued) in.advance();
    wait_lds();
    if (issued) wait_vmcnt<T::AHEAD>();
    raw_barrier();
    slot = slot + 1 == SLOTS ? 0 : slot + 1;
  };
  for (int t = in.first; t < in.total; t += in.nb) {
    const Tile cur = in.find(t);
    v4i acc[FN][FM];
    clear(acc);
    if (turn) {
      in.issue();
      turn_ends(true);
    }
    for (int s = 0; s < in.stages; s += 2) {
      Int8Operands<FN, FM, KU, T> f;
      f.read(smem + slot * T::STAGE, wn, wm, lane);
      in.issue();
      turn_ends(true);
      const bool more = !turn || s + 2 < in.stages;       // the tile's stages are as many as its turns that issue
      if (more) in.issue();
      f.multiply(acc);
      if (more) turn_ends(true);
    }
    // (its last reads were done before the last barrier)
    uint8_t* last = smem + (slot == 0 ? SLOTS - 1 : slot - 1) * T::STAGE;
    v4i mine[FN][FM / 2];
#pragma unroll
    for (int j = 0; j < FM / 2; ++j) {
      // wave w gives to w ^ 4 and takes what that gives
      v4i* give = reinterpret_cast<v4i*>(last + w * (FN * 1024)) + lane;
      const v4i* take = reinterpret_cast<const v4i*>(last + (w ^ 4) * (FN * 1024)) + lane;
#pragma unroll
      for (int i = 0; i < FN; ++i) give[i * 64] = turn ? acc[i][j] : acc[i][j + FM / 2];
      wait_lds();
      raw_barrier();
#pragma unroll
      for (int i = 0; i < FN; ++i) mine[i][j] = (turn ? acc[i][j + FM / 2] : acc[i][j]) + take[i * 64];
      wait_lds();
      raw_barrier();
    }
    const int m0 = wm * T::WM + turn * (T::WM / 2);
    if (wn * T::WN < cur.cols && m0 < cur.rows)
      store_sums<FN, FM / 2, T>(p, cur, mine, wn * T::WN, m0, smem + T::LDS + w * T::OUT_BYTES, lane);
  }
  wait_vmcnt<0>();
}

// ---------------------------------------------------------------------------
// Product of few tokens
//
// A workgroup has NF fragments of 16 channels and up to MF fragments of 16 tokens of
// one expert; its eight waves split the contraction and meet in LDS at the end.
// 32-bit sums are whole numbers, so their order does not matter. A wave brings its
// 64-code steps to a ring of its own in LDS and waits for its own loads only.
// (Straight to registers a lane would load 16 bytes of another row than its
// neighbour does, which takes the address unit a cycle a lane.)
//
// What bounds it: reading the weights. 64 rows of 128 experts, 2048 x 7168: 110 us for
// the 620 MB of the experts that have any (5.7 TB/s; a plain read reaches 6.4); one row,
// 4096 x 7168: 7 us, of which 4.6 are for the 29 MB.

constexpr int kFewWaves = 8;
constexpr int few_slots(int nf, int mf) { return nf + mf <= 2 ? 4 : nf + mf <= 3 ? 3 : nf + mf <= 4 ? 4 : nf + mf <= 6 ? 3 : 2; }
constexpr int few_lds(int nf, int mf) { return kFewWaves * few_slots(nf, mf) * (nf + mf) * 1024; }

// Expert and rows of piece `seg`, when an expert's tokens go `each` at a time
struct Piece {
  int g, row0, rows;
};
__device__ __forceinline__ Piece find_piece(const SplitArgs& sp, int seg, int each) {
  if (sp.G == 1) return Piece{0, seg * each, min(sp.m[0] - seg * each, each)};
  const int lane = threadIdx.x & 63, per = (sp.G + 63) / 64;
  // pieces (high half) and rows of the lane's experts, then of those before
  uint64_t sum = 0;
  for (int i = 0; i < per; ++i) {
    const int e = lane * per + i, m = e < sp.G ? sp.m[e] : 0;
    sum += (uint64_t)token_pieces(m, each) << 32 | (uint32_t)m;
  }
  uint64_t upto = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint64_t o = __shfl_up((unsigned long long)upto, d, 64);
    if (lane >= d) upto += o;
  }
  const int owner = __popcll(__ballot((int)(upto >> 32) <= seg));   // lanes whose pieces all come before
  const uint64_t before = __shfl((unsigned long long)(upto - sum), owner, 64);
  Piece p;
  int left = uniform(seg - (int)(before >> 32)), row = uniform((int)(uint32_t)before);
  p.g = uniform(owner) * per;
  for (; p.g < sp.G; ++p.g) {
    const int n = token_pieces(sp.m[p.g], each);
    if (left < n) break;
    left -= n;
    row += sp.m[p.g];
  }
  p.row0 = row + left * each;
  p.rows = min(sp.m[p.g] - left * each, each);
  return p;
}

template <int NF, int MF>
__global__ __launch_bounds__(kFewWaves * 64) void few_int8_kernel(const Int8Params p) {
  constexpr int S = few_slots(NF, MF), LOADS = NF + MF, SLOT = LOADS * 1024;
  static_assert(S * LOADS >= NF * MF, "a wave's sums fit in its ring");
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6);
  uint8_t* ring = smem + w * (S * SLOT);
  const Piece pc = find_piece(p.sp, blockIdx.y, 16 * MF);
  const int K = p.k, col0 = (int)blockIdx.x * (16 * NF), cols = (int)min(p.n - col0, (int64_t)(16 * NF));
  const __amdgpu_buffer_rsrc_t bw = uniform_buffer(p.w + ((int64_t)pc.g * p.n + col0) * K, (uint32_t)(cols * K));
  const __amdgpu_buffer_rsrc_t ba = uniform_buffer(p.a + (int64_t)pc.row0 * K, (uint32_t)(pc.rows * K));
  const int steps = (K + 63) / 64, per = (steps + kFewWaves - 1) / kFewWaves;
  const int begin = min(w * per, steps), end = min(begin + per, steps);
  // chunk c of row r lies at c ^ (r/4 % 4), as in the stages above
  const int lc = ((lane % 4) ^ (lane / 16)) * 16;
  const uint32_t row = (uint32_t)(lane / 4 * K + lc);
  const auto issue = [&](int s, int slot) {
    // past the wave's part or the contraction's end: zeros
    const uint32_t off = s < end && s * 64 + lc < K ? row + (uint32_t)(s * 64) : kOutside;
#pragma unroll
    for (int i = 0; i < NF; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(bw, (MXGG_LDS void*)(ring + slot * SLOT + i * 1024), 16,
                                               off + (uint32_t)(i * 16 * K), 0, 0, 0);
#pragma unroll
    for (int j = 0; j < MF; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ba, (MXGG_LDS void*)(ring + slot * SLOT + (NF + j) * 1024), 16,
                                               off + (uint32_t)(j * 16 * K), 0, 0, 0);
  };
  // Scales of the fragments that this wave will store: register c of lane l of
  // fragment (i, j) is channel 16 i + 4 (l / 16) + c of token 16 j + l % 16.
  constexpr int PER = (NF * MF + kFewWaves - 1) / kFewWaves;
  const __amdgpu_buffer_rsrc_t bs = uniform_buffer(p.ws + (int64_t)pc.g * p.n + col0, (uint32_t)cols * 4);
  float sa[PER];
  v4f sw[PER];
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    const int f = w + q * kFewWaves, n = f / MF * 16 + lane / 16 * 4, m = f % MF * 16 + lane % 16;
    sa[q] = p.as[pc.row0 + min(m, pc.rows - 1)];
    sw[q] = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(bs, n * 4, 0, 0));
  }
  v4i acc[NF][MF];
#pragma unroll
  for (int i = 0; i < NF; ++i)
#pragma unroll
    for (int j = 0; j < MF; ++j) acc[i][j] = v4i{};
#pragma unroll
  for (int s = 0; s < S; ++s) issue(begin + s, s);
  const uint8_t* mine = ring + lane % 16 * 64 + ((lane / 16) ^ (lane / 4 % 4)) * 16;
  int slot = 0;
  for (int s = begin; s < end; ++s) {
    wait_vmcnt<(S - 1) * LOADS>();
    __builtin_amdgcn_sched_barrier(0);
    v4i wf[NF], af[MF];
#pragma unroll
    for (int i = 0; i < NF; ++i) wf[i] = *reinterpret_cast<const v4i*>(mine + slot * SLOT + i * 1024);
#pragma unroll
    for (int j = 0; j < MF; ++j) af[j] = *reinterpret_cast<const v4i*>(mine + slot * SLOT + (NF + j) * 1024);
    wait_lds();
    __builtin_amdgcn_sched_barrier(0);
    issue(s + S, slot);
    slot = slot + 1 == S ? 0 : slot + 1;
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
      for (int j = 0; j < MF; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[i], af[j], acc[i][j], 0, 0, 0);
  }
  wait_vmcnt<0>();                                       // zeros still on their way to the ring
  const auto sums_of = [&](int v) { return reinterpret_cast<v4i*>(smem + v * (S * SLOT)) + lane; };
#pragma unroll
  for (int i = 0; i < NF; ++i)
#pragma unroll
    for (int j = 0; j < MF; ++j) sums_of(w)[(i * MF + j) * 64] = acc[i][j];
  __syncthreads();
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    const int f = w + q * kFewWaves;
    if (f >= NF * MF) break;
    v4i sum = sums_of(0)[f * 64];
#pragma unroll
    for (int v = 1; v < kFewWaves; ++v) sum += sums_of(v)[f * 64];
    const int n = f / MF * 16 + lane / 16 * 4, m = f % MF * 16 + lane % 16, left = cols - n;
    if (m >= pc.rows) continue;
    float o[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) o[c] = (float)sum[c] * sa[q] * sw[q][c];
    uint16_t* out = p.out + ((int64_t)pc.row0 + m) * p.n + col0 + n;
    const uint32_t d[2] = {bf16_pair(o[0], o[1]), bf16_pair(o[2], o[3])};
    if (left >= 4) memcpy(out, d, 8);
    else if (left > 0) store_some(out, d[0], d[1], 0, 0, left);
  }
}

template <int NF, int MF>
hipError_t few_int8(const Int8Params& p, hipStream_t st) {
  const hipError_t e = ensure_dynamic_lds((const void*)few_int8_kernel<NF, MF>, few_lds(NF, MF), st);
  if (e != hipSuccess) return e;
  const dim3 grid((uint32_t)((p.n + 16 * NF - 1) / (16 * NF)), (uint32_t)int8_pieces(p.sp, 16 * MF));
  few_int8_kernel<NF, MF><<<grid, kFewWaves * 64, few_lds(NF, MF), st>>>(p);
  return hipGetLastError();
}

template <class T>
hipError_t tile_int8(void (*kernel)(Int8Params), const Int8Params& p, int num_cus, hipStream_t st) {
  const hipError_t e = ensure_dynamic_lds((const void*)kernel, T::SMEM, st);
  if (e != hipSuccess) return e;
  const int64_t tiles = int8_pieces(p.sp, T::TM) * ((p.n + T::TN - 1) / T::TN);
  // Whole eights, so that neighbouring tiles meet on an XCD (a workgroup without a tile
  // ends at once): 2999 rows of 5 experts, 1111 x 2000, 20.3 -> 18.1 us.
  const int64_t grid = (tiles + 7) / 8 * 8;
  kernel<<<(uint32_t)(grid < num_cus ? grid : num_cus), kThreads, T::SMEM, st>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quant_int8(const uint16_t* x, int64_t rows, int64_t cols, int64_t ldx, int8_t* q, float* scales,
                             hipStream_t st) {
  // As many lanes as hold the row in two chunks each: with twice as many, half of them
  // idle, 65536 x 512 took 21 us for 18, 16384 x 1536 19 for 15, 32768 x 2048 37 for 31.
  if (cols <= 16 * 2 * 8) return quant_int8<16, 2>(x, rows, cols, ldx, q, scales, st);
  if (cols <= 32 * 2 * 8) return quant_int8<32, 2>(x, rows, cols, ldx, q, scales, st);
  if (cols <= 64 * 2 * 8) return quant_int8<64, 2>(x, rows, cols, ldx, q, scales, st);
  if (cols <= 128 * 2 * 8) return quant_int8<128, 2>(x, rows, cols, ldx, q, scales, st);
  if (cols <= 256 * 2 * 8) return quant_int8<256, 2>(x, rows, cols, ldx, q, scales, st);
  if (cols <= 512 * 2 * 8) return quant_int8<512, 2>(x, rows, cols, ldx, q, scales, st);
  if (cols <= 1024 * 2 * 8) return quant_int8<1024, 2>(x, rows, cols, ldx, q, scales, st);
  return quant_int8<1024, 2, false>(x, rows, cols, ldx, q, scales, st);
}

hipError_t launch_grouped_int8(const Int8Params& p, int num_cus, hipStream_t st) {
  switch (int8_form(p.sp, p.n, p.k, num_cus)) {
    case kInt8Big: return tile_int8<Int8Tile<8, 4, 1, 4, false>>(grouped_int8_kernel<8, 4, 1, 4>, p, num_cus, st);
    case kInt8Small: return tile_int8<Int8Tile<4, 4, 2, 4, true>>(split_int8_kernel<4, 4, 2, 4>, p, num_cus, st);
    case kInt8Few11: return few_int8<1, 1>(p, st);
    case kInt8Few12: return few_int8<1, 2>(p, st);
    case kInt8Few21: return few_int8<2, 1>(p, st);
    case kInt8Few22: return few_int8<2, 2>(p, st);
    case kInt8Few24: return few_int8<2, 4>(p, st);
    case kInt8Few42: return few_int8<4, 2>(p, st);
    case kInt8Few44: return few_int8<4, 4>(p, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace mxgg
