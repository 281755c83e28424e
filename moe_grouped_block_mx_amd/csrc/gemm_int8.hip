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

typedef int v16i __attribute__((ext_vector_type(16)));

// ---------------------------------------------------------------------------
// Quantizer
//
// A row belongs to L lanes that keep it in registers, so it is read once. The
// code of an element is exact: 127 x / amax is first approximated with the
// reciprocal and then corrected by its remainder, so a quotient half way between
// two integers is seen as that and goes to the even one (any other is at least
// 2^-9 away from half way, far more than the approximation is off).

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
  const int64_t r = (int64_t)blockIdx.x * PER + threadIdx.x / L;
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
  if constexpr (L >= 64) {
    top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
    top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
  }
  if constexpr (L > 64) {
    if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WAVES; ++w) top = max(top, part[threadIdx.x / L * WAVES + w]);
  }
  const Int8Row s(top);
  if (!here) return;
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

template <int L, int NV, bool STAY = true>
hipError_t quant_int8(const uint16_t* x, int64_t rows, int64_t cols, int64_t ldx, int8_t* q, float* scales, hipStream_t st) {
  constexpr int THREADS = L < 256 ? 256 : L, PER = THREADS / L;
  const int64_t blocks = (rows + PER - 1) / PER;
  quant_int8_kernel<L, NV, THREADS, STAY><<<(uint32_t)blocks, THREADS, 0, st>>>(x, rows, (int)(cols / 8), ldx, q, scales);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Product
//
// Weights are the MFMA's first operand, tokens the second: register i of a
// 32x32 result is then channel 8 (i/4) + 4 (lane/32) + i%4 of token lane%32, four
// neighbouring channels of one row.
//
// A workgroup has 256 channels and 256 tokens at a time, and its eight waves 128 x
// 64 of them each. Stages of 64 codes of every row come to LDS by DMA, four slots in
// a ring that runs on over the workgroup's tiles. The two waves of a SIMD take
// turns: while one reads a stage's operands from LDS and issues loads, the other
// has the matrix unit to itself, and a barrier swaps them.

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
// A buffer from a wave-uniform base: reads past its end give zeros
__device__ __forceinline__ __amdgpu_buffer_rsrc_t uniform_buffer(const void* base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(((uint64_t)hi << 32) | lo), 0,
                                           (int)__builtin_amdgcn_readfirstlane(bytes), 0x00020000);
}
constexpr uint32_t kOutside = 0x80000000u;   // an offset past every buffer's end

constexpr int kTile = 256;            // channels and tokens of a tile
constexpr int kStageK = 64;           // codes of a row in a stage
constexpr int kOperand = kTile * kStageK, kStage = 2 * kOperand, kSlots = 4;
constexpr int kThreads = 512, kWaves = kThreads / 64;
constexpr int kWaveN = 128, kWaveM = 64;      // 2 x 4 waves
constexpr int kFN = kWaveN / 32, kFM = kWaveM / 32;
constexpr int kLoads = kOperand / (kWaves * 1024);   // 1 KiB loads of an operand, a wave and stage
constexpr int kTileGroup = 4;

struct Tile {
  int row0, g, col0, rows, cols;
};
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

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

__global__ __launch_bounds__(kThreads, 1) void grouped_int8_kernel(const Int8Params p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ int64_t pref[kMaxExperts + 1], tpref[kMaxExperts + 1], wtot[kWaves];
  __shared__ int32_t offs[kMaxExperts + 1];
  const int G = p.sp.G, nt = (int)((p.n + kTile - 1) / kTile);
  block_prefix64<kThreads>(G, [&](int g) { return (int64_t)p.sp.m[g]; }, pref, wtot);
  block_prefix64<kThreads>(G, [&](int g) { return (int64_t)((p.sp.m[g] + kTile - 1) / kTile); }, tpref, wtot);
  for (int g = threadIdx.x; g <= G; g += kThreads) offs[g] = (int32_t)tpref[g] * nt;
  __syncthreads();

  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int turn = w / 4, wn = turn, wm = turn ? 3 - w % 4 : w % 4, h = lane >> 5, l32 = lane & 31;
  const int K = p.k, total = __builtin_amdgcn_readfirstlane(offs[G]), stages = (K + kStageK - 1) / kStageK;
  const int nb = gridDim.x, b = blockIdx.x;
  // neighbouring tiles on one XCD (workgroups are dealt round the 8 of them):
  // they share operands in its L2
  const int first = nb % 8 == 0 ? (b % 8) * (nb / 8) + b / 8 : b;

  const auto find = [&](int t) {
    Tile o;
    o.g = uniform(upper_bound_i32(offs, G + 1, t) - 1);
    const int o0 = uniform(offs[o.g]), mt = (uniform(offs[o.g + 1]) - o0) / nt, local = t - o0;
    const int r0 = local / (kTileGroup * nt) * kTileGroup, hgt = min(mt - r0, kTileGroup), in = local - r0 * nt;
    const int ct = in / hgt, rt = r0 + in % hgt;
    o.row0 = uniform((int)pref[o.g]) + rt * kTile;
    o.col0 = ct * kTile;
    o.rows = min(p.sp.m[o.g] - rt * kTile, kTile);
    o.cols = (int)min(p.n - o.col0, (int64_t)kTile);
    return o;
  };

  // Issuing side. A load brings 16 rows; chunk c of row r lies at c ^ (r/4 % 4)
  // of the row's four: the fragments' reads are then without bank conflicts.
  const int lr = w * 16 + lane / 4, lc = (lane % 4) ^ (lane / 16);
  const uint32_t lane_off = (uint32_t)(lr * K + lc * 16);
  const int last_k = K - (stages - 1) * kStageK;          // codes of the last stage
  const bool lane_in_last = lc * 16 < last_k;
  int it = first, is = 0, slot_issue = 0;
  const uint8_t *base_w = p.w, *base_a = p.a;
  uint32_t size_w = 0, size_a = 0;
  const auto aim = [&]() {
    size_w = size_a = 0;                                  // nothing left: zeros, that the counts go on
    if (it >= total) return;
    const Tile o = find(it);
    base_w = p.w + ((int64_t)o.g * p.n + o.col0) * K;
    base_a = p.a + (int64_t)o.row0 * K;
    size_w = (uint32_t)(o.cols * K);
    size_a = (uint32_t)(o.rows * K);
  };
  const auto issue = [&]() {
    uint8_t* at = smem + slot_issue * kStage + w * 1024;
    const __amdgpu_buffer_rsrc_t bw = uniform_buffer(base_w, size_w), ba = uniform_buffer(base_a, size_a);
    // zeros behind the contraction's end, of the tokens (the weights may be anything)
    const uint32_t wo = lane_off + (uint32_t)(is * kStageK);
    const uint32_t ao = is + 1 < stages || lane_in_last ? wo : kOutside;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(bw, (MXGG_LDS void*)(at + i * (kWaves * 1024)), 16,
                                               wo + (uint32_t)(i * 128 * K), 0, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ba, (MXGG_LDS void*)(at + kOperand + i * (kWaves * 1024)), 16,
                                               ao + (uint32_t)(i * 128 * K), 0, 0, 0);
    }
  };
  const auto advance = [&]() {
    slot_issue = (slot_issue + 1) & (kSlots - 1);
    if (++is == stages) {
      is = 0;
      it += nb;
      aim();
    }
  };

  if (first >= total) return;
  aim();
#pragma unroll
  for (int s = 0; s < kSlots - 1; ++s) {
    issue();
    advance();
  }
  constexpr int kAhead = 2 * 2 * kLoads;                  // loads of the two stages behind the awaited one
  wait_vmcnt<kAhead>();
  raw_barrier();
  if (turn) raw_barrier();                                // the second four waves are one turn behind
  int slot = 0;
  // a lane's pieces: codes 16 (2u + h) .. of row l32 of a fragment
  const int piece0 = l32 * kStageK + (h ^ ((l32 >> 2) & 3)) * 16, piece1 = piece0 ^ 32;
  const int at_w = wn * kWaveN * kStageK, at_a = kOperand + wm * kWaveM * kStageK;
  for (int t = first; t < total; t += nb) {
    const Tile cur = find(t);
    const bool busy = wn * kWaveN < cur.cols && wm * kWaveM < cur.rows;   // else nothing of the wave's is stored
    v16i acc[kFN][kFM];
#pragma unroll
    for (int i = 0; i < kFN; ++i)
#pragma unroll
      for (int j = 0; j < kFM; ++j) acc[i][j] = v16i{};
    for (int s = 0; s < stages; ++s) {
      v4i wf[2][kFN], af[2][kFM];
      if (busy) {
        const uint8_t* st = smem + slot * kStage;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint8_t* pw = st + at_w + (u ? piece1 : piece0);
          const uint8_t* pa = st + at_a + (u ? piece1 : piece0);
#pragma unroll
          for (int i = 0; i < kFN; ++i) wf[u][i] = *reinterpret_cast<const v4i*>(pw + i * 32 * kStageK);
#pragma unroll
          for (int j = 0; j < kFM; ++j) af[u][j] = *reinterpret_cast<const v4i*>(pa + j * 32 * kStageK);
        }
      }
      slot = (slot + 1) & (kSlots - 1);
      issue();
      advance();
      wait_lds();
      if (turn) wait_vmcnt<kAhead>();
      raw_barrier();
      if (busy) {
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < kFN; ++i)
#pragma unroll
            for (int j = 0; j < kFM; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[u][i], af[u][j], acc[i][j], 0, 0, 0);
        __builtin_amdgcn_s_setprio(0);
      }
      if (!turn) wait_vmcnt<kAhead>();
      raw_barrier();
    }
    // Epilogue: a lane has channels 8q + 4h .. +3 of token l32 in registers 4q ..
    // 4q + 3; the two halves of a wave exchange every other group, so that each
    // lane stores eight neighbouring channels.
    if (!busy) continue;
    const __amdgpu_buffer_rsrc_t scales =
        uniform_buffer(p.ws + (int64_t)cur.g * p.n + cur.col0, (uint32_t)cur.cols * 4);
    uint16_t* row[kFM];
    float sa[kFM];
    bool have[kFM];
#pragma unroll
    for (int j = 0; j < kFM; ++j) {
      const int m = wm * kWaveM + j * 32 + l32;
      have[j] = m < cur.rows;
      sa[j] = p.as[cur.row0 + min(m, cur.rows - 1)];
      row[j] = p.out + (int64_t)(cur.row0 + m) * p.n + cur.col0;
    }
#pragma unroll
    for (int i = 0; i < kFN; ++i) {
      const int n0 = wn * kWaveN + i * 32;
      v4f sw[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        sw[q] = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(scales, (n0 + 8 * q + 4 * h) * 4, 0, 0));
#pragma unroll
      for (int j = 0; j < kFM; ++j)
#pragma unroll
        for (int q = 0; q < 4; q += 2) {
          uint32_t v[4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float o[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) o[c] = (float)acc[i][j][4 * (q + e) + c] * sa[j] * sw[q + e][c];
            v[2 * e] = bf16_pair(o[0], o[1]);
            v[2 * e + 1] = bf16_pair(o[2], o[3]);
          }
          // lower half: group q of both halves; upper half: group q + 1
          const auto lo = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
          const auto hi = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
          const uint32_t d[4] = {lo[0], hi[0], lo[1], hi[1]};
          const int n = n0 + 8 * (q + h), left = cur.cols - n;
          if (have[j] && left >= 8) memcpy(row[j] + n, d, 16);
          if (cur.cols % 8 && have[j] && left > 0 && left < 8) store_some(row[j] + n, d[0], d[1], d[2], d[3], left);
        }
    }
  }
  if (!turn) raw_barrier();
  wait_vmcnt<0>();
}

}  // namespace

hipError_t launch_quant_int8(const uint16_t* x, int64_t rows, int64_t cols, int64_t ldx, int8_t* q, float* scales,
                             hipStream_t st) {
  if (cols <= 16 * 2 * 8) return quant_int8<16, 2>(x, rows, cols, ldx, q, scales, st);
  if (cols <= 64 * 2 * 8) return quant_int8<64, 2>(x, rows, cols, ldx, q, scales, st);
  if (cols <= 256 * 2 * 8) return quant_int8<256, 2>(x, rows, cols, ldx, q, scales, st);
  if (cols <= 512 * 2 * 8) return quant_int8<512, 2>(x, rows, cols, ldx, q, scales, st);
  if (cols <= 1024 * 2 * 8) return quant_int8<1024, 2>(x, rows, cols, ldx, q, scales, st);
  return quant_int8<1024, 2, false>(x, rows, cols, ldx, q, scales, st);
}

hipError_t launch_grouped_int8(const Int8Params& p, int num_cus, hipStream_t st) {
  const hipError_t e = ensure_dynamic_lds((const void*)grouped_int8_kernel, kSlots * kStage, st);
  if (e != hipSuccess) return e;
  int64_t tiles = 0;
  for (int g = 0; g < p.sp.G; ++g) tiles += (p.sp.m[g] + kTile - 1) / kTile;
  tiles *= (p.n + kTile - 1) / kTile;
  const uint32_t grid = (uint32_t)(tiles < num_cus ? tiles : num_cus);
  grouped_int8_kernel<<<grid, kThreads, kSlots * kStage, st>>>(p);
  return hipGetLastError();
}

}  // namespace mxgg
