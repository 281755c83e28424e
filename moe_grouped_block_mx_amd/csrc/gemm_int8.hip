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

#define MXGG_LDS __attribute__((address_space(3)))

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}
// Workgroup barrier without a memory fence (which would wait for every load to
// LDS in flight)
__device__ __forceinline__ void raw_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
__device__ __forceinline__ void dma16(const uint8_t* src, uint8_t* lds) {
  __builtin_amdgcn_global_load_lds((const void*)src, (MXGG_LDS void*)lds, 16, 0, 0);
}
// what stands in for the codes behind the contraction's end
static __device__ __attribute__((aligned(64))) uint32_t g_zeros[16];

constexpr int kTile = 256;            // channels and tokens of a tile
constexpr int kStageK = 128;          // codes of a row in a stage
constexpr int kOperand = kTile * kStageK, kStage = 2 * kOperand, kSlots = 2;
constexpr int kThreads = 512, kWaves = kThreads / 64;
constexpr int kWaveN = 128, kWaveM = 64;      // 2 x 4 waves
constexpr int kFN = kWaveN / 32, kFM = kWaveM / 32;
constexpr int kLoads = kOperand / (kWaves * 1024);   // 1 KiB loads of an operand, a wave and stage
constexpr int kTileGroup = 4;

struct Tile {
  const uint8_t* w;       // first channel's codes
  const uint8_t* a;       // first token's
  int64_t row0;
  int g, col0, rows, cols;
};

struct Offsets {
  uint32_t w[kLoads], a[kLoads];
};

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
  const int wn = w / 4, wm = w % 4, h = lane >> 5, l32 = lane & 31;
  const int total = offs[G], stages = (p.k + kStageK - 1) / kStageK;
  const int nb = gridDim.x, b = blockIdx.x;
  // neighbouring tiles on one XCD (workgroups are dealt round the 8 of them):
  // they share operands in its L2
  const int first = nb % 8 == 0 ? (b % 8) * (nb / 8) + b / 8 : b;

  const auto find = [&](int t) {
    Tile o;
    o.g = upper_bound_i32(offs, G + 1, t) - 1;
    const int mt = (offs[o.g + 1] - offs[o.g]) / nt, local = t - offs[o.g];
    const int r0 = local / (kTileGroup * nt) * kTileGroup, hgt = min(mt - r0, kTileGroup), in = local - r0 * nt;
    const int ct = in / hgt, rt = r0 + in % hgt;
    o.row0 = pref[o.g] + (int64_t)rt * kTile;
    o.col0 = ct * kTile;
    o.rows = min(p.sp.m[o.g] - rt * kTile, kTile);
    o.cols = (int)min(p.n - o.col0, (int64_t)kTile);
    o.w = p.w + ((int64_t)o.g * p.n + o.col0) * p.k;
    o.a = p.a + o.row0 * p.k;
    return o;
  };
  // chunk c of row r lies at c ^ (r/2 % 8): the fragments' reads are then
  // without bank conflicts
  const int lr = lane / 8, lc = lane % 8;
  const auto plan = [&](const Tile& o) {
    Offsets f;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int r = (i * kWaves + w) * 8 + lr, c = lc ^ ((r >> 1) & 7);
      f.w[i] = (uint32_t)(min(r, o.cols - 1) * p.k + c * 16);
      f.a[i] = (uint32_t)(min(r, o.rows - 1) * p.k + c * 16);
    }
    return f;
  };
  const auto issue = [&](const Tile& o, const Offsets& f, int s, int slot) {
    uint8_t* at = smem + slot * kStage;
    const uint8_t* zero = reinterpret_cast<const uint8_t*>(g_zeros);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int r = (i * kWaves + w) * 8 + lr, c = lc ^ ((r >> 1) & 7);
      const bool in = s * kStageK + c * 16 < p.k;
      dma16(in ? o.w + s * kStageK + f.w[i] : zero, at + (i * kWaves + w) * 1024);
      dma16(in ? o.a + s * kStageK + f.a[i] : zero, at + kOperand + (i * kWaves + w) * 1024);
    }
  };

  if (first >= total) return;
  Tile cur = find(first);
  Offsets f = plan(cur);
  int slot = 0;
  issue(cur, f, 0, 0);
  for (int t = first; t < total; t += nb) {
    v16i acc[kFN][kFM];
#pragma unroll
    for (int i = 0; i < kFN; ++i)
#pragma unroll
      for (int j = 0; j < kFM; ++j) acc[i][j] = v16i{};
    Tile next = cur;
    for (int s = 0; s < stages; ++s) {
      wait_vmcnt<0>();
      raw_barrier();
      if (s + 1 < stages) {
        issue(cur, f, s + 1, slot ^ 1);
      } else if (t + nb < total) {
        next = find(t + nb);
        f = plan(next);
        issue(next, f, 0, slot ^ 1);
      }
      const uint8_t* wt = smem + slot * kStage + wn * kWaveN * kStageK;
      const uint8_t* at = smem + slot * kStage + kOperand + wm * kWaveM * kStageK;
#pragma unroll
      for (int u = 0; u < kStageK / 32; ++u) {
        v4i wf[kFN], af[kFM];
#pragma unroll
        for (int i = 0; i < kFN; ++i) {
          const int r = i * 32 + l32;
          wf[i] = *reinterpret_cast<const v4i*>(wt + r * kStageK + ((2 * u + h) ^ ((r >> 1) & 7)) * 16);
        }
#pragma unroll
        for (int j = 0; j < kFM; ++j) {
          const int r = j * 32 + l32;
          af[j] = *reinterpret_cast<const v4i*>(at + r * kStageK + ((2 * u + h) ^ ((r >> 1) & 7)) * 16);
        }
#pragma unroll
        for (int i = 0; i < kFN; ++i)
#pragma unroll
          for (int j = 0; j < kFM; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[i], af[j], acc[i][j], 0, 0, 0);
      }
      slot ^= 1;
    }
    // Epilogue: a lane has channels 8q + 4h .. +3 of token l32 in registers 4q ..
    // 4q + 3; the two halves of a wave exchange every other group, so that each
    // lane stores eight neighbouring channels.
#pragma unroll
    for (int j = 0; j < kFM; ++j) {
      const int m = wm * kWaveM + j * 32 + l32;
      const float sa = p.as[cur.row0 + min(m, cur.rows - 1)];
#pragma unroll
      for (int i = 0; i < kFN; ++i)
#pragma unroll
        for (int q = 0; q < 4; q += 2) {
          uint32_t v[4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int n0 = wn * kWaveN + i * 32 + 8 * (q + e) + 4 * h;
            float o[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int n = min(n0 + c, cur.cols - 1);
              o[c] = (float)acc[i][j][4 * (q + e) + c] * sa * p.ws[(int64_t)cur.g * p.n + cur.col0 + n];
            }
            v[2 * e] = bf16_pair(o[0], o[1]);
            v[2 * e + 1] = bf16_pair(o[2], o[3]);
          }
          // lower half: group q of both halves; upper half: group q + 1
          const auto lo = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
          const auto hi = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
          const uint32_t d[4] = {lo[0], hi[0], lo[1], hi[1]};
          const int n0 = wn * kWaveN + i * 32 + 8 * (q + h);
          if (m < cur.rows) {
            uint16_t* out = p.out + (cur.row0 + m) * p.n + cur.col0 + n0;
            if (n0 + 8 <= cur.cols) memcpy(out, d, 16);
            else
              for (int c = 0; c < 8; ++c)
                if (n0 + c < cur.cols) out[c] = (uint16_t)(d[c / 2] >> (16 * (c % 2)));
          }
        }
    }
    cur = next;
  }
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
