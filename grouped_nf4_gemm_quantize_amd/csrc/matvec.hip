// Products of a few activation rows with one 4-bit matrix that has group
// scales: y[t, n] = bias[n] + sum_g s[n, g] sum_{k in g} (v(code) - z[n, g]) x[t, k].
//
// Bound by the read of the codes, so the arithmetic has to stay below it: 4-bit
// codes at 5 TB/s are 10^13 weights a second, four vector operations each. The
// products go through the matrix unit (16x16x32 fp16, sums in fp32), whose
// 16 rows of x cost the same for one token as for sixteen; a weight costs half a
// v_perm_b32 and half an LDS read to decode, through a table byte -> two
// fp16 values with one copy per lane slot, so that random bytes never share a
// bank.
//
// The eight waves of a workgroup share the K axis of 16 output rows (a tile) in
// chunks of 128, chunk c of wave c % 8.  A lane reads 16 consecutive packed bytes
// (32 codes) of one row; four lane swaps then give each of the chunk's four matrix
// steps 32 consecutive k, all of one scale group, whose sum is scaled in fp32.
// A wave's part of x stays in registers from tile to tile.  The waves' sums meet in LDS.
//
// nf4's levels are no fp16 values: each is held as a sum of two (22 bits),
// scaled by 2^8 so that the small parts stay normal, and multiplied twice.  All
// other formats' values are exact in fp16 (fp4's 1/6 and the 2^-8 are applied to
// the final sum).

#include "common.h"
#include "launch.h"

namespace nf4moe {

namespace {

constexpr int kMvThreads = 512;
constexpr int kMvWaves = kMvThreads / 64;
constexpr int kMvTile = 16;     // output rows of one matrix step
constexpr int kMvTokens = 16;   // rows of x of one matrix step
constexpr int kMvChunk = 128;   // k of one lane-wide read

enum MvKind { kPlain = 0, kSplit = 1, kZeros = 2 };  // fp16 table; two tables; minus zeros

struct MvScales {
  uint32_t s[4];  // raw scales of a chunk's groups
  uint32_t z;     // raw zeros, one byte a group
};

// Raw scale i of the matrix (its bits, widened).
__device__ __forceinline__ uint32_t mv_raw(const MatvecArgs& a, int64_t i) {
  if (a.qt == kMvMXFP4) return reinterpret_cast<const uint8_t*>(a.scales)[i];
  if (a.scale_dtype == kF32) return reinterpret_cast<const uint32_t*>(a.scales)[i];
  return reinterpret_cast<const uint16_t*>(a.scales)[i];
}

__device__ __forceinline__ float mv_value(const MatvecArgs& a, uint32_t raw) {
  if (a.qt == kMvMXFP4)  // 2^(raw - 127), 255 is NaN
    return raw == 255u ? __builtin_nanf("") : ldexpf(1.0f, (int)raw - 127);
  if (a.scale_dtype == kF32) return __uint_as_float(raw);
  return a.scale_dtype == kBF16 ? bf16_bits_to_f32(raw)
                                : (float)__builtin_bit_cast(_Float16, (uint16_t)raw);
}

// The raw scales (and zeros) of chunk c of row n: `left` of its k exist.
template <int kKind>
__device__ __forceinline__ MvScales mv_load_scales(const MatvecArgs& a, int n, int c, int left) {
  MvScales r;
  const int per = kMvChunk / a.group;  // 1, 2 or 4
  const int64_t i0 = (int64_t)n * (a.K / a.group) + c * per;
  r.z = 0;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    r.s[g] = 0;
    if (g < per && g * a.group < left) {
      r.s[g] = mv_raw(a, i0 + g);
      if constexpr (kKind == kZeros) r.z |= (uint32_t)a.zeros[i0 + g] << (8 * g);
    }
  }
  return r;
}

// Transposes 4 words x 4 lane rows of 16: lane row q, word s <-> lane row s, word q.
__device__ __forceinline__ void quad_transpose(uint32_t (&d)[4]) {
  auto p = __builtin_amdgcn_permlane32_swap(d[0], d[2], false, false);
  auto q = __builtin_amdgcn_permlane32_swap(d[1], d[3], false, false);
  auto u = __builtin_amdgcn_permlane16_swap(p[0], q[0], false, false);
  auto v = __builtin_amdgcn_permlane16_swap(p[1], q[1], false, false);
  d[0] = u[0], d[1] = u[1], d[2] = v[0], d[3] = v[1];
}

// tot += the products of one chunk of one row tile.
template <int kKind, int kRegs>
__device__ __forceinline__ void mv_chunk(const MatvecArgs& a, const char* lut, uint32_t lane_off,
                                         u32x4 w, const MvScales& sc, const f16x8 (&x)[4],
                                         int left, float (&tot)[kRegs]) {
  uint32_t d[4] = {w.x, w.y, w.z, w.w};
  quad_transpose(d);
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    if (32 * s >= left) break;
    const int g = a.group == 32 ? s : a.group == 64 ? s >> 1 : 0;
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // table address: byte j of the codes in bits 8..15, the lane's slot below
      const uint32_t at =
          __builtin_amdgcn_perm(d[s], lane_off, 0x0c0c0000u | ((4u + j) << 8));
      if constexpr (kKind == kSplit) {
        const u32x2 e = *reinterpret_cast<const u32x2*>(lut + at);
        hi[j] = e.x;
        lo[j] = e.y;
      } else {
        hi[j] = *reinterpret_cast<const uint32_t*>(lut + at);
      }
    }
    if constexpr (kKind == kZeros) {
      const _Float16 z = (_Float16)(float)((sc.z >> (8 * g)) & 0xffu);
      const f16x2 z2 = {z, z};
#pragma unroll
      for (int j = 0; j < 4; ++j) hi[j] = half2_as_u32(u32_as_half2(hi[j]) - z2);
    }
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    const u32x4 h4 = {hi[0], hi[1], hi[2], hi[3]};
    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[s], __builtin_bit_cast(f16x8, h4), acc, 0, 0, 0);
    if constexpr (kKind == kSplit) {
      const u32x4 l4 = {lo[0], lo[1], lo[2], lo[3]};
      acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[s], __builtin_bit_cast(f16x8, l4), acc, 0, 0,
                                                   0);
    }
    const float f = mv_value(a, sc.s[g]);
#pragma unroll
    for (int i = 0; i < kRegs; ++i) tot[i] = fmaf(f, acc[i], tot[i]);
  }
}

// The matrix unit's x operand of step s of chunk c: row m of the 16 is token
// (m / 4) kRegs + m % 4 where m % 4 < kRegs, so that the first kRegs result
// registers of a lane hold all tokens.
template <int kRegs>
__device__ __forceinline__ void mv_load_x(const MatvecArgs& a, int64_t t0, int nt, int c, int left,
                                          int lane, f16x8 (&x)[4]) {
  const int m = lane & 15, q = lane >> 4;
  const int t = (m >> 2) * kRegs + (m & 3);
  const bool live = (m & 3) < kRegs && t < nt;
  const uint16_t* p = reinterpret_cast<const uint16_t*>(a.x) + (t0 + t) * a.K + c * kMvChunk + 8 * q;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    u32x4 v = {0u, 0u, 0u, 0u};
    if (live && 32 * s < left) v = *reinterpret_cast<const u32x4*>(p + 32 * s);
    if (a.x_bf16) {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o[i] = pack_half2((_Float16)bf16_bits_to_f32(w[i] & 0xffffu),
                          (_Float16)bf16_bits_to_f32(w[i] >> 16));
      v = u32x4{o[0], o[1], o[2], o[3]};
    }
    x[s] = __builtin_bit_cast(f16x8, v);
  }
}

// The decode table: 256 byte values x 256 bytes, as 32 copies of two words
// (kSplit) or 64 of one.  Ends with a barrier.
template <int kKind>
__device__ __forceinline__ void mv_fill(const MatvecArgs& a, u32x4* lut, uint32_t* stage, int tid) {
  const float nf4[16] = NF4MOE_LEVELS_INIT;
  const float e2m1[16] = NF4MOE_E2M1_VALUES_INIT;
  if (tid < 16) {
    const float v = kKind == kSplit       ? 256.0f * nf4[tid]
                    : kKind == kZeros     ? (float)tid
                    : a.qt == kMvINT4     ? (float)tid - 8.0f
                                          : e2m1[tid];
    const _Float16 hi = (_Float16)v, lo = (_Float16)(v - (float)hi);
    stage[tid] = pack_half2(hi, lo);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4096 / kMvThreads; ++i) {
    const int u = i * kMvThreads + tid, b = u >> 4;  // 16 16-byte units an entry
    const uint32_t first = stage[a.qt == kMvMXFP4 ? b & 15 : b >> 4];
    const uint32_t second = stage[a.qt == kMvMXFP4 ? b >> 4 : b & 15];
    const uint32_t h = (first & 0xffffu) | (second << 16);
    const uint32_t l = (first >> 16) | (second & 0xffff0000u);
    lut[u] = kKind == kSplit ? u32x4{h, l, h, l} : u32x4{h, h, h, h};
  }
  __syncthreads();
}

}  // namespace

// kCpw: chunks of a wave that stay in registers as x (0: x is read for every
// tile, any K).
template <int kKind, int kRegs, int kCpw>
__global__ __launch_bounds__(kMvThreads) void matvec_kernel(MatvecArgs a) {
  constexpr int kX = kCpw ? kCpw : 1;
  __shared__ u32x4 lut[4096];
  __shared__ float red[2][kMvWaves][kRegs][64];
  __shared__ uint32_t stage[16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t t0 = (int64_t)blockIdx.y * kMvTokens;
  const int nt = a.T - t0 < kMvTokens ? (int)(a.T - t0) : kMvTokens;
  const int chunks = (a.K + kMvChunk - 1) / kMvChunk;
  const int tiles = (a.N + kMvTile - 1) / kMvTile;
  const int q = lane >> 4;
  const uint32_t lane_off = kKind == kSplit ? (lane & 31) * 8 : lane * 4;
  const int64_t row_bytes = a.K / 2;
  const auto left_of = [&](int c) { return a.K - c * kMvChunk; };
  const auto row_of = [&](int tile) {
    const int n = tile * kMvTile + (lane & 15);
    return n < a.N ? n : a.N - 1;
  };
  // 16 packed bytes of chunk c: the lane's 32 codes, or the row's first where the
  // row has ended (x is zero there)
  const auto load_w = [&](int n, int c) {
    const int64_t at = 32 * q < left_of(c) ? c * (kMvChunk / 2) + 16 * q : 0;
    return *reinterpret_cast<const u32x4*>(a.codes + n * row_bytes + at);
  };

  f16x8 x[kX][4];
  u32x4 w[kX];
  MvScales sc[kX];
  int tile = blockIdx.x;
  if constexpr (kCpw > 0) {
    const int n = row_of(tile);
#pragma unroll
    for (int j = 0; j < kX; ++j) {
      const int c = wave + j * kMvWaves;
      if (c >= chunks) break;
      w[j] = load_w(n, c);
      sc[j] = mv_load_scales<kKind>(a, n, c, left_of(c));
      mv_load_x<kRegs>(a, t0, nt, c, left_of(c), lane, x[j]);
    }
  }
  mv_fill<kKind>(a, lut, stage, tid);
  const char* table = reinterpret_cast<const char*>(lut);
  const float last = kKind == kSplit ? 1.0f / 256.0f : 1.0f;

  for (int buf = 0; tile < tiles; tile += gridDim.x, buf ^= 1) {
    float tot[kRegs] = {};
    if constexpr (kCpw > 0) {
      const int next = tile + (int)gridDim.x;
      const int n = row_of(next);
      u32x4 w2[kX];
      MvScales sc2[kX];
#pragma unroll
      for (int j = 0; j < kX; ++j) {
        const int c = wave + j * kMvWaves;
        if (c >= chunks || next >= tiles) break;
        w2[j] = load_w(n, c);
        sc2[j] = mv_load_scales<kKind>(a, n, c, left_of(c));
      }
#pragma unroll
      for (int j = 0; j < kX; ++j) {
        const int c = wave + j * kMvWaves;
        if (c >= chunks) break;
        mv_chunk<kKind, kRegs>(a, table, lane_off, w[j], sc[j], x[j], left_of(c), tot);
      }
#pragma unroll
      for (int j = 0; j < kX; ++j) w[j] = w2[j], sc[j] = sc2[j];
    } else {
      const int n = row_of(tile);
      for (int c = wave; c < chunks; c += kMvWaves) {
        const u32x4 wc = load_w(n, c);
        const MvScales s = mv_load_scales<kKind>(a, n, c, left_of(c));
        mv_load_x<kRegs>(a, t0, nt, c, left_of(c), lane, x[0]);
        mv_chunk<kKind, kRegs>(a, table, lane_off, wc, s, x[0], left_of(c), tot);
      }
    }
#pragma unroll
    for (int i = 0; i < kRegs; ++i) red[buf][wave][i][lane] = tot[i];
    __syncthreads();  // red[buf] is written again two tiles on, after the next barrier
    if (wave < kRegs) {
      float v = 0.f;
#pragma unroll
      for (int u = 0; u < kMvWaves; ++u) v += red[buf][u][wave][lane];
      const int t = q * kRegs + wave, n = tile * kMvTile + (lane & 15);
      if (t < nt && n < a.N) {
        v = (a.qt == kMvFP4 ? v * (1.0f / 6.0f) : v * last) + (a.bias ? a.bias[n] : 0.f);
        const int64_t i = (t0 + t) * a.N + n;
        if (a.y_dtype == kF32) reinterpret_cast<float*>(a.y)[i] = v;
        else if (a.y_dtype == kBF16) reinterpret_cast<uint16_t*>(a.y)[i] = f32_to_bf16_bits(v);
        else reinterpret_cast<_Float16*>(a.y)[i] = (_Float16)v;
      }
    }
  }
}

namespace {

template <int kKind, int kRegs>
void mv_launch(const MatvecArgs& a, dim3 grid, hipStream_t s) {
  const int per = (a.K + kMvChunk * kMvWaves - 1) / (kMvChunk * kMvWaves);
  if (per <= 1)
    hipLaunchKernelGGL((matvec_kernel<kKind, kRegs, 1>), grid, dim3(kMvThreads), 0, s, a);
  else if (per <= 2)
    hipLaunchKernelGGL((matvec_kernel<kKind, kRegs, 2>), grid, dim3(kMvThreads), 0, s, a);
  else if (per <= 4)
    hipLaunchKernelGGL((matvec_kernel<kKind, kRegs, 4>), grid, dim3(kMvThreads), 0, s, a);
  else
    hipLaunchKernelGGL((matvec_kernel<kKind, kRegs, 0>), grid, dim3(kMvThreads), 0, s, a);
}

template <int kKind>
void mv_launch_rows(const MatvecArgs& a, dim3 grid, hipStream_t s) {
  if (a.T <= 4) mv_launch<kKind, 1>(a, grid, s);
  else if (a.T <= 8) mv_launch<kKind, 2>(a, grid, s);
  else mv_launch<kKind, 4>(a, grid, s);
}

}  // namespace

hipError_t launch_matvec(const MatvecArgs& a, int num_cus, hipStream_t s) {
  const unsigned ny = (unsigned)((a.T + kMvTokens - 1) / kMvTokens);
  const int tiles = (a.N + kMvTile - 1) / kMvTile;
  // one workgroup per compute unit, shared by the token blocks; a multiple of 8, so
  // that the blocks of one tile run on the same XCD and share its L2
  int nx = num_cus / (int)ny / 8 * 8;
  if (nx < 8) nx = 8;
  if (nx > tiles) nx = tiles;
  const dim3 grid((unsigned)nx, ny);
  if (a.qt == kMvNF4) mv_launch_rows<kSplit>(a, grid, s);
  else if (a.zeros) mv_launch_rows<kZeros>(a, grid, s);
  else mv_launch_rows<kPlain>(a, grid, s);
  return hipGetLastError();
}

}  // namespace nf4moe
