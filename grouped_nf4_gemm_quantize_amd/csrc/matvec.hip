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

// What a kernel is compiled for: how the table's values are held, and the groups.
enum MvFormat {
  kMvfNF4,      // two fp16 tables, fp32 scales of 64
  kMvfFP4,      // fp32 scales of 64
  kMvfMX,       // e8m0 scales of 32
  kMvfInt32,    // codes minus zeros, scales of 32, 64 or 128 of any float type
  kMvfInt64,
  kMvfInt128
};
constexpr bool mv_split(int f) { return f == kMvfNF4; }
constexpr bool mv_int(int f) { return f >= kMvfInt32; }
// scale groups of a chunk
constexpr int mv_groups(int f) { return f == kMvfMX || f == kMvfInt32 ? 4 : f == kMvfInt128 ? 1 : 2; }

// Raw scales of a chunk's groups (their bits, widened), and zeros, a byte each.
template <int kFmt>
struct MvScales {
  uint32_t s[mv_groups(kFmt)];
  uint32_t z;
};

template <int kFmt>
__device__ __forceinline__ float mv_value(const MatvecArgs& a, uint32_t raw) {
  if constexpr (kFmt == kMvfMX)  // 2^(raw - 127), 255 is NaN
    return __uint_as_float(raw == 0u ? 0x00400000u : raw == 255u ? 0x7fc00000u : raw << 23);
  if (!mv_int(kFmt) || a.scale_dtype == kF32) return __uint_as_float(raw);
  return a.scale_dtype == kBF16 ? bf16_bits_to_f32(raw)
                                : (float)__builtin_bit_cast(_Float16, (uint16_t)raw);
}

// The raw scales (and zeros) of chunk c of row n, 0 for groups beyond the row. Rows of
// whole chunks read a chunk's scales at once.
template <int kFmt>
__device__ __forceinline__ void mv_load_scales(const MatvecArgs& a, int n, int c, bool whole,
                                               MvScales<kFmt>& r) {
  constexpr int kPer = mv_groups(kFmt), kGroup = kMvChunk / kPer;
  const int groups = a.K / kGroup;
  const int64_t i0 = (int64_t)n * groups + c * kPer;
  const bool wide = !mv_int(kFmt) || a.scale_dtype == kF32;
  r.z = 0x08080808u;
  if (whole) {
    if constexpr (kFmt == kMvfMX) {
      uint32_t v;
      __builtin_memcpy(&v, reinterpret_cast<const uint8_t*>(a.scales) + i0, 4);
#pragma unroll
      for (int g = 0; g < kPer; ++g) r.s[g] = (v >> (8 * g)) & 0xffu;
    } else if (wide) {
      __builtin_memcpy(r.s, reinterpret_cast<const uint32_t*>(a.scales) + i0, 4 * kPer);
    } else {
      uint16_t v[kPer];
      __builtin_memcpy(v, reinterpret_cast<const uint16_t*>(a.scales) + i0, 2 * kPer);
#pragma unroll
      for (int g = 0; g < kPer; ++g) r.s[g] = v[g];
    }
    if constexpr (mv_int(kFmt))
      if (a.zeros) __builtin_memcpy(&r.z, a.zeros + i0, kPer);
    return;
  }
#pragma unroll
  for (int g = 0; g < kPer; ++g) {
    const bool in = c * kPer + g < groups;
    const int64_t i = in ? i0 + g : i0;
    uint32_t v;
    if constexpr (kFmt == kMvfMX) v = reinterpret_cast<const uint8_t*>(a.scales)[i];
    else if (wide) v = reinterpret_cast<const uint32_t*>(a.scales)[i];
    else v = reinterpret_cast<const uint16_t*>(a.scales)[i];
    r.s[g] = in ? v : 0u;
    if constexpr (mv_int(kFmt))
      if (a.zeros) r.z = (r.z & ~(0xffu << (8 * g))) | ((uint32_t)a.zeros[i] << (8 * g));
  }
}

// Transposes 4 words x 4 lane rows of 16: lane row q, word s <-> lane row s, word q.
__device__ __forceinline__ void quad_transpose(uint32_t (&d)[4]) {
  auto p = __builtin_amdgcn_permlane32_swap(d[0], d[2], false, false);
  auto q = __builtin_amdgcn_permlane32_swap(d[1], d[3], false, false);
  auto u = __builtin_amdgcn_permlane16_swap(p[0], q[0], false, false);
  auto v = __builtin_amdgcn_permlane16_swap(p[1], q[1], false, false);
  d[0] = u[0], d[1] = u[1], d[2] = v[0], d[3] = v[1];
}

// tot += the products of one chunk of one row tile. Steps beyond the end of the row
// have x = 0 and a scale of 0.
template <int kFmt, int kRegs>
__device__ __forceinline__ void mv_chunk(const MatvecArgs& a, const char* lut, uint32_t lane_off,
                                         u32x4 w, const MvScales<kFmt>& sc, const f16x8 (&x)[4],
                                         float (&tot)[kRegs]) {
  uint32_t d[4] = {w.x, w.y, w.z, w.w};
  quad_transpose(d);
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int g = s * mv_groups(kFmt) / 4;
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // table address: byte j of the codes in bits 8..15, the lane's slot below
      const uint32_t at =
          __builtin_amdgcn_perm(d[s], lane_off, 0x0c0c0000u | ((4u + j) << 8));
      if constexpr (mv_split(kFmt)) {
        const u32x2 e = *reinterpret_cast<const u32x2*>(lut + at);
        hi[j] = e.x;
        lo[j] = e.y;
      } else {
        hi[j] = *reinterpret_cast<const uint32_t*>(lut + at);
      }
    }
    if constexpr (mv_int(kFmt)) {
      const _Float16 z = (_Float16)(float)((sc.z >> (8 * g)) & 0xffu);
      const f16x2 z2 = {z, z};
#pragma unroll
      for (int j = 0; j < 4; ++j) hi[j] = half2_as_u32(u32_as_half2(hi[j]) - z2);
    }
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    const u32x4 h4 = {hi[0], hi[1], hi[2], hi[3]};
    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[s], __builtin_bit_cast(f16x8, h4), acc, 0, 0, 0);
    if constexpr (mv_split(kFmt)) {
      const u32x4 l4 = {lo[0], lo[1], lo[2], lo[3]};
      acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[s], __builtin_bit_cast(f16x8, l4), acc, 0, 0,
                                                   0);
    }
    const float f = mv_value<kFmt>(a, sc.s[g]);
#pragma unroll
    for (int i = 0; i < kRegs; ++i) tot[i] = fmaf(f, acc[i], tot[i]);
  }
}

// The matrix unit's x operand of step s of chunk c: row m of the 16 is token
// (m / 4) kRegs + m % 4 where m % 4 < kRegs, so that the first kRegs result
// registers of a lane hold all tokens.
template <int kRegs>
__device__ __forceinline__ void mv_load_x(const MatvecArgs& a, int64_t t0, int nt, int c, int lane,
                                          f16x8 (&x)[4]) {
  const int left = a.K - c * kMvChunk;
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
// (nf4) or 64 of one.  Ends with a barrier.
template <int kFmt>
__device__ __forceinline__ void mv_fill(u32x4* lut, uint32_t* stage, int tid) {
  const float nf4[16] = NF4MOE_LEVELS_INIT;
  const float e2m1[16] = NF4MOE_E2M1_VALUES_INIT;
  if (tid < 16) {
    const float v = mv_split(kFmt) ? 256.0f * nf4[tid] : mv_int(kFmt) ? (float)tid : e2m1[tid];
    const _Float16 hi = (_Float16)v, lo = (_Float16)(v - (float)hi);
    stage[tid] = pack_half2(hi, lo);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4096 / kMvThreads; ++i) {
    const int u = i * kMvThreads + tid, b = u >> 4;  // 16 16-byte units an entry
    const uint32_t first = stage[kFmt == kMvfMX ? b & 15 : b >> 4];
    const uint32_t second = stage[kFmt == kMvfMX ? b >> 4 : b & 15];
    const uint32_t h = (first & 0xffffu) | (second << 16);
    const uint32_t l = (first >> 16) | (second & 0xffff0000u);
    lut[u] = mv_split(kFmt) ? u32x4{h, l, h, l} : u32x4{h, h, h, h};
  }
  __syncthreads();
}

}  // namespace

// kCpw: chunks of a wave that stay in registers as x (0: x is read for every
// tile, any K).
template <int kFmt, int kRegs, int kCpw>
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
  const bool whole = a.K % kMvChunk == 0;
  const int tiles = (a.N + kMvTile - 1) / kMvTile;
  const int q = lane >> 4;
  const uint32_t lane_off = mv_split(kFmt) ? (lane & 31) * 8 : lane * 4;
  const int64_t row_bytes = a.K / 2;
  const auto row_of = [&](int tile) {
    const int n = tile * kMvTile + (lane & 15);
    return n < a.N ? n : a.N - 1;
  };
  // 16 packed bytes of chunk c: the lane's 32 codes, or the row's first where the
  // row has ended (x is zero there)
  const auto load_w = [&](int n, int c) {
    const int at = c * (kMvChunk / 2) + 16 * q;
    return *reinterpret_cast<const u32x4*>(a.codes + n * row_bytes + (at < row_bytes ? at : 0));
  };

  f16x8 x[kX][4];
  u32x4 w[kX] = {};
  MvScales<kFmt> sc[kX] = {};
  int tile = blockIdx.x;
  const auto load_tile = [&](int tl) {
    const int n = row_of(tl);
#pragma unroll
    for (int j = 0; j < kX; ++j) {
      const int c = wave + j * kMvWaves;
      if (c >= chunks) continue;
      w[j] = load_w(n, c);
      mv_load_scales<kFmt>(a, n, c, whole, sc[j]);
    }
  };
  if constexpr (kCpw > 0) {
    load_tile(tile);
#pragma unroll
    for (int j = 0; j < kX; ++j)
      mv_load_x<kRegs>(a, t0, nt, wave + j * kMvWaves, lane, x[j]);
  }
  mv_fill<kFmt>(lut, stage, tid);
  const char* table = reinterpret_cast<const char*>(lut);
  const float last = mv_split(kFmt) ? 1.0f / 256.0f : kFmt == kMvfFP4 ? 1.0f / 6.0f : 1.0f;

  for (int buf = 0; tile < tiles; tile += gridDim.x, buf ^= 1) {
    float tot[kRegs] = {};
    if constexpr (kCpw > 0) {
      u32x4 w1[kX];
      MvScales<kFmt> sc1[kX];
#pragma unroll
      for (int j = 0; j < kX; ++j) w1[j] = w[j], sc1[j] = sc[j];
      if (tile + (int)gridDim.x < tiles) load_tile(tile + gridDim.x);
#pragma unroll
      for (int j = 0; j < kX; ++j)
        mv_chunk<kFmt, kRegs>(a, table, lane_off, w1[j], sc1[j], x[j], tot);
    } else {
      const int n = row_of(tile);
      for (int c = wave; c < chunks; c += kMvWaves) {
        const u32x4 wc = load_w(n, c);
        MvScales<kFmt> s;
        mv_load_scales<kFmt>(a, n, c, whole, s);
        mv_load_x<kRegs>(a, t0, nt, c, lane, x[0]);
        mv_chunk<kFmt, kRegs>(a, table, lane_off, wc, s, x[0], tot);
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
        v = v * last + (a.bias ? a.bias[n] : 0.f);
        const int64_t i = (t0 + t) * a.N + n;
        if (a.y_dtype == kF32) reinterpret_cast<float*>(a.y)[i] = v;
        else if (a.y_dtype == kBF16) reinterpret_cast<uint16_t*>(a.y)[i] = f32_to_bf16_bits(v);
        else reinterpret_cast<_Float16*>(a.y)[i] = (_Float16)v;
      }
    }
  }
}

namespace {

template <int kFmt, int kRegs>
void mv_launch(const MatvecArgs& a, dim3 grid, hipStream_t s) {
  const int per = (a.K + kMvChunk * kMvWaves - 1) / (kMvChunk * kMvWaves);
  if (per <= 1)
    hipLaunchKernelGGL((matvec_kernel<kFmt, kRegs, 1>), grid, dim3(kMvThreads), 0, s, a);
  else if (per <= 2)
    hipLaunchKernelGGL((matvec_kernel<kFmt, kRegs, 2>), grid, dim3(kMvThreads), 0, s, a);
  else if (per <= 4)
    hipLaunchKernelGGL((matvec_kernel<kFmt, kRegs, 4>), grid, dim3(kMvThreads), 0, s, a);
  else
    hipLaunchKernelGGL((matvec_kernel<kFmt, kRegs, 0>), grid, dim3(kMvThreads), 0, s, a);
}

template <int kFmt>
void mv_launch_rows(const MatvecArgs& a, dim3 grid, hipStream_t s) {
  if (a.T <= 4) mv_launch<kFmt, 1>(a, grid, s);
  else mv_launch<kFmt, 4>(a, grid, s);
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
  if (a.qt == kMvNF4) mv_launch_rows<kMvfNF4>(a, grid, s);
  else if (a.qt == kMvFP4) mv_launch_rows<kMvfFP4>(a, grid, s);
  else if (a.qt == kMvMXFP4) mv_launch_rows<kMvfMX>(a, grid, s);
  else if (a.group == 32) mv_launch_rows<kMvfInt32>(a, grid, s);
  else if (a.group == 64) mv_launch_rows<kMvfInt64>(a, grid, s);
  else mv_launch_rows<kMvfInt128>(a, grid, s);
  return hipGetLastError();
}

}  // namespace nf4moe
