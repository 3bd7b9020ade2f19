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

constexpr int kMvThreads = 1024;
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

typedef __amdgpu_buffer_rsrc_t Rsrc;

// The rows of a tile as a buffer: reads beyond its end return 0 without
// touching memory, which covers rows beyond N and tiles beyond the last.
__device__ __forceinline__ Rsrc mv_rsrc(const void* p, int64_t offset, int64_t bytes) {
  char* at = const_cast<char*>(reinterpret_cast<const char*>(p)) + offset;
  return __builtin_amdgcn_make_buffer_rsrc(at, 0, bytes > 0 ? (int)bytes : 0, 0x00020000);
}

// Raw scales of a chunk's groups as they are read, and zeros, a byte each.  Nothing is
// computed on them before they are used, so that a read can stay in flight.
template <int kFmt, bool kWhole>
struct MvScales {
  static constexpr int kPer = mv_groups(kFmt);
  uint32_t s[kPer];  // kWhole: packed as in memory
  uint32_t z[kPer];  // kWhole: all in z[0]
};

// What a lane needs of a tile's scales: byte offsets of its row.
struct MvScaleRow {
  int size;  // bytes of a scale
  int s, z;  // offset of the row's first scale, and first zero
  int groups;
};

template <int kFmt, bool kWhole>
__device__ __forceinline__ void mv_load_scales(Rsrc rs, Rsrc rz, const MvScaleRow& row, int c,
                                               MvScales<kFmt, kWhole>& r) {
  constexpr int kPer = mv_groups(kFmt);
  if constexpr (kWhole) {
    const int at = row.s + c * kPer * row.size;
    if constexpr (kFmt == kMvfMX) {
      r.s[0] = __builtin_amdgcn_raw_buffer_load_b32(rs, at, 0, 0);
    } else if constexpr (!mv_int(kFmt)) {
      const auto v = __builtin_amdgcn_raw_buffer_load_b64(rs, at, 0, 0);
      r.s[0] = v[0], r.s[1] = v[1];
    } else if (row.size == 4) {
      if constexpr (kPer == 4) {
        const auto v = __builtin_amdgcn_raw_buffer_load_b128(rs, at, 0, 0);
        r.s[0] = v[0], r.s[1] = v[1], r.s[2] = v[2], r.s[3] = v[3];
      } else if constexpr (kPer == 2) {
        const auto v = __builtin_amdgcn_raw_buffer_load_b64(rs, at, 0, 0);
        r.s[0] = v[0], r.s[1] = v[1];
      } else {
        r.s[0] = __builtin_amdgcn_raw_buffer_load_b32(rs, at, 0, 0);
      }
    } else {
      if constexpr (kPer == 4) {
        const auto v = __builtin_amdgcn_raw_buffer_load_b64(rs, at, 0, 0);
        r.s[0] = v[0], r.s[1] = v[1];
      } else if constexpr (kPer == 2) {
        r.s[0] = __builtin_amdgcn_raw_buffer_load_b32(rs, at, 0, 0);
      } else {
        r.s[0] = __builtin_amdgcn_raw_buffer_load_b16(rs, at, 0, 0);
      }
    }
    if constexpr (mv_int(kFmt)) {
      const int zat = row.z + c * kPer;
      if constexpr (kPer == 4) r.z[0] = __builtin_amdgcn_raw_buffer_load_b32(rz, zat, 0, 0);
      else if constexpr (kPer == 2) r.z[0] = __builtin_amdgcn_raw_buffer_load_b16(rz, zat, 0, 0);
      else r.z[0] = __builtin_amdgcn_raw_buffer_load_b8(rz, zat, 0, 0);
    }
  } else {
#pragma unroll
    for (int g = 0; g < kPer; ++g) {
      // groups beyond the row (x is zero there) read its last one
      const int i = c * kPer + g < row.groups ? c * kPer + g : row.groups - 1;
      const int at = row.s + i * row.size;
      if constexpr (kFmt == kMvfMX)
        r.s[g] = __builtin_amdgcn_raw_buffer_load_b8(rs, at, 0, 0);
      else if (!mv_int(kFmt) || row.size == 4)
        r.s[g] = __builtin_amdgcn_raw_buffer_load_b32(rs, at, 0, 0);
      else
        r.s[g] = __builtin_amdgcn_raw_buffer_load_b16(rs, at, 0, 0);
      if constexpr (mv_int(kFmt)) r.z[g] = __builtin_amdgcn_raw_buffer_load_b8(rz, row.z + i, 0, 0);
    }
  }
}

// Scale g of a chunk as fp32.
template <int kFmt, bool kWhole>
__device__ __forceinline__ float mv_scale(const MvScales<kFmt, kWhole>& r, int g, int dtype) {
  if constexpr (kFmt == kMvfMX) {  // 2^(raw - 127), 255 is NaN
    const uint32_t raw = kWhole ? (r.s[0] >> (8 * g)) & 0xffu : r.s[g];
    return __uint_as_float(raw == 0u ? 0x00400000u : raw == 255u ? 0x7fc00000u : raw << 23);
  }
  if (!mv_int(kFmt) || dtype == kF32) return __uint_as_float(r.s[g]);
  const uint32_t raw = kWhole ? (r.s[g >> 1] >> (16 * (g & 1))) & 0xffffu : r.s[g];
  return dtype == kBF16 ? bf16_bits_to_f32(raw)
                        : (float)__builtin_bit_cast(_Float16, (uint16_t)raw);
}

// Transposes 4 words x 4 lane rows of 16: lane row q, word s <-> lane row s, word q.
__device__ __forceinline__ void quad_transpose(uint32_t (&d)[4]) {
  auto p = __builtin_amdgcn_permlane32_swap(d[0], d[2], false, false);
  auto q = __builtin_amdgcn_permlane32_swap(d[1], d[3], false, false);
  auto u = __builtin_amdgcn_permlane16_swap(p[0], q[0], false, false);
  auto v = __builtin_amdgcn_permlane16_swap(p[1], q[1], false, false);
  d[0] = u[0], d[1] = u[1], d[2] = v[0], d[3] = v[1];
}

// x of one matrix step: for nf4 each pair of values twice, against the two words of
// a table entry as they are read.
template <int kFmt>
struct MvX {
  f16x8 v[mv_split(kFmt) ? 2 : 1];
};

// tot += the products of one chunk of one row tile.  Steps beyond the end of the row
// have x = 0.
template <int kFmt, bool kWhole, int kRegs>
__device__ __forceinline__ void mv_chunk(const MatvecArgs& a, const char* lut, uint32_t lane_off,
                                         u32x4 w, const MvScales<kFmt, kWhole>& sc,
                                         const MvX<kFmt> (&x)[4], float* tot) {
  uint32_t d[4] = {w.x, w.y, w.z, w.w};
  quad_transpose(d);
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int g = s * mv_groups(kFmt) / 4;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    uint32_t at[4];
    // table address: byte j of the codes in bits 8..15, the lane's slot below
#pragma unroll
    for (int j = 0; j < 4; ++j)
      at[j] = __builtin_amdgcn_perm(d[s], lane_off, 0x0c0c0000u | ((4u + j) << 8));
    if constexpr (mv_split(kFmt)) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const u32x2 e = *reinterpret_cast<const u32x2*>(lut + at[2 * h]);
        const u32x2 f = *reinterpret_cast<const u32x2*>(lut + at[2 * h + 1]);
        const u32x4 b = {e.x, e.y, f.x, f.y};
        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[s].v[h], __builtin_bit_cast(f16x8, b), acc,
                                                     0, 0, 0);
      }
    } else {
      uint32_t b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const uint32_t*>(lut + at[j]);
      if constexpr (mv_int(kFmt)) {
        const uint32_t raw = kWhole ? (sc.z[0] >> (8 * g)) & 0xffu : sc.z[g];
        const _Float16 z = (_Float16)(float)(a.zeros ? raw : 8u);
        const f16x2 z2 = {z, z};
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = half2_as_u32(u32_as_half2(b[j]) - z2);
      }
      const u32x4 b4 = {b[0], b[1], b[2], b[3]};
      acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[s].v[0], __builtin_bit_cast(f16x8, b4), acc, 0,
                                                   0, 0);
    }
    const float f = mv_scale<kFmt, kWhole>(sc, g, a.scale_dtype);
#pragma unroll
    for (int i = 0; i < kRegs; ++i) tot[i] = fmaf(f, acc[i], tot[i]);
  }
}

// The matrix unit's x operand of step s of chunk c: row m of the 16 is token
// (m / 4) kRegs + m % 4 where m % 4 < kRegs, so that the first kRegs result
// registers of a lane hold all tokens.
template <int kFmt, int kRegs>
__device__ __forceinline__ void mv_load_x(const MatvecArgs& a, int64_t t0, int nt, int c, int lane,
                                          MvX<kFmt> (&x)[4]) {
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
    if constexpr (mv_split(kFmt)) {
      x[s].v[0] = __builtin_bit_cast(f16x8, (u32x4{v.x, v.x, v.y, v.y}));
      x[s].v[1] = __builtin_bit_cast(f16x8, (u32x4{v.z, v.z, v.w, v.w}));
    } else {
      x[s].v[0] = __builtin_bit_cast(f16x8, v);
    }
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

// kWhole: rows are whole chunks and a chunk's scales one aligned read.  kRegs:
// result registers of a lane (1: up to 4 tokens, 4: up to 16).  kCpw: chunks of a wave
// whose x stays in registers (0: x is read again for every kRows tiles, any K).
// kRows: tiles between two barriers.
template <int kFmt, bool kWhole, int kRegs, int kCpw, int kRows>
__global__ __launch_bounds__(kMvThreads) void matvec_kernel(MatvecArgs a) {
  constexpr int kX = kCpw ? kCpw : 1;
  constexpr int kOut = kRows * kRegs;  // result registers of a lane between barriers
  __shared__ u32x4 lut[4096];
  __shared__ float red[2][kMvWaves][kOut][64];
  __shared__ uint32_t stage[16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t t0 = (int64_t)blockIdx.y * kMvTokens;
  const int nt = a.T - t0 < kMvTokens ? (int)(a.T - t0) : kMvTokens;
  const int chunks = (a.K + kMvChunk - 1) / kMvChunk;
  const int tiles = (a.N + kMvTile - 1) / kMvTile;
  const int n_lane = lane & 15, q = lane >> 4;
  const uint32_t lane_off = mv_split(kFmt) ? (lane & 31) * 8 : lane * 4;
  const int row_bytes = a.K / 2;
  MvScaleRow sr;
  sr.groups = a.K / (kMvChunk / mv_groups(kFmt));
  sr.size = kFmt == kMvfMX ? 1 : !mv_int(kFmt) || a.scale_dtype == kF32 ? 4 : 2;
  sr.s = n_lane * sr.groups * sr.size;
  sr.z = n_lane * sr.groups;
  const uint8_t* zeros = a.zeros ? a.zeros : a.codes;  // read but not used

  MvX<kFmt> x[kX][4];
  u32x4 w[kRows][kX];
  MvScales<kFmt, kWhole> sc[kRows][kX];
  const int lane_w = n_lane * row_bytes + 16 * q;

  // reads chunk c of row tile `tile` (all zeros beyond the last tile)
  const auto load = [&](int tile, int c, u32x4& wo, MvScales<kFmt, kWhole>& so) {
    const int64_t n0 = (int64_t)tile * kMvTile;
    const int64_t rows = a.N - n0 < kMvTile ? a.N - n0 : kMvTile;
    const Rsrc rw = mv_rsrc(a.codes, n0 * row_bytes, rows * row_bytes);
    const Rsrc rs = mv_rsrc(a.scales, n0 * sr.groups * sr.size, rows * sr.groups * sr.size);
    const Rsrc rz = mv_rsrc(zeros, n0 * sr.groups, rows * sr.groups);
    wo = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                       rw, lane_w, c * (kMvChunk / 2), 0));
    mv_load_scales<kFmt, kWhole>(rs, rz, sr, c, so);
  };
  const auto chunk_of = [&](int j) {
    // a wave without a j-th chunk repeats the last one with x = 0
    const int c = wave + j * kMvWaves;
    return c < chunks ? c : chunks - 1;
  };

  int tile = blockIdx.x * kRows;
  if constexpr (kCpw > 0) {
#pragma unroll
    for (int j = 0; j < kX; ++j)
#pragma unroll
      for (int u = 0; u < kRows; ++u) load(tile + u, chunk_of(j), w[u][j], sc[u][j]);
#pragma unroll
    for (int j = 0; j < kX; ++j)
      mv_load_x<kFmt, kRegs>(a, t0, nt, wave + j * kMvWaves, lane, x[j]);
  }
  mv_fill<kFmt>(lut, stage, tid);
  const char* table = reinterpret_cast<const char*>(lut);
  const float last = mv_split(kFmt) ? 1.0f / 256.0f : kFmt == kMvfFP4 ? 1.0f / 6.0f : 1.0f;
  const int step = gridDim.x * kRows;

  for (int buf = 0; tile < tiles; tile += step, buf ^= 1) {
    float tot[kOut] = {};
    if constexpr (kCpw > 0) {
#pragma unroll
      for (int j = 0; j < kX; ++j)
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          const u32x4 w1 = w[u][j];
          const MvScales<kFmt, kWhole> s1 = sc[u][j];
          load(tile + step + u, chunk_of(j), w[u][j], sc[u][j]);
          mv_chunk<kFmt, kWhole, kRegs>(a, table, lane_off, w1, s1, x[j], tot + u * kRegs);
        }
    } else {
      for (int c = wave; c < chunks; c += kMvWaves) {
#pragma unroll
        for (int u = 0; u < kRows; ++u) load(tile + u, c, w[u][0], sc[u][0]);
        mv_load_x<kFmt, kRegs>(a, t0, nt, c, lane, x[0]);
#pragma unroll
        for (int u = 0; u < kRows; ++u)
          mv_chunk<kFmt, kWhole, kRegs>(a, table, lane_off, w[u][0], sc[u][0], x[0],
                                        tot + u * kRegs);
      }
    }
#pragma unroll
    for (int i = 0; i < kOut; ++i) red[buf][wave][i][lane] = tot[i];
    __syncthreads();  // red[buf] is written again two rounds on, after the next barrier
    if (wave < kOut) {
      float v = 0.f;
#pragma unroll
      for (int u = 0; u < kMvWaves; ++u) v += red[buf][u][wave][lane];
      const int t = q * kRegs + wave % kRegs;
      const int64_t n = (int64_t)(tile + wave / kRegs) * kMvTile + n_lane;
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

template <int kFmt, bool kWhole, int kRegs, int kCpw, int kRows>
void mv_go(const MatvecArgs& a, int nx, unsigned ny, hipStream_t s) {
  hipLaunchKernelGGL((matvec_kernel<kFmt, kWhole, kRegs, kCpw, kRows>), dim3((unsigned)nx, ny),
                     dim3(kMvThreads), 0, s, a);
}

template <int kFmt, bool kWhole, int kRegs>
void mv_launch(const MatvecArgs& a, int cus, hipStream_t s) {
  constexpr int kMany = kRegs == 1 ? 4 : 2;
  const unsigned ny = (unsigned)((a.T + kMvTokens - 1) / kMvTokens);
  const int tiles = (a.N + kMvTile - 1) / kMvTile;
  // one workgroup per compute unit, shared by the token blocks; a multiple of 8, so
  // that the blocks of one tile run on the same XCD and share its L2
  int nx = cus / (int)ny / 8 * 8;
  if (nx < 8) nx = 8;
  const bool many = tiles >= 2 * kMany * nx;
  const int rounds = many ? (tiles + kMany - 1) / kMany : tiles;
  if (nx > rounds) nx = rounds;
  const int per = (a.K + kMvChunk * kMvWaves - 1) / (kMvChunk * kMvWaves);
  if (per <= 1 && many) mv_go<kFmt, kWhole, kRegs, 1, kMany>(a, nx, ny, s);
  else if (per <= 1) mv_go<kFmt, kWhole, kRegs, 1, 1>(a, nx, ny, s);
  else if (per <= 2) mv_go<kFmt, kWhole, kRegs, 2, 1>(a, nx, ny, s);
  else if (many) mv_go<kFmt, kWhole, kRegs, 0, kMany>(a, nx, ny, s);
  else mv_go<kFmt, kWhole, kRegs, 0, 1>(a, nx, ny, s);
}

template <int kFmt>
void mv_launch_format(const MatvecArgs& a, int cus, hipStream_t s) {
  constexpr int kPer = mv_groups(kFmt);
  const int size = kFmt == kMvfMX ? 1 : !mv_int(kFmt) || a.scale_dtype == kF32 ? 4 : 2;
  const int read = kPer * size < 4 ? kPer * size : 4;
  const bool whole = a.K % kMvChunk == 0 && (uintptr_t)a.scales % read == 0 &&
                     (uintptr_t)a.zeros % kPer == 0;
  if (whole && a.T <= 4) mv_launch<kFmt, true, 1>(a, cus, s);
  else if (whole) mv_launch<kFmt, true, 4>(a, cus, s);
  else if (a.T <= 4) mv_launch<kFmt, false, 1>(a, cus, s);
  else mv_launch<kFmt, false, 4>(a, cus, s);
}

}  // namespace

hipError_t launch_matvec(const MatvecArgs& a, int num_cus, hipStream_t s) {
  if (a.qt == kMvNF4) mv_launch_format<kMvfNF4>(a, num_cus, s);
  else if (a.qt == kMvFP4) mv_launch_format<kMvfFP4>(a, num_cus, s);
  else if (a.qt == kMvMXFP4) mv_launch_format<kMvfMX>(a, num_cus, s);
  else if (a.group == 32) mv_launch_format<kMvfInt32>(a, num_cus, s);
  else if (a.group == 64) mv_launch_format<kMvfInt64>(a, num_cus, s);
  else mv_launch_format<kMvfInt128>(a, num_cus, s);
  return hipGetLastError();
}

}  // namespace nf4moe
