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
// The waves of a workgroup (up to sixteen) share the K axis of 16 output rows (a
// tile) in chunks of 128, chunk c going to wave c % waves.  A lane reads 16 consecutive
// packed bytes (32 codes) of one row; four lane swaps then give each of the chunk's four
// matrix steps 32 consecutive k, all of one scale group, whose sum is scaled in fp32.
// A wave's part of x stays in registers from tile to tile (up to K = 4096), and the
// next tiles' codes are in flight while a tile is computed.  The waves' sums meet in LDS.
// Measured (one MI355X, a call among others): nf4 151936 x 2048, four tokens, fp32 out
// 39.8 us = 4.4 TB/s of codes and scales; int4 28672 x 4096, one token 16.2 us = 3.8 TB/s; below
// some 10 MB launch and first reads set the time (2048 x 2048, one token: 4.9 us in a graph).
//
// Scales and zeros go through LDS too: read by the wave that uses them, a chunk's few
// bytes of 16 rows cost as many cache lines as its codes.  The workgroup reads a round's
// as consecutive elements instead, two steps ahead: when this was changed, int4 28672 x 4096
// in groups of 128, one token, went from 28.7 to 16.5 us (15.9 with no scales read at all).
//
// nf4's levels are no fp16 values: each is held as a sum of two (22 bits),
// scaled by 2^8 so that the small parts stay normal, and multiplied twice.  All
// other formats' values are exact in fp16 (fp4's 1/6 and the 2^-8 are applied to
// the final sum).
// fp4's and MXFP4's values are exact in bf16 too, so bf16 x is multiplied as it is.  For
// nf4 it becomes fp16 (as in the expert stacks): bf16 parts of 22-bit levels would be
// three products.  For int4 as well: code - zero in pairs is an fp16 operation, bf16 has none.

#include "common.h"
#include "launch.h"
#include "matvec_index.h"

namespace nf4moe {

namespace {

constexpr int kMvWaves = 16;    // waves of a workgroup, at most
constexpr int kMvTile = 16;     // output rows of one matrix step
constexpr int kMvTokens = 16;   // rows of x of one matrix step

// What a kernel is compiled for: how the table's values are held, and the groups.
enum MvFormat {
  kMvfNF4,      // two fp16 tables, fp32 scales of 64
  kMvfFP4,      // fp32 scales of 64
  kMvfFP4b,     // the same for bf16 x
  kMvfMX,       // e8m0 scales of 32
  kMvfMXb,      // the same for bf16 x
  kMvfInt32,    // codes minus zeros, scales of 32, 64 or 128 of any float type
  kMvfInt64,
  kMvfInt128
};
constexpr bool mv_split(int f) { return f == kMvfNF4; }
constexpr bool mv_mx(int f) { return f == kMvfMX || f == kMvfMXb; }
constexpr bool mv_bf16(int f) { return f == kMvfFP4b || f == kMvfMXb; }  // products of bf16 values
constexpr bool mv_int(int f) { return f >= kMvfInt32; }
// scale groups of a chunk
constexpr int mv_groups(int f) { return mv_mx(f) || f == kMvfInt32 ? 4 : f == kMvfInt128 ? 1 : 2; }

typedef __amdgpu_buffer_rsrc_t Rsrc;
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ Rsrc mv_rsrc(const void* p, int64_t offset, uint32_t bytes) {
  char* at = const_cast<char*>(reinterpret_cast<const char*>(p)) + offset;
  return __builtin_amdgcn_make_buffer_rsrc(at, 0, (int)bytes, 0x00020000);
}

// Raw scale -> fp32.
template <int kFmt>
__device__ __forceinline__ float mv_scale(uint32_t raw, int dtype) {
  if constexpr (mv_mx(kFmt))  // 2^(raw - 127), 255 is NaN
    return __uint_as_float(raw == 0u ? 0x00400000u : raw == 255u ? 0x7fc00000u : raw << 23);
  if (!mv_int(kFmt) || dtype == kF32) return __uint_as_float(raw);
  return dtype == kBF16 ? bf16_bits_to_f32(raw)
                        : (float)__builtin_bit_cast(_Float16, (uint16_t)raw);
}

// The scales (fp32) and zeros (fp16) of kRows tiles x 16 kX chunks in LDS.
// Rows are kStride words apart: 16 rows of one chunk lie in different banks.
template <int kFmt, int kX, int kRows>
struct MvStage {
  static constexpr int kStride = (16 * kX + 1) * mv_groups(kFmt);
  // elements of a thread: waves * kX chunks of each row over 64 * waves threads
  static constexpr int kReads = (kRows * kMvTile * kX * mv_groups(kFmt) + 63) / 64;
  float s[kRows * kMvTile * kStride];
  _Float16 z[mv_int(kFmt) ? kRows * kMvTile * kStride : 2];
};

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
  u32x4 v[mv_split(kFmt) ? 2 : 1];
};

template <int kFmt>
__device__ __forceinline__ f32x4 mv_mfma(u32x4 x, u32x4 w, f32x4 c) {
  if constexpr (mv_bf16(kFmt))
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x),
                                                   __builtin_bit_cast(bf16x8, w), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, x),
                                                  __builtin_bit_cast(f16x8, w), c, 0, 0, 0);
}

// tot += the products of one chunk of one row tile, whose scales and zeros begin at
// `scales` and `zeros`.  Steps beyond the end of the row have x = 0.
template <int kFmt, int kRegs>
__device__ __forceinline__ void mv_chunk(const char* lut, uint32_t lane_off, u32x4 w,
                                         const float* scales, const _Float16* zeros,
                                         const MvX<kFmt> (&x)[4], float* tot) {
  constexpr int kGroups = mv_groups(kFmt);
  uint32_t d[4] = {w.x, w.y, w.z, w.w};
  quad_transpose(d);
  typedef float Scales __attribute__((ext_vector_type(kGroups == 1 ? 2 : kGroups)));
  typedef _Float16 Zeros __attribute__((ext_vector_type(kGroups == 1 ? 2 : kGroups)));
  float scale[kGroups];
  f16x2 zero[kGroups];
  if constexpr (kGroups == 1) {
    scale[0] = scales[0];
    if constexpr (mv_int(kFmt)) zero[0] = f16x2{zeros[0], zeros[0]};
  } else {
    const Scales v = *reinterpret_cast<const Scales*>(scales);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) scale[g] = v[g];
    if constexpr (mv_int(kFmt)) {
      const Zeros z = *reinterpret_cast<const Zeros*>(zeros);
#pragma unroll
      for (int g = 0; g < kGroups; ++g) zero[g] = f16x2{z[g], z[g]};
    }
  }
  // all table reads first, then the four steps, then their sums: each waits once
  uint32_t hi[4][4], lo[4][4];
#pragma unroll
  for (int s = 0; s < 4; ++s)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // table address: byte j of the codes in bits 8..15, the lane's slot below
      const uint32_t at = __builtin_amdgcn_perm(d[s], lane_off, 0x0c0c0000u | ((4u + j) << 8));
      if constexpr (mv_split(kFmt)) {
        const u32x2 e = *reinterpret_cast<const u32x2*>(lut + at);
        hi[s][j] = e.x;
        lo[s][j] = e.y;
      } else {
        hi[s][j] = *reinterpret_cast<const uint32_t*>(lut + at);
      }
    }
  f32x4 acc[4];
  const f32x4 none = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    if constexpr (mv_split(kFmt)) {
      const u32x4 b0 = {hi[s][0], lo[s][0], hi[s][1], lo[s][1]};
      const u32x4 b1 = {hi[s][2], lo[s][2], hi[s][3], lo[s][3]};
      acc[s] = mv_mfma<kFmt>(x[s].v[0], b0, none);
      acc[s] = mv_mfma<kFmt>(x[s].v[1], b1, acc[s]);
    } else {
      if constexpr (mv_int(kFmt)) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          hi[s][j] = half2_as_u32(u32_as_half2(hi[s][j]) - zero[s * kGroups / 4]);
      }
      acc[s] = mv_mfma<kFmt>(x[s].v[0], u32x4{hi[s][0], hi[s][1], hi[s][2], hi[s][3]}, none);
    }
  }
#pragma unroll
  for (int s = 0; s < 4; ++s)
#pragma unroll
    for (int i = 0; i < kRegs; ++i)
      tot[i] = fmaf(scale[s * kGroups / 4], acc[s][i], tot[i]);
}

// The matrix unit's x operand of step s of chunk c as it is read (zero beyond the row
// or the tokens): row m of the 16 is token (m / 4) kRegs + m % 4 where m % 4 < kRegs,
// so that the first kRegs result registers of a lane hold all tokens.
template <int kRegs>
__device__ __forceinline__ void mv_read_x(const MatvecArgs& a, int64_t t0, int nt, int c, int lane,
                                          u32x4 (&v)[4]) {
  const int left = a.K - c * kMvChunk;
  const int m = lane & 15, q = lane >> 4;
  const int t = (m >> 2) * kRegs + (m & 3);
  const bool live = (m & 3) < kRegs && t < nt;
  // beyond the end the offset is out of the buffer's bounds, and the read gives 0
  const Rsrc r = mv_rsrc(a.x, t0 * a.K * 2, (uint32_t)(nt * a.K * 2));
  const int at = (t * a.K + c * kMvChunk + 8 * q) * 2;
#pragma unroll
  for (int s = 0; s < 4; ++s)
    v[s] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                         r, live && 32 * s < left ? at + 64 * s : 0x7ffffff0, 0, 0));
}

template <int kFmt>
__device__ __forceinline__ void mv_set_x(const MatvecArgs& a, const u32x4 (&raw)[4],
                                         MvX<kFmt> (&x)[4]) {
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    u32x4 v = raw[s];
    if (!mv_bf16(kFmt) && a.x_bf16) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = pack_half2((_Float16)bf16_bits_to_f32(v[i] & 0xffffu),
                          (_Float16)bf16_bits_to_f32(v[i] >> 16));
    }
    if constexpr (mv_split(kFmt)) {
      x[s].v[0] = u32x4{v.x, v.x, v.y, v.y};
      x[s].v[1] = u32x4{v.z, v.z, v.w, v.w};
    } else {
      x[s].v[0] = v;
    }
  }
}

// The decode table: 256 byte values x 256 bytes, as 32 copies of two words
// (nf4) or 64 of one.  A barrier has to follow.
template <int kFmt>
__device__ __forceinline__ void mv_fill(u32x4* lut, uint32_t* stage, int tid) {
  const float nf4[16] = NF4MOE_LEVELS_INIT;
  const float e2m1[16] = NF4MOE_E2M1_VALUES_INIT;
  if (tid < 16) {
    // selected from literals: a read of the levels would wait for the codes' reads
    // issued before it
    float v = (float)tid;
    if constexpr (!mv_int(kFmt)) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (tid == i) v = mv_split(kFmt) ? 256.0f * nf4[i] : e2m1[i];
    }
    const _Float16 hi = (_Float16)v, lo = (_Float16)(v - (float)hi);
    stage[tid] = mv_bf16(kFmt) ? f32_to_bf16_bits(v) : pack_half2(hi, lo);
  }
  __syncthreads();
  for (int u = tid; u < 4096; u += blockDim.x) {
    const int b = u >> 4;  // 16 16-byte units an entry
    const uint32_t first = stage[mv_mx(kFmt) ? b & 15 : b >> 4];
    const uint32_t second = stage[mv_mx(kFmt) ? b >> 4 : b & 15];
    const uint32_t h = (first & 0xffffu) | (second << 16);
    const uint32_t l = (first >> 16) | (second & 0xffff0000u);
    lut[u] = mv_split(kFmt) ? u32x4{h, l, h, l} : u32x4{h, h, h, h};
  }
}

}  // namespace

// kRegs: result registers of a lane (1: up to 4 tokens, 4: up to 16).  kCpw: chunks of a
// wave whose x stays in registers (0: any number, x is read with the codes).  kRows:
// tiles of a round.  A round is one step, or (kCpw 0) one for every 16 chunks.
template <int kFmt, int kRegs, int kCpw, int kRows>
__global__ __launch_bounds__(64 * kMvWaves) void matvec_kernel(MatvecArgs a) {
  constexpr int kX = kCpw ? kCpw : 1;
  constexpr int kOut = kRows * kRegs;  // result registers of a lane in a round
  constexpr int kGroups = mv_groups(kFmt);
  typedef MvStage<kFmt, kX, kRows> Stage;
  __shared__ u32x4 lut[4096];
  __shared__ float red[2][kMvWaves][kOut][64];
  __shared__ __attribute__((aligned(16))) Stage stage[2];
  __shared__ uint32_t levels[16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), waves = blockDim.x >> 6;
  const int64_t t0 = (int64_t)blockIdx.y * kMvTokens;
  const int nt = a.T - t0 < kMvTokens ? (int)(a.T - t0) : kMvTokens;
  const int chunks = (a.K + kMvChunk - 1) / kMvChunk;
  const int tiles = (a.N + kMvTile - 1) / kMvTile;
  const int n_lane = lane & 15, q = lane >> 4;
  const uint32_t lane_off = mv_split(kFmt) ? (lane & 31) * 8 : lane * 4;
  const int row_bytes = a.K / 2;
  const int groups = a.K / (kMvChunk / kGroups);
  const int size = mv_mx(kFmt) ? 1 : !mv_int(kFmt) || a.scale_dtype == kF32 ? 4 : 2;
  const uint8_t* zeros = a.zeros ? a.zeros : a.codes;  // read but not used
  const int lane_row = n_lane * row_bytes;
  const int panels = kCpw ? 1 : (chunks + kMvWaves - 1) / kMvWaves;
  const int grid_step = gridDim.x * kRows;

  // chunk j of this wave in a panel; a wave without one repeats the last with x = 0
  const auto chunk_of = [&](int panel, int j) {
    const int c = panel * kMvWaves + wave + j * waves;
    return c < chunks ? c : chunks - 1;
  };
  // The rows of a round as buffers: reads beyond N return 0 without touching memory.
  const auto rows_of = [&](int tile) {
    const int64_t left = a.N - (int64_t)tile * kMvTile;
    return (uint32_t)(left < 0 ? 0 : left < kMvTile * kRows ? left : kMvTile * kRows);
  };
  // codes of a step.  The whole offset is in the vector operand: the record count bounds
  // that one, a scalar offset may be added after the check.
  u32x4 w[kRows][kX];
  const auto load_w = [&](int tile, int panel, int u, int j) {
    const Rsrc r = mv_rsrc(a.codes, (int64_t)tile * kMvTile * row_bytes, rows_of(tile) * row_bytes);
    const int at = lane_row + mv_code_byte(chunk_of(panel, j), q, row_bytes);
    w[u][j] = __builtin_bit_cast(
        u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at + u * kMvTile * row_bytes, 0, 0));
  };
  // scales and zeros of a step, element i of the workgroup: raw, then into LDS.  Beyond
  // the end of a row its last scale is read (x is zero there).
  uint32_t raw_s[Stage::kReads], raw_z[Stage::kReads];
  const int seg = waves * kX * kGroups;                    // scales of a row
  const uint32_t magic = ((1u << 20) + seg - 1) / seg;     // i / seg = i * magic >> 20, exact
  const int stage_count = kRows * kMvTile * seg;           // for i up to 64 seg <= 2^13
  const auto load_stage = [&](int tile, int panel) {
    const int64_t first = (int64_t)tile * kMvTile * groups;
    const uint32_t count = rows_of(tile) * groups;
    const Rsrc rs = mv_rsrc(a.scales, first * size, count * size);
    const Rsrc rz = mv_rsrc(zeros, first, count);
#pragma unroll
    for (int k = 0; k < Stage::kReads; ++k) {
      const int i = tid + k * blockDim.x, row = (int)(i * magic >> 20);
      const int g = panel * kMvWaves * kGroups + i - row * seg;
      const int at = row * groups + (g < groups ? g : groups - 1);
      if (mv_mx(kFmt)) raw_s[k] = __builtin_amdgcn_raw_buffer_load_b8(rs, at, 0, 0);
      else if (size == 4) raw_s[k] = __builtin_amdgcn_raw_buffer_load_b32(rs, at * 4, 0, 0);
      else raw_s[k] = __builtin_amdgcn_raw_buffer_load_b16(rs, at * 2, 0, 0);
      if constexpr (mv_int(kFmt)) raw_z[k] = __builtin_amdgcn_raw_buffer_load_b8(rz, at, 0, 0);
    }
  };
  const auto put_stage = [&](Stage& to) {
#pragma unroll
    for (int k = 0; k < Stage::kReads; ++k) {
      const int i = tid + k * blockDim.x, row = (int)(i * magic >> 20);
      if (i >= stage_count) break;
      const int at = row * Stage::kStride + i - row * seg;
      to.s[at] = mv_scale<kFmt>(raw_s[k], a.scale_dtype);
      if constexpr (mv_int(kFmt)) to.z[at] = (_Float16)(float)(a.zeros ? raw_z[k] : 8u);
    }
  };

  // the step after (tile, panel)
  const auto after = [&](int& tile, int& panel) {
    const bool end = ++panel == panels;
    if (end) panel = 0, tile += grid_step;
    return end;
  };

  int tile = blockIdx.x * kRows, panel = 0;
  int next_tile = tile, next_panel = panel;  // of the codes in flight
  // x and the first steps' reads are in flight while the table is made
  u32x4 raw_x[kX][4];
  load_stage(tile, 0);
#pragma unroll
  for (int j = 0; j < kX; ++j) mv_read_x<kRegs>(a, t0, nt, wave + j * waves, lane, raw_x[j]);
#pragma unroll
  for (int j = 0; j < kX; ++j)
#pragma unroll
    for (int u = 0; u < kRows; ++u) load_w(tile, 0, u, j);
  mv_fill<kFmt>(lut, levels, tid);
  put_stage(stage[0]);
  after(next_tile, next_panel);
  load_stage(next_tile, next_panel);
  __syncthreads();
  MvX<kFmt> x[kX][4];
#pragma unroll
  for (int j = 0; j < kCpw; ++j) mv_set_x<kFmt>(a, raw_x[j], x[j]);
  const char* table = reinterpret_cast<const char*>(lut);
  const float last = mv_split(kFmt) ? 1.0f / 256.0f : kFmt == kMvfFP4 || kFmt == kMvfFP4b ? 1.0f / 6.0f : 1.0f;

  float tot[kOut] = {};
  for (int buf = 0, out = 0; tile < tiles; buf ^= 1) {
    // the next step's codes, and the scales of the one after it, are in flight
    // during this step
    const bool end = panel + 1 == panels;
    int ahead_tile = next_tile, ahead_panel = next_panel;
    after(ahead_tile, ahead_panel);
    put_stage(stage[buf ^ 1]);
    load_stage(ahead_tile, ahead_panel);
    const Stage& now = stage[buf];
    if constexpr (kCpw > 0) {
#pragma unroll
      for (int j = 0; j < kX; ++j)
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          const u32x4 w1 = w[u][j];
          load_w(next_tile, 0, u, j);
          const int at = (u * kMvTile + n_lane) * Stage::kStride + (wave + j * waves) * kGroups;
          mv_chunk<kFmt, kRegs>(table, lane_off, w1, now.s + at, now.z + at, x[j], tot + u * kRegs);
        }
    } else {
      mv_set_x<kFmt>(a, raw_x[0], x[0]);
      mv_read_x<kRegs>(a, t0, nt, next_panel * kMvWaves + wave, lane, raw_x[0]);
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const u32x4 w1 = w[u][0];
        load_w(next_tile, next_panel, u, 0);
        const int at = (u * kMvTile + n_lane) * Stage::kStride + wave * kGroups;
        mv_chunk<kFmt, kRegs>(table, lane_off, w1, now.s + at, now.z + at, x[0], tot + u * kRegs);
      }
    }
    if (end) {
#pragma unroll
      for (int i = 0; i < kOut; ++i) red[out][wave][i][lane] = tot[i], tot[i] = 0.f;
    }
    // orders this step's LDS writes before their readers, and its reads of stage[buf] before
    // the next step's writes; red[out] is written again two rounds on
    __syncthreads();
    if (end) {
      for (int i = wave; i < kOut; i += waves) {
        float v = 0.f;
        for (int u = 0; u < waves; ++u) v += red[out][u][i][lane];
        const int t = q * kRegs + i % kRegs;
        const int64_t n = (int64_t)(tile + i / kRegs) * kMvTile + n_lane;
        if (t < nt && n < a.N) {
          v = v * last + (a.bias ? a.bias[n] : 0.f);
          const int64_t at = (t0 + t) * a.N + n;
          if (a.y_dtype == kF32) reinterpret_cast<float*>(a.y)[at] = v;
          else if (a.y_dtype == kBF16) reinterpret_cast<uint16_t*>(a.y)[at] = f32_to_bf16_bits(v);
          else reinterpret_cast<_Float16*>(a.y)[at] = (_Float16)v;
        }
      }
      out ^= 1;
    }
    tile = next_tile, panel = next_panel;
    next_tile = ahead_tile, next_panel = ahead_panel;
  }
}

namespace {

template <int kFmt, int kRegs, int kCpw, int kRows>
void mv_go(const MatvecArgs& a, int nx, unsigned ny, int waves, hipStream_t s) {
  const int rounds = ((a.N + kMvTile - 1) / kMvTile + kRows - 1) / kRows;
  hipLaunchKernelGGL((matvec_kernel<kFmt, kRegs, kCpw, kRows>),
                     dim3((unsigned)(nx < rounds ? nx : rounds), ny), dim3(64 * waves), 0, s, a);
}

template <int kFmt, int kRegs>
void mv_launch(const MatvecArgs& a, int cus, hipStream_t s) {
  const unsigned ny = (unsigned)((a.T + kMvTokens - 1) / kMvTokens);
  const int tiles = (a.N + kMvTile - 1) / kMvTile;
  // one workgroup per compute unit, shared by the token blocks; a multiple of 8, so
  // that the blocks of one tile run on the same XCD and share its L2
  int nx = cus / (int)ny / 8 * 8;
  if (nx < 8) nx = 8;
  const int chunks = (a.K + kMvChunk - 1) / kMvChunk;
  const int per = (chunks + kMvWaves - 1) / kMvWaves;
  // as few waves as take the chunks in as many turns
  const int waves = (chunks + per - 1) / per;
  // Tiles of a round: several save barriers and reads of x and cost balance between
  // workgroups; sixteen tokens' sums leave LDS for two.  us for one and several, in a graph:
  //   up to 4 tokens, K 2048, one | four    nf4           MXFP4         int4 (128)
  //     N 4096                              5.1 | 7.5     4.8 | 7.3     5.5 | 7.7
  //     N 24576                             11.8 | 13.3   11.5 | 12.7   12.7 | 11.9
  //     N 32768                             14.6 | 13.9   14.1 | 13.4   15.6 | 12.1
  //     N 65536                             24.6 | 20.7   24.5 | 19.8   27.1 | 17.9
  //   (int4 in groups of 32: N 24576 12.0 | 13.6, 32768 14.6 | 14.0)
  //   16 tokens, K 2048, one | two: N 4096  6.4 | 7.2     6.1 | 7.1     6.5 | 7.4
  //     N 8192                              8.0 | 7.3     7.6 | 7.2     7.8 | 7.5
  //   64 tokens, K 2048, N 16384            27.6 | 21.9   27.6 | 22.6   27.4 | 21.6
  //   one token, K 8192, one | two | four   nf4                  MXFP4
  //     N 4096                              10.0 | 12.5 | 17.9   8.8 | 11.6 | 17.3
  //     N 8192                              16.6 | 14.7 | 19.9   15.4 | 14.1 | 19.5
  //     N 16384                             28.3 | 23.4 | 23.0   26.2 | 22.4 | 22.7
  //     N 32768                             52.6 | 41.8 | 38.9   47.9 | 39.6 | 37.4
  //   16 tokens, K 8192, one | two: N 4096  13.5 | 15.8   13.5 | 15.6
  //     N 8192                              24.1 | 18.1   23.2 | 17.2
  // Where a wave has two chunks of K they were even (int4, K 4096, N 28672 17.0 | 16.9).
  constexpr int kMany = kRegs == 1 ? 4 : 2;
  if (per == 1 && tiles >= (kRegs == 1 ? 8 : 2) * nx)
    mv_go<kFmt, kRegs, 1, kMany>(a, nx, ny, waves, s);
  else if (per == 1) mv_go<kFmt, kRegs, 1, 1>(a, nx, ny, waves, s);
  else if (per == 2) mv_go<kFmt, kRegs, 2, 1>(a, nx, ny, waves, s);
  else if (tiles >= kMany * nx) mv_go<kFmt, kRegs, 0, kMany>(a, nx, ny, kMvWaves, s);
  else if (kRegs == 1 && tiles >= 2 * nx) mv_go<kFmt, kRegs, 0, 2>(a, nx, ny, kMvWaves, s);
  else mv_go<kFmt, kRegs, 0, 1>(a, nx, ny, kMvWaves, s);
}

template <int kFmt>
void mv_launch_format(const MatvecArgs& a, int cus, hipStream_t s) {
  // results of up to four tokens are one register a lane: fewer sums, and more tiles a round (one
  // register | four, nf4: one token 4096x2048 5.0 | 5.5 us, four 65536x2048 21.0 | 24.1,
  // 32768x8192 40.0 | 46.3; MXFP4 and int4 alike)
  if (a.T <= 4) mv_launch<kFmt, 1>(a, cus, s);
  else mv_launch<kFmt, 4>(a, cus, s);
}

}  // namespace

hipError_t launch_matvec(const MatvecArgs& a, int num_cus, hipStream_t s) {
  if (a.qt == kMvNF4) mv_launch_format<kMvfNF4>(a, num_cus, s);
  else if (a.qt == kMvFP4 && a.x_bf16) mv_launch_format<kMvfFP4b>(a, num_cus, s);
  else if (a.qt == kMvFP4) mv_launch_format<kMvfFP4>(a, num_cus, s);
  else if (a.qt == kMvMXFP4 && a.x_bf16) mv_launch_format<kMvfMXb>(a, num_cus, s);
  else if (a.qt == kMvMXFP4) mv_launch_format<kMvfMX>(a, num_cus, s);
  else if (a.group == 32) mv_launch_format<kMvfInt32>(a, num_cus, s);
  else if (a.group == 64) mv_launch_format<kMvfInt64>(a, num_cus, s);
  else mv_launch_format<kMvfInt128>(a, num_cus, s);
  return hipGetLastError();
}

}  // namespace nf4moe
