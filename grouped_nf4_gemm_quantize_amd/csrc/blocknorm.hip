// RMS norms after and before a block, fused with the block's gate and residual
// scale, and their gradients (block_norm_forward / block_norm_backward):
//   z = y * rstd(y) * (w_post + off),  r = beta * residual + alpha * gate * z,
//   h = r * rstd(r) * (w_pre + off),   rstd(v) = 1 / sqrt(mean(v^2) + eps).
//
// Bound by memory: every matrix is read once (twice by the backward beyond 8192 columns)
// and written once.  The waves of a row hold it in registers, eight consecutive columns a
// lane (sixteen beyond 8192 columns): few registers, so that sixteen waves and their reads
// are in flight on a compute unit.  A row has a wave at least: at 128 columns 48 of 64 lanes
// have none (65536 x 128 bf16 39 us forward and 62 backward, against 13 and 19 for the bytes).  All of a row's reads are issued together, before any of them is
// converted; they go through buffer bounds, so that columns and rows beyond the end
// need no branch between them.  r is rounded to its type before it is normalised, so
// h follows from what is stored.
//
// Measured at 4096 x 2048, bf16, both norms and a token gate: 15.4 us = 4.4 TB/s.  With
// branches between the reads (types and bounds decided by each) it took 31 us.
//
// The backward's sums over T stay in registers over a workgroup's rows, are added over
// its waves in LDS and go to one partial row a workgroup; a second kernel adds
// the partial rows.  The same case: 28 us = 3.6 TB/s of the 12 bytes an element (24 us
// and 4 us; the partial sums add 8 MB to 101).

#include "common.h"
#include "launch.h"

namespace nf4moe {

namespace {

constexpr int kNormWaves = 8;      // waves of a workgroup of several rows, forward
constexpr int kNormBwdWaves = 16;  // and backward: fewer partial rows
constexpr int kNormMaxWaves = 16;  // waves of a workgroup of one row
constexpr int kNormPartials = 256; // partial rows of the weight gradients, at most

typedef __amdgpu_buffer_rsrc_t Rsrc;

// Eight consecutive elements as they are read; kBytes is an element's size.
template <int kBytes>
struct Raw8 {
  u32x4 v[kBytes / 2];
};

// `bytes` bytes at p: reads beyond them return 0, writes are dropped.
__device__ __forceinline__ Rsrc span_of(const void* p, int64_t offset, int bytes) {
  char* at = const_cast<char*>(reinterpret_cast<const char*>(p)) + offset;
  return __builtin_amdgcn_make_buffer_rsrc(at, 0, bytes, 0x00020000);
}

__device__ __forceinline__ u32x4 read16(Rsrc r, int offset) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, offset, 0, 0));
}

template <int kBytes>
__device__ __forceinline__ void fetch8(Rsrc r, int col, Raw8<kBytes>& o) {
  o.v[0] = read16(r, col * kBytes);
  if constexpr (kBytes == 4) o.v[1] = read16(r, col * 4 + 16);
}

// Weights of either size: the second half of 16-bit ones is read beyond the end.
__device__ __forceinline__ void fetch8_any(Rsrc r, int size, int col, Raw8<4>& o) {
  o.v[0] = read16(r, col * size);
  o.v[1] = read16(r, size == 4 ? col * 4 + 16 : 0x7ffffff0);
}

template <int kBytes>
__device__ __forceinline__ void widen8(const Raw8<kBytes>& r, int dtype, float (&v)[8]) {
  if (kBytes == 4 && dtype == kF32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r.v[kBytes / 2 * i / 8][i & 3]);
  } else if (dtype == kBF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(r.v[0][i] << 16);
      v[2 * i + 1] = __uint_as_float(r.v[0][i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f16x2 h = u32_as_half2(r.v[0][i]);
      v[2 * i] = (float)h.x;
      v[2 * i + 1] = (float)h.y;
    }
  }
}

// Rounds v to dtype, stores it and leaves the stored values in v.
__device__ __forceinline__ void write8(Rsrc r, int dtype, int col, float (&v)[8]) {
  u32x4 q;
  if (dtype == kF32) {
    const u32x4 a = {__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                     __float_as_uint(v[3])};
    const u32x4 b = {__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]),
                     __float_as_uint(v[7])};
    __builtin_amdgcn_raw_buffer_store_b128(a, r, col * 4, 0, 0);
    __builtin_amdgcn_raw_buffer_store_b128(b, r, col * 4 + 16, 0, 0);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (dtype == kBF16) {
      const uint32_t a = f32_to_bf16_bits(v[2 * i]), b = f32_to_bf16_bits(v[2 * i + 1]);
      q[i] = a | (b << 16);
      v[2 * i] = bf16_bits_to_f32(a);
      v[2 * i + 1] = bf16_bits_to_f32(b);
    } else {
      const _Float16 a = (_Float16)v[2 * i], b = (_Float16)v[2 * i + 1];
      q[i] = pack_half2(a, b);
      v[2 * i] = (float)a;
      v[2 * i + 1] = (float)b;
    }
  }
  __builtin_amdgcn_raw_buffer_store_b128(q, r, col * 2, 0, 0);
}

// How the waves of a workgroup share rows: kRowWaves waves a row in workgroups of kAll;
// or five to eight waves a row (0), as many rows as kAll has eights; or all waves of
// a workgroup of up to 16 (-1).
template <int kRowWaves>
constexpr int norm_waves(int all) {
  return kRowWaves >= 0 ? all : kNormMaxWaves;
}

template <int kRowWaves, int kAll>
struct NormShape {
  static constexpr int kRows = kRowWaves > 0 ? kAll / kRowWaves : kRowWaves ? 1 : kAll / 8;
  static constexpr int kWaves = norm_waves<kRowWaves>(kAll);
  int lane, sub, part, row_waves;  // sub: row of the workgroup; part: wave of the row
  __device__ NormShape() {
    lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    row_waves = kRowWaves > 0 ? kRowWaves : (blockDim.x >> 6) / kRows;
    sub = kRowWaves > 0 ? wave / row_waves : kRows > 1 && wave >= row_waves;
    part = wave - sub * row_waves;
  }
  __device__ int col(int u) const { return ((u * row_waves + part) * 64 + lane) * 8; }
};

// Sums of kN values over the waves of a row, in every lane.  A barrier has to come
// between two uses of `red`.
template <int kN, int kRowWaves, int kAll>
__device__ __forceinline__ void row_sum(float (&v)[kN], float (*red)[kNormMaxWaves],
                                        const NormShape<kRowWaves, kAll>& at) {
#pragma unroll
  for (int i = 0; i < kN; ++i) v[i] = wave_sum(v[i]);
  if constexpr (kRowWaves != 1) {
    const int first = at.sub * at.row_waves;
    if (at.lane == 0)
#pragma unroll
      for (int i = 0; i < kN; ++i) red[i][first + at.part] = v[i];
    __syncthreads();
    if constexpr (kRowWaves > 0) {
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        v[i] = red[i][first];
#pragma unroll
        for (int w = 1; w < kRowWaves; ++w) v[i] += red[i][first + w];
      }
    } else {
      // lane l of each 16 takes wave l's sum: one read for any number of waves
      const int w = at.lane & 15;
      const bool in = w < at.row_waves;
#pragma unroll
      for (int i = 0; i < kN; ++i) v[i] = in ? red[i][first + w] : 0.f;
#pragma unroll
      for (int i = 0; i < kN; ++i) v[i] = row16_sum(v[i]);
    }
  }
}

// 1 / sqrt(mean + eps), correctly rounded operations
__device__ __forceinline__ float rstd_of(float sum, int H, float eps) {
  return 1.0f / sqrtf(sum / (float)H + eps);
}

}  // namespace

// kRes, kY: element sizes of the residual and of y (2 where there is none).
template <int kRes, int kY, int kVec, int kRowWaves>
__global__ __launch_bounds__(64 * norm_waves<kRowWaves>(kNormWaves), kVec == 1 ? 8 : 4) void
block_norm_kernel(BlockNormArgs a) {
  const NormShape<kRowWaves, kNormWaves> at;
  __shared__ float red[2][1][kNormMaxWaves];
  constexpr int kRows = at.kRows;
  const int ws = a.w_dtype == kF32 ? 4 : 2;
  const Rsrc r_pre = span_of(a.w_pre, 0, a.w_pre ? a.H * ws : 0);
  const Rsrc r_post = span_of(a.w_post, 0, a.w_post ? a.H * ws : 0);
  const Rsrc r_gate = span_of(a.gate, 0, a.gate_axis == 2 ? a.H * 4 : 0);
  const int hs = a.h_dtype == kF32 ? 4 : 2;
  for (int64_t first = (int64_t)blockIdx.x * kRows; first < a.T;
       first += (int64_t)gridDim.x * kRows) {
    // the waves of a row beyond the last take part in the barriers only
    const int64_t t = first + at.sub;
    const bool live = t < a.T;
    const int n = live ? a.H : 0;
    const int64_t row = live ? t * a.H : 0;
    const Rsrc r_res = span_of(a.residual, row * kRes, n * kRes);
    const Rsrc r_y = span_of(a.y, row * kY, a.y ? n * kY : 0);
    Raw8<kRes> r0[kVec];
    Raw8<kY> y0[kVec];
    Raw8<4> w0[kVec], w1[kVec], g0[kVec];
#pragma unroll
    for (int u = 0; u < kVec; ++u) {
      fetch8<kY>(r_y, at.col(u), y0[u]);
      fetch8<kRes>(r_res, at.col(u), r0[u]);
    }
#pragma unroll
    for (int u = 0; u < kVec; ++u) {
      fetch8_any(r_post, ws, at.col(u), w0[u]);
      fetch8_any(r_pre, ws, at.col(u), w1[u]);
      if (a.gate_axis == 2) fetch8<4>(r_gate, at.col(u), g0[u]);
    }
    float gt = a.alpha;
    if (a.gate_axis == 1 && live) gt *= a.gate[t];
    float r[kVec][8], z[kVec][8], wv[8];
#pragma unroll
    for (int u = 0; u < kVec; ++u) {
      widen8<kRes>(r0[u], a.res_dtype, r[u]);
      widen8<kY>(y0[u], a.y_dtype, z[u]);
    }
    if (a.y) {
      float rstd = 1.f;
      if (a.w_post) {
        float s[1] = {0.f};
#pragma unroll
        for (int u = 0; u < kVec; ++u)
#pragma unroll
          for (int i = 0; i < 8; ++i) s[0] += z[u][i] * z[u][i];
        row_sum<1>(s, red[0], at);
        rstd = rstd_of(s[0], a.H, a.eps);
      }
      const Rsrc r_out = span_of(a.r_out, row * kRes, n * kRes);
#pragma unroll
      for (int u = 0; u < kVec; ++u) {
        if (a.w_post) {
          widen8<4>(w0[u], a.w_dtype, wv);
#pragma unroll
          for (int i = 0; i < 8; ++i) z[u][i] *= rstd * (wv[i] + a.w_offset);
        }
        if (a.gate_axis == 2) {
          widen8<4>(g0[u], kF32, wv);
#pragma unroll
          for (int i = 0; i < 8; ++i) z[u][i] *= wv[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) r[u][i] = a.beta * r[u][i] + gt * z[u][i];
        write8(r_out, a.res_dtype, at.col(u), r[u]);
      }
    }
    if (a.w_pre) {
      float s[1] = {0.f};
#pragma unroll
      for (int u = 0; u < kVec; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0] += r[u][i] * r[u][i];
      row_sum<1>(s, red[1], at);
      const float rstd = rstd_of(s[0], a.H, a.eps);
      const Rsrc r_h = span_of(a.h, row * hs, n * hs);
#pragma unroll
      for (int u = 0; u < kVec; ++u) {
        widen8<4>(w1[u], a.w_dtype, wv);
#pragma unroll
        for (int i = 0; i < 8; ++i) r[u][i] = r[u][i] * rstd * (wv[i] + a.w_offset);
        write8(r_h, a.h_dtype, at.col(u), r[u]);
      }
    }
    if constexpr (kRowWaves != 1) __syncthreads();  // `red` is written again for the next row
  }
}

// A lane's part of one row's matrices as they are read.
template <int kRes, int kY, int kDh>
struct NormRow {
  Raw8<kRes> r, d;
  Raw8<kY> y;
  Raw8<kDh> h;
};

__device__ __forceinline__ f32x4 four(const float (&v)[8], int half) {
  return f32x4{v[4 * half], v[4 * half + 1], v[4 * half + 2], v[4 * half + 3]};
}

// A lane's weights, with the offset; without w_post z is y: weight 1.
struct NormCols {
  float pre[8], post[8], gate[8];
};

// Waves of a backward's workgroup: sixteen, or eight for one row of five to eight waves with
// fp32 residual and a channel gate, which need more than 128 registers.  us of one row | two, in a
// graph: y fp32 1531 x 2888 27.1 | 31.8, 4096 x 2560 46.3 | 53.2, 2048 x 4096 39.6 | 48.6;
// y bf16 1531 x 2888 28.4 | 28.7, 4096 x 2560 55.8 | 50.4, 4096 x 3584 57.2 | 63.0, 2048 x 4096
// 35.3 | 43.3.  bf16 without a gate, 4096 x 2880: 51 | 38.
template <int kRes, int kRowWaves, bool kGate>
constexpr int norm_bwd_waves() {
  return kRowWaves == 0 && kRes == 4 && kGate ? 8 : kNormBwdWaves;
}

// A workgroup takes rows in turn with the others; its sums over them of the column
// gradients go to row blockIdx.x of the partial sums (dw_pre, dw_post, dgate by
// channel).  kDh: element size of dh (2 where there is none).
// All sums of a row are taken at once: with dr = d + rstd_r dh w_pre - k_r r and
// q = gate w_post y, sum dr q = sum d q + rstd_r sum dh w_pre q - k_r sum r q.
//
// Registers: sixteen waves have 128 a lane, and a spill among the next row's reads waits for
// them.  With eight columns a lane (kVec 1, kHold) the next row's reads are in flight and the
// weights stay in registers; in LDS with a channel gate or fp32 rows of four waves or more
// (kKeep; 2048 x 5120 fp32, channel gate 87 | 62 us).  With sixteen columns, values and
// sums alone fill the registers: the row and its weights are read again after the
// row's sums, and two column sums are held in LDS (275 x 8536 fp16, channel gate 85 | 33 us, 53 x
// 13808 fp32 55 | 23).  The second reading is not all from L2: 512 x 16384 bf16 fetches 1.7 times
// the matrices' bytes, 2.6 times with a channel gate.
// Spills are fewer than without this, not gone: 38 of the 96 kernels have some.  Up to 8192
// columns 8 to 40 bytes a lane, all but one with a channel gate; beyond, 20 to 36 bytes, 92 to
// 116 with a channel gate; 16-bit rows without one have none up to 8192.
template <int kRes, int kY, int kDh, int kVec, int kRowWaves, bool kGate>
__global__ __launch_bounds__(
    64 * norm_waves<kRowWaves>((norm_bwd_waves<kRes, kRowWaves, kGate>())),
    ((norm_bwd_waves<kRes, kRowWaves, kGate>()) == 8 ? 3 : 4)) void
block_norm_bwd_kernel(BlockNormArgs a) {
  constexpr int kAll = norm_bwd_waves<kRes, kRowWaves, kGate>();
  const NormShape<kRowWaves, kAll> at;
  constexpr int kRows = at.kRows, kCols = kVec * (kRowWaves > 0 ? kRowWaves : 8) * 512;
  constexpr bool kHold = kVec == 1;
  constexpr bool kKeep = kHold && kAll == kNormBwdWaves &&
                         (kGate || (kRes == 4 && (kRowWaves == 4 || kRowWaves == 0)));
  __shared__ float red[2][6][kNormMaxWaves];
  // partial sums of the waves that share columns
  __shared__ f32x4 all[kRows > 1 ? kRows / 2 : 1][kRows > 1 ? kCols / 4 : 1];
  const int ws = a.w_dtype == kF32 ? 4 : 2;
  const Rsrc r_pre = span_of(a.w_pre, 0, a.w_pre ? a.H * ws : 0);
  const Rsrc r_post = span_of(a.w_post, 0, a.w_post ? a.H * ws : 0);
  const Rsrc r_gate = span_of(a.gate, 0, kGate ? a.H * 4 : 0);
  typedef NormRow<kRes, kY, kDh> Row;
  // a column the compiler cannot know, where it would otherwise keep what is to be read again
  const auto col_of = [&](int u) {
    int col = at.col(u);
    if constexpr (!kHold) asm volatile("" : "+v"(col));
    return col;
  };
  const auto read = [&](int64_t t, int u, Row& o) {
    const bool live = t < a.T;
    const int n = live ? a.H : 0, col = col_of(u);
    const int64_t row = live ? t * a.H : 0;
    fetch8<kRes>(span_of(a.residual, row * kRes, a.w_pre ? n * kRes : 0), col, o.r);
    fetch8<kDh>(span_of(a.dh, row * kDh, a.dh ? n * kDh : 0), col, o.h);
    fetch8<kY>(span_of(a.y, row * kY, a.y ? n * kY : 0), col, o.y);
    fetch8<kRes>(span_of(a.d_r_out, row * kRes, a.d_r_out ? n * kRes : 0), col, o.d);
  };
  const auto gate_of = [&](int64_t t) { return a.gate_axis == 1 && t < a.T ? a.gate[t] : 1.f; };
  const auto columns = [&](int u, NormCols& w) {
    Raw8<4> p, q, g;
    const int col = col_of(u);
    fetch8_any(r_pre, ws, col, p);
    fetch8_any(r_post, ws, col, q);
    if constexpr (kGate) fetch8<4>(r_gate, col, g);
    widen8<4>(p, a.w_dtype, w.pre);
    widen8<4>(q, a.w_dtype, w.post);
    if constexpr (kGate) widen8<4>(g, kF32, w.gate);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w.pre[i] += a.w_offset;
      w.post[i] = a.w_post ? w.post[i] + a.w_offset : 1.f;
    }
  };
  float r[8], d[8], y[8], g[8];
  const auto widen = [&](const Row& o) {
    widen8<kRes>(o.r, a.res_dtype, r);
    widen8<kDh>(o.h, a.h_dtype, g);
    widen8<kY>(o.y, a.y_dtype, y);
    widen8<kRes>(o.d, a.res_dtype, d);
  };
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t t = (int64_t)blockIdx.x * kRows + at.sub;
  Row next;
  float next_gate = gate_of(t);
  NormCols w;
  // the weights in LDS, in the lane's own places, where they do not fit the registers
  __shared__ f32x4 kept[3][2][kKeep ? 64 * kNormMaxWaves : 1];
  const auto kept_columns = [&]() {
    int at = threadIdx.x;
    asm volatile("" : "+v"(at));  // read here, not before the loop
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w.pre[e] = kept[0][e >> 2][at][e & 3];
      w.post[e] = kept[1][e >> 2][at][e & 3];
      if constexpr (kGate) w.gate[e] = kept[2][e >> 2][at][e & 3];
    }
  };
  if constexpr (kHold) {
    read(t, 0, next);
    columns(0, w);
  }
  if constexpr (kKeep) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      kept[0][e][threadIdx.x] = four(w.pre, e);
      kept[1][e][threadIdx.x] = four(w.post, e);
      if constexpr (kGate) kept[2][e][threadIdx.x] = four(w.gate, e);
    }
  }
  // sums of the column gradients; of long rows the last two in LDS, in the lane's own places
  float s_pre[kVec][8] = {}, s_post[8] = {}, s_gate[8] = {};
  __shared__ f32x4 mine[kGate ? 2 : 1][kVec][2][kHold ? 1 : 64 * kNormMaxWaves];
  const auto add_mine = [&](int which, int u, const float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 2; ++e) mine[which][u][e][threadIdx.x] += four(v, e);
  };
  if constexpr (!kHold) {
    const f32x4 none = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 2 * kVec; ++k) {
      mine[0][k >> 1][k & 1][threadIdx.x] = none;
      if constexpr (kGate) mine[1][k >> 1][k & 1][threadIdx.x] = none;
    }
  }
  const float inv_h = 1.0f / (float)a.H;
  // waves whose row is beyond the last (t >= T) take part in the barriers only
  for (int buf = 0; t - at.sub < a.T; t += step, buf ^= 1) {
    const bool live = t < a.T;
    const int n = live ? a.H : 0;
    const int64_t row = live ? t * a.H : 0;
    const float gt = a.alpha * next_gate;
    if constexpr (kHold) {
      widen(next);
      read(t + step, 0, next);
    }
    next_gate = gate_of(t + step);
    // r^2, dh w r, y^2; d q, dh w q, r q
    float s[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < kVec; ++u) {
      if constexpr (!kHold) {
        __builtin_amdgcn_sched_barrier(0);  // one u's values at a time
        read(t, u, next);
        columns(u, w);
        widen(next);
      }
      if constexpr (kKeep) kept_columns();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float hw = g[i] * w.pre[i];
        const float q = (kGate ? w.gate[i] * w.post[i] : w.post[i]) * y[i];
        s[0] += r[i] * r[i];
        s[1] += hw * r[i];
        s[2] += y[i] * y[i];
        s[3] += d[i] * q;
        s[4] += hw * q;
        s[5] += r[i] * q;
      }
    }
    row_sum<6>(s, red[buf], at);
    // without w_pre (or a row) r and dh are zero here, and so is all they give.  The third
    // power of a small row's rstd can pass fp32's range, its products with the sums do not.
    const float rstd_r = a.w_pre && live ? rstd_of(s[0], a.H, a.eps) : 0.f;
    const float k_r = rstd_r * (rstd_r * (rstd_r * (s[1] * inv_h)));
    const float rstd_y = !a.w_post ? 1.f : live ? rstd_of(s[2], a.H, a.eps) : 0.f;
    const float dr_q = s[3] + rstd_r * s[4] - k_r * s[5];
    if (a.gate_axis == 1 && live && at.part == 0 && at.lane == 0)
      a.dgate[t] = a.alpha * rstd_y * dr_q;
    const float k_y = a.w_post ? rstd_y * (rstd_y * (rstd_y * (gt * dr_q * inv_h))) : 0.f;
    const Rsrc r_out = span_of(a.r_out, row * kRes, n * kRes);
    const Rsrc r_dy = span_of(a.h, row * kY, a.y ? n * kY : 0);
#pragma unroll
    for (int u = 0; u < kVec; ++u) {
      if constexpr (!kHold) {
        __builtin_amdgcn_sched_barrier(0);  // one u's values at a time
        read(t, u, next);
        columns(u, w);
        widen(next);
      }
      if constexpr (kKeep) kept_columns();
      float post[8], gate[8];  // this row's part of the sums
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s_pre[u][i] += g[i] * r[i] * rstd_r;
        // d becomes dr, r dresidual
        d[i] += rstd_r * g[i] * w.pre[i] - r[i] * k_r;
        r[i] = a.beta * d[i];
        // g becomes the gradient dz of z, then dy
        g[i] = gt * d[i];
        const float yn = y[i] * rstd_y;
        if constexpr (kGate) {
          gate[i] = a.alpha * d[i] * (yn * w.post[i]);
          g[i] *= w.gate[i];
        }
        post[i] = g[i] * yn;
        g[i] = rstd_y * (g[i] * w.post[i]) - y[i] * k_y;
      }
      if constexpr (kHold) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          s_post[i] += post[i];
          if constexpr (kGate) s_gate[i] += gate[i];
        }
      } else {
        add_mine(0, u, post);
        if constexpr (kGate) add_mine(1, u, gate);
      }
      write8(r_out, a.res_dtype, at.col(u), r);
      write8(r_dy, a.y_dtype, at.col(u), g);
    }
  }
  // the sums of waves that share columns, in halves: the upper half hands over
  const auto join = [&](float (&v)[kVec][8]) {
#pragma unroll
    for (int half = kRows / 2; half > 0; half /= 2) {
      __syncthreads();
      if (at.sub >= half && at.sub < 2 * half)
#pragma unroll
        for (int u = 0; u < kVec; ++u) {
          f32x4* o = &all[at.sub - half][at.col(u) / 4];
          o[0] = f32x4{v[u][0], v[u][1], v[u][2], v[u][3]};
          o[1] = f32x4{v[u][4], v[u][5], v[u][6], v[u][7]};
        }
      __syncthreads();
      if (at.sub < half)
#pragma unroll
        for (int u = 0; u < kVec; ++u) {
          const f32x4 *o = &all[at.sub][at.col(u) / 4], p = o[0], q = o[1];
#pragma unroll
          for (int i = 0; i < 4; ++i) v[u][i] += p[i], v[u][4 + i] += q[i];
        }
    }
  };
  const auto put = [&](float (&v)[kVec][8], int p) {
    join(v);
    const int64_t row = ((int64_t)p * gridDim.x + blockIdx.x) * a.H;
    const Rsrc r_part = span_of(a.part, row * 4, at.sub == 0 ? a.H * 4 : 0);
#pragma unroll
    for (int u = 0; u < kVec; ++u) write8(r_part, kF32, at.col(u), v[u]);
  };
  if (a.w_pre) put(s_pre, 0);
#pragma unroll
  for (int p = 1; p < (kGate ? 3 : 2); ++p) {
#pragma unroll
    for (int u = 0; u < kVec; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (kHold) s_pre[u][i] = p == 1 ? s_post[i] : s_gate[i];
        else s_pre[u][i] = mine[p - 1][u][i >> 2][threadIdx.x][i & 3];
      }
    if (p == 2 || a.w_post) put(s_pre, p);
  }
}

// out[c] = sum over the partial rows: 16 lanes of four columns, the 16 x 4 row
// classes of a workgroup each in order, then joined in order.
__global__ __launch_bounds__(1024) void block_norm_reduce_kernel(BlockNormArgs a, int groups) {
  __shared__ f32x4 red[64][16];
  const int plane = blockIdx.y;
  float* out = plane == 0 ? a.dw_pre : plane == 1 ? a.dw_post : a.dgate;
  if (plane == 0 ? !a.w_pre : plane == 1 ? !a.w_post : a.gate_axis != 2) return;
  const int q = threadIdx.x & 15, k = threadIdx.x >> 4;
  const int c = (blockIdx.x * 16 + q) * 4;
  const float* p = a.part + (int64_t)plane * groups * a.H + c;
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  if (c < a.H)
    for (int i = k; i < groups; i += 64) s += *reinterpret_cast<const f32x4*>(p + (int64_t)i * a.H);
  red[k][q] = s;
  __syncthreads();
  if (threadIdx.x < 64) {
    // thread (column lane, word) of the 64 columns
    const int col = blockIdx.x * 64 + threadIdx.x;
    float v = 0.f;
    for (int i = 0; i < 64; ++i) v += red[i][threadIdx.x >> 2][threadIdx.x & 3];
    if (col < a.H) out[col] = v;
  }
}

namespace {

// Waves of a row, eight columns a lane: 1, 2 and 4 in workgroups of kNormWaves (backward
// kNormBwdWaves, which takes two rows of 5 to 8 as well), more in one of their own; sixteen
// columns a lane where they would be more than sixteen.
int norm_row_waves(int H) {
  const int vec = H > 512 * kNormMaxWaves ? 2 : 1;
  const int w = (H + 512 * vec - 1) / (512 * vec);
  return w == 3 ? 4 : w;
}

template <int kRes, int kY, int kDh, int kVec, int kRowWaves, bool kGate>
void norm_bwd_go(const BlockNormArgs& a, int groups, hipStream_t s) {
  constexpr int kAll = norm_bwd_waves<kRes, kRowWaves, kGate>();
  constexpr int kRows = NormShape<kRowWaves, kAll>::kRows;
  const dim3 block(64 * (kRowWaves > 0 ? kAll : norm_row_waves(a.H) * kRows));
  hipLaunchKernelGGL((block_norm_bwd_kernel<kRes, kY, kDh, kVec, kRowWaves, kGate>), dim3(groups),
                     block, 0, s, a);
}

template <int kRes, int kY, int kDh, int kVec, int kRowWaves>
void norm_bwd_gate(const BlockNormArgs& a, int groups, hipStream_t s) {
  if (a.gate_axis == 2) norm_bwd_go<kRes, kY, kDh, kVec, kRowWaves, true>(a, groups, s);
  else norm_bwd_go<kRes, kY, kDh, kVec, kRowWaves, false>(a, groups, s);
}

template <int kRes, int kY, int kVec, int kRowWaves>
void norm_go(const BlockNormArgs& a, int bwd_groups, hipStream_t s) {
  if (bwd_groups) {
    if (a.dh && a.h_dtype == kF32) norm_bwd_gate<kRes, kY, 4, kVec, kRowWaves>(a, bwd_groups, s);
    else norm_bwd_gate<kRes, kY, 2, kVec, kRowWaves>(a, bwd_groups, s);
    return;
  }
  const dim3 block(64 * (kRowWaves > 0 ? kNormWaves : norm_row_waves(a.H)));
  constexpr int kRows = NormShape<kRowWaves, kNormWaves>::kRows;
  const int64_t rounds = (a.T + kRows - 1) / kRows;
  hipLaunchKernelGGL((block_norm_kernel<kRes, kY, kVec, kRowWaves>),
                     dim3((unsigned)(rounds < (1 << 20) ? rounds : (1 << 20))), block, 0, s, a);
}

template <int kRes, int kY>
void norm_sizes(const BlockNormArgs& a, int bwd_groups, hipStream_t s) {
  switch (norm_row_waves(a.H)) {
    case 1: return norm_go<kRes, kY, 1, 1>(a, bwd_groups, s);
    case 2: return norm_go<kRes, kY, 1, 2>(a, bwd_groups, s);
    case 4: return norm_go<kRes, kY, 1, 4>(a, bwd_groups, s);
  }
  if (a.H <= 512 * kNormMaxWaves / 2) norm_go<kRes, kY, 1, 0>(a, bwd_groups, s);
  else if (a.H <= 512 * kNormMaxWaves) norm_go<kRes, kY, 1, -1>(a, bwd_groups, s);
  else norm_go<kRes, kY, 2, -1>(a, bwd_groups, s);
}

void norm_launch(const BlockNormArgs& a, int bwd_groups, hipStream_t s) {
  const bool wide_y = a.y && a.y_dtype == kF32;
  if (a.res_dtype == kF32 && wide_y) norm_sizes<4, 4>(a, bwd_groups, s);
  else if (a.res_dtype == kF32) norm_sizes<4, 2>(a, bwd_groups, s);
  else if (wide_y) norm_sizes<2, 4>(a, bwd_groups, s);
  else norm_sizes<2, 2>(a, bwd_groups, s);
}

}  // namespace

// One workgroup a compute unit: with two of six waves for 1531 x 2888 the partial rows cost more
// than the waves gained (31 us, one 26.5).  Counted for workgroups of sixteen waves; fewer
// rows at a time take more turns.  Not the device's count: the workspace's size
// follows from it, and is asked for without a device.
int block_norm_groups(int64_t T, int H) {
  const int waves = norm_row_waves(H);
  const int64_t rows = waves <= 4 ? kNormBwdWaves / waves : waves <= 8 ? 2 : 1;
  const int64_t rounds = (T + rows - 1) / rows;
  // as few as finish in as many turns: fewer partial rows (275 x 8536 39 | 33 us)
  const int64_t turns = (rounds + kNormPartials - 1) / kNormPartials;
  return (int)((rounds + turns - 1) / turns);
}

hipError_t launch_block_norm(const BlockNormArgs& a, hipStream_t s) {
  norm_launch(a, 0, s);
  return hipGetLastError();
}

hipError_t launch_block_norm_bwd(const BlockNormArgs& a, hipStream_t s) {
  const int groups = block_norm_groups(a.T, a.H);
  norm_launch(a, groups, s);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || (!a.w_pre && !a.w_post && a.gate_axis != 2)) return err;
  hipLaunchKernelGGL(block_norm_reduce_kernel, dim3((a.H + 63) / 64, 3), dim3(1024), 0, s, a,
                     groups);
  return hipGetLastError();
}

}  // namespace nf4moe
