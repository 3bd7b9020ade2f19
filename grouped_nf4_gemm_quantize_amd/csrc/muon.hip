// The optimiser step of per-expert adapter factors, orthogonalised by
// Newton-Schulz products (lora_muon_step, lora_orthogonalize).
//
// A factor u is r x n with r <= 16.  The iteration
//   X <- a X + b (X X^T) X + c (X X^T)^2 X,  X_0 = u / (|u| + eps)
// stays in the row space: with X_k = P_k X_0 and G_k = X_k X_k^T,
//   Q = a I + b G_k + c G_k^2,  P_{k+1} = Q P_k,  G_{k+1} = Q G_k Q,
// so the long axis is needed only for G_0 and for O = P u / (|u| + eps).  A direction of
// singular value s << 1 grows a-fold a step (485-fold in five with a = 3.4445)
// and an error of its G a^2-fold, which 32 bits cannot hold: G, P and
// O are 64-bit, on the matrix unit's fp64 form (16x16x4).
//
// Two launches over (factor, chunk of the long axis): the first updates m and
// leaves each chunk's part of u u^T in the workspace, the second adds the parts in
// chunk order, does the r x r algebra and applies P to its chunk.
//
// Slots: the 16 rows of a matrix step hold p = floor(16 / r) stretches of the long
// axis side by side, slot f = stretch * r + rank, so that small ranks fill it too; the
// matrices between them are block diagonal, p copies of the r x r ones.
//  - For u u^T lane 16 q + i holds slot i and contracts over q: products of a
//    register with itself.
//  - For P u lane 16 q + c holds, for step s, slot 4 s + q (A factors) or 4 q + s (B
//    factors, whose four are then consecutive in memory) of column c; the result
//    registers hold the same elements as the operands.
//  - G, Q and P are polynomials of one symmetric matrix, so symmetric and commuting;
//    the result registers of a symmetric matrix (row 4 j + q, column i) are its operand
//    registers (row i, column 4 j + q): no product needs an exchange between lanes.

#include "common.h"
#include "launch.h"

namespace nf4moe {

namespace {

typedef double f64x4 __attribute__((ext_vector_type(4)));

constexpr int kMuonThreads = 512;
constexpr int kMuonWaves = kMuonThreads / 64;

__device__ __forceinline__ f64x4 mfma64(double a, double b, f64x4 c) {
  return __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, c, 0, 0, 0);
}

// Four elements i .. i + 3 of an array of any type; kVec: aligned, else one by one
// those that `in` names.
template <bool kVec>
__device__ __forceinline__ f32x4 load4(const void* p, int dtype, const int64_t (&i)[4],
                                       const bool (&in)[4]) {
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  if constexpr (kVec) {
    if (!in[0]) return v;
    if (dtype == kF32) return *reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(p) + i[0]);
    const u32x2 h = *reinterpret_cast<const u32x2*>(reinterpret_cast<const uint16_t*>(p) + i[0]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t raw = (h[e >> 1] >> (16 * (e & 1))) & 0xffffu;
      v[e] = dtype == kBF16 ? bf16_bits_to_f32(raw)
                            : (float)__builtin_bit_cast(_Float16, (uint16_t)raw);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (!in[e]) continue;
      if (dtype == kF32) {
        v[e] = reinterpret_cast<const float*>(p)[i[e]];
      } else {
        const uint16_t raw = reinterpret_cast<const uint16_t*>(p)[i[e]];
        v[e] = dtype == kBF16 ? bf16_bits_to_f32(raw) : (float)__builtin_bit_cast(_Float16, raw);
      }
    }
  }
  return v;
}

__device__ __forceinline__ uint16_t bits16(float v, int dtype) {
  return dtype == kBF16 ? f32_to_bf16_bits(v) : __builtin_bit_cast(uint16_t, (_Float16)v);
}

template <bool kVec>
__device__ __forceinline__ void store4(void* p, int dtype, const int64_t (&i)[4],
                                       const bool (&in)[4], f32x4 v) {
  if constexpr (kVec) {
    if (!in[0]) return;
    if (dtype == kF32) {
      *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(p) + i[0]) = v;
    } else {
      *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(p) + i[0]) =
          u32x2{bits16(v[0], dtype) | ((uint32_t)bits16(v[1], dtype) << 16),
                bits16(v[2], dtype) | ((uint32_t)bits16(v[3], dtype) << 16)};
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (!in[e]) continue;
      if (dtype == kF32) reinterpret_cast<float*>(p)[i[e]] = v[e];
      else reinterpret_cast<uint16_t*>(p)[i[e]] = bits16(v[e], dtype);
    }
  }
}

// Where a lane's four elements lie in its factor (i) and which exist (in): of a
// workgroup's columns c0 .. c0 + cols - 1, block `blk`.
struct Place {
  int64_t i[4];
  bool in[4];
};

// u u^T, A factors: slot f, columns 16 blk + 4 q .. + 3 of its stretch.
// u u^T, B factors: slot f, groups 4 e + q of the block's sixteen: whole rows of
// 64 consecutive elements (r divides 16) are read at a time.
template <bool kRank>
__device__ __forceinline__ Place gram_place(const MuonTensor& t, int64_t c0, int cols, int p,
                                            int blk, int f, int q) {
  Place w;
  const int seg = f / t.r, rank = f - seg * t.r;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int c = kRank ? blk * 16 * p + seg * 16 + 4 * q + e : (blk * 16 + 4 * e + q) * p + seg;
    w.in[e] = f < p * t.r && c < cols;
    w.i[e] = kRank ? rank * t.n + c0 + c : (c0 + c) * t.r + rank;
  }
  return w;
}

// P u, A factors: slot 4 s + q, columns 4 c .. 4 c + 3 of a stretch of 64.
// P u, B factors: slots 4 q .. 4 q + 3 of group c.
template <bool kRank>
__device__ __forceinline__ Place apply_place(const MuonTensor& t, int64_t c0, int cols, int p,
                                             int blk, int s, int q, int lane_c) {
  Place w;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int f = kRank ? 4 * s + q : 4 * q + e;
    const int seg = f / t.r, rank = f - seg * t.r;
    const int c = kRank ? blk * 64 * p + seg * 64 + 4 * lane_c + e : (blk * 16 + lane_c) * p + seg;
    w.in[e] = f < p * t.r && c < cols;
    w.i[e] = kRank ? rank * t.n + c0 + c : (c0 + c) * t.r + rank;
  }
  return w;
}

struct MuonBlock {
  int ti, e, chunk, cols, p;
  int64_t c0, base;
};

__device__ __forceinline__ MuonBlock muon_block(const MuonArgs& a) {
  MuonBlock b;
  b.ti = 0;
  while (b.ti + 1 < a.count && (int)blockIdx.x >= a.t[b.ti + 1].block0) ++b.ti;
  const MuonTensor& t = a.t[b.ti];
  const int local = blockIdx.x - t.block0;
  b.e = local / t.chunks;
  b.chunk = local - b.e * t.chunks;
  b.c0 = (int64_t)b.chunk * t.chunk_cols;
  b.cols = t.n - b.c0 < t.chunk_cols ? (int)(t.n - b.c0) : t.chunk_cols;
  b.base = (int64_t)b.e * t.r * t.n;
  b.p = 16 / t.r;
  return b;
}

// A factor's arrays from its expert's first element on.
__device__ __forceinline__ const void* at_base(const void* p, int dtype, int64_t base) {
  return reinterpret_cast<const char*>(p) + base * (dtype == kF32 ? 4 : 2);
}

template <bool kRank, bool kVec>
__device__ __forceinline__ f64x4 gram_chunk(const MuonArgs& a, const MuonTensor& t,
                                            const MuonBlock& b, int wave, int lane) {
  constexpr bool kWide = kRank && kVec;  // B factors: one element a lane, rows together
  constexpr int kUnroll = 4;
  const int f = lane & 15, q = lane >> 4;
  const int blocks = (b.cols + 16 * b.p - 1) / (16 * b.p);
  const void* g = at_base(t.g, t.g_dtype, b.base);
  const float* m = t.m ? t.m + b.base : nullptr;
  float* m_out = t.m ? t.m_out + b.base : nullptr;
  f64x4 acc = {0.0, 0.0, 0.0, 0.0};
  for (int blk = wave; blk < blocks; blk += kMuonWaves * kUnroll) {
    Place w[kUnroll];
    f32x4 gv[kUnroll], mv[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      w[k] = gram_place<kRank>(t, b.c0, b.cols, b.p, blk + k * kMuonWaves, f, q);
      gv[k] = load4<kWide>(g, t.g_dtype, w[k].i, w[k].in);
      if (m) mv[k] = load4<kWide>(m, kF32, w[k].i, w[k].in);
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      f32x4 u = gv[k];
      if (m) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          mv[k][e] = fmaf(a.mu, mv[k][e], gv[k][e]);
          u[e] = a.nesterov ? fmaf(a.mu, mv[k][e], gv[k][e]) : mv[k][e];
        }
        store4<kWide>(m_out, kF32, w[k].i, w[k].in, mv[k]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) acc = mfma64((double)u[e], (double)u[e], acc);
    }
  }
  return acc;
}

template <bool kRank, bool kVec>
__device__ __forceinline__ void apply_chunk(const MuonArgs& a, const MuonTensor& t,
                                            const MuonBlock& b, const double (&pm)[4], int wave,
                                            int lane) {
  const int lane_c = lane & 15, q = lane >> 4;
  const int width = kRank ? 64 * b.p : 16 * b.p;
  const int blocks = (b.cols + width - 1) / width;
  const void* g = at_base(t.g, t.g_dtype, b.base);
  const float* m = t.m ? t.m_out + b.base : nullptr;
  const void* w = at_base(t.w, t.w_dtype, b.base);
  void* w_out = const_cast<void*>(at_base(t.w_out, t.w_dtype, b.base));
  void* w16 = const_cast<void*>(at_base(t.w16, kF16, b.base));
  const double keep = 1.0 - a.lr * a.weight_decay, step = -a.lr * t.scale;
  // four reads of four elements: the slots of one block (A), four blocks (B)
  constexpr int kStep = kRank ? 1 : 4;
  for (int blk = wave * kStep; blk < blocks; blk += kMuonWaves * kStep) {
    Place pl[4];
    f32x4 u[4], wv[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      pl[k] = apply_place<kRank>(t, b.c0, b.cols, b.p, kRank ? blk : blk + k, k, q, lane_c);
      u[k] = load4<kVec>(g, t.g_dtype, pl[k].i, pl[k].in);
      if (m) {
        const f32x4 mv = load4<kVec>(m, kF32, pl[k].i, pl[k].in);
#pragma unroll
        for (int e = 0; e < 4; ++e) u[k][e] = a.nesterov ? fmaf(a.mu, mv[e], u[k][e]) : mv[e];
      }
      if (t.w) wv[k] = load4<kVec>(w, t.w_dtype, pl[k].i, pl[k].in);
    }
    f32x4 o[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      f64x4 d = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
      for (int s = 0; s < 4; ++s) d = mfma64(pm[s], (double)(kRank ? u[s][x] : u[x][s]), d);
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        double v = d[s];
        if (t.w) v = keep * (double)(kRank ? wv[s][x] : wv[x][s]) + step * v;
        if constexpr (kRank) o[s][x] = (float)v;
        else o[x][s] = (float)v;
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      store4<kVec>(w_out, t.w_dtype, pl[k].i, pl[k].in, o[k]);
      if (t.w16) {
        f32x4 r = o[k];
        store4<kVec>(w16, t.w16_dtype, pl[k].i, pl[k].in, r);
      }
    }
  }
}

}  // namespace

__global__ __launch_bounds__(kMuonThreads) void muon_gram_kernel(MuonArgs a) {
  __shared__ double part[kMuonWaves][16][17];
  const MuonBlock b = muon_block(a);
  const MuonTensor& t = a.t[b.ti];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  f64x4 acc;
  if (t.rank_major)
    acc = t.vec ? gram_chunk<true, true>(a, t, b, wave, lane)
                : gram_chunk<true, false>(a, t, b, wave, lane);
  else
    acc = gram_chunk<false, false>(a, t, b, wave, lane);
#pragma unroll
  for (int j = 0; j < 4; ++j) part[wave][4 * j + (lane >> 4)][lane & 15] = acc[j];
  __syncthreads();
  const int r = t.r, i = tid / r, j = tid - i * r;
  if (i >= r) return;
  double s = 0.0;
  for (int k = 0; k < b.p; ++k)
    for (int w = 0; w < kMuonWaves; ++w) s += part[w][k * r + i][k * r + j];
  t.gram[((int64_t)b.e * t.chunks + b.chunk) * r * r + tid] = s;
}

__global__ __launch_bounds__(kMuonThreads) void muon_apply_kernel(MuonArgs a) {
  __shared__ double gm[16][17];
  __shared__ double pm[4][64];
  const MuonBlock b = muon_block(a);
  const MuonTensor& t = a.t[b.ti];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = t.r;
  if (tid < r * r) {
    const double* gram = t.gram + (int64_t)b.e * t.chunks * r * r + tid;
    double s = 0.0;
    for (int c = 0; c < t.chunks; ++c) s += gram[(int64_t)c * r * r];
    gm[tid / r][tid % r] = s;
  }
  __syncthreads();
  if (wave == 0) {
    double norm2 = 0.0;
    for (int k = 0; k < r; ++k) norm2 += gm[k][k];
    const double inv = norm2 == 0.0 ? 0.0 : 1.0 / (sqrt(norm2) + a.eps);
    f64x4 g, p, id;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k0 = 4 * j + (lane >> 4), k1 = lane & 15;
      const int f0 = t.rank_major ? k0 : 4 * (k0 & 3) + (k0 >> 2);
      const int f1 = t.rank_major ? k1 : 4 * (k1 & 3) + (k1 >> 2);
      const bool in = f0 / r == f1 / r && f0 < b.p * r && f1 < b.p * r;
      g[j] = in ? gm[f0 % r][f1 % r] * inv * inv : 0.0;
      id[j] = k0 == k1 ? 1.0 : 0.0;
    }
    const auto product = [&](const f64x4& x, const f64x4& y) {
      f64x4 d = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
      for (int s = 0; s < 4; ++s) d = mfma64(x[s], y[s], d);
      return d;
    };
    p = id;
    for (int step = 0; step < a.steps; ++step) {
      const f64x4 g2 = product(g, g);
      f64x4 q;
#pragma unroll
      for (int j = 0; j < 4; ++j) q[j] = a.a * id[j] + a.b * g[j] + a.c * g2[j];
      const f64x4 h = product(q, g);
      p = product(q, p);
      g = product(h, q);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) pm[j][lane] = p[j] * inv;
  }
  __syncthreads();
  const double pr[4] = {pm[0][lane], pm[1][lane], pm[2][lane], pm[3][lane]};
  if (t.rank_major) {
    if (t.vec) apply_chunk<true, true>(a, t, b, pr, wave, lane);
    else apply_chunk<true, false>(a, t, b, pr, wave, lane);
  } else {
    if (t.vec) apply_chunk<false, true>(a, t, b, pr, wave, lane);
    else apply_chunk<false, false>(a, t, b, pr, wave, lane);
  }
}

// Long-axis elements of a workgroup: 8192 elements of the factor and whole blocks of both
// kernels, fewer where a tensor would not fill the card.
int muon_chunk_cols(int E, int64_t n, int r) {
  const int unit = 64 * (16 / r);
  int64_t cols = (8192 / r + unit - 1) / unit * unit;
  while (cols > unit && E * ((n + cols - 1) / cols) < 256) cols = (cols / 2 + unit - 1) / unit * unit;
  return (int)cols;
}

hipError_t launch_muon(const MuonArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(muon_gram_kernel, dim3(a.blocks), dim3(kMuonThreads), 0, s, a);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL(muon_apply_kernel, dim3(a.blocks), dim3(kMuonThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace nf4moe
