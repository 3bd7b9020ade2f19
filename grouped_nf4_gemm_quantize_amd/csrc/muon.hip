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
//
// Bound by memory: 16 to 22 bytes an element.  One workgroup takes a whole factor where
// factors are small, or enough to fill the card and each fits LDS: one launch, every array
// read once, u kept in LDS (A factors with rows 16 bytes longer, so that the 16 ranks
// of a column lie in different banks).  Otherwise two launches over (factor, chunk of
// the long axis): the first updates m and leaves each chunk's part of u u^T in the
// workspace, the second adds the parts in chunk order, does the algebra and applies P
// to its chunk.  Measured: four fp32 factors of each of 64 experts (H 2048, I 1024,
// r 8; 81 MB) 24.5 us = 3.3 TB/s, bf16 factors of 128 experts (H 2048, I 768, r 16; 210 MB)
// 79 us = 2.7 TB/s: a factor's fp64 products (8 k cycles each for u u^T and P u at 16 x
// 2048) and the algebra (0.5 us a step) are not covered by another factor's reads.
// 8 factors of 8 x 1000 take 11 us.  One tensor of a call whose elements are not four to an
// aligned read (r n or its row no multiple of four, an unaligned pointer) puts the whole call on
// the kernels with single reads, which spill 44 (factor) and 121 registers (apply): 64 experts'
// factors of rank 7 (H 2048, I 768) take 42 us against 12 for the bytes.

#include "common.h"
#include "launch.h"

namespace nf4moe {

namespace {

typedef double f64x4 __attribute__((ext_vector_type(4)));

constexpr int kMuonThreads = 512;  // of the two launches
constexpr int kMuonWaves = kMuonThreads / 64;
constexpr int kFactorThreads = 1024;  // of the one
constexpr int kFactorWaves = kFactorThreads / 64;
constexpr int kFactorReads = 9;       // reads of four elements a thread: 36864 elements
constexpr int kFactorFloats = 33792;  // LDS copy of u, with its padding
// Small factors, which get no workspace, always fit: rows of at most 7 elements more, 16 ranks.
static_assert(kMuonSmall + 16 * 7 <= kFactorFloats, "small factors take one launch");

__device__ __forceinline__ f64x4 mfma64(double a, double b, f64x4 c) {
  return __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, c, 0, 0, 0);
}

// A lane's four elements: their places in the factor and which exist.  Accesses
// compiled for kVec take i[0] .. i[0] + 3 at once, all or none.
struct Place {
  int i[4];
  bool in[4];
};

// Four elements as they are read; nothing is converted before it is used, so
// that reads stay in flight.
struct Raw4 {
  u32x4 v;
};

template <bool kVec>
__device__ __forceinline__ Raw4 fetch4(const void* p, int dtype, const Place& w) {
  Raw4 r = {{0u, 0u, 0u, 0u}};
  if constexpr (kVec) {
    if (w.in[0]) {
      if (dtype == kF32) {
        r.v = *reinterpret_cast<const u32x4*>(reinterpret_cast<const float*>(p) + w.i[0]);
      } else {
        const u32x2 h = *reinterpret_cast<const u32x2*>(reinterpret_cast<const uint16_t*>(p) + w.i[0]);
        r.v.x = h.x;
        r.v.y = h.y;
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (w.in[e])
        r.v[e] = dtype == kF32 ? reinterpret_cast<const uint32_t*>(p)[w.i[e]]
                               : reinterpret_cast<const uint16_t*>(p)[w.i[e]];
  }
  return r;
}

template <bool kVec>
__device__ __forceinline__ f32x4 widen4(const Raw4& r, int dtype) {
  f32x4 v;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (dtype == kF32) {
      v[e] = __uint_as_float(r.v[e]);
    } else {
      const uint32_t raw = kVec ? (r.v[e >> 1] >> (16 * (e & 1))) & 0xffffu : r.v[e];
      v[e] = dtype == kBF16 ? bf16_bits_to_f32(raw)
                            : (float)__builtin_bit_cast(_Float16, (uint16_t)raw);
    }
  }
  return v;
}

__device__ __forceinline__ uint16_t bits16(float v, int dtype) {
  return dtype == kBF16 ? f32_to_bf16_bits(v) : __builtin_bit_cast(uint16_t, (_Float16)v);
}

template <bool kVec>
__device__ __forceinline__ void store4(void* p, int dtype, const Place& w, f32x4 v) {
  if constexpr (kVec) {
    if (!w.in[0]) return;
    if (dtype == kF32) {
      *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(p) + w.i[0]) = v;
    } else {
      *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(p) + w.i[0]) =
          u32x2{bits16(v[0], dtype) | ((uint32_t)bits16(v[1], dtype) << 16),
                bits16(v[2], dtype) | ((uint32_t)bits16(v[3], dtype) << 16)};
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (!w.in[e]) continue;
      if (dtype == kF32) reinterpret_cast<float*>(p)[w.i[e]] = v[e];
      else reinterpret_cast<uint16_t*>(p)[w.i[e]] = bits16(v[e], dtype);
    }
  }
}

// What dtype holds of v: the 16-bit copy is taken of the weight as it is stored.
__device__ __forceinline__ f32x4 held4(f32x4 v, int dtype) {
  if (dtype != kF32) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      v[e] = dtype == kBF16 ? bf16_bits_to_f32(f32_to_bf16_bits(v[e])) : (float)(_Float16)v[e];
  }
  return v;
}

// A factor's shape: slots, its columns c0 .. c0 + cols - 1 in hand, and the distance of its
// ranks (A factors).
struct Shape {
  int r, p, inv;  // inv: f / r = f * inv >> 8 for f < 16
  int c0, cols, ld;
};

__device__ __forceinline__ Shape shape_of(int r, int c0, int cols, int ld) {
  return Shape{r, 16 / r, (256 + r - 1) / r, c0, cols, ld};
}

// u u^T, A factors: slot f, columns 16 blk + 4 q .. + 3 of its stretch.
// u u^T, B factors: slot f, groups 4 e + q of the block's sixteen, so that a lane row
// of 16 reads consecutive elements.
template <bool kRank>
__device__ __forceinline__ Place gram_place(const Shape& h, int blk, int f, int q) {
  Place w;
  const int seg = f * h.inv >> 8, rank = f - seg * h.r;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int c = kRank ? (blk * h.p + seg) * 16 + 4 * q + e : (blk * 16 + 4 * e + q) * h.p + seg;
    w.in[e] = seg < h.p && c < h.cols;
    w.i[e] = kRank ? rank * h.ld + h.c0 + c : (h.c0 + c) * h.r + rank;
  }
  return w;
}

// P u, A factors: slot 4 s + q, columns 4 c .. 4 c + 3 of a stretch of 64.
// P u, B factors: slots 4 q .. 4 q + 3 of group c of block blk + s.
template <bool kRank>
__device__ __forceinline__ Place apply_place(const Shape& h, int blk, int s, int lane) {
  Place w;
  const int q = lane >> 4, lane_c = lane & 15;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int f = kRank ? 4 * s + q : 4 * q + e;
    const int seg = f * h.inv >> 8, rank = f - seg * h.r;
    const int c = kRank ? (blk * h.p + seg) * 64 + 4 * lane_c + e
                        : ((blk + s) * 16 + lane_c) * h.p + seg;
    w.in[e] = seg < h.p && c < h.cols;
    w.i[e] = kRank ? rank * h.ld + h.c0 + c : (h.c0 + c) * h.r + rank;
  }
  return w;
}

// Blocks of a wave's turn, and of the shape.
template <bool kRank>
__device__ __forceinline__ int apply_blocks(const Shape& h) {
  const int width = (kRank ? 64 : 16) * h.p;
  return (h.cols + width - 1) / width;
}

// A factor's arrays from its expert's first element on.
__device__ __forceinline__ const void* at_base(const void* p, int dtype, int64_t base) {
  return reinterpret_cast<const char*>(p) + base * (dtype == kF32 ? 4 : 2);
}

// One wave: P / (|u| + eps) from the Gram matrix gm (zeros beyond r x r), as operand
// registers of P u.
template <bool kRank>
__device__ __forceinline__ void newton_schulz(const MuonArgs& a, const Shape& h,
                                              const double (&gm)[16][17], int lane,
                                              double (&pm)[4][64]) {
  double norm2 = 0.0;
#pragma unroll
  for (int k = 0; k < 16; ++k) norm2 += gm[k][k];
  const double inv = norm2 == 0.0 ? 0.0 : 1.0 / (sqrt(norm2) + a.eps);
  f64x4 g, id;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int k0 = 4 * j + (lane >> 4), k1 = lane & 15;
    const int f0 = kRank ? k0 : 4 * (k0 & 3) + (k0 >> 2);
    const int f1 = kRank ? k1 : 4 * (k1 & 3) + (k1 >> 2);
    const int s0 = f0 * h.inv >> 8, s1 = f1 * h.inv >> 8;
    const double v = gm[f0 - s0 * h.r][f1 - s1 * h.r] * inv * inv;
    g[j] = s0 == s1 && s0 < h.p ? v : 0.0;
    id[j] = k0 == k1 ? 1.0 : 0.0;
  }
  // two chains of two steps: a chain of four waits for each step's result
  const auto product = [&](const f64x4& x, const f64x4& y) {
    const f64x4 zero = {0.0, 0.0, 0.0, 0.0};
    f64x4 d = mfma64(x[0], y[0], zero), e = mfma64(x[1], y[1], zero);
    d = mfma64(x[2], y[2], d);
    e = mfma64(x[3], y[3], e);
    return d + e;
  };
  const auto quintic = [&](const f64x4& x) {
    const f64x4 x2 = product(x, x);
    f64x4 q;
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = a.a * id[j] + a.b * x[j] + a.c * x2[j];
    return q;
  };
  f64x4 q = quintic(g), p = q;
  for (int step = 1; step < a.steps; ++step) {
    const f64x4 w = product(q, g);
    g = product(w, q);
    q = quintic(g);
    p = product(q, p);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) pm[j][lane] = p[j] * inv;
}

// o = P u of a wave's turn: u[k][e] and the result in the places of apply_place.
template <bool kRank>
__device__ __forceinline__ void apply_products(const double (&pr)[4], const f32x4 (&u)[4],
                                               f64x4 (&o)[4]) {
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    f64x4 d = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
    for (int s = 0; s < 4; ++s) d = mfma64(pr[s], (double)(kRank ? u[s][x] : u[x][s]), d);
    o[x] = d;
  }
}

// The sums over waves and stretches of a wave's results for u u^T: element tid of r x r.
__device__ __forceinline__ double fold_gram(const double (*part)[16][17], int waves, const Shape& h,
                                            int tid) {
  const int i = tid / h.r, j = tid - i * h.r;
  double s = 0.0;
  for (int k = 0; k < h.p; ++k)
    for (int w = 0; w < waves; ++w) s += part[w][k * h.r + i][k * h.r + j];
  return s;
}

struct MuonBlock {
  int ti, e, chunk;
  int64_t base;
};

__device__ __forceinline__ MuonBlock muon_block(const MuonArgs& a) {
  MuonBlock b;
  b.ti = 0;
  while (b.ti + 1 < a.count && (int)blockIdx.x >= a.t[b.ti + 1].block0) ++b.ti;
  const MuonTensor& t = a.t[b.ti];
  const int local = blockIdx.x - t.block0;
  b.e = local / t.chunks;
  b.chunk = local - b.e * t.chunks;
  b.base = (int64_t)b.e * t.r * t.n;
  return b;
}

__device__ __forceinline__ Shape chunk_shape(const MuonTensor& t, const MuonBlock& b) {
  const int c0 = b.chunk * t.chunk_cols;
  return shape_of(t.r, c0, t.n - c0 < t.chunk_cols ? (int)(t.n - c0) : t.chunk_cols, (int)t.n);
}

template <bool kRank, bool kVec>
__device__ __forceinline__ f64x4 gram_chunk(const MuonArgs& a, const MuonTensor& t,
                                            const MuonBlock& b, const Shape& h, int wave,
                                            int lane) {
  constexpr bool kWide = kRank && kVec;  // B factors: one element a lane, rows together
  constexpr int kUnroll = 4;
  const int blocks = (h.cols + 16 * h.p - 1) / (16 * h.p);
  const void* g = at_base(t.g, t.g_dtype, b.base);
  f64x4 acc = {0.0, 0.0, 0.0, 0.0};
  for (int blk = wave; blk < blocks; blk += kMuonWaves * kUnroll) {
    Raw4 gv[kUnroll], mv[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const Place w = gram_place<kRank>(h, blk + k * kMuonWaves, lane & 15, lane >> 4);
      gv[k] = fetch4<kWide>(g, t.g_dtype, w);
      if (t.m) mv[k] = fetch4<kWide>(t.m + b.base, kF32, w);
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const f32x4 gw = widen4<kWide>(gv[k], t.g_dtype);
      f32x4 u = gw;
      if (t.m) {
        f32x4 m = widen4<kWide>(mv[k], kF32);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          m[e] = fmaf(a.mu, m[e], gw[e]);
          u[e] = a.nesterov ? fmaf(a.mu, m[e], gw[e]) : m[e];
        }
        const Place w = gram_place<kRank>(h, blk + k * kMuonWaves, lane & 15, lane >> 4);
        store4<kWide>(t.m_out + b.base, kF32, w, m);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) acc = mfma64((double)u[e], (double)u[e], acc);
    }
  }
  return acc;
}

template <bool kRank, bool kVec>
__device__ __forceinline__ void apply_factor(const MuonArgs& a, const MuonTensor& t,
                                             const MuonBlock& b, double (&gm)[16][17],
                                             double (&pm)[4][64]) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Shape h = chunk_shape(t, b);
  constexpr int kStep = kRank ? 1 : 4;
  const int blocks = apply_blocks<kRank>(h);
  const void* g = at_base(t.g, t.g_dtype, b.base);
  const void* w = at_base(t.w, t.w_dtype, b.base);
  void* w_out = const_cast<void*>(at_base(t.w_out, t.w_dtype, b.base));
  void* w16 = const_cast<void*>(at_base(t.w16, kF16, b.base));
  const double keep = 1.0 - a.lr * a.weight_decay, step = -a.lr * t.scale;
  Raw4 gv[4], mv[4], wv[4];
  const auto read = [&](int blk) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const Place pl = apply_place<kRank>(h, blk, k, lane);
      gv[k] = fetch4<kVec>(g, t.g_dtype, pl);
      if (t.m) mv[k] = fetch4<kVec>(t.m_out + b.base, kF32, pl);
      if (t.w) wv[k] = fetch4<kVec>(w, t.w_dtype, pl);
    }
  };
  double sum = 0.0;
  if (tid < 256) {
    const int i = tid >> 4, j = tid & 15;
    if (i < h.r && j < h.r) {
      const double* gram = t.gram + (int64_t)b.e * t.chunks * h.r * h.r + i * h.r + j;
      for (int c = 0; c < t.chunks; ++c) sum += gram[(int64_t)c * h.r * h.r];
    }
  }
  // the first reads (all of a usual chunk's) are in flight during the algebra
  int blk = wave * kStep;
  read(blk);
  if (tid < 256) gm[tid >> 4][tid & 15] = sum;
  __syncthreads();
  if (wave == 0) newton_schulz<kRank>(a, h, gm, lane, pm);
  __syncthreads();
  const double pr[4] = {pm[0][lane], pm[1][lane], pm[2][lane], pm[3][lane]};
  while (blk < blocks) {
    f32x4 u[4], o4[4];
    f64x4 o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      u[k] = widen4<kVec>(gv[k], t.g_dtype);
      if (t.m) {
        const f32x4 m = widen4<kVec>(mv[k], kF32);
#pragma unroll
        for (int e = 0; e < 4; ++e) u[k][e] = a.nesterov ? fmaf(a.mu, m[e], u[k][e]) : m[e];
      }
    }
    apply_products<kRank>(pr, u, o);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const f32x4 wf = widen4<kVec>(wv[k], t.w_dtype);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const double d = kRank ? o[e][k] : o[k][e];
        o4[k][e] = (float)(t.w ? keep * (double)wf[e] + step * d : d);
      }
      const Place pl = apply_place<kRank>(h, blk, k, lane);
      store4<kVec>(w_out, t.w_dtype, pl, o4[k]);
      if (t.w16) store4<kVec>(w16, t.w16_dtype, pl, held4(o4[k], t.w_dtype));
    }
    blk += kMuonWaves * kStep;
    if (blk < blocks) read(blk);
  }
}

// One workgroup, one factor: u in LDS (A factors with padded rows), everything else in
// registers.
template <bool kRank, bool kVec>
__device__ __forceinline__ void whole_factor(const MuonArgs& a, const MuonTensor& t,
                                             const MuonBlock& b, float* u,
                                             double (*part)[16][17], double (&gm)[16][17],
                                             double (&pm)[4][64]) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = (int)t.n, size = t.r * n, ld = t.lds_row;
  const Shape h = shape_of(t.r, 0, n, ld);
  const void* g = at_base(t.g, t.g_dtype, b.base);
  const void* w = at_base(t.w, t.w_dtype, b.base);
  // read k of a thread: four consecutive elements in memory order
  const auto flat = [&](int k) {
    Place pl;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      pl.i[e] = (tid + k * kFactorThreads) * 4 + e;
      pl.in[e] = pl.i[e] < size;
    }
    return pl;
  };
  // an element's place in LDS: rows of A factors are ld apart
  const auto slot = [&](int i) {
    return kRank ? i + (int)__umulhi((uint32_t)i, t.n_magic) * (ld - n) : i;
  };
  const auto turn = [&](int first, int last) {
    Raw4 gv[5], mv[5];
#pragma unroll
    for (int k = 0; k < 5; ++k) {
      if (first + k >= last) break;
      const Place pl = flat(first + k);
      gv[k] = fetch4<kVec>(g, t.g_dtype, pl);
      if (t.m) mv[k] = fetch4<kVec>(t.m + b.base, kF32, pl);
    }
#pragma unroll
    for (int k = 0; k < 5; ++k) {
      if (first + k >= last) break;
      const Place pl = flat(first + k);
      f32x4 x = widen4<kVec>(gv[k], t.g_dtype);
      if (t.m) {
        f32x4 m = widen4<kVec>(mv[k], kF32);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          m[e] = fmaf(a.mu, m[e], x[e]);
          x[e] = a.nesterov ? fmaf(a.mu, m[e], x[e]) : m[e];
        }
        store4<kVec>(t.m_out + b.base, kF32, pl, m);
      }
      if constexpr (kVec) {
        if (pl.in[0]) *reinterpret_cast<f32x4*>(u + slot(pl.i[0])) = x;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (pl.in[e]) u[slot(pl.i[e])] = x[e];
      }
    }
  };
  // zeros behind the rows (A) or the factor (B), which wide LDS reads touch
  const int tail = kRank ? ld - n : 16;
  for (int i = tid; i < (kRank ? h.r : 1) * tail; i += kFactorThreads) {
    const int row = i / tail;
    u[kRank ? row * ld + n + (i - row * tail) : size + i] = 0.f;
  }
  turn(0, 5);
  if (size > 5 * 4 * kFactorThreads) turn(5, kFactorReads);
  Raw4 wv[kFactorReads];
  if (t.w) {
#pragma unroll
    for (int k = 0; k < kFactorReads; ++k) wv[k] = fetch4<kVec>(w, t.w_dtype, flat(k));
  }
  __syncthreads();
  const int gblocks = (n + 16 * h.p - 1) / (16 * h.p);
  f64x4 acc = {0.0, 0.0, 0.0, 0.0};
  for (int blk = wave; blk < gblocks; blk += kFactorWaves) {
    const Place pl = gram_place<kRank>(h, blk, lane & 15, lane >> 4);
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
    if constexpr (kRank) {
      if (pl.in[0]) x = *reinterpret_cast<const f32x4*>(u + pl.i[0]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (pl.in[e]) x[e] = u[pl.i[e]];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) acc = mfma64((double)x[e], (double)x[e], acc);
  }
  // the upper eight waves hand their sums to the lower
  constexpr int kHalf = kFactorWaves / 2;
  if (wave >= kHalf)
#pragma unroll
    for (int j = 0; j < 4; ++j) part[wave - kHalf][4 * j + (lane >> 4)][lane & 15] = acc[j];
  __syncthreads();
  if (wave < kHalf)
#pragma unroll
    for (int j = 0; j < 4; ++j) part[wave][4 * j + (lane >> 4)][lane & 15] += acc[j];
  if (tid < 256) gm[tid >> 4][tid & 15] = 0.0;
  __syncthreads();
  if (tid < h.r * h.r) gm[tid / h.r][tid % h.r] = fold_gram(part, kHalf, h, tid);
  __syncthreads();
  if (wave == 0) newton_schulz<kRank>(a, h, gm, lane, pm);
  __syncthreads();
  const double pr[4] = {pm[0][lane], pm[1][lane], pm[2][lane], pm[3][lane]};
  constexpr int kStep = kRank ? 1 : 4;
  const int blocks = apply_blocks<kRank>(h);
  // four B slots are one LDS access where a group has a multiple of four
  const bool wide = kRank || h.p * h.r % 4 == 0;
  for (int blk = wave * kStep; blk < blocks; blk += kFactorWaves * kStep) {
    f32x4 x[4];
    f64x4 o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const Place pl = apply_place<kRank>(h, blk, k, lane);
      x[k] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (wide) {
        if (pl.in[0]) x[k] = *reinterpret_cast<const f32x4*>(u + pl.i[0]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (pl.in[e]) x[k][e] = u[pl.i[e]];
      }
    }
    apply_products<kRank>(pr, x, o);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const Place pl = apply_place<kRank>(h, blk, k, lane);
      // O in fp32, as LDS has room for no more: half a unit in 2^24 of the step.  w' is
      // rounded to its type after that, so where w is (nearly) zero it is rounded twice.
      f32x4 y;
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = (float)(kRank ? o[e][k] : o[k][e]);
      if (wide) {
        if (pl.in[0]) *reinterpret_cast<f32x4*>(u + pl.i[0]) = y;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (pl.in[e]) u[pl.i[e]] = y[e];
      }
    }
  }
  __syncthreads();
  void* w_out = const_cast<void*>(at_base(t.w_out, t.w_dtype, b.base));
  void* w16 = const_cast<void*>(at_base(t.w16, kF16, b.base));
  const double keep = 1.0 - a.lr * a.weight_decay, step = -a.lr * t.scale;
#pragma unroll
  for (int k = 0; k < kFactorReads; ++k) {
    const Place pl = flat(k);
    if (!pl.in[0]) break;
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    if constexpr (kVec) {
      o = *reinterpret_cast<const f32x4*>(u + slot(pl.i[0]));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (pl.in[e]) o[e] = u[slot(pl.i[e])];
    }
    if (t.w) {
      const f32x4 wf = widen4<kVec>(wv[k], t.w_dtype);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = (float)(keep * (double)wf[e] + step * (double)o[e]);
    }
    store4<kVec>(w_out, t.w_dtype, pl, o);
    if (t.w16) store4<kVec>(w16, t.w16_dtype, pl, held4(o, t.w_dtype));
  }
}

}  // namespace

// kVec: every tensor of the call has aligned reads of four.
template <bool kVec>
__global__ __launch_bounds__(kMuonThreads) void muon_gram_kernel(MuonArgs a) {
  __shared__ double part[kMuonWaves][16][17];
  const MuonBlock b = muon_block(a);
  const MuonTensor& t = a.t[b.ti];
  const Shape h = chunk_shape(t, b);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const f64x4 acc =
      t.rank_major ? gram_chunk<true, kVec>(a, t, b, h, wave, lane)
                   : gram_chunk<false, kVec>(a, t, b, h, wave, lane);
#pragma unroll
  for (int j = 0; j < 4; ++j) part[wave][4 * j + (lane >> 4)][lane & 15] = acc[j];
  __syncthreads();
  if (tid < t.r * t.r)
    t.gram[((int64_t)b.e * t.chunks + b.chunk) * t.r * t.r + tid] =
        fold_gram(part, kMuonWaves, h, tid);
}

template <bool kVec>
__global__ __launch_bounds__(kMuonThreads, 4) void muon_apply_kernel(MuonArgs a) {
  __shared__ double gm[16][17];
  __shared__ double pm[4][64];
  const MuonBlock b = muon_block(a);
  const MuonTensor& t = a.t[b.ti];
  if (t.rank_major) apply_factor<true, kVec>(a, t, b, gm, pm);
  else apply_factor<false, kVec>(a, t, b, gm, pm);
}

template <bool kVec>
__global__ __launch_bounds__(kFactorThreads) void muon_factor_kernel(MuonArgs a) {
  extern __shared__ float lds_u[];
  __shared__ double part[kFactorWaves / 2][16][17];
  __shared__ double gm[16][17];
  __shared__ double pm[4][64];
  const MuonBlock b = muon_block(a);
  const MuonTensor& t = a.t[b.ti];
  if (t.rank_major) whole_factor<true, kVec>(a, t, b, lds_u, part, gm, pm);
  else whole_factor<false, kVec>(a, t, b, lds_u, part, gm, pm);
}

// Long-axis elements of a workgroup: 8192 elements of the factor and whole blocks of both
// kernels, fewer where a tensor would not fill the card.
int muon_chunk_cols(int E, int64_t n, int r) {
  const int unit = 64 * (16 / r);
  int64_t cols = (8192 / r + unit - 1) / unit * unit;
  while (cols > unit && E * ((n + cols - 1) / cols) < 256) cols = (cols / 2 + unit - 1) / unit * unit;
  return (int)cols;
}

namespace {

template <bool kVec>
hipError_t muon_go(const MuonArgs& a, int lds, hipStream_t s) {
  if (lds > 0) {
    if (lds > 32768) {  // beyond 64 KiB with the kernel's own
      // The limit is the function's, not the launch's: always the same, so that a smaller call
      // of another host thread does not lower it between here and the launch.
      const void* k = reinterpret_cast<const void*>(muon_factor_kernel<kVec>);
      hipError_t err = hipFuncSetAttribute(k, hipFuncAttributeMaxDynamicSharedMemorySize,
                                           kFactorFloats * 4);
      if (err != hipSuccess) return err;
    }
    hipLaunchKernelGGL(muon_factor_kernel<kVec>, dim3(a.blocks), dim3(kFactorThreads), lds, s, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(muon_gram_kernel<kVec>, dim3(a.blocks), dim3(kMuonThreads), 0, s, a);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL(muon_apply_kernel<kVec>, dim3(a.blocks), dim3(kMuonThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_muon(MuonArgs& a, int num_cus, hipStream_t s) {
  // One workgroup a factor where all fit, and either half the compute units or more get one, or
  // factors are small: 64 factors of 8 x 2048 take 20-24 us in two launches, 128 of them 19-20
  // in one; 64 of 16 x 2048 take 22-25 us in two, 128 of them 31 in one.
  int64_t factors = 0, floats = 0;
  bool small = true;
  bool vec = true;
  for (int i = 0; i < a.count; ++i) {
    MuonTensor& t = a.t[i];
    if (t.n == 1) t.rank_major = 0;  // the same memory either way
    t.lds_row = t.rank_major ? (int)((t.n + 3) / 4 * 4 + 4) : 0;
    const int64_t need = t.rank_major ? (int64_t)t.r * t.lds_row : t.r * t.n + 16;
    floats = need > floats ? need : floats;
    factors += t.E;
    small = small && muon_small(t.r, t.n);
    vec = vec && t.vec;
  }
  int lds = 0;
  if (floats <= kFactorFloats && (2 * factors >= num_cus || small)) {
    lds = (int)floats * 4;
    a.blocks = 0;
    for (int i = 0; i < a.count; ++i) {
      a.t[i].chunks = 1;
      a.t[i].block0 = a.blocks;
      a.blocks += a.t[i].E;
      // i / n = umulhi(i, n_magic): exact, as i and n are below 2^16; A factors have n > 1
      a.t[i].n_magic =
          a.t[i].rank_major ? (uint32_t)((((uint64_t)1 << 32) + a.t[i].n - 1) / a.t[i].n) : 0u;
    }
  }
  return vec ? muon_go<true>(a, lds, s) : muon_go<false>(a, lds, s);
}

}  // namespace nf4moe
