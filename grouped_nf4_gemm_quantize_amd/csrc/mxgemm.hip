// The grouped product of two MXFP4 operands (grouped_mx4_gemm): rows of one
// expert times that expert's matrix,
//   out[i, n] = sum over blocks b of 2^(sa[i,b] + sw[n,b] - 254) * sum_{k in b} va[i,k] vw[n,k],
// on the matrix unit's scaled 4-bit instructions: v_mfma_scale_f32_16x16x128
// takes 16 x 128 codes of either operand, one block of 32 and its scale byte a
// lane, and adds the scaled sums to fp32 accumulators (2^-24 of the terms'
// magnitudes a step, as measured: less than one fp32 rounding).
//
// K need only be a multiple of 32: blocks beyond a row's end get the scale byte
// 0 on both sides, so whatever codes are read there count 2^-254 times at most
// 1152 a block, which is nothing beside any fp32 number and 0 alone.

#include <algorithm>

#include "common.h"
#include "launch.h"
#include "mfma_common.h"

namespace nf4moe {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kWaves = 4;
constexpr int kThreads = kWaves * 64;

__shared__ int32_t s_tiles[kMaxExperts + 1];
__shared__ int32_t s_wsum[kWaves];
__shared__ float s_part[kWaves][2][16][17];

// Two values rounded to the nearest 16-bit ones.
template <int kOut>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  if constexpr (kOut == kBF16) return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
  else return pack_half2((_Float16)a, (_Float16)b);
}

template <int kOut>
__device__ __forceinline__ void store4(void* out, int64_t idx, const float (&v)[4]) {
  if constexpr (kOut == kF32) {
    *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(out) + idx) = f32x4{v[0], v[1], v[2], v[3]};
  } else {
    *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(out) + idx) =
        u32x2{pack2<kOut>(v[0], v[1]), pack2<kOut>(v[2], v[3])};
  }
}

__device__ __forceinline__ i32x8 codes8(u32x4 v) {
  return i32x8{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
}

}  // namespace

// 16 rows of one expert by 32 weight rows (SwiGLU: 16 gate and their 16 up rows) a
// workgroup; its waves take every fourth 128 of K and join in LDS.
template <bool kSwiglu, int kOut>
__global__ __launch_bounds__(kThreads) void mx_small_kernel(MxGemmArgs g, int n_tiles) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r16 = lane & 15, q = lane >> 4;
  build_tile_table<kThreads, 16>(g.offsets, g.E, s_tiles, s_wsum, tid);
  const int N = g.N, I = N >> 1, KB = g.K / 32;
  const int total = s_tiles[g.E] * n_tiles;
  for (int tix = blockIdx.x; tix < total; tix += gridDim.x) {
    const int mt = tix / n_tiles, nt = tix - mt * n_tiles;
    int lo = 0, hi = g.E;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_tiles[mid] <= mt) lo = mid; else hi = mid;
    }
    const int e = lo;
    const int row0 = g.offsets[e] + (mt - s_tiles[e]) * 16;
    const int rows = min(16, min(g.offsets[e + 1], (int)g.P) - row0);
    if (rows <= 0) continue;  // behind P
    const int row = row0 + (r16 < rows ? r16 : 0);
    int64_t src = g.gather ? g.gather[row] / g.gather_div : row;
    src = src < 0 ? 0 : src >= g.a_rows ? g.a_rows - 1 : src;
    const uint8_t* ac = g.a + src * KB * 16;
    const uint8_t* as = g.a_scales + src * KB;
    // weight rows of the tile's two halves, clamped to valid ones
    const uint8_t* wc[2];
    const uint8_t* ws[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      int n = kSwiglu ? min(nt * 16 + r16, I - 1) + h * I : min(nt * 32 + h * 16 + r16, N - 1);
      const int64_t at = (int64_t)e * N + n;
      wc[h] = g.blocks + at * KB * 16;
      ws[h] = g.scales + at * KB;
    }
    f32x4 acc[2] = {};
    for (int b0 = wave * 4; b0 < KB; b0 += kWaves * 4) {
      const int b = min(b0 + q, KB - 1);
      const bool in = b0 + q < KB;
      const u32x4 av = *reinterpret_cast<const u32x4*>(ac + (int64_t)b * 16);
      const int sa = in ? as[b] : 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const u32x4 wv = *reinterpret_cast<const u32x4*>(wc[h] + (int64_t)b * 16);
        const int sw = in ? ws[h][b] : 0;
        // the weights first: a lane's four sums are consecutive output columns
        acc[h] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(codes8(wv), codes8(av), acc[h],
                                                                  4, 4, 0, sw, 0, sa);
      }
    }
    __syncthreads();  // the last tile's sums are read
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) s_part[wave][h][r16][4 * q + i] = acc[h][i];
    __syncthreads();
    // 16 rows x 32 columns (SwiGLU: 16), two (one) a thread
    const int c = tid & 15, r = tid >> 4;
    float v[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      v[h] = (s_part[0][h][r][c] + s_part[1][h][r][c]) + (s_part[2][h][r][c] + s_part[3][h][r][c]);
    if (r < rows) {
      const int i = row0 + r;
      const int64_t o = g.scatter ? g.scatter[i] : i;
      if (o >= 0 && o < g.out_rows) {
        const float rs = g.row_scale ? g.row_scale[i] : 1.f;
        if constexpr (kSwiglu) {
          const int col = nt * 16 + c;
          if (col < I) store_out<kOut>(g.out, o * I + col, silu_f(v[0]) * v[1] * rs);
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int col = nt * 32 + h * 16 + c;
            if (col < N) store_out<kOut>(g.out, o * N + col, v[h] * rs);
          }
        }
      }
    }
  }
}

// ---- many rows: tiles through LDS ---------------------------------------------------

namespace {

// A tile: WM x WN waves, each MT x NT accumulator tiles of 32 x 32 (v_mfma_scale 32x32x64, the
// weights first: a lane holds row lane & 31, columns 8 (j / 4) + 4 (lane / 32) + j % 4).
#ifndef FENCE
#define FENCE __builtin_amdgcn_sched_barrier(0)
#endif
template <int kWM, int kWN, int kMT, int kNT, int kPerCu>
struct Tile {
  static constexpr int PER_CU = kPerCu;  // workgroups on a compute unit
  static constexpr int WM = kWM, WN = kWN, MT = kMT, NT = kNT;
  static constexpr int WAVES = WM * WN, THREADS = WAVES * 64;
  static constexpr int BM = WM * MT * 32, BN = WN * NT * 32;
  static constexpr int A_DMA = BM / 8 / WAVES, B_DMA = BN / 8 / WAVES;  // copies of 8 rows a wave
  static constexpr int S_GROUPS = (BM + BN) / 64;  // of 64 rows' scales, a copy each
  static constexpr int S_DMA = (S_GROUPS + WAVES - 1) / WAVES;  // a wave (the last group's twice)
  static_assert(BM % (8 * WAVES) == 0 && BN % (8 * WAVES) == 0, "whole copies a wave");
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;  // 256 codes of a row
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int WINDOW = (BM + BN) * 16;  // 16 scale bytes of a row
  static constexpr int LDS = 2 * (STAGE + WINDOW);
};

template <class T>
struct Copies {
  i32x4 a_rsrc, b_rsrc, sa_rsrc, sb_rsrc;
  uint32_t a_off[T::A_DMA], b_off[T::B_DMA], s_off[T::S_DMA];
};

// dma16 for the lanes of `due`, all or none (every lane of the wave is at work here).
__device__ __forceinline__ void dma16_if(i32x4 rsrc, uint32_t voff, uint32_t soff, uint32_t lds,
                                         uint32_t due) {
  asm volatile("s_mov_b32 m0, %3\n\ts_mov_b32 exec_lo, %4\n\ts_mov_b32 exec_hi, %4\n\t"
               "s_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds\n\ts_mov_b64 exec, -1"
               :: "v"(voff), "s"(rsrc), "s"(soff), "s"(lds), "s"(due) : "memory", "m0");
}

// Copy j of a wave's A_DMA + B_DMA of step kb, to the stage at LDS address st.
template <class T>
__device__ __forceinline__ void issue_one(const Copies<T>& c, int j, int kb, uint32_t st, int wave,
                                          uint32_t due) {
  if (j < T::A_DMA)
    dma16_if(c.a_rsrc, c.a_off[j], (uint32_t)kb * 128u, st + (wave * T::A_DMA + j) * 1024,
             due);
  else
    dma16_if(c.b_rsrc, c.b_off[j - T::A_DMA], (uint32_t)kb * 128u,
          st + T::A_BYTES + (wave * T::B_DMA + j - T::A_DMA) * 1024, due);
}

// The scales of step kb on (kPerStep bytes of the row a step): 16 bytes from the aligned word
// that holds the first.
template <class T>
__device__ __forceinline__ void issue_scales(const Copies<T>& c, int kb, uint32_t window, int wave,
                                             uint32_t due) {
#pragma unroll
  for (int i = 0; i < T::S_DMA; ++i) {
    // rows 64 g .. of the activations, then of the weights
    const int g = min(wave * T::S_DMA + i, T::S_GROUPS - 1);
    dma16_if(g * 64 < T::BM ? c.sa_rsrc : c.sb_rsrc, c.s_off[i], (uint32_t)kb * 8u,
             window + g * 1024, due);
  }
}

// Where a wave finds its operands in a stage, and its rows' scale bytes in their windows.
template <class T>
struct Place {
  uint32_t ro[4], a_base, b_base;
  int a_row, b_row;  // this lane's first row among the stage's rows
  uint32_t a_shift[T::MT], b_shift;
  uint32_t mask[2];  // of the last step's halves: scale bytes inside the row
  uint32_t lane_shift;
};

// The scale bytes of a row's step, four a half; the two of this lane's blocks at bytes 0 and 2.
template <class T, bool kSplit>
__device__ __forceinline__ void scale_words(const char* window, int row, int odd, uint32_t shift,
                                            const uint32_t (&mask)[2], uint32_t lane_shift,
                                            int (&v)[2]) {
  const uint32_t* p = reinterpret_cast<const uint32_t*>(window) + row * 4;
  u32x2 w;
  if constexpr (kSplit) {
    const u32x4 x = *reinterpret_cast<const u32x4*>(p);
    w = u32x2{__builtin_amdgcn_alignbyte(x.y, x.x, shift), __builtin_amdgcn_alignbyte(x.z, x.y, shift)};
  } else {
    w = *reinterpret_cast<const u32x2*>(p + odd * 2);
  }
  v[0] = (int)((w.x & mask[0]) >> lane_shift);
  v[1] = (int)((w.y & mask[1]) >> lane_shift);
}

template <class T>
struct Frags {
  u32x4 a[T::MT], b[T::NT];
};

template <class T, int M>
__device__ __forceinline__ void load_frags(const char* st, uint32_t ro, const Place<T>& p,
                                           Frags<T>& f) {
  if constexpr (M == 0) return;
#pragma unroll
  for (int m = 0; m < M; ++m)
    f.a[m] = *reinterpret_cast<const u32x4*>(st + p.a_base + m * 4096 + ro);
#pragma unroll
  for (int n = 0; n < T::NT; ++n)
    f.b[n] = *reinterpret_cast<const u32x4*>(st + T::A_BYTES + p.b_base + n * 4096 + ro);
}

// A quarter of a step; `between(m)` runs after each row tile's instructions.
template <class T, int M, int kQuarter, class F>
__device__ __forceinline__ void multiply(const Frags<T>& f, const int (&sa)[T::MT][2],
                                         const int (&sb)[T::NT][2],
                                         f32x16 (&acc)[M ? M : 1][T::NT], F between) {
  constexpr int kHalf = kQuarter / 2, kSel = kQuarter % 2 * 2;
#pragma unroll
  for (int m = 0; m < T::MT; ++m) {
    if constexpr (M > 0) {
      if (m < M) {
#pragma unroll
        for (int n = 0; n < T::NT; ++n)
          acc[m][n] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              codes8(f.b[n]), codes8(f.a[m]), acc[m][n], 4, 4, kSel, sb[n][kHalf], kSel,
              sa[m][kHalf]);
      }
    }
    between(m);
  }
}

// The k loop of a tile for a wave with M row tiles that hold rows.  Step kb (256 of K: whole
// 128-byte lines of the codes' rows) is in stage kb % 2, the scales of one step (kSplit) or two in
// a window of their own.  The barrier of a step stands before its last quarter, where every wave
// has read the stage: the copies of step kb + 2 go there then, among the quarter's products.  A
// copy that is not due is issued for no lane: with a branch in its place the products of
// the whole step were moved behind the barrier.
template <class T, int M, bool kSplit>
__device__ __forceinline__ void kloop(const Copies<T>& c, const Place<T>& p, int nk,
                                      const char* ring, uint32_t ring_at, int wave,
                                      f32x16 (&acc)[M ? M : 1][T::NT]) {
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int n = 0; n < T::NT; ++n)
#pragma unroll
      for (int j = 0; j < 16; ++j) acc[m][n][j] = 0.f;
  wait_vm_barrier<T::A_DMA + T::B_DMA>();  // all but step 1's codes landed
  Frags<T> f0, f1;
  load_frags<T, M>(ring, p.ro[0], p, f0);
  const auto nothing = [](int) {};
  for (int kb = 0; kb < nk; ++kb) {
    const int odd = kb & 1;
    const char* st = ring + odd * T::STAGE;
    const int slot = kSplit ? odd : (kb >> 1) & 1;
    const char* win = ring + 2 * T::STAGE + slot * T::WINDOW;
    int sa[T::MT][2], sb[T::NT][2];
    if constexpr (M > 0) {
      const uint32_t mask[2] = {kb == nk - 1 ? p.mask[0] : ~0u, kb == nk - 1 ? p.mask[1] : ~0u};
#pragma unroll
      for (int m = 0; m < M; ++m)
        scale_words<T, kSplit>(win, p.a_row + m * 32, odd, p.a_shift[m], mask, p.lane_shift, sa[m]);
#pragma unroll
      for (int n = 0; n < T::NT; ++n)
        scale_words<T, kSplit>(win, p.b_row + n * 32, odd, p.b_shift, mask, p.lane_shift, sb[n]);
    }
    load_frags<T, M>(st, p.ro[1], p, f1);
    multiply<T, M, 0>(f0, sa, sb, acc, nothing);
    FENCE;
    load_frags<T, M>(st, p.ro[2], p, f0);
    multiply<T, M, 1>(f1, sa, sb, acc, nothing);
    FENCE;
    load_frags<T, M>(st, p.ro[3], p, f1);
    multiply<T, M, 2>(f0, sa, sb, acc, nothing);
    FENCE;
    wait_vm_barrier<0>();
    FENCE;
    load_frags<T, M>(ring + (odd ^ 1) * T::STAGE, p.ro[0], p, f0);
    const int next = kb + 2;
    const uint32_t due = __builtin_amdgcn_readfirstlane(next < nk ? ~0u : 0u);
    issue_scales<T>(c, next, ring_at + 2 * T::STAGE + (kSplit ? slot : slot ^ 1) * T::WINDOW, wave,
                    kSplit ? due : due & (uint32_t)(odd - 1));
    multiply<T, M, 3>(f1, sa, sb, acc, [&](int m) {
      constexpr int kAll = T::A_DMA + T::B_DMA, kPart = (kAll + T::MT - 1) / T::MT;
#pragma unroll
      for (int j = m * kPart; j < min((m + 1) * kPart, kAll); ++j)
        issue_one<T>(c, j, next, ring_at + odd * T::STAGE, wave, due);
    });
    FENCE;
  }
}

template <int V>
struct Const {
  static constexpr int value = V;
};

// The wave's rows of a tile, from its accumulators, to their places in out.
template <class T, int M, bool kSwiglu, int kOut>
__device__ __forceinline__ void store_tile(const MxGemmArgs& g, const int32_t* orow,
                                           const float* rscale, int rows_valid, int col0, int wm,
                                           int wn, int n32, int g2,
                                           const f32x16 (&acc)[M][T::NT]) {
  const int ncols = kSwiglu ? g.N >> 1 : g.N;
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const int trow = (wm * T::MT + m) * 32 + n32;
    if (trow >= rows_valid) continue;
    const int64_t o = orow[trow];
    if (o < 0 || o >= g.out_rows) continue;
    const float rs = rscale[trow];
    constexpr int NTO = kSwiglu ? T::NT / 2 : T::NT;
#pragma unroll
    for (int n = 0; n < NTO; ++n) {
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
        const int col = col0 + (wn * NTO + n) * 32 + 8 * jj + 4 * g2;
        if (col >= ncols) continue;
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = 4 * jj + i;
          if constexpr (kSwiglu) v[i] = silu_f(acc[m][n][j]) * acc[m][n + NTO][j] * rs;
          else v[i] = acc[m][n][j] * rs;
        }
        store4<kOut>(g.out, o * ncols + col, v);
      }
    }
  }
}

}  // namespace

template <class T, bool kSwiglu, int kOut, bool kSplit>
__global__ __launch_bounds__(T::THREADS, T::PER_CU) void mx_tile_kernel(MxGemmArgs g, int n_tiles) {
  __shared__ __attribute__((aligned(1024))) char ring[T::LDS];
  __shared__ int32_t tiles[kMaxExperts + 1];
  __shared__ int32_t wsum[T::WAVES];
  __shared__ int32_t orow[2][T::BM];
  __shared__ float rscale[2][T::BM];
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / T::WN, wn = wave % T::WN;
  const int n32 = lane & 31, g2 = lane >> 5;
  build_tile_table<T::THREADS, T::BM>(g.offsets, g.E, tiles, wsum, tid);

  const int N = g.N, I = N >> 1, KB = g.K / 32;
  const int nk = (KB + 7) / 8;
  const uint32_t row_bytes = (uint32_t)KB * 16u;
  Place<T> p;
#pragma unroll
  for (int q = 0; q < 4; ++q) p.ro[q] = n32 * 128 + (((2 * q + g2) ^ (n32 & 7)) << 4);
  p.a_base = (uint32_t)wm * T::MT * 4096;
  p.b_base = (uint32_t)wn * T::NT * 4096;
  p.a_row = wm * T::MT * 32 + n32;
  p.b_row = T::BM + wn * T::NT * 32 + n32;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int inside = KB - (nk - 1) * 8 - 4 * h;  // scale bytes of the last step's half
    p.mask[h] = inside >= 4 ? ~0u : inside > 0 ? (1u << (8 * inside)) - 1u : 0u;
  }
  p.lane_shift = 8 * g2;
  constexpr int kCols = kSwiglu ? T::BN / 2 : T::BN;  // output columns of a tile

  // weight row of LDS row l, clamped to a valid one.  SwiGLU: of a wave's NT groups of 32 the
  // first half are gate rows, the others the up rows of the same columns.
  auto weight_row = [&](int l, int n_idx) -> int {
    if constexpr (kSwiglu) {
      constexpr int H = T::NT / 2;
      const int w = l / (T::NT * 32), nt = (l >> 5) % T::NT, n = l & 31;
      const int col = n_idx * kCols + (w * H + nt % H) * 32 + n;
      return min(col, I - 1) + (nt >= H ? I : 0);
    } else {
      return min(n_idx * T::BN + l, N - 1);
    }
  };
  // scales are read as aligned words: byte offsets from the array's start rounded down
  auto scale_rsrc = [&](const uint8_t* p, int64_t bytes, uint32_t& skip) -> i32x4 {
    skip = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 3);
    return make_rsrc(p - skip, ((uint32_t)bytes + skip + 3u) & ~3u);
  };

  Copies<T> c;
  uint32_t a_skip, b_skip;
  c.a_rsrc = make_rsrc(g.a, (uint32_t)g.a_rows * row_bytes);
  c.sa_rsrc = scale_rsrc(g.a_scales, g.a_rows * KB, a_skip);
  const int total_m = __builtin_amdgcn_readfirstlane(tiles[g.E]);
  const int total = total_m * n_tiles;
  const int G = gridDim.x;  // a multiple of 8
  const int u = (blockIdx.x & 7) * (G >> 3) + (blockIdx.x >> 3);
  const uint32_t ring_at = lds_addr(ring);
  for (int r = 0;; ++r) {
    const int tix = r * G + u;
    if (tix >= total) break;
    // groups of four row tiles, the row tile changing fastest
    const int group = tix / (4 * n_tiles), in = tix - group * 4 * n_tiles;
    const int gm = min(4, total_m - group * 4);
    const int n_idx = in / gm, mt_global = group * 4 + (in - n_idx * gm);
    int lo = 0, hi = g.E;  // tiles[lo] <= mt_global < tiles[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tiles[mid] <= mt_global) lo = mid; else hi = mid;
    }
    const int e = __builtin_amdgcn_readfirstlane(lo);
    const int m_local = mt_global - __builtin_amdgcn_readfirstlane(tiles[e]);
    const int row0 = __builtin_amdgcn_readfirstlane(g.offsets[e]) + m_local * T::BM;
    const int end = min(__builtin_amdgcn_readfirstlane(g.offsets[e + 1]), (int)g.P);
    const int rows_valid = min(T::BM, end - row0);
    if (rows_valid <= 0) continue;  // behind P
    const int mtv = max(0, min(T::MT, (rows_valid - wm * T::MT * 32 + 31) >> 5));

    auto source = [&](int row) -> uint32_t {
      const int idx = row0 + (row < rows_valid ? row : 0);
      const int s = g.gather ? g.gather[idx] / g.gather_div : idx;
      return (uint32_t)min(max(s, 0), (int)g.a_rows - 1);
    };
    const int64_t w_at = (int64_t)e * N;
    c.b_rsrc = make_rsrc(g.blocks + w_at * row_bytes, (uint32_t)N * row_bytes);
    c.sb_rsrc = scale_rsrc(g.scales + w_at * KB, (int64_t)N * KB, b_skip);
#pragma unroll
    for (int i = 0; i < T::A_DMA; ++i) {
      const int row = (wave * T::A_DMA + i) * 8 + (lane >> 3);
      c.a_off[i] = source(row) * row_bytes + (((lane & 7) ^ (row & 7)) << 4);
    }
#pragma unroll
    for (int i = 0; i < T::B_DMA; ++i) {
      const int l = (wave * T::B_DMA + i) * 8 + (lane >> 3);
      c.b_off[i] = (uint32_t)weight_row(l, n_idx) * row_bytes + (((lane & 7) ^ (l & 7)) << 4);
    }
#pragma unroll
    for (int i = 0; i < T::S_DMA; ++i) {
      const int l = min(wave * T::S_DMA + i, T::S_GROUPS - 1) * 64 + lane;
      c.s_off[i] = (l < T::BM ? source(l) * (uint32_t)KB + a_skip
                              : (uint32_t)weight_row(l - T::BM, n_idx) * (uint32_t)KB + b_skip) & ~3u;
    }
    // where in its first word a row's scales begin; the same for all of a lane's weight rows
    if constexpr (kSplit) {
#pragma unroll
      for (int m = 0; m < T::MT; ++m)
        p.a_shift[m] = (source((wm * T::MT + m) * 32 + n32) * (uint32_t)KB + a_skip) & 3u;
      p.b_shift = ((uint32_t)weight_row(wn * T::NT * 32 + n32, n_idx) * (uint32_t)KB + b_skip) & 3u;
    }
    const int par = r & 1;
    for (int l = tid; l < T::BM; l += T::THREADS) {
      const int row = row0 + (l < rows_valid ? l : 0);
      orow[par][l] = g.scatter ? g.scatter[row] : row;
      rscale[par][l] = g.row_scale ? g.row_scale[row] : 1.0f;
    }

    // every wave is done with the previous tile's ring
    lds_barrier();
    issue_scales<T>(c, 0, ring_at + 2 * T::STAGE, wave, ~0u);
    if (kSplit) issue_scales<T>(c, min(1, nk - 1), ring_at + 2 * T::STAGE + T::WINDOW, wave, ~0u);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < T::A_DMA + T::B_DMA; ++j)
        issue_one<T>(c, j, min(i, nk - 1), ring_at + i * T::STAGE, wave, ~0u);
    auto tile = [&](auto rows) {
      constexpr int M = decltype(rows)::value;
      f32x16 acc[M ? M : 1][T::NT];
      kloop<T, M, kSplit>(c, p, nk, ring, ring_at, wave, acc);
      if constexpr (M > 0)
        store_tile<T, M, kSwiglu, kOut>(g, orow[par], rscale[par], rows_valid, n_idx * kCols, wm,
                                        wn, n32, g2, acc);
    };
    if (mtv > T::MT / 2) tile(Const<T::MT>{});
    else if (T::MT > 2 && mtv == 2) tile(Const<T::MT / 2>{});
    else if (mtv == 1) tile(Const<1>{});
    else tile(Const<0>{});
  }
  // no copy of the wave is left in flight when it ends
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

namespace {

template <bool kSwiglu>
void launch_small(const MxGemmArgs& g, dim3 grid, int n_tiles, hipStream_t s) {
  if (g.out_dtype == kF32)
    hipLaunchKernelGGL((mx_small_kernel<kSwiglu, kF32>), grid, dim3(kThreads), 0, s, g, n_tiles);
  else if (g.out_dtype == kBF16)
    hipLaunchKernelGGL((mx_small_kernel<kSwiglu, kBF16>), grid, dim3(kThreads), 0, s, g, n_tiles);
  else
    hipLaunchKernelGGL((mx_small_kernel<kSwiglu, kF16>), grid, dim3(kThreads), 0, s, g, n_tiles);
}

template <class T, bool kSwiglu, bool kSplit>
void launch_tile(const MxGemmArgs& g, dim3 grid, int n_tiles, hipStream_t s) {
  if (g.out_dtype == kF32)
    hipLaunchKernelGGL((mx_tile_kernel<T, kSwiglu, kF32, kSplit>), grid, dim3(T::THREADS), 0, s, g, n_tiles);
  else if (g.out_dtype == kBF16)
    hipLaunchKernelGGL((mx_tile_kernel<T, kSwiglu, kBF16, kSplit>), grid, dim3(T::THREADS), 0, s, g, n_tiles);
  else
    hipLaunchKernelGGL((mx_tile_kernel<T, kSwiglu, kF16, kSplit>), grid, dim3(T::THREADS), 0, s, g, n_tiles);
}

template <class T>
void launch_tiles(const MxGemmArgs& g, int num_cus, hipStream_t s) {
  const int cols = g.swiglu ? T::BN / 2 : T::BN;
  const int n_tiles = ((g.swiglu ? g.N / 2 : g.N) + cols - 1) / cols;
  const int64_t tiles = ((g.P + T::BM - 1) / T::BM + std::min<int64_t>(g.E, g.P)) * n_tiles;
  const dim3 grid((unsigned)((std::min<int64_t>(tiles, num_cus * T::PER_CU) + 7) / 8 * 8));
  const bool split = g.K % 128 || (reinterpret_cast<uintptr_t>(g.a_scales) & 3) ||
                     (reinterpret_cast<uintptr_t>(g.scales) & 3);
  if (g.swiglu) {
    if (split) launch_tile<T, true, true>(g, grid, n_tiles, s);
    else launch_tile<T, true, false>(g, grid, n_tiles, s);
  } else {
    if (split) launch_tile<T, false, true>(g, grid, n_tiles, s);
    else launch_tile<T, false, false>(g, grid, n_tiles, s);
  }
}

#ifndef TILE_BIG
#define TILE_BIG 4, 2, 2, 4, 1
#endif
using Tile256 = Tile<TILE_BIG>;  // 256 x 256
#ifndef TILE_SMALL
#define TILE_SMALL 2, 2, 1, 2, 2
#endif
using Tile64 = Tile<TILE_SMALL>;

}  // namespace

hipError_t launch_mx_gemm(const MxGemmArgs& g, int num_cus, hipStream_t s) {
  const int64_t rows = g.P / std::min<int64_t>(g.E, g.P);  // of an expert, at least
  if (rows >= 128) {
    launch_tiles<Tile256>(g, num_cus, s);
    return hipGetLastError();
  }
  if (rows >= 24) {
    launch_tiles<Tile64>(g, num_cus, s);
    return hipGetLastError();
  }
  const int n_tiles = g.swiglu ? (g.N / 2 + 15) / 16 : (g.N + 31) / 32;
  // an expert's rows begin a tile of their own: at most one more for each that has rows
  const int64_t tiles = ((g.P + 15) / 16 + std::min<int64_t>(g.E, g.P)) * n_tiles;
  const dim3 grid((unsigned)std::min<int64_t>(tiles, num_cus * 8));
  if (g.swiglu) launch_small<true>(g, grid, n_tiles, s);
  else launch_small<false>(g, grid, n_tiles, s);
  return hipGetLastError();
}

}  // namespace nf4moe
