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
//
// Three ways, by the rows an expert has (rules and both sides' figures at the launchers): 16-row
// tiles of one launch that makes the rows' blocks too; 64 x 128 tiles, which stream the weights at
// the rate of a large copy; 256 x 256 tiles.  Measured (kernels alone, blocks of the rows made before
// but for the first): one token, 8 of 64 experts, gate and up of H 2048 I 1024 7.3-8.0 us; 64 tokens
// 28.9 us = 4.97 TB/s; 4096 tokens 101-103 us = 2.7 PFLOP/s; one 8192 x 8192 matrix, 8192
// rows 261-268 us = 4.1-4.2 PFLOP/s (a 16-bit library product of the size reaches 1.43).

#include <algorithm>

#include "common.h"
#include "launch.h"
#include "mfma_common.h"
#include "mx_common.h"

namespace nf4moe {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kWaves = 4;
constexpr int kThreads = kWaves * 64;

// Two values rounded to the nearest 16-bit ones.
template <int kOut>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (kOut == kBF16) return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
  else return pack_half2((_Float16)a, (_Float16)b);
}

// build_tile_table with the rows at and beyond P left out; rows[e] is expert e's first row.
template <int kThreads, int kBM>
__device__ __forceinline__ void build_tiles(const int32_t* __restrict__ offsets, int E, int P,
                                            int32_t* tiles, int32_t* rows, int32_t* wsum, int tid) {
  constexpr int kPer = kMaxExperts / kThreads;
  const int lane = tid & 63, wave = tid >> 6;
  int32_t cnt[kPer];
  int32_t local = 0;
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int ex = tid * kPer + u;
    cnt[u] = 0;
    if (ex < E) {
      const int from = max(0, min(offsets[ex], P)), to = max(from, min(offsets[ex + 1], P));
      cnt[u] = (to - from + kBM - 1) / kBM;
      rows[ex] = from;
      if (ex == E - 1) rows[E] = to;
    }
    local += cnt[u];
  }
  int32_t incl = local;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int32_t v = __shfl_up(incl, off, 64);
    if (lane >= off) incl += v;
  }
  if (lane == 63) wsum[wave] = incl;
  __syncthreads();
  int32_t run = incl - local;
  for (int w = 0; w < wave; ++w) run += wsum[w];
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int ex = tid * kPer + u;
    if (ex < E) tiles[ex] = run;
    run += cnt[u];
  }
  if (tid == kThreads - 1) tiles[E] = run;
  __syncthreads();
}

__device__ __forceinline__ i32x8 codes8(u32x4 v) {
  return i32x8{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
}

}  // namespace

// 16 rows of one expert by 32 weight rows (SwiGLU: 16 gate and their 16 up rows) a workgroup.  Of
// every 4096 of K a wave takes four runs of 256 (whole lines of the codes, eight scale bytes at
// a time), whose reads are all in flight while the workgroup lays the rows' blocks into LDS; the
// waves join in LDS.  kA: the activations' type, or kCodes for blocks made before: making them
// here costs one launch less.
constexpr int kCodes = 3;
constexpr int kSmallRows = 32;  // P of a call, at most
constexpr int kChunk = 128;     // blocks of K at a time
constexpr int kRuns = kChunk / 8 / kWaves;
constexpr int kRowBytes = kChunk * 16 + 16;  // of a row's codes in LDS: 16 rows on 16 bank groups

template <int kA>
struct ABlock {
  Eight<kA> v[4];
};
template <>
struct ABlock<kCodes> {
  u32x4 c;
  uint8_t s;
};

template <int kA>
__device__ __forceinline__ void load_block(const MxGemmArgs& g, int64_t block, ABlock<kA>& o) {
  if constexpr (kA == kCodes) {
    o.c = reinterpret_cast<const u32x4*>(g.a)[block];
    o.s = g.a_scales[block];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) load_eight<kA>(g.a, block * 4 + i, o.v[i]);
  }
}

template <int kA>
__device__ __forceinline__ u32x4 block_codes(const ABlock<kA>& x, int& scale) {
  if constexpr (kA == kCodes) {
    scale = x.s;
    return x.c;
  } else {
    uint32_t top = max(max(eight_top<kA>(x.v[0]), eight_top<kA>(x.v[1])),
                       max(eight_top<kA>(x.v[2]), eight_top<kA>(x.v[3])));
    if constexpr (kA != kF32) top = wide_bits<kA>(top);
    const uint32_t byte = scale_byte(top);
    const float s = scale_value(byte);
    scale = (int)byte;
    u32x4 c;
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = byte == 255u ? 0u : eight_codes<kA>(x.v[i], s);
    return c;
  }
}

// The expert, first row and rows of 16-row tile mt, by one wave: 64 experts at a time, a lane's tiles
// counted over the lanes below it by ballots (an expert has at most kSmallRows / 16).  False
// behind the last tile.
__device__ __forceinline__ bool find_tile(const int32_t* __restrict__ offsets, int E, int P, int mt,
                                          int lane, int& e, int& row0, int& rows) {
  int before = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int ex = e0 + lane;
    const int from = max(0, min(ex < E ? offsets[ex] : P, P));
    const int to = max(from, min(ex < E ? offsets[ex + 1] : P, P));
    const int n = (to - from + 15) / 16;
    int below = before, all = 0;
#pragma unroll
    for (int k = 1; k <= kSmallRows / 16; ++k) {
      const uint64_t has = __ballot(n >= k);
      below += __builtin_amdgcn_mbcnt_hi((uint32_t)(has >> 32),
                                         __builtin_amdgcn_mbcnt_lo((uint32_t)has, 0));
      all += __popcll(has);
    }
    if (mt < before + all) {
      const uint64_t mine = __ballot(mt >= below && mt < below + n);
      const int l = __ffsll((unsigned long long)mine) - 1;
      e = e0 + l;
      row0 = __builtin_amdgcn_readlane(from, l) + (mt - __builtin_amdgcn_readlane(below, l)) * 16;
      rows = min(16, __builtin_amdgcn_readlane(to, l) - row0);
      return true;
    }
    before += all;
  }
  return false;
}

// The scale bytes of blocks b0 .. b0 + 7 of a row of KB; 0 behind the row's end.
__device__ __forceinline__ uint64_t run_scales(const uint8_t* row, int b0, int KB) {
  uint64_t v = 0;
  if (KB >= 8) {
    // eight bytes at any place, none behind the row
    const int from = min(b0, KB - 8);
    __builtin_memcpy(&v, row + from, 8);
    return v >> (8 * (b0 - from));
  }
  for (int i = 0; i < KB; ++i) v |= (uint64_t)row[i] << (8 * i);
  return v;
}

template <bool kSwiglu, int kOut, int kA>
__global__ __launch_bounds__(kThreads) void mx_small_kernel(MxGemmArgs g, int n_tiles) {
  __shared__ __attribute__((aligned(16))) char s_codes[16 * kRowBytes];
  __shared__ uint8_t s_scales[16 * kChunk];
  __shared__ int32_t s_src[16];
  __shared__ float s_part[kWaves][2][16][17];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, q = lane >> 4;
  const int N = g.N, I = N >> 1, KB = g.K / 32;
  for (int tix = blockIdx.x;; tix += gridDim.x) {
    const int mt = tix / n_tiles, nt = tix - mt * n_tiles;
    int e, row0, rows;
    if (!find_tile(g.offsets, g.E, (int)g.P, mt, lane, e, row0, rows)) break;
    if (tid < 16) {
      const int row = row0 + min(tid, rows - 1);
      const int s = g.gather ? g.gather[row] / g.gather_div : row;
      s_src[tid] = min(max(s, 0), (int)g.a_rows - 1);
    }
    // weight rows of the tile's two halves, clamped to valid ones
    int64_t w_block[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int n = kSwiglu ? min(nt * 16 + r16, I - 1) + h * I : min(nt * 32 + h * 16 + r16, N - 1);
      w_block[h] = ((int64_t)e * N + n) * KB;
    }
    f32x4 acc[2] = {};
    for (int c0 = 0; c0 < KB; c0 += kChunk) {
      u32x4 w[kRuns][2][2];
      uint64_t sw[kRuns][2];
#pragma unroll
      for (int i = 0; i < kRuns; ++i) {
        const int b0 = c0 + (i * kWaves + wave) * 8;
        if (b0 >= KB) break;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
            w[i][h][j] = reinterpret_cast<const u32x4*>(g.blocks)[w_block[h] + min(b0 + 4 * j + q, KB - 1)];
          sw[i][h] = run_scales(g.scales + w_block[h], b0, KB);
        }
      }
      __syncthreads();  // s_src is there, the last chunk is read
      const int here = min(kChunk, KB - c0);
      for (int x = tid; x < rows * here; x += kThreads) {
        const int r = x / here, b = x - r * here;
        ABlock<kA> v;
        load_block<kA>(g, (int64_t)s_src[r] * KB + c0 + b, v);
        int scale;
        *reinterpret_cast<u32x4*>(s_codes + r * kRowBytes + b * 16) = block_codes<kA>(v, scale);
        s_scales[r * kChunk + b] = (uint8_t)scale;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kRuns; ++i) {
        const int b0 = c0 + (i * kWaves + wave) * 8;
        if (b0 >= KB) break;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          // rows behind the last multiply what lies in LDS; their results are not stored
          const int b = b0 + 4 * j + q;
          const u32x4 av = *reinterpret_cast<const u32x4*>(s_codes + r16 * kRowBytes + (b - c0) * 16);
          const int sa = b < KB ? s_scales[r16 * kChunk + b - c0] : 0;
          // the weights first: a lane's four sums are consecutive output columns
#pragma unroll
          for (int h = 0; h < 2; ++h)
            acc[h] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                codes8(w[i][h][j]), codes8(av), acc[h], 4, 4, 0,
                (int)(sw[i][h] >> (8 * (4 * j + q))) & 255, 0, sa);
        }
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
    if (r >= rows) continue;
    float v[2] = {0.f, 0.f};
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v[h] += s_part[w][h][r][c];
    {
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
//
// 256 x 256 (144 KB of LDS) because the copies bound it: a step of 256 of K brings 64 KB of codes
// from the L2 to a compute unit for 2048 cycles of matrix instructions.  8192^3 takes 261-268 us; with
// copies that hit the first-level cache 205, without any copy 169.  Waiting for the copies is not
// what they cost (without the waits nothing is gained): the L2s deliver 12 TB/s then, at 1.9 GHz,
// with the matrix units busy 49 % of the time.  Four waves of 128 x 128 each were slower than eight
// of 64 x 128 (316 against 299 us in one run, of an earlier state of both).

namespace {

// A tile: WM x WN waves, each MT x NT accumulator tiles of 32 x 32 (v_mfma_scale 32x32x64: a lane
// holds column lane & 31 of rows 8 (j / 4) + 4 (lane / 32) + j % 4).  The weight rows are laid out
// so that a lane's NT columns are neighbours: a row's results leave as whole lines.
template <int kWM, int kWN, int kMT, int kNT, int kPerCu>
struct Tile {
  static constexpr int PER_CU = kPerCu;  // workgroups on a compute unit
  static constexpr int WM = kWM, WN = kWN, MT = kMT, NT = kNT;
  static constexpr int WAVES = WM * WN, THREADS = WAVES * 64;
  static constexpr int BM = WM * MT * 32, BN = WN * NT * 32;
  static constexpr int A_DMA = BM / 8 / WAVES, B_DMA = BN / 8 / WAVES;  // copies of 8 rows a wave
  static constexpr int S_GROUPS = (BM + BN) / 64;  // of 64 rows' scales, a copy each
  static constexpr int S_DMA = (S_GROUPS + WAVES - 1) / WAVES;  // a wave (the last group's twice)
  static_assert(MT <= 2, "a wave has all, one or none of its row tiles");
  static_assert(BM % (8 * WAVES) == 0 && BM % 64 == 0, "whole copies a wave");
  static_assert(32 % (B_DMA * 8) == 0, "a wave copies rows of one group of 32 weight rows");
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;  // 256 codes of a row
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int WINDOW = (BM + BN) * 16;  // 16 scale bytes of a row
  static constexpr int LDS = 2 * (STAGE + WINDOW);
};

constexpr int kDescs = 32;  // tiles of a workgroup that are looked up at a time

// Which rows and columns a tile has.
struct TileDesc {
  int e, row0, rows, n_idx;
};

// What a wave copies: offsets of its lanes in the arrays at step 0 of a tile.
template <class T>
struct Copies {
  i32x4 a_rsrc, b_rsrc, sa_rsrc, sb_rsrc;
  uint32_t a_off[T::A_DMA], b_off[2], s_off[T::S_DMA];  // b_off: even and odd copies
};

// The weight copies of a step that are issued in the next one's first half.
struct Pending {
  i32x4 rsrc;
  uint32_t off[2], where;
  int kb;
};

// The value of every lane, for a scalar register.
__device__ __forceinline__ int scalar(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ i32x4 scalar(i32x4 v) {
  return i32x4{scalar(v.x), scalar(v.y), scalar(v.z), scalar(v.w)};
}

// dma16 and dma4 with the resource and the place in scalar registers, wherever they are.
__device__ __forceinline__ void copy16(i32x4 rsrc, uint32_t voff, uint32_t lds) {
  dma16(scalar(rsrc), voff, 0, (uint32_t)scalar((int)lds));
}
__device__ __forceinline__ void copy4(i32x4 rsrc, uint32_t voff, uint32_t lds) {
  dma4(scalar(rsrc), voff, 0, (uint32_t)scalar((int)lds));
}

// An offset that no array has: a copy from there writes zeros and reads no memory.
constexpr uint32_t kNowhere = 0xf0000000u;

// Copy j of a wave's A_DMA and of its B_DMA, to the stage at LDS address st.  Bounds are checked on
// the lane's offset alone, so it is the whole one; `where` is 0 or kNowhere.  A lane's weight rows
// are b_step bytes apart.
template <class T>
__device__ __forceinline__ void issue_a(const Copies<T>& c, int j, int kb, uint32_t st, int wave,
                                        uint32_t where) {
  copy16(c.a_rsrc, (c.a_off[j] + (uint32_t)kb * 128u) | where, st + (wave * T::A_DMA + j) * 1024);
}
template <class T>
__device__ __forceinline__ void issue_b(const Pending& d, int j, uint32_t b_step, uint32_t st,
                                        int wave) {
  copy16(d.rsrc, (d.off[j & 1] + ((uint32_t)j * b_step + (uint32_t)d.kb * 128u)) | d.where,
        st + T::A_BYTES + (wave * T::B_DMA + j) * 1024);
}

// The scales of step kb on (eight bytes of the row a step): 16 bytes from the aligned word that
// holds the first.
template <class T>
__device__ __forceinline__ void issue_scales(const Copies<T>& c, int kb, uint32_t window, int wave,
                                             uint32_t trash, uint32_t where) {
#pragma unroll
  for (int i = 0; i < T::S_DMA; ++i) {
    // rows 64 g .. of the activations, then of the weights
    const int g = min(wave * T::S_DMA + i, T::S_GROUPS - 1);
    copy16(g * 64 < T::BM ? c.sa_rsrc : c.sb_rsrc, (c.s_off[i] + (uint32_t)kb * 8u) | where,
          where ? trash : window + g * 1024);
  }
}

// Where a wave finds its operands in a stage, and its rows' scale bytes in their windows.
template <class T>
struct Place {
  uint32_t ro[4], a_base, b_base;
  int a_row, b_row;  // this lane's first row among the stage's rows
  uint32_t a_shift[T::MT], b_shift[T::NT];
  uint32_t mask[2];  // of the last step's halves: scale bytes inside the row
  int last;          // that step
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
              codes8(f.a[m]), codes8(f.b[n]), acc[m][n], 4, 4, kSel, sa[m][kHalf], kSel,
              sb[n][kHalf]);
      }
    }
    between(m);
  }
}

// The k loop of a tile for a wave with M row tiles that hold rows.  Step kb (256 of K: whole
// 128-byte lines of the codes' rows) is in the stage of its parity, counted on over the tiles, the
// scales of one step (kSplit) or two in a window of their own.  The barrier of a step stands before
// its last quarter, where every wave has read the stage: the copies of the step after next go
// there then, the activations' among the quarter's products, the weights' among those of the next
// step's first half (all in one quarter kept the waves from their products: the copies' addresses
// take the compute unit 16 cycles each).  At the end of a tile they are those of the next
// tile's first steps, for which `next_copies` changes c.  A copy that is not due comes from nowhere:
// with a branch in its place the products of the whole step were moved behind the barrier.
template <class T, int M, bool kSplit, class F>
__device__ __forceinline__ void kloop(Copies<T>& c, Pending& d, const Place<T>& p, int nk,
                                      uint32_t b_step,
                                      const char* ring, uint32_t ring_at, int wave, int& stage_,
                                      int& window_, bool more, F next_copies,
                                      f32x16 (&acc)[M ? M : 1][T::NT]) {
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int n = 0; n < T::NT; ++n)
#pragma unroll
      for (int j = 0; j < 16; ++j) acc[m][n][j] = 0.f;
  Frags<T> f0, f1;
  load_frags<T, M>(ring + scalar(stage_) * T::STAGE, p.ro[0], p, f0);
  const auto nothing = [](int) {};
  const auto part = [](int m, int n) { return n * m / T::MT; };
  for (int kb = 0; kb < nk; ++kb) {
    if (kb == nk - 2) next_copies();
    const int stage = scalar(stage_), window = scalar(window_);
    const char* st = ring + stage * T::STAGE;
    const char* win = ring + 2 * T::STAGE + window * T::WINDOW;
    int sa[T::MT][2], sb[T::NT][2];
    if constexpr (M > 0) {
      const int left = p.last - kb;  // a step behind the last has no scales
      const uint32_t mask[2] = {left > 0 ? ~0u : left ? 0u : p.mask[0],
                                left > 0 ? ~0u : left ? 0u : p.mask[1]};
#pragma unroll
      for (int m = 0; m < M; ++m)
        scale_words<T, kSplit>(win, p.a_row + m * 32, kb & 1, p.a_shift[m], mask, p.lane_shift, sa[m]);
#pragma unroll
      for (int n = 0; n < T::NT; ++n)
        scale_words<T, kSplit>(win, p.b_row + n * 32, kb & 1, p.b_shift[n], mask, p.lane_shift, sb[n]);
    }
    const uint32_t other = ring_at + (stage ^ 1) * T::STAGE;
    load_frags<T, M>(st, p.ro[1], p, f1);
    multiply<T, M, 0>(f0, sa, sb, acc, [&](int m) {
#pragma unroll
      for (int j = part(m, T::B_DMA / 2); j < part(m + 1, T::B_DMA / 2); ++j)
        issue_b<T>(d, j, b_step, other, wave);
    });
    __builtin_amdgcn_sched_barrier(0);
    load_frags<T, M>(st, p.ro[2], p, f0);
    multiply<T, M, 1>(f1, sa, sb, acc, [&](int m) {
#pragma unroll
      for (int j = part(m, T::B_DMA - T::B_DMA / 2); j < part(m + 1, T::B_DMA - T::B_DMA / 2); ++j)
        issue_b<T>(d, j + T::B_DMA / 2, b_step, other, wave);
    });
    __builtin_amdgcn_sched_barrier(0);
    load_frags<T, M>(st, p.ro[3], p, f1);
    multiply<T, M, 2>(f0, sa, sb, acc, nothing);
    __builtin_amdgcn_sched_barrier(0);
    wait_vm_barrier<0>();
    __builtin_amdgcn_sched_barrier(0);
    load_frags<T, M>(ring + (stage ^ 1) * T::STAGE, p.ro[0], p, f0);
    const int ahead = kb + 2 < nk ? kb + 2 : kb + 2 - nk;
    const uint32_t where = scalar(kb + 2 < nk || more ? 0 : (int)kNowhere);
    // a window read for the last time gives its place (an odd step); at an even one the other
    // window's is free
    const int slot = kSplit || (kb & 1) ? window : window ^ 1;
    issue_scales<T>(c, ahead, ring_at + 2 * T::STAGE + slot * T::WINDOW, wave,
                    ring_at + T::LDS, kSplit || !(ahead & 1) ? where : kNowhere);
    multiply<T, M, 3>(f1, sa, sb, acc, [&](int m) {
#pragma unroll
      for (int j = part(m, T::A_DMA); j < part(m + 1, T::A_DMA); ++j)
        issue_a<T>(c, j, ahead, ring_at + stage * T::STAGE, wave, where);
    });
    d = Pending{c.b_rsrc, {c.b_off[0], c.b_off[1]}, where, ahead};
    __builtin_amdgcn_sched_barrier(0);
    stage_ = stage ^ 1;
    window_ = kSplit || (kb & 1) || kb == nk - 1 ? window ^ 1 : window;
  }
}

template <int V>
struct Const {
  static constexpr int value = V;
};

// N neighbouring values.
template <int kOut, int N>
__device__ __forceinline__ void store_run(void* out, int64_t at, const float (&v)[N]) {
  if constexpr (kOut == kF32) {
    float* p = reinterpret_cast<float*>(out) + at;
    if constexpr (N == 4) *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
    else if constexpr (N == 2) *reinterpret_cast<f32x2*>(p) = f32x2{v[0], v[1]};
    else p[0] = v[0];
  } else {
    uint16_t* p = reinterpret_cast<uint16_t*>(out) + at;
    if constexpr (N == 4)
      *reinterpret_cast<u32x2*>(p) = u32x2{pack2<kOut>(v[0], v[1]), pack2<kOut>(v[2], v[3])};
    else if constexpr (N == 2) *reinterpret_cast<uint32_t*>(p) = pack2<kOut>(v[0], v[1]);
    else p[0] = (uint16_t)pack2<kOut>(v[0], 0.f);
  }
}

// The results of row j of row tile m: its C columns.
template <class T, int M, bool kSwiglu, int C>
__device__ __forceinline__ void row_of(const f32x16 (&acc)[M][T::NT], int m, int j, float (&v)[C]) {
#pragma unroll
  for (int n = 0; n < C; ++n) {
    if constexpr (kSwiglu) v[n] = silu_f(acc[m][n][j]) * acc[m][n + C][j];
    else v[n] = acc[m][n][j];
  }
}

// The wave's rows of a tile, from its accumulators, to their places in out.
template <class T, int M, bool kSwiglu, int kOut>
__device__ __forceinline__ void store_tile(const MxGemmArgs& g, const TileDesc& d,
                                           const int32_t* orow, const float* rscale, int wm,
                                           int wn, int n32, int g2,
                                           const f32x16 (&acc)[M][T::NT]) {
  constexpr int C = kSwiglu ? T::NT / 2 : T::NT;  // columns of a lane
  const int ncols = kSwiglu ? g.N >> 1 : g.N;
  const int col0 = (d.n_idx * T::WN + wn) * 32 * C, row0 = wm * T::MT * 32;
  if (!g.scatter && !g.row_scale && row0 + M * 32 <= d.rows && col0 + 32 * C <= ncols &&
      d.row0 + d.rows <= g.out_rows) {
    // whole and in order: the rows' places follow from a scalar, the lane's part is the same
    constexpr int kSize = kOut == kF32 ? 4 : 2;
    const uint32_t lane_at = (uint32_t)(4 * g2 * ncols + n32 * C) * kSize;
    char* at = reinterpret_cast<char*>(g.out) + ((int64_t)(d.row0 + row0) * ncols + col0) * kSize;
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        float v[C];
        row_of<T, M, kSwiglu, C>(acc, m, j, v);
        store_run<kOut, C>(at + (int64_t)(m * 32 + 8 * (j / 4) + j % 4) * ncols * kSize + lane_at, 0, v);
      }
    return;
  }
  const int col = col0 + n32 * C;
  if (col >= ncols) return;  // ncols is a multiple of 16: all of a lane's columns or none
#pragma unroll
  for (int m = 0; m < M; ++m) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int trow = row0 + m * 32 + 8 * q + 4 * g2;
      i32x4 o = i32x4{0, 1, 2, 3} + (d.row0 + trow);
      f32x4 rs = {1.f, 1.f, 1.f, 1.f};
      if (g.scatter) o = *reinterpret_cast<const i32x4*>(orow + trow);
      if (g.row_scale) rs = *reinterpret_cast<const f32x4*>(rscale + trow);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (trow + i >= d.rows || o[i] < 0 || o[i] >= g.out_rows) continue;
        float v[C];
        row_of<T, M, kSwiglu, C>(acc, m, 4 * q + i, v);
#pragma unroll
        for (int n = 0; n < C; ++n) v[n] *= rs[i];
        store_run<kOut, C>(g.out, (int64_t)o[i] * ncols + col, v);
      }
    }
  }
}

}  // namespace

template <class T, bool kSwiglu, int kOut, bool kSplit>
__global__ __launch_bounds__(T::THREADS, T::PER_CU) void mx_tile_kernel(MxGemmArgs g, int n_tiles) {
  __shared__ __attribute__((aligned(1024))) char ring[T::LDS + 1024];  // with a place for copies of nothing
  __shared__ __attribute__((aligned(16))) int32_t srow[2][T::BM];   // gather entry of each row
  __shared__ __attribute__((aligned(16))) int32_t orow[2][T::BM];   // and its scatter entry
  __shared__ __attribute__((aligned(16))) float rscale[2][T::BM];   // and row scale
  __shared__ TileDesc descs[kDescs];
  __shared__ int32_t tiles[kMaxExperts + 1];
  __shared__ int32_t first[kMaxExperts + 1];
  __shared__ int32_t wsum[T::WAVES];
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / T::WN, wn = wave % T::WN;
  const int n32 = lane & 31, g2 = lane >> 5;
  build_tiles<T::THREADS, T::BM>(g.offsets, g.E, (int)g.P, tiles, first, wsum, tid);

  const int N = g.N, I = N >> 1, KB = g.K / 32;
  const int nk = max(2, (KB + 7) / 8);
  const uint32_t row_bytes = (uint32_t)KB * 16u;
  constexpr int C = kSwiglu ? T::NT / 2 : T::NT;  // neighbouring columns of a lane
  const uint32_t b_step = 8u * C * row_bytes;
  Place<T> p;
#pragma unroll
  for (int q = 0; q < 4; ++q) p.ro[q] = n32 * 128 + (((2 * q + g2) ^ ((n32 >> 1) & 7)) << 4);
  p.a_base = (uint32_t)wm * T::MT * 4096;
  p.b_base = (uint32_t)wn * T::NT * 4096;
  p.a_row = wm * T::MT * 32 + n32;
  p.b_row = T::BM + wn * T::NT * 32 + n32;
  p.last = (KB + 7) / 8 - 1;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int inside = KB - p.last * 8 - 4 * h;  // scale bytes of the last step's half
    p.mask[h] = inside >= 4 ? ~0u : inside > 0 ? (1u << (8 * inside)) - 1u : 0u;
  }
  p.lane_shift = 8 * g2;

  // The weight row of LDS row l = (wave column, group of 32, i): columns C i .. of a wave column
  // go to its first C groups; SwiGLU: their up rows to the others.  Rows behind the
  // matrix are read as zeros, gate rows behind I are up rows; neither's results are stored.
  auto weight_row = [&](int l, int n_idx) -> int {
    const int w = l / (T::NT * 32), nt = (l >> 5) % T::NT, i = l & 31;
    return ((n_idx * T::WN + w) * 32 + i) * C + nt % C + (nt >= C ? I : 0);
  };
  // scales are read as aligned words: byte offsets from the array's start rounded down
  auto scale_rsrc = [&](const uint8_t* at, int64_t bytes, uint32_t& skip) -> i32x4 {
    skip = (uint32_t)(reinterpret_cast<uintptr_t>(at) & 3);
    return make_rsrc(at - skip, ((uint32_t)bytes + skip + 3u) & ~3u);
  };
  const int total_m = __builtin_amdgcn_readfirstlane(tiles[g.E]);
  const int total = total_m * n_tiles;
  const int G = gridDim.x;  // a multiple of 8
  const int u = (blockIdx.x & 7) * (G >> 3) + (blockIdx.x >> 3);
  if (u >= total) return;
  // Tiles r .. r + kDescs - 1 of this workgroup: groups of four row tiles, the row tile changing fastest.
  auto look_up = [&](int r) {
    const int64_t t = (int64_t)(r + tid) * G + u;
    if (tid < kDescs && t < total) {
      const int tix = (int)t;
      const int group = tix / (4 * n_tiles), in = tix - group * 4 * n_tiles;
      const int gm = min(4, total_m - group * 4);
      const int n_idx = in / gm, mt = group * 4 + (in - n_idx * gm);
      int lo = 0, hi = g.E;  // tiles[lo] <= mt < tiles[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tiles[mid] <= mt) lo = mid; else hi = mid;
      }
      const int row0 = first[lo] + (mt - tiles[lo]) * T::BM;
      descs[tid] = TileDesc{lo, row0, min(T::BM, first[lo + 1] - row0), n_idx};
    }
  };
  auto desc = [&](int r) -> TileDesc {
    const TileDesc d = descs[r & (kDescs - 1)];
    return TileDesc{__builtin_amdgcn_readfirstlane(d.e), __builtin_amdgcn_readfirstlane(d.row0),
                    __builtin_amdgcn_readfirstlane(d.rows), __builtin_amdgcn_readfirstlane(d.n_idx)};
  };
  const i32x4 ga_rsrc = make_rsrc(g.gather, g.gather ? (uint32_t)g.P * 4u : 0u);
  const i32x4 sc_rsrc = make_rsrc(g.scatter, g.scatter ? (uint32_t)g.P * 4u : 0u);
  const i32x4 rs_rsrc = make_rsrc(g.row_scale, g.row_scale ? (uint32_t)g.P * 4u : 0u);
  // The index arrays' entries of a tile's rows (the last row's for the rows behind it).
  auto copy_indices = [&](const TileDesc& d, int par) {
    for (int grp = wave; grp < T::BM / 64; grp += T::WAVES) {
      const uint32_t at = (uint32_t)(d.row0 + min(grp * 64 + lane, d.rows - 1)) * 4u;
      if (g.gather) copy4(ga_rsrc, at, lds_addr(&srow[par][grp * 64]));
      if (g.scatter) copy4(sc_rsrc, at, lds_addr(&orow[par][grp * 64]));
      if (g.row_scale) copy4(rs_rsrc, at, lds_addr(&rscale[par][grp * 64]));
    }
  };
  auto source = [&](const TileDesc& d, int par, int row) -> uint32_t {
    const int s = g.gather ? srow[par][row] / g.gather_div : d.row0 + min(row, d.rows - 1);
    return (uint32_t)min(max(s, 0), (int)g.a_rows - 1);
  };
  Copies<T> c;
  uint32_t a_skip, b_skip = 0;
  c.a_rsrc = make_rsrc(g.a, (uint32_t)g.a_rows * row_bytes);
  c.sa_rsrc = scale_rsrc(g.a_scales, g.a_rows * KB, a_skip);
  auto copies_of = [&](const TileDesc& d, int par) {
    const int64_t w_at = (int64_t)d.e * N;
    c.b_rsrc = make_rsrc(g.blocks + w_at * row_bytes, (uint32_t)N * row_bytes);
    c.sb_rsrc = scale_rsrc(g.scales + w_at * KB, (int64_t)N * KB, b_skip);
#pragma unroll
    for (int i = 0; i < T::A_DMA; ++i) {
      const int row = (wave * T::A_DMA + i) * 8 + (lane >> 3);
      c.a_off[i] = row < d.rows ? source(d, par, row) * row_bytes + (((lane & 7) ^ ((row >> 1) & 7)) << 4)
                                : kNowhere;
    }
    const int l0 = wave * T::B_DMA * 8 + (lane >> 3);
    // chunks are exchanged by the row's second to fourth bit: eight rows on, by four more
    const uint32_t chunk = (lane & 7) ^ ((l0 >> 1) & 7);
    c.b_off[0] = (uint32_t)weight_row(l0, d.n_idx) * row_bytes + (chunk << 4);
    c.b_off[1] = (uint32_t)weight_row(l0, d.n_idx) * row_bytes + ((chunk ^ 4) << 4);
#pragma unroll
    for (int i = 0; i < T::S_DMA; ++i) {
      const int l = min(wave * T::S_DMA + i, T::S_GROUPS - 1) * 64 + lane;
      c.s_off[i] = (l < T::BM ? source(d, par, l) * (uint32_t)KB + a_skip
                              : (uint32_t)weight_row(l - T::BM, d.n_idx) * (uint32_t)KB + b_skip) & ~3u;
    }
  };

  const uint32_t ring_at = lds_addr(ring);
  look_up(0);
  __syncthreads();
  TileDesc cur = desc(0);
  copy_indices(cur, 0);
  wait_vm_barrier<0>();
  copies_of(cur, 0);
  issue_scales<T>(c, 0, ring_at + 2 * T::STAGE, wave, 0, 0);
  if (kSplit) issue_scales<T>(c, 1, ring_at + 2 * T::STAGE + T::WINDOW, wave, 0, 0);
  Pending d{c.b_rsrc, {c.b_off[0], c.b_off[1]}, 0, 0};
#pragma unroll
  for (int j = 0; j < T::A_DMA; ++j) issue_a<T>(c, j, 0, ring_at, wave, 0);
#pragma unroll
  for (int j = 0; j < T::B_DMA; ++j) issue_b<T>(d, j, b_step, ring_at, wave);
#pragma unroll
  for (int j = 0; j < T::A_DMA; ++j) issue_a<T>(c, j, 1, ring_at + T::STAGE, wave, 0);
  d.kb = 1;
  wait_vm_barrier<T::A_DMA>();  // step 0 landed
  int stage = 0, window = 0;
  for (int r = 0;; ++r) {
    const int par = r & 1;
    const bool more = (int64_t)(r + 1) * G + u < total;
    TileDesc next = cur;
    if (more) {
      if (((r + 1) & (kDescs - 1)) == 0) {
        __syncthreads();
        look_up(r + 1);
        __syncthreads();
      }
      next = desc(r + 1);
      copy_indices(next, par ^ 1);
      // they are read two steps before the tile's end, behind a step's barrier
      if (nk < 3) wait_vm_barrier<0>();
    }
    // where in its first word a row's scales begin
    if constexpr (kSplit) {
#pragma unroll
      for (int m = 0; m < T::MT; ++m)
        p.a_shift[m] = (source(cur, par, (wm * T::MT + m) * 32 + n32) * (uint32_t)KB + a_skip) & 3u;
      const uint32_t at = (uint32_t)reinterpret_cast<uintptr_t>(g.scales + (int64_t)cur.e * N * KB);
#pragma unroll
      for (int n = 0; n < T::NT; ++n)
        p.b_shift[n] = (at + (uint32_t)weight_row((wn * T::NT + n) * 32 + n32, cur.n_idx) * KB) & 3u;
    }
    const int mtv = max(0, min(T::MT, (cur.rows - wm * T::MT * 32 + 31) >> 5));
    auto tile = [&](auto rows) {
      constexpr int M = decltype(rows)::value;
      f32x16 acc[M ? M : 1][T::NT];
      kloop<T, M, kSplit>(c, d, p, nk, b_step, ring, ring_at, wave, stage, window, more,
                          [&] { copies_of(next, par ^ 1); }, acc);
      if constexpr (M > 0)
        store_tile<T, M, kSwiglu, kOut>(g, cur, orow[par], rscale[par], wm, wn, n32, g2, acc);
    };
    if (mtv > T::MT / 2) tile(Const<T::MT>{});
    else if (mtv == 1) tile(Const<1>{});
    else tile(Const<0>{});
    if (!more) break;
    cur = next;
    // every wave has read this tile's indices, whose place the next but one's take
    lds_barrier();
  }
  // no copy of the wave is left in flight when it ends
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

namespace {

template <bool kSwiglu, int kA>
void launch_small(const MxGemmArgs& g, dim3 grid, int n_tiles, hipStream_t s) {
  if (g.out_dtype == kF32)
    hipLaunchKernelGGL((mx_small_kernel<kSwiglu, kF32, kA>), grid, dim3(kThreads), 0, s, g, n_tiles);
  else if (g.out_dtype == kBF16)
    hipLaunchKernelGGL((mx_small_kernel<kSwiglu, kBF16, kA>), grid, dim3(kThreads), 0, s, g, n_tiles);
  else
    hipLaunchKernelGGL((mx_small_kernel<kSwiglu, kF16, kA>), grid, dim3(kThreads), 0, s, g, n_tiles);
}

template <bool kSwiglu>
void launch_small(const MxGemmArgs& g, dim3 grid, int n_tiles, hipStream_t s) {
  if (g.a_dtype == kF32) launch_small<kSwiglu, kF32>(g, grid, n_tiles, s);
  else if (g.a_dtype == kBF16) launch_small<kSwiglu, kBF16>(g, grid, n_tiles, s);
  else if (g.a_dtype == kF16) launch_small<kSwiglu, kF16>(g, grid, n_tiles, s);
  else launch_small<kSwiglu, kCodes>(g, grid, n_tiles, s);
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

using Tile256 = Tile<4, 2, 2, 4, 1>;  // 256 x 256
using Tile64 = Tile<2, 2, 1, 2, 2>;   // 64 x 128
// Columns of a 16-row tile's workgroup, and the tiles of a call, at most: an expert's rows begin one
// of their own.
int small_n_tiles(int64_t N, bool swiglu) { return (int)(swiglu ? (N / 2 + 15) / 16 : (N + 31) / 32); }
int64_t small_tiles(int E, int64_t P, int64_t N, bool swiglu) {
  const int64_t hit = std::min<int64_t>(E, P);
  return (hit + (P - hit) / 16) * small_n_tiles(N, swiglu);
}

}  // namespace

// One launch of 16-row tiles while they are few, each reading its weights for itself.  Measured,
// small against quantising and 64-row tiles (us, in a graph): 16 pairs on 64 experts of 2048 x 2048
// (1024 tiles) 14.1 against 15.9, 24 pairs (1536) 16.9 and 17.3, 32 pairs (2048) 21.9 and 19.4;
// 32 rows of one 4096 x 4096 (256) 12.1 and 16.6; 24 rows of 28672 x 2048 (1792) 24.2 and 17.6.
bool mx_gemm_small(int E, int64_t P, int64_t N, bool swiglu) {
  return P <= kSmallRows && small_tiles(E, P, N, swiglu) <= 1536;
}

// 256-row tiles from 80 rows an expert on, where 64-row ones are more than one round of the card's
// places (an expert's last tile counted half).  Measured, 64 against 256 (us):
//   64 experts of 2048 x 2048: 32 rows each 28.6 and 33.2, 64 rows 32.3 and 40.7, 96 rows 43.8
//   and 36.6, 128 rows 46.6 and 37.6;
//   one round: 1024 rows of one 2048 x 2048 12.7 and 19.1, of one 4096 x 4096 23.7 and 31.5, 512 of
//   8192 x 8192 37.9 and 55.3, 128 of 28672 x 4096 23.8 and 29.3, 1536 on 8 experts 16.3 and 24.3;
//   a little more: 1088 rows of one 4096 x 4096 34.9 and 32.2, 576 of 8192 x 8192 67.9 and 53.5,
//   2048 on 16 experts of 2048 x 2048 25.5 and 22.1; the other way round, 8 experts of 256 rows each
//   (512 tiles, counted as 576) 14.3 and 23.7.
static bool mx_gemm_wide(const MxGemmArgs& g, int num_cus) {
  const int64_t hit = std::min<int64_t>(g.E, g.P);
  if (g.P / hit < 80) return false;
  return ((g.P + 63) / 64 + hit / 2) * ((g.N + 127) / 128) > (int64_t)num_cus * Tile64::PER_CU;
}

hipError_t launch_mx_gemm(const MxGemmArgs& g, int num_cus, hipStream_t s) {
  if (mx_gemm_small(g.E, g.P, g.N, g.swiglu)) {
    const int n_tiles = small_n_tiles(g.N, g.swiglu);
    const dim3 grid((unsigned)small_tiles(g.E, g.P, g.N, g.swiglu));
    if (g.swiglu) launch_small<true>(g, grid, n_tiles, s);
    else launch_small<false>(g, grid, n_tiles, s);
  } else if (mx_gemm_wide(g, num_cus)) {
    launch_tiles<Tile256>(g, num_cus, s);
  } else {
    launch_tiles<Tile64>(g, num_cus, s);
  }
  return hipGetLastError();
}

}  // namespace nf4moe
