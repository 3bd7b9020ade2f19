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

}  // namespace

hipError_t launch_mx_gemm(const MxGemmArgs& g, int num_cus, hipStream_t s) {
  const int n_tiles = g.swiglu ? (g.N / 2 + 15) / 16 : (g.N + 31) / 32;
  // an expert's rows begin a tile of their own: at most one more for each that has rows
  const int64_t tiles = ((g.P + 15) / 16 + std::min<int64_t>(g.E, g.P)) * n_tiles;
  const dim3 grid((unsigned)std::min<int64_t>(tiles, num_cus * 8));
  if (g.swiglu) launch_small<true>(g, grid, n_tiles, s);
  else launch_small<false>(g, grid, n_tiles, s);
  return hipGetLastError();
}

}  // namespace nf4moe
