// MXFP4 blocks made of 16- and 32-bit values and read back (mxfp4_quantize,
// mxfp4_dequantize).  A block is 32 values along the contraction axis:
//   e = max(floor(log2 max|x|) - 2, -127);  code = e2m1(x / 2^e), ties to even,
//   beyond 6 saturated;  scale byte = e + 127, 255 (NaN) for a block with an
//   infinity or a NaN.
// floor(log2) is the exponent field of the largest magnitude; the division by a
// power of two is exact and the conversion instructions do it and the rounding.
//
// Bound by memory: 2.53 bytes an element for bf16 one way, and the same back.  Measured, 16 x 2048
// x 2048 bf16, between other calls: along the rows 26-30 us = 5.7-6.5 TB/s, along the columns 35 us
// (25 on the same input again, part of which is in the cache behind the L2s), back 26-27 us.

#include <algorithm>

#include "common.h"
#include "launch.h"
#include "mfma_common.h"
#include "mx_common.h"

namespace nf4moe {

namespace {

template <int kCtrl>
__device__ __forceinline__ uint32_t dpp_u(uint32_t v) {
  return (uint32_t)dpp_i<kCtrl>((int)v);
}

// Blocks along the rows: the matrix is a flat run of blocks, eight values a lane.
template <int kT>
__global__ __launch_bounds__(256) void mx_quantize_kernel(const void* x, int64_t n8,
                                                          uint32_t* codes, uint8_t* scales) {
  // n8 is a multiple of 4, so the lanes of a block are in or out together
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n8; i += (int64_t)gridDim.x * 256) {
    Eight<kT> v;
    load_eight<kT>(x, i, v);
    uint32_t top = eight_top<kT>(v);  // of the four lanes of a block
    top = max(top, dpp_u<kDppXor1>(top));
    top = max(top, dpp_u<kDppXor2>(top));
    if constexpr (kT != kF32) top = wide_bits<kT>(top);
    const uint32_t byte = scale_byte(top);
    const uint32_t c = eight_codes<kT>(v, scale_value(byte));
    codes[i] = byte == 255u ? 0u : c;
    if ((threadIdx.x & 3) == 0) scales[i >> 2] = (uint8_t)byte;
  }
}

// Blocks along the columns of [R, K]: a lane takes 32 rows of one column, or of two neighbours as
// they lie in a word (16-bit values, K even).  A workgroup's eight waves have row blocks beside each
// other: their codes, 128 bytes of a column, and scales go through LDS and leave as whole
// lines (16 x 2048 x 2048 bf16, both in one run: 31.5 us; 46.5 with a lane's 16 bytes and scale byte stored
// as they are).
constexpr int kColWaves = 8;

template <int kT, int kCols>
__global__ __launch_bounds__(kColWaves * 64) void mx_quantize_cols_kernel(const void* x, int64_t R,
                                                                          int64_t K, uint8_t* codes,
                                                                          uint8_t* scales) {
  constexpr int kStride = kColWaves * 16 + 16;  // of a column's codes in LDS
  __shared__ __attribute__((aligned(16))) char s_codes[64 * kCols * kStride];
  __shared__ __attribute__((aligned(8))) uint8_t s_scales[64 * kCols * kColWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t col0 = (int64_t)blockIdx.x * 64 * kCols, blocks = R / 32;
  const int64_t rb0 = (int64_t)blockIdx.y * kColWaves, e = blockIdx.z;
  const int cols = (int)min((int64_t)64 * kCols, K - col0);
  const int rbs = (int)min((int64_t)kColWaves, blocks - rb0);
  // lanes behind the last column or row block read its values again
  const int c0 = min(lane * kCols, cols - kCols), rb = min(wave, rbs - 1);
  const int64_t at = (e * R + (rb0 + rb) * 32) * K + col0 + c0;
  uint32_t v[32];
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    if constexpr (kT == kF32) v[j] = reinterpret_cast<const uint32_t*>(x)[at + j * K];
    else if constexpr (kCols == 2)
      v[j] = *reinterpret_cast<const uint32_t*>(reinterpret_cast<const uint16_t*>(x) + at + j * K);
    else v[j] = reinterpret_cast<const uint16_t*>(x)[at + j * K];
  }
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    if constexpr (kT == kF32) m = max(m, v[j] & 0x7fffffffu);
    else m = pk_max_u16(m, v[j] & 0x7fff7fffu);
  }
#pragma unroll
  for (int c = 0; c < kCols; ++c) {
    uint32_t top = m;
    if constexpr (kT != kF32) top = wide_bits<kT>(c ? m >> 16 : m & 0xffffu);
    const uint32_t byte = scale_byte(top);
    const float s = scale_value(byte);
    u32x4 o;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t w = 0;
      if constexpr (kT == kF32) {
        w = cvt_two<0>(w, v[8 * q], v[8 * q + 1], s);
        w = cvt_two<1>(w, v[8 * q + 2], v[8 * q + 3], s);
        w = cvt_two<2>(w, v[8 * q + 4], v[8 * q + 5], s);
        w = cvt_two<3>(w, v[8 * q + 6], v[8 * q + 7], s);
      } else {
        // this column's half of two rows' words
        constexpr uint32_t kLow = 0x05040100u, kHigh = 0x07060302u;
        const uint32_t sel = c ? kHigh : kLow;
        w = cvt_pair<kT, 0>(w, __builtin_amdgcn_perm(v[8 * q + 1], v[8 * q], sel), s);
        w = cvt_pair<kT, 1>(w, __builtin_amdgcn_perm(v[8 * q + 3], v[8 * q + 2], sel), s);
        w = cvt_pair<kT, 2>(w, __builtin_amdgcn_perm(v[8 * q + 5], v[8 * q + 4], sel), s);
        w = cvt_pair<kT, 3>(w, __builtin_amdgcn_perm(v[8 * q + 7], v[8 * q + 6], sel), s);
      }
      o[q] = byte == 255u ? 0u : w;
    }
    *reinterpret_cast<u32x4*>(s_codes + (c0 + c) * kStride + rb * 16) = o;
    s_scales[(c0 + c) * kColWaves + rb] = (uint8_t)byte;
  }
  __syncthreads();
  // eight threads a column; K and the row blocks set how many columns and blocks there are
  for (int i = threadIdx.x; i < cols * kColWaves; i += kColWaves * 64) {
    const int c = i / kColWaves, b = i % kColWaves;
    if (b >= rbs) continue;
    const int64_t ob = (e * K + col0 + c) * blocks + rb0 + b;
    reinterpret_cast<u32x4*>(codes)[ob] = *reinterpret_cast<const u32x4*>(s_codes + c * kStride + b * 16);
    if (blocks % kColWaves == 0 && (reinterpret_cast<uintptr_t>(scales) & 7) == 0) {
      if (b == 0)
        *reinterpret_cast<uint64_t*>(scales + ob) = *reinterpret_cast<const uint64_t*>(s_scales + c * kColWaves);
    } else {
      scales[ob] = s_scales[c * kColWaves + b];
    }
  }
}

template <int kSel>
__device__ __forceinline__ void two_values(uint32_t c, float s, float* v) {
  const f32x2 p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, kSel);
  v[0] = p.x;
  v[1] = p.y;
}

template <int kOut>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(const uint32_t* codes,
                                                            const uint8_t* scales, int64_t n8,
                                                            void* out) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n8; i += (int64_t)gridDim.x * 256) {
    const uint32_t c = codes[i];
    const uint32_t byte = scales[i >> 2];
    const float s = scale_value(byte);
    float v[8];
    two_values<0>(c, s, v);
    two_values<1>(c, s, v + 2);
    two_values<2>(c, s, v + 4);
    two_values<3>(c, s, v + 6);
    if (byte == 255u) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(0x7fc00000u);
    }
    store8<kOut>(out, i * 8, v);
  }
}

}  // namespace

// Workgroups of 256 for n lanes; a grid's threads are counted in 32 bits.
static unsigned flat_grid(int64_t n) { return (unsigned)std::min<int64_t>((n + 255) / 256, 1 << 22); }

hipError_t launch_mx_quantize(const void* x, int x_dtype, int64_t E, int64_t R, int64_t K,
                              bool cols, uint8_t* codes, uint8_t* scales, hipStream_t s) {
  if (!cols) {
    const int64_t n8 = E * R * K / 8;
    const dim3 grid(flat_grid(n8));
    uint32_t* c = reinterpret_cast<uint32_t*>(codes);
    if (x_dtype == kF32)
      hipLaunchKernelGGL(mx_quantize_kernel<kF32>, grid, dim3(256), 0, s, x, n8, c, scales);
    else if (x_dtype == kBF16)
      hipLaunchKernelGGL(mx_quantize_kernel<kBF16>, grid, dim3(256), 0, s, x, n8, c, scales);
    else
      hipLaunchKernelGGL(mx_quantize_kernel<kF16>, grid, dim3(256), 0, s, x, n8, c, scales);
    return hipGetLastError();
  }
  const bool pairs = x_dtype != kF32 && K % 2 == 0 && (reinterpret_cast<uintptr_t>(x) & 3) == 0;
  const int64_t width = pairs ? 128 : 64;
  const dim3 grid((unsigned)((K + width - 1) / width), (unsigned)((R / 32 + kColWaves - 1) / kColWaves),
                  (unsigned)E);
  const dim3 block(kColWaves * 64);
  if (x_dtype == kF32)
    hipLaunchKernelGGL((mx_quantize_cols_kernel<kF32, 1>), grid, block, 0, s, x, R, K, codes, scales);
  else if (x_dtype == kBF16 && pairs)
    hipLaunchKernelGGL((mx_quantize_cols_kernel<kBF16, 2>), grid, block, 0, s, x, R, K, codes, scales);
  else if (x_dtype == kBF16)
    hipLaunchKernelGGL((mx_quantize_cols_kernel<kBF16, 1>), grid, block, 0, s, x, R, K, codes, scales);
  else if (pairs)
    hipLaunchKernelGGL((mx_quantize_cols_kernel<kF16, 2>), grid, block, 0, s, x, R, K, codes, scales);
  else
    hipLaunchKernelGGL((mx_quantize_cols_kernel<kF16, 1>), grid, block, 0, s, x, R, K, codes, scales);
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t n, void* out,
                                int out_dtype, hipStream_t s) {
  const int64_t n8 = n / 8;
  const dim3 grid(flat_grid(n8));
  const uint32_t* c = reinterpret_cast<const uint32_t*>(codes);
  if (out_dtype == kF32)
    hipLaunchKernelGGL(mx_dequantize_kernel<kF32>, grid, dim3(256), 0, s, c, scales, n8, out);
  else if (out_dtype == kBF16)
    hipLaunchKernelGGL(mx_dequantize_kernel<kBF16>, grid, dim3(256), 0, s, c, scales, n8, out);
  else
    hipLaunchKernelGGL(mx_dequantize_kernel<kF16>, grid, dim3(256), 0, s, c, scales, n8, out);
  return hipGetLastError();
}

}  // namespace nf4moe
