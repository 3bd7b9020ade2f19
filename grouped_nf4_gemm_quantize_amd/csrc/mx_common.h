// Device helpers of the MXFP4 kernels: a block's scale and the codes of its values.
#pragma once

#include "common.h"

namespace nf4moe {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// The scale byte of a block whose largest magnitude has these fp32 bits (infinity
// or NaN: 255), and the power of two the conversion divides by.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  const uint32_t e = top >> 23;
  return top >= 0x7f800000u ? 255u : e > 2u ? e - 2u : 0u;
}
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __uint_as_float(byte == 0u ? 0x400000u : byte == 255u ? 0x3f800000u : byte << 23);
}

// fp32 bits of a 16-bit magnitude.
template <int kT>
__device__ __forceinline__ uint32_t wide_bits(uint32_t mag16) {
  if constexpr (kT == kBF16) return mag16 << 16;
  else return __float_as_uint((float)__builtin_bit_cast(_Float16, (uint16_t)mag16));
}

__device__ __forceinline__ uint32_t pk_max_u16(uint32_t a, uint32_t b) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                __builtin_bit_cast(u16x2, b)));
}

// Two 16-bit values to the codes of byte kSel of `old`.
template <int kT, int kSel>
__device__ __forceinline__ uint32_t cvt_pair(uint32_t old, uint32_t pair, float scale) {
  if constexpr (kT == kBF16)
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, __builtin_bit_cast(bf16x2, pair), scale,
                                                     kSel);
  else
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(old, u32_as_half2(pair), scale, kSel);
}
template <int kSel>
__device__ __forceinline__ uint32_t cvt_two(uint32_t old, uint32_t a, uint32_t b, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, __uint_as_float(a), __uint_as_float(b),
                                                  scale, kSel);
}

// Eight values as they are read (fp32: two words of four).
template <int kT>
struct Eight {
  u32x4 v[kT == kF32 ? 2 : 1];
};

template <int kT>
__device__ __forceinline__ void load_eight(const void* x, int64_t i, Eight<kT>& o) {
  const u32x4* p = reinterpret_cast<const u32x4*>(x) + i * (kT == kF32 ? 2 : 1);
#pragma unroll
  for (int j = 0; j < (kT == kF32 ? 2 : 1); ++j) o.v[j] = p[j];
}

// The largest magnitude of eight values: fp32 bits, or 16-bit ones for wide_bits.
template <int kT>
__device__ __forceinline__ uint32_t eight_top(const Eight<kT>& x) {
  if constexpr (kT == kF32) {
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, x.v[j >> 2][j & 3] & 0x7fffffffu);
    return top;
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) m = pk_max_u16(m, x.v[0][j] & 0x7fff7fffu);
    return max(m & 0xffffu, m >> 16);
  }
}

// The codes of eight values.
template <int kT>
__device__ __forceinline__ uint32_t eight_codes(const Eight<kT>& x, float s) {
  uint32_t c = 0;
  if constexpr (kT == kF32) {
    c = cvt_two<0>(c, x.v[0][0], x.v[0][1], s);
    c = cvt_two<1>(c, x.v[0][2], x.v[0][3], s);
    c = cvt_two<2>(c, x.v[1][0], x.v[1][1], s);
    c = cvt_two<3>(c, x.v[1][2], x.v[1][3], s);
  } else {
    c = cvt_pair<kT, 0>(c, x.v[0][0], s);
    c = cvt_pair<kT, 1>(c, x.v[0][1], s);
    c = cvt_pair<kT, 2>(c, x.v[0][2], s);
    c = cvt_pair<kT, 3>(c, x.v[0][3], s);
  }
  return c;
}

}  // namespace

}  // namespace nf4moe
