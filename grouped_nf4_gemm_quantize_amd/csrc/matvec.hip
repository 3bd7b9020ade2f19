// Products of a few activation rows with one 4-bit matrix that has group
// scales: y[t, n] = bias[n] + sum_g s[n, g] sum_{k in g} (v(code) - z[n, g]) x[t, k].
//
// One wave per output row n: its lanes take eight consecutive k at a time
// (4 packed bytes, inside one group), multiply in fp32 and the wave sums.

#include "common.h"
#include "launch.h"

namespace nf4moe {

namespace {

constexpr int kMvTokens = 8;  // rows of x per workgroup

__device__ __forceinline__ float mv_scale(const MatvecArgs& a, int64_t i) {
  if (a.qt == kMvMXFP4) {
    const uint32_t b = reinterpret_cast<const uint8_t*>(a.scales)[i];
    return b == 255u ? __builtin_nanf("") : ldexpf(1.0f, (int)b - 127);
  }
  if (a.scale_dtype == kF32) return reinterpret_cast<const float*>(a.scales)[i];
  const uint16_t raw = reinterpret_cast<const uint16_t*>(a.scales)[i];
  return a.scale_dtype == kBF16 ? bf16_bits_to_f32(raw)
                                : (float)__builtin_bit_cast(_Float16, raw);
}

}  // namespace

__global__ __launch_bounds__(256) void matvec_kernel(MatvecArgs a) {
  __shared__ float level[16];
  const float nf4[16] = NF4MOE_LEVELS_INIT;
  const float fp4[16] = NF4MOE_FP4_LEVELS_INIT;
  const float e2m1[16] = NF4MOE_E2M1_VALUES_INIT;
  const int tid = threadIdx.x, lane = tid & 63;
  if (tid < 16)
    level[tid] = a.qt == kMvNF4   ? nf4[tid]
                 : a.qt == kMvFP4 ? fp4[tid]
                 : a.qt == kMvINT4 ? (float)tid
                                   : e2m1[tid];
  __syncthreads();
  const int n = blockIdx.x * 4 + (tid >> 6);
  if (n >= a.N) return;
  const int64_t t0 = (int64_t)blockIdx.y * kMvTokens;
  const int nt = a.T - t0 < kMvTokens ? (int)(a.T - t0) : kMvTokens;
  const int groups = a.K / a.group;
  const uint32_t* codes = reinterpret_cast<const uint32_t*>(a.codes + (int64_t)n * (a.K / 2));
  float acc[kMvTokens] = {};
  for (int c = lane; c < a.K / 8; c += 64) {
    const uint32_t q = codes[c];
    const int64_t gi = (int64_t)n * groups + c * 8 / a.group;
    const float s = mv_scale(a, gi);
    float z = 0.f;
    if (a.qt == kMvINT4) z = a.zeros ? (float)a.zeros[gi] : 8.f;
    float w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int nib = a.qt == kMvMXFP4 ? j : j ^ 1;
      w[j] = level[(q >> (4 * nib)) & 15] - z;
    }
#pragma unroll
    for (int t = 0; t < kMvTokens; ++t) {
      if (t >= nt) break;
      const uint16_t* x = reinterpret_cast<const uint16_t*>(a.x) + (t0 + t) * a.K + c * 8;
      float p = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const _Float16 xv = a.x_bf16 ? (_Float16)bf16_bits_to_f32(x[j])
                                     : __builtin_bit_cast(_Float16, x[j]);
        p += w[j] * (float)xv;
      }
      acc[t] += s * p;
    }
  }
  const float b = a.bias ? a.bias[n] : 0.f;
#pragma unroll
  for (int t = 0; t < kMvTokens; ++t) {
    const float v = wave_sum(acc[t]) + b;
    if (t >= nt || lane != 0) continue;
    const int64_t i = (t0 + t) * a.N + n;
    if (a.y_dtype == kF32) reinterpret_cast<float*>(a.y)[i] = v;
    else if (a.y_dtype == kBF16) reinterpret_cast<uint16_t*>(a.y)[i] = f32_to_bf16_bits(v);
    else reinterpret_cast<_Float16*>(a.y)[i] = (_Float16)v;
  }
}

hipError_t launch_matvec(const MatvecArgs& a, int num_cus, hipStream_t s) {
  (void)num_cus;
  const dim3 grid((unsigned)((a.N + 3) / 4), (unsigned)((a.T + kMvTokens - 1) / kMvTokens));
  hipLaunchKernelGGL(matvec_kernel, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace nf4moe
