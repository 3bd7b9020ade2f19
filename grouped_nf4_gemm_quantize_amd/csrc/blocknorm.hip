// RMS norms after and before a block, fused with the block's gate and residual
// scale, and their gradients (block_norm_forward / block_norm_backward):
//   z = y * rstd(y) * (w_post + off),  r = beta * residual + alpha * gate * z,
//   h = r * rstd(r) * (w_pre + off),   rstd(v) = 1 / sqrt(mean(v^2) + eps).
//
// One workgroup holds one row: a thread has eight consecutive columns (or two
// such vectors beyond 8192 columns) in fp32 registers, so every matrix is read
// once and written once; the row sums go through the waves and LDS.  r is rounded
// to its type before it is normalised, so h follows from what is stored.

#include "common.h"
#include "launch.h"

namespace nf4moe {

namespace {

constexpr int kNormGroups = 512;  // workgroups (and partial rows) of the backward

// Eight consecutive elements from element idx (a multiple of 8; rows are
// 16-byte aligned).
__device__ __forceinline__ void load8(const void* p, int dtype, int64_t idx, float (&v)[8]) {
  if (dtype == kF32) {
    const f32x4* q = reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(p) + idx);
    const f32x4 a = q[0], b = q[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
    return;
  }
  const u32x4 q = *reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(p) + idx);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (dtype == kBF16) {
      v[2 * i] = bf16_bits_to_f32(q[i] & 0xffffu);
      v[2 * i + 1] = bf16_bits_to_f32(q[i] >> 16);
    } else {
      const f16x2 h = u32_as_half2(q[i]);
      v[2 * i] = (float)h.x;
      v[2 * i + 1] = (float)h.y;
    }
  }
}

// Rounds v to dtype, stores it and leaves the stored values in v.
__device__ __forceinline__ void store8(void* p, int dtype, int64_t idx, float (&v)[8]) {
  if (dtype == kF32) {
    f32x4* q = reinterpret_cast<f32x4*>(reinterpret_cast<float*>(p) + idx);
    q[0] = f32x4{v[0], v[1], v[2], v[3]};
    q[1] = f32x4{v[4], v[5], v[6], v[7]};
    return;
  }
  u32x4 q;
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
  *reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(p) + idx) = q;
}

// Sums of kN values over the workgroup, in every thread.  `red` holds kN * 16
// floats; the caller alternates between two of them from call to call.
template <int kN>
__device__ __forceinline__ void block_sum(float (&v)[kN], float* red) {
  const int wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
#pragma unroll
  for (int i = 0; i < kN; ++i) v[i] = wave_sum(v[i]);
  if (waves == 1) return;
  if ((threadIdx.x & 63) == 0)
#pragma unroll
    for (int i = 0; i < kN; ++i) red[i * 16 + wave] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    float s = 0.f;
    for (int w = 0; w < waves; ++w) s += red[i * 16 + w];
    v[i] = s;
  }
}

// 1 / sqrt(mean + eps), correctly rounded operations
__device__ __forceinline__ float rstd_of(float sum, int H, float eps) {
  return 1.0f / sqrtf(sum / (float)H + eps);
}

}  // namespace

template <int kVec>
__global__ __launch_bounds__(1024) void block_norm_kernel(BlockNormArgs a) {
  __shared__ float red[2][16];
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
  const int64_t row = t * a.H;
  float r[kVec][8], z[kVec][8], wv[8];
#pragma unroll
  for (int u = 0; u < kVec; ++u) {
    const int c = (threadIdx.x + u * blockDim.x) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[u][i] = z[u][i] = 0.f;
    if (c >= a.H) continue;
    load8(a.residual, a.res_dtype, row + c, r[u]);
    if (a.y) load8(a.y, a.y_dtype, row + c, z[u]);
  }
  if (a.y) {
    float rstd = 1.f;
    if (a.w_post) {
      float s[1] = {0.f};
#pragma unroll
      for (int u = 0; u < kVec; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0] += z[u][i] * z[u][i];
      block_sum(s, red[0]);
      rstd = rstd_of(s[0], a.H, a.eps);
    }
    const float gt = a.gate_axis == 1 ? a.alpha * a.gate[t] : a.alpha;
#pragma unroll
    for (int u = 0; u < kVec; ++u) {
      const int c = (threadIdx.x + u * blockDim.x) * 8;
      if (c >= a.H) continue;
      if (a.w_post) {
        load8(a.w_post, a.w_dtype, c, wv);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[u][i] *= rstd * (wv[i] + a.w_offset);
      }
      if (a.gate_axis == 2) {
        for (int i = 0; i < 8; ++i) z[u][i] *= a.gate[c + i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) r[u][i] = a.beta * r[u][i] + gt * z[u][i];
      store8(a.r_out, a.res_dtype, row + c, r[u]);
    }
  }
  if (!a.w_pre) {
    __syncthreads();  // the sums' LDS is written again for the next row
    continue;
  }
  float s[1] = {0.f};
#pragma unroll
  for (int u = 0; u < kVec; ++u)
#pragma unroll
    for (int i = 0; i < 8; ++i) s[0] += r[u][i] * r[u][i];
  block_sum(s, red[1]);
  const float rstd = rstd_of(s[0], a.H, a.eps);
#pragma unroll
  for (int u = 0; u < kVec; ++u) {
    const int c = (threadIdx.x + u * blockDim.x) * 8;
    if (c >= a.H) continue;
    load8(a.w_pre, a.w_dtype, c, wv);
#pragma unroll
    for (int i = 0; i < 8; ++i) r[u][i] = r[u][i] * rstd * (wv[i] + a.w_offset);
    store8(a.h, a.h_dtype, row + c, r[u]);
  }
  __syncthreads();
  }
}

// A workgroup takes rows blockIdx.x, blockIdx.x + gridDim.x, ...; its sums over
// them of the column gradients stay in registers and go to row blockIdx.x of the
// partial sums (dw_pre, dw_post, dgate by channel).
template <int kVec>
__global__ __launch_bounds__(1024) void block_norm_bwd_kernel(BlockNormArgs a) {
  __shared__ float red[2][3 * 16];
  __shared__ float red_g[2 * 16];
  float s_pre[kVec][8] = {}, s_post[kVec][8] = {}, s_gate[kVec][8] = {};
  const float inv_h = 1.0f / (float)a.H;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int64_t row = t * a.H;
    float r[kVec][8], d[kVec][8], y[kVec][8], g[kVec][8], wv[8];
    float s[3] = {0.f, 0.f, 0.f};  // r^2, dh * w * r, y^2
#pragma unroll
    for (int u = 0; u < kVec; ++u) {
      const int c = (threadIdx.x + u * blockDim.x) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) r[u][i] = d[u][i] = y[u][i] = g[u][i] = 0.f;
      if (c >= a.H) continue;
      if (a.w_pre) {
        load8(a.residual, a.res_dtype, row + c, r[u]);
        load8(a.dh, a.h_dtype, row + c, g[u]);
        load8(a.w_pre, a.w_dtype, c, wv);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          s[0] += r[u][i] * r[u][i];
          s[1] += g[u][i] * (wv[i] + a.w_offset) * r[u][i];
        }
      }
      if (a.d_r_out) load8(a.d_r_out, a.res_dtype, row + c, d[u]);
      if (a.y) {
        load8(a.y, a.y_dtype, row + c, y[u]);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[2] += y[u][i] * y[u][i];
      }
    }
    block_sum(s, red[0]);
    const float rstd_r = rstd_of(s[0], a.H, a.eps);
    const float k_r = rstd_r * rstd_r * rstd_r * (s[1] * inv_h);
    const float rstd_y = a.w_post ? rstd_of(s[2], a.H, a.eps) : 1.f;
    const float gt = a.gate_axis == 1 ? a.alpha * a.gate[t] : a.alpha;
    float s2[2] = {0.f, 0.f};  // dz * w * y, dr * z
#pragma unroll
    for (int u = 0; u < kVec; ++u) {
      const int c = (threadIdx.x + u * blockDim.x) * 8;
      if (c >= a.H) continue;
      if (a.w_pre) {
        load8(a.w_pre, a.w_dtype, c, wv);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          s_pre[u][i] += g[u][i] * r[u][i] * rstd_r;
          d[u][i] += rstd_r * g[u][i] * (wv[i] + a.w_offset) - r[u][i] * k_r;
        }
      }
      // d is dr; r becomes dresidual, g the gradient dz of z
#pragma unroll
      for (int i = 0; i < 8; ++i) r[u][i] = a.beta * d[u][i];
      store8(a.r_out, a.res_dtype, row + c, r[u]);
      if (!a.y) continue;
      if (a.w_post) load8(a.w_post, a.w_dtype, c, wv);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float w = a.w_post ? wv[i] + a.w_offset : 1.f;
        const float z = y[u][i] * rstd_y * w;
        g[u][i] = gt * d[u][i];
        if (a.gate_axis == 2) {
          s_gate[u][i] += a.alpha * d[u][i] * z;
          g[u][i] *= a.gate[c + i];
        }
        s2[0] += g[u][i] * w * y[u][i];
        s2[1] += d[u][i] * z;
        s_post[u][i] += g[u][i] * y[u][i] * rstd_y;
        g[u][i] *= w;
      }
    }
    if (a.y) {
      block_sum(s2, red_g);
      if (a.gate_axis == 1 && threadIdx.x == 0) a.dgate[t] = a.alpha * s2[1];
      const float k_y = a.w_post ? rstd_y * rstd_y * rstd_y * (s2[0] * inv_h) : 0.f;
#pragma unroll
      for (int u = 0; u < kVec; ++u) {
        const int c = (threadIdx.x + u * blockDim.x) * 8;
        if (c >= a.H) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) g[u][i] = rstd_y * g[u][i] - y[u][i] * k_y;
        store8(a.h, a.y_dtype, row + c, g[u]);
      }
    }
    __syncthreads();  // the sums' LDS is written again for the next row
  }
  float* part = a.part + (int64_t)blockIdx.x * a.H;
  const int64_t plane = (int64_t)gridDim.x * a.H;
#pragma unroll
  for (int u = 0; u < kVec; ++u) {
    const int c = (threadIdx.x + u * blockDim.x) * 8;
    if (c >= a.H) continue;
    if (a.w_pre) store8(part, kF32, c, s_pre[u]);
    if (a.w_post) store8(part + plane, kF32, c, s_post[u]);
    if (a.gate_axis == 2) store8(part + 2 * plane, kF32, c, s_gate[u]);
  }
}

// out[c] = sum over the partial rows, one thread a column.
__global__ __launch_bounds__(64) void block_norm_reduce_kernel(BlockNormArgs a, int groups) {
  const int c = blockIdx.x * 64 + threadIdx.x;
  float* out = blockIdx.y == 0 ? a.dw_pre : blockIdx.y == 1 ? a.dw_post : a.dgate;
  if (blockIdx.y == 0 && !a.w_pre) return;
  if (blockIdx.y == 1 && !a.w_post) return;
  if (blockIdx.y == 2 && a.gate_axis != 2) return;
  if (c >= a.H) return;
  const float* p = a.part + (int64_t)blockIdx.y * groups * a.H + c;
  float s = 0.f;
  for (int i = 0; i < groups; ++i) s += p[(int64_t)i * a.H];
  out[c] = s;
}

int block_norm_groups(int64_t T, int H) {
  (void)H;
  return (int)(T < kNormGroups ? T : kNormGroups);
}

namespace {
// threads of a workgroup that holds a row: eight columns each, two vectors
// a thread where one would need more than 1024 threads
int norm_threads(int H, int vec) { return (H / 8 + 64 * vec - 1) / (64 * vec) * 64; }
}  // namespace

hipError_t launch_block_norm(const BlockNormArgs& a, int num_cus, hipStream_t s) {
  (void)num_cus;
  const dim3 grid((unsigned)(a.T < (1 << 20) ? a.T : (1 << 20)));
  if (a.H <= 8192)
    hipLaunchKernelGGL(block_norm_kernel<1>, grid, dim3(norm_threads(a.H, 1)), 0, s, a);
  else
    hipLaunchKernelGGL(block_norm_kernel<2>, grid, dim3(norm_threads(a.H, 2)), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_block_norm_bwd(const BlockNormArgs& a, hipStream_t s) {
  const int groups = block_norm_groups(a.T, a.H);
  if (a.H <= 8192)
    hipLaunchKernelGGL(block_norm_bwd_kernel<1>, dim3(groups), dim3(norm_threads(a.H, 1)), 0, s, a);
  else
    hipLaunchKernelGGL(block_norm_bwd_kernel<2>, dim3(groups), dim3(norm_threads(a.H, 2)), 0, s, a);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || (!a.w_pre && !a.w_post && a.gate_axis != 2)) return err;
  hipLaunchKernelGGL(block_norm_reduce_kernel, dim3((a.H + 63) / 64, 3), dim3(64), 0, s, a, groups);
  return hipGetLastError();
}

}  // namespace nf4moe
