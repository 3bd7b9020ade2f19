// Token rows into the experts' rows and back, with the routing weights, and the
// gradients (moe_dispatch, moe_combine, moe_combine_backward, moe_route_backward).
// Pair p = t k + j has its row at pos[p]; one outside [0, R) has none.
//   dispatch          rows[pos[p]] = w[p] x[t]
//   combine           y[t] = sum_j w[p] rows[pos[p]], j ascending, fp32
//   combine backward  drows[pos[p]] = w[p] dy[t],  dw[p] = <dy[t], rows[pos[p]]>
//   route backward    weights over the k chosen:  dl[id_j] += w_j (dw_j - sum_i w_i dw_i)
//                     weights of the softmax p over all:  dl[e] = p_e (g_e - sum_j p_j dw_j),
//                     g_e the sum of dw_j with id_j = e
//
// All go by token, so that a token's row is read (or written) once for its k pairs; sums over a
// token's columns stay in one workgroup and have one order.  Bound by memory.  Measured, 4096
// tokens of 2048 columns, k 8, bf16 tokens and fp16 rows: dispatch 24-25 us alone = 6.0-6.3 TB/s (most of
// it writes), combine 27-28 us = 5.4-5.6 TB/s, its gradient 50-52 us = 5.5-5.7 TB/s and the router's
// 4.1-4.8 us (a launch and reads in turn).  With one row's read at a time combine took 34 us in a row of calls,
// with several 31.

#include <algorithm>

#include "common.h"
#include "launch.h"
#include "mfma_common.h"

namespace nf4moe {

namespace {

// Eight consecutive elements at element index i.
template <int kT>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&v)[8]) {
  if constexpr (kT == kF32) {
    const f32x4* q = reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(p) + i);
    const f32x4 a = q[0], b = q[1];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = a[j];
      v[4 + j] = b[j];
    }
  } else {
    unpack8<kT == kBF16>(
        *reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(p) + i), v);
  }
}

// The same in two parts, so that several reads are in flight before the first is used.
template <int kT>
struct Raw8 {
  u32x4 w[kT == kF32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const u32x4* q = reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(p) +
                                                    i * (kT == kF32 ? 4 : 2));
#pragma unroll
    for (int j = 0; j < (kT == kF32 ? 2 : 1); ++j) w[j] = q[j];
  }
  __device__ __forceinline__ void widen(float (&v)[8]) const {
    if constexpr (kT == kF32) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j >> 2][j & 3]);
    } else {
      unpack8<kT == kBF16>(w[0], v);
    }
  }
};

__device__ __forceinline__ bool has_row(int32_t at, int64_t R) {
  return at >= 0 && at < R;
}

// Rows that no pair names become 0: the first g.clear workgroups of a launch do that beside the
// others, each for a run of rows, with a bit a row in LDS set from all positions.  The rows are
// other ones than the pairs' own, so nothing is waited for.  4096 tokens, k 8, 2048 columns fp16:
// dispatch 25.3 us with it and 25.0 without, 42.9 with a launch that clears all rows before; combine's
// gradient 51.2, 49.9 and 66.9.
constexpr int kClearGroups = 128;
constexpr int kClearRows = 1 << 16;  // of a workgroup, at most

__device__ __forceinline__ void clear_unnamed(const DispatchArgs& g, int row_chunks) {
  __shared__ uint32_t s_named[kClearRows / 32];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t per = ((g.R + g.clear - 1) / g.clear + 31) / 32 * 32, first = blockIdx.x * per;
  if (first >= g.R) return;
  const int n = (int)min(per, g.R - first);
  // the bits behind the last row stand for rows with a pair
  for (int i = threadIdx.x; i * 32 < n; i += 256)
    s_named[i] = n - i * 32 >= 32 ? 0u : ~0u << (n - i * 32);
  __syncthreads();
  const auto name = [&](int32_t at) {
    const int64_t r = at - first;  // below 0 for a pair without a row
    if (r >= 0 && r < n) atomicOr(&s_named[r >> 5], 1u << (r & 31));
  };
  const int64_t pairs = g.T * g.k;
  constexpr int kAhead = 4;  // reads of four positions in flight
  int64_t p = 0;
  for (; p + kAhead * 1024 <= pairs; p += kAhead * 1024) {
    i32x4 v[kAhead];  // at any word
#pragma unroll
    for (int j = 0; j < kAhead; ++j) __builtin_memcpy(&v[j], g.pos + p + j * 1024 + threadIdx.x * 4, 16);
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) name(v[j][i]);
  }
  for (p += threadIdx.x; p < pairs; p += 256) name(g.pos[p]);
  __syncthreads();
  for (int i = wave; i * 32 < n; i += 4) {
    uint32_t free = ~(uint32_t)__builtin_amdgcn_readfirstlane((int)s_named[i]);
    for (; free; free &= free - 1) {
      u32x4* row = reinterpret_cast<u32x4*>(g.out) + (first + i * 32 + __ffs(free) - 1) * row_chunks;
      for (int c = lane; c < row_chunks; c += 64) row[c] = u32x4{0, 0, 0, 0};
    }
  }
}

}  // namespace

__global__ __launch_bounds__(256) void clear_kernel(u32x4* out, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    out[i] = u32x4{0, 0, 0, 0};
}

// A workgroup takes `toks` tokens (one if a row has 256 chunks of eight or more).
template <int kX, int kRows>
__global__ __launch_bounds__(256) void dispatch_kernel(DispatchArgs g, int c8, int toks) {
  if ((int)blockIdx.x < g.clear) {
    clear_unnamed(g, kRows == kF32 ? 2 * c8 : c8);
    return;
  }
  const int group = blockIdx.x - g.clear, all = gridDim.x - g.clear;
  const int tl = c8 < 256 ? threadIdx.x / c8 : 0;
  const int c0 = threadIdx.x - tl * c8;
  if (tl >= toks) return;
  for (int64_t t = (int64_t)group * toks + tl; t < g.T; t += (int64_t)all * toks) {
    const int32_t* pos = g.pos + t * g.k;
    for (int c = c0; c < c8; c += 256) {
      float v[8];
      load8<kX>(g.x, t * g.H + c * 8, v);
      for (int j = 0; j < g.k; ++j) {
        const int32_t at = pos[j];
        if (!has_row(at, g.R)) continue;
        float o[8];
        const float w = g.w ? g.w[t * g.k + j] : 1.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = g.w ? w * v[i] : v[i];
        store8<kRows>(g.out, (int64_t)at * g.H + c * 8, o);
      }
    }
  }
}

template <int kRows, int kY>
__global__ __launch_bounds__(256) void combine_rows_kernel(DispatchArgs g, int c8, int toks) {
  const int tl = c8 < 256 ? threadIdx.x / c8 : 0;
  const int c0 = threadIdx.x - tl * c8;
  if (tl >= toks) return;
  for (int64_t t = (int64_t)blockIdx.x * toks + tl; t < g.T; t += (int64_t)gridDim.x * toks) {
    const int32_t* pos = g.pos + t * g.k;
    for (int c = c0; c < c8; c += 256) {
      float y[8] = {};
      // four pairs' rows are read together; a pair without one reads row 0 and adds nothing
      for (int j0 = 0; j0 < g.k && g.R > 0; j0 += 4) {
        Raw8<kRows> v[4];
        bool has[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int32_t at = j0 + j < g.k ? pos[j0 + j] : -1;
          has[j] = has_row(at, g.R);
          v[j].load(g.x, (int64_t)(has[j] ? at : 0) * g.H + c * 8);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float w = g.w && has[j] ? g.w[t * g.k + j0 + j] : 1.f;
          float f[8];
          v[j].widen(f);
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = has[j] ? y[i] + w * f[i] : y[i];
        }
      }
      store8<kY>(g.out, t * g.H + c * 8, y);
    }
  }
}

// kWaves waves of a workgroup take one token (one for rows of 512 columns or less: four tokens a
// workgroup), eight pairs at a time: their rows are read together, a pair without one reads
// row 0 and leaves nothing.
template <int kDy, int kRows, int kD, int kWaves>
__global__ __launch_bounds__(256) void combine_bwd_kernel(DispatchArgs g, int c8) {
  constexpr int kToks = 4 / kWaves;
  __shared__ float s_sum[4][8];
  if ((int)blockIdx.x < g.clear) {
    clear_unnamed(g, kD == kF32 ? 2 * c8 : c8);
    return;
  }
  const int group = blockIdx.x - g.clear, all = gridDim.x - g.clear;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int64_t t = (int64_t)group * kToks + wave / kWaves; t < g.T; t += (int64_t)all * kToks) {
    const int32_t* pos = g.pos + t * g.k;
    for (int j0 = 0; j0 < g.k; j0 += 8) {
      float sum[8] = {};
      int32_t at[8];
      float w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        at[j] = j0 + j < g.k ? pos[j0 + j] : -1;
        w[j] = g.w && j0 + j < g.k ? g.w[t * g.k + j0 + j] : 1.f;
      }
      for (int c = threadIdx.x % (64 * kWaves); c < c8 && g.R > 0; c += 64 * kWaves) {
        Raw8<kDy> d;
        Raw8<kRows> v[8];
        d.load(g.x, t * g.H + c * 8);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[j].load(g.rows, (int64_t)(has_row(at[j], g.R) ? at[j] : 0) * g.H + c * 8);
        float dy[8];
        d.widen(dy);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (!has_row(at[j], g.R)) continue;
          float f[8], o[8];
          v[j].widen(f);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            sum[j] += dy[i] * f[i];
            o[i] = w[j] * dy[i];
          }
          if (g.out) store8<kD>(g.out, (int64_t)at[j] * g.H + c * 8, o);
        }
      }
      float* dw = g.dw + t * g.k + j0;
      if constexpr (kWaves == 1) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float all = wave_sum(sum[j]);
          if (lane == j && j0 + j < g.k) dw[j] = all;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float all = wave_sum(sum[j]);
          if (lane == 0) s_sum[wave][j] = all;
        }
        __syncthreads();
        if (threadIdx.x < 8 && j0 + (int)threadIdx.x < g.k) {
          const int j = threadIdx.x;
          dw[j] = (s_sum[0][j] + s_sum[1][j]) + (s_sum[2][j] + s_sum[3][j]);
        }
        __syncthreads();
      }
    }
  }
}

// A wave takes one token.
template <bool kRenorm>
__global__ __launch_bounds__(256) void route_bwd_kernel(RouteBwdArgs g) {
  const int lane = threadIdx.x & 63;
  for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < g.T; t += (int64_t)gridDim.x * 4) {
    const float* l = g.logits + t * g.E;
    int id = -1;
    float dw = 0.f;
    if (lane < g.k) {
      id = g.ids[t * g.k + lane];
      if (id < 0 || id >= g.E) id = -1;
      if (id >= 0) dw = g.dw[t * g.k + lane];
    }
    const bool any = __ballot(id >= 0) != 0;
    const float mine = id >= 0 ? l[id] : -INFINITY;
    float top = mine, all = 0.f;
    if constexpr (!kRenorm) {
      for (int e = lane; e < g.E; e += 64) top = fmaxf(top, l[e]);
    }
    top = wave_max(top);
    const float ex = id >= 0 ? expf(mine - top) : 0.f;
    if constexpr (kRenorm) {
      all = wave_sum(ex);
    } else {
      for (int e = lane; e < g.E; e += 64) all += expf(l[e] - top);
      all = wave_sum(all);
    }
    const float w = id >= 0 ? ex / all : 0.f;
    const float mean = wave_sum(w * dw);
    const float mine_g = kRenorm ? w * (dw - mean) : dw;
    for (int e = lane; e - lane < g.E; e += 64) {
      float v = 0.f;
      for (int j = 0; j < g.k; ++j) {
        const int ij = __builtin_amdgcn_readlane(id, j);
        const float gj = lane_f(mine_g, j);
        if (ij == e) v += gj;
      }
      if (e < g.E) {
        // without a choice nothing was weighted, whatever the logits are (all -inf: p is NaN)
        if constexpr (!kRenorm) v = any ? expf(l[e] - top) / all * (v - mean) : 0.f;
        g.dlogits[t * g.E + e] = v;
      }
    }
  }
}

namespace {

#define NF4MOE_BY_TYPE(dtype, T, ...)          \
  if ((dtype) == kF32) {                       \
    constexpr int T = kF32;                    \
    __VA_ARGS__;                               \
  } else if ((dtype) == kBF16) {               \
    constexpr int T = kBF16;                   \
    __VA_ARGS__;                               \
  } else {                                     \
    constexpr int T = kF16;                    \
    __VA_ARGS__;                               \
  }

// Workgroups of 256; a grid's threads are counted in 32 bits.
unsigned groups(int64_t n) { return (unsigned)std::min<int64_t>(n, 1 << 22); }

// Where g.clear asks for rows without a pair to be cleared: how many workgroups do it, or 0 after a
// launch that has cleared all rows, if they are so short that this is cheaper, or too many.  By
// the bytes of the rows for a pair, with workgroups against a launch before, 524288 pairs (us): 512,
// dispatch 154 and 97, combine's gradient 169 and 180; 1024, 192 and 209, 254 and 330.
hipError_t clear_groups(DispatchArgs& g, hipStream_t s) {
  const int64_t row_bytes = (int64_t)g.H * (g.out_dtype == kF32 ? 4 : 2);
  if (!g.clear) return hipSuccess;
  g.clear = 0;
  if (g.out == nullptr || g.R == 0) return hipSuccess;
  const int n = (int)std::min<int64_t>(kClearGroups, (g.R + 63) / 64);
  if (g.R <= (int64_t)n * kClearRows && g.R * row_bytes >= 1024 * g.T * g.k) {
    g.clear = n;
    return hipSuccess;
  }
  const int64_t n16 = g.R * row_bytes / 16;
  hipLaunchKernelGGL(clear_kernel, dim3(groups((n16 + 255) / 256)), dim3(256), 0, s,
                     reinterpret_cast<u32x4*>(g.out), n16);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dispatch(DispatchArgs g, hipStream_t s) {
  const hipError_t err = clear_groups(g, s);
  if (err != hipSuccess) return err;
  const int c8 = g.H / 8, toks = c8 < 256 ? 256 / c8 : 1;
  const dim3 grid(g.clear + groups((g.T + toks - 1) / toks));
  NF4MOE_BY_TYPE(g.x_dtype, kX, NF4MOE_BY_TYPE(g.out_dtype, kO,
      hipLaunchKernelGGL((dispatch_kernel<kX, kO>), grid, dim3(256), 0, s, g, c8, toks)))
  return hipGetLastError();
}

hipError_t launch_combine_rows(const DispatchArgs& g, hipStream_t s) {
  const int c8 = g.H / 8, toks = c8 < 256 ? 256 / c8 : 1;
  const dim3 grid(groups((g.T + toks - 1) / toks));
  NF4MOE_BY_TYPE(g.x_dtype, kX, NF4MOE_BY_TYPE(g.out_dtype, kO,
      hipLaunchKernelGGL((combine_rows_kernel<kX, kO>), grid, dim3(256), 0, s, g, c8, toks)))
  return hipGetLastError();
}

hipError_t launch_combine_bwd(DispatchArgs g, hipStream_t s) {
  const hipError_t err = clear_groups(g, s);
  if (err != hipSuccess) return err;
  const int c8 = g.H / 8;
  if (c8 <= 64) {
    const dim3 grid(g.clear + groups((g.T + 3) / 4));
    NF4MOE_BY_TYPE(g.x_dtype, kX, NF4MOE_BY_TYPE(g.rows_dtype, kR, NF4MOE_BY_TYPE(g.out_dtype, kO,
        hipLaunchKernelGGL((combine_bwd_kernel<kX, kR, kO, 1>), grid, dim3(256), 0, s, g, c8))))
  } else {
    const dim3 grid(g.clear + groups(g.T));
    NF4MOE_BY_TYPE(g.x_dtype, kX, NF4MOE_BY_TYPE(g.rows_dtype, kR, NF4MOE_BY_TYPE(g.out_dtype, kO,
        hipLaunchKernelGGL((combine_bwd_kernel<kX, kR, kO, 4>), grid, dim3(256), 0, s, g, c8))))
  }
  return hipGetLastError();
}

hipError_t launch_route_bwd(const RouteBwdArgs& g, hipStream_t s) {
  const dim3 grid(groups((g.T + 3) / 4));
  if (g.renormalize)
    hipLaunchKernelGGL(route_bwd_kernel<true>, grid, dim3(256), 0, s, g);
  else
    hipLaunchKernelGGL(route_bwd_kernel<false>, grid, dim3(256), 0, s, g);
  return hipGetLastError();
}

}  // namespace nf4moe
