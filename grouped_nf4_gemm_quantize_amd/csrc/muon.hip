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
// O are 64-bit.
//
// Two launches over (factor, chunk of the long axis): the first updates m and
// leaves each chunk's part of u u^T in the workspace, the second adds the parts in
// chunk order, does the r x r algebra and applies P to its chunk.

#include "common.h"
#include "launch.h"

namespace nf4moe {

namespace {

constexpr int kCols = 256;  // long-axis elements of a workgroup

__device__ __forceinline__ float load1(const void* p, int dtype, int64_t i) {
  if (dtype == kF32) return reinterpret_cast<const float*>(p)[i];
  const uint16_t raw = reinterpret_cast<const uint16_t*>(p)[i];
  return dtype == kBF16 ? bf16_bits_to_f32(raw) : (float)__builtin_bit_cast(_Float16, raw);
}

__device__ __forceinline__ void store1(void* p, int dtype, int64_t i, float v) {
  if (dtype == kF32) reinterpret_cast<float*>(p)[i] = v;
  else if (dtype == kBF16) reinterpret_cast<uint16_t*>(p)[i] = f32_to_bf16_bits(v);
  else reinterpret_cast<_Float16*>(p)[i] = (_Float16)v;
}

}  // namespace

template <bool kApply>
__global__ __launch_bounds__(256) void muon_kernel(MuonArgs a) {
  __shared__ float u[16][kCols + 1];
  __shared__ double gm[16][17], pm[16][17], qm[16][17], tm[16][17];
  int ti = 0;
  while (ti + 1 < a.count && (int)blockIdx.x >= a.t[ti + 1].block0) ++ti;
  const MuonTensor& t = a.t[ti];
  const int local = blockIdx.x - t.block0;
  const int e = local / t.chunks, chunk = local - e * t.chunks;
  const int r = t.r, tid = threadIdx.x;
  const int64_t c0 = (int64_t)chunk * kCols;
  const int nc = t.n - c0 < kCols ? (int)(t.n - c0) : kCols;
  const int64_t base = (int64_t)e * r * t.n;
  const int64_t sr = t.rank_major ? t.n : 1, sc = t.rank_major ? 1 : r;

  for (int q = tid; q < r * kCols; q += 256) {
    const int j = t.rank_major ? q / kCols : q % r, c = t.rank_major ? q % kCols : q / r;
    float v = 0.f;
    if (c < nc) {
      const int64_t i = base + j * sr + (c0 + c) * sc;
      const float g = load1(t.g, t.g_dtype, i);
      v = g;
      if (t.m) {
        // the second launch reads the updated m, which may be in place
        const float m = kApply ? t.m_out[i] : fmaf(a.mu, t.m[i], g);
        if (!kApply) t.m_out[i] = m;
        v = a.nesterov ? fmaf(a.mu, m, g) : m;
      }
    }
    u[j][c] = v;
  }
  const int i = tid >> 4, j = tid & 15;
  const bool in = i < r && j < r;
  double* gram = t.gram + (int64_t)e * t.chunks * r * r;
  if constexpr (!kApply) {
    __syncthreads();
    if (!in) return;
    double s = 0.0;
    for (int c = 0; c < nc; ++c) s += (double)u[i][c] * (double)u[j][c];
    gram[(int64_t)chunk * r * r + i * r + j] = s;
  } else {
    double g0 = 0.0;
    if (in)
      for (int c = 0; c < t.chunks; ++c) g0 += gram[(int64_t)c * r * r + i * r + j];
    gm[i][j] = g0;
    __syncthreads();
    double norm2 = 0.0;
    for (int k = 0; k < r; ++k) norm2 += gm[k][k];
    const double scale = 1.0 / (sqrt(norm2) + a.eps);
    const double inv = norm2 == 0.0 ? 0.0 : scale;
    __syncthreads();
    gm[i][j] = g0 * inv * inv;
    pm[i][j] = i == j ? 1.0 : 0.0;
    __syncthreads();
    for (int step = 0; step < a.steps; ++step) {
      double g2 = 0.0;
      for (int k = 0; k < 16; ++k) g2 += gm[i][k] * gm[k][j];
      qm[i][j] = (i == j ? a.a : 0.0) + a.b * gm[i][j] + a.c * g2;
      __syncthreads();
      double p = 0.0, w = 0.0;
      for (int k = 0; k < 16; ++k) {
        p += qm[i][k] * pm[k][j];
        w += qm[i][k] * gm[k][j];
      }
      tm[i][j] = w;
      __syncthreads();
      double g = 0.0;
      for (int k = 0; k < 16; ++k) g += tm[i][k] * qm[k][j];
      pm[i][j] = p;
      gm[i][j] = g;
      __syncthreads();
    }
    for (int q = tid; q < r * kCols; q += 256) {
      const int jj = t.rank_major ? q / kCols : q % r, c = t.rank_major ? q % kCols : q / r;
      if (c >= nc) continue;
      double o = 0.0;
      for (int k = 0; k < r; ++k) o += pm[jj][k] * (double)u[k][c];
      o *= inv;
      const int64_t at = base + jj * sr + (c0 + c) * sc;
      float w;
      if (t.w)
        w = (float)((double)load1(t.w, t.w_dtype, at) * (1.0 - a.lr * a.weight_decay) -
                    a.lr * t.scale * o);
      else
        w = (float)o;
      store1(t.w_out, t.w_dtype, at, w);
      if (t.w16) store1(t.w16, t.w16_dtype, at, w);
    }
  }
}

int muon_chunks(int64_t n, int r) {
  (void)r;
  return (int)((n + kCols - 1) / kCols);
}

hipError_t launch_muon(const MuonArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(muon_kernel<false>, dim3(a.blocks), dim3(256), 0, s, a);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL(muon_kernel<true>, dim3(a.blocks), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace nf4moe
