// Orthogonalisation of a stack of matrices by Newton-Schulz products, for
// sm_100a (as the Muon optimiser applies to an update before it is taken).
//
//   X <- G / (|G|_F + 1e-7), transposed if it has more rows than columns
//   steps times:  A = X X^T,  X <- a X + (b A + c A A) X,   (a, b, c) = (3.4445, -4.7750, 2.0315)
//   out = scale X (transposed back)
//
// On the singular values each step is the polynomial a s + b s^3 + c s^5,
// which lifts small values by a and keeps every value in [0, 1.21]: it stays
// bounded for any number of steps.
#include <cuda_runtime.h>
#include <stdint.h>

#include "train_ops.h"

namespace cgtp {
namespace {

constexpr float kNsA = 3.4445f, kNsB = -4.7750f, kNsC = 2.0315f;
constexpr double kNsEps = 1e-7;

// One block per matrix: X [m][n] (m <= n) = G / (|G|_F + eps).  The squares are
// summed in 64 bits: they can neither overflow nor vanish.
__global__ void __launch_bounds__(512) ortho_start_kernel(int rows, int cols, const float* __restrict__ g,
                                                           float* __restrict__ x) {
  __shared__ double red[512];
  const long long size = (long long)rows * cols;
  g += blockIdx.x * size;
  x += blockIdx.x * size;
  double s = 0.0;
  for (long long i = threadIdx.x; i < size; i += 512) s += (double)g[i] * g[i];
  red[threadIdx.x] = s;
  __syncthreads();
  for (int o = 256; o > 0; o >>= 1) {
    if (threadIdx.x < o) red[threadIdx.x] += red[threadIdx.x + o];
    __syncthreads();
  }
  const double inv = 1.0 / (sqrt(red[0]) + kNsEps);
  for (long long i = threadIdx.x; i < size; i += 512) {
    const long long r = i / cols, c = i % cols;
    x[rows > cols ? c * rows + r : i] = (float)(g[i] * inv);
  }
}

// d = alpha a b + beta e for a stack of matrices, 64 x 64 tiles; B_T: b is
// given transposed.  OUT_T: d is written transposed and scaled.
constexpr int kTile = 64, kDepth = 16;
template <bool B_T>
__global__ void __launch_bounds__(256)
    ortho_product_kernel(int m, int n, int k, const float* __restrict__ a, const float* __restrict__ b, float alpha,
                         float beta, const float* __restrict__ e, float scale, int out_t, float* __restrict__ d) {
  __shared__ float as[kDepth][kTile + 4], bs[kDepth][kTile + 4];
  const long long z = blockIdx.z;
  a += z * m * k;
  b += z * n * k;
  e += z * m * n;
  d += z * m * n;
  const int m0 = blockIdx.y * kTile, n0 = blockIdx.x * kTile;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < k; k0 += kDepth) {
    for (int i = threadIdx.x; i < kTile * kDepth; i += 256) {
      const int r = i / kDepth, q = i % kDepth;
      as[q][r] = m0 + r < m && k0 + q < k ? a[(long long)(m0 + r) * k + k0 + q] : 0.f;
      if (B_T) bs[q][r] = n0 + r < n && k0 + q < k ? b[(long long)(n0 + r) * k + k0 + q] : 0.f;
    }
    if (!B_T)
      for (int i = threadIdx.x; i < kTile * kDepth; i += 256) {
        const int q = i / kTile, r = i % kTile;
        bs[q][r] = n0 + r < n && k0 + q < k ? b[(long long)(k0 + q) * n + n0 + r] : 0.f;
      }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kDepth; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(as[q][ty * 4 + i], bs[q][tx * 4 + j], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int r = m0 + ty * 4 + i, c = n0 + tx * 4 + j;
      if (r < m && c < n)
        d[out_t ? (long long)c * m + r : (long long)r * n + c] =
            scale * fmaf(alpha, acc[i][j], beta == 0.f ? 0.f : beta * e[(long long)r * n + c]);
    }
}

}  // namespace

size_t ortho_workspace(int batch, int rows, int cols) {
  const size_t m = rows < cols ? rows : cols, n = rows < cols ? cols : rows;
  return 2 * pad256(sizeof(float) * batch * m * n) + 2 * pad256(sizeof(float) * batch * m * m);
}

cudaError_t launch_ortho(int batch, int rows, int cols, int steps, float scale, const float* g, float* out, void* ws,
                         cudaStream_t stream) {
  if (batch == 0 || rows == 0 || cols == 0) return cudaSuccess;
  const int m = rows < cols ? rows : cols, n = rows < cols ? cols : rows;
  const size_t xb = pad256(sizeof(float) * (size_t)batch * m * n), ab = pad256(sizeof(float) * (size_t)batch * m * m);
  float* x[2] = {(float*)ws, (float*)((char*)ws + xb)};
  float* a = (float*)((char*)ws + 2 * xb);
  float* p = (float*)((char*)ws + 2 * xb + ab);
  ortho_start_kernel<<<batch, 512, 0, stream>>>(rows, cols, g, x[0]);
  cudaError_t e = cudaGetLastError();
  const unsigned tm = (m + kTile - 1) / kTile, tn = (n + kTile - 1) / kTile;
  for (int s = 0; s < steps && e == cudaSuccess; ++s) {
    const bool last = s + 1 == steps;
    ortho_product_kernel<true><<<dim3(tm, tm, batch), 256, 0, stream>>>(m, m, n, x[0], x[0], 1.f, 0.f, x[0], 1.f, 0, a);
    ortho_product_kernel<true><<<dim3(tm, tm, batch), 256, 0, stream>>>(m, m, m, a, a, kNsC, kNsB, a, 1.f, 0, p);
    ortho_product_kernel<false><<<dim3(tn, tm, batch), 256, 0, stream>>>(
        m, n, m, p, x[0], 1.f, kNsA, x[0], last ? scale : 1.f, last && rows > cols, last ? out : x[1]);
    float* t = x[0];
    x[0] = x[1];
    x[1] = t;
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace cgtp
