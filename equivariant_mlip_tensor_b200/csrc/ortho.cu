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
//
// The products run on the tensor cores in fp16 pairs: x 2^k = high + low holds 22
// bits of x, and low high + high low + high high, summed in fp32, leaves out
// only low low (2^-22 of a product and less), so three fp16 products give a
// product of fp32 accuracy.  That the values stay bounded makes fixed powers
// of two fit: entries of X and of X X^T are at most 1.21 and 1.45 (x 2^14 <
// 65504), those of a + b A + c A A at most 3.45 (x 2^13).  Norms and sums stay
// in fp32 and above; a X is taken into the last product by adding a to the diagonal of
// b A + c A A.
#include <cuda_runtime.h>
#include <stdint.h>

#include "tc.cuh"
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

// ---------------------------------------------------------- the short side up to 128
// All steps of one matrix in one launch: a cluster of 1, 2, 4 or 8 blocks holds
// X, each its own columns, as fp16 pairs in shared memory from the first step
// to the last; A and a + b A + c A A (at most 128 x 128) are in every block.
// The same tile of X is read along its rows for X X^T and down its rows for
// the last product.  With more than one block, the blocks' parts of X X^T meet
// in cluster shared memory: each block sums its share of the entries over the
// blocks in order and writes it to all.
constexpr int kSmallThreads = 256;
constexpr int kSmallSide = 128;                // rows of X
constexpr int kSmallColumns = 256;             // columns of X in one block
constexpr float kXScale = 16384.f, kPScale = 8192.f;

struct SmallArgs {
  int rows, cols, steps, m, n, tall;
  int mp, nj;  // rows (padded to 16) and columns of X per block (a multiple of 16)
  float scale;
  const float* g;
  float* out;
};

// Shared memory of a block: X as two sets of 64-column tiles, then A (two sets
// again), whose place the fp32 parts of X X^T take before A is known; a full
// set of 128 rows behind the last tile is always inside the allocation,
// because an operand of M = 128 rows reads that far (those rows of the result
// are not used).
struct SmallLayout {
  int x_set, a_set, part_stride, bytes;
};
__host__ __device__ inline SmallLayout small_layout(int mp, int nj, int blocks) {
  SmallLayout L;
  L.x_set = (nj + 63) / 64 * mp * 128;
  L.a_set = (mp + 63) / 64 * mp * 128;
  L.part_stride = mp + 4;  // floats: rows 16 bytes apart modulo 128, no bank conflicts of 16-byte stores
  const int part = blocks > 1 ? mp * L.part_stride * 4 : 0;
  const int a_bytes = 2 * L.a_set > part ? 2 * L.a_set : part;
  L.bytes = 2 * L.x_set + a_bytes + (128 - mp) * 128 + 1024;
  return L;
}

// Element (r, c) of X before scaling: row r of G, or column r where G is tall.
__device__ __forceinline__ float small_input(const SmallArgs& a, const float* g, int r, int c) {
  if (r >= a.m || c >= a.n) return 0.f;
  return g[a.tall ? (long long)c * a.cols + r : (long long)r * a.cols + c];
}

__global__ void __launch_bounds__(kSmallThreads, 1) ortho_small_kernel(SmallArgs a, int blocks) {
  extern __shared__ uint8_t raw[];
  __shared__ double sums[kSmallThreads / 32];
  __shared__ double block_sum;
  __shared__ uint32_t tmem_slot;
  __shared__ uint64_t bar_word;
  const SmallLayout L = small_layout(a.mp, a.nj, blocks);
  uint8_t* base = raw + ((1024 - (tc::smem_addr(raw) & 1023)) & 1023);
  uint8_t* xs = base;
  uint8_t* as = base + 2 * L.x_set;
  float* part = reinterpret_cast<float*>(as);
  const uint32_t x_addr = tc::smem_addr(xs), a_addr = tc::smem_addr(as), bar = tc::smem_addr(&bar_word);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x % blocks, matrix = blockIdx.x / blocks;
  const int c0 = rank * a.nj;
  const float* g = a.g + (long long)matrix * a.rows * a.cols;
  float* out = a.out + (long long)matrix * a.rows * a.cols;
  uint32_t columns = 32;
  while ((int)columns < a.mp || (int)columns < a.nj) columns <<= 1;

  if (warp == 0) tc::tmem_alloc(tc::smem_addr(&tmem_slot), columns);
  if (tid == 0) tc::mbar_init(bar, 1);

  // Frobenius norm, squares in 64 bits: they neither overflow nor vanish
  const int units = a.nj / 8;  // 8-column units of a row
  double s = 0.0;
  for (int q = tid; q < a.mp * units; q += kSmallThreads) {
    const int r = a.tall ? q % a.mp : q / units, u = a.tall ? q / a.mp : q % units;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double v = small_input(a, g, r, c0 + 8 * u + i);
      s = fma(v, v, s);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) sums[warp] = s;
  __syncthreads();
  if (tid == 0) {
    s = 0.0;
    for (int w = 0; w < kSmallThreads / 32; ++w) s += sums[w];
    block_sum = s;
  }
  if (blocks > 1) tc::cluster_sync();
  else __syncthreads();
  s = 0.0;
  for (int k = 0; k < blocks; ++k)
    s += blocks > 1 ? tc::peer_load_double(tc::peer_addr(tc::smem_addr(&block_sum), k)) : block_sum;
  const double inv = 1.0 / (sqrt(s) + kNsEps);

  // X as fp16 pairs; rows m.. and columns n.. are zero
  for (int q = tid; q < a.mp * units; q += kSmallThreads) {
    const int r = a.tall ? q % a.mp : q / units, u = a.tall ? q / a.mp : q % units;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)(small_input(a, g, r, c0 + 8 * u + i) * inv);
    uint4 hi, lo;
    tc::split8(v, kXScale, hi, lo);
    const uint32_t at = (u >> 3) * a.mp * 128 + tc::tile_unit(r, u & 7);
    *reinterpret_cast<uint4*>(xs + at) = hi;
    *reinterpret_cast<uint4*>(xs + L.x_set + at) = lo;
  }
  tc::fence_async();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = tmem_slot;

  // One thread issues the three products of a contraction: low high, high low, high high
  const uint32_t row_set = a.mp * 128;
  auto rows_by_rows = [&](uint32_t addr, uint32_t set, int k) {  // tile tile^T
    for (int p = 0; p < 3; ++p) {
      const uint32_t oa = p == 0 ? set : 0, ob = p == 1 ? set : 0;
      for (int i = 0; i < k / 16; ++i) {
        const uint32_t at = addr + (i >> 2) * row_set + (i & 3) * 32;
        tc::mma(tmem, tc::desc_k(at + oa), tc::desc_k(at + ob), tc::instruction(a.mp, false), p > 0 || i > 0);
      }
    }
    tc::commit(bar);
  };
  auto rows_by_columns = [&]() {  // P X
    for (int p = 0; p < 3; ++p) {
      const uint32_t oa = p == 0 ? L.a_set : 0, ob = p == 1 ? L.x_set : 0;
      for (int i = 0; i < a.mp / 16; ++i)
        tc::mma(tmem, tc::desc_k(a_addr + oa + (i >> 2) * row_set + (i & 3) * 32),
                tc::desc_mn(x_addr + ob + i * 2048, row_set), tc::instruction(a.nj, true), p > 0 || i > 0);
    }
    tc::commit(bar);
  };
  // this thread's row of the accumulator, and every other 16 of its columns
  const int r = (warp & 3) * 32 + lane, half = warp >> 2;
  const uint32_t t_row = tmem + ((uint32_t)((warp & 3) * 32) << 16);
  const bool live = (warp & 3) * 32 < a.mp;  // the warp's rows hold part of the result
  uint32_t parity = 0;
  bool ok = true;
  auto wait = [&]() {
    if (ok) ok = tc::mbar_wait(bar, parity);
    parity ^= 1;
    tc::fence_after_sync();
  };
  auto ready = [&]() {  // what the threads wrote is there for the next products
    tc::fence_async();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
  };

  for (int step = 0; step < a.steps; ++step) {
    // A = X X^T
    if (tid == 0) rows_by_rows(x_addr, L.x_set, a.nj);
    wait();
    if (live) {
      for (int c = half * 16; c < a.mp; c += 32) {
        float v[16];
        tc::tmem_load16(t_row + c, v);
        if (r < a.mp) {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] *= 1.f / (kXScale * kXScale);
          if (blocks > 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              reinterpret_cast<float4*>(part + r * L.part_stride + c)[i] =
                  make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float w[8] = {v[8 * h],     v[8 * h + 1], v[8 * h + 2], v[8 * h + 3],
                                  v[8 * h + 4], v[8 * h + 5], v[8 * h + 6], v[8 * h + 7]};
              uint4 hi, lo;
              tc::split8(w, kXScale, hi, lo);
              const uint32_t at = (c >> 6) * row_set + tc::tile_unit(r, ((c >> 3) + h) & 7);
              *reinterpret_cast<uint4*>(as + at) = hi;
              *reinterpret_cast<uint4*>(as + L.a_set + at) = lo;
            }
          }
        }
      }
    }
    if (blocks > 1) {
      tc::cluster_sync();  // every block's part is there
      const int row_units = a.mp / 8, all = a.mp * row_units;
      const int u0 = rank * all / blocks, u1 = (rank + 1) * all / blocks;
      constexpr int kMost = kSmallSide * kSmallSide / 8 / 2 / kSmallThreads;  // units a thread, 2 blocks
      uint4 hi[kMost], lo[kMost];
#pragma unroll
      for (int k = 0; k < kMost; ++k) {
        const int u = u0 + tid + k * kSmallThreads;
        float w[8] = {};
        if (u < u1) {
          const uint32_t at = a_addr + ((u / row_units) * L.part_stride + u % row_units * 8) * 4;
          for (int b = 0; b < blocks; ++b) {
            const uint32_t from = tc::peer_addr(at, b);
            const float4 p = tc::peer_load4(from), q = tc::peer_load4(from + 16);
            w[0] += p.x, w[1] += p.y, w[2] += p.z, w[3] += p.w;
            w[4] += q.x, w[5] += q.y, w[6] += q.z, w[7] += q.w;
          }
        }
        tc::split8(w, kXScale, hi[k], lo[k]);
      }
      tc::cluster_sync();  // every part has been read: A may take its place
#pragma unroll
      for (int k = 0; k < kMost; ++k) {
        const int u = u0 + tid + k * kSmallThreads;
        if (u >= u1) continue;
        const int rr = u / row_units, cu = u % row_units;
        const uint32_t at = a_addr + (cu >> 3) * row_set + tc::tile_unit(rr, cu & 7);
        for (int b = 0; b < blocks; ++b) {
          tc::peer_store16(tc::peer_addr(at, b), hi[k]);
          tc::peer_store16(tc::peer_addr(at + L.a_set, b), lo[k]);
        }
      }
      tc::fence_async();
      tc::cluster_sync();
    }
    ready();
    // A A
    if (tid == 0) rows_by_rows(a_addr, L.a_set, a.mp);
    wait();
    if (live) {
      for (int c = half * 16; c < a.mp; c += 32) {
        float v[16];
        tc::tmem_load16(t_row + c, v);
        if (r < a.mp) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t at = (c >> 6) * row_set + tc::tile_unit(r, ((c >> 3) + h) & 7);
            uint4 hi = *reinterpret_cast<const uint4*>(as + at), lo = *reinterpret_cast<const uint4*>(as + L.a_set + at);
            float w[8];
            tc::join8(hi, lo, 1.f / kXScale, w);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              w[i] = fmaf(kNsC / (kXScale * kXScale), v[8 * h + i], fmaf(kNsB, w[i], c + 8 * h + i == r ? kNsA : 0.f));
            tc::split8(w, kPScale, hi, lo);
            *reinterpret_cast<uint4*>(as + at) = hi;
            *reinterpret_cast<uint4*>(as + L.a_set + at) = lo;
          }
        }
      }
    }
    ready();
    // X = (a + b A + c A A) X
    if (tid == 0) rows_by_columns();
    wait();
    const bool last = step + 1 == a.steps;
    if (live) {
      for (int c = half * 16; c < a.nj; c += 32) {
        float v[16];
        tc::tmem_load16(t_row + c, v);
        if (r < a.mp) {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] *= 1.f / (kXScale * kPScale);
          if (!last) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float w[8] = {v[8 * h],     v[8 * h + 1], v[8 * h + 2], v[8 * h + 3],
                                  v[8 * h + 4], v[8 * h + 5], v[8 * h + 6], v[8 * h + 7]};
              uint4 hi, lo;
              tc::split8(w, kXScale, hi, lo);
              const uint32_t at = (c >> 6) * row_set + tc::tile_unit(r, ((c >> 3) + h) & 7);
              *reinterpret_cast<uint4*>(xs + at) = hi;
              *reinterpret_cast<uint4*>(xs + L.x_set + at) = lo;
            }
          } else if (r < a.m) {
            const float bad = __int_as_float(0x7fffffff);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = ok ? v[i] * a.scale : bad;
            if (a.tall) {
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (c0 + c + i < a.n) out[(long long)(c0 + c + i) * a.cols + r] = v[i];
            } else if (a.cols % 4 == 0 && (reinterpret_cast<uintptr_t>(a.out) & 15) == 0) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (c0 + c + 4 * i < a.n)
                  *reinterpret_cast<float4*>(out + (long long)r * a.cols + c0 + c + 4 * i) =
                      make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (c0 + c + i < a.n) out[(long long)r * a.cols + c0 + c + i] = v[i];
            }
          }
        }
      }
    }
    ready();
  }
  if (warp == 0) tc::tmem_free(tmem, columns);
  if (blocks > 1) tc::cluster_sync();  // no block leaves while another may still read its shared memory
}

// Blocks per matrix: as few as hold its columns (1, 2, 4 or 8).
int small_blocks(int m, int n) {
  if (m > kSmallSide) return 0;
  for (int b = 1; b <= 8; b *= 2)
    if (n <= b * kSmallColumns) return b;
  return 0;
}

cudaError_t launch_small(int batch, int rows, int cols, int steps, float scale, const float* g, float* out,
                         cudaStream_t stream) {
  SmallArgs a{};
  a.rows = rows;
  a.cols = cols;
  a.steps = steps;
  a.tall = rows > cols;
  a.m = a.tall ? cols : rows;
  a.n = a.tall ? rows : cols;
  const int blocks = small_blocks(a.m, a.n);
  a.mp = (a.m + 15) / 16 * 16;
  a.nj = ((a.n + blocks - 1) / blocks + 15) / 16 * 16;
  a.scale = scale;
  a.g = g;
  a.out = out;
  const int bytes = small_layout(a.mp, a.nj, blocks).bytes;
  cudaError_t e = cudaFuncSetAttribute(ortho_small_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)batch * blocks);
  cfg.blockDim = dim3(kSmallThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = blocks;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = blocks > 1 ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, ortho_small_kernel, a, blocks);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t ortho_workspace(int batch, int rows, int cols) {
  const size_t m = rows < cols ? rows : cols, n = rows < cols ? cols : rows;
  if (small_blocks((int)m, (int)n) > 0) return 0;
  return 2 * pad256(sizeof(float) * batch * m * n) + 2 * pad256(sizeof(float) * batch * m * m);
}

cudaError_t launch_ortho(int batch, int rows, int cols, int steps, float scale, const float* g, float* out, void* ws,
                         cudaStream_t stream) {
  if (batch == 0 || rows == 0 || cols == 0) return cudaSuccess;
  const int m = rows < cols ? rows : cols, n = rows < cols ? cols : rows;
  if (small_blocks(m, n) > 0) return launch_small(batch, rows, cols, steps, scale, g, out, stream);
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
