// Group norm with an activation over channels-last rows, one normalisation
// per graph (sample) and channel group, forward and backward, for sm_100a.
//
//   over the rows of a sample x the channels of a group: mean, var (biased)
//   h = (x - mean) rstd, rstd = 1 / sqrt(var + eps);  z = gamma h + beta;  y = act(z)
//   gz = grad_y act'(z);  t = gamma gz
//   grad_x = rstd (t - <t> - h <t h>);  grad_gamma = sum gz h;  grad_beta = sum gz
//
// Bound by memory: the forward has to read x and write y, the backward to read
// x and grad_y and write grad_x.  Samples may have any length (graph offsets
// on the device), and two splits of the work share that:
//
// Fused: a block, or a cluster of 2, 4 or 8 that cut the sample's rows, owns one
// sample and one slab of whole groups.  The rows stay in registers between the
// statistics and the result; rows beyond the registers are read again, which
// finds them in L2.
//
// Tiles, for samples so long that a cluster's few blocks could not draw on the
// memory: the rows are cut into tiles of equal length whatever the samples are.
// The part of sample s in tile t has the slot t + s of its own: going down the
// rows, each step moves to the next tile or the next sample, so no two parts
// share a slot.
//   1. each tile reduces each of its parts per channel into the part's slot;
//   2. one group of threads per (sample, group) joins the slots in order;
//   3. each tile reads its rows again and writes the result.
//
// Statistics are means and sums of squared deviations from a mean, joined as
// such, in fp32: deviations are from the mean of their own rows or of the whole group, so no
// sum of squares has an offset or an outlier to cancel.
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "tc.cuh"
#include "train_ops.h"

namespace cgtp {
namespace {

constexpr int kNormThreads = 256;  // of the tiles
constexpr int kNormRows = 8;       // rows per thread of the tiles, held in registers
constexpr int kFusedMost = 512;    // threads of a fused block, at most

// VEC columns of a row; the packed fp32 operations take two at a time.
template <int VEC>
struct Vec {
  float v[VEC];
};
template <int VEC>
__device__ __forceinline__ Vec<VEC> load_vec(const float* p) {
  Vec<VEC> r;
  if constexpr (VEC == 4) {
    const float4 q = *reinterpret_cast<const float4*>(p);
    r.v[0] = q.x;
    r.v[1] = q.y;
    r.v[2] = q.z;
    r.v[3] = q.w;
  } else {
    r.v[0] = *p;
  }
  return r;
}
template <int VEC>
__device__ __forceinline__ void store_vec(float* p, const Vec<VEC>& a) {
  if constexpr (VEC == 4) *reinterpret_cast<float4*>(p) = make_float4(a.v[0], a.v[1], a.v[2], a.v[3]);
  else *p = a.v[0];
}
template <int VEC>
__device__ __forceinline__ Vec<VEC> fma(const Vec<VEC>& a, const Vec<VEC>& b, const Vec<VEC>& c) {
  Vec<VEC> r;
  if constexpr (VEC == 4) {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const float2 q = __ffma2_rn(make_float2(a.v[i], a.v[i + 1]), make_float2(b.v[i], b.v[i + 1]),
                                  make_float2(c.v[i], c.v[i + 1]));
      r.v[i] = q.x;
      r.v[i + 1] = q.y;
    }
  } else {
    r.v[0] = fmaf(a.v[0], b.v[0], c.v[0]);
  }
  return r;
}
template <int VEC>
__device__ __forceinline__ Vec<VEC> operator+(const Vec<VEC>& a, const Vec<VEC>& b) {
  Vec<VEC> r;
  if constexpr (VEC == 4) {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const float2 q = __fadd2_rn(make_float2(a.v[i], a.v[i + 1]), make_float2(b.v[i], b.v[i + 1]));
      r.v[i] = q.x;
      r.v[i + 1] = q.y;
    }
  } else {
    r.v[0] = a.v[0] + b.v[0];
  }
  return r;
}
template <int VEC>
__device__ __forceinline__ Vec<VEC> operator*(const Vec<VEC>& a, const Vec<VEC>& b) {
  Vec<VEC> r;
  if constexpr (VEC == 4) {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const float2 q = __fmul2_rn(make_float2(a.v[i], a.v[i + 1]), make_float2(b.v[i], b.v[i + 1]));
      r.v[i] = q.x;
      r.v[i + 1] = q.y;
    }
  } else {
    r.v[0] = a.v[0] * b.v[0];
  }
  return r;
}
template <int VEC>
__device__ __forceinline__ Vec<VEC> all(float s) {
  Vec<VEC> r;
#pragma unroll
  for (int i = 0; i < VEC; ++i) r.v[i] = s;
  return r;
}

// 1 / (1 + exp(-z)) by the hardware's base-2 exponential and reciprocal, and 0 or 1
// at the ends.  The exponential is off by some (|z| + 3) 2^-24 of itself, of which 1 - s
// reaches s; the sum 1 + e and the reciprocal add some 3 x 2^-24 wherever z lies.
__device__ __forceinline__ float sigmoid(float z) {
  float e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + e));
  return s;
}
template <bool SILU, int VEC>
__device__ __forceinline__ Vec<VEC> activate(const Vec<VEC>& z) {
  Vec<VEC> s = all<VEC>(1.f);
  if (SILU)
#pragma unroll
    for (int i = 0; i < VEC; ++i) s.v[i] = sigmoid(z.v[i]);
  return SILU ? z * s : z;
}
// g act'(z)
template <bool SILU, int VEC>
__device__ __forceinline__ Vec<VEC> activate_grad(const Vec<VEC>& z, const Vec<VEC>& g) {
  const Vec<VEC> one = all<VEC>(1.f);
  Vec<VEC> s = one;
  if (SILU)
#pragma unroll
    for (int i = 0; i < VEC; ++i) s.v[i] = sigmoid(z.v[i]);
  return SILU ? g * s * fma(z, fma(s, all<VEC>(-1.f), one), one) : g;
}

// Bounds of sample s, clamped into [0, n].
__device__ __forceinline__ int2 sample_rows(const NormArgs& a, int s) {
  if (a.ptr == nullptr) return make_int2(0, a.n);
  const int lo = min(max(a.ptr[s], 0), a.n);
  return make_int2(lo, min(max(a.ptr[s + 1], lo), a.n));
}

// The scale, shift, -mean and rstd of a thread's columns in sample s.
template <int VEC>
struct Columns {
  Vec<VEC> gamma, beta, minus_mean, rstd;
  __device__ __forceinline__ void load_params(const NormArgs& a, int col) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      gamma.v[j] = a.gamma == nullptr ? 1.f : a.gamma[col + j];
      beta.v[j] = a.beta == nullptr ? 0.f : a.beta[col + j];
    }
  }
  __device__ __forceinline__ void load_stats(const NormArgs& a, int col, int s) {
    const int cpg = a.channels / a.groups;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const long long k = (long long)s * a.groups + (col + j) / cpg;
      minus_mean.v[j] = -a.mean[k];
      rstd.v[j] = a.rstd[k];
    }
  }
  __device__ __forceinline__ Vec<VEC> normalised(const Vec<VEC>& x) const { return (x + minus_mean) * rstd; }
};

// ------------------------------------------------------------------- fused
constexpr int kSlabColumns = 128;
struct Slabs {
  int lanes;        // threads across a slab's columns (a power of two, at most 32)
  int groups;       // whole groups of a slab
  int count;        // slabs
  int blocks;       // blocks per sample and slab (a cluster): 1 << shift
  int threads;      // of a block
  int rows;         // rows per thread, held in registers
  int shift;
  unsigned per_cpg; // 2^20 / channels per group, rounded up
  int team;         // threads that sum one group (a power of two, at most 32)
};
// x / (channels per group), x < 16 * 128: the product is over by less than 2^11 of 2^20, a step is 2^13 at least
__device__ __forceinline__ int group_of(const Slabs& f, int x) { return (int)((unsigned)x * f.per_cpg >> 20); }

// What the threads of a block share: column sums by warp, then by column or by group.
struct FusedShared {
  float red[2][kFusedMost / 32][kSlabColumns];
  float col[2][kSlabColumns];
  float sum[2][kSlabColumns];    // by group: this block's
  float total[2][kSlabColumns];  // by group: the results that every block of the cluster has
};

struct Place {
  int sample, part, lane, ty, nty, c0, columns, groups, cpg, g0, col, r0, r1, rows;
  bool on;
};
template <int VEC>
__device__ __forceinline__ Place place_of(const NormArgs& a, const Slabs& f) {
  Place p;
  p.part = blockIdx.x & (f.blocks - 1);
  p.sample = blockIdx.x >> f.shift;
  int slab = 0;
  if (f.count > 1) {
    slab = p.sample % f.count;
    p.sample /= f.count;
  }
  p.cpg = a.channels / a.groups;
  p.lane = threadIdx.x & (f.lanes - 1);
  p.ty = threadIdx.x / f.lanes;
  p.nty = blockDim.x / f.lanes;
  p.g0 = slab * f.groups;
  p.groups = min(f.groups, a.groups - p.g0);
  p.c0 = p.g0 * p.cpg;
  p.columns = p.groups * p.cpg;
  p.col = p.c0 + p.lane * VEC;
  p.on = p.lane * VEC < p.columns;
  const int2 b = sample_rows(a, p.sample);
  p.rows = b.y - b.x;
  p.r0 = b.x + (int)((long long)p.rows * p.part >> f.shift);
  p.r1 = b.x + (int)((long long)p.rows * (p.part + 1) >> f.shift);
  return p;
}

// Sums over the rows of a block: lanes of a warp with the same columns, then
// (in shared memory) the warps, in a fixed order.
template <int VEC>
__device__ __forceinline__ void sum_rows(Vec<VEC> v, const Place& p, int lanes, float (*red)[kSlabColumns]) {
  for (int o = lanes; o < 32; o <<= 1)
#pragma unroll
    for (int j = 0; j < VEC; ++j) v.v[j] += __shfl_xor_sync(0xffffffffu, v.v[j], o);
  if ((threadIdx.x & 31) < lanes && p.lane * VEC < kSlabColumns) store_vec<VEC>(&red[threadIdx.x >> 5][p.lane * VEC], v);
}

// For each group of the slab, value(g, e) summed over e < count by a team of
// threads, in a fixed order; last(g, sum) on one thread.
template <class V, class L>
__device__ __forceinline__ void team_sums(const Place& p, int team, int count, V&& value, L&& last) {
  const int mine = threadIdx.x & (team - 1), teams = blockDim.x / team;
  for (int g0 = 0; g0 < p.groups; g0 += teams) {  // the same for every thread
    const int g = g0 + threadIdx.x / team;
    float s = 0.f;
    if (g < p.groups)
      for (int e = mine; e < count; e += team) s += value(g, e);
    for (int o = team >> 1; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (g < p.groups && mine == 0) last(g, s);
  }
}
// result(sum) of each group over the columns (and warps) of red and over the cluster, into total.
template <class R>
__device__ __forceinline__ void sum_groups(const Place& p, const Slabs& f, const float (*red)[kSlabColumns], float* sum,
                                           float* total, R&& result) {
  __syncthreads();
  const auto value = [&](int g, int e) {
    const int w = group_of(f, e);
    return red[w][g * p.cpg + e - w * p.cpg];
  };
  const int count = (int)(blockDim.x >> 5) * p.cpg;
  if (f.blocks == 1) {
    team_sums(p, f.team, count, value, [&](int g, float s) { total[g] = result(g, s); });
  } else {
    team_sums(p, f.team, count, value, [&](int g, float s) { sum[g] = s; });
    __syncwarp();
    tc::cluster_sync();
    for (int g = threadIdx.x; g < p.groups; g += blockDim.x) {
      float s = 0.f;
      for (int k = 0; k < f.blocks; ++k) s += tc::peer_load(tc::peer_addr(tc::smem_addr(sum + g), k));
      total[g] = result(g, s);
    }
  }
  __syncthreads();
}

template <int VEC, bool SILU, int ROWS>
__global__ void __launch_bounds__(kFusedMost) norm_fused_kernel(NormArgs a, Slabs f) {
  __shared__ __align__(16) FusedShared sh;
  const Place p = place_of<VEC>(a, f);
  const long long stat0 = (long long)p.sample * a.groups + p.g0;
  if (p.rows == 0) {
    if (p.part == 0)
      for (int g = threadIdx.x; g < p.groups; g += blockDim.x) {
        a.mean[stat0 + g] = 0.f;
        a.rstd[stat0 + g] = 1.f / sqrtf(a.eps);
      }
    return;  // every block of the cluster
  }
  const int step = p.nty * ROWS;
  const bool held = p.r1 - p.r0 <= step;
  Columns<VEC> c{};
  if (p.on) c.load_params(a, p.col);
  const float* x = a.x + (long long)(p.r0 + p.ty) * a.x_stride + p.col;
  const long long x_row = p.nty * a.x_stride, x_step = ROWS * x_row;
  Vec<VEC> v[ROWS];
  const auto read = [&](const float* from, int left) {  // rows that are not there are zero
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      v[i] = Vec<VEC>{};
      if (p.on && i * p.nty < left) v[i] = load_vec<VEC>(from + i * x_row);
    }
  };
  const int rows_left = p.r1 - p.r0 - p.ty;  // of this thread, from its first row on
  // the sums of this thread's rows; when they do not stay in registers also their
  // count, mean and squared deviations from it
  float count = 0.f;
  Vec<VEC> mean{}, dev{}, sum{};
  if (held) {
    read(x, rows_left);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) sum = sum + v[i];
  } else {
    const float* from = x;
    for (int left = rows_left; left > 0; left -= step, from += x_step) {
      read(from, left);
      float n = 0.f;
      Vec<VEC> s{}, d{};
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        n += i * p.nty < left ? 1.f : 0.f;
        s = s + v[i];
      }
      const Vec<VEC> m = s * all<VEC>(1.f / n), minus = m * all<VEC>(-1.f);
#pragma unroll
      for (int i = 0; i < ROWS; ++i)
        if (i * p.nty < left) {
          const Vec<VEC> q = v[i] + minus;
          d = fma(q, q, d);
        }
      const float both = count + n;  // join with the rows before
      const Vec<VEC> q = m + mean * all<VEC>(-1.f);
      mean = fma(q, all<VEC>(n / both), mean);
      dev = fma(q * q, all<VEC>(count * n / both), dev + d);
      count = both;
    }
    sum = mean * all<VEC>(count);
  }
  const float per_value = float(p.rows) * float(p.cpg);
  sum_rows<VEC>(sum, p, f.lanes, sh.red[0]);
  sum_groups(p, f, sh.red[0], sh.sum[0], sh.total[0], [&](int g, float s) {
    const float m = s / per_value;
    if (p.part == 0) a.mean[stat0 + g] = m;
    return -m;
  });
  int group[VEC];  // of this thread's columns
#pragma unroll
  for (int j = 0; j < VEC; ++j) group[j] = p.on ? group_of(f, p.lane * VEC + j) : 0;
#pragma unroll
  for (int j = 0; j < VEC; ++j) c.minus_mean.v[j] = sh.total[0][group[j]];
  if (held) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
      if (i * p.nty < rows_left && p.on) {
        v[i] = v[i] + c.minus_mean;
        dev = fma(v[i], v[i], dev);
      }
  } else if (p.on) {
    const Vec<VEC> q = mean + c.minus_mean;
    dev = fma(q * q, all<VEC>(count), dev);
  }
  sum_rows<VEC>(dev, p, f.lanes, sh.red[1]);
  sum_groups(p, f, sh.red[1], sh.sum[1], sh.total[1], [&](int g, float s) {
    const float r = 1.f / sqrtf(s / per_value + a.eps);
    if (p.part == 0) a.rstd[stat0 + g] = r;
    return r;
  });
  if (p.on) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) c.rstd.v[j] = sh.total[1][group[j]];
    const Vec<VEC> w = c.gamma * c.rstd;
    float* y = a.y + (long long)(p.r0 + p.ty) * a.y_stride + p.col;
    const long long y_row = p.nty * a.y_stride, y_step = ROWS * y_row;
    for (int left = rows_left; left > 0; left -= step, x += x_step, y += y_step) {
      if (!held) {
        read(x, left);
#pragma unroll
        for (int i = 0; i < ROWS; ++i) v[i] = v[i] + c.minus_mean;
      }
#pragma unroll
      for (int i = 0; i < ROWS; ++i)
        if (i * p.nty < left) store_vec<VEC>(y + i * y_row, activate<SILU>(fma(w, v[i], c.beta)));
    }
  }
  if (f.blocks > 1) {
    __syncwarp();
    tc::cluster_sync();  // no block leaves while another may still read its sums
  }
}

// slots [sample * blocks + part][channel]: (sum gz, sum gz h) of the block's rows
template <int VEC, bool SILU, int ROWS>
__global__ void __launch_bounds__(kFusedMost) norm_bwd_fused_kernel(NormArgs a, Slabs f, float2* __restrict__ slots) {
  grid_dependents_launch();
  __shared__ __align__(16) FusedShared sh;
  const Place p = place_of<VEC>(a, f);
  float2* slot = slots + (((long long)p.sample << f.shift) + p.part) * a.channels + p.c0;
  if (p.rows == 0) {
    for (int k = threadIdx.x; k < p.columns; k += blockDim.x) slot[k] = make_float2(0.f, 0.f);
    return;  // every block of the cluster
  }
  const int step = p.nty * ROWS;
  const bool held = p.r1 - p.r0 <= step;
  Columns<VEC> c{};
  int group[VEC];  // of this thread's columns
#pragma unroll
  for (int j = 0; j < VEC; ++j) group[j] = p.on ? group_of(f, p.lane * VEC + j) : 0;
  if (p.on) {
    c.load_params(a, p.col);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const long long k = (long long)p.sample * a.groups + p.g0 + group[j];
      c.minus_mean.v[j] = -a.mean[k];
      c.rstd.v[j] = a.rstd[k];
    }
  }
  const float* x = a.x + (long long)(p.r0 + p.ty) * a.x_stride + p.col;
  const float* gy = a.grad_y + (long long)(p.r0 + p.ty) * a.gy_stride + p.col;
  const long long x_row = p.nty * a.x_stride, gy_row = p.nty * a.gy_stride;
  Vec<VEC> h[ROWS], gz[ROWS];
  const auto read = [&](const float* fx, const float* fg, int left) {  // rows that are not there are zero
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      h[i] = Vec<VEC>{};
      gz[i] = Vec<VEC>{};
      if (p.on && i * p.nty < left) {
        h[i] = load_vec<VEC>(fx + i * x_row);
        gz[i] = load_vec<VEC>(fg + i * gy_row);
      }
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      if (i * p.nty < left) {
        h[i] = c.normalised(h[i]);
        gz[i] = activate_grad<SILU>(fma(c.gamma, h[i], c.beta), gz[i]);
      }
    }
  };
  const int rows_left = p.r1 - p.r0 - p.ty;  // of this thread, from its first row on
  Vec<VEC> s1{}, s2{};
  {
    const float *fx = x, *fg = gy;
    for (int left = rows_left; left > 0; left -= step, fx += ROWS * x_row, fg += ROWS * gy_row) {
      read(fx, fg, left);
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        s1 = s1 + gz[i];
        s2 = fma(gz[i], h[i], s2);
      }
    }
  }
  sum_rows<VEC>(s1, p, f.lanes, sh.red[0]);
  sum_rows<VEC>(s2, p, f.lanes, sh.red[1]);
  __syncthreads();
  for (int k = threadIdx.x; k < p.columns; k += blockDim.x) {
    float u = 0.f, q = 0.f;
#pragma unroll 4
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
      u += sh.red[0][w][k];
      q += sh.red[1][w][k];
    }
    slot[k] = make_float2(u, q);
    const float w = a.gamma == nullptr ? 1.f : a.gamma[p.c0 + k];
    sh.col[0][k] = w * u;
    sh.col[1][k] = w * q;
  }
  if (a.grad_x == nullptr) return;  // every block
  __syncthreads();
  const float per_value = -1.f / (float(p.rows) * float(p.cpg));
#pragma unroll
  for (int q = 0; q < 2; ++q)
    team_sums(p, f.team, p.cpg, [&](int g, int e) { return sh.col[q][g * p.cpg + e]; },
              [&](int g, float s) { (f.blocks > 1 ? sh.sum : sh.total)[q][g] = s * per_value; });
  if (f.blocks > 1) {
    __syncwarp();
    tc::cluster_sync();
    for (int g = threadIdx.x; g < 2 * p.groups; g += blockDim.x) {
      const int q = g >= p.groups, i = g - q * p.groups;
      float s = 0.f;
      for (int k = 0; k < f.blocks; ++k) s += tc::peer_load(tc::peer_addr(tc::smem_addr(&sh.sum[q][i]), k));
      sh.total[q][i] = s;
    }
  }
  __syncthreads();
  if (p.on) {
    Vec<VEC> m1, m2;  // less the means of t and t h
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      m1.v[j] = sh.total[0][group[j]];
      m2.v[j] = sh.total[1][group[j]];
    }
    float* gx = a.grad_x + (long long)(p.r0 + p.ty) * a.gx_stride + p.col;
    const long long gx_row = p.nty * a.gx_stride;
    for (int left = rows_left; left > 0; left -= step, x += ROWS * x_row, gy += ROWS * gy_row, gx += ROWS * gx_row) {
      if (!held) read(x, gy, left);
#pragma unroll
      for (int i = 0; i < ROWS; ++i)
        if (i * p.nty < left)
          store_vec<VEC>(gx + i * gx_row, c.rstd * fma(h[i], m2, fma(c.gamma, gz[i], m1)));
    }
  }
  if (f.blocks > 1) {
    __syncwarp();
    tc::cluster_sync();  // no block leaves while another may still read its sums
  }
}

// ------------------------------------------------------------------- tiles
// The sample that row r belongs to: the last one that starts at or before r
// (-1: none).  Whole warps call: 32 offsets at a time, so that 1 000 samples
// take two loads in a row instead of ten.
__device__ __forceinline__ int sample_of(const NormArgs& a, int r) {
  if (a.ptr == nullptr) return 0;
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = a.samples;  // the first sample with ptr > r is in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step + step - 1;
    const unsigned below = __ballot_sync(0xffffffffu, at < hi && a.ptr[at] <= r);
    lo += __popc(below) * step;
    hi = step == 1 ? lo : min(hi, lo + step - 1);
  }
  return min(lo, a.samples) - 1;
}

// Calls f(sample, first row, last row + 1) for each part of the tile's rows
// [r0, r1) that belongs to a sample.  The same for every thread of the block.
template <class F>
__device__ __forceinline__ void for_parts(const NormArgs& a, int r0, int r1, F&& f) {
  for (int r = r0; r < r1;) {
    const int s = sample_of(a, r);
    if (s < 0) {
      r = max(r + 1, min(r1, a.ptr[0]));
      continue;
    }
    const int2 b = sample_rows(a, s);
    const int hi = min(b.y, r1);
    if (hi <= r) {  // behind the last sample (or between samples of disordered offsets)
      if (s == a.samples - 1) return;
      ++r;
      continue;
    }
    f(s, r, hi);
    r = hi;
  }
}

// The same from the last row down.
template <class F>
__device__ __forceinline__ void for_parts_down(const NormArgs& a, int r0, int r1, F&& f) {
  for (int r = r1 - 1; r >= r0;) {
    const int s = sample_of(a, r);
    if (s < 0) return;
    const int2 b = sample_rows(a, s);
    if (b.y <= r) {  // behind the last sample (or between samples of disordered offsets)
      r = b.y - 1;
      continue;
    }
    const int lo = min(max(b.x, r0), r);  // each step goes down, disordered offsets too
    f(s, lo, r + 1);
    r = lo - 1;
  }
}

// Sums v over the block's row groups (threads with the same lane), in a fixed
// order; the result is valid in every thread of row group 0.
template <int K>
__device__ __forceinline__ void sum_row_groups(float (&v)[K], float* red, int ty, int nty) {
  float* mine = red + threadIdx.x;
#pragma unroll
  for (int j = 0; j < K; ++j) mine[j * kNormThreads] = v[j];
  const int lpr = kNormThreads / nty;
  for (int o = nty >> 1; o > 0; o >>= 1) {
    __syncthreads();
    if (ty < o)
#pragma unroll
      for (int j = 0; j < K; ++j) mine[j * kNormThreads] += mine[j * kNormThreads + o * lpr];
  }
#pragma unroll
  for (int j = 0; j < K; ++j) v[j] = mine[j * kNormThreads];
}

struct Tile {
  int lane, ty, nty, r0, r1, col, index;
  bool on;  // the thread has columns
};
// Tile `index` of `per` times the rows that the block's registers hold.
template <int VEC>
__device__ __forceinline__ Tile make_tile(const NormArgs& a, int lpr, int per, int index) {
  Tile t;
  t.index = index;
  t.lane = threadIdx.x & (lpr - 1);
  t.ty = threadIdx.x / lpr;
  t.nty = kNormThreads / lpr;
  const int rows = t.nty * kNormRows * per;
  t.r0 = index * rows;
  t.r1 = min(a.n - t.r0, rows) + t.r0;
  t.col = (blockIdx.y * lpr + t.lane) * VEC;
  t.on = t.col < a.channels;
  return t;
}

// 1, forward: slot [channel] = (mean, sum of squared deviations) of the part.
template <int VEC>
__global__ void __launch_bounds__(kNormThreads) norm_part_kernel(NormArgs a, int lpr, int per, float2* __restrict__ slots) {
  grid_dependents_launch();
  __shared__ float red[VEC * kNormThreads];
  __shared__ float mean_of[VEC * 32];
  const Tile t = make_tile<VEC>(a, lpr, per, blockIdx.x);
  for_parts(a, t.r0, t.r1, [&](int s, int lo, int hi) {
    // this thread's rows: count, mean, squared deviations from it
    float count = 0.f;
    Vec<VEC> mean{}, dev{};
    const int step = t.nty * kNormRows;
    const auto read = [&](Vec<VEC>(&v)[kNormRows], int base) {
#pragma unroll
      for (int i = 0; i < kNormRows; ++i) {
        const int r = base + i * t.nty;
        v[i] = Vec<VEC>{};
        if (t.on && r < hi) v[i] = load_vec<VEC>(a.x + r * a.x_stride + t.col);
      }
    };
    const auto add = [&](const Vec<VEC>(&v)[kNormRows], int base) {
      float n = 0.f;
      Vec<VEC> sum{}, d{};
#pragma unroll
      for (int i = 0; i < kNormRows; ++i) {
        n += base + i * t.nty < hi ? 1.f : 0.f;
        sum = sum + v[i];
      }
      if (n == 0.f) return;
      const Vec<VEC> m = sum * all<VEC>(1.f / n), minus = m * all<VEC>(-1.f);
#pragma unroll
      for (int i = 0; i < kNormRows; ++i)
        if (base + i * t.nty < hi) {
          const Vec<VEC> q = v[i] + minus;
          d = fma(q, q, d);
        }
      // join with the rows before
      const float both = count + n, part = n / both;
      const Vec<VEC> q = m + mean * all<VEC>(-1.f);
      mean = fma(q, all<VEC>(part), mean);
      dev = fma(q * q, all<VEC>(count * part), dev + d);
      count = both;
    };
    Vec<VEC> u[kNormRows], v[kNormRows];  // one is read while the other is used
    read(u, lo + t.ty);
    for (int base = lo + t.ty; base < hi; base += 2 * step) {
      read(v, base + step);
      add(u, base);
      read(u, base + 2 * step);
      add(v, base + step);
    }
    Vec<VEC> sum = mean * all<VEC>(count);
    __syncthreads();
    sum_row_groups<VEC>(sum.v, red, t.ty, t.nty);
    if (t.ty == 0)
#pragma unroll
      for (int j = 0; j < VEC; ++j) mean_of[t.lane * VEC + j] = sum.v[j] / float(hi - lo);
    __syncthreads();
    Vec<VEC> whole;
#pragma unroll
    for (int j = 0; j < VEC; ++j) whole.v[j] = mean_of[t.lane * VEC + j];
    const Vec<VEC> q = mean + whole * all<VEC>(-1.f);
    dev = fma(q * q, all<VEC>(count), dev);
    __syncthreads();
    sum_row_groups<VEC>(dev.v, red, t.ty, t.nty);
    if (t.ty == 0 && t.on)
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        slots[((long long)t.index + s) * a.channels + t.col + j] = make_float2(whole.v[j], dev.v[j]);
  });
}

// Sums over the TPI threads of one item, in a fixed order, valid in all of them.
template <int TPI, int K>
__device__ __forceinline__ void item_sums(float (&v)[K], float (*red)[32]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if constexpr (TPI > 32) {
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int i = 0; i < K; ++i) red[i][threadIdx.x >> 5] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < K; ++i) {
      v[i] = 0.f;
#pragma unroll
      for (int q = 0; q < TPI / 32; ++q) v[i] += red[i][q];
    }
  }
}

// 2: TPI threads per (sample, group) join the slots.  Forward: the mean of all
// values, then, from the slots once more (they come from L2), the squared deviations from it:
// each part's own plus its mean's.  A part may be one row that is like no other, so no part's
// mean can stand for the whole one: squares about it would cancel.  What the mean's own
// rounding leaves of the first moment is taken off the variance and the mean.
// Backward: the group's means of t and t h.
constexpr int kJoinThreads = 1024;
template <int TPI, bool BWD>
__global__ void __launch_bounds__(TPI > 32 ? TPI : kNormThreads)
    norm_join_kernel(NormArgs a, int rows_per_tile, const float2* __restrict__ slots, float2* __restrict__ terms) {
  grid_dependents_launch();
  grid_dependency_wait();
  __shared__ float red[3][32];  // of the mean, and of the two sums
  const long long item = ((long long)blockIdx.x * blockDim.x + threadIdx.x) / TPI;
  if (item >= (long long)a.samples * a.groups) return;  // whole items leave together
  const int s = (int)(item / a.groups), g = (int)(item % a.groups), cpg = a.channels / a.groups;
  const int2 b = sample_rows(a, s);
  const int t0 = b.x / rows_per_tile, t1 = b.y > b.x ? (b.y - 1) / rows_per_tile : t0 - 1;
  const long long entries = (long long)(t1 - t0 + 1) * cpg;
  const float count = float(b.y - b.x) * float(cpg);
  const float2* base = slots + ((long long)t0 + s) * a.channels + (long long)g * cpg;
  const int tid = threadIdx.x % TPI;
  auto rows_of = [&](int t) { return min(b.y, (t + 1) * rows_per_tile) - max(b.x, t * rows_per_tile); };
  // Every TPI-th entry, parts in order.  The forward, which takes them twice, keeps the first ones: f(rows, slot).
  constexpr int kHeld = BWD ? 0 : 4;
  int k = tid / cpg, c = tid % cpg;
  const auto next = [&]() {
    k += TPI / cpg;
    c += TPI % cpg;
    if (c >= cpg) {
      c -= cpg;
      ++k;
    }
  };
  float2 held[kHeld + 1];
  float rows[kHeld + 1];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const bool there = tid + (long long)i * TPI < entries;
    held[i] = there ? base[(long long)k * a.channels + c] : make_float2(0.f, 0.f);
    rows[i] = there ? float(rows_of(t0 + k)) : 0.f;
    next();
  }
  const int k0 = k, c0 = c;
  const auto for_slots = [&](auto&& f) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) f(rows[i], held[i]);
    k = k0;
    c = c0;
#pragma unroll 8
    for (long long q = tid + kHeld * TPI; q < entries; q += TPI) {
      f(float(rows_of(t0 + k)), base[(long long)k * a.channels + c]);
      next();
    }
  };
  float mean = 0.f, sum[2] = {};
  if constexpr (!BWD) {
    float all[1] = {};
    for_slots([&](float n, float2 v) { all[0] = fmaf(n, v.x, all[0]); });
    item_sums<TPI>(all, red + 2);
    mean = entries > 0 ? all[0] / count : 0.f;
  }
  for_slots([&](float n, float2 v) {
    if constexpr (BWD) {
      const float w = a.gamma == nullptr ? 1.f : a.gamma[g * cpg + c];
      sum[0] = fmaf(w, v.x, sum[0]);
      sum[1] = fmaf(w, v.y, sum[1]);
    } else {
      const float d = v.x - mean;
      sum[0] = fmaf(n, d, sum[0]);
      sum[1] += fmaf(n * d, d, v.y);
    }
  });
  item_sums<TPI>(sum, red);
  if (tid != 0) return;
  const float m1 = entries > 0 ? sum[0] / count : 0.f, m2 = entries > 0 ? sum[1] / count : 0.f;
  if constexpr (BWD) {
    terms[item] = make_float2(m1, m2);
  } else {
    const float var = fmaf(-m1, m1, m2);
    a.mean[item] = mean + m1;
    a.rstd[item] = 1.f / sqrtf((var < 0.f ? 0.f : var) + a.eps);  // NaN stays
  }
}

// 3, forward.  The tiles from the last to the first: what step 1 read last is
// still in L2.  The rows, which no launch of this call writes, are read before
// the wait for step 2.
template <int VEC, bool SILU>
__global__ void __launch_bounds__(kNormThreads) norm_apply_kernel(NormArgs a, int lpr) {
  const Tile t = make_tile<VEC>(a, lpr, 1, gridDim.x - 1 - blockIdx.x);
  Vec<VEC> v[kNormRows];
#pragma unroll
  for (int i = 0; i < kNormRows; ++i) {
    const int r = t.r0 + t.ty + i * t.nty;
    if (t.on && r < t.r1) v[i] = load_vec<VEC>(a.x + r * a.x_stride + t.col);
  }
  Columns<VEC> c;
  if (t.on) c.load_params(a, t.col);
  grid_dependency_wait();
  for_parts(a, t.r0, t.r1, [&](int s, int lo, int hi) {
    if (!t.on) return;
    c.load_stats(a, t.col, s);
#pragma unroll
    for (int i = 0; i < kNormRows; ++i) {
      const int r = t.r0 + t.ty + i * t.nty;
      if (r >= lo && r < hi)
        store_vec<VEC>(a.y + r * a.y_stride + t.col, activate<SILU>(fma(c.gamma, c.normalised(v[i]), c.beta)));
    }
  });
}

// A thread's rows of x and grad_y, every `step` rows from the first, on their way through
// a ring of its own in shared memory: kRing rows are in flight while one is used, 192
// KB an SM, without registers.  (A load takes some 2 to 3 us when the memory is busy, so 6.5
// TB/s want 100 KB in flight an SM all the time.  The backward of 131 101 x 256 in 61 samples takes
// 121 us so, 135 us with 8 rows in registers that are read in one go and then used, 150 us with two
// halves of them in turn.)
constexpr int kRing = 8;
constexpr int kRingBlocks = 3;  // blocks an SM
template <int VEC>
constexpr int ring_bytes() {
  return kRing * 2 * kNormThreads * VEC * (int)sizeof(float);
}
template <int VEC>
struct RowRing {
  const float *x, *g;
  long long x_step, g_step;
  int left;   // rows not yet under way
  int place;  // of the next row
  float* mine;
  __device__ __forceinline__ RowRing(const NormArgs& a, float* ring, int row, int step, int rows, int col)
      : x(a.x + row * a.x_stride + col),
        g(a.grad_y + row * a.gy_stride + col),
        x_step(step * a.x_stride),
        g_step(step * a.gy_stride),
        left(rows),
        place(0),
        mine(ring + threadIdx.x * VEC) {
    for (int i = 0; i < kRing; ++i) next();
  }
  // The next row into the place of the one that was used.
  __device__ __forceinline__ void next() {
    if (left > 0) {
      float* to = mine + place * (2 * kNormThreads * VEC);
      copy(to, x);
      copy(to + kNormThreads * VEC, g);
      x += x_step;
      g += g_step;
      --left;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    place = (place + 1) % kRing;
  }
  __device__ __forceinline__ void read(Vec<VEC>& vx, Vec<VEC>& vg) const {
    asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
    vx = load_vec<VEC>(mine + place * (2 * kNormThreads * VEC));
    vg = load_vec<VEC>(mine + place * (2 * kNormThreads * VEC) + kNormThreads * VEC);
  }
  static __device__ __forceinline__ void copy(float* to, const float* from) {
    if constexpr (VEC == 4)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_addr(to)), "l"(from) : "memory");
    else
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(tc::smem_addr(to)), "l"(from) : "memory");
  }
  static __device__ __forceinline__ void finish() { asm volatile("cp.async.wait_all;" ::: "memory"); }
};
// Rows of a tile that belong to the thread's row group.
__device__ __forceinline__ int rows_of_group(const Tile& t) {
  return t.on && t.r1 - t.r0 > t.ty ? (t.r1 - t.r0 - t.ty + t.nty - 1) / t.nty : 0;
}

// 1, backward: slot [channel] = (sum gz, sum gz h) of the part.
template <int VEC, bool SILU>
__global__ void __launch_bounds__(kNormThreads, kRingBlocks)
    norm_bwd_part_kernel(NormArgs a, int lpr, int per, float2* __restrict__ slots) {
  grid_dependents_launch();
  extern __shared__ __align__(16) float norm_ring[];
  __shared__ float red[2 * VEC * kNormThreads];
  const Tile t = make_tile<VEC>(a, lpr, per, blockIdx.x);
  int row = t.r0 + t.ty;
  RowRing<VEC> ring(a, norm_ring, row, t.nty, rows_of_group(t), t.col);
  Columns<VEC> c{};
  if (t.on) c.load_params(a, t.col);
  for_parts(a, t.r0, t.r1, [&](int s, int lo, int hi) {
    Vec<VEC> s1{}, s2{};
    if (t.on) {
      c.load_stats(a, t.col, s);
      for (; row < hi; row += t.nty) {
        Vec<VEC> x, g;
        ring.read(x, g);
        if (row >= lo) {
          const Vec<VEC> h = c.normalised(x), gz = activate_grad<SILU>(fma(c.gamma, h, c.beta), g);
          s1 = s1 + gz;
          s2 = fma(gz, h, s2);
        }
        ring.next();
      }
    }
    float sum[2 * VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      sum[j] = s1.v[j];
      sum[VEC + j] = s2.v[j];
    }
    __syncthreads();
    sum_row_groups<2 * VEC>(sum, red, t.ty, t.nty);
    if (t.ty == 0 && t.on)
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        slots[((long long)t.index + s) * a.channels + t.col + j] = make_float2(sum[j], sum[VEC + j]);
  });
  ring.finish();
}

// 3, backward: the tiles of step 1, their rows from the last to the first (what
// step 1 read last is still in L2).  The rows, which no launch of this call
// writes before, are under way before the wait for step 2.
template <int VEC, bool SILU>
__global__ void __launch_bounds__(kNormThreads, kRingBlocks)
    norm_bwd_apply_kernel(NormArgs a, int lpr, int per, const float2* __restrict__ terms) {
  extern __shared__ __align__(16) float norm_ring[];
  const Tile t = make_tile<VEC>(a, lpr, per, blockIdx.x);
  int row = t.r1 - 1 - t.ty;
  RowRing<VEC> ring(a, norm_ring, row, -t.nty, rows_of_group(t), t.col);
  float* gx = a.grad_x + row * a.gx_stride + t.col;
  const long long gx_step = t.nty * a.gx_stride;
  Columns<VEC> c{};
  if (t.on) c.load_params(a, t.col);
  grid_dependents_launch();
  grid_dependency_wait();
  for_parts_down(a, t.r0, t.r1, [&](int s, int lo, int hi) {
    if (!t.on) return;
    c.load_stats(a, t.col, s);
    Vec<VEC> m1, m2;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float2 m = terms[(long long)s * a.groups + (t.col + j) / (a.channels / a.groups)];
      m1.v[j] = -m.x;
      m2.v[j] = -m.y;
    }
    for (; row >= lo; row -= t.nty, gx -= gx_step) {
      Vec<VEC> x, g;
      ring.read(x, g);
      if (row < hi) {
        const Vec<VEC> h = c.normalised(x), gz = activate_grad<SILU>(fma(c.gamma, h, c.beta), g);
        store_vec<VEC>(gx, c.rstd * fma(h, m2, fma(c.gamma, gz, m1)));
      }
      ring.next();
    }
  });
  ring.finish();
}

// -------------------------------------------------------------- parameters
// Sums of rows of slots per channel, 32 channels a block: rows
// [y per, (y + 1) per) into row y of `sums`, or into the gradients.
__global__ void __launch_bounds__(1024)
    norm_param_kernel(int rows, int per, int channels, const float2* __restrict__ slots, float2* __restrict__ sums,
                      float* __restrict__ grad_gamma, float* __restrict__ grad_beta) {
  grid_dependency_wait();
  __shared__ float2 red[32][33];
  const int lane = threadIdx.x & 31, ty = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  const long long r0 = (long long)blockIdx.y * per, r1 = min((long long)rows, r0 + per);
  float2 s = make_float2(0.f, 0.f);
  if (c < channels) {
#pragma unroll 8
    for (long long r = r0 + ty; r < r1; r += 32) s = __fadd2_rn(s, slots[r * channels + c]);
  }
  red[ty][lane] = s;
  __syncthreads();
  s = red[lane][ty];  // warp ty sums channel ty of the block over the 32 row groups
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
    s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
  }
  const int k = blockIdx.x * 32 + ty;
  if (lane == 0 && k < channels) {
    if (sums != nullptr) {
      sums[(long long)blockIdx.y * channels + k] = s;
    } else {
      if (grad_beta != nullptr) grad_beta[k] = s.x;
      if (grad_gamma != nullptr) grad_gamma[k] = s.y;
    }
  }
}
constexpr int kParamRows = 1024, kParamParts = 64;

// after_kernel: the launch before this one in the stream is a kernel of the same call.
cudaError_t sum_params(const NormArgs& a, long long rows, const float2* slots, float2* sums, bool after_kernel,
                       cudaStream_t stream) {
  if (a.grad_gamma == nullptr && a.grad_beta == nullptr) return cudaSuccess;
  const unsigned columns = (unsigned)((a.channels + 31) / 32);
  cudaError_t e = cudaSuccess;
  if (rows > kParamRows) {
    const int per = (int)((rows + kParamParts - 1) / kParamParts);
    e = launch_kernel(norm_param_kernel, dim3(columns, kParamParts), dim3(1024), 0, stream, after_kernel,
                      (int)rows, per, a.channels, slots, sums, (float*)nullptr, (float*)nullptr);
    if (e != cudaSuccess) return e;
    slots = sums;
    rows = kParamParts;
    after_kernel = true;
  }
  return launch_kernel(norm_param_kernel, dim3(columns), dim3(1024), 0, stream, after_kernel, (int)rows, (int)rows,
                       a.channels, slots, (float2*)nullptr, a.grad_gamma, a.grad_beta);
}

// ---------------------------------------------------------------- launching
int lanes_per_row(int width, int vec) {
  const int need = (width + vec - 1) / vec;
  int l = 1;
  while (l < 32 && l < need) l <<= 1;
  return l;
}
int rows_per_tile(int channels, int vec) { return kNormRows * (kNormThreads / lanes_per_row(channels, vec)); }
long long tiles_of(int n, int rows) { return ((long long)n + rows - 1) / rows; }
bool vec4_rows(const void* p, long long stride) { return stride % 4 == 0 && ((uintptr_t)p & 15u) == 0; }

// The fused split for these sizes, or count = 0 for the tiles.  Measured on
// fp32 rows with SiLU, forward / backward in microseconds:
//   256 samples x 30 rows x 128 channels: whole rows, 256 threads, 4 rows each 4.6 / 6.9 (tiles 20 / 26);
//   254 samples, 130 000 rows x 256: 128-byte slabs 59 / 105 (whole rows in clusters of 4 84 / 124, tiles 80 / 124);
//   4 000 samples, 130 000 rows x 256: whole rows 83 / 132 (256-byte slabs 113 / 159, tiles 270 / 241);
//   61 samples, 131 101 rows x 256: 64-byte slabs 98 / 164, the tiles 80 / 121;
//   1 sample of 130 000 rows x 256: a cluster of 8 per 128-byte slab 110 / 174, the tiles 71 / 116;
//   1 sample of 20 000 rows x 128: a cluster of 8 per 64-byte slab 13 / 20, the tiles 12 / 20 in three and six launches.
//   400 samples of up to 3 013 rows, 200 000 rows x 64: 64-byte slabs 38 / 72, the tiles 47 / 58;
//   100 samples of up to 2 441 rows, 60 000 rows x 256: 64-byte slabs 39 / 68, the tiles 44 / 57.
// Index arithmetic and reductions that every thread repeats are what small
// samples pay for: group numbers by a product, row addresses by steps and one
// thread per statistic took the forward from 6.6 to 4.6 and, at 4 000 samples,
// from 137 to 83.
// So slabs narrow, down to 64 bytes a row, while the usual sample does not fit
// the registers and there are not yet many blocks; then few blocks become a
// cluster of larger ones.  Long samples of a tensor that leaves L2 go to the
// tiles, which read whole rows, as do longest samples that would keep their
// blocks reading long after the others (in the backward, which reads twice as
// much, sooner).
constexpr long long kFewBlocks = 148, kManyBlocks = 8 * kFewBlocks;
template <int VEC>
Slabs fused_slabs(const NormArgs& a, int max_rows, bool backward) {
  Slabs f{};
  const int cpg = a.channels / a.groups;
  const int most = VEC == 4 ? kSlabColumns : 32;  // 32 lanes across
  if (a.n == 0 || a.samples == 0 || cpg > most) return f;
  // slabs start on a vector: their groups are a multiple of this
  int unit = 1;
  while (unit * cpg % VEC != 0) ++unit;
  if (unit * cpg > most) return f;
  const long long average = ((long long)a.n + a.samples - 1) / a.samples;
  // the longest sample: the caller's bound, else four times the average is expected
  long long longest = max_rows > 0 ? max_rows : a.samples == 1 ? a.n : 4 * average + 64;
  if (longest > a.n) longest = a.n;
  const long long usual = longest < 2 * average ? longest : 2 * average;
  if (average > 1024 && (long long)a.n * a.channels > (16 << 20)) return f;
  auto set = [&](int groups) {
    f.groups = groups < a.groups ? groups : a.groups;
    f.count = (a.groups + f.groups - 1) / f.groups;
    f.lanes = lanes_per_row(f.groups * cpg, VEC);
  };
  auto held = [&]() { return (long long)f.rows * (f.threads / f.lanes); };
  auto blocks = [&]() { return (long long)a.samples * f.count; };
  f.threads = 256;
  f.rows = 8;
  f.per_cpg = ((1u << 20) + cpg - 1) / cpg;
  set(most / (unit * cpg) * unit);
  while (f.groups > unit && f.groups * cpg > 16 && blocks() < kManyBlocks && (held() < usual || blocks() < kFewBlocks)) {
    const int half = (f.groups / unit + 1) / 2 * unit;
    if (half == f.groups) break;
    set(half);
  }
  f.blocks = 1;
  while (f.blocks < 8 && held() * f.blocks < longest && blocks() * f.blocks < kFewBlocks) f.blocks *= 2;
  if (blocks() * f.blocks <= kFewBlocks && held() * f.blocks < longest) f.threads = kFusedMost;
  if (f.blocks == 1) {
    if (blocks() >= kManyBlocks) f.threads = 128;  // small blocks overlap better
    if (held() / 2 >= usual) f.rows = 4;  // small samples
    while (f.threads > 128 && held() / 2 >= usual) f.threads /= 2;
  }
  while (1 << f.shift < f.blocks) ++f.shift;
  f.team = 32;
  while (f.team > 1 && f.team * f.groups > f.threads) f.team /= 2;
  if (backward && max_rows > 1024 && max_rows > 4 * average && max_rows > 4 * held() * f.blocks &&
      (long long)a.n * a.channels > (8 << 20))
    f.count = 0;
  if (held() * f.blocks * (blocks() < 4 * kFewBlocks ? 8 : 32) < longest || blocks() * f.blocks > 0x7fffffffLL) f.count = 0;
  return f;
}

template <class... P, class... A>
cudaError_t launch_cluster(void (*kernel)(P...), const NormArgs& a, const Slabs& f, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((long long)a.samples * f.count * f.blocks));
  cfg.blockDim = dim3(f.threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = f.blocks;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = f.blocks > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, a, f, args...);
}

// Rows of a tile of step 1, as a multiple of a block's registers: as many tiles as
// are resident at once, `resident` blocks an SM (131 101 x 256: forward 80 us, with twice as many
// tiles 84), which leaves few slots to join.
int part_rows(const NormArgs& a, int rows, unsigned columns, int resident) {
  const long long blocks = tiles_of(a.n, rows) * columns, most = resident * kFewBlocks, per = (blocks + most - 1) / most;
  return (int)(per < 1 ? 1 : per > 64 ? 64 : per);
}

template <bool BWD>
cudaError_t join(const NormArgs& a, int rows, const float2* slots, float2* terms, cudaStream_t stream) {
  const long long items = (long long)a.samples * a.groups;
  // a warp per item while a sample has few slots; a block for long samples
  // (launched dependent on step 1: each waits for it before its first read)
  const bool wide = ((double)a.n / a.samples / rows + 1) * (a.channels / a.groups) > 512;
  const long long blocks = wide ? items : (items * 32 + kNormThreads - 1) / kNormThreads;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  return wide ? launch_kernel(norm_join_kernel<kJoinThreads, BWD>, dim3((unsigned)blocks), dim3(kJoinThreads), 0, stream,
                              a.n > 0, a, rows, slots, terms)
              : launch_kernel(norm_join_kernel<32, BWD>, dim3((unsigned)blocks), dim3(kNormThreads), 0, stream,
                              a.n > 0, a, rows, slots, terms);
}

template <int VEC, bool SILU>
cudaError_t norm_fwd(const NormArgs& a, int max_rows, void* ws, cudaStream_t stream) {
  const Slabs f = fused_slabs<VEC>(a, max_rows, false);
  if (f.count > 0)
    return f.rows == 4 ? launch_cluster(norm_fused_kernel<VEC, SILU, 4>, a, f, stream)
                       : launch_cluster(norm_fused_kernel<VEC, SILU, 8>, a, f, stream);
  const int lpr = lanes_per_row(a.channels, VEC), rows = rows_per_tile(a.channels, VEC);
  const unsigned columns = (unsigned)((a.channels + lpr * VEC - 1) / (lpr * VEC));
  const int per = part_rows(a, rows, columns, 2);
  cudaError_t e = cudaSuccess;
  if (a.n > 0) {
    norm_part_kernel<VEC><<<dim3((unsigned)tiles_of(a.n, per * rows), columns), kNormThreads, 0, stream>>>(a, lpr, per,
                                                                                                          (float2*)ws);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) e = join<false>(a, per * rows, (float2*)ws, nullptr, stream);
  if (e == cudaSuccess && a.n > 0)
    e = launch_kernel(norm_apply_kernel<VEC, SILU>, dim3((unsigned)tiles_of(a.n, rows), columns), dim3(kNormThreads), 0,
                      stream, true, a, lpr);
  return e;
}

// Workspace: terms, partial sums of the parameters, slots.
size_t terms_bytes(const NormArgs& a) { return pad256(sizeof(float2) * (size_t)a.samples * a.groups); }
size_t sums_bytes(const NormArgs& a) { return pad256(sizeof(float2) * (size_t)kParamParts * a.channels); }

template <int VEC, bool SILU>
cudaError_t norm_bwd(const NormArgs& a, int max_rows, void* ws, cudaStream_t stream) {
  float2* terms = (float2*)ws;
  float2* sums = (float2*)((char*)ws + terms_bytes(a));
  float2* slots = (float2*)((char*)ws + terms_bytes(a) + sums_bytes(a));
  const Slabs f = fused_slabs<VEC>(a, max_rows, true);
  if (f.count > 0) {
    const cudaError_t e = f.rows == 4 ? launch_cluster(norm_bwd_fused_kernel<VEC, SILU, 4>, a, f, stream, slots)
                                      : launch_cluster(norm_bwd_fused_kernel<VEC, SILU, 8>, a, f, stream, slots);
    return e != cudaSuccess ? e : sum_params(a, (long long)a.samples * f.blocks, slots, sums, true, stream);
  }
  const int lpr = lanes_per_row(a.channels, VEC), rows = rows_per_tile(a.channels, VEC);
  const unsigned columns = (unsigned)((a.channels + lpr * VEC - 1) / (lpr * VEC));
  const int per = part_rows(a, rows, columns, kRingBlocks);
  constexpr int ring = ring_bytes<VEC>();
  const long long tiles = tiles_of(a.n, per * rows), n_slots = tiles + a.samples;
  cudaError_t e = cudaMemsetAsync(slots, 0, sizeof(float2) * (size_t)n_slots * a.channels, stream);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(norm_bwd_part_kernel<VEC, SILU>, cudaFuncAttributeMaxDynamicSharedMemorySize, ring);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(norm_bwd_apply_kernel<VEC, SILU>, cudaFuncAttributeMaxDynamicSharedMemorySize, ring);
  if (e == cudaSuccess && a.n > 0) {
    norm_bwd_part_kernel<VEC, SILU><<<dim3((unsigned)tiles, columns), kNormThreads, ring, stream>>>(a, lpr, per, slots);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess && a.grad_x != nullptr && a.samples > 0) {
    e = join<true>(a, per * rows, slots, terms, stream);
    if (e == cudaSuccess && a.n > 0)
      e = launch_kernel(norm_bwd_apply_kernel<VEC, SILU>, dim3((unsigned)tiles, columns), dim3(kNormThreads), ring,
                        stream, true, a, lpr, per, (const float2*)terms);
  }
  return e != cudaSuccess ? e : sum_params(a, n_slots, slots, sums, a.n > 0, stream);
}

}  // namespace

// Enough for rows of any alignment.
size_t norm_workspace(int n, int samples, int channels, int groups, int max_rows, bool backward) {
  NormArgs a{};
  a.n = n;
  a.samples = samples;
  a.channels = channels;
  a.groups = groups;
  const Slabs one = fused_slabs<1>(a, max_rows, backward);
  const Slabs four = channels % 4 == 0 ? fused_slabs<4>(a, max_rows, backward) : one;
  const bool fused = one.count > 0 && four.count > 0;
  if (fused && !backward) return 0;
  const int blocks = one.blocks > four.blocks ? one.blocks : four.blocks;
  size_t slots = (size_t)samples * (fused ? blocks : 1);
  if (!fused) {
    slots += (size_t)tiles_of(n, rows_per_tile(channels, 1));
    const size_t other = (size_t)samples * blocks;  // the alignment that is fused
    if (other > slots) slots = other;
  }
  return terms_bytes(a) + sums_bytes(a) + pad256(sizeof(float2) * slots * (size_t)channels);
}

cudaError_t launch_norm_fwd(const NormArgs& a, int max_rows, void* ws, cudaStream_t stream) {
  if (a.samples == 0) return cudaSuccess;
  const bool v4 = a.channels % 4 == 0 && vec4_rows(a.x, a.x_stride) && vec4_rows(a.y, a.y_stride);
  if (v4) return a.act ? norm_fwd<4, true>(a, max_rows, ws, stream) : norm_fwd<4, false>(a, max_rows, ws, stream);
  return a.act ? norm_fwd<1, true>(a, max_rows, ws, stream) : norm_fwd<1, false>(a, max_rows, ws, stream);
}

cudaError_t launch_norm_bwd(const NormArgs& a, int max_rows, void* ws, cudaStream_t stream) {
  const bool v4 = a.channels % 4 == 0 && vec4_rows(a.x, a.x_stride) && vec4_rows(a.grad_y, a.gy_stride) &&
                  (a.grad_x == nullptr || vec4_rows(a.grad_x, a.gx_stride));
  if (v4) return a.act ? norm_bwd<4, true>(a, max_rows, ws, stream) : norm_bwd<4, false>(a, max_rows, ws, stream);
  return a.act ? norm_bwd<1, true>(a, max_rows, ws, stream) : norm_bwd<1, false>(a, max_rows, ws, stream);
}

}  // namespace cgtp
