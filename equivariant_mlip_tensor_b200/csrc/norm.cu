// Group norm with an activation over channels-last rows, one normalisation
// per graph (sample) and channel group, forward and backward, for sm_100a.
//
//   over the rows of a sample x the channels of a group: mean, var (biased)
//   h = (x - mean) rstd, rstd = 1 / sqrt(var + eps);  z = gamma h + beta;  y = act(z)
//   gz = grad_y act'(z);  t = gamma gz
//   grad_x = rstd (t - <t> - h <t h>);  grad_gamma = sum gz h;  grad_beta = sum gz
//
// Bound by memory: the forward has to read x and write y, the backward to read
// x and grad_y and write grad_x.
//
// Samples may have any length (graph offsets on the device), so the rows are
// cut into tiles of equal length whatever the samples are.  The part of sample
// s in tile t has the slot t + s of its own: going down the rows, each step
// moves to the next tile or the next sample, so no two parts share a slot.
//   1. each tile reduces each of its parts per channel into the part's slot
//      (forward: mean and sum of squared deviations, two passes over values
//      held in registers; backward: sums of gz and gz h);
//   2. one group of threads per (sample, group) joins the slots in order;
//   3. each tile reads its rows again and writes the result.
#include <cuda_runtime.h>
#include <stdint.h>

#include "train_ops.h"

namespace cgtp {
namespace {

constexpr int kNormThreads = 256;
constexpr int kNormRows = 8;  // rows per thread, held in registers

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

// Bounds of sample s, clamped into [0, n].
__device__ __forceinline__ int2 sample_rows(const NormArgs& a, int s) {
  if (a.ptr == nullptr) return make_int2(0, a.n);
  const int lo = min(max(a.ptr[s], 0), a.n);
  return make_int2(lo, min(max(a.ptr[s + 1], lo), a.n));
}
// The sample that row r belongs to: the last one that starts at or before r
// (-1: none), found in log2(samples) steps.
__device__ __forceinline__ int sample_of(const NormArgs& a, int r) {
  if (a.ptr == nullptr) return 0;
  int lo = 0, hi = a.samples;  // first sample with ptr > r
  while (lo < hi) {
    const int mid = lo + (hi - lo) / 2;
    if (a.ptr[mid] <= r) lo = mid + 1;
    else hi = mid;
  }
  return lo - 1;
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

template <bool SILU>
__device__ __forceinline__ float act(float z) {
  return SILU ? z / (1.f + expf(-z)) : z;
}
template <bool SILU>
__device__ __forceinline__ float act_grad(float z) {
  if (!SILU) return 1.f;
  const float s = 1.f / (1.f + expf(-z));
  return s * (1.f + z * (1.f - s));
}

struct Tile {
  int lane, ty, nty, r0, r1, col;
  bool on;  // the thread has columns
};
template <int VEC>
__device__ __forceinline__ Tile make_tile(const NormArgs& a, int lpr) {
  Tile t;
  t.lane = threadIdx.x & (lpr - 1);
  t.ty = threadIdx.x / lpr;
  t.nty = kNormThreads / lpr;
  t.r0 = blockIdx.x * (t.nty * kNormRows);
  t.r1 = min(a.n - t.r0, t.nty * kNormRows) + t.r0;
  t.col = (blockIdx.y * lpr + t.lane) * VEC;
  t.on = t.col < a.channels;
  return t;
}

// 1, forward: slot [channel] = (mean, sum of squared deviations) of the part.
template <int VEC>
__global__ void __launch_bounds__(kNormThreads) norm_part_kernel(NormArgs a, int lpr, float2* __restrict__ slots) {
  __shared__ float red[VEC * kNormThreads];
  __shared__ float mean_of[VEC * 32];
  const Tile t = make_tile<VEC>(a, lpr);
  Vec<VEC> v[kNormRows];
#pragma unroll
  for (int i = 0; i < kNormRows; ++i) {
    const int r = t.r0 + t.ty + i * t.nty;
    v[i] = Vec<VEC>{};
    if (t.on && r < t.r1) v[i] = load_vec<VEC>(a.x + r * a.x_stride + t.col);
  }
  for_parts(a, t.r0, t.r1, [&](int s, int lo, int hi) {
    float sum[VEC] = {};
#pragma unroll
    for (int i = 0; i < kNormRows; ++i) {
      const int r = t.r0 + t.ty + i * t.nty;
      if (r >= lo && r < hi)
#pragma unroll
        for (int j = 0; j < VEC; ++j) sum[j] += v[i].v[j];
    }
    __syncthreads();
    sum_row_groups<VEC>(sum, red, t.ty, t.nty);
    if (t.ty == 0)
#pragma unroll
      for (int j = 0; j < VEC; ++j) mean_of[t.lane * VEC + j] = sum[j] / float(hi - lo);
    __syncthreads();
    float mean[VEC], dev[VEC] = {};
#pragma unroll
    for (int j = 0; j < VEC; ++j) mean[j] = mean_of[t.lane * VEC + j];
#pragma unroll
    for (int i = 0; i < kNormRows; ++i) {
      const int r = t.r0 + t.ty + i * t.nty;
      if (r >= lo && r < hi)
#pragma unroll
        for (int j = 0; j < VEC; ++j) dev[j] = fmaf(v[i].v[j] - mean[j], v[i].v[j] - mean[j], dev[j]);
    }
    __syncthreads();
    sum_row_groups<VEC>(dev, red, t.ty, t.nty);
    if (t.ty == 0 && t.on)
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        slots[((long long)blockIdx.x + s) * a.channels + t.col + j] = make_float2(mean[j], dev[j]);
  });
}

// Sum over the TPI threads of one item, in a fixed order, valid in all of them.
template <int TPI>
__device__ __forceinline__ float item_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (TPI > 32) {
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int q = 0; q < TPI / 32; ++q) v += red[q];
  }
  return v;
}

// 2: TPI threads per (sample, group) join the slots.  Forward: the mean of all
// values, then the squared deviations from it (each part's own plus its
// mean's); backward: the group's means of t and t h.
template <int TPI, bool BWD>
__global__ void __launch_bounds__(kNormThreads)
    norm_join_kernel(NormArgs a, int rows_per_tile, const float2* __restrict__ slots, float2* __restrict__ terms) {
  __shared__ float red[kNormThreads / 32];
  const long long item = ((long long)blockIdx.x * kNormThreads + threadIdx.x) / TPI;
  if (item >= (long long)a.samples * a.groups) return;  // whole items leave together
  const int s = (int)(item / a.groups), g = (int)(item % a.groups), cpg = a.channels / a.groups;
  const int2 b = sample_rows(a, s);
  const int t0 = b.x / rows_per_tile, t1 = b.y > b.x ? (b.y - 1) / rows_per_tile : t0 - 1;
  const long long entries = (long long)(t1 - t0 + 1) * cpg;
  const float count = float(b.y - b.x) * float(cpg);
  const float2* base = slots + ((long long)t0 + s) * a.channels + (long long)g * cpg;
  const int tid = threadIdx.x % TPI;
  auto rows_of = [&](int t) { return min(b.y, (t + 1) * rows_per_tile) - max(b.x, t * rows_per_tile); };
  float s1 = 0.f, s2 = 0.f;
  for (long long q = tid; q < entries; q += TPI) {
    const int k = (int)(q / cpg), c = (int)(q % cpg);
    const float2 v = base[(long long)k * a.channels + c];
    if (BWD) {
      const float w = a.gamma == nullptr ? 1.f : a.gamma[g * cpg + c];
      s1 = fmaf(w, v.x, s1);
      s2 = fmaf(w, v.y, s2);
    } else {
      s1 = fmaf(float(rows_of(t0 + k)), v.x, s1);
    }
  }
  s1 = item_sum<TPI>(s1, red);
  const float mean = entries > 0 ? s1 / count : 0.f;
  if constexpr (BWD) {
    s2 = item_sum<TPI>(s2, red);
    if (tid == 0) terms[item] = make_float2(mean, entries > 0 ? s2 / count : 0.f);
  } else {
    for (long long q = tid; q < entries; q += TPI) {
      const int k = (int)(q / cpg), c = (int)(q % cpg);
      const float2 v = base[(long long)k * a.channels + c];
      const float d = v.x - mean;
      s2 += fmaf(float(rows_of(t0 + k)) * d, d, v.y);
    }
    s2 = item_sum<TPI>(s2, red);
    if (tid == 0) {
      a.mean[item] = mean;
      a.rstd[item] = 1.f / sqrtf((entries > 0 ? s2 / count : 0.f) + a.eps);
    }
  }
}

// The scale, shift, mean and rstd of a thread's columns in sample s.
template <int VEC>
struct Columns {
  float gamma[VEC], beta[VEC], mean[VEC], rstd[VEC];
  __device__ __forceinline__ void load(const NormArgs& a, int col, int s) {
    const int cpg = a.channels / a.groups;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const long long k = (long long)s * a.groups + (col + j) / cpg;
      gamma[j] = a.gamma == nullptr ? 1.f : a.gamma[col + j];
      beta[j] = a.beta == nullptr ? 0.f : a.beta[col + j];
      mean[j] = a.mean[k];
      rstd[j] = a.rstd[k];
    }
  }
};

// 3, forward
template <int VEC, bool SILU>
__global__ void __launch_bounds__(kNormThreads) norm_apply_kernel(NormArgs a, int lpr) {
  const Tile t = make_tile<VEC>(a, lpr);
  if (!t.on) return;
  Vec<VEC> v[kNormRows];
#pragma unroll
  for (int i = 0; i < kNormRows; ++i) {
    const int r = t.r0 + t.ty + i * t.nty;
    if (r < t.r1) v[i] = load_vec<VEC>(a.x + r * a.x_stride + t.col);
  }
  for_parts(a, t.r0, t.r1, [&](int s, int lo, int hi) {
    Columns<VEC> c;
    c.load(a, t.col, s);
#pragma unroll
    for (int i = 0; i < kNormRows; ++i) {
      const int r = t.r0 + t.ty + i * t.nty;
      if (r >= lo && r < hi) {
        Vec<VEC> o;
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          o.v[j] = act<SILU>(fmaf(c.gamma[j], (v[i].v[j] - c.mean[j]) * c.rstd[j], c.beta[j]));
        store_vec<VEC>(a.y + r * a.y_stride + t.col, o);
      }
    }
  });
}

// 1, backward: slot [channel] = (sum gz, sum gz h) of the part.
template <int VEC, bool SILU>
__global__ void __launch_bounds__(kNormThreads) norm_bwd_part_kernel(NormArgs a, int lpr, float2* __restrict__ slots) {
  __shared__ float red[2 * VEC * kNormThreads];
  const Tile t = make_tile<VEC>(a, lpr);
  Vec<VEC> v[kNormRows], g[kNormRows];
#pragma unroll
  for (int i = 0; i < kNormRows; ++i) {
    const int r = t.r0 + t.ty + i * t.nty;
    v[i] = Vec<VEC>{};
    g[i] = Vec<VEC>{};
    if (t.on && r < t.r1) {
      v[i] = load_vec<VEC>(a.x + r * a.x_stride + t.col);
      g[i] = load_vec<VEC>(a.grad_y + r * a.gy_stride + t.col);
    }
  }
  for_parts(a, t.r0, t.r1, [&](int s, int lo, int hi) {
    float sum[2 * VEC] = {};
    if (t.on) {
      Columns<VEC> c;
      c.load(a, t.col, s);
#pragma unroll
      for (int i = 0; i < kNormRows; ++i) {
        const int r = t.r0 + t.ty + i * t.nty;
        if (r >= lo && r < hi)
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const float h = (v[i].v[j] - c.mean[j]) * c.rstd[j];
            const float gz = g[i].v[j] * act_grad<SILU>(fmaf(c.gamma[j], h, c.beta[j]));
            sum[j] += gz;
            sum[VEC + j] = fmaf(gz, h, sum[VEC + j]);
          }
      }
    }
    __syncthreads();
    sum_row_groups<2 * VEC>(sum, red, t.ty, t.nty);
    if (t.ty == 0 && t.on)
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        slots[((long long)blockIdx.x + s) * a.channels + t.col + j] = make_float2(sum[j], sum[VEC + j]);
  });
}

// grad_gamma and grad_beta: the sum of every slot (unused ones are zero), 32
// channels a block.
__global__ void __launch_bounds__(1024) norm_param_kernel(int rows, int channels, const float2* __restrict__ slots,
                                                          float* __restrict__ grad_gamma, float* __restrict__ grad_beta) {
  __shared__ float2 red[32][33];
  const int lane = threadIdx.x & 31, ty = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float2 s = make_float2(0.f, 0.f);
  if (c < channels) {
#pragma unroll 4
    for (int r = ty; r < rows; r += 32) {
      const float2 v = slots[(long long)r * channels + c];
      s.x += v.x;
      s.y += v.y;
    }
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
    if (grad_beta != nullptr) grad_beta[k] = s.x;
    if (grad_gamma != nullptr) grad_gamma[k] = s.y;
  }
}

// 3, backward
template <int VEC, bool SILU>
__global__ void __launch_bounds__(kNormThreads)
    norm_bwd_apply_kernel(NormArgs a, int lpr, const float2* __restrict__ terms) {
  const Tile t = make_tile<VEC>(a, lpr);
  if (!t.on) return;
  Vec<VEC> v[kNormRows], g[kNormRows];
#pragma unroll
  for (int i = 0; i < kNormRows; ++i) {
    const int r = t.r0 + t.ty + i * t.nty;
    if (r < t.r1) {
      v[i] = load_vec<VEC>(a.x + r * a.x_stride + t.col);
      g[i] = load_vec<VEC>(a.grad_y + r * a.gy_stride + t.col);
    }
  }
  for_parts(a, t.r0, t.r1, [&](int s, int lo, int hi) {
    Columns<VEC> c;
    c.load(a, t.col, s);
    float2 m[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      m[j] = terms[(long long)s * a.groups + (t.col + j) / (a.channels / a.groups)];
#pragma unroll
    for (int i = 0; i < kNormRows; ++i) {
      const int r = t.r0 + t.ty + i * t.nty;
      if (r >= lo && r < hi) {
        Vec<VEC> o;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float h = (v[i].v[j] - c.mean[j]) * c.rstd[j];
          const float gz = g[i].v[j] * act_grad<SILU>(fmaf(c.gamma[j], h, c.beta[j]));
          o.v[j] = c.rstd[j] * (fmaf(c.gamma[j], gz, -m[j].x) - h * m[j].y);
        }
        store_vec<VEC>(a.grad_x + r * a.gx_stride + t.col, o);
      }
    }
  });
}

int lanes_per_row(int width, int vec) {
  const int need = (width + vec - 1) / vec;
  int l = 1;
  while (l < 32 && l < need) l <<= 1;
  return l;
}
int rows_per_tile(int channels, int vec) { return kNormRows * (kNormThreads / lanes_per_row(channels, vec)); }
long long tiles_of(int n, int rows) { return ((long long)n + rows - 1) / rows; }
bool vec4_rows(const void* p, long long stride) { return stride % 4 == 0 && ((uintptr_t)p & 15u) == 0; }

template <bool BWD>
cudaError_t join(const NormArgs& a, int rows, const float2* slots, float2* terms, cudaStream_t stream) {
  const long long items = (long long)a.samples * a.groups;
  // a warp per item while a sample has few slots; a block for long samples
  const bool wide = ((double)a.n / a.samples / rows + 1) * (a.channels / a.groups) > 512;
  const long long blocks = wide ? items : (items * 32 + kNormThreads - 1) / kNormThreads;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (wide) norm_join_kernel<kNormThreads, BWD><<<(unsigned)blocks, kNormThreads, 0, stream>>>(a, rows, slots, terms);
  else norm_join_kernel<32, BWD><<<(unsigned)blocks, kNormThreads, 0, stream>>>(a, rows, slots, terms);
  return cudaGetLastError();
}

template <int VEC, bool SILU>
cudaError_t norm_fwd(const NormArgs& a, void* ws, cudaStream_t stream) {
  const int lpr = lanes_per_row(a.channels, VEC), rows = rows_per_tile(a.channels, VEC);
  const dim3 grid((unsigned)tiles_of(a.n, rows), (unsigned)((a.channels + lpr * VEC - 1) / (lpr * VEC)));
  cudaError_t e = cudaSuccess;
  if (a.n > 0) {
    norm_part_kernel<VEC><<<grid, kNormThreads, 0, stream>>>(a, lpr, (float2*)ws);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) e = join<false>(a, rows, (float2*)ws, nullptr, stream);
  if (e == cudaSuccess && a.n > 0) {
    norm_apply_kernel<VEC, SILU><<<grid, kNormThreads, 0, stream>>>(a, lpr);
    e = cudaGetLastError();
  }
  return e;
}

template <int VEC, bool SILU>
cudaError_t norm_bwd(const NormArgs& a, void* ws, cudaStream_t stream) {
  const int lpr = lanes_per_row(a.channels, VEC), rows = rows_per_tile(a.channels, VEC);
  const long long tiles = tiles_of(a.n, rows), n_slots = tiles + a.samples;
  const dim3 grid((unsigned)tiles, (unsigned)((a.channels + lpr * VEC - 1) / (lpr * VEC)));
  float2* terms = (float2*)ws;
  float2* slots = (float2*)((char*)ws + pad256(sizeof(float2) * (size_t)a.samples * a.groups));
  cudaError_t e = cudaMemsetAsync(slots, 0, sizeof(float2) * (size_t)n_slots * a.channels, stream);
  if (e == cudaSuccess && a.n > 0) {
    norm_bwd_part_kernel<VEC, SILU><<<grid, kNormThreads, 0, stream>>>(a, lpr, slots);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess && a.grad_x != nullptr) {
    e = join<true>(a, rows, slots, terms, stream);
    if (e == cudaSuccess && a.n > 0) {
      norm_bwd_apply_kernel<VEC, SILU><<<grid, kNormThreads, 0, stream>>>(a, lpr, terms);
      e = cudaGetLastError();
    }
  }
  if (e == cudaSuccess && (a.grad_gamma != nullptr || a.grad_beta != nullptr)) {
    norm_param_kernel<<<(a.channels + 31) / 32, 1024, 0, stream>>>((int)n_slots, a.channels, slots, a.grad_gamma,
                                                                   a.grad_beta);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace

// Enough for both directions and for rows of any alignment.
size_t norm_workspace(int n, int samples, int channels, int groups) {
  const size_t slots = (size_t)tiles_of(n, rows_per_tile(channels, 1)) + (size_t)samples;
  return pad256(sizeof(float2) * (size_t)samples * groups) + pad256(sizeof(float2) * slots * (size_t)channels);
}

cudaError_t launch_norm_fwd(const NormArgs& a, int max_rows, void* ws, cudaStream_t stream) {
  (void)max_rows;
  if (a.samples == 0 || a.channels == 0) return cudaSuccess;
  const bool v4 = a.channels % 4 == 0 && vec4_rows(a.x, a.x_stride) && vec4_rows(a.y, a.y_stride);
  if (v4) return a.act ? norm_fwd<4, true>(a, ws, stream) : norm_fwd<4, false>(a, ws, stream);
  return a.act ? norm_fwd<1, true>(a, ws, stream) : norm_fwd<1, false>(a, ws, stream);
}

cudaError_t launch_norm_bwd(const NormArgs& a, int max_rows, void* ws, cudaStream_t stream) {
  (void)max_rows;
  if (a.channels == 0) return cudaSuccess;
  const bool v4 = a.channels % 4 == 0 && vec4_rows(a.x, a.x_stride) && vec4_rows(a.grad_y, a.gy_stride) &&
                  (a.grad_x == nullptr || vec4_rows(a.grad_x, a.gx_stride));
  if (v4) return a.act ? norm_bwd<4, true>(a, ws, stream) : norm_bwd<4, false>(a, ws, stream);
  return a.act ? norm_bwd<1, true>(a, ws, stream) : norm_bwd<1, false>(a, ws, stream);
}

}  // namespace cgtp
