// Launchers of the training-side operators: token sort and embedding
// (embed.cu), per-graph group norm (norm.cu) and the Newton-Schulz
// orthogonalisation (ortho.cu).  None of them uses the coefficient tables.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

namespace cgtp {

inline size_t pad256(size_t b) { return (b + 255) & ~(size_t)255; }

// ---- embed.cu ----
size_t token_sort_workspace(int n, int n_rows);
cudaError_t launch_token_sort(int n, int n_rows, const int* tokens, int* order, int* sorted, void* ws, cudaStream_t stream);
cudaError_t launch_embed_fwd(int n, int n_rows, int width, const int* tokens, const float* table, float scale,
                             float* out, long long out_stride, cudaStream_t stream);
size_t embed_bwd_workspace(int n, int width);
cudaError_t launch_embed_bwd(int n, int n_rows, int width, const int* order, const int* sorted, const float* grad_out,
                             long long grad_stride, float scale, float* grad_table, void* ws, cudaStream_t stream);

// ---- norm.cu ----
// Arguments of the per-graph group norm: samples are the row ranges
// [ptr[s], ptr[s + 1]) (ptr = nullptr: one sample of all n rows).
struct NormArgs {
  int n, samples, channels, groups;
  const int* ptr;
  const float* x;
  long long x_stride;
  const float *gamma, *beta;  // nullable: 1 and 0
  float eps;
  int act;  // 0 none, 1 SiLU
  // forward
  float* y;
  long long y_stride;
  float *mean, *rstd;  // [samples][groups], written by the forward, read by the backward
  // backward
  const float* grad_y;
  long long gy_stride;
  float* grad_x;
  long long gx_stride;
  float *grad_gamma, *grad_beta;  // nullable
};
size_t norm_workspace(int n, int samples, int channels, int groups, int max_rows, bool backward);
cudaError_t launch_norm_fwd(const NormArgs& a, int max_rows, void* ws, cudaStream_t stream);
cudaError_t launch_norm_bwd(const NormArgs& a, int max_rows, void* ws, cudaStream_t stream);

// ---- ortho.cu ----
size_t ortho_workspace(int batch, int rows, int cols);
cudaError_t launch_ortho(int batch, int rows, int cols, int steps, float scale, const float* g, float* out, void* ws,
                         cudaStream_t stream);

}  // namespace cgtp
