// Internal declarations of the residual RMS norm's kernels (residual_norm_fwd.cu, residual_norm_bwd.cu).
#pragma once

#include "llp_internal.h"

namespace llp {

enum GateKind { kGateNone = 0, kGateColumns = 1, kGateRows = 2 };

struct ResidualNormParams {
  const void* x;  // the backward's s
  const void* branch;
  const void* gate;
  const void* gs;  // the backward's upstream gradients
  const void* gh;
  long long x_stride, b_stride, gate_stride, gs_stride, gh_stride;  // elements between rows
  const void* post_weight;
  const void* weight;
  int gate_kind;
  int N, D;
  int dtype, param_dtype;
  float scale, eps;
};

struct ResidualNormOut {
  void* s;
  void* h;
  float* post_rstd;
  float* rstd;
};

struct ResidualNormGrads {
  const float* post_rstd;
  const float* rstd;
  void* gx;
  void* gb;
  void* ggate;
  void* gpost;
  void* gweight;
  void* workspace;
};

cudaError_t residual_norm_fwd_setup();
cudaError_t residual_norm_bwd_setup();
cudaError_t launch_residual_norm_fwd(const ResidualNormParams& p, const ResidualNormOut& o, cudaStream_t s);
size_t residual_norm_bwd_workspace(long long N, long long D);
cudaError_t launch_residual_norm_bwd(const ResidualNormParams& p, const ResidualNormGrads& o, cudaStream_t s);

}  // namespace llp
