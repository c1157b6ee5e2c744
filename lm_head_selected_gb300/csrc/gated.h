// Internal declarations of the gated linear layer's kernels (gated.cu).
#pragma once

#include "llp_internal.h"

namespace llp {

// Resident CTA pairs of each GEMM.
struct GatedCaps {
  int fwd_groups, gx_groups, gw_groups;
};

struct GatedFwdParams {
  int N, D, F;
  int num_m, num_ft, group_m;
  int keep;  // the projections are stored too
  int act;
  int f16, kps;
  unsigned int* err;
};

struct GatedBwdParams {
  const void* gy;
  const void* pre;   // [2][N][F]
  void* dpre;        // [N][2][F_pad]
  int* sched;        // [kNumSchedCounters] ticket counters of the two GEMMs, zeroed here
  int N, F, F_pad;
  int dtype, act;
};

struct GatedGradXParams : GradGemmParams {
  int half_blocks;  // K blocks of each half
};

struct GatedGradWParams : GradGemmParams {
  int F_pad;
  int tiles;       // row tiles of one weight
  int first_tile;  // of the launch: 0, or `tiles` where only Wu's gradient is asked for
};

cudaError_t gated_setup(GatedCaps* caps);
cudaError_t launch_gated_fwd(const CUtensorMap& x, const CUtensorMap& wg, const CUtensorMap& wu, const CUtensorMap& y,
                             const CUtensorMap& pre, const GatedFwdParams& p, const GatedCaps& caps, cudaStream_t s);
cudaError_t launch_gated_dpre(const GatedBwdParams& p, int num_sms, cudaStream_t s);
cudaError_t launch_gated_grad_x(const CUtensorMap& dpre, const CUtensorMap& wg, const CUtensorMap& wu,
                                const CUtensorMap& gx, const GatedGradXParams& p, const GatedCaps& caps,
                                cudaStream_t s);
cudaError_t launch_gated_grad_w(const CUtensorMap& dpre, const CUtensorMap& x, const CUtensorMap& gwg,
                                const CUtensorMap& gwu, const GatedGradWParams& p, const GatedCaps& caps,
                                cudaStream_t s);

}  // namespace llp
