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

// The forward of few tokens, weights on the MMA's M side (gated_small.cu).
constexpr int kSmallGatedMaxN = 128;
constexpr int kGatedSmallSmem = 232448;

struct GatedSmallParams {
  int N, D, F;
  int BN;      // MMA N: N rounded up to 16
  int R;       // rows of each weight to a CTA (height of the weights' boxes)
  int units;   // of R rows
  int c;       // K blocks of a stage
  int stages;
  int tmem_cols;
  int chunked;  // the maps are 3-D {64, rows, D / 64}: one copy per operand and stage (D % 64 == 0), else 2-D
  int act, f16;
  uint16_t* y;
  uint16_t* pre;  // [2][N][F], or nullptr
  unsigned int* err;
};
// Fills all up to tmem_cols; false when the batch is too large for the kernel.
bool gated_small_plan(int N, int D, int F, int num_sms, GatedSmallParams* p);
cudaError_t gated_small_setup();
cudaError_t launch_gated_small(const CUtensorMap& wg, const CUtensorMap& wu, const CUtensorMap& x,
                               const GatedSmallParams& p, int num_sms, cudaStream_t s);

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
