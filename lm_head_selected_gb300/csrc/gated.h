// Internal declarations of the gated linear layer's kernels (gated.cu).
#pragma once

#include "llp_internal.h"

namespace llp {

// Resident CTA pairs of each GEMM.
struct GatedCaps {
  int fwd_groups[2];  // of 128 and of 64 columns of y to a tile
  int gx_groups, gw_groups;
};

constexpr int kGatedPairs = 76;  // CTA pairs that the choices below are made for

// Columns of y to a tile: 64 where tiles of 128 leave more of the pairs idle in their last wave than narrow
// tiles cost (their MMAs read the same rows of x for half the columns).
inline int gated_cols(long long N, long long F) {
  const long long m = (N + kUnitM - 1) / kUnitM;
  const long long wide = (m * ((F + 127) / 128) + kGatedPairs - 1) / kGatedPairs;
  const long long narrow = (m * ((F + 63) / 64) + kGatedPairs - 1) / kGatedPairs;
  return narrow * 75 < wide * 100 ? 64 : 128;
}

// Segments of the long sum of grad_x: with fewer tiles than pairs, the K blocks are split among pairs, and
// the segments' fp32 partials are summed in ascending order.  In units of a K block's time on a pair
// (0.27 us): a segment's blocks and about 8 for its start and end, for each wave; the partials' way
// through memory at 5 TB/s.
inline int gated_segments(long long N, long long D, long long F_pad) {
  const long long tiles = ((N + kUnitM - 1) / kUnitM) * ((D + kTileN - 1) / kTileN), blocks = 2 * F_pad / kTileK;
  long long best = 1, best_cost = ((tiles + kGatedPairs - 1) / kGatedPairs) * (blocks + 8);
  for (long long n = 2; n <= 16 && n * tiles <= 2 * kGatedPairs; ++n) {
    const long long per = (blocks + n - 1) / n;
    if ((blocks + per - 1) / per != n) continue;
    const long long cost = ((tiles * n + kGatedPairs - 1) / kGatedPairs) * (per + 8) + 16 + n * N * D * 8 / 1350000;
    if (cost < best_cost) best = n, best_cost = cost;
  }
  return static_cast<int>(best);
}

struct GatedFwdParams {
  int N, D, F;
  int cols;  // of y to a tile, 128 or 64
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
