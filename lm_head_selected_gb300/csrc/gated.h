// Internal declarations of the gated linear layer's kernels (gated.cu).
#pragma once

#include "llp_internal.h"

namespace llp {

constexpr int kGatedPairs = 76;  // CTA pairs that the choices below are made for

// Resident CTA pairs of each GEMM.
struct GatedCaps {
  int fwd_groups[2];  // of 128 and of 64 columns of y to a tile
  int gx_groups, gw_groups;
};

// Columns of y to a tile: 64 where all of those tiles run at once.  They take 0.73 of the time of 128 (512
// tokens or fewer, 2048 x 4096: 12.5 us, 16.5 with 128); with more waves they lose (4096 x 4096 x 8192
// 383 us, 288 with 128).
inline int gated_cols(long long N, long long F) {
  return ((N + kUnitM - 1) / kUnitM) * ((F + 63) / 64) <= kGatedPairs ? 64 : 128;
}

// Segments of a gradient's long sum: with fewer tiles than pairs, the K blocks are split among pairs, and
// the segments' fp32 partials of its `count` elements are summed in ascending order.  In units of a K block's
// time on a pair (0.27 us): a segment's blocks and about 8 for its start and end, for each wave; the
// partials' way through memory at 5 TB/s.  `per`: blocks of a segment, a multiple of `step`.
struct GatedSplit {
  int nseg, per;
};
inline GatedSplit gated_split(long long tiles, long long blocks, long long count, long long step) {
  long long best = 1, best_per = blocks, best_cost = ((tiles + kGatedPairs - 1) / kGatedPairs) * (blocks + 8);
  for (long long n = 2; n <= 16 && n * tiles <= 2 * kGatedPairs; ++n) {
    const long long per = ((blocks + n - 1) / n + step - 1) / step * step;
    if ((blocks + per - 1) / per != n) continue;
    const long long cost = ((tiles * n + kGatedPairs - 1) / kGatedPairs) * (per + 8) + 16 + n * count * 8 / 1350000;
    if (cost < best_cost) best = n, best_per = per, best_cost = cost;
  }
  return {static_cast<int>(best), static_cast<int>(best_per)};
}
inline long long gated_tiles(long long rows, long long cols) {
  return ((rows + kUnitM - 1) / kUnitM) * ((cols + kTileN - 1) / kTileN);
}
inline GatedSplit gated_split_x(long long N, long long D, long long F_pad) {
  return gated_split(gated_tiles(N, D), 2 * F_pad / kTileK, N * D, 1);
}
// Of both weights' gradients, whichever is asked for: the same bits then.  A stage may hold two blocks.
inline GatedSplit gated_split_w(long long N, long long D, long long F) {
  return gated_split(2 * gated_tiles(F, D), (N + kTileK - 1) / kTileK, 2 * F * D, 2);
}

struct GatedFwdParams {
  int N, D, F;
  int cols;  // of y to a tile
  int num_m, num_ft, group_m;
  int keep;  // the projections are stored too
  int act;
  int f16, kps;
  unsigned int* err;
};

// The forward of few tokens, weights on the MMA's M side (gated_small.cu).
constexpr int kGatedSmallSmem = 232448;

// Most tokens that it takes.  The CTA-pair tiles of 128 columns take one time whatever the batch up to 256
// tokens, which is short where they all run at once and only half the pairs have one: 2048 x 4096 12.5 us,
// this kernel 12.2 of 32 tokens, 13.6 of 64; 2048 x 8192 19.0, 17.8 of 96 and 20.0 of 128; with a second
// wave 2688 x 10752 36.7, 34.9 of 224 and 37.9 of 256.
inline int gated_small_most(long long F) {
  const long long tiles = (F + 127) / 128;
  return tiles <= kGatedPairs / 2 ? 32 : tiles <= kGatedPairs ? 96 : 224;
}

struct GatedSmallParams {
  int N, D, F;
  int BN;      // MMA N: N rounded up to 16
  int R;       // rows of each weight to a CTA (height of the weights' boxes)
  int joint;   // both weights' rows in one MMA: where R is at most 64
  int units;   // of R rows
  int c;       // K blocks of a stage
  int stages;
  int tmem_cols;
  int chunked;  // the maps reach several K blocks: one copy per operand and stage (D % 64 == 0), else 2-D
  int act, f16;
  uint16_t* y;
  uint16_t* pre;  // [2][N][F], or nullptr
  unsigned int* err;
};
// Fills all up to chunked; false when the batch is too large for the kernel.
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
// out[k][i] = the sum over s of part[k][s][i], rounded; either may be null.
cudaError_t launch_gated_join(const float* part, int nseg, long long count, void* gate, void* up, bool f16, int num_sms,
                              cudaStream_t s);
cudaError_t launch_gated_grad_w(const CUtensorMap& dpre, const CUtensorMap& x, const CUtensorMap& gwg,
                                const CUtensorMap& gwu, const GatedGradWParams& p, const GatedCaps& caps,
                                cudaStream_t s);

}  // namespace llp
