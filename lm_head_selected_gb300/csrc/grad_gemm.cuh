// The gradient GEMMs' configuration of the tcgen05 core, shared by the linear log-prob's backward
// and the gated linear layer's, and the rounding to the path's 16-bit type.
#pragma once

#include "gemm_core.cuh"

namespace llp {

__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b) {
  __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t pack_f16x2(float a, float b) {
  __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}

// Two floats rounded to the path's 16-bit type (fp16 when f16, else bf16).
__device__ __forceinline__ uint32_t pack16x2(bool f16, float a, float b) {
  return f16 ? pack_f16x2(a, b) : pack_bf16x2(a, b);
}

// ----------------------------------------------------------------------------
// Gradient GEMMs with fixed K segments (B2 and B3 of the linear log-prob).
// ----------------------------------------------------------------------------
template <bool A_MN_, bool B_MN_>
struct GradCfg : PlainOperands {
  static constexpr bool A_MN = A_MN_;
  static constexpr bool B_MN = B_MN_;
  static_assert(B_MN, "half-width column tiles load B in 64-row MN-major boxes");
  static constexpr bool PAIR = kPairMMA;
  static constexpr int BN = kTileN;
  static constexpr int A_ROWS = BM;
  static constexpr int STAGES = PAIR ? kPairStages : 4;
  static constexpr int EXTRA_SMEM = kEpiSmemBytes;
  static constexpr int UM = kUnitM;
  using Params = GradGemmParams;

  struct RowState {
    int r;
  };

  static __device__ __forceinline__ uint64_t policy_a() { return l2_policy_evict_normal(); }
  // grad_weight's B, the hidden states, is re-read by every unit
  static __device__ __forceinline__ uint64_t policy_b() {
    return (A_MN && LLP_GW_H_EVICT_LAST) ? l2_policy_evict_last() : l2_policy_evict_normal();
  }
  // units are claimed in ascending order from a ticket counter, so the tiles
  // that share A rows or a K window of B run together
  static constexpr bool DYNAMIC = (LLP_DYNAMIC_SCHED & (A_MN ? 2 : 1)) != 0;
  static __device__ __forceinline__ int* sched_counter(const Params& p) { return p.sched; }
  static __device__ __forceinline__ unsigned int* progress_counter(const Params& p) { return p.progress; }
  static __device__ __forceinline__ bool a_chunked(const Params& p) { return p.a_chunked != 0; }
  static __device__ __forceinline__ bool b_chunked(const Params& p) { return p.b_chunked != 0; }
  static __device__ __forceinline__ int kps(const Params& p) { return p.kps; }
  // grad_weight's B is the hidden states
  static __device__ __forceinline__ void on_launch(const Params&) {}

  // The odd CTA's half of a last column tile may lie past the end: it loads the even one's columns then, for
  // accumulator columns that no one reads.  A copy from outside the tensor is not free: those of all pairs went
  // to the same few lines of L2 (the gated layer's elementwise pass and grad_x at 16384 x 128 x 384 27 us, 16
  // with this).
  static __device__ __forceinline__ int b_row(const Params& p, int n0, int, int, int rank, int rows) {
    return n0 + rank * rows < p.D ? n0 + rank * rows : n0;
  }

  static __device__ __forceinline__ int num_units(const Params& p) { return p.nseg * p.num_m * p.num_d; }

  // Segment is the slowest index, then M tile, then the output column tile, so the
  // CTAs that run together share A rows and the same K window of B.
  static __device__ __forceinline__ UnitInfo unit(const Params& p, int u) {
    const int per_seg = p.num_m * p.num_d;
    const int seg = u / per_seg;
    const int r = u - seg * per_seg;
    const int mt = r / p.num_d;
    const int dt = r - mt * p.num_d;
    const int total_kb = (p.K + BK - 1) / BK;
    UnitInfo ui;
    ui.m0 = mt * UM;
    ui.n0 = dt * BN;
    ui.ntiles = 1;
    ui.kb0 = seg * p.kseg_blocks;
    ui.nkb = min(p.kseg_blocks, total_kb - ui.kb0);
    ui.bn = (LLP_HALF_TILE && p.D - ui.n0 <= BN / 2) ? BN / 2 : BN;  // ragged last column tile: half-width MMA
    return ui;
  }

  static __device__ __forceinline__ void unit_begin(const Params&, const UnitInfo& ui, int, int row, RowState& rs) {
    rs.r = ui.m0 + row;
  }

  // Output through 32-row slabs and TMA stores: bf16 [rows][D] with one
  // segment, else the fp32 partial of this segment in [nseg][rows][D] (a 3-D
  // tensor map, so rows past `rows` are clipped inside the segment).
  static __device__ __forceinline__ void tile(const Params& p, const UnitInfo& ui, int u, int, int row, int lane,
                                              uint32_t taddr, RowState&, EpiStore& es) {
    const int seg = u / (p.num_m * p.num_d);
    const int row0 = ui.m0 + row - lane;
    if (row0 >= p.rows) return;  // this warp's rows are all past the end (warp-uniform)
    if (p.nseg == 1 && !p.f32_out) {
      const bool f16 = p.f16 != 0;
#pragma unroll 1
      for (int q = 0; q < BN / 64; ++q) {
        const int d0 = ui.n0 + 64 * q;
        if (d0 >= p.D) break;  // warp-uniform
        const uint32_t sbuf = epi_slab_begin(es);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float a[32];
          tmem_load_32cols(taddr + 64 * q + 32 * h, a);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            epi_slab_put(sbuf, lane, 4 * h + k, pack16x2(f16, a[8 * k + 0], a[8 * k + 1]),
                         pack16x2(f16, a[8 * k + 2], a[8 * k + 3]), pack16x2(f16, a[8 * k + 4], a[8 * k + 5]),
                         pack16x2(f16, a[8 * k + 6], a[8 * k + 7]));
        }
        epi_slab_store_2d(es, sbuf, d0, row0);
      }
    } else {
#pragma unroll 1
      for (int c = 0; c < BN / 32; ++c) {
        const int d0 = ui.n0 + 32 * c;
        if (d0 >= p.D) break;  // warp-uniform
        const uint32_t sbuf = epi_slab_begin(es);
        float a[32];
        tmem_load_32cols(taddr + 32 * c, a);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          epi_slab_put(sbuf, lane, k, __float_as_uint(a[4 * k + 0]), __float_as_uint(a[4 * k + 1]),
                       __float_as_uint(a[4 * k + 2]), __float_as_uint(a[4 * k + 3]));
        epi_slab_store_3d(es, sbuf, d0, row0, seg);
      }
    }
  }

  static __device__ __forceinline__ void unit_end(const Params&, const UnitInfo&, int, int, RowState&) {}
};

template <class Cfg>
inline cudaError_t launch_units(const typename Cfg::Maps& maps, const typename Cfg::Params& p, long long units,
                                int groups, cudaStream_t s) {
  const long long g = units < groups ? units : groups;
  return launch_gemm<Cfg>(maps, p, static_cast<int>(g) * Plan<Cfg>::NCTA, s);
}

}  // namespace llp
