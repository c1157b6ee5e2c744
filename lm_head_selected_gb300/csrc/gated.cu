// Gated linear layer y = act(x Wg^T) * (x Wu^T) and its gradient, on the tcgen05 core.
//
// Forward: one GEMM over both projections.  A CTA pair's 256 x 256 (or 256 x 128) tile has 128 (64) columns of each:
// of the tile's B rows the even CTA loads its half from Wg and the odd CTA its half from Wu, so
// that the accumulator's first half is the gate and its second half the up projection of the same
// 128 columns of y, and every thread of the epilogue holds both factors of its row.  The
// projections never leave the SM unless they are kept for the gradient; y is formed from the
// fp32 accumulators.
//
// Backward, from the kept projections:
//   dG = grad_y * up * act'(gate),  dU = grad_y * act(gate)       one elementwise pass
//   grad_x   = dG . Wg + dU . Wu        one GEMM over K = 2 F: the K blocks of the first half
//                                       take B from Wg, those of the second from Wu
//   grad_Wg  = dG^T . x,  grad_Wu = dU^T . x      one launch over the tiles of both
// dG and dU are rounded to the tensors' 16-bit type, as the tensor cores take them; they lie in
// one workspace [N][2][F_pad], F_pad a multiple of 128 with zeros in the padding.
//
// Bound by the tensor cores for batches.  16384 x 2688 x 10752 bf16: forward with both projections kept
// 1.05 to 1.17 ms as the power-capped clock has it (1.61 to 1.8 PFLOP/s, 94 to 105% of the measured sustained
// rate); gradient 2.52 to 2.65 ms: the elementwise pass 0.275 (6.4 TB/s), the GEMMs 1.07 each (1.77
// PFLOP/s).  512 x 2688 x 10752: gradient 104 us, 158 without the split of grad_x's sum.  24772 x 544 x 360: 71
// us, 169 without the split of the weights' sums over the tokens.
#include "gated.h"

#include "grad_gemm.cuh"

#include "elem.cuh"
#include "gated.cuh"

namespace llp {

namespace {

struct GatedMaps {
  CUtensorMap a, b, c;  // x, Wg, y
  CUtensorMap b2, c2;   // Wu, the kept projections [2][N][F]
};

// COLS: columns of y in a tile, 128 or 64.
template <int COLS>
struct GatedFwdCfg : PlainOperands {
  using Maps = GatedMaps;
  using Params = GatedFwdParams;
  static constexpr bool A_MN = false;
  static constexpr bool B_MN = false;
  static constexpr bool PAIR = true;
  static constexpr int BN = 2 * COLS;
  static constexpr int A_ROWS = kTileM;
  static constexpr int STAGES = COLS == 128 ? kPairStages : 8;  // of 32 or 24 KB
  static constexpr int EXTRA_SMEM = kEpiSmemBytes;

  struct RowState {};

  static __device__ __forceinline__ const CUtensorMap* b_map(const Maps& m, const Params&, uint32_t rank, int) {
    return rank == 0 ? &m.b : &m.b2;
  }
  static __device__ __forceinline__ int b_row(const Params&, int n0, int, int, int, int) { return n0; }
  static __device__ __forceinline__ const CUtensorMap* c_map2(const Maps& m) { return &m.c2; }
  static __device__ __forceinline__ uint64_t policy_a() { return l2_policy_evict_last(); }
  static __device__ __forceinline__ uint64_t policy_b() { return l2_policy_evict_normal(); }
  static constexpr bool DYNAMIC = false;
  static __device__ __forceinline__ int* sched_counter(const Params&) { return nullptr; }
  static __device__ __forceinline__ unsigned int* progress_counter(const Params&) { return nullptr; }
  static __device__ __forceinline__ bool a_chunked(const Params&) { return false; }
  static __device__ __forceinline__ bool b_chunked(const Params&) { return false; }
  static __device__ __forceinline__ int kps(const Params& p) { return p.kps; }
  static __device__ __forceinline__ void on_launch(const Params&) {}

  static __device__ __forceinline__ int num_units(const Params& p) { return p.num_m * p.num_ft; }

  // groups of group_m row tiles; inside a group the column tile is the slow index, so that the
  // pairs that run together share weight tiles in L2
  static __device__ __forceinline__ UnitInfo unit(const Params& p, int u) {
    const int gsize = p.group_m * p.num_ft;
    const int grp = u / gsize;
    const int r = u - grp * gsize;
    const int gm = min(p.group_m, p.num_m - grp * p.group_m);
    const int ft = r / gm;
    UnitInfo ui;
    ui.m0 = (grp * p.group_m + (r - ft * gm)) * kUnitM;
    ui.n0 = ft * COLS;
    ui.ntiles = 1;
    ui.kb0 = 0;
    ui.nkb = (p.D + BK - 1) / BK;
    ui.bn = BN;
    return ui;
  }

  static __device__ __forceinline__ void unit_begin(const Params&, const UnitInfo&, int, int, RowState&) {}
  static __device__ __forceinline__ void unit_end(const Params&, const UnitInfo&, int, int, RowState&) {}

  static __device__ __forceinline__ void put32(uint32_t sbuf, int lane, int h, bool f16, const float (&z)[32]) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      epi_slab_put(sbuf, lane, 4 * h + k, pack16x2(f16, z[8 * k + 0], z[8 * k + 1]),
                   pack16x2(f16, z[8 * k + 2], z[8 * k + 3]), pack16x2(f16, z[8 * k + 4], z[8 * k + 5]),
                   pack16x2(f16, z[8 * k + 6], z[8 * k + 7]));
  }

  template <int ACT>
  static __device__ __forceinline__ void product(float (&g)[32], const float (&u)[32]) {
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const F2 v = mul2(gated_act<ACT>(f2(g[i], g[i + 1])), f2(u[i], u[i + 1]));
      g[i] = v.x;
      g[i + 1] = v.y;
    }
  }

  static __device__ __forceinline__ void tile(const Params& p, const UnitInfo& ui, int, int, int row, int lane,
                                              uint32_t taddr, RowState&, EpiStore& es) {
    const int row0 = ui.m0 + row - lane;
    if (row0 >= p.N) return;  // this warp's rows are all past the end (warp-uniform)
    const bool f16 = p.f16 != 0;
#pragma unroll 1
    for (int q = 0; q < COLS / 64; ++q) {  // 64-column slabs; rows and columns past the end are clipped
      const int f0 = ui.n0 + 64 * q;
      if (f0 >= p.F) break;  // warp-uniform
      if (p.keep) {
#pragma unroll 1
        for (int z = 0; z < 2; ++z) {
          const uint32_t sbuf = epi_slab_begin(es);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float v[32];
            tmem_load_32cols(taddr + COLS * z + 64 * q + 32 * h, v);
            put32(sbuf, lane, h, f16, v);
          }
          epi_slab_store_3d_to(es, es.map2, sbuf, f0, row0, z);
        }
      }
      const uint32_t sbuf = epi_slab_begin(es);
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        float g[32], u[32];
        tmem_load_32cols(taddr + 64 * q + 32 * h, g);
        tmem_load_32cols(taddr + COLS + 64 * q + 32 * h, u);
        if (p.act == kActSilu)
          product<kActSilu>(g, u);
        else if (p.act == kActGelu)
          product<kActGelu>(g, u);
        else
          product<kActGeluTanh>(g, u);
        put32(sbuf, lane, h, f16, g);
      }
      epi_slab_store_2d(es, sbuf, f0, row0);
    }
  }
};

// ---------------------------------------------------------------- backward

// grad_x: the K blocks of the second half come from Wu.
struct GatedGradXCfg : GradCfg<false, true> {
  struct Maps {
    CUtensorMap a, b, c;  // dG and dU side by side, Wg, grad_x
    CUtensorMap b2;       // Wu
  };
  using Params = GatedGradXParams;
  static __device__ __forceinline__ const CUtensorMap* b_map(const Maps& m, const Params& p, uint32_t, int kb) {
    return kb < p.half_blocks ? &m.b : &m.b2;
  }
  static __device__ __forceinline__ int b_kx(const Params& p, int kb) {
    return (kb < p.half_blocks ? kb : kb - p.half_blocks) * BK;
  }
};

// grad_Wg and grad_Wu: row tiles [0, tiles) are of Wg, [tiles, 2 tiles) of Wu.
struct GatedGradWCfg : GradCfg<true, true> {
  using Base = GradCfg<true, true>;
  struct Maps {
    CUtensorMap a, b, c;  // dG and dU side by side, x, grad_Wg
    CUtensorMap c2;       // grad_Wu
  };
  using Params = GatedGradWParams;
  static __device__ __forceinline__ const CUtensorMap* c_map2(const Maps& m) { return &m.c2; }
  static __device__ __forceinline__ UnitInfo unit(const Params& p, int u) {
    UnitInfo ui = Base::unit(p, u);
    const int mt = ui.m0 / kUnitM + p.first_tile;
    ui.m0 = mt < p.tiles ? mt * kUnitM : p.F_pad + (mt - p.tiles) * kUnitM;
    return ui;
  }
  static __device__ __forceinline__ void tile(const Params& p, const UnitInfo& ui, int u, int j, int row, int lane,
                                              uint32_t taddr, RowState& rs, EpiStore& es) {
    const CUtensorMap* const gate = es.map;
    UnitInfo v = ui;
    // a tile of the first half may end past F_pad but starts before it
    if (v.m0 >= p.F_pad) {
      v.m0 -= p.F_pad;
      es.map = es.map2;
    }
    Base::tile(p, v, u, j, row, lane, taddr, rs, es);
    es.map = gate;
  }
};

// dG and dU of 8 columns of a row per step.  Bound by memory: three tensors read, two written.
constexpr int kDpreThreads = 256;
template <int DT, int ACT>
__global__ void __launch_bounds__(kDpreThreads) gated_dpre_kernel(const uint4* __restrict__ gy,
                                                                  const uint4* __restrict__ gate,
                                                                  const uint4* __restrict__ up, int N, int F, int F_pad,
                                                                  uint4* __restrict__ dpre, int* sched) {
  constexpr int W = 8;
  if (blockIdx.x == 0 && threadIdx.x < kNumSchedCounters) sched[threadIdx.x] = 0;  // of the GEMMs that follow
  const int vecs = F / W, pitch = F_pad / W;  // of a row, and with its padding
  const long long step = static_cast<long long>(gridDim.x) * kDpreThreads;
  const long long at = static_cast<long long>(blockIdx.x) * kDpreThreads + threadIdx.x;
  long long n = at / pitch;
  int c = static_cast<int>(at - n * pitch);
  const long long n_step = step / pitch;
  const int c_step = static_cast<int>(step - n_step * pitch);
  while (n < N) {
    uint4* const out = dpre + n * 2 * pitch + c;
    if (c < vecs) {
      const long long i = n * vecs + c;
      F2 y[W / 2], g[W / 2], u[W / 2];
      unpack2<DT, W>(__ldg(gy + i), y);
      unpack2<DT, W>(__ldg(gate + i), g);
      unpack2<DT, W>(__ldg(up + i), u);
#pragma unroll
      for (int k = 0; k < W / 2; ++k) {
        F2 a, slope;
        gated_act_slope<ACT>(g[k], a, slope);
        g[k] = mul2(mul2(y[k], u[k]), slope);
        u[k] = mul2(y[k], a);
      }
      out[0] = pack2<DT, W>(g);
      out[pitch] = pack2<DT, W>(u);
    } else {
      out[0] = out[pitch] = make_uint4(0, 0, 0, 0);
    }
    n += n_step;
    c += c_step;
    if (c >= pitch) {
      c -= pitch;
      ++n;
    }
  }
}

template <int DT>
cudaError_t dpre(const GatedBwdParams& p, int blocks, cudaStream_t s) {
  const uint4* const gy = static_cast<const uint4*>(p.gy);
  const uint4* const gate = static_cast<const uint4*>(p.pre);
  const uint4* const up = gate + static_cast<size_t>(p.N) * p.F / 8;
  const auto kernel = p.act == kActSilu   ? gated_dpre_kernel<DT, kActSilu>
                      : p.act == kActGelu ? gated_dpre_kernel<DT, kActGelu>
                                          : gated_dpre_kernel<DT, kActGeluTanh>;
  kernel<<<blocks, kDpreThreads, 0, s>>>(gy, gate, up, p.N, p.F, p.F_pad, static_cast<uint4*>(p.dpre), p.sched);
  return launch_result();
}

// The segments' partials of the weights' gradients, part [2][nseg][count], one weight to each blockIdx.y.
constexpr int kJoinThreads = 256;
__global__ void __launch_bounds__(kJoinThreads) gated_join_kernel(const float4* __restrict__ part, int nseg,
                                                                  long long count4, uint2* gate, uint2* up, bool f16) {
  uint2* const out = blockIdx.y == 0 ? gate : up;
  if (out == nullptr) return;
  part += static_cast<size_t>(blockIdx.y) * nseg * count4;
  const long long step = static_cast<long long>(gridDim.x) * kJoinThreads;
  for (long long i = static_cast<long long>(blockIdx.x) * kJoinThreads + threadIdx.x; i < count4; i += step) {
    float4 sum = __ldg(part + i);
#pragma unroll 8
    for (int s = 1; s < nseg; ++s) {
      const float4 v = __ldg(part + s * count4 + i);
      sum = make_float4(sum.x + v.x, sum.y + v.y, sum.z + v.z, sum.w + v.w);
    }
    out[i] = make_uint2(pack16x2(f16, sum.x, sum.y), pack16x2(f16, sum.z, sum.w));
  }
}

}  // namespace

cudaError_t launch_gated_join(const float* part, int nseg, long long count, void* gate, void* up, bool f16, int num_sms,
                              cudaStream_t s) {
  const long long want = (count / 4 + kJoinThreads - 1) / kJoinThreads, most = 4LL * num_sms;
  const dim3 grid(static_cast<unsigned>(want < most ? want : most), 2);
  gated_join_kernel<<<grid, kJoinThreads, 0, s>>>(reinterpret_cast<const float4*>(part), nseg, count / 4,
                                                  static_cast<uint2*>(gate), static_cast<uint2*>(up), f16);
  return launch_result();
}

cudaError_t gated_setup(GatedCaps* caps) {
  cudaError_t e = note_cuda(setup_gemm<GatedFwdCfg<128>>(&caps->fwd_groups[0]));
  if (e == cudaSuccess) e = note_cuda(setup_gemm<GatedFwdCfg<64>>(&caps->fwd_groups[1]));
  if (e == cudaSuccess) e = note_cuda(setup_gemm<GatedGradXCfg>(&caps->gx_groups));
  if (e == cudaSuccess) e = note_cuda(setup_gemm<GatedGradWCfg>(&caps->gw_groups));
  return e;
}

cudaError_t launch_gated_fwd(const CUtensorMap& x, const CUtensorMap& wg, const CUtensorMap& wu, const CUtensorMap& y,
                             const CUtensorMap& pre, const GatedFwdParams& p, const GatedCaps& caps, cudaStream_t s) {
  const long long units = static_cast<long long>(p.num_m) * p.num_ft;
  return p.cols == 128 ? launch_units<GatedFwdCfg<128>>({x, wg, y, wu, pre}, p, units, caps.fwd_groups[0], s)
                       : launch_units<GatedFwdCfg<64>>({x, wg, y, wu, pre}, p, units, caps.fwd_groups[1], s);
}

cudaError_t launch_gated_dpre(const GatedBwdParams& p, int num_sms, cudaStream_t s) {
  const long long vecs = static_cast<long long>(p.N) * (p.F_pad / 8);
  const long long want = (vecs + kDpreThreads - 1) / kDpreThreads, most = 8LL * num_sms;
  const int blocks = static_cast<int>(want < most ? want : most);
  return p.dtype == kDtypeF16 ? dpre<kDtypeF16>(p, blocks, s) : dpre<kDtypeBF16>(p, blocks, s);
}

cudaError_t launch_gated_grad_x(const CUtensorMap& dpre, const CUtensorMap& wg, const CUtensorMap& wu,
                                const CUtensorMap& gx, const GatedGradXParams& p, const GatedCaps& caps,
                                cudaStream_t s) {
  const long long units = static_cast<long long>(p.nseg) * p.num_m * p.num_d;
  return launch_units<GatedGradXCfg>({dpre, wg, gx, wu}, p, units, caps.gx_groups, s);
}

cudaError_t launch_gated_grad_w(const CUtensorMap& dpre, const CUtensorMap& x, const CUtensorMap& gwg,
                                const CUtensorMap& gwu, const GatedGradWParams& p, const GatedCaps& caps,
                                cudaStream_t s) {
  const long long units = static_cast<long long>(p.nseg) * p.num_m * p.num_d;
  return launch_units<GatedGradWCfg>({dpre, x, gwg, gwu}, p, units, caps.gw_groups, s);
}

}  // namespace llp
