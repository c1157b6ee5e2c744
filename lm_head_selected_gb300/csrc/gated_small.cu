// The gated linear layer's forward for few tokens (gated_small_most), with the operands of the
// contraction swapped:
//
//     gate^T [F, N] = Wg [F, D] . x^T [D, N],   up^T likewise
//
// so that the weights' rows lie on the MMA's M side and the few tokens on its N side (rounded up to 16).
// The kernel is a stream of the weights.  A CTA takes R rows of Wg and the same R rows of Wu (R a multiple
// of 8, at most 128, chosen so that the rows are spread evenly over the SMs: 10752 rows are 150 CTAs of
// 72), one MMA each per 16-deep step into two accumulators, so that lane j of one holds the gate and of
// the other the up projection of one column of y, for every token.  An MMA reads 128 rows: what lies
// behind the R-th belongs to other operands and feeds only accumulator lanes that no one reads.
//
// Where R is at most 64 (JOINT) both weights' rows go into one MMA, lanes 0..R-1 and R..2R-1: an MMA of few
// tokens takes about 80 cycles, mostly to read its 128 rows, and with two of them a step the K loop took
// 0.34 us per K block whatever the weights' size (2048 x 4096 of one token 15.6 us, together 11.1).
// The rows lie in groups of 8 (1024 bytes of a K block) at one stride: a copy of several K blocks brings each
// group's blocks side by side, so that the up projection's first group follows the gate's last.
// The epilogue then brings the two halves together through shared memory.
//
// Each weight has a map of its own.  One map over both, its third dimension stepping from one to the other,
// needed a copy less for each stage, but the copies' columns past D were then fetched behind the lower weight's
// last row, which faults where a mapped region ends there.
//
// An SM issues only about four tensor copies per microsecond whatever their size, so a stage is c K blocks
// of 64 (c = 1, 2 or 4) and comes as three copies: the gate's rows, the up projection's, x (in L2).
// Every element accumulates the same 16-wide steps in the same ascending order as in the CTA-pair GEMM,
// so that a token's row is bitwise the same in any batch.
//
// Bound by the weights' stream: 1 x 4096 x 16384 41.8 us in a captured graph (6.4 TB/s, 96% of the measured
// copy peak; CTA-pair tiles 87), 32 x 2688 x 10752 22.2 us (5.2 TB/s, 78%: 14 us of MMAs one after another
// and the start and end show beside 17 us of stream; CTA-pair tiles 35).
//
// Roles: warp 0 copies, warp 1 owns TMEM and issues the MMAs, warps 2..5 are the epilogue (a thread per
// weight row; one token's 32 neighbouring columns to a warp's store).  Every wait is bounded.
#include "elem.cuh"
#include "gated.cuh"
#include "gated.h"
#include "sm103_ptx.cuh"

namespace llp {

namespace {

constexpr int kGsThreads = 192;
constexpr int kGsMaxStages = 8;
constexpr int kGsBarBytes = 256;  // two rings of kGsMaxStages barriers, three more, two words

__host__ __device__ inline int gs_acc_cols(int BN) { return (BN + 31) / 32 * 32; }
__host__ __device__ inline int gs_stage_bytes(const GatedSmallParams& p) { return (2 * p.R + p.BN) * 128 * p.c; }

template <int ACT>
__device__ __forceinline__ void product32(float (&g)[32], const float (&u)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    const F2 v = mul2(gated_act<ACT>(f2(g[i], g[i + 1])), f2(u[i], u[i + 1]));
    g[i] = v.x;
    g[i + 1] = v.y;
  }
}

__device__ __forceinline__ uint16_t to16(bool f16, float x) {
  if (f16) {
    const __half h = __float2half_rn(x);
    return *reinterpret_cast<const uint16_t*>(&h);
  }
  const __nv_bfloat16 b = __float2bfloat16_rn(x);
  return *reinterpret_cast<const uint16_t*>(&b);
}

constexpr int kXchPitch = 33;  // floats of a row of the JOINT epilogue's exchange

template <bool JOINT>
__global__ void __launch_bounds__(kGsThreads, 1)
    gated_small_kernel(const __grid_constant__ CUtensorMap tm_g, const __grid_constant__ CUtensorMap tm_u,
                       const __grid_constant__ CUtensorMap tm_x, const GatedSmallParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // the barriers come first: what an MMA reads past its operand lies behind them
  uint64_t* const full = reinterpret_cast<uint64_t*>(smem);
  uint64_t* const empty = full + kGsMaxStages;
  uint64_t* const tmem_full = empty + kGsMaxStages;
  uint64_t* const tmem_empty = tmem_full + 1;
  uint64_t* const drain = tmem_empty + 1;
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint8_t* const ring = smem + 1024;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stage_bytes = gs_stage_bytes(p);
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(tmem_full, 1);
    mbar_init(tmem_empty, 4);  // one arrive per epilogue warp
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_g);
    tma_prefetch_desc(&tm_u);
    tma_prefetch_desc(&tm_x);
  }
  __syncwarp();
  if (warp == 1) {
    tmem_alloc(tmem_slot, p.tmem_cols);
    tmem_relinquish_alloc_permit();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t acc_cols = gs_acc_cols(p.BN);
  const int steps = (p.D + 64 * p.c - 1) / (64 * p.c);  // stages of a unit

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol_w = l2_policy_evict_first();  // streamed once
      const uint64_t pol_x = l2_policy_evict_last();   // re-read by every CTA
      int st = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int u = blockIdx.x; u < p.units && ok; u += gridDim.x) {
        for (int g = 0; g < steps; ++g) {
          if (!mbar_wait(&empty[st], ph ^ 1u, abort_flag, p.err, kDevTimeoutEmpty)) {
            ok = false;
            break;
          }
          const uint32_t base = smem_u32(ring + st * stage_bytes);
          const uint32_t up = base + p.R * 128 * p.c, x = up + p.R * 128 * p.c;
          mbar_arrive_expect_tx(&full[st], static_cast<uint32_t>(stage_bytes));
          if (JOINT && p.chunked) {
            tma_load_4d(base, &tm_g, &full[st], 0, 0, g * p.c, u * (p.R / 8), pol_w);
            tma_load_4d(up, &tm_u, &full[st], 0, 0, g * p.c, u * (p.R / 8), pol_w);
            tma_load_3d(x, &tm_x, &full[st], 0, 0, g * p.c, pol_x);
          } else if (p.chunked) {
            tma_load_3d(base, &tm_g, &full[st], 0, u * p.R, g * p.c, pol_w);
            tma_load_3d(up, &tm_u, &full[st], 0, u * p.R, g * p.c, pol_w);
            tma_load_3d(x, &tm_x, &full[st], 0, 0, g * p.c, pol_x);
          } else {
            for (int c = 0; c < p.c; ++c) {
              const int kx = (g * p.c + c) * 64;
              const uint32_t at = c * p.R * 128;  // JOINT: the two weights' rows of a K block lie together
              tma_load_2d(JOINT ? base + 2 * at : base + at, &tm_g, &full[st], kx, u * p.R, pol_w);
              tma_load_2d(JOINT ? base + 2 * at + p.R * 128 : up + at, &tm_u, &full[st], kx, u * p.R, pol_w);
              tma_load_2d(x + c * p.BN * 128, &tm_x, &full[st], kx, 0, pol_x);
            }
          }
          if (++st == p.stages) {
            st = 0;
            ph ^= 1u;
          }
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = make_idesc_16_f32(128, p.BN, false, false, p.f16 != 0);
      // JOINT: from a K block to the next, and between groups of 8 rows
      const uint32_t w_step = p.chunked ? 1024 : 2 * p.R * 128, w_group = p.chunked ? p.c * 1024 : 1024;
      int st = 0;
      uint32_t ph = 0, acc_ph = 0;
      for (int u = blockIdx.x; u < p.units; u += gridDim.x) {
        if (!mbar_wait(tmem_empty, acc_ph ^ 1u, abort_flag, p.err, kDevTimeoutTmemEmpty)) break;
        acc_ph ^= 1u;
        tc_fence_after_sync();
        bool ok = true;
        for (int g = 0; g < steps; ++g) {
          if (!mbar_wait(&full[st], ph, abort_flag, p.err, kDevTimeoutFull)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t base = smem_u32(ring + st * stage_bytes);
          for (int c = 0; c < p.c; ++c) {
            if (JOINT) {
              const uint64_t wd = make_smem_desc_sw128(base + c * w_step, 16, w_group);
              const uint64_t xd = make_smem_desc_sw128(base + 2 * p.c * p.R * 128 + c * p.BN * 128, 16, 1024);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                umma_bf16_f32(tmem_base, wd + 2 * kk, xd + 2 * kk, idesc, (g > 0 || c > 0 || kk > 0) ? 1u : 0u);
              continue;
            }
            const uint64_t gd = make_smem_desc_sw128(base + c * p.R * 128, 16, 1024);
            const uint64_t ud = make_smem_desc_sw128(base + (p.c + c) * p.R * 128, 16, 1024);
            const uint64_t xd = make_smem_desc_sw128(base + 2 * p.c * p.R * 128 + c * p.BN * 128, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {  // 16 elements, 32 bytes on in the swizzled row
              const uint32_t acc = (g > 0 || c > 0 || kk > 0) ? 1u : 0u;
              umma_bf16_f32(tmem_base, gd + 2 * kk, xd + 2 * kk, idesc, acc);
              umma_bf16_f32(tmem_base + acc_cols, ud + 2 * kk, xd + 2 * kk, idesc, acc);
            }
          }
          umma_commit(&empty[st]);
          if (++st == p.stages) {
            st = 0;
            ph ^= 1u;
          }
        }
        if (!ok) break;
        umma_commit(tmem_full);
      }
      umma_commit(drain);
      if (!mbar_wait_drain(drain, 0, 100000000ull)) atomicCAS(p.err, 0u, kDevTimeoutDrain);
    }
  } else {
    const int row = (warp & 3) * 32 + lane;  // TMEM lane, row of the unit
    const uint32_t taddr = tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const bool f16 = p.f16 != 0;
    uint32_t acc_ph = 0;
    for (int u = blockIdx.x; u < p.units; u += gridDim.x, acc_ph ^= 1u) {
      bool ok = mbar_wait(tmem_full, acc_ph, abort_flag, p.err, kDevTimeoutTmemFull);
      // the four warps meet at barriers below: all of them go on, or none
      if (JOINT) ok = named_bar_and(1, 128, ok);
      if (!ok) break;
      tc_fence_after_sync();
      if (JOINT) {
        // the ring is free: this CTA has one unit, and its MMAs are through
        float* const xch = reinterpret_cast<float*>(ring);
        const int tid = threadIdx.x - 64;  // warps 2..5
        const int r = tid & 63, half = tid >> 6;
        const long long f = static_cast<long long>(u) * p.R + r;
        const bool mine = r < p.R && f < p.F;
        const float* const gate_row = xch + r * kXchPitch;
        const float* const up_row = xch + (p.R + r) * kXchPitch;
        for (int n0 = 0; n0 < p.N; n0 += 32) {
          if ((warp & 3) * 32 < 2 * p.R) {  // warp-uniform
            float v[32];
            tmem_load_32cols(taddr + n0, v);
#pragma unroll
            for (int j = 0; j < 32; ++j) xch[row * kXchPitch + j] = v[j];
          }
          named_bar_sync(1, 128);
          if (mine) {
#pragma unroll 1
            for (int j = 16 * half; j < 16 * half + 16 && n0 + j < p.N; j += 2) {
              const bool two = n0 + j + 1 < p.N;
              const F2 g = f2(gate_row[j], gate_row[j + 1]), v = f2(up_row[j], up_row[j + 1]);
              const long long at = static_cast<long long>(n0 + j) * p.F + f;
              if (p.pre != nullptr) {
                uint16_t* const up = p.pre + static_cast<long long>(p.N) * p.F;
                p.pre[at] = to16(f16, g.x);
                up[at] = to16(f16, v.x);
                if (two) {
                  p.pre[at + p.F] = to16(f16, g.y);
                  up[at + p.F] = to16(f16, v.y);
                }
              }
              const F2 a = p.act == kActSilu   ? gated_act<kActSilu>(g)
                           : p.act == kActGelu ? gated_act<kActGelu>(g)
                                               : gated_act<kActGeluTanh>(g);
              const F2 y = mul2(a, v);
              p.y[at] = to16(f16, y.x);
              if (two) p.y[at + p.F] = to16(f16, y.y);
            }
          }
          named_bar_sync(1, 128);
        }
        break;
      }
      const long long f = static_cast<long long>(u) * p.R + row;
      const bool mine = row < p.R && f < p.F;
      if ((warp & 3) * 32 < p.R) {  // warp-uniform
        for (int n0 = 0; n0 < p.N; n0 += 32) {
          float g[32], v[32];
          tmem_load_32cols(taddr + n0, g);
          tmem_load_32cols(taddr + acc_cols + n0, v);
          if (p.pre != nullptr && mine) {
            uint16_t* const gate = p.pre + static_cast<long long>(n0) * p.F + f;
            uint16_t* const up = gate + static_cast<long long>(p.N) * p.F;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              if (n0 + j < p.N) {
                gate[static_cast<long long>(j) * p.F] = to16(f16, g[j]);
                up[static_cast<long long>(j) * p.F] = to16(f16, v[j]);
              }
            }
          }
          if (p.act == kActSilu)
            product32<kActSilu>(g, v);
          else if (p.act == kActGelu)
            product32<kActGelu>(g, v);
          else
            product32<kActGeluTanh>(g, v);
          if (mine) {
            uint16_t* const y = p.y + static_cast<long long>(n0) * p.F + f;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (n0 + j < p.N) y[static_cast<long long>(j) * p.F] = to16(f16, g[j]);
          }
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(tmem_empty);
    }
  }
  tc_fence_before_sync();
  __syncwarp();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 1) tmem_dealloc(tmem_base, p.tmem_cols);
}

// What an MMA reads behind the last stage's last rows: it takes 16 groups, p.c K blocks apart in the joint maps'
// layout, from the last K block's first.
int gs_slack(const GatedSmallParams& p) {
  const bool apart = p.joint && p.chunked;
  const int reads = apart ? 16384 * p.c : 16384;
  const int there = apart ? gs_stage_bytes(p) : (p.joint ? 2 : 1) * p.R * 128 + p.c * p.BN * 128;
  return there < reads ? reads - there : 0;
}
int gs_smem(const GatedSmallParams& p) { return 2048 + p.stages * gs_stage_bytes(p) + gs_slack(p); }

}  // namespace

bool gated_small_plan(int N, int D, int F, int num_sms, GatedSmallParams* p) {
  if (N < 1 || N > gated_small_most(F)) return false;
  p->N = N;
  p->D = D;
  p->F = F;
  p->BN = (N + 15) / 16 * 16;
  const long long sms = num_sms > 0 ? num_sms : 1;
  const long long waves = (F + sms * 128 - 1) / (sms * 128);
  const long long rows = (F + sms * waves - 1) / (sms * waves);
  p->R = static_cast<int>((rows + 7) / 8 * 8);
  p->units = (F + p->R - 1) / p->R;
  p->joint = p->R <= 64 ? 1 : 0;
  p->chunked = D % 64 == 0 ? 1 : 0;
  // K blocks per stage: as few as make a stage of 40 KB, at most four, and no more than there are
  const int blocks = (D + 63) / 64;
  p->c = 1;
  while (p->c < 4 && gs_stage_bytes(*p) < 40 * 1024 && p->c < blocks) p->c *= 2;
  p->stages = 1;
  while (p->stages < kGsMaxStages) {
    ++p->stages;
    if (gs_smem(*p) > kGatedSmallSmem) {
      --p->stages;
      break;
    }
  }
  int cols = 32;
  while (cols < (p->joint ? 1 : 2) * gs_acc_cols(p->BN)) cols *= 2;
  p->tmem_cols = cols;
  return p->stages >= 2;
}

cudaError_t gated_small_setup() {
  const cudaError_t e = note_cuda(cudaFuncSetAttribute(gated_small_kernel<false>,
                                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kGatedSmallSmem));
  return e != cudaSuccess ? e
                          : note_cuda(cudaFuncSetAttribute(gated_small_kernel<true>,
                                                           cudaFuncAttributeMaxDynamicSharedMemorySize, kGatedSmallSmem));
}

cudaError_t launch_gated_small(const CUtensorMap& wg, const CUtensorMap& wu, const CUtensorMap& x,
                               const GatedSmallParams& p, int num_sms, cudaStream_t s) {
  const int grid = p.units < num_sms ? p.units : num_sms;
  if (p.joint)
    gated_small_kernel<true><<<grid, kGsThreads, gs_smem(p), s>>>(wg, wu, x, p);
  else
    gated_small_kernel<false><<<grid, kGsThreads, gs_smem(p), s>>>(wg, wu, x, p);
  return launch_result();
}

}  // namespace llp
