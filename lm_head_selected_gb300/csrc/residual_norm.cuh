// Shared by the residual RMS norm's kernels (forward and backward): a group of warps owns a row at a time,
// each thread K of its vectors, which it copies itself with cp.async into its own slots of a ring of rows.
#pragma once

#include "layer_norm.cuh"
#include "residual_norm.h"

namespace llp {

constexpr int kResThreads = 512;           // of a CTA, one per SM: 128 registers per thread
constexpr int kResSmem = 232448 - 2048;    // dynamic shared memory: what an SM has, less the static arrays

// W parameters in fp32, those at or past n reading as 0; src of the rows' type, or fp32.
template <int DT, int W, bool AL>
__device__ __forceinline__ void param_vector(const void* src, bool f32, int at, int n, F2 (&v)[W / 2]) {
  if (f32)
    load_params<kDtypeF32, W, AL>(static_cast<const float*>(src) + at, n, 0.f, v);
  else
    load_params<DT, W, AL>(static_cast<const typename Elem<DT>::T*>(src) + at, n, 0.f, v);
}

// scale * gate * post_weight of W columns, a gate per column and a post_weight where there are some.
template <int DT, int W, bool AL>
__device__ __forceinline__ void coefficient_vector(const ResidualNormParams& p, bool f32, int at, int n, F2 (&v)[W / 2]) {
#pragma unroll
  for (int i = 0; i < W / 2; ++i) v[i] = f2(p.scale);
  F2 t[W / 2];
  if (p.gate_kind == kGateColumns) {
    param_vector<DT, W, AL>(p.gate, f32, at, n, t);
#pragma unroll
    for (int i = 0; i < W / 2; ++i) v[i] = mul2(v[i], t[i]);
  }
  if (p.post_weight != nullptr) {
    param_vector<DT, W, AL>(p.post_weight, f32, at, n, t);
#pragma unroll
    for (int i = 0; i < W / 2; ++i) v[i] = mul2(v[i], t[i]);
  }
}

// Both as a CTA keeps them for all of its rows, in fp32: [2][W / 4][units] float4, the first four
// columns of every vector, then the others, so that neighbouring threads read neighbouring vectors.
template <int DT, bool AL>
__device__ __forceinline__ void keep_coefficients(float4* kept, const ResidualNormParams& p) {
  constexpr int W = Elem<DT>::W;
  const bool f32 = p.param_dtype == kDtypeF32;
  const int units = (p.D + W - 1) / W;
  for (int u = threadIdx.x; u < units; u += kResThreads) {
    const int n = min(p.D - u * W, W);
    F2 v[W / 2];
    coefficient_vector<DT, W, AL>(p, f32, u * W, n, v);
#pragma unroll
    for (int i = 0; i < W / 4; ++i) kept[i * units + u] = make_float4(v[2 * i].x, v[2 * i].y, v[2 * i + 1].x, v[2 * i + 1].y);
    if (p.weight != nullptr) {
      param_vector<DT, W, AL>(p.weight, f32, u * W, n, v);
#pragma unroll
      for (int i = 0; i < W / 4; ++i)
        kept[(W / 4 + i) * units + u] = make_float4(v[2 * i].x, v[2 * i].y, v[2 * i + 1].x, v[2 * i + 1].y);
    }
  }
}
template <int W>
__device__ __forceinline__ void kept_vector(const float4* kept, int which, int units, int u, F2 (&v)[W / 2]) {
#pragma unroll
  for (int i = 0; i < W / 4; ++i) {
    const float4 f = kept[(which * (W / 4) + i) * units + u];
    v[2 * i] = f2(f.x, f.y);
    v[2 * i + 1] = f2(f.z, f.w);
  }
}

// Sum over a group of `warps` (1, 2, 4, 8 or 16) warps: butterflies, then over its warps, which meet in
// sm[16] at named barrier `id`.  The same bits in every thread.  A group alternates between two arrays:
// a warp that is a sum ahead must not write over what another still reads.
__device__ __forceinline__ float group_sum(float v, float* sm, int warp, int warps, int id) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if (warps > 1) {
    if (lane == 0) sm[warp] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(32 * warps) : "memory");
    v = sm[lane & (warps - 1)];
    for (int off = warps / 2; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  }
  return v;
}

__device__ __forceinline__ void copies_left(int rows) {  // waits until at most `rows` (0 or 1) groups are in flight
  if (rows == 0)
    copy_wait<0>();
  else
    copy_wait<1>();
}

// Warps of a group and vectors of a thread for a row of `units` vectors, at most `most` vectors to a lane.
struct ResShape {
  int warps, K;
};
inline ResShape res_shape(int units, int most) {
  int warps = 1;
  while (warps < 16 && most * 32 * warps < units) warps *= 2;
  return {warps, (units + 32 * warps - 1) / (32 * warps)};
}

// Rows of the ring: two where shared memory holds them beside what is kept.  Three were slower (forward
// 16384 x 2688 62.2 us, 58.5 with two; gradient 16384 x 4096 136.5 and 134.2).
inline int res_stages(size_t per_stage, size_t kept) { return 2 * per_stage + kept <= kResSmem ? 2 : 1; }

// Whether rows of more than kPipeUnits vectors keep their coefficients too: where that costs no row of the
// ring.  Otherwise they are read anew for each row, as much from L2 as the row itself has in HBM.
inline bool res_keep(size_t per_stage, size_t kept) {
  return res_stages(per_stage, 0) * per_stage + kept <= kResSmem;
}

}  // namespace llp
