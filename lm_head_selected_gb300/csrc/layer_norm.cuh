// Shared by the layer norm kernels (forward and backward).
#pragma once

#include "elem.cuh"

namespace llp {

// A row is D elements in `units` 16-byte vectors of W; the last one may be ragged.
// AL: rows are whole vectors, 16-byte aligned, and so are the parameters (a template
// parameter: as a run-time flag it cost the aligned kernels the predicated-off
// instructions of the other form, 1.5 times the time).

// W parameters from `src`, those at or past `n` reading as `none`.
template <int PT, int W, bool AL>
__device__ __forceinline__ void load_params(const typename Elem<PT>::T* src, int n, float none, F2 (&v)[W / 2]) {
  float f[W];
  if constexpr (AL) {
#pragma unroll
    for (int i = 0; i < W / Elem<PT>::W; ++i)
      Elem<PT>::unpack(__ldg(reinterpret_cast<const uint4*>(src) + i),
                       *reinterpret_cast<float(*)[Elem<PT>::W]>(f + i * Elem<PT>::W));
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) f[i] = i < n ? Elem<PT>::get(__ldg(src + i)) : none;
  }
#pragma unroll
  for (int i = 0; i < W / 2; ++i) v[i] = f2(f[2 * i], f[2 * i + 1]);
}

// Sums of a and b over the `warps` (1, 2, 4, 8 or 16) warps of a group (named barrier `id`),
// the same bits in every thread.  After one exchange the lower half of each warp sums a
// and the upper half b, so that both take little more than the shuffles of one; the warps
// meet in sm[2][16].
__device__ __forceinline__ void group_sums(float& a, float& b, float* sm, int warp, int warps, int id) {
  const int lane = threadIdx.x & 31;
  const bool upper = lane >= 16;
  float v = (upper ? b : a) + __shfl_xor_sync(0xffffffffu, upper ? a : b, 16);
#pragma unroll
  for (int off = 8; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if (warps > 1) {
    float* const half = sm + (lane & 16);
    if ((lane & 15) == 0) half[warp] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(32 * warps) : "memory");
    v = half[lane & (warps - 1)];
    for (int off = warps / 2; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  }
  a = __shfl_sync(0xffffffffu, v, 0);
  b = __shfl_sync(0xffffffffu, v, 16);
}

// The parameters of the row's columns as a CTA keeps them: in fp32, so that a row need not
// convert them again, as W / 4 arrays of `units` float4s (the first four columns of every
// vector, then the others), so that neighbouring threads read neighbouring vectors.
template <int PT, int W, bool AL>
__device__ __forceinline__ void keep_params(float4* kept, const typename Elem<PT>::T* src, float none, int D) {
  const int units = (D + W - 1) / W;
  for (int u = threadIdx.x; u < units; u += blockDim.x) {
    F2 v[W / 2];
#pragma unroll
    for (int i = 0; i < W / 2; ++i) v[i] = f2(none);
    if (src != nullptr) load_params<PT, W, AL>(src + u * W, min(D - u * W, W), 0.f, v);
#pragma unroll
    for (int i = 0; i < W / 4; ++i) kept[i * units + u] = make_float4(v[2 * i].x, v[2 * i].y, v[2 * i + 1].x, v[2 * i + 1].y);
  }
}

constexpr int kPipeSMs = 152;     // SMs that the persistent grids are made for
constexpr int kPipeUnits = 1024;  // vectors of the widest row that takes up to three per thread; twice as many take four

// Vectors of a thread that lie within the row for sure.
template <int K>
constexpr int kFull = K == 4 ? 2 : K - 1;

// Fixed-order sum over a CTA of THREADS threads: butterflies, then the warps in ascending order.
template <int THREADS>
__device__ __forceinline__ float cta_sum(float v, float* sm) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  v = sm[0];
#pragma unroll
  for (int w = 1; w < THREADS / 32; ++w) v += sm[w];
  return v;
}

}  // namespace llp
