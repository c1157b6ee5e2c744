// Shared by the layer norm kernels (forward and backward).
#pragma once

#include "elem.cuh"

namespace llp {

// Two fp32 values in one register pair, for the packed fp32 instructions.
using F2 = float2;
__device__ __forceinline__ F2 f2(float a, float b) { return make_float2(a, b); }
__device__ __forceinline__ F2 f2(float a) { return make_float2(a, a); }
__device__ __forceinline__ F2 add2(F2 a, F2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ F2 mul2(F2 a, F2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float sum2(F2 a) { return __fadd_rn(a.x, a.y); }

// A row is D elements in `units` 16-byte vectors of W; the last one may be ragged.

template <int DT, int W>
__device__ __forceinline__ void unpack2(const uint4& r, F2 (&v)[W / 2]) {
  float f[W];
  Elem<DT>::unpack(r, f);
#pragma unroll
  for (int i = 0; i < W / 2; ++i) v[i] = f2(f[2 * i], f[2 * i + 1]);
}
template <int DT, int W>
__device__ __forceinline__ uint4 pack2(const F2 (&v)[W / 2]) {
  float f[W];
#pragma unroll
  for (int i = 0; i < W / 2; ++i) f[2 * i] = v[i].x, f[2 * i + 1] = v[i].y;
  return Elem<DT>::pack(f);
}

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

__device__ __forceinline__ void copy_async(void* slot, const void* p) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(slot))),
               "l"(p)
               : "memory");
}
__device__ __forceinline__ void copy_async4(void* slot, const void* p) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(slot))),
               "l"(p)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// A thread's copy of one vector of a row in shared memory, and what it takes to fill and
// read it.  Aligned: 16 bytes, one cp.async.  Otherwise 4-byte words: an odd row of 16-bit
// elements may start in the middle of one, so that its vectors take five words; they keep
// that shift until they are read.  `span`: the tensor's first and one past its last
// element; a word that sticks out of it is put together from elements instead.
template <int DT, bool AL>
struct Slot {
  using T = typename Elem<DT>::T;
  static constexpr int W = Elem<DT>::W;
  static constexpr bool FIVE = !AL && DT != kDtypeF32;
  static constexpr int BYTES = FIVE ? 20 : 16;  // per vector
  static __device__ __forceinline__ bool shifted(const T* p) { return FIVE && (reinterpret_cast<uintptr_t>(p) & 2) != 0; }
  static __device__ __forceinline__ void copy(uint4* slot, uint32_t* fifth, const T* p, int n, const T* lo, const T* hi) {
    if constexpr (AL) {
      copy_async(slot, p);
    } else if constexpr (DT == kDtypeF32) {
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (i < n) copy_async4(reinterpret_cast<float*>(slot) + i, p + i);
    } else {
      const T* q = shifted(p) ? p - 1 : p;  // 4-byte aligned
      const int words = (static_cast<int>(p - q) + n + 1) / 2;
      if (q >= lo && q + 2 * words <= hi) {
#pragma unroll
        for (int i = 0; i < 5; ++i)
          if (i < words) copy_async4(i < 4 ? reinterpret_cast<uint32_t*>(slot) + i : fifth, q + 2 * i);
      } else {
        uint32_t w[5];
#pragma unroll
        for (int i = 0; i < 5; ++i) {
          const T *a = q + 2 * i, *b = a + 1;
          const uint32_t l = a >= p && a < p + n ? *reinterpret_cast<const uint16_t*>(a) : 0;
          const uint32_t h = b >= p && b < p + n ? *reinterpret_cast<const uint16_t*>(b) : 0;
          w[i] = l | h << 16;
        }
        *slot = make_uint4(w[0], w[1], w[2], w[3]);
        *fifth = w[4];
      }
    }
  }
  // The vector, elements at or past n reading as 0.
  static __device__ __forceinline__ uint4 read(const uint4* slot, const uint32_t* fifth, bool shift, int n) {
    uint4 r = *slot;
    if constexpr (FIVE) {
      if (shift) {
        r.x = __funnelshift_r(r.x, r.y, 16);
        r.y = __funnelshift_r(r.y, r.z, 16);
        r.z = __funnelshift_r(r.z, r.w, 16);
        r.w = __funnelshift_r(r.w, *fifth, 16);
      }
      if (n < W) {
        uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = 2 * i >= n ? 0 : 2 * i + 1 >= n ? w[i] & 0xFFFFu : w[i];
        r = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    return r;
  }
  // The first n elements of a vector to a row.
  static __device__ __forceinline__ void store(T* p, const uint4& v, int n) {
    if constexpr (AL) {
      *reinterpret_cast<uint4*>(p) = v;
    } else {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      if constexpr (DT == kDtypeF32) {
#pragma unroll
        for (int i = 0; i < W; ++i)
          if (i < n) reinterpret_cast<uint32_t*>(p)[i] = w[i];
      } else {
        uint16_t* const h = reinterpret_cast<uint16_t*>(p);
        if (n == W && !shifted(p)) {
#pragma unroll
          for (int i = 0; i < 4; ++i) reinterpret_cast<uint32_t*>(p)[i] = w[i];
        } else if (n == W) {
          h[0] = static_cast<uint16_t>(w[0]);
#pragma unroll
          for (int i = 0; i < 3; ++i) reinterpret_cast<uint32_t*>(p + 1)[i] = __funnelshift_r(w[i], w[i + 1], 16);
          h[7] = static_cast<uint16_t>(w[3] >> 16);
        } else {
#pragma unroll
          for (int i = 0; i < W; ++i)
            if (i < n) h[i] = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
        }
      }
    }
  }
};

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
constexpr int kPipeUnits = 1024;  // vectors of the widest row of the one-pass kernels

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
