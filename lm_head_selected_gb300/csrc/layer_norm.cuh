// Shared by the layer norm kernels (forward and backward).
#pragma once

#include "elem.cuh"

namespace llp {

// The thread layout of a row: LANES threads own it together, lane l the units l,
// l + LANES, ... (K of them).  A unit is W = 16 bytes of elements when D is whole
// vectors, else one element.  The layout, and with it the order of every sum,
// depends on D and the types alone; `al` only chooses between one 16-byte access
// and W single ones.
template <int DT, int W>
struct RowUnit {
  using T = typename Elem<DT>::T;
  // W elements at p, as fp32
  static __device__ __forceinline__ void load(const T* p, bool al, float (&v)[W]) {
    if constexpr (W == 1) {
      v[0] = Elem<DT>::get(__ldg(p));
    } else if constexpr (W == Elem<DT>::W) {
      if (al) {
        Elem<DT>::unpack(__ldg(reinterpret_cast<const uint4*>(p)), v);
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = Elem<DT>::get(__ldg(p + i));
      }
    } else {  // fp32 parameters next to 16-bit rows: two vectors
      static_assert(DT == kDtypeF32 && W == 8, "");
      if (al) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = __ldg(p + i);
      }
    }
  }
  // W elements kept as stored (16 bytes, or one element) until they are needed
  using Raw = typename std::conditional<W == 1, T, uint4>::type;
  static __device__ __forceinline__ Raw load_raw(const T* p, bool al) {
    if constexpr (W == 1) {
      return __ldg(p);
    } else {
      static_assert(W == Elem<DT>::W, "");
      if (al) return __ldg(reinterpret_cast<const uint4*>(p));
      float v[W];
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] = Elem<DT>::get(__ldg(p + i));
      return Elem<DT>::pack(v);  // exact: the values are of this type
    }
  }
  static __device__ __forceinline__ Raw zero() {
    if constexpr (W == 1) return Elem<DT>::put(0.f);
    else return make_uint4(0, 0, 0, 0);
  }
  static __device__ __forceinline__ void unpack(const Raw& r, float (&v)[W]) {
    if constexpr (W == 1) v[0] = Elem<DT>::get(r);
    else Elem<DT>::unpack(r, v);
  }
  static __device__ __forceinline__ void store(T* p, bool al, const float (&v)[W]) {
    if constexpr (W == 1) {
      *p = Elem<DT>::put(v[0]);
    } else {
      if (al) {
        *reinterpret_cast<uint4*>(p) = Elem<DT>::pack(v);
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i) p[i] = Elem<DT>::put(v[i]);
      }
    }
  }
};

// NaN payloads may change in an unaligned load_raw; nothing else.

// Waits for the LANES threads of a row (a whole number of warps) that share the
// named barrier `id`.
template <int LANES>
__device__ __forceinline__ void row_barrier(int id) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(LANES) : "memory");
}

// Sums of M values over the LANES threads of a row, the same bits in each of them:
// butterflies within the warp, then the warps in ascending order through `sm`
// (LANES / 32 * M floats, not used again before the next row_barrier of the row).
template <int LANES, int M>
__device__ __forceinline__ void row_sum(float (&v)[M], float* sm, int id) {
#pragma unroll
  for (int off = (LANES < 32 ? LANES : 32) / 2; off >= 1; off >>= 1)
#pragma unroll
    for (int m = 0; m < M; ++m) v[m] += __shfl_xor_sync(0xffffffffu, v[m], off);
  if constexpr (LANES > 32) {
    constexpr int WARPS = LANES / 32;
    const int w = (threadIdx.x % LANES) >> 5;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int m = 0; m < M; ++m) sm[w * M + m] = v[m];
    }
    row_barrier<LANES>(id);
#pragma unroll
    for (int m = 0; m < M; ++m) v[m] = 0.f;
#pragma unroll
    for (int i = 0; i < WARPS; ++i)
#pragma unroll
      for (int m = 0; m < M; ++m) v[m] += sm[i * M + m];
  }
}

// Sum over a CTA of THREADS threads, in the same order.
template <int THREADS>
__device__ __forceinline__ float cta_sum(float v, float* sm) {
  float a[1] = {v};
  __syncthreads();
  row_sum<THREADS, 1>(a, sm, 0);
  return a[0];
}

}  // namespace llp
