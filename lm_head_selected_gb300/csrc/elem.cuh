// Elements of the three tensor types (bf16, fp32, fp16) as fp32 values, one at
// a time or as 16-byte vectors.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <type_traits>

#include "llp_internal.h"

namespace llp {

template <int DT>
struct Elem;

template <>
struct Elem<kDtypeBF16> {
  using T = __nv_bfloat16;
  static constexpr int W = 8;  // elements of a 16-byte vector
  static __device__ __forceinline__ float get(T v) { return __bfloat162float(v); }
  static __device__ __forceinline__ T put(float v) { return __float2bfloat16_rn(v); }
  static __device__ __forceinline__ void unpack(const uint4& r, float (&v)[W]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[W]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

template <>
struct Elem<kDtypeF16> {
  using T = __half;
  static constexpr int W = 8;
  static __device__ __forceinline__ float get(T v) { return __half2float(v); }
  static __device__ __forceinline__ T put(float v) { return __float2half_rn(v); }
  static __device__ __forceinline__ void unpack(const uint4& r, float (&v)[W]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[W]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 p = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

template <>
struct Elem<kDtypeF32> {
  using T = float;
  static constexpr int W = 4;
  static __device__ __forceinline__ float get(T v) { return v; }
  static __device__ __forceinline__ T put(float v) { return v; }
  static __device__ __forceinline__ void unpack(const uint4& r, float (&v)[W]) {
    v[0] = __uint_as_float(r.x);
    v[1] = __uint_as_float(r.y);
    v[2] = __uint_as_float(r.z);
    v[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[W]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
};

// A unit is what one thread moves at a time: a 16-byte vector, or one element
// where rows are not 16-byte aligned.
template <int DT, bool VEC>
struct Unit {
  using T = typename Elem<DT>::T;
  static constexpr int W = VEC ? Elem<DT>::W : 1;
  using Raw = typename std::conditional<VEC, uint4, T>::type;
  static __device__ __forceinline__ Raw load(const T* p) {
    if constexpr (VEC) return __ldg(reinterpret_cast<const uint4*>(p));
    else return __ldg(p);
  }
  static __device__ __forceinline__ Raw zero() {
    if constexpr (VEC) return make_uint4(0, 0, 0, 0);
    else return Elem<DT>::put(0.f);
  }
  static __device__ __forceinline__ void unpack(const Raw& r, float (&v)[W]) {
    if constexpr (VEC) Elem<DT>::unpack(r, v);
    else v[0] = Elem<DT>::get(r);
  }
  static __device__ __forceinline__ void store(T* p, const float (&v)[W]) {
    if constexpr (VEC) *reinterpret_cast<uint4*>(p) = Elem<DT>::pack(v);
    else *p = Elem<DT>::put(v[0]);
  }
  static __device__ __forceinline__ void store_raw(T* p, const Raw& r) { *reinterpret_cast<Raw*>(p) = r; }
};

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline int elem_bytes(int dtype) { return dtype == kDtypeF32 ? 4 : 2; }

}  // namespace llp
