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

// Two fp32 values in one register pair, for the packed fp32 instructions.
using F2 = float2;
__device__ __forceinline__ F2 f2(float a, float b) { return make_float2(a, b); }
__device__ __forceinline__ F2 f2(float a) { return make_float2(a, a); }
__device__ __forceinline__ F2 add2(F2 a, F2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ F2 mul2(F2 a, F2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float sum2(F2 a) { return __fadd_rn(a.x, a.y); }

// One instruction each, within two units in the last place; subnormals count as 0.
__device__ __forceinline__ float root_ftz(float v) {
  float r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float inverse_ftz(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

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

// Loads of what another launch or another CTA of this one writes while this kernel is there
// already: from L2, not through the read-only path, which needs memory that stays the same
// for the whole life of the kernel.  Volatile and with a clobber, so that none is merged with
// another or moved above the griddepcontrol.wait or the fence before it.
__device__ __forceinline__ int load_written(const int* p) {
  int v;
  asm volatile("ld.global.cg.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ unsigned load_written(const unsigned* p) {
  unsigned v;
  asm volatile("ld.global.cg.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ float load_written(const float* p) {
  float v;
  asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ int4 load_written(const int4* p) {
  int4 v;
  asm volatile("ld.global.cg.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ float4 load_written(const float4* p) {
  float4 v;
  asm volatile("ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "l"(p)
               : "memory");
  return v;
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
// that shift until they are read.  `lo`, `hi`: the tensor's first and one past its last
// element; a word that sticks out of it is put together from elements instead.  Neighbouring
// lanes' words lie 16 bytes apart, so that a warp's access takes four lines for 128 bytes, five
// times per vector each way, and L1 is the busiest unit (75 to 77% of its peak, HBM at 15 to
// 26%): layer norm of 16384 x 1001 bf16 28.0 us, its gradient 36.0, where x 1000 takes 15.8
// and 21.9.
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
  // The same vector straight from global memory.
  static __device__ __forceinline__ uint4 load(const T* p, int n, const T* lo, const T* hi) {
    if constexpr (AL) {
      return __ldg(reinterpret_cast<const uint4*>(p));
    } else {
      uint32_t w[5] = {0, 0, 0, 0, 0};
      if constexpr (DT == kDtypeF32) {
#pragma unroll
        for (int i = 0; i < W; ++i)
          if (i < n) w[i] = __ldg(reinterpret_cast<const uint32_t*>(p) + i);
        return make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        const T* q = shifted(p) ? p - 1 : p;
        const int words = (static_cast<int>(p - q) + n + 1) / 2;
        const bool wide = q >= lo && q + 2 * words <= hi;
        const uint16_t* const h = reinterpret_cast<const uint16_t*>(q);
#pragma unroll
        for (int i = 0; i < 5; ++i) {
          if (wide) {
            if (i < words) w[i] = __ldg(reinterpret_cast<const uint32_t*>(q) + i);
          } else {
            const T *a = q + 2 * i, *b = a + 1;
            if (a >= p && a < p + n) w[i] = __ldg(h + 2 * i);
            if (b >= p && b < p + n) w[i] |= static_cast<uint32_t>(__ldg(h + 2 * i + 1)) << 16;
          }
        }
        const uint4 v = make_uint4(w[0], w[1], w[2], w[3]);
        return read(&v, w + 4, q != p, n);
      }
    }
  }
  // The same for memory that this kernel writes too, element by element unless aligned.
  static __device__ __forceinline__ uint4 load_changed(const T* p, int n) {
    if constexpr (AL) {
      return *reinterpret_cast<const uint4*>(p);
    } else {
      float f[W];
#pragma unroll
      for (int i = 0; i < W; ++i) f[i] = i < n ? Elem<DT>::get(p[i]) : 0.f;
      return Elem<DT>::pack(f);  // exact, but for the payload of a NaN
    }
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

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline int elem_bytes(int dtype) { return dtype == kDtypeF32 ? 4 : 2; }

}  // namespace llp
