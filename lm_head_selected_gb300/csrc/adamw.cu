// AdamW over many tensors in one launch.  The tensors' addresses come as kernel parameters, so that a
// step copies nothing to the device and can be captured; a CTA takes chunks of 4096 elements round
// robin, and finds a chunk's tensor by bisection.
//
// Bound by memory: 28 bytes per bf16 parameter with an fp32 master copy and states in 32 bits,
// 10 per bf16 parameter with states in 8 bits.
#include <cuda_fp8.h>

#include "adamw_internal.h"
#include "elem.cuh"

namespace llp {

namespace {

constexpr int kAdamThreads = 256;
constexpr int W = 8;  // elements of a thread's step
constexpr float kTop8 = 448.f;              // largest e4m3 value
constexpr float kLeast8 = 0.001953125f;     // smallest above 0, 2^-9
constexpr float kSmall8 = 1e-30f;           // scales above this and below its reciprocal have a normal reciprocal

struct Step {
  float b1, c1, b2, c2, eps, rate, rate_m, root_v, scale;
};

// beta^t by repeated squaring, in 64 bits.
__device__ double power(double b, long long t) {
  double r = 1.0;
  for (; t > 0; t >>= 1, b *= b)
    if (t & 1) r *= b;
  return r;
}

__device__ Step read_step(const AdamScalars& k) {
  Step s = {k.b1, k.c1, k.b2, k.c2, k.eps, k.rate, k.rate_m, k.root_v, 1.f};
  if (k.device_step != nullptr) {
    const long long t = k.step + *k.device_step;
    s.rate_m = static_cast<float>(k.rate / (1.0 - power(k.beta1, t)));
    s.root_v = static_cast<float>(1.0 / sqrt(1.0 - power(k.beta2, t)));
  }
  if (k.device_lr != nullptr) {
    const float lr = *k.device_lr;
    s.rate *= lr;
    s.rate_m *= lr;
  }
  if (k.grad_scale != nullptr) s.scale = *k.grad_scale;
  return s;
}

// N consecutive elements as fp32, whole vectors or one by one.
template <int DT, int N>
__device__ __forceinline__ void load_wide(const typename Elem<DT>::T* p, float (&v)[N]) {
  constexpr int E = Elem<DT>::W;
#pragma unroll
  for (int i = 0; i < N / E; ++i) {
    float f[E];
    Elem<DT>::unpack(*reinterpret_cast<const uint4*>(p + i * E), f);
#pragma unroll
    for (int j = 0; j < E; ++j) v[i * E + j] = f[j];
  }
}
template <int DT, int N>
__device__ __forceinline__ void store_wide(typename Elem<DT>::T* p, const float (&v)[N]) {
  constexpr int E = Elem<DT>::W;
#pragma unroll
  for (int i = 0; i < N / E; ++i) {
    float f[E];
#pragma unroll
    for (int j = 0; j < E; ++j) f[j] = v[i * E + j];
    *reinterpret_cast<uint4*>(p + i * E) = Elem<DT>::pack(f);
  }
}
template <int DT, int N>
__device__ __forceinline__ void load_few(const typename Elem<DT>::T* p, int n, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = i < n ? Elem<DT>::get(p[i]) : 0.f;
}
template <int DT, int N>
__device__ __forceinline__ void store_few(typename Elem<DT>::T* p, int n, const float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i < n) p[i] = Elem<DT>::put(v[i]);
}

// The moments and the parameter's new value.
__device__ __forceinline__ void update(const Step& s, float shrink, float g, float& m, float& v, float& root, float& p) {
  g *= s.scale;
  m = fmaf(s.b1, m, s.c1 * g);
  v = fmaf(s.b2, v, s.c2 * g * g);
  root = __fsqrt_rn(v);
  p = fmaf(p, shrink, -s.rate_m * __fdividef(m, fmaf(root, s.root_v, s.eps)));
}

// 32-bit states: N elements from `at`; VEC: all of them, whole vectors.
template <int PD, int GD, int N, bool VEC>
__device__ __forceinline__ void plain_elements(const AdamTensor& t, const Step& s, float shrink, long long at, int n) {
  using P = typename Elem<PD>::T;
  using G = typename Elem<GD>::T;
  P* const p = static_cast<P*>(t.p) + at;
  float* const m = static_cast<float*>(t.m) + at;
  float* const v = static_cast<float*>(t.v) + at;
  float pv[N], gv[N], mv[N], vv[N], root;
  if (VEC) {
    load_wide<GD, N>(static_cast<const G*>(t.g) + at, gv);
    load_wide<kDtypeF32, N>(m, mv);
    load_wide<kDtypeF32, N>(v, vv);
    if (t.master != nullptr)
      load_wide<kDtypeF32, N>(t.master + at, pv);
    else
      load_wide<PD, N>(p, pv);
  } else {
    load_few<GD, N>(static_cast<const G*>(t.g) + at, n, gv);
    load_few<kDtypeF32, N>(m, n, mv);
    load_few<kDtypeF32, N>(v, n, vv);
    if (t.master != nullptr)
      load_few<kDtypeF32, N>(t.master + at, n, pv);
    else
      load_few<PD, N>(p, n, pv);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) update(s, shrink, gv[i], mv[i], vv[i], root, pv[i]);
  if (VEC) {
    store_wide<kDtypeF32, N>(m, mv);
    store_wide<kDtypeF32, N>(v, vv);
    if (t.master != nullptr) store_wide<kDtypeF32, N>(t.master + at, pv);
    store_wide<PD, N>(p, pv);
  } else {
    store_few<kDtypeF32, N>(m, n, mv);
    store_few<kDtypeF32, N>(v, n, vv);
    if (t.master != nullptr) store_few<kDtypeF32, N>(t.master + at, n, pv);
    store_few<PD, N>(p, n, pv);
  }
}

template <int PD, int GD>
__device__ __forceinline__ void plain_chunk(const AdamTensor& t, const Step& s, int chunk) {
  const float shrink = 1.f - s.rate * t.decay;
  const int head = t.head < 0 ? 0 : t.head;
  const long long at = head + static_cast<long long>(chunk) * kAdamChunk;
  const int n = static_cast<int>(t.n - at < kAdamChunk ? t.n - at : kAdamChunk);  // head <= t.n: never below 0
  if (chunk == 0 && static_cast<int>(threadIdx.x) < head)
    plain_elements<PD, GD, 1, false>(t, s, shrink, threadIdx.x, 1);
  if (t.head < 0) {
    for (int i = threadIdx.x; i < n; i += kAdamThreads) plain_elements<PD, GD, 1, false>(t, s, shrink, at + i, 1);
    return;
  }
#pragma unroll 1
  for (int i = threadIdx.x * W; i < n; i += kAdamThreads * W) {
    if (i + W <= n)
      plain_elements<PD, GD, W, true>(t, s, shrink, at + i, W);
    else
      plain_elements<PD, GD, W, false>(t, s, shrink, at + i, n - i);
  }
}

// Eight e4m3 codes as fp32: e4m3 widens to fp16 exactly.
__device__ __forceinline__ void codes_to_float(uint2 c, float (&v)[W]) {
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i / 2] >> (16 * (i & 1))),
                                                     __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ uint2 float_to_codes(const float (&v)[W]) {
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t c = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i], v[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    w[i / 2] |= c << (16 * (i & 1));
  }
  return make_uint2(w[0], w[1]);
}

// The larger of two magnitudes; NaN if one is.
__device__ __forceinline__ float nan_max(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 8-bit states: a warp takes a block of kAdamBlock elements, eight per lane.
template <int PD, int GD>
__device__ __forceinline__ void block_elements(const AdamTensor& t, const Step& s, float shrink, long long block) {
  using P = typename Elem<PD>::T;
  using G = typename Elem<GD>::T;
  const int lane = threadIdx.x & 31;
  const long long at = block * kAdamBlock + lane * W;
  const int n = static_cast<int>(t.n - at < W ? (t.n - at > 0 ? t.n - at : 0) : W);
  P* const p = static_cast<P*>(t.p) + at;
  const G* const g = static_cast<const G*>(t.g) + at;
  unsigned char* const mc = static_cast<unsigned char*>(t.m) + at;
  unsigned char* const vc = static_cast<unsigned char*>(t.v) + at;
  const bool wide = t.head == 0 && n == W;
  float pv[W], gv[W], mv[W], vv[W], root[W];
  uint2 m8 = make_uint2(0, 0), v8 = make_uint2(0, 0);
  if (wide) {
    load_wide<GD, W>(g, gv);
    m8 = *reinterpret_cast<const uint2*>(mc);
    v8 = *reinterpret_cast<const uint2*>(vc);
    if (t.master != nullptr)
      load_wide<kDtypeF32, W>(t.master + at, pv);
    else
      load_wide<PD, W>(p, pv);
  } else {
    load_few<GD, W>(g, n, gv);
    if (t.master != nullptr)
      load_few<kDtypeF32, W>(t.master + at, n, pv);
    else
      load_few<PD, W>(p, n, pv);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const uint32_t a = i < n ? mc[i] : 0, b = i < n ? vc[i] : 0;
      if (i < 4) m8.x |= a << (8 * i), v8.x |= b << (8 * i);
      else m8.y |= a << (8 * i - 32), v8.y |= b << (8 * i - 32);
    }
  }
  const float ms = t.m_scale[block], vs = t.v_scale[block];
  codes_to_float(m8, mv);
  codes_to_float(v8, vv);
  float mt = 0.f, vt = 0.f;  // largest |m| and root of v
#pragma unroll
  for (int i = 0; i < W; ++i) {
    mv[i] *= ms;
    vv[i] *= vs;
    vv[i] *= vv[i];
    update(s, shrink, gv[i], mv[i], vv[i], root[i], pv[i]);
    mt = nan_max(mt, fabsf(mv[i]));
    vt = nan_max(vt, root[i]);
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) {
    mt = nan_max(mt, __shfl_xor_sync(0xffffffffu, mt, off));
    vt = nan_max(vt, __shfl_xor_sync(0xffffffffu, vt, off));
  }
  const float m_new = __fdiv_rn(mt, kTop8), v_new = __fdiv_rn(vt, kTop8);
  const float m_by = m_new != 0.f ? m_new : 1.f, v_by = v_new != 0.f ? v_new : 1.f;
  if (fminf(m_by, v_by) > kSmall8 && fmaxf(m_by, v_by) < 1.f / kSmall8) {
    const float m_inv = __fdiv_rn(1.f, m_by), v_inv = __fdiv_rn(1.f, v_by);
#pragma unroll
    for (int i = 0; i < W; ++i) mv[i] *= m_inv, vv[i] = root[i] * v_inv;
  } else {  // the reciprocal would be infinite or lose digits (or a value is not finite)
#pragma unroll
    for (int i = 0; i < W; ++i) mv[i] = __fdiv_rn(mv[i], m_by), vv[i] = __fdiv_rn(root[i], v_by);
  }
#pragma unroll
  for (int i = 0; i < W; ++i) vv[i] = vv[i] > 0.f ? fmaxf(vv[i], kLeast8) : vv[i];
  m8 = float_to_codes(mv);
  v8 = float_to_codes(vv);
  if (wide) {
    *reinterpret_cast<uint2*>(mc) = m8;
    *reinterpret_cast<uint2*>(vc) = v8;
    if (t.master != nullptr) store_wide<kDtypeF32, W>(t.master + at, pv);
    store_wide<PD, W>(p, pv);
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if (i < n) {
        mc[i] = static_cast<unsigned char>((i < 4 ? m8.x >> (8 * i) : m8.y >> (8 * i - 32)) & 0xFF);
        vc[i] = static_cast<unsigned char>((i < 4 ? v8.x >> (8 * i) : v8.y >> (8 * i - 32)) & 0xFF);
      }
    }
    if (t.master != nullptr) store_few<kDtypeF32, W>(t.master + at, n, pv);
    store_few<PD, W>(p, n, pv);
  }
  if (lane == 0) {
    t.m_scale[block] = m_new;
    t.v_scale[block] = v_new;
  }
}

template <int PD, int GD>
__device__ __forceinline__ void block_chunk(const AdamTensor& t, const Step& s, int chunk) {
  const float shrink = 1.f - s.rate * t.decay;
  const long long blocks = (t.n + kAdamBlock - 1) / kAdamBlock;
  long long b = static_cast<long long>(chunk) * (kAdamChunk / kAdamBlock) + (threadIdx.x >> 5);
#pragma unroll 1
  for (int i = 0; i < kAdamChunk / kAdamBlock / (kAdamThreads / 32); ++i, b += kAdamThreads / 32)
    if (b < blocks) block_elements<PD, GD>(t, s, shrink, b);
}

template <int PD, int GD, int BITS>
__device__ __forceinline__ void chunk_of(const AdamTensor& t, const Step& s, int chunk) {
  if constexpr (BITS == 8)
    block_chunk<PD, GD>(t, s, chunk);
  else
    plain_chunk<PD, GD>(t, s, chunk);
}

template <int MOST, int BITS>
__global__ void __launch_bounds__(kAdamThreads) adamw_kernel(const __grid_constant__ AdamTable<MOST> table) {
  __shared__ Step shared;
  if (threadIdx.x == 0) shared = read_step(table.k);
  __syncthreads();
  const Step s = shared;
  for (int c = blockIdx.x; c < table.chunks; c += gridDim.x) {
    int lo = 0, hi = table.count;  // the last tensor whose first chunk is not past c
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (table.t[mid].first_chunk <= c) lo = mid;
      else hi = mid;
    }
    const AdamTensor& t = table.t[lo];
    const int chunk = c - t.first_chunk;
    if (t.param_dtype == kDtypeF32) chunk_of<kDtypeF32, kDtypeF32, BITS>(t, s, chunk);
    else if (t.param_dtype == kDtypeBF16) {
      if (t.grad_dtype == kDtypeBF16) chunk_of<kDtypeBF16, kDtypeBF16, BITS>(t, s, chunk);
      else chunk_of<kDtypeBF16, kDtypeF32, BITS>(t, s, chunk);
    } else {
      if (t.grad_dtype == kDtypeF16) chunk_of<kDtypeF16, kDtypeF16, BITS>(t, s, chunk);
      else chunk_of<kDtypeF16, kDtypeF32, BITS>(t, s, chunk);
    }
  }
}

}  // namespace

template <int MOST>
cudaError_t launch_adamw(const AdamTable<MOST>& table, int bits, int num_sms, cudaStream_t s) {
  const int most = 8 * num_sms;
  const int blocks = table.chunks < most ? table.chunks : most;
  if (bits == 8)
    adamw_kernel<MOST, 8><<<blocks, kAdamThreads, 0, s>>>(table);
  else
    adamw_kernel<MOST, 32><<<blocks, kAdamThreads, 0, s>>>(table);
  return launch_result();
}

template cudaError_t launch_adamw<kAdamFew>(const AdamTable<kAdamFew>&, int, int, cudaStream_t);
template cudaError_t launch_adamw<kAdamMany>(const AdamTable<kAdamMany>&, int, int, cudaStream_t);

}  // namespace llp
