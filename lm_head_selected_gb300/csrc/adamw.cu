// AdamW over many tensors in one launch.  The tensors' addresses come as kernel parameters, so that a
// step copies nothing to the device and can be captured; a CTA takes chunks of the tensors round robin,
// and finds a chunk's tensor by bisection.
//
// Bound by memory.  States in 32 bits: 28 bytes per bf16 parameter with an fp32 master copy.  439 M of
// them 1850 us (6.6 TB/s, 99% of the measured copy peak) with 512 threads and chunks of 4096 elements to an
// SM; four CTAs of 256 took 2075: with more streams at once each has less of a DRAM page.
// States in 8 bits: 10 bytes per bf16 parameter.  369 M of them, with gradients everywhere, 605 us (6.1 TB/s,
// 91%).  What it took, from 1123 us: the blocks to come in a ring of shared memory (828), codes in 16-byte
// copies and scales not loaded by themselves (755), scales stored 64 bytes at a time (698), fewer warps with
// deeper rings and no spills (652), codes exact to the border (669), the warps' rings on banks of their own
// (600), the decay subtracted with the update (605).  Blocks with an element that has had no gradient yet are read
// twice and take the general form: 352 M parameters 572 us, 1.29 ms at the first step, 3.12 ms where 97% of a
// table's rows never had a gradient.
#include <cfloat>

#include <cuda_fp8.h>

#include "adamw_internal.h"
#include "elem.cuh"

namespace llp {

namespace {

constexpr int kAdamThreads = 256;   // of a CTA, states in 32 bits
constexpr int kPackedThreads = 128;  // and in 8
constexpr int kWarpBlocks = kAdamPackedChunk / kAdamBlock / (kPackedThreads / 32);  // to a warp of a chunk
static_assert(kAdamPackedChunk % (2 * kAdamBlock * (kPackedThreads / 32)) == 0 && kWarpBlocks <= 16, "a lane for each scale");
template <int BITS>
constexpr int kAdamResident = BITS == 8 ? 4 : 2;  // CTAs to an SM
constexpr int W = 8;  // elements of a thread's step
constexpr float kTop8 = 448.f;              // largest e4m3 value
constexpr float kLeast8 = 0.001953125f;     // smallest above 0, 2^-9

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

// The parameter less decay * p and the update, one rounding for the three: a factor 1 - decay would be rounded to
// 2^-25 beforehand, for every element and step alike (a decay of 1e-7 19% too large, one of 1e-8 lost).  An
// infinite parameter stays what it is.
__device__ __forceinline__ float bounded(float p) { return fminf(fmaxf(p, -FLT_MAX), FLT_MAX); }
__device__ __forceinline__ F2 moved(F2 p, float decay, F2 minus_update) {
  return add2(p, fma2(f2(bounded(p.x), bounded(p.y)), f2(-decay), minus_update));
}

// The moments and the parameter's new value.
__device__ __forceinline__ void update(const Step& s, float decay, float g, float& m, float& v, float& root, float& p) {
  g *= s.scale;
  m = fmaf(s.b1, m, s.c1 * g);
  v = fmaf(s.b2, v, s.c2 * g * g);
  root = sqrtf(v);
  p -= fmaf(bounded(p), decay, s.rate_m * __fdividef(m, fmaf(root, s.root_v, s.eps)));
}

// 32-bit states: N elements from `at`; VEC: all of them, whole vectors.
template <int PD, int GD, int N, bool VEC>
__device__ __forceinline__ void plain_elements(const AdamTensor& t, const Step& s, float decay, long long at, int n) {
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
  for (int i = 0; i < N; ++i) update(s, decay, gv[i], mv[i], vv[i], root, pv[i]);
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
__device__ __forceinline__ void plain_chunk(const AdamTensor& t, const Step* shared, int chunk) {
  const Step s = *shared;
  const float decay = s.rate * t.decay;
  const int head = t.head < 0 ? 0 : t.head;
  const long long at = head + static_cast<long long>(chunk) * kAdamChunk;
  const int n = static_cast<int>(t.n - at < kAdamChunk ? t.n - at : kAdamChunk);  // head <= t.n: never below 0
  if (chunk == 0 && static_cast<int>(threadIdx.x) < head)
    plain_elements<PD, GD, 1, false>(t, s, decay, threadIdx.x, 1);
  if (t.head < 0) {
    for (int i = threadIdx.x; i < n; i += kAdamThreads) plain_elements<PD, GD, 1, false>(t, s, decay, at + i, 1);
    return;
  }
#pragma unroll 1
  for (int i = threadIdx.x * W; i < n; i += kAdamThreads * W) {
    if (i + W <= n)
      plain_elements<PD, GD, W, true>(t, s, decay, at + i, W);
    else
      plain_elements<PD, GD, W, false>(t, s, decay, at + i, n - i);
  }
}

// Two e4m3 codes (the low or the high half of a word's four) as fp32: e4m3 widens to fp16 exactly.
__device__ __forceinline__ F2 codes_to_f2(uint32_t word, int half) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(word >> (16 * half)), __NV_E4M3);
  return __half22float2(__half2(h));
}
__device__ __forceinline__ uint32_t f2_to_codes(F2 v) {
  return __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint2 all_codes(const F2 (&v)[W / 2]) {
  return make_uint2(f2_to_codes(v[0]) | f2_to_codes(v[1]) << 16, f2_to_codes(v[2]) | f2_to_codes(v[3]) << 16);
}

// The larger of two magnitudes; NaN if one is.
__device__ __forceinline__ float nan_max(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Of three, in one instruction: max.NaN of magnitudes, and min.
__device__ __forceinline__ float nan_max3_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// A lane's eight elements of a block with 8-bit states, as they lie in memory.
template <int PD, int GD, bool MASTER>
struct Packed {
  static constexpr int PV = MASTER || PD == kDtypeF32 ? 2 : 1, GV = GD == kDtypeF32 ? 2 : 1;
  uint4 p[PV], g[GV];
  uint2 m, v;
  float ms, vs;
};

// The blocks to come are under way in a ring of shared memory, two neighbours to a slot, so that their codes
// too come in 16-byte copies, which go past L1 (8-byte ones need lines of it, and there is little left
// beside the ring).
template <int PD, int GD, bool MASTER>
struct Slot8 {
  using R = Packed<PD, GD, MASTER>;
  uint4 p[2][R::PV * 32];  // as in memory: neighbouring lanes copy neighbouring vectors
  uint4 g[2][R::GV * 32];
  uint2 m[2][32];
  uint2 v[2][32];
};
// Bytes of a warp's ring: four slots of 16-bit parameters and gradients, two or three of others, and an odd
// multiple of 16 bytes, so that the CTA's rings do not all start on the same banks (bf16, 186 M
// parameters: 282 us, 306 with multiples of 32, 319 of 128).
constexpr int kWarpRing = 12400;

// The pair's blocks below `stop`.
template <int PD, int GD, bool MASTER>
__device__ __forceinline__ void copy_pair(const AdamTensor& t, long long block, long long stop, Slot8<PD, GD, MASTER>* slot) {
  using R = Packed<PD, GD, MASTER>;
  const int lane = threadIdx.x & 31;
  const bool both = block + 1 < stop;
  const long long at = block * kAdamBlock;
  const uint4* const p = (MASTER ? reinterpret_cast<const uint4*>(t.master + at)
                                 : reinterpret_cast<const uint4*>(static_cast<const typename Elem<PD>::T*>(t.p) + at)) + lane;
  const uint4* const g = reinterpret_cast<const uint4*>(static_cast<const typename Elem<GD>::T*>(t.g) + at) + lane;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (k == 0 || both) {
#pragma unroll
      for (int i = 0; i < R::PV; ++i) copy_async(&slot->p[k][i * 32 + lane], p + (k * R::PV + i) * 32);
#pragma unroll
      for (int i = 0; i < R::GV; ++i) copy_async(&slot->g[k][i * 32 + lane], g + (k * R::GV + i) * 32);
    }
  }
  if (lane < 16 || both) {
    copy_async(reinterpret_cast<uint4*>(slot->m) + lane, static_cast<const unsigned char*>(t.m) + at + 16 * lane);
    copy_async(reinterpret_cast<uint4*>(slot->v) + lane, static_cast<const unsigned char*>(t.v) + at + 16 * lane);
  }
}

template <int PD, int GD, bool MASTER>
__device__ __forceinline__ void read_packed(const Slot8<PD, GD, MASTER>* slot, int k, Packed<PD, GD, MASTER>& r) {
  using R = Packed<PD, GD, MASTER>;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < R::PV; ++i) r.p[i] = slot->p[k][lane * R::PV + i];
#pragma unroll
  for (int i = 0; i < R::GV; ++i) r.g[i] = slot->g[k][lane * R::GV + i];
  r.m = slot->m[k][lane];
  r.v = slot->v[k][lane];
}

// A block's elements straight from memory: whole vectors, or at the tensor's end and off the vectors'
// boundaries one by one; what is not there is 0.
template <int PD, int GD, bool MASTER>
__device__ __forceinline__ void load_packed(const AdamTensor& t, long long block, Packed<PD, GD, MASTER>& r) {
  using R = Packed<PD, GD, MASTER>;
  const long long at = block * kAdamBlock + (threadIdx.x & 31) * W;
  const uint4* const p = MASTER ? reinterpret_cast<const uint4*>(t.master + at)
                                : reinterpret_cast<const uint4*>(static_cast<const typename Elem<PD>::T*>(t.p) + at);
  const uint4* const g = reinterpret_cast<const uint4*>(static_cast<const typename Elem<GD>::T*>(t.g) + at);
#pragma unroll
  for (int i = 0; i < R::PV; ++i) r.p[i] = p[i];
#pragma unroll
  for (int i = 0; i < R::GV; ++i) r.g[i] = g[i];
  r.m = *reinterpret_cast<const uint2*>(static_cast<const unsigned char*>(t.m) + at);
  r.v = *reinterpret_cast<const uint2*>(static_cast<const unsigned char*>(t.v) + at);
  r.ms = t.m_scale[block];
  r.vs = t.v_scale[block];
}
template <int PD, int GD, bool MASTER>
__device__ __forceinline__ void load_packed_few(const AdamTensor& t, long long block, int n, Packed<PD, GD, MASTER>& r) {
  using P = typename Elem<PD>::T;
  using G = typename Elem<GD>::T;
  using R = Packed<PD, GD, MASTER>;
  const long long at = block * kAdamBlock + (threadIdx.x & 31) * W;
  r.ms = t.m_scale[block];
  r.vs = t.v_scale[block];
  float f[8];
  load_few<GD, W>(static_cast<const G*>(t.g) + at, n, f);
#pragma unroll
  for (int i = 0; i < R::GV; ++i) {
    float part[Elem<GD>::W];
#pragma unroll
    for (int j = 0; j < Elem<GD>::W; ++j) part[j] = f[i * Elem<GD>::W + j];
    r.g[i] = Elem<GD>::pack(part);
  }
  constexpr int PDT = MASTER ? kDtypeF32 : PD;
  if constexpr (MASTER)
    load_few<kDtypeF32, W>(t.master + at, n, f);
  else
    load_few<PD, W>(static_cast<const P*>(t.p) + at, n, f);
#pragma unroll
  for (int i = 0; i < R::PV; ++i) {
    float part[Elem<PDT>::W];
#pragma unroll
    for (int j = 0; j < Elem<PDT>::W; ++j) part[j] = f[i * Elem<PDT>::W + j];
    r.p[i] = Elem<PDT>::pack(part);
  }
  const unsigned char* const mc = static_cast<const unsigned char*>(t.m) + at;
  const unsigned char* const vc = static_cast<const unsigned char*>(t.v) + at;
  r.m = r.v = make_uint2(0, 0);
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const uint32_t a = i < n ? mc[i] : 0u, c = i < n ? vc[i] : 0u;
    if (i < 4) {
      r.m.x |= a << (8 * i);
      r.v.x |= c << (8 * i);
    } else {
      r.m.y |= a << (8 * i - 32);
      r.v.y |= c << (8 * i - 32);
    }
  }
}

template <int PD, int GD, bool MASTER>
__device__ __forceinline__ void unpack_packed(const Packed<PD, GD, MASTER>& r, F2 (&p)[W / 2], F2 (&g)[W / 2]) {
  using R = Packed<PD, GD, MASTER>;
  constexpr int H = W / 2, PDT = MASTER ? kDtypeF32 : PD;
#pragma unroll
  for (int i = 0; i < R::PV; ++i) {
    F2 part[H / R::PV];
    unpack2<PDT, W / R::PV>(r.p[i], part);
#pragma unroll
    for (int j = 0; j < H / R::PV; ++j) p[i * (H / R::PV) + j] = part[j];
  }
#pragma unroll
  for (int i = 0; i < R::GV; ++i) {
    F2 part[H / R::GV];
    unpack2<GD, W / R::GV>(r.g[i], part);
#pragma unroll
    for (int j = 0; j < H / R::GV; ++j) g[i * (H / R::GV) + j] = part[j];
  }
}

// n of the lane's elements (W where WHOLE) and their codes.
template <int PD, int GD, bool MASTER, bool WHOLE>
__device__ __forceinline__ void store_packed(const AdamTensor& t, long long block, int n, const F2 (&p)[W / 2], uint2 m8,
                                             uint2 v8) {
  using P = typename Elem<PD>::T;
  const long long at = block * kAdamBlock + (threadIdx.x & 31) * W;
  P* const out = static_cast<P*>(t.p) + at;
  unsigned char* const mc = static_cast<unsigned char*>(t.m) + at;
  unsigned char* const vc = static_cast<unsigned char*>(t.v) + at;
  float pv[W];
#pragma unroll
  for (int i = 0; i < W / 2; ++i) pv[2 * i] = p[i].x, pv[2 * i + 1] = p[i].y;
  if (WHOLE) {
    *reinterpret_cast<uint2*>(mc) = m8;
    *reinterpret_cast<uint2*>(vc) = v8;
    if (MASTER) store_wide<kDtypeF32, W>(t.master + at, pv);
    store_wide<PD, W>(out, pv);
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if (i < n) {
        mc[i] = static_cast<unsigned char>((i < 4 ? m8.x : m8.y) >> (8 * (i & 3)));
        vc[i] = static_cast<unsigned char>((i < 4 ? v8.x : v8.y) >> (8 * (i & 3)));
      }
    }
    if (MASTER) store_few<kDtypeF32, W>(t.master + at, n, pv);
    store_few<PD, W>(out, n, pv);
  }
}
__device__ __forceinline__ void store_scales(const AdamTensor& t, long long block, float ms, float us) {
  if ((threadIdx.x & 31) == 0) {
    t.m_scale[block] = ms;
    t.v_scale[block] = us;
  }
}

// The block's largest of non-negative values; NaN, whose bits are above infinity's, wins.
__device__ __forceinline__ float warp_top(float v) { return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v))); }

// a b + c d, each operation rounded by itself.  The sums are scalar: a packed product and a packed sum were
// contracted into one operation, with the instructions' explicit rounding too (seen in the results).
__device__ __forceinline__ F2 sum_of_products(F2 a, F2 b, F2 c, F2 d) {
  const F2 u = mul2(a, b), v = mul2(c, d);
  return f2(__fadd_rn(u.x, v.x), __fadd_rn(u.y, v.y));
}
__device__ __forceinline__ F2 first_moment(const Step& s, F2 code, float scale, F2 g) {
  return sum_of_products(mul2(code, f2(scale)), f2(s.b1), g, f2(s.c1));
}
__device__ __forceinline__ F2 second_moment(const Step& s, F2 code, float scale, F2 g) {
  const F2 root = mul2(code, f2(scale));
  return sum_of_products(mul2(root, root), f2(s.b2), mul2(g, g), f2(s.c2));
}

// A block's step for any values, each operation rounded by itself: a stored code then is what the
// definition in fp32 gives, which a value next to the border between two codes would otherwise miss by
// an eighth.  The warp's lanes share the two maxima; all of them must come here.
template <int PD, int GD, bool MASTER, bool WHOLE>
__device__ __forceinline__ void step_any(const AdamTensor& t, const Step& s, float decay, long long block, int n,
                                         const Packed<PD, GD, MASTER>& r) {
  constexpr int H = W / 2;
  F2 p[H], m[H], u[H];
  unpack_packed(r, p, u);
  float mt = 0.f, ut = 0.f;  // largest |m| and root of v
#pragma unroll
  for (int i = 0; i < H; ++i) {
    const F2 g = mul2(u[i], f2(s.scale));
    const F2 v = second_moment(s, codes_to_f2(i < 2 ? r.v.x : r.v.y, i & 1), r.vs, g);
    m[i] = first_moment(s, codes_to_f2(i < 2 ? r.m.x : r.m.y, i & 1), r.ms, g);
    u[i] = f2(sqrtf(v.x), sqrtf(v.y));
    const F2 d = fma2(u[i], f2(s.root_v), f2(s.eps));
    p[i] = moved(p[i], decay, mul2(f2(__fdiv_rn(m[i].x, d.x), __fdiv_rn(m[i].y, d.y)), f2(-s.rate_m)));
    mt = nan_max(mt, nan_max(fabsf(m[i].x), fabsf(m[i].y)));
    ut = nan_max(ut, nan_max(u[i].x, u[i].y));
  }
  const float ms = warp_top(mt) * (1.f / kTop8), us = warp_top(ut) * (1.f / kTop8);
  const float m_by = ms != 0.f ? ms : 1.f, u_by = us != 0.f ? us : 1.f;
#pragma unroll
  for (int i = 0; i < H; ++i) {
    m[i] = f2(__fdiv_rn(m[i].x, m_by), __fdiv_rn(m[i].y, m_by));
    u[i] = f2(__fdiv_rn(u[i].x, u_by), __fdiv_rn(u[i].y, u_by));
    // a root above 0 is not stored as 0
    u[i] = f2(u[i].x > 0.f ? fmaxf(u[i].x, kLeast8) : u[i].x, u[i].y > 0.f ? fmaxf(u[i].y, kLeast8) : u[i].y);
  }
  store_packed<PD, GD, MASTER, WHOLE>(t, block, n, p, all_codes(m), all_codes(u));
  store_scales(t, block, ms, us);
}

// The same of a whole block whose values lie in the middle of fp32's range and whose roots are all above 0,
// in fewer instructions: roots and reciprocals come from the instructions that are within 2^-23 and flush
// subnormals to 0, and values are multiplied by a reciprocal of the scale.  All in all a quotient is
// within 13 2^-24 of the exactly rounded one; where 2^-19 to either side would give another code, the
// block is left to step_any (about one in a hundred).  The new scales are the caller's to store.  False,
// and nothing written, where this form will not do.
template <int PD, int GD, bool MASTER, bool WHOLE>
__device__ __forceinline__ bool step_usual(const AdamTensor& t, const Step& s, float decay, long long block,
                                           const Packed<PD, GD, MASTER>& r, float& ms, float& us) {
  constexpr int H = W / 2;
  constexpr float kLow = 1e-15f, kHigh = 1e15f, kMargin = 1.f / 524288.f;
  if (!(r.vs > kLow && r.vs < kHigh && r.ms < kHigh)) return false;  // the same in all lanes
  F2 p[H], m[H], u[H];
  unpack_packed(r, p, u);
  float mt = 0.f, vt = 0.f, pt = 0.f, least = kHigh;
#pragma unroll
  for (int i = 0; i < H; ++i) {
    const F2 g = mul2(u[i], f2(s.scale));
    const F2 v = second_moment(s, codes_to_f2(i < 2 ? r.v.x : r.v.y, i & 1), r.vs, g);
    m[i] = first_moment(s, codes_to_f2(i < 2 ? r.m.x : r.m.y, i & 1), r.ms, g);
    vt = nan_max3_abs(vt, v.x, v.y);
    least = min3(least, v.x, v.y);
    mt = nan_max3_abs(mt, m[i].x, m[i].y);
    u[i] = f2(root_ftz(v.x), root_ftz(v.y));
    const F2 d = fma2(u[i], f2(s.root_v), f2(s.eps));
    pt = nan_max3_abs(pt, p[i].x, p[i].y);
    const F2 update = mul2(mul2(m[i], f2(inverse_ftz(d.x), inverse_ftz(d.y))), f2(-s.rate_m));
    p[i] = add2(p[i], fma2(p[i], f2(-decay), update));
  }
  mt = warp_top(mt);
  vt = warp_top(vt);
  bool fine = least > 1e-36f && mt > 1e-25f && mt < kHigh && vt < kHigh * kHigh && pt < kHigh;  // no: a NaN too
  const float ut = __fsqrt_rn(vt);  // the largest root
  ms = mt * (1.f / kTop8);
  us = ut * (1.f / kTop8);
  const float m_inv = kTop8 * inverse_ftz(mt), u_inv = kTop8 * inverse_ftz(ut);
  const F2 m_lo = f2(m_inv * (1.f - kMargin)), m_hi = f2(m_inv * (1.f + kMargin));
  const F2 u_lo = f2(u_inv * (1.f - kMargin)), u_hi = f2(u_inv * (1.f + kMargin));
  uint2 m8 = make_uint2(0, 0), v8 = make_uint2(0, 0);
  uint32_t differ = 0;
#pragma unroll
  for (int i = 0; i < H; ++i) {
    const uint32_t a = f2_to_codes(mul2(m[i], m_lo)), b = f2_to_codes(mul2(m[i], m_hi));
    const F2 x = mul2(u[i], u_lo), y = mul2(u[i], u_hi);
    const uint32_t c = f2_to_codes(f2(fmaxf(x.x, kLeast8), fmaxf(x.y, kLeast8)));
    const uint32_t d = f2_to_codes(f2(fmaxf(y.x, kLeast8), fmaxf(y.y, kLeast8)));
    differ |= (a ^ b) | (c ^ d);
    (i < 2 ? m8.x : m8.y) |= a << (16 * (i & 1));
    (i < 2 ? v8.x : v8.y) |= c << (16 * (i & 1));
  }
  fine = fine && differ == 0;
  if (!__all_sync(0xffffffffu, fine)) return false;
  store_packed<PD, GD, MASTER, WHOLE>(t, block, W, p, m8, v8);
  return true;
}

// What step_usual left of a warp's blocks of a chunk (bit i of `done`: the i-th is not), those off the
// vectors' boundaries and the tensor's last.  A call, so that its registers are not the whole blocks'.
template <int PD, int GD, bool MASTER>
__device__ __noinline__ void packed_rest(const AdamTensor& t, const Step* shared, long long mine, long long end,
                                         long long stop, unsigned done) {
  const Step s = *shared;
  const float decay = s.rate * t.decay;
  Packed<PD, GD, MASTER> r;
#pragma unroll 1
  for (int i = 0; i < kWarpBlocks && mine + i < end; ++i) {
    const long long b = mine + i;
    if (done >> i & 1) continue;
    if (b < stop) {
      load_packed(t, b, r);
      step_any<PD, GD, MASTER, true>(t, s, decay, b, W, r);
    } else {
      const long long left = t.n - (b * kAdamBlock + (threadIdx.x & 31) * W);
      const int n = left < W ? (left > 0 ? static_cast<int>(left) : 0) : W;
      load_packed_few(t, b, n, r);
      // wherever a block lies, the same steps give the same bits
      float ms, us;
      if ((b + 1) * kAdamBlock <= t.n && step_usual<PD, GD, MASTER, false>(t, s, decay, b, r, ms, us))
        store_scales(t, b, ms, us);
      else
        step_any<PD, GD, MASTER, false>(t, s, decay, b, n, r);
    }
  }
}

// 8-bit states: each warp of the CTA takes kWarpBlocks neighbouring blocks of the chunk, two at a time.  Their
// scales, a 32-byte sector of each array, are read and written at once: four bytes at a time the writes
// alone cost a sixth of the time.  Lane i holds the i-th block's scale of m, lane 16 + i that of the root.
template <int PD, int GD, bool MASTER>
__device__ __forceinline__ void packed_chunk(const AdamTensor& t, const Step* shared, int chunk) {
  using Ring = Slot8<PD, GD, MASTER>;
  extern __shared__ uint4 adam_ring[];
  Ring* const ring = reinterpret_cast<Ring*>(reinterpret_cast<unsigned char*>(adam_ring) + (threadIdx.x >> 5) * kWarpRing);
  constexpr int kAhead = kWarpRing / sizeof(Ring);
  static_assert(kAhead >= 2 && sizeof(Ring) % 16 == 0 && kWarpRing % 16 == 0, "slots of the ring");
  const int lane = threadIdx.x & 31;
  const long long blocks = (t.n + kAdamBlock - 1) / kAdamBlock;
  const long long mine = static_cast<long long>(chunk) * (kAdamPackedChunk / kAdamBlock) + (threadIdx.x >> 5) * kWarpBlocks;
  const long long end = mine + kWarpBlocks < blocks ? mine + kWarpBlocks : blocks;
  const long long whole = t.head < 0 ? 0 : t.n / kAdamBlock;  // blocks that come in whole vectors
  const long long stop = end < whole ? end : whole;
  if (mine >= end) return;
  unsigned done = 0;
  if (mine < stop) {
    const Step s = *shared;
    const float decay = s.rate * t.decay;
    const int count = static_cast<int>(stop - mine);
#pragma unroll
    for (int i = 0; i < kAhead - 1; ++i) {
      if (2 * i < count) copy_pair<PD, GD, MASTER>(t, mine + 2 * i, stop, ring + i);
      copy_commit();
    }
    const int j = lane & 15;
    float* const scale_at = (lane < 16 ? t.m_scale : t.v_scale) + mine + j;
    float scales = j < count ? *scale_at : 0.f;
    int slot = 0;
#pragma unroll 1
    for (int i = 0; i < count; i += 2) {
      // lanes read what others copied: all of them are past the last reading of the slot, and through with
      // their copies, before any goes on
      __syncwarp();
      if (i + 2 * (kAhead - 1) < count)
        copy_pair<PD, GD, MASTER>(t, mine + i + 2 * (kAhead - 1), stop, ring + (slot == 0 ? kAhead - 1 : slot - 1));
      copy_commit();
      copy_wait<kAhead - 1>();
      __syncwarp();
#pragma unroll 1
      for (int k = i; k < i + 2 && k < count; ++k) {
        Packed<PD, GD, MASTER> r;
        read_packed(ring + slot, k - i, r);
        r.ms = __shfl_sync(0xffffffffu, scales, k);
        r.vs = __shfl_sync(0xffffffffu, scales, 16 + k);
        float ms, us;
        if (step_usual<PD, GD, MASTER, true>(t, s, decay, mine + k, r, ms, us)) {
          done |= 1u << k;
          if (j == k) scales = lane < 16 ? ms : us;
        }
      }
      slot = slot + 1 == kAhead ? 0 : slot + 1;
    }
    copy_wait<0>();
    __syncwarp();  // before the next chunk's copies
    if (done >> j & 1) *scale_at = scales;
  }
  if (done != (1u << (end - mine)) - 1) packed_rest<PD, GD, MASTER>(t, shared, mine, end, stop, done);
}
template <int PD, int GD>
__device__ __forceinline__ void block_chunk(const AdamTensor& t, const Step* shared, int chunk) {
  if (t.master != nullptr)
    packed_chunk<PD, GD, true>(t, shared, chunk);
  else
    packed_chunk<PD, GD, false>(t, shared, chunk);
}

template <int PD, int GD, int BITS>
__device__ __forceinline__ void chunk_of(const AdamTensor& t, const Step* shared, int chunk) {
  if constexpr (BITS == 8)
    block_chunk<PD, GD>(t, shared, chunk);
  else
    plain_chunk<PD, GD>(t, shared, chunk);
}

template <int MOST, int BITS>
__global__ void __launch_bounds__(BITS == 8 ? kPackedThreads : kAdamThreads, kAdamResident<BITS>)
    adamw_kernel(const __grid_constant__ AdamTable<MOST> table) {
  __shared__ Step shared;
  if (threadIdx.x == 0) shared = read_step(table.k);
  __syncthreads();
  for (int c = blockIdx.x; c < table.chunks; c += gridDim.x) {
    int lo = 0, hi = table.count;  // the last tensor whose first chunk is not past c
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (table.t[mid].first_chunk <= c) lo = mid;
      else hi = mid;
    }
    const AdamTensor& t = table.t[lo];
    const int chunk = c - t.first_chunk;
    if (t.param_dtype == kDtypeF32) chunk_of<kDtypeF32, kDtypeF32, BITS>(t, &shared, chunk);
    else if (t.param_dtype == kDtypeBF16) {
      if (t.grad_dtype == kDtypeBF16) chunk_of<kDtypeBF16, kDtypeBF16, BITS>(t, &shared, chunk);
      else chunk_of<kDtypeBF16, kDtypeF32, BITS>(t, &shared, chunk);
    } else {
      if (t.grad_dtype == kDtypeF16) chunk_of<kDtypeF16, kDtypeF16, BITS>(t, &shared, chunk);
      else chunk_of<kDtypeF16, kDtypeF32, BITS>(t, &shared, chunk);
    }
  }
}

}  // namespace

cudaError_t adamw_setup() {
  const int bytes = kPackedThreads / 32 * kWarpRing;
  cudaError_t e = note_cuda(cudaFuncSetAttribute(adamw_kernel<kAdamFew, 8>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
  if (e == cudaSuccess)
    e = note_cuda(cudaFuncSetAttribute(adamw_kernel<kAdamMany, 8>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
  return e;
}

template <int MOST>
cudaError_t launch_adamw(const AdamTable<MOST>& table, int bits, int num_sms, cudaStream_t s) {
  const int most = (bits == 8 ? kAdamResident<8> : kAdamResident<32>) * num_sms;
  const int blocks = table.chunks < most ? table.chunks : most;
  if (bits == 8)
    adamw_kernel<MOST, 8><<<blocks, kPackedThreads, kPackedThreads / 32 * kWarpRing, s>>>(table);
  else
    adamw_kernel<MOST, 32><<<blocks, kAdamThreads, 0, s>>>(table);
  return launch_result();
}

template cudaError_t launch_adamw<kAdamFew>(const AdamTable<kAdamFew>&, int, int, cudaStream_t);
template cudaError_t launch_adamw<kAdamMany>(const AdamTable<kAdamMany>&, int, int, cudaStream_t);

}  // namespace llp
