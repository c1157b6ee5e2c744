// RMS norms around a block: s = x + scale * gate * norm(branch), h = norm(s), in one launch.
//
// One CTA per row, three passes over it (the second and third from L2).
#include "layer_norm.cuh"
#include "residual_norm.h"

namespace llp {

namespace {

constexpr int kWideThreads = 512;

template <int DT, int PT>
__global__ void __launch_bounds__(kWideThreads) residual_norm_fwd_wide_kernel(ResidualNormParams p, ResidualNormOut o) {
  using E = Elem<DT>;
  using T = typename E::T;
  using P = Elem<PT>;
  using PE = typename P::T;
  __shared__ float sm[kWideThreads / 32];
  const long long n = blockIdx.x;
  const T* const x = static_cast<const T*>(p.x) + n * p.x_stride;
  const T* const b = p.branch == nullptr ? nullptr : static_cast<const T*>(p.branch) + n * p.b_stride;
  const T* const gr = p.gate_kind == kGateRows ? static_cast<const T*>(p.gate) + n * p.gate_stride : nullptr;
  const PE* const gc = p.gate_kind == kGateColumns ? static_cast<const PE*>(p.gate) : nullptr;
  const PE* const pw = static_cast<const PE*>(p.post_weight);
  const PE* const w = static_cast<const PE*>(p.weight);
  const float inv = 1.f / static_cast<float>(p.D);
  float pr = 1.f;
  if (pw != nullptr) {
    float t = 0.f;
#pragma unroll 8
    for (int c = threadIdx.x; c < p.D; c += kWideThreads) {
      const float v = E::get(b[c]);
      t = fmaf(v, v, t);
    }
    pr = rsqrtf(fmaf(cta_sum<kWideThreads>(t, sm), inv, p.eps));
    if (threadIdx.x == 0) o.post_rstd[n] = pr;
  }
  auto stream = [&](int c) {
    float v = E::get(x[c]);
    if (b != nullptr) {
      float m = E::get(b[c]) * pr * p.scale;
      if (pw != nullptr) m *= P::get(__ldg(pw + c));
      if (gc != nullptr) m *= P::get(__ldg(gc + c));
      if (gr != nullptr) m *= E::get(__ldg(gr + c));
      v += m;
    }
    return v;
  };
  T* const s = static_cast<T*>(o.s) + n * p.D;
  T* const h = static_cast<T*>(o.h) + n * p.D;
  if (w == nullptr) {
#pragma unroll 4
    for (int c = threadIdx.x; c < p.D; c += kWideThreads) s[c] = E::put(stream(c));
    return;
  }
  float t = 0.f;
#pragma unroll 4
  for (int c = threadIdx.x; c < p.D; c += kWideThreads) {
    const float v = stream(c);
    t = fmaf(v, v, t);
  }
  const float r = rsqrtf(fmaf(cta_sum<kWideThreads>(t, sm), inv, p.eps));
  if (threadIdx.x == 0) o.rstd[n] = r;
#pragma unroll 4
  for (int c = threadIdx.x; c < p.D; c += kWideThreads) {
    const float v = stream(c);
    if (o.s != nullptr) s[c] = E::put(v);
    h[c] = E::put(v * r * P::get(__ldg(w + c)));
  }
}

template <int DT, int PT>
cudaError_t run(const ResidualNormParams& p, const ResidualNormOut& o, cudaStream_t s) {
  residual_norm_fwd_wide_kernel<DT, PT><<<p.N, kWideThreads, 0, s>>>(p, o);
  return launch_result();
}

}  // namespace

cudaError_t launch_residual_norm_fwd(const ResidualNormParams& p, const ResidualNormOut& o, cudaStream_t s) {
  const bool pf = p.param_dtype == kDtypeF32;
  if (p.dtype == kDtypeF32) return run<kDtypeF32, kDtypeF32>(p, o, s);
  if (p.dtype == kDtypeBF16) return pf ? run<kDtypeBF16, kDtypeF32>(p, o, s) : run<kDtypeBF16, kDtypeBF16>(p, o, s);
  return pf ? run<kDtypeF16, kDtypeF32>(p, o, s) : run<kDtypeF16, kDtypeF16>(p, o, s);
}

}  // namespace llp
