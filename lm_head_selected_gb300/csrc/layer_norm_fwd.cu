// Layer norm over the last dimension: y = (x - mean) * rstd * weight + bias.
//
// A row is read once and stays in the registers of the LANES threads that own it
// while its mean and then its centred second moment are summed: two reductions,
// no cancellation, one pass over memory.  Rows beyond 4096 units are read three
// times by one CTA each (from L2 after the first).
#include "layer_norm.cuh"

namespace llp {

namespace {

template <int DT, int PT, int W, int LANES, int K>
__global__ void __launch_bounds__(LANES < 128 ? 128 : LANES) layer_norm_fwd_kernel(
    LayerNormParams p, bool al, typename Elem<DT>::T* __restrict__ y, float* __restrict__ mean_out,
    float* __restrict__ rstd_out) {
  using U = RowUnit<DT, W>;
  using P = RowUnit<PT, W>;
  constexpr int ROWS = LANES < 128 ? 128 / LANES : 1;
  __shared__ float sm[2][ROWS * (LANES < 32 ? 1 : LANES / 32)];
  const int group = threadIdx.x / LANES, lane = threadIdx.x % LANES;
  const long long n = static_cast<long long>(blockIdx.x) * ROWS + group;
  const bool live = n < p.N;
  if (LANES > 32 && !live) return;  // the row's own barrier is not needed then
  const typename U::T* x = static_cast<const typename U::T*>(p.x) + (live ? n : 0) * p.x_stride;
  const int units = p.D / W;
  float* s0 = sm[0] + group * (LANES / 32);
  float* s1 = sm[1] + group * (LANES / 32);
  typename U::Raw raw[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int u = lane + k * LANES;
    raw[k] = u < units ? U::load_raw(x + static_cast<size_t>(u) * W, al) : U::zero();
  }
  float sum[1] = {0.f};
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float v[W];
    U::unpack(raw[k], v);
#pragma unroll
    for (int i = 0; i < W; ++i) sum[0] += v[i];
  }
  row_sum<LANES, 1>(sum, s0, 1 + group);
  const float inv = 1.f / static_cast<float>(p.D);
  const float mean = sum[0] * inv;
  sum[0] = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (lane + k * LANES < units) {
      float v[W];
      U::unpack(raw[k], v);
#pragma unroll
      for (int i = 0; i < W; ++i) sum[0] = fmaf(v[i] - mean, v[i] - mean, sum[0]);
    }
  }
  row_sum<LANES, 1>(sum, s1, 1 + group);
  const float rstd = 1.f / sqrtf(fmaf(sum[0], inv, p.eps));
  if (!live) return;
  typename U::T* out = y + static_cast<size_t>(n) * p.D;
  const typename P::T* w = static_cast<const typename P::T*>(p.weight);
  const typename P::T* b = static_cast<const typename P::T*>(p.bias);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int u = lane + k * LANES;
    if (u < units) {
      float v[W], wv[W], bv[W];
      U::unpack(raw[k], v);
      if (w != nullptr) P::load(w + u * W, al, wv);
      if (b != nullptr) P::load(b + u * W, al, bv);
#pragma unroll
      for (int i = 0; i < W; ++i) {
        float h = (v[i] - mean) * rstd;
        if (w != nullptr) h *= wv[i];
        v[i] = b != nullptr ? h + bv[i] : h;
      }
      U::store(out + static_cast<size_t>(u) * W, al, v);
    }
  }
  if (lane == 0) {
    mean_out[n] = mean;
    rstd_out[n] = rstd;
  }
}

constexpr int kWideThreads = 512;

template <int DT, int PT>
__global__ void __launch_bounds__(kWideThreads) layer_norm_fwd_wide_kernel(LayerNormParams p,
                                                                           typename Elem<DT>::T* __restrict__ y,
                                                                           float* __restrict__ mean_out,
                                                                           float* __restrict__ rstd_out) {
  using E = Elem<DT>;
  using P = Elem<PT>;
  __shared__ float sm[kWideThreads / 32];
  const long long n = blockIdx.x;
  const typename E::T* x = static_cast<const typename E::T*>(p.x) + n * p.x_stride;
  const typename P::T* w = static_cast<const typename P::T*>(p.weight);
  const typename P::T* b = static_cast<const typename P::T*>(p.bias);
  const float inv = 1.f / static_cast<float>(p.D);
  float s = 0.f;
#pragma unroll 8
  for (int c = threadIdx.x; c < p.D; c += kWideThreads) s += E::get(__ldg(x + c));
  const float mean = cta_sum<kWideThreads>(s, sm) * inv;
  s = 0.f;
#pragma unroll 8
  for (int c = threadIdx.x; c < p.D; c += kWideThreads) {
    const float d = E::get(__ldg(x + c)) - mean;
    s = fmaf(d, d, s);
  }
  const float rstd = 1.f / sqrtf(fmaf(cta_sum<kWideThreads>(s, sm), inv, p.eps));
#pragma unroll 4
  for (int c = threadIdx.x; c < p.D; c += kWideThreads) {
    float h = (E::get(__ldg(x + c)) - mean) * rstd;
    if (w != nullptr) h *= P::get(__ldg(w + c));
    y[static_cast<size_t>(n) * p.D + c] = E::put(b != nullptr ? h + P::get(__ldg(b + c)) : h);
  }
  if (threadIdx.x == 0) {
    mean_out[n] = mean;
    rstd_out[n] = rstd;
  }
}

template <int DT, int PT, int W, int LANES, int K>
cudaError_t rows(const LayerNormParams& p, bool al, void* y, float* mean, float* rstd, cudaStream_t s) {
  constexpr int ROWS = LANES < 128 ? 128 / LANES : 1;
  layer_norm_fwd_kernel<DT, PT, W, LANES, K><<<(p.N + ROWS - 1) / ROWS, LANES < 128 ? 128 : LANES, 0, s>>>(
      p, al, static_cast<typename Elem<DT>::T*>(y), mean, rstd);
  return launch_result();
}

template <int DT, int PT>
cudaError_t run(const LayerNormParams& p, void* y, float* mean, float* rstd, cudaStream_t s) {
  constexpr int W = Elem<DT>::W;
  const bool al = aligned16(p.x) && (p.x_stride * elem_bytes(DT)) % 16 == 0 && aligned16(y) && aligned16(p.weight) &&
                  aligned16(p.bias);
  if (p.D % W == 0) {
    const int units = p.D / W;
    if (units <= 8) return rows<DT, PT, W, 8, 1>(p, al, y, mean, rstd, s);
    if (units <= 32) return rows<DT, PT, W, 32, 1>(p, al, y, mean, rstd, s);
    if (units <= 128) return rows<DT, PT, W, 32, 4>(p, al, y, mean, rstd, s);
    if (units <= 384) return rows<DT, PT, W, 128, 3>(p, al, y, mean, rstd, s);
    if (units <= 512) return rows<DT, PT, W, 128, 4>(p, al, y, mean, rstd, s);
    if (units <= 1024) return rows<DT, PT, W, 256, 4>(p, al, y, mean, rstd, s);
    if (units <= 2048) return rows<DT, PT, W, 512, 4>(p, al, y, mean, rstd, s);
    if (units <= 4096) return rows<DT, PT, W, 512, 8>(p, al, y, mean, rstd, s);
  } else {
    if (p.D <= 256) return rows<DT, PT, 1, 32, 8>(p, al, y, mean, rstd, s);
    if (p.D <= 1024) return rows<DT, PT, 1, 128, 8>(p, al, y, mean, rstd, s);
    if (p.D <= 4096) return rows<DT, PT, 1, 256, 16>(p, al, y, mean, rstd, s);
  }
  layer_norm_fwd_wide_kernel<DT, PT><<<p.N, kWideThreads, 0, s>>>(p, static_cast<typename Elem<DT>::T*>(y), mean, rstd);
  return launch_result();
}

}  // namespace

cudaError_t launch_layer_norm_fwd(const LayerNormParams& p, void* y, float* mean, float* rstd, cudaStream_t s) {
  const bool pf = p.param_dtype == kDtypeF32;
  if (p.dtype == kDtypeF32) return run<kDtypeF32, kDtypeF32>(p, y, mean, rstd, s);
  if (p.dtype == kDtypeBF16)
    return pf ? run<kDtypeBF16, kDtypeF32>(p, y, mean, rstd, s) : run<kDtypeBF16, kDtypeBF16>(p, y, mean, rstd, s);
  return pf ? run<kDtypeF16, kDtypeF32>(p, y, mean, rstd, s) : run<kDtypeF16, kDtypeF16>(p, y, mean, rstd, s);
}

}  // namespace llp
