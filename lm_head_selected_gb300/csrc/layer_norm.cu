// Layer norm over the last dimension, and its gradients.
#include "elem.cuh"

namespace llp {

namespace {

constexpr int kThreads = 256;

// Fixed-order block sum: butterflies in the warps, then the warps in ascending order.
__device__ __forceinline__ float block_sum(float v, float* sm) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
  for (int w = 0; w < kThreads / 32; ++w) v += sm[w];
  __syncthreads();
  return v;
}

// One CTA per row, three passes over it.
template <int DT, int PT>
__global__ void __launch_bounds__(kThreads) layer_norm_fwd_kernel(LayerNormParams p,
                                                                  typename Elem<DT>::T* __restrict__ y,
                                                                  float* __restrict__ mean_out,
                                                                  float* __restrict__ rstd_out) {
  using E = Elem<DT>;
  using P = Elem<PT>;
  __shared__ float sm[kThreads / 32];
  const long long n = blockIdx.x;
  const typename E::T* x = static_cast<const typename E::T*>(p.x) + n * p.x_stride;
  const typename P::T* w = static_cast<const typename P::T*>(p.weight);
  const typename P::T* b = static_cast<const typename P::T*>(p.bias);
  float s = 0.f;
  for (int c = threadIdx.x; c < p.D; c += kThreads) s += E::get(x[c]);
  const float mean = block_sum(s, sm) / static_cast<float>(p.D);
  s = 0.f;
  for (int c = threadIdx.x; c < p.D; c += kThreads) {
    const float d = E::get(x[c]) - mean;
    s = fmaf(d, d, s);
  }
  const float rstd = 1.f / sqrtf(block_sum(s, sm) / static_cast<float>(p.D) + p.eps);
  for (int c = threadIdx.x; c < p.D; c += kThreads) {
    const float h = (E::get(x[c]) - mean) * rstd;
    y[n * p.D + c] = E::put(fmaf(h, w ? P::get(w[c]) : 1.f, b ? P::get(b[c]) : 0.f));
  }
  if (threadIdx.x == 0) {
    mean_out[n] = mean;
    rstd_out[n] = rstd;
  }
}

// One CTA per row.
template <int DT, int PT>
__global__ void __launch_bounds__(kThreads) layer_norm_bwd_x_kernel(LayerNormParams p, const float* __restrict__ mean,
                                                                    const float* __restrict__ rstd,
                                                                    typename Elem<DT>::T* __restrict__ gx) {
  using E = Elem<DT>;
  using P = Elem<PT>;
  __shared__ float sm[kThreads / 32];
  const long long n = blockIdx.x;
  const typename E::T* x = static_cast<const typename E::T*>(p.x) + n * p.x_stride;
  const typename E::T* g = static_cast<const typename E::T*>(p.gy) + n * p.gy_stride;
  const typename P::T* w = static_cast<const typename P::T*>(p.weight);
  const float m = mean[n], r = rstd[n];
  float s1 = 0.f, s2 = 0.f;
  for (int c = threadIdx.x; c < p.D; c += kThreads) {
    const float a = E::get(g[c]) * (w ? P::get(w[c]) : 1.f);
    s1 += a;
    s2 = fmaf(a, (E::get(x[c]) - m) * r, s2);
  }
  s1 = block_sum(s1, sm) / static_cast<float>(p.D);
  s2 = block_sum(s2, sm) / static_cast<float>(p.D);
  for (int c = threadIdx.x; c < p.D; c += kThreads) {
    const float a = E::get(g[c]) * (w ? P::get(w[c]) : 1.f);
    gx[n * p.D + c] = E::put((a - s1 - (E::get(x[c]) - m) * r * s2) * r);
  }
}

// One thread per column, rows in ascending order in blocks of 256.
template <int DT, int PT>
__global__ void __launch_bounds__(kThreads) layer_norm_bwd_params_kernel(LayerNormParams p,
                                                                         const float* __restrict__ mean,
                                                                         const float* __restrict__ rstd,
                                                                         typename Elem<PT>::T* __restrict__ gw,
                                                                         typename Elem<PT>::T* __restrict__ gb) {
  using E = Elem<DT>;
  using P = Elem<PT>;
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= p.D) return;
  const typename E::T* x = static_cast<const typename E::T*>(p.x) + c;
  const typename E::T* g = static_cast<const typename E::T*>(p.gy) + c;
  float sw = 0.f, sb = 0.f;
  for (int n0 = 0; n0 < p.N; n0 += 256) {
    float tw = 0.f, tb = 0.f;
    for (int n = n0; n < p.N && n < n0 + 256; ++n) {
      const float gv = E::get(g[n * p.gy_stride]);
      tb += gv;
      tw = fmaf(gv, (E::get(x[n * p.x_stride]) - mean[n]) * rstd[n], tw);
    }
    sw += tw;
    sb += tb;
  }
  if (gw) gw[c] = P::put(sw);
  if (gb) gb[c] = P::put(sb);
}

template <int DT, int PT>
cudaError_t fwd(const LayerNormParams& p, void* y, float* mean, float* rstd, cudaStream_t s) {
  layer_norm_fwd_kernel<DT, PT><<<p.N, kThreads, 0, s>>>(p, static_cast<typename Elem<DT>::T*>(y), mean, rstd);
  return launch_result();
}

template <int DT, int PT>
cudaError_t bwd(const LayerNormParams& p, const float* mean, const float* rstd, void* gx, void* gw, void* gb,
                cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (gx != nullptr) {
    layer_norm_bwd_x_kernel<DT, PT><<<p.N, kThreads, 0, s>>>(p, mean, rstd, static_cast<typename Elem<DT>::T*>(gx));
    e = launch_result();
  }
  if (e == cudaSuccess && (gw != nullptr || gb != nullptr)) {
    layer_norm_bwd_params_kernel<DT, PT><<<(p.D + kThreads - 1) / kThreads, kThreads, 0, s>>>(
        p, mean, rstd, static_cast<typename Elem<PT>::T*>(gw), static_cast<typename Elem<PT>::T*>(gb));
    e = launch_result();
  }
  return e;
}

}  // namespace

size_t layer_norm_bwd_workspace(long long, long long) { return 256; }

cudaError_t launch_layer_norm_fwd(const LayerNormParams& p, void* y, float* mean, float* rstd, cudaStream_t s) {
  const bool pf = p.param_dtype == kDtypeF32;
  if (p.dtype == kDtypeF32) return fwd<kDtypeF32, kDtypeF32>(p, y, mean, rstd, s);
  if (p.dtype == kDtypeBF16)
    return pf ? fwd<kDtypeBF16, kDtypeF32>(p, y, mean, rstd, s) : fwd<kDtypeBF16, kDtypeBF16>(p, y, mean, rstd, s);
  return pf ? fwd<kDtypeF16, kDtypeF32>(p, y, mean, rstd, s) : fwd<kDtypeF16, kDtypeF16>(p, y, mean, rstd, s);
}

cudaError_t launch_layer_norm_bwd(const LayerNormParams& p, const float* mean, const float* rstd, void* gx, void* gw,
                                  void* gb, void* workspace, int num_sms, cudaStream_t s) {
  (void)workspace;
  (void)num_sms;
  const bool pf = p.param_dtype == kDtypeF32;
  if (p.dtype == kDtypeF32) return bwd<kDtypeF32, kDtypeF32>(p, mean, rstd, gx, gw, gb, s);
  if (p.dtype == kDtypeBF16)
    return pf ? bwd<kDtypeBF16, kDtypeF32>(p, mean, rstd, gx, gw, gb, s)
              : bwd<kDtypeBF16, kDtypeBF16>(p, mean, rstd, gx, gw, gb, s);
  return pf ? bwd<kDtypeF16, kDtypeF32>(p, mean, rstd, gx, gw, gb, s)
            : bwd<kDtypeF16, kDtypeF16>(p, mean, rstd, gx, gw, gb, s);
}

}  // namespace llp
