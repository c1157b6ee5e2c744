// Gradients of layer norm.  With h = (x - mean) * rstd and a = grad_y * weight,
//
//   grad_x      = rstd * (a - sum a / D - h * (sum a h) / D)
//   grad_weight = sum over rows of grad_y * h,   grad_bias = sum over rows of grad_y
//
// One pass over grad_y and x gives all three: LANES threads own a row at a time,
// hold it in registers while the two row sums are joined, and write grad_x; the
// columns a thread owns are the same for every row, so it keeps their share of
// the two column sums in registers too.  The next row's loads are in flight
// meanwhile.  The grid is fixed by the sizes; every group of LANES threads takes
// the rows group, group + groups, ...; a second launch joins the CTAs' column
// sums in ascending order.  Rows beyond the register layouts take three kernels.
#include "layer_norm.cuh"

namespace llp {

namespace {

constexpr int kMaxParts = 608;  // partial column sums: CTAs of the row pass (4 per SM)

// part: [gridDim.x][2][D], the CTA's column sums of grad_y * h and of grad_y; null to skip them.
template <int DT, int PT, int W, int LANES, int K>
__global__ void __launch_bounds__(LANES < 256 ? 256 : LANES) layer_norm_bwd_kernel(
    LayerNormParams p, bool al, const float* __restrict__ mean, const float* __restrict__ rstd,
    typename Elem<DT>::T* __restrict__ gx, float* __restrict__ part) {
  using U = RowUnit<DT, W>;
  using P = RowUnit<PT, W>;
  constexpr int THREADS = LANES < 256 ? 256 : LANES;
  constexpr int GROUPS = THREADS / LANES;
  __shared__ float sm[2][GROUPS * (LANES / 32) * 2];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int group = threadIdx.x / LANES, lane = threadIdx.x % LANES;
  const int units = p.D / W;
  const typename U::T* xb = static_cast<const typename U::T*>(p.x);
  const typename U::T* gb = static_cast<const typename U::T*>(p.gy);
  const typename P::T* wb = static_cast<const typename P::T*>(p.weight);
  const long long step = static_cast<long long>(gridDim.x) * GROUPS;
  const float inv = 1.f / static_cast<float>(p.D);

  float wv[K][W], aw[K][W], ab[K][W];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int u = lane + k * LANES;
#pragma unroll
    for (int i = 0; i < W; ++i) wv[k][i] = 1.f, aw[k][i] = ab[k][i] = 0.f;
    if (wb != nullptr && u < units) P::load(wb + u * W, al, wv[k]);
  }
  typename U::Raw xr[K], gr[K];
  float m = 0.f, r = 0.f;
  auto fetch = [&](long long n) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int u = lane + k * LANES;
      const bool on = n < p.N && u < units;
      gr[k] = on ? U::load_raw(gb + n * p.gy_stride + static_cast<size_t>(u) * W, al) : U::zero();
      xr[k] = on ? U::load_raw(xb + n * p.x_stride + static_cast<size_t>(u) * W, al) : U::zero();
    }
    if (n < p.N) m = __ldg(mean + n), r = __ldg(rstd + n);
  };
  long long n = static_cast<long long>(blockIdx.x) * GROUPS + group;
  fetch(n);
  for (int odd = 0; n < p.N; n += step, odd ^= 1) {
    typename U::Raw xc[K], gc[K];
    const float mc = m, rc = r;
#pragma unroll
    for (int k = 0; k < K; ++k) xc[k] = xr[k], gc[k] = gr[k];
    fetch(n + step);
    float s[2] = {0.f, 0.f};
    float h[K][W], a[K][W];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const bool on = lane + k * LANES < units;
      U::unpack(xc[k], h[k]);
      U::unpack(gc[k], a[k]);
#pragma unroll
      for (int i = 0; i < W; ++i) {
        h[k][i] = on ? (h[k][i] - mc) * rc : 0.f;
        aw[k][i] = fmaf(a[k][i], h[k][i], aw[k][i]);
        ab[k][i] += a[k][i];
        a[k][i] *= wv[k][i];
        s[0] += a[k][i];
        s[1] = fmaf(a[k][i], h[k][i], s[1]);
      }
    }
    row_sum<LANES, 2>(s, sm[odd] + group * (LANES / 32) * 2, 1 + group);
    if (gx != nullptr) {
      const float s0 = s[0] * inv, s1 = s[1] * inv;
      typename U::T* out = gx + static_cast<size_t>(n) * p.D;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int u = lane + k * LANES;
        if (u < units) {
#pragma unroll
          for (int i = 0; i < W; ++i) a[k][i] = (fmaf(-h[k][i], s1, a[k][i]) - s0) * rc;
          U::store(out + static_cast<size_t>(u) * W, al, a[k]);
        }
      }
    }
  }
  if (part == nullptr) return;
  if constexpr (GROUPS > 1) {  // the CTA's groups in ascending order
    __shared__ float join[2 * LANES * K * W];
    for (int g = 1; g < GROUPS; ++g) {
      __syncthreads();
      if (group == g) {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int i = 0; i < W; ++i) {
            join[(k * W + i) * LANES + lane] = aw[k][i];
            join[((K + k) * W + i) * LANES + lane] = ab[k][i];
          }
      }
      __syncthreads();
      if (group == 0) {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int i = 0; i < W; ++i) {
            aw[k][i] += join[(k * W + i) * LANES + lane];
            ab[k][i] += join[((K + k) * W + i) * LANES + lane];
          }
      }
    }
    if (group != 0) return;
  }
  float* pw = part + static_cast<size_t>(blockIdx.x) * 2 * p.D;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int u = lane + k * LANES;
    if (u < units) {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        pw[static_cast<size_t>(u) * W + i] = aw[k][i];
        pw[p.D + static_cast<size_t>(u) * W + i] = ab[k][i];
      }
    }
  }
}

// 32 of the 2 D column sums per CTA; warp w adds the parts w, w + 8, ..., then the warps
// are joined in ascending order.
template <int PT>
__global__ void __launch_bounds__(256) layer_norm_join_kernel(const float* __restrict__ part, int parts, int D,
                                                              typename Elem<PT>::T* __restrict__ gw,
                                                              typename Elem<PT>::T* __restrict__ gb) {
  __shared__ float sm[8][32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < 2 * D) {
#pragma unroll 8
    for (int i = warp; i < parts; i += 8) s += __ldcg(part + static_cast<size_t>(i) * 2 * D + c);
  }
  sm[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || c >= 2 * D) return;
  s = sm[0][lane];
#pragma unroll
  for (int w = 1; w < 8; ++w) s += sm[w][lane];
  if (c < D) {
    if (gw != nullptr) gw[c] = Elem<PT>::put(s);
  } else {
    if (gb != nullptr) gb[c - D] = Elem<PT>::put(s);
  }
}

// ---------------------------------------------------------------- wide rows

constexpr int kWideThreads = 512;

template <int DT, int PT>
__global__ void __launch_bounds__(kWideThreads) layer_norm_bwd_wide_x_kernel(LayerNormParams p,
                                                                             const float* __restrict__ mean,
                                                                             const float* __restrict__ rstd,
                                                                             typename Elem<DT>::T* __restrict__ gx) {
  using E = Elem<DT>;
  using P = Elem<PT>;
  __shared__ float sm[kWideThreads / 32];
  const long long n = blockIdx.x;
  const typename E::T* x = static_cast<const typename E::T*>(p.x) + n * p.x_stride;
  const typename E::T* g = static_cast<const typename E::T*>(p.gy) + n * p.gy_stride;
  const typename P::T* w = static_cast<const typename P::T*>(p.weight);
  const float m = mean[n], r = rstd[n], inv = 1.f / static_cast<float>(p.D);
  float s0 = 0.f, s1 = 0.f;
#pragma unroll 4
  for (int c = threadIdx.x; c < p.D; c += kWideThreads) {
    const float a = E::get(__ldg(g + c)) * (w != nullptr ? P::get(__ldg(w + c)) : 1.f);
    s0 += a;
    s1 = fmaf(a, (E::get(__ldg(x + c)) - m) * r, s1);
  }
  s0 = cta_sum<kWideThreads>(s0, sm) * inv;
  s1 = cta_sum<kWideThreads>(s1, sm) * inv;
#pragma unroll 4
  for (int c = threadIdx.x; c < p.D; c += kWideThreads) {
    const float a = E::get(__ldg(g + c)) * (w != nullptr ? P::get(__ldg(w + c)) : 1.f);
    const float h = (E::get(__ldg(x + c)) - m) * r;
    gx[static_cast<size_t>(n) * p.D + c] = E::put((fmaf(-h, s1, a) - s0) * r);
  }
}

// One thread per column; blockIdx.y takes the rows y, y + gridDim.y, ...
template <int DT>
__global__ void __launch_bounds__(256) layer_norm_bwd_wide_params_kernel(LayerNormParams p,
                                                                         const float* __restrict__ mean,
                                                                         const float* __restrict__ rstd,
                                                                         float* __restrict__ part) {
  using E = Elem<DT>;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= p.D) return;
  const typename E::T* x = static_cast<const typename E::T*>(p.x) + c;
  const typename E::T* g = static_cast<const typename E::T*>(p.gy) + c;
  float sw = 0.f, sb = 0.f;
#pragma unroll 4
  for (long long n = blockIdx.y; n < p.N; n += gridDim.y) {
    const float gv = E::get(__ldg(g + n * p.gy_stride));
    sb += gv;
    sw = fmaf(gv, (E::get(__ldg(x + n * p.x_stride)) - __ldg(mean + n)) * __ldg(rstd + n), sw);
  }
  float* o = part + static_cast<size_t>(blockIdx.y) * 2 * p.D;
  o[c] = sw;
  o[p.D + c] = sb;
}

// ---------------------------------------------------------------- launches

struct Grads {
  const float* mean;
  const float* rstd;
  void* gx;
  void* gw;
  void* gb;
  float* part;
};

template <int PT>
cudaError_t join(const LayerNormParams& p, const Grads& o, int parts, cudaStream_t s) {
  using T = typename Elem<PT>::T;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((2 * p.D + 31) / 32);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return note_cuda(cudaLaunchKernelEx(&cfg, layer_norm_join_kernel<PT>, static_cast<const float*>(o.part), parts, p.D,
                                      static_cast<T*>(o.gw), static_cast<T*>(o.gb)));
}

template <int DT, int PT, int W, int LANES, int K>
cudaError_t rows(const LayerNormParams& p, bool al, const Grads& o, cudaStream_t s) {
  constexpr int THREADS = LANES < 256 ? 256 : LANES;
  constexpr int GROUPS = THREADS / LANES;
  constexpr int PER_SM = THREADS <= 256 ? 4 : THREADS <= 512 ? 2 : 1;
  const bool params = o.gw != nullptr || o.gb != nullptr;
  const long long want = (static_cast<long long>(p.N) + GROUPS - 1) / GROUPS;
  const int grid = static_cast<int>(want < 152 * PER_SM ? want : 152 * PER_SM);
  layer_norm_bwd_kernel<DT, PT, W, LANES, K><<<grid, THREADS, 0, s>>>(
      p, al, o.mean, o.rstd, static_cast<typename Elem<DT>::T*>(o.gx), params ? o.part : nullptr);
  const cudaError_t e = launch_result();
  return e != cudaSuccess || !params ? e : join<PT>(p, o, grid, s);
}

template <int DT, int PT>
cudaError_t wide(const LayerNormParams& p, const Grads& o, cudaStream_t s) {
  if (o.gx != nullptr) {
    layer_norm_bwd_wide_x_kernel<DT, PT><<<p.N, kWideThreads, 0, s>>>(p, o.mean, o.rstd,
                                                                      static_cast<typename Elem<DT>::T*>(o.gx));
    const cudaError_t e = launch_result();
    if (e != cudaSuccess) return e;
  }
  if (o.gw == nullptr && o.gb == nullptr) return cudaSuccess;
  const int parts = p.N < 64 ? 1 : p.N < 1024 ? p.N / 32 : 32;
  layer_norm_bwd_wide_params_kernel<DT><<<dim3((p.D + 255) / 256, parts), 256, 0, s>>>(p, o.mean, o.rstd, o.part);
  const cudaError_t e = launch_result();
  return e != cudaSuccess ? e : join<PT>(p, o, parts, s);
}

template <int DT, int PT>
cudaError_t run(const LayerNormParams& p, const Grads& o, cudaStream_t s) {
  constexpr int W = Elem<DT>::W;
  const bool al = aligned16(p.x) && (p.x_stride * elem_bytes(DT)) % 16 == 0 && aligned16(p.gy) &&
                  (p.gy_stride * elem_bytes(DT)) % 16 == 0 && aligned16(o.gx) && aligned16(p.weight);
  if (p.D % W == 0) {
    const int units = p.D / W;
    if (units <= 32) return rows<DT, PT, W, 32, 1>(p, al, o, s);
    if (units <= 128) return rows<DT, PT, W, 128, 1>(p, al, o, s);
    if (units <= 256) return rows<DT, PT, W, 256, 1>(p, al, o, s);
    if (units <= 384) return rows<DT, PT, W, 384, 1>(p, al, o, s);
    if (units <= 512) return rows<DT, PT, W, 512, 1>(p, al, o, s);
    if (units <= 768) return rows<DT, PT, W, 384, 2>(p, al, o, s);
    if (units <= 1024) return rows<DT, PT, W, 512, 2>(p, al, o, s);
    if (units <= 2048) return rows<DT, PT, W, 1024, 2>(p, al, o, s);
  } else {
    if (p.D <= 256) return rows<DT, PT, 1, 32, 8>(p, al, o, s);
    if (p.D <= 1024) return rows<DT, PT, 1, 256, 4>(p, al, o, s);
    if (p.D <= 4096) return rows<DT, PT, 1, 512, 8>(p, al, o, s);
  }
  return wide<DT, PT>(p, o, s);
}

}  // namespace

size_t layer_norm_bwd_workspace(long long N, long long D) {
  const long long parts = N < kMaxParts ? N : kMaxParts;
  return static_cast<size_t>(parts) * 2 * D * sizeof(float);
}

cudaError_t launch_layer_norm_bwd(const LayerNormParams& p, const float* mean, const float* rstd, void* gx, void* gw,
                                  void* gb, void* workspace, cudaStream_t s) {
  const Grads o = {mean, rstd, gx, gw, gb, static_cast<float*>(workspace)};
  const bool pf = p.param_dtype == kDtypeF32;
  if (p.dtype == kDtypeF32) return run<kDtypeF32, kDtypeF32>(p, o, s);
  if (p.dtype == kDtypeBF16) return pf ? run<kDtypeBF16, kDtypeF32>(p, o, s) : run<kDtypeBF16, kDtypeBF16>(p, o, s);
  return pf ? run<kDtypeF16, kDtypeF32>(p, o, s) : run<kDtypeF16, kDtypeF16>(p, o, s);
}

}  // namespace llp
