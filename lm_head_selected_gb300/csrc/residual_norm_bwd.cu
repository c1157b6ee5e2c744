// Gradient of the RMS norms around a block.  With c = s * rstd, a = grad_h * weight, k = branch * post_rstd:
//
//   G = grad_s + rstd * (a - c * sum(a c) / D)                    grad_x
//   e = scale * gate * G * post_weight,  grad_branch = post_rstd * (e - k * sum(e k) / D)
//   sums over rows: grad_h * c for the weight, and S = scale * G * k (times the row's own gate), of which
//   the gradients of post_weight and of a gate per column are multiples: gate * S and post_weight * S.
//
// One CTA per row writes the rows' gradients; one thread per column sums the columns over a range of
// rows, and a third launch joins the ranges in ascending order.
#include "layer_norm.cuh"
#include "residual_norm.h"

namespace llp {

namespace {

constexpr int kWideThreads = 512;
constexpr int kParts = kPipeSMs;  // most ranges of rows with column sums of their own

template <int DT, int PT>
struct Row {
  using E = Elem<DT>;
  using T = typename E::T;
  using P = Elem<PT>;
  using PE = typename P::T;
  const T *gs, *gh, *s, *b, *gr;
  const PE *gc, *pw, *w;
  float r, pr, scale;
  __device__ __forceinline__ Row(const ResidualNormParams& p, const ResidualNormGrads& o, long long n) {
    gs = p.gs == nullptr ? nullptr : static_cast<const T*>(p.gs) + n * p.gs_stride;
    w = static_cast<const PE*>(p.weight);
    gh = w == nullptr ? nullptr : static_cast<const T*>(p.gh) + n * p.gh_stride;
    s = w == nullptr ? nullptr : static_cast<const T*>(p.x) + n * p.x_stride;
    b = p.branch == nullptr ? nullptr : static_cast<const T*>(p.branch) + n * p.b_stride;
    gr = p.gate_kind == kGateRows ? static_cast<const T*>(p.gate) + n * p.gate_stride : nullptr;
    gc = p.gate_kind == kGateColumns ? static_cast<const PE*>(p.gate) : nullptr;
    pw = static_cast<const PE*>(p.post_weight);
    r = w == nullptr ? 0.f : o.rstd[n];
    pr = pw == nullptr ? 1.f : o.post_rstd[n];
    scale = p.scale;
  }
  __device__ __forceinline__ float a(int c) const { return E::get(__ldg(gh + c)) * P::get(__ldg(w + c)); }
  __device__ __forceinline__ float cs(int c) const { return E::get(__ldg(s + c)) * r; }
  __device__ __forceinline__ float k(int c) const { return E::get(__ldg(b + c)) * pr; }
  // G, given sum(a c) / D
  __device__ __forceinline__ float G(int c, float mean) const {
    const float up = gs == nullptr ? 0.f : E::get(__ldg(gs + c));
    return w == nullptr ? up : fmaf(r, fmaf(-cs(c), mean, a(c)), up);
  }
  __device__ __forceinline__ float column_gate(int c) const { return gc == nullptr ? 1.f : P::get(__ldg(gc + c)); }
  __device__ __forceinline__ float row_gate(int c) const { return gr == nullptr ? 1.f : E::get(__ldg(gr + c)); }
  __device__ __forceinline__ float post(int c) const { return pw == nullptr ? 1.f : P::get(__ldg(pw + c)); }
};

// means: sum(a c) / D of each row, for the column sums.
template <int DT, int PT>
__global__ void __launch_bounds__(kWideThreads) residual_norm_bwd_wide_x_kernel(ResidualNormParams p,
                                                                                ResidualNormGrads o, float* means) {
  using E = Elem<DT>;
  using T = typename E::T;
  __shared__ float sm[kWideThreads / 32];
  const long long n = blockIdx.x;
  const Row<DT, PT> row(p, o, n);
  const float inv = 1.f / static_cast<float>(p.D);
  float mean = 0.f;
  if (row.w != nullptr) {
    float t = 0.f;
#pragma unroll 4
    for (int c = threadIdx.x; c < p.D; c += kWideThreads) t = fmaf(row.a(c), row.cs(c), t);
    mean = cta_sum<kWideThreads>(t, sm) * inv;
    if (threadIdx.x == 0) means[n] = mean;
  }
  T* const gx = o.gx == nullptr ? nullptr : static_cast<T*>(o.gx) + n * p.D;
  T* const gb = o.gb == nullptr ? nullptr : static_cast<T*>(o.gb) + n * p.D;
  T* const gg = o.ggate != nullptr && p.gate_kind == kGateRows ? static_cast<T*>(o.ggate) + n * p.D : nullptr;
  float t = 0.f;
#pragma unroll 2
  for (int c = threadIdx.x; c < p.D; c += kWideThreads) {
    const float G = row.G(c, mean), u = row.scale * G;
    if (gx != nullptr) gx[c] = E::put(G);
    if (gg != nullptr) gg[c] = E::put(u * row.k(c) * row.post(c));
    if (gb != nullptr) {
      const float e = u * row.column_gate(c) * row.row_gate(c) * row.post(c);
      if (row.pw == nullptr)
        gb[c] = E::put(e);
      else
        t = fmaf(e, row.k(c), t);
    }
  }
  if (gb == nullptr || row.pw == nullptr) return;
  const float along = cta_sum<kWideThreads>(t, sm) * inv;
#pragma unroll 2
  for (int c = threadIdx.x; c < p.D; c += kWideThreads) {
    const float e = row.scale * row.G(c, mean) * row.column_gate(c) * row.row_gate(c) * row.post(c);
    gb[c] = E::put(row.pr * fmaf(-row.k(c), along, e));
  }
}

// One thread per column; blockIdx.y takes the rows y, y + gridDim.y, ...  part [gridDim.y][2][D].
template <int DT, int PT>
__global__ void __launch_bounds__(256) residual_norm_bwd_wide_columns_kernel(ResidualNormParams p, ResidualNormGrads o,
                                                                             const float* __restrict__ means,
                                                                             float* __restrict__ part) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= p.D) return;
  float sw = 0.f, ss = 0.f;
  for (long long n = blockIdx.y; n < p.N; n += gridDim.y) {
    const Row<DT, PT> row(p, o, n);
    if (row.w != nullptr) sw = fmaf(Elem<DT>::get(__ldg(row.gh + c)), row.cs(c), sw);
    if (row.b != nullptr) {
      const float G = row.G(c, row.w == nullptr ? 0.f : __ldg(means + n));
      ss = fmaf(row.scale * G * row.row_gate(c), row.k(c), ss);
    }
  }
  float* const out = part + static_cast<size_t>(blockIdx.y) * 2 * p.D;
  out[c] = sw;
  out[p.D + c] = ss;
}

// 32 of the 2 D column sums per CTA; warp w adds the parts w, w + 32, ..., then the warps are joined
// in ascending order.
constexpr int kJoinWarps = 32;

template <int PT>
__global__ void __launch_bounds__(32 * kJoinWarps) residual_norm_join_kernel(ResidualNormParams p, ResidualNormGrads o,
                                                                             const float* __restrict__ part, int parts) {
  using P = Elem<PT>;
  using PE = typename P::T;
  __shared__ float sm[kJoinWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < 2 * p.D) {
#pragma unroll 5
    for (int i = warp; i < parts; i += kJoinWarps) s += part[static_cast<size_t>(i) * 2 * p.D + c];
  }
  sm[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || c >= 2 * p.D) return;
  s = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) s += sm[w][lane];
  if (c < p.D) {
    if (o.gweight != nullptr) static_cast<PE*>(o.gweight)[c] = P::put(s);
    return;
  }
  const int d = c - p.D;
  const PE* const gate = p.gate_kind == kGateColumns ? static_cast<const PE*>(p.gate) : nullptr;
  const PE* const pw = static_cast<const PE*>(p.post_weight);
  if (o.gpost != nullptr) static_cast<PE*>(o.gpost)[d] = P::put(gate == nullptr ? s : s * P::get(gate[d]));
  if (o.ggate != nullptr && gate != nullptr) static_cast<PE*>(o.ggate)[d] = P::put(pw == nullptr ? s : s * P::get(pw[d]));
}

template <int DT, int PT>
cudaError_t run(const ResidualNormParams& p, const ResidualNormGrads& o, cudaStream_t s) {
  float* const part = static_cast<float*>(o.workspace);
  float* const means = part + static_cast<size_t>(p.N < kParts ? p.N : kParts) * 2 * p.D;
  residual_norm_bwd_wide_x_kernel<DT, PT><<<p.N, kWideThreads, 0, s>>>(p, o, means);
  cudaError_t e = launch_result();
  const bool columns = o.gweight != nullptr || o.gpost != nullptr || (o.ggate != nullptr && p.gate_kind == kGateColumns);
  if (e != cudaSuccess || !columns) return e;
  const int parts = p.N < 64 ? 1 : p.N < 1024 ? p.N / 32 : 32;
  residual_norm_bwd_wide_columns_kernel<DT, PT><<<dim3((p.D + 255) / 256, parts), 256, 0, s>>>(p, o, means, part);
  if ((e = launch_result()) != cudaSuccess) return e;
  residual_norm_join_kernel<PT><<<(2 * p.D + 31) / 32, 32 * kJoinWarps, 0, s>>>(p, o, part, parts);
  return launch_result();
}

}  // namespace

size_t residual_norm_bwd_workspace(long long N, long long D) {
  const long long parts = N < kParts ? N : kParts;
  return (static_cast<size_t>(parts) * 2 * D + N) * sizeof(float);
}

cudaError_t launch_residual_norm_bwd(const ResidualNormParams& p, const ResidualNormGrads& o, cudaStream_t s) {
  const bool pf = p.param_dtype == kDtypeF32;
  if (p.dtype == kDtypeF32) return run<kDtypeF32, kDtypeF32>(p, o, s);
  if (p.dtype == kDtypeBF16) return pf ? run<kDtypeBF16, kDtypeF32>(p, o, s) : run<kDtypeBF16, kDtypeBF16>(p, o, s);
  return pf ? run<kDtypeF16, kDtypeF32>(p, o, s) : run<kDtypeF16, kDtypeF16>(p, o, s);
}

}  // namespace llp
