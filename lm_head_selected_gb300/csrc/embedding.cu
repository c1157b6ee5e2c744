// Token embedding: lookup with scaling, and its gradient.
//
//   out[n, :]         = scale * weight[t_n, :]
//   grad_weight[v, :] = scale * sum over n with t_n = v, ascending, of grad_out[n, :]
#include "elem.cuh"

namespace llp {

namespace {

__device__ __forceinline__ bool token_ok(long long t, long long V, long long ignore_index) {
  return t != ignore_index && t >= 0 && t < V;
}

constexpr int kThreads = 256;

// One CTA per token row.
template <int DT>
__global__ void __launch_bounds__(kThreads) embedding_fwd_kernel(const long long* __restrict__ tokens,
                                                                 const typename Elem<DT>::T* __restrict__ weight,
                                                                 int V, int D, float scale, long long ignore_index,
                                                                 typename Elem<DT>::T* __restrict__ out) {
  using E = Elem<DT>;
  const long long t = tokens[blockIdx.x];
  const bool ok = token_ok(t, V, ignore_index);
  typename E::T* o = out + static_cast<size_t>(blockIdx.x) * D;
  const typename E::T* w = weight + (ok ? static_cast<size_t>(t) * D : 0);
  for (int c = threadIdx.x; c < D; c += kThreads) o[c] = E::put(ok ? E::get(w[c]) * scale : 0.f);
}

// One CTA per table row: scans the tokens in ascending order, kThreads at a
// time, and adds the rows of those that name it.
template <int DT>
__global__ void __launch_bounds__(kThreads) embedding_bwd_kernel(const long long* __restrict__ tokens,
                                                                 const typename Elem<DT>::T* __restrict__ grad_out,
                                                                 long long stride, int N, int D, float scale,
                                                                 long long ignore_index, int accumulate,
                                                                 typename Elem<DT>::T* __restrict__ grad_weight) {
  using E = Elem<DT>;
  __shared__ unsigned hit[kThreads / 32];
  const long long v = blockIdx.x;
  typename E::T* o = grad_weight + static_cast<size_t>(v) * D;
  for (int c0 = 0; c0 < D; c0 += kThreads) {
    const int c = c0 + threadIdx.x;
    float acc = 0.f;
    bool any = false;
    for (int n0 = 0; n0 < N; n0 += kThreads) {
      const int n = n0 + threadIdx.x;
      const unsigned m = __ballot_sync(0xffffffffu, n < N && v != ignore_index && tokens[n] == v);
      if ((threadIdx.x & 31) == 0) hit[threadIdx.x >> 5] = m;
      __syncthreads();
      for (int w = 0; w < kThreads / 32; ++w) {
        for (unsigned b = hit[w]; b != 0; b &= b - 1) {
          any = true;
          const int at = n0 + 32 * w + __ffs(b) - 1;
          if (c < D) acc += E::get(grad_out[at * stride + c]);
        }
      }
      __syncthreads();
    }
    if (c < D && (any || !accumulate)) o[c] = E::put(fmaf(scale, acc, accumulate ? E::get(o[c]) : 0.f));
  }
}

template <int DT>
cudaError_t fwd(const EmbeddingParams& p, const void* weight, void* out, cudaStream_t s) {
  using T = typename Elem<DT>::T;
  embedding_fwd_kernel<DT><<<p.N, kThreads, 0, s>>>(p.tokens, static_cast<const T*>(weight), p.V, p.D, p.scale,
                                                    p.ignore_index, static_cast<T*>(out));
  return launch_result();
}

template <int DT>
cudaError_t bwd(const EmbeddingParams& p, const void* grad_out, long long stride, int accumulate, void* grad_weight,
                cudaStream_t s) {
  using T = typename Elem<DT>::T;
  embedding_bwd_kernel<DT><<<p.V, kThreads, 0, s>>>(p.tokens, static_cast<const T*>(grad_out), stride, p.N, p.D,
                                                    p.scale, p.ignore_index, accumulate, static_cast<T*>(grad_weight));
  return launch_result();
}

}  // namespace

size_t embedding_bwd_workspace(long long, long long, long long) { return 256; }

cudaError_t launch_embedding_fwd(const EmbeddingParams& p, const void* weight, void* out, cudaStream_t s) {
  if (p.dtype == kDtypeBF16) return fwd<kDtypeBF16>(p, weight, out, s);
  if (p.dtype == kDtypeF16) return fwd<kDtypeF16>(p, weight, out, s);
  return fwd<kDtypeF32>(p, weight, out, s);
}

cudaError_t launch_embedding_bwd(const EmbeddingParams& p, const void* grad_out, long long stride, int accumulate,
                                 void* grad_weight, void* workspace, cudaStream_t s) {
  (void)workspace;
  if (p.dtype == kDtypeBF16) return bwd<kDtypeBF16>(p, grad_out, stride, accumulate, grad_weight, s);
  if (p.dtype == kDtypeF16) return bwd<kDtypeF16>(p, grad_out, stride, accumulate, grad_weight, s);
  return bwd<kDtypeF32>(p, grad_out, stride, accumulate, grad_weight, s);
}

}  // namespace llp
