// Dropout with the mask drawn from a counter-based generator, in the forward
// and again in the backward pass.
#include "elem.cuh"

namespace llp {

namespace {

constexpr int kThreads = 256;

// Philox4x32-10 (Salmon, Moraes, Dror, Shaw: "Parallel random numbers: as easy
// as 1, 2, 3", SC 2011).
__device__ __forceinline__ uint4 philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0,
                                        uint32_t k1) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const unsigned long long a = 0xD2511F53ull * c0, b = 0xCD9E8D57ull * c2;
    const uint32_t n0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0, n2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
    c1 = static_cast<uint32_t>(b);
    c3 = static_cast<uint32_t>(a);
    c0 = n0;
    c2 = n2;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// One thread per block of eight elements.
template <int DT>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const typename Elem<DT>::T* x,
                                                           const typename Elem<DT>::T* residual, long long count,
                                                           uint32_t threshold, float scale, uint64_t seed,
                                                           uint64_t offset, const long long* device_offset,
                                                           typename Elem<DT>::T* y) {
  using E = Elem<DT>;
  const uint64_t blk = static_cast<uint64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const long long e0 = static_cast<long long>(blk) * 8;
  if (e0 >= count) return;
  if (device_offset != nullptr) offset += static_cast<uint64_t>(*device_offset);
  const uint4 r = philox(static_cast<uint32_t>(blk), static_cast<uint32_t>(blk >> 32), static_cast<uint32_t>(offset),
                         static_cast<uint32_t>(offset >> 32), static_cast<uint32_t>(seed),
                         static_cast<uint32_t>(seed >> 32));
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (e0 + i >= count) break;
    const uint32_t lane = (i & 1) ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu;
    float v = lane >= threshold ? E::get(x[e0 + i]) * scale : 0.f;
    if (residual != nullptr) v += E::get(residual[e0 + i]);
    y[e0 + i] = E::put(v);
  }
}

template <int DT>
cudaError_t run(const DropoutParams& p, cudaStream_t s) {
  using T = typename Elem<DT>::T;
  const long long blocks = ((p.count + 7) / 8 + kThreads - 1) / kThreads;
  dropout_kernel<DT><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(
      static_cast<const T*>(p.x), static_cast<const T*>(p.residual), p.count, p.threshold, p.scale, p.seed, p.offset,
      p.device_offset, static_cast<T*>(p.y));
  return launch_result();
}

}  // namespace

cudaError_t launch_dropout(const DropoutParams& p, int num_sms, cudaStream_t s) {
  (void)num_sms;
  if (p.dtype == kDtypeBF16) return run<kDtypeBF16>(p, s);
  if (p.dtype == kDtypeF16) return run<kDtypeF16>(p, s);
  return run<kDtypeF32>(p, s);
}

}  // namespace llp
