// Dropout with the mask drawn from a counter-based generator, in the forward
// and again in the backward pass:
//   y[e] = (16-bit lane e % 8 of Philox block e / 8 >= threshold ? x[e] * scale : 0) + residual[e]
//
// One thread moves the eight elements of a Philox block, several blocks with
// their loads in flight together; the rounds run while they are.  16 bits per
// element halve the generator's work: 32 would cost 40 wide multiplies per eight
// elements, about what the multiplier pipe can do in the time their 32 bytes
// take through HBM.
//
// Bound by memory.  Measured, bf16: 16384 x 2688 with a residual 38.4 us (6.9 TB/s, the
// measured copy peak), without one 30.0 (5.9 TB/s, 87%); 65600 x 2688 without one 112.5
// (6.3 TB/s, 93%).
#include "elem.cuh"

namespace llp {

namespace {

constexpr int kThreads = 256;
// Blocks of eight elements per thread, their loads in flight together, measured at 65600 x
// 2688 bf16 (and with a residual at 16384 x 2688): 1 block 130 (38.1) us, 2 119 (38.4),
// 3 112.5 (38.4), 4 112.8 (39.0), 8 114.5 (43.0).
constexpr int kBlocks = 3;

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

// Applies one block's lanes to v[0..7].
__device__ __forceinline__ void drop8(const uint4& r, uint32_t threshold, float scale, float (&v)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = (w[i] & 0xFFFFu) >= threshold ? v[2 * i] * scale : 0.f;
    v[2 * i + 1] = (w[i] >> 16) >= threshold ? v[2 * i + 1] * scale : 0.f;
  }
}

// x and residual are read before y is written at the same place, so y may be either of
// them: neither is read through the read-only path.
template <int DT, bool RES, int BLOCKS>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const typename Elem<DT>::T* x,
                                                           const typename Elem<DT>::T* residual, long long count,
                                                           uint32_t threshold, float scale, uint64_t seed,
                                                           uint64_t offset, const long long* device_offset,
                                                           typename Elem<DT>::T* y) {
  using E = Elem<DT>;
  constexpr int VECS = 8 / E::W;  // 16-byte vectors of eight elements
  if (device_offset != nullptr) offset += static_cast<uint64_t>(*device_offset);
  const long long first = static_cast<long long>(blockIdx.x) * (kThreads * BLOCKS) + threadIdx.x;
  const long long whole = count / 8;
  uint4 xv[BLOCKS][VECS], rv[BLOCKS][VECS];
#pragma unroll
  for (int j = 0; j < BLOCKS; ++j) {
    const long long blk = first + j * kThreads;
    if (blk < whole) {
#pragma unroll
      for (int k = 0; k < VECS; ++k) xv[j][k] = reinterpret_cast<const uint4*>(x)[blk * VECS + k];
      if (RES) {
#pragma unroll
        for (int k = 0; k < VECS; ++k) rv[j][k] = reinterpret_cast<const uint4*>(residual)[blk * VECS + k];
      }
    }
  }
#pragma unroll
  for (int j = 0; j < BLOCKS; ++j) {
    const long long blk = first + j * kThreads;
    if (blk > whole || blk * 8 >= count) break;
    const uint4 r = philox(static_cast<uint32_t>(blk), static_cast<uint32_t>(blk >> 32), static_cast<uint32_t>(offset),
                           static_cast<uint32_t>(offset >> 32), static_cast<uint32_t>(seed),
                           static_cast<uint32_t>(seed >> 32));
    float v[8];
    if (blk < whole) {
#pragma unroll
      for (int k = 0; k < VECS; ++k) E::unpack(xv[j][k], *reinterpret_cast<float(*)[E::W]>(v + k * E::W));
      drop8(r, threshold, scale, v);
#pragma unroll
      for (int k = 0; k < VECS; ++k) {
        float(&o)[E::W] = *reinterpret_cast<float(*)[E::W]>(v + k * E::W);
        if (RES) {
          float t[E::W];
          E::unpack(rv[j][k], t);
#pragma unroll
          for (int i = 0; i < E::W; ++i) o[i] += t[i];
        }
        reinterpret_cast<uint4*>(y)[blk * VECS + k] = E::pack(o);
      }
    } else {  // the last, partial block
      const int n = static_cast<int>(count - blk * 8);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < n ? E::get(x[blk * 8 + i]) : 0.f;
      drop8(r, threshold, scale, v);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) y[blk * 8 + i] = E::put(RES ? v[i] + E::get(residual[blk * 8 + i]) : v[i]);
    }
  }
}

// Tensors that do not start on a 16-byte boundary: element by element, one thread per block of
// eight.  One element late, bf16: 16384 x 2688 with a residual 110 us, without one 78, 65600 x
// 2688 305: 2.6 to 2.9 times the vectors' time.
template <int DT>
__global__ void __launch_bounds__(kThreads) dropout_unaligned_kernel(const typename Elem<DT>::T* x,
                                                                     const typename Elem<DT>::T* residual,
                                                                     long long count, uint32_t threshold, float scale,
                                                                     uint64_t seed, uint64_t offset,
                                                                     const long long* device_offset,
                                                                     typename Elem<DT>::T* y) {
  using E = Elem<DT>;
  const long long blk = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  if (blk * 8 >= count) return;
  if (device_offset != nullptr) offset += static_cast<uint64_t>(*device_offset);
  const uint4 r = philox(static_cast<uint32_t>(blk), static_cast<uint32_t>(blk >> 32), static_cast<uint32_t>(offset),
                         static_cast<uint32_t>(offset >> 32), static_cast<uint32_t>(seed),
                         static_cast<uint32_t>(seed >> 32));
  const int n = static_cast<int>(count - blk * 8 < 8 ? count - blk * 8 : 8);
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = i < n ? E::get(x[blk * 8 + i]) : 0.f;
  drop8(r, threshold, scale, v);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) y[blk * 8 + i] = E::put(residual != nullptr ? v[i] + E::get(residual[blk * 8 + i]) : v[i]);
}

template <int DT, bool RES, int BLOCKS>
cudaError_t launch(const DropoutParams& p, cudaStream_t s) {
  using T = typename Elem<DT>::T;
  const long long blocks = (p.count + 7) / 8;
  const long long per = kThreads * BLOCKS;
  dropout_kernel<DT, RES, BLOCKS><<<static_cast<unsigned>((blocks + per - 1) / per), kThreads, 0, s>>>(
      static_cast<const T*>(p.x), static_cast<const T*>(p.residual), p.count, p.threshold, p.scale, p.seed, p.offset,
      p.device_offset, static_cast<T*>(p.y));
  return launch_result();
}

template <int DT>
cudaError_t run(const DropoutParams& p, int num_sms, cudaStream_t s) {
  using T = typename Elem<DT>::T;
  const long long blocks = (p.count + 7) / 8;
  if (!aligned16(p.x) || !aligned16(p.residual) || !aligned16(p.y)) {
    dropout_unaligned_kernel<DT><<<static_cast<unsigned>((blocks + kThreads - 1) / kThreads), kThreads, 0, s>>>(
        static_cast<const T*>(p.x), static_cast<const T*>(p.residual), p.count, p.threshold, p.scale, p.seed, p.offset,
        p.device_offset, static_cast<T*>(p.y));
    return launch_result();
  }
  // several blocks per thread once every SM has its fill of threads without them
  const bool deep = blocks > static_cast<long long>(num_sms) * 2048 * 2;
  if (p.residual != nullptr) return deep ? launch<DT, true, kBlocks>(p, s) : launch<DT, true, 1>(p, s);
  return deep ? launch<DT, false, kBlocks>(p, s) : launch<DT, false, 1>(p, s);
}

}  // namespace

cudaError_t launch_dropout(const DropoutParams& p, int num_sms, cudaStream_t s) {
  if (p.dtype == kDtypeBF16) return run<kDtypeBF16>(p, num_sms, s);
  if (p.dtype == kDtypeF16) return run<kDtypeF16>(p, num_sms, s);
  return run<kDtypeF32>(p, num_sms, s);
}

}  // namespace llp
