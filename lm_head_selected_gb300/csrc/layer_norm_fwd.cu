// Layer norm over the last dimension: y = (x - mean) * rstd * weight + bias.
//
// A warp owns a row (a quarter of a warp a very short one, up to four warps a wide
// one) and reads it once: the row stays in registers while its mean and then its
// centred second moment are summed, two reductions without cancellation.  Up to 11
// vectors per lane keep the reductions' instructions few against the row's own, and a
// row that one warp owns needs no barrier.  Each lane copies its vectors of the next
// row with cp.async into its own slots of shared memory meanwhile; the parameters lie
// there too, in fp32.  With a row spread over six warps, two vectors per lane, the
// exchange between the warps set the pace: 36.4 us against %FWD% at 16384 rows of
// 2688.  Rows beyond 1024 vectors are read three times by one CTA each (from L2 after
// the first).
#include "layer_norm.cuh"

namespace llp {

namespace {

template <int K>
struct FwdShape {
  static constexpr int WARPS = K <= 4 ? 32 : K <= 6 ? 24 : 16;  // of a CTA, one per SM: 64, 80 or 128 registers
};

// LANES: lanes of a row's warps that own a row (8 or 32); `warps` warps per row.
template <int DT, int PT, int K, int LANES, bool AL>
__global__ void __launch_bounds__(32 * FwdShape<K>::WARPS, 1) layer_norm_fwd_kernel(
    LayerNormParams p, int warps, RowRanges ranges, typename Elem<DT>::T* __restrict__ y,
    float* __restrict__ mean_out, float* __restrict__ rstd_out) {
  using T = typename Elem<DT>::T;
  using P = typename Elem<PT>::T;
  constexpr int W = Elem<DT>::W, H = W / 2;
  extern __shared__ uint4 slots[];  // [2][K][threads], then weight and bias [W / 4][units] float4 each
  __shared__ float red[2][FwdShape<K>::WARPS];
  const int threads = blockDim.x, lane = threadIdx.x & (LANES - 1);
  const int units = (p.D + W - 1) / W;
  const int group = LANES < 32 ? threadIdx.x / LANES : (threadIdx.x >> 5) / warps;
  const int warp = LANES < 32 ? 0 : (threadIdx.x >> 5) - group * warps;
  const int first = warp * K * LANES + lane;  // this lane's vectors: first + k * LANES
  const int groups = LANES < 32 ? threads / LANES : (threads >> 5) / warps;
  unsigned r0, r1;
  row_range(ranges, blockIdx.x * groups + group, r0, r1);
  const T* src = static_cast<const T*>(p.x) + static_cast<long long>(r0) * p.x_stride + first * W;
  uint4* const mine = slots + threadIdx.x;
  auto valid = [&](int k) { return min(p.D - (first + k * LANES) * W, W); };  // elements of vector k
  for (int i = 0; i < 2 * K; ++i) mine[i * threads] = make_uint4(0, 0, 0, 0);  // what no copy writes stays 0
  unsigned next = r0;
  auto issue = [&](int b) {  // the next row, if there is one
    if (next < r1) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (first + k * LANES < units)
          copy_vector<DT, AL>(mine + (b * K + k) * threads, src + k * LANES * W, valid(k));
      src += p.x_stride;
      ++next;
    }
    copy_commit();
  };
  issue(0);
  float4* const kept = reinterpret_cast<float4*>(slots + 2 * K * threads);
  keep_params<PT, W, AL>(kept, static_cast<const P*>(p.weight), 1.f, p.D);
  keep_params<PT, W, AL>(kept + W / 4 * units, static_cast<const P*>(p.bias), 0.f, p.D);
  __syncthreads();
  const float inv = 1.f / static_cast<float>(p.D);
  // sum over the row's lanes: butterflies, then its warps in ascending order
  auto row_sum = [&](float v, float* sm) {
#pragma unroll
    for (int off = LANES / 2; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if (LANES == 32 && warps > 1) {
      if (lane == 0) sm[group * warps + warp] = v;
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * warps) : "memory");
      v = sm[group * warps];
      for (int w = 1; w < warps; ++w) v += sm[group * warps + w];
    }
    return v;
  };
  T* out = y + static_cast<size_t>(r0) * p.D + first * W;
  // the lanes of a warp stay together: its groups' ranges differ by one row at most
  unsigned rounds = r1 - r0;
  if (LANES < 32) rounds = __reduce_max_sync(0xffffffffu, rounds);
  for (unsigned i = 0; i < rounds; ++i) {
    const int b = i & 1;
    issue(b ^ 1);
    copy_wait<1>();
    F2 x[K][H], t[H];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      unpack2<DT, W>(mine[(b * K + k) * threads], x[k]);
#pragma unroll
      for (int h = 0; h < H; ++h) t[h] = k == 0 ? x[k][h] : add2(t[h], x[k][h]);
    }
#pragma unroll
    for (int h = 1; h < H; ++h) t[0] = add2(t[0], t[h]);
    const float mean = row_sum(sum2(t[0]), red[0]) * inv;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const float m = first + k * LANES < units ? -mean : 0.f;  // past the row's end x is and stays 0
#pragma unroll
      for (int h = 0; h < H; ++h) x[k][h] = add2(x[k][h], f2(m));
      if constexpr (!AL) {  // a ragged last vector
        const int n = valid(k);
#pragma unroll
        for (int h = 0; h < H; ++h)
          x[k][h] = f2(2 * h < n ? x[k][h].x : 0.f, 2 * h + 1 < n ? x[k][h].y : 0.f);
      }
#pragma unroll
      for (int h = 0; h < H; ++h) t[h] = k == 0 ? mul2(x[k][h], x[k][h]) : fma2(x[k][h], x[k][h], t[h]);
    }
#pragma unroll
    for (int h = 1; h < H; ++h) t[0] = add2(t[0], t[h]);
    // rsqrtf is within two units in the last place
    const float rstd = rsqrtf(fmaf(row_sum(sum2(t[0]), red[1]), inv, p.eps));
    const unsigned n = r0 + i;
    if (LANES < 32 && n >= r1) continue;
    const F2 sc = f2(rstd);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int u = first + k * LANES;
      if (u < units) {
#pragma unroll
        for (int q = 0; q < W / 4; ++q) {
          const float4 w = kept[q * units + u], c = kept[(W / 4 + q) * units + u];
          x[k][2 * q] = fma2(mul2(x[k][2 * q], sc), f2(w.x, w.y), f2(c.x, c.y));
          x[k][2 * q + 1] = fma2(mul2(x[k][2 * q + 1], sc), f2(w.z, w.w), f2(c.z, c.w));
        }
        store_vector<DT, AL>(out + k * LANES * W, pack2<DT, W>(x[k]), valid(k));
      }
    }
    out += p.D;
    if (first == 0) {
      mean_out[n] = mean;
      rstd_out[n] = rstd;
    }
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
  const float rstd = rsqrtf(fmaf(cta_sum<kWideThreads>(s, sm), inv, p.eps));
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

template <int DT, int PT, int K, int LANES = 32>
cudaError_t rows(const LayerNormParams& p, int warps, void* y, float* mean, float* rstd, cudaStream_t s) {
  constexpr int W = Elem<DT>::W;
  const int units = (p.D + W - 1) / W;
  const bool al = p.D % W == 0 && aligned16(p.x) && (p.x_stride * elem_bytes(DT)) % 16 == 0 && aligned16(y) &&
                  aligned16(p.weight) && aligned16(p.bias);
  const auto kernel = al ? layer_norm_fwd_kernel<DT, PT, K, LANES, true> : layer_norm_fwd_kernel<DT, PT, K, LANES, false>;
  const int groups = LANES < 32 ? FwdShape<K>::WARPS * (32 / LANES) : FwdShape<K>::WARPS / warps;
  const int threads = LANES < 32 ? 32 * FwdShape<K>::WARPS : 32 * warps * groups;
  const size_t smem = (static_cast<size_t>(2) * K * threads + 2 * (W / 4) * static_cast<size_t>(units)) * 16;
  const long long want = (static_cast<long long>(p.N) + groups - 1) / groups;
  const int grid = static_cast<int>(want < kPipeSMs ? want : kPipeSMs);
  kernel<<<grid, threads, smem, s>>>(
      p, warps, row_ranges(p.N, static_cast<long long>(grid) * groups),
      static_cast<typename Elem<DT>::T*>(y), mean, rstd);
  return launch_result();
}

// Vectors per lane: few lanes with many vectors, see above; more than one warp per row
// where they would not fit its registers.
template <int DT, int PT>
cudaError_t run(const LayerNormParams& p, void* y, float* mean, float* rstd, cudaStream_t s) {
  const int units = (p.D + Elem<DT>::W - 1) / Elem<DT>::W;
  if (units <= 8) return rows<DT, PT, 1, 8>(p, 1, y, mean, rstd, s);
  if (units <= 32) return rows<DT, PT, 1>(p, 1, y, mean, rstd, s);
  if (units <= 64) return rows<DT, PT, 2>(p, 1, y, mean, rstd, s);
  if (units <= 128) return rows<DT, PT, 4>(p, 1, y, mean, rstd, s);
  if (units <= 192) return rows<DT, PT, 6>(p, 1, y, mean, rstd, s);
  if (units <= 256) return rows<DT, PT, 8>(p, 1, y, mean, rstd, s);
  if (units <= 352) return rows<DT, PT, 11>(p, 1, y, mean, rstd, s);
  if (units <= kPipeUnits) return rows<DT, PT, 8>(p, units <= 512 ? 2 : 4, y, mean, rstd, s);
  layer_norm_fwd_wide_kernel<DT, PT><<<p.N, kWideThreads, 0, s>>>(p, static_cast<typename Elem<DT>::T*>(y), mean, rstd);
  return launch_result();
}

constexpr int kFwdSmem = 220 * 1024;  // most that a layout above takes

template <int DT, int PT, int K, int LANES = 32>
cudaError_t allow() {
  const cudaError_t e = note_cuda(cudaFuncSetAttribute(layer_norm_fwd_kernel<DT, PT, K, LANES, true>,
                                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kFwdSmem));
  return e != cudaSuccess ? e
                          : note_cuda(cudaFuncSetAttribute(layer_norm_fwd_kernel<DT, PT, K, LANES, false>,
                                                           cudaFuncAttributeMaxDynamicSharedMemorySize, kFwdSmem));
}

template <int DT, int PT>
cudaError_t setup() {
  cudaError_t e = allow<DT, PT, 1, 8>();
  if (e == cudaSuccess) e = allow<DT, PT, 1>();
  if (e == cudaSuccess) e = allow<DT, PT, 2>();
  if (e == cudaSuccess) e = allow<DT, PT, 4>();
  if (e == cudaSuccess) e = allow<DT, PT, 6>();
  if (e == cudaSuccess) e = allow<DT, PT, 8>();
  if (e == cudaSuccess) e = allow<DT, PT, 11>();
  return e;
}

}  // namespace

cudaError_t layer_norm_fwd_setup() {
  cudaError_t e = setup<kDtypeF32, kDtypeF32>();
  if (e == cudaSuccess) e = setup<kDtypeBF16, kDtypeF32>();
  if (e == cudaSuccess) e = setup<kDtypeBF16, kDtypeBF16>();
  if (e == cudaSuccess) e = setup<kDtypeF16, kDtypeF32>();
  if (e == cudaSuccess) e = setup<kDtypeF16, kDtypeF16>();
  return e;
}

cudaError_t launch_layer_norm_fwd(const LayerNormParams& p, void* y, float* mean, float* rstd, cudaStream_t s) {
  const bool pf = p.param_dtype == kDtypeF32;
  if (p.dtype == kDtypeF32) return run<kDtypeF32, kDtypeF32>(p, y, mean, rstd, s);
  if (p.dtype == kDtypeBF16)
    return pf ? run<kDtypeBF16, kDtypeF32>(p, y, mean, rstd, s) : run<kDtypeBF16, kDtypeBF16>(p, y, mean, rstd, s);
  return pf ? run<kDtypeF16, kDtypeF32>(p, y, mean, rstd, s) : run<kDtypeF16, kDtypeF16>(p, y, mean, rstd, s);
}

}  // namespace llp
