// Layer norm over the last dimension: y = (x - mean) * rstd * weight + bias.
//
// A group of warps owns a row at a time, up to three vectors per thread, and reads it
// once: the row stays in registers while its mean and then its centred second moment
// are summed, two reductions without cancellation.  The rows to come are in flight
// meanwhile: each thread copies the vectors it will use itself, with cp.async into its
// own slots of a ring of rows; the parameters lie in shared memory too, in fp32.  Group
// q of G takes the rows q, q + G, ...: the rows under way at one time are neighbours.
// Rows of 1025 to 2048 vectors have a CTA each and four per thread; wider ones are read
// three times by one CTA each (from L2 after the first).
//
// Bound by memory, both ways.  Measured, bf16: 16384 x 2688 31.0 us (5.7 TB/s, 84% of
// the measured copy peak; an elementwise kernel of the same traffic takes 30.0), 65600 x
// 2688 108.6 us (96%).  One vector per thread, with six warps to a row, took 36.4 us, one
// warp to a row with eleven 32.6, contiguous ranges of rows 31.1 and 121.  4096 x 16384
// 52.0 us (76%), 4096 x 8448 41.7 (49%: a CTA has one row at a time, and its sums' latency
// shows; read three times 86 and 49).
#include "layer_norm.cuh"

namespace llp {

namespace {

template <int K>
struct FwdShape {
  static constexpr int THREADS = K <= 2 ? 1024 : K == 3 ? 768 : 512;  // of a CTA, one per SM: 64, 80 or 128 registers
  static constexpr int STAGES = K <= 3 ? 3 : 2;                       // rows of the ring
};

// Vectors per lane: K = ceil(units / (32 * warps)), or 4 for more than kPipeUnits vectors and 16
// warps.  Those from kFull<K> on may lie past the row's end.
template <int DT, int PT, int K, bool AL>
__global__ void __launch_bounds__(FwdShape<K>::THREADS, 1) layer_norm_fwd_kernel(
    LayerNormParams p, int warps, int groups, typename Elem<DT>::T* __restrict__ y,
    float* __restrict__ mean_out, float* __restrict__ rstd_out) {
  using T = typename Elem<DT>::T;
  using P = typename Elem<PT>::T;
  constexpr int W = Elem<DT>::W, H = W / 2, STAGES = FwdShape<K>::STAGES;
  using S = Slot<DT, AL>;
  extern __shared__ uint4 ring[];  // [STAGES][K][threads]; then weight and bias; then the slots' fifth words
  __shared__ float red[2][FwdShape<K>::THREADS / 32];
  constexpr int threads = FwdShape<K>::THREADS;
  const int lane = threadIdx.x & 31;
  const int group = (threadIdx.x >> 5) / warps, warp = (threadIdx.x >> 5) - group * warps;
  const int units = (p.D + W - 1) / W;
  const int first = 32 * warp + lane, width = 32 * warps;  // this lane's vectors: first + k * width
  const int last = first + (K - 1) * width;
  const bool tail = last < units;
  const int tail_n = min(p.D - last * W, W);  // elements of the last vector
  auto on = [&](int k) { return k < kFull<K> || (k == K - 1 ? tail : first + k * width < units); };
  auto left = [&](int k) { return k < kFull<K> ? W : k == K - 1 ? tail_n : min(p.D - (first + k * width) * W, W); };
  // this group's rows: r0, r0 + step, ...; none when there are more groups than named barriers
  const unsigned step = gridDim.x * groups, r0 = blockIdx.x * groups + group, r1 = group < groups ? p.N : 0;
  const T* src = static_cast<const T*>(p.x) + static_cast<long long>(r0) * p.x_stride + first * W;
  const T* const lo = static_cast<const T*>(p.x);
  const T* const hi = lo + static_cast<long long>(p.N - 1) * p.x_stride + p.D;
  uint4* const mine = ring + threadIdx.x;
  constexpr int pitch = K * threads;  // of a stage
  float4* const kept = reinterpret_cast<float4*>(ring + STAGES * pitch);
  uint32_t* const fifth = reinterpret_cast<uint32_t*>(kept + W / 2 * units) + threadIdx.x;
#pragma unroll
  for (int k = kFull<K>; k < K; ++k)
    if (!AL || !on(k))  // what no copy writes stays 0
      for (int i = 0; i < STAGES; ++i) mine[(i * K + k) * threads] = make_uint4(0, 0, 0, 0);
  auto issue = [&](unsigned n, int stage) {  // row n, the next one, if there is one
    if (n < r1) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (on(k))
          S::copy(mine + stage * pitch + k * threads, fifth + stage * pitch + k * threads, src + k * width * W, left(k),
                  lo, hi);
      src += step * p.x_stride;
    }
    copy_commit();
  };
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) issue(r0 + s * step, s);
  keep_params<PT, W, AL>(kept, static_cast<const P*>(p.weight), 1.f, p.D);
  keep_params<PT, W, AL>(kept + W / 4 * units, static_cast<const P*>(p.bias), 0.f, p.D);
  __syncthreads();
  const float inv = 1.f / static_cast<float>(p.D);
  // sum over the group: butterflies, then over its warps
  auto row_sum = [&](float v, float* sm) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if (warps > 1) {
      if (lane == 0) sm[group * warps + warp] = v;
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * warps) : "memory");
      v = sm[group * warps + (lane & (warps - 1))];
      for (int off = warps / 2; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    }
    return v;
  };
  T* out = y + static_cast<size_t>(r0) * p.D + first * W;
  int stage = 0;
  for (unsigned n = r0; n < r1; n += step) {
    copy_wait<STAGES - 2>();
    const int at = stage * pitch;
    const bool shift = S::shifted(lo + static_cast<long long>(n) * p.x_stride);
    F2 x[K][H], t[2] = {f2(0.f), f2(0.f)};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      unpack2<DT, W>(S::read(mine + at + k * threads, fifth + at + k * threads, shift, left(k)), x[k]);
#pragma unroll
      for (int i = 0; i < H; ++i) t[i & 1] = add2(t[i & 1], x[k][i]);
    }
    issue(n + (STAGES - 1) * step, stage == 0 ? STAGES - 1 : stage - 1);
    stage = stage + 1 == STAGES ? 0 : stage + 1;
    // a quotient, not a product with 1 / D: the mean of equal values has to be that value (0.08 in
    // place of 0 came out of 1000 columns of 3000)
    const float mean = row_sum(sum2(add2(t[0], t[1])), red[0]) / static_cast<float>(p.D);
    t[0] = t[1] = f2(0.f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const float m = on(k) ? -mean : 0.f;  // past the row's end x is and stays 0
#pragma unroll
      for (int i = 0; i < H; ++i) {
        x[k][i] = add2(x[k][i], f2(m));
        if constexpr (!AL) {  // a ragged last vector
          if (k >= kFull<K>) x[k][i] = f2(2 * i < left(k) ? x[k][i].x : 0.f, 2 * i + 1 < left(k) ? x[k][i].y : 0.f);
        }
        t[i & 1] = fma2(x[k][i], x[k][i], t[i & 1]);
      }
    }
    // rsqrtf is within two units in the last place
    const float rstd = rsqrtf(fmaf(row_sum(sum2(add2(t[0], t[1])), red[1]), inv, p.eps));
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (on(k)) {
        const int u = first + k * width;
#pragma unroll
        for (int q = 0; q < W / 4; ++q) {
          const float4 w = kept[q * units + u], c = kept[(W / 4 + q) * units + u];
          x[k][2 * q] = fma2(mul2(x[k][2 * q], f2(rstd)), f2(w.x, w.y), f2(c.x, c.y));
          x[k][2 * q + 1] = fma2(mul2(x[k][2 * q + 1], f2(rstd)), f2(w.z, w.w), f2(c.z, c.w));
        }
        S::store(out + k * width * W, pack2<DT, W>(x[k]), left(k));
      }
    }
    out += static_cast<size_t>(step) * p.D;
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
  const float mean = cta_sum<kWideThreads>(s, sm) / static_cast<float>(p.D);
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

template <int DT, int PT, int K>
cudaError_t rows(const LayerNormParams& p, int warps, bool al, void* y, float* mean, float* rstd, cudaStream_t s) {
  using Shape = FwdShape<K>;
  const int units = (p.D + Elem<DT>::W - 1) / Elem<DT>::W;
  int groups = Shape::THREADS / 32 / warps;
  if (warps > 1 && groups > 15) groups = 15;  // named barriers 1 .. 15
  const size_t smem = static_cast<size_t>(Shape::STAGES) * K * Shape::THREADS * (al ? 16 : Slot<DT, false>::BYTES) +
                      static_cast<size_t>(Elem<DT>::W / 2) * units * 16;
  const long long want = (static_cast<long long>(p.N) + groups - 1) / groups;
  const int grid = static_cast<int>(want < kPipeSMs ? want : kPipeSMs);
  const auto kernel = al ? layer_norm_fwd_kernel<DT, PT, K, true> : layer_norm_fwd_kernel<DT, PT, K, false>;
  kernel<<<grid, Shape::THREADS, smem, s>>>(p, warps, groups, static_cast<typename Elem<DT>::T*>(y), mean, rstd);
  return launch_result();
}

template <int DT, int PT>
cudaError_t run(const LayerNormParams& p, void* y, float* mean, float* rstd, cudaStream_t s) {
  const int units = (p.D + Elem<DT>::W - 1) / Elem<DT>::W;
  const bool al = p.D % Elem<DT>::W == 0 && aligned16(p.x) && (p.x_stride * elem_bytes(DT)) % 16 == 0 &&
                  aligned16(y) && aligned16(p.weight) && aligned16(p.bias);
  if (units <= kPipeUnits) {
    int warps = 1;
    while (96 * warps < units) warps *= 2;
    const int K = (units + 32 * warps - 1) / (32 * warps);
    if (K == 1) return rows<DT, PT, 1>(p, warps, al, y, mean, rstd, s);
    if (K == 2) return rows<DT, PT, 2>(p, warps, al, y, mean, rstd, s);
    return rows<DT, PT, 3>(p, warps, al, y, mean, rstd, s);
  }
  if (units <= 2 * kPipeUnits) return rows<DT, PT, 4>(p, 16, al, y, mean, rstd, s);
  layer_norm_fwd_wide_kernel<DT, PT><<<p.N, kWideThreads, 0, s>>>(p, static_cast<typename Elem<DT>::T*>(y), mean, rstd);
  return launch_result();
}

template <int DT, int PT, int K>
cudaError_t allow() {
  const int bytes = 220 * 1024;  // more than any layout takes
  const cudaError_t e = note_cuda(cudaFuncSetAttribute(layer_norm_fwd_kernel<DT, PT, K, true>,
                                                       cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
  return e != cudaSuccess ? e
                          : note_cuda(cudaFuncSetAttribute(layer_norm_fwd_kernel<DT, PT, K, false>,
                                                           cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
}

template <int DT, int PT>
cudaError_t setup() {
  cudaError_t e = allow<DT, PT, 1>();
  if (e == cudaSuccess) e = allow<DT, PT, 2>();
  if (e == cudaSuccess) e = allow<DT, PT, 3>();
  if (e == cudaSuccess) e = allow<DT, PT, 4>();
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
