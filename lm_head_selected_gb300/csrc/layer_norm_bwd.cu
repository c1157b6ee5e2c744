// Gradients of layer norm.  With h = (x - mean) * rstd and a = grad_y * weight,
//
//   grad_x      = rstd * (a - sum a / D - h * (sum a h) / D)
//   grad_weight = sum over rows of grad_y * h,   grad_bias = sum over rows of grad_y
//
// One pass over grad_y and x gives all three.  A group of warps owns a row at a time,
// up to three vectors per thread: it holds the row in registers while its two sums
// are joined, writes grad_x, and as a thread's columns are the same in every row it
// keeps their share of the column sums in registers too.  Few threads with several
// vectors each, because the instructions of the sums (shuffles, a barrier, the
// exchange between the warps) weigh as much as those of a vector and the issue of
// instructions is what bounds this kernel next to memory: at 65600 rows of 2688 bf16
// one vector per thread takes 256 us (80 registers, two rows at once), two 213, three
// 171.  Each thread copies the vectors it will use itself, with cp.async into its own
// slots of a ring of rows, so that nothing but the sums makes threads wait for one
// another and the rows to come are in flight whatever the registers hold.  Group q of
// G takes the rows q, q + G, ...: the rows under way at one time are neighbours
// (contiguous ranges instead: 190 us).  A second launch joins the CTAs' column sums in
// ascending order.  Rows of 1025 to 2048 vectors take four per thread, read from the
// ring once more for grad_x because the registers hold no more than the column sums;
// wider ones take three plain kernels.
//
// Measured, bf16, three tensors of traffic: 16384 x 4096 66.2 us (6.1 TB/s, 90% of the
// measured copy peak), 65600 x 2688 164 to 166 us (94%), 16384 x 2688 45.1 us (87%: 5 us are the
// join and the two launches' ends), 4096 x 16384 71 us (84%), 4096 x 8448 55 us (56%; three
// plain kernels: 142).
#include "layer_norm.cuh"

namespace llp {

namespace {

constexpr int kBwdThreads = 512;  // of a CTA, one per SM: 128 registers per thread
template <int K, bool AL>
struct BwdRing {
  static constexpr int STAGES = K == 4 ? 2 : AL ? 4 : 3;  // rows
};

// part: [gridDim.x][2][D], the CTA's column sums of grad_y * h and of grad_y; null to skip them.
// Vectors per thread: K = ceil(units / (32 * warps)), or 4 for more than kPipeUnits vectors and 16
// warps; those from kFull<K> on may lie past the row's end.  Four are too many to hold beside their
// columns' sums: they are read from the ring once more for grad_x.
template <int DT, int PT, int K, bool AL>
__global__ void __launch_bounds__(kBwdThreads, 1) layer_norm_bwd_kernel(
    LayerNormParams p, int warps, const float* __restrict__ mean, const float* __restrict__ rstd,
    typename Elem<DT>::T* __restrict__ gx, float* __restrict__ part) {
  using T = typename Elem<DT>::T;
  constexpr int W = Elem<DT>::W, H = W / 2, STAGES = BwdRing<K, AL>::STAGES;
  constexpr bool HOLD = K < 4;
  using S = Slot<DT, AL>;
  extern __shared__ uint4 ring[];  // [STAGES][2][K][threads]: grad_y and x; then the weight; then the slots' fifth words
  __shared__ float red[2][K == 4 ? 1 : kBwdThreads / 32][32];  // [groups]: one of 16 warps when K is 4
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int threads = kBwdThreads;
  const int lane = threadIdx.x & 31;
  const int group = (threadIdx.x >> 5) / warps, warp = (threadIdx.x >> 5) - group * warps;
  const int groups = (threads >> 5) / warps;
  const int units = (p.D + W - 1) / W;
  const int first = 32 * warp + lane, width = 32 * warps;  // this thread's vectors: first + k * width
  const int last = first + (K - 1) * width;
  const bool tail = last < units;
  const int tail_n = min(p.D - last * W, W);  // elements of the last vector
  auto on = [&](int k) { return k < kFull<K> || (k == K - 1 ? tail : first + k * width < units); };
  auto left = [&](int k) { return k < kFull<K> ? W : k == K - 1 ? tail_n : min(p.D - (first + k * width) * W, W); };
  // this group's rows: r0, r0 + step, ...
  const unsigned step = gridDim.x * groups, r0 = blockIdx.x * groups + group, r1 = p.N;
  const T* gsrc = static_cast<const T*>(p.gy) + static_cast<long long>(r0) * p.gy_stride + first * W;
  const T* xsrc = static_cast<const T*>(p.x) + static_cast<long long>(r0) * p.x_stride + first * W;
  const T* const glo = static_cast<const T*>(p.gy);
  const T* const xlo = static_cast<const T*>(p.x);
  const T* const ghi = glo + static_cast<long long>(p.N - 1) * p.gy_stride + p.D;
  const T* const xhi = xlo + static_cast<long long>(p.N - 1) * p.x_stride + p.D;
  uint4* const mine = ring + threadIdx.x;
  constexpr int pitch = 2 * K * threads;  // of a stage
  float4* const kept = reinterpret_cast<float4*>(ring + STAGES * pitch);
  uint32_t* const fifth = reinterpret_cast<uint32_t*>(kept + W / 4 * units) + threadIdx.x;
  // what no copy writes stays 0: grad_y past the row's end adds nothing to any sum
#pragma unroll
  for (int k = kFull<K>; k < K; ++k)
    if (!AL || !on(k))
      for (int i = 0; i < 2 * STAGES; ++i) mine[(i * K + k) * threads] = make_uint4(0, 0, 0, 0);
  auto issue = [&](unsigned n, int stage) {  // row n, the next one, if there is one
    if (n < r1) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (on(k)) {
          const int g = stage * pitch + k * threads, x = g + K * threads, n = left(k);
          S::copy(mine + g, fifth + g, gsrc + k * width * W, n, glo, ghi);
          S::copy(mine + x, fifth + x, xsrc + k * width * W, n, xlo, xhi);
        }
      }
      gsrc += step * p.gy_stride;
      xsrc += step * p.x_stride;
    }
    copy_commit();
  };
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) issue(r0 + s * step, s);
  keep_params<PT, W, AL>(kept, static_cast<const typename Elem<PT>::T*>(p.weight), 1.f, p.D);
  // lane l holds the statistics of the group's row 32 b + l, and of the next 32
  auto stats = [&](const float* s, unsigned n) { return n + lane * step < r1 ? __ldg(s + n + lane * step) : 0.f; };
  float m_next = stats(mean, r0), s_next = stats(rstd, r0), m_lane = 0.f, s_lane = 0.f;
  F2 aw[K][H], ab[K][H];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < H; ++i) aw[k][i] = ab[k][i] = f2(0.f);
  const float inv = 1.f / static_cast<float>(p.D);
  T* out = gx == nullptr ? nullptr : gx + static_cast<size_t>(r0) * p.D + first * W;
  __syncthreads();  // the weight is kept
  int stage = 0;
  unsigned i = 0;  // rows taken
  for (unsigned n = r0; n < r1; n += step, ++i) {
    const unsigned i0 = i & 31;
    if (i0 == 0) {
      m_lane = m_next, s_lane = s_next;
      m_next = stats(mean, n + 32 * step), s_next = stats(rstd, n + 32 * step);
    }
    const float sc = __shfl_sync(0xffffffffu, s_lane, i0), minus = -__shfl_sync(0xffffffffu, m_lane, i0);
    const int now = stage;
    if (!HOLD) issue(n + step, stage ^ 1);
    copy_wait<HOLD ? STAGES - 2 : 1>();
    const bool gshift = S::shifted(glo + static_cast<long long>(n) * p.gy_stride);
    const bool xshift = S::shifted(xlo + static_cast<long long>(n) * p.x_stride);
    F2 a[HOLD ? K : 1][H], h[HOLD ? K : 1][H], t0 = f2(0.f), t1 = f2(0.f);
    // grad_y * weight and h of a vector, and on the first pass its share of the sums
    auto vector = [&](int k, F2 (&a)[H], F2 (&h)[H], bool sums) {
      const int g = now * pitch + k * threads, x = g + K * threads;
      unpack2<DT, W>(S::read(mine + g, fifth + g, gshift, left(k)), a);
      unpack2<DT, W>(S::read(mine + x, fifth + x, xshift, left(k)), h);
      const float m = on(k) ? minus : 0.f;  // past the row's end x is and stays 0
#pragma unroll
      for (int q = 0; q < W / 4; ++q) {
        const float4 w = on(k) ? kept[q * units + first + k * width] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 2 * q; i < 2 * q + 2; ++i) {
          // The mean is subtracted first, as in the forward: x - mean is exact where they are close.
          // x * rstd - mean * rstd in one step saves an instruction and adds half a unit of mean *
          // rstd to every h: 2.7e-3 in place of 0 for a row of 1000s.
          h[i] = add2(h[i], f2(m));
          if constexpr (!AL) {  // a ragged last vector; the second pass stores none of what is past the end
            if (sums && k >= kFull<K>)
              h[i] = f2(2 * i < left(k) ? h[i].x : 0.f, 2 * i + 1 < left(k) ? h[i].y : 0.f);
          }
          h[i] = mul2(h[i], f2(sc));
          if (sums) {
            ab[k][i] = add2(ab[k][i], a[i]);
            aw[k][i] = fma2(a[i], h[i], aw[k][i]);
          }
          a[i] = mul2(a[i], i == 2 * q ? f2(w.x, w.y) : f2(w.z, w.w));
          if (sums) {
            t0 = add2(t0, a[i]);
            t1 = fma2(a[i], h[i], t1);
          }
        }
      }
    };
#pragma unroll
    for (int k = 0; k < K; ++k) vector(k, a[HOLD ? k : 0], h[HOLD ? k : 0], true);
    if (HOLD) issue(n + (STAGES - 1) * step, stage == 0 ? STAGES - 1 : stage - 1);
    stage = stage + 1 == STAGES ? 0 : stage + 1;
    float s0 = sum2(t0), s1 = sum2(t1);
    group_sums(s0, s1, red[i & 1][group], warp, warps, 1 + group);
    if (out != nullptr) {
      // rstd * (a - s0 / D - h * s1 / D), rstd last: where grad_y * weight is one value in all of a
      // row, nothing of it is left.  For that s0 / D has to be a quotient.  Its remainder under the
      // product with 1 / D is exact in one fma, and the remainder's share corrects the product
      // (Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor",
      // 1990); the division took registers that 2688 columns do not have (44.8 -> 52.1 us).
      const float q = s0 * inv;
      const float c0 = -fmaf(fmaf(-q, static_cast<float>(p.D), s0), inv, q), c1 = -s1 * inv;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (on(k)) {
          F2(&av)[H] = a[HOLD ? k : 0], (&hv)[H] = h[HOLD ? k : 0];
          if (!HOLD) vector(k, av, hv, false);
#pragma unroll
          for (int i = 0; i < H; ++i) av[i] = mul2(fma2(hv[i], f2(c1), add2(av[i], f2(c0))), f2(sc));
          S::store(out + k * width * W, pack2<DT, W>(av), left(k));
        }
      }
      out += static_cast<size_t>(step) * p.D;
    }
  }
  if (part == nullptr) return;
  copy_wait<0>();
  __syncthreads();
  // the CTA's column sums: its groups in ascending order, through the ring's memory
  float* const join = reinterpret_cast<float*>(ring);  // [groups][2][units * W]
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (on(k)) {
      F2* const o = reinterpret_cast<F2*>(join + (group * 2 * units + first + k * width) * W);
#pragma unroll
      for (int i = 0; i < H; ++i) o[i] = aw[k][i], o[units * H + i] = ab[k][i];
    }
  }
  __syncthreads();
  float* const sum = part + static_cast<size_t>(blockIdx.x) * 2 * p.D;
  for (int c = threadIdx.x; c < 2 * p.D; c += threads) {
    const int at = c < p.D ? c : units * W + c - p.D;
    float s = join[at];
    for (int g = 1; g < groups; ++g) s += join[g * 2 * units * W + at];
    sum[c] = s;
  }
}

// 32 of the 2 D column sums per CTA; warp w adds the parts w, w + 32, ..., then the warps
// are joined in ascending order.
constexpr int kJoinWarps = 32;

template <int PT>
__global__ void __launch_bounds__(32 * kJoinWarps) layer_norm_join_kernel(const float* part, int parts,
                                                                          int D, typename Elem<PT>::T* __restrict__ gw,
                                                                          typename Elem<PT>::T* __restrict__ gb) {
  __shared__ float sm[kJoinWarps][32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  // the loads go out together: a part past the end is read again and not added
  constexpr int MOST = (kPipeSMs + kJoinWarps - 1) / kJoinWarps;
  float v[MOST], s = 0.f;
#pragma unroll
  for (int i = 0; i < MOST; ++i)
    v[i] = load_written(part + static_cast<size_t>(min(warp + i * kJoinWarps, parts - 1)) * 2 * D + min(c, 2 * D - 1));
#pragma unroll
  for (int i = 0; i < MOST; ++i)
    if (warp + i * kJoinWarps < parts) s += v[i];
  sm[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || c >= 2 * D) return;
  s = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) s += sm[w][lane];
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
  s0 = cta_sum<kWideThreads>(s0, sm) / static_cast<float>(p.D);
  s1 = cta_sum<kWideThreads>(s1, sm) * inv;
#pragma unroll 4
  for (int c = threadIdx.x; c < p.D; c += kWideThreads) {
    const float a = E::get(__ldg(g + c)) * (w != nullptr ? P::get(__ldg(w + c)) : 1.f);
    const float h = (E::get(__ldg(x + c)) - m) * r;
    gx[static_cast<size_t>(n) * p.D + c] = E::put(fmaf(-h, s1, a - s0) * r);
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
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return note_cuda(cudaLaunchKernelEx(&cfg, layer_norm_join_kernel<PT>, static_cast<const float*>(o.part), parts, p.D,
                                      static_cast<T*>(o.gw), static_cast<T*>(o.gb)));
}

template <int DT, int PT, int K>
cudaError_t rows(const LayerNormParams& p, int warps, bool al, const Grads& o, cudaStream_t s) {
  const int units = (p.D + Elem<DT>::W - 1) / Elem<DT>::W;
  const int groups = kBwdThreads / 32 / warps;  // warps is 1, 2, 4, 8 or 16
  const long long want = (static_cast<long long>(p.N) + groups - 1) / groups;
  const int grid = static_cast<int>(want < kPipeSMs ? want : kPipeSMs);
  const size_t slots = static_cast<size_t>(al ? BwdRing<K, true>::STAGES : BwdRing<K, false>::STAGES) * 2 * K * kBwdThreads;
  const size_t smem = slots * (al ? 16 : Slot<DT, false>::BYTES) + static_cast<size_t>(units) * (Elem<DT>::W / 4) * 16;
  const bool params = o.gw != nullptr || o.gb != nullptr;
  const auto kernel = al ? layer_norm_bwd_kernel<DT, PT, K, true> : layer_norm_bwd_kernel<DT, PT, K, false>;
  kernel<<<grid, kBwdThreads, smem, s>>>(p, warps, o.mean, o.rstd, static_cast<typename Elem<DT>::T*>(o.gx),
                                         params ? o.part : nullptr);
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
  const bool al = p.D % W == 0 && aligned16(p.x) && (p.x_stride * elem_bytes(DT)) % 16 == 0 && aligned16(p.gy) &&
                  (p.gy_stride * elem_bytes(DT)) % 16 == 0 && aligned16(o.gx) && aligned16(p.weight);
  const int units = (p.D + W - 1) / W;
  if (units <= kPipeUnits) {
    // three vectors per thread, two where ragged rows need registers of their own
    const int most = p.D % W == 0 ? 96 : 64;
    int warps = 1;
    while (most * warps < units) warps *= 2;
    const int K = (units + 32 * warps - 1) / (32 * warps);
    if (K == 1) return rows<DT, PT, 1>(p, warps, al, o, s);
    if (K == 2) return rows<DT, PT, 2>(p, warps, al, o, s);
    return rows<DT, PT, 3>(p, warps, al, o, s);
  }
  if (units <= 2 * kPipeUnits) return rows<DT, PT, 4>(p, 16, al, o, s);
  return wide<DT, PT>(p, o, s);
}

template <int DT, int PT, int K>
cudaError_t allow() {
  // K = 3: 192 KB of the ring, 24 KB of the weight; K = 4: 128 (odd 16-bit rows 160) and 64
  const int bytes = (K == 4 ? 224 : 222) * 1024;
  cudaError_t e = note_cuda(cudaFuncSetAttribute(layer_norm_bwd_kernel<DT, PT, K, true>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
  if (e == cudaSuccess)
    e = note_cuda(cudaFuncSetAttribute(layer_norm_bwd_kernel<DT, PT, K, false>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
  return e;
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

cudaError_t layer_norm_bwd_setup() {
  cudaError_t e = setup<kDtypeF32, kDtypeF32>();
  if (e == cudaSuccess) e = setup<kDtypeBF16, kDtypeF32>();
  if (e == cudaSuccess) e = setup<kDtypeBF16, kDtypeBF16>();
  if (e == cudaSuccess) e = setup<kDtypeF16, kDtypeF32>();
  if (e == cudaSuccess) e = setup<kDtypeF16, kDtypeF16>();
  return e;
}

size_t layer_norm_bwd_workspace(long long N, long long D) {
  const long long parts = N < kPipeSMs ? N : kPipeSMs;
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
