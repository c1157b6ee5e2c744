// RMS norms around a block: s = x + scale * gate * norm(branch), h = norm(s), in one launch.
//
// A group of warps owns a row at a time, up to three vectors per thread (four for more than 1024
// vectors), and reads x, branch and a gate of the row's own once.  The branch stays in registers while
// its squares are summed, becomes s there, and s while its squares are summed.  The rows to come are in
// flight meanwhile in a ring of shared memory that every thread fills for itself; the columns'
// coefficients, scale * gate * post_weight and weight, lie beside it in fp32.  Group q of G takes the
// rows q, q + G, ...  Rows of more than 2048 vectors are read three times by one CTA each (from L2 after
// the first).
//
// Bound by memory: two tensors read and two written.  Measured in a captured graph, bf16 with a gate per
// column and both norms: 16384 x 2688 53.5 to 58.5 us by machine (6.0 to 6.6 TB/s, 90 to 98% of
// the measured copy peak; one CTA per row with three passes 235); with two vectors per thread in place of three 68.7.  32 x 2688 4.1 us, of which most is
// latency.  16384 x 2688 without a branch, the plain RMS norm, 32.5 us (81%): two rows of one tensor are half
// the bytes on the way.  Odd rows are bound by their 4-byte copies, as in layer norm.
#include "residual_norm.cuh"

namespace llp {

namespace {

// Vectors per lane: K = ceil(units / (32 * warps)); those from kFull<K> on may lie past the row's end.
// What no copy writes stays 0 in the ring, and adds nothing to any sum.
template <int DT, int K, bool AL, bool ROWS>
__global__ void __launch_bounds__(kResThreads, 1) residual_norm_fwd_kernel(const ResidualNormParams p,
                                                                           const ResidualNormOut o, int warps,
                                                                           int stages, bool keep_wide) {
  using T = typename Elem<DT>::T;
  constexpr int W = Elem<DT>::W, H = W / 2, N_IN = ROWS ? 3 : 2, threads = kResThreads;
  const bool keep = K < 4 || keep_wide;  // the coefficients lie in shared memory
  using S = Slot<DT, AL>;
  extern __shared__ uint4 ring[];  // [stages][N_IN][K][threads]; then the coefficients; then the slots' fifth words
  __shared__ float red[2][2][threads / 32];
  const int lane = threadIdx.x & 31;
  const int group = (threadIdx.x >> 5) / warps, warp = (threadIdx.x >> 5) - group * warps;
  const int groups = (threads >> 5) / warps;
  const int units = (p.D + W - 1) / W;
  const int first = 32 * warp + lane, width = 32 * warps;  // this lane's vectors: first + k * width
  auto on = [&](int k) { return k < kFull<K> || first + k * width < units; };
  auto left = [&](int k) { return k < kFull<K> ? W : min(p.D - (first + k * width) * W, W); };
  const unsigned step = gridDim.x * groups, r0 = blockIdx.x * groups + group, r1 = p.N;  // this group's rows
  constexpr int pitch = N_IN * K * threads;  // of a stage
  uint4* const mine = ring + threadIdx.x;
  float4* const kept = reinterpret_cast<float4*>(ring + stages * pitch);
  uint32_t* const fifth = reinterpret_cast<uint32_t*>(kept + (keep ? W / 2 * units : 0)) + threadIdx.x;
  const bool has_b = p.branch != nullptr, f32 = p.param_dtype == kDtypeF32;
  for (int i = 0; i < stages * N_IN; ++i)
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (!AL || !on(k) || (!has_b && i % N_IN == 1)) mine[(i * K + k) * threads] = make_uint4(0, 0, 0, 0);
      if (S::FIVE) fifth[(i * K + k) * threads] = 0;  // read wherever a row starts in the middle of a word
    }
  auto copy = [&](const void* base, long long stride, unsigned n, int at) {
    const T* const lo = static_cast<const T*>(base);
    const T* const src = lo + static_cast<long long>(n) * stride + first * W;
    const T* const hi = lo + static_cast<long long>(p.N - 1) * stride + p.D;
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (on(k)) S::copy(mine + at + k * threads, fifth + at + k * threads, src + k * width * W, left(k), lo, hi);
  };
  auto issue = [&](unsigned n, int stage) {  // row n, if there is one
    if (n < r1) {
      copy(p.x, p.x_stride, n, stage * pitch);
      if (has_b) copy(p.branch, p.b_stride, n, stage * pitch + K * threads);
      if (ROWS) copy(p.gate, p.gate_stride, n, stage * pitch + 2 * K * threads);
    }
    copy_commit();
  };
  for (int s = 0; s < stages - 1; ++s) issue(r0 + s * step, s);
  if (keep) keep_coefficients<DT, AL>(kept, p);
  __syncthreads();
  const float inv = 1.f / static_cast<float>(p.D);
  int stage = 0;
  unsigned i = 0;
  for (unsigned n = r0; n < r1; n += step, ++i) {
    issue(n + (stages - 1) * step, stage == 0 ? stages - 1 : stage - 1);
    copies_left(stages - 1);
    const int at = stage * pitch;
    stage = stage + 1 == stages ? 0 : stage + 1;
    auto read = [&](int t, int k, const void* base, long long stride, F2 (&v)[H]) {
      const bool shift = S::shifted(static_cast<const T*>(base) + static_cast<long long>(n) * stride);
      const int slot = at + (t * K + k) * threads;
      unpack2<DT, W>(S::read(mine + slot, fifth + slot, shift, left(k)), v);
    };
    F2 s[K][H];
#pragma unroll
    for (int k = 0; k < K; ++k) read(1, k, p.branch, p.b_stride, s[k]);
    float pr = 1.f;
    if (p.post_weight != nullptr) {
      F2 t[2] = {f2(0.f), f2(0.f)};
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < H; ++j) t[j & 1] = fma2(s[k][j], s[k][j], t[j & 1]);
      // rsqrtf is within two units in the last place
      pr = rsqrtf(fmaf(group_sum(sum2(add2(t[0], t[1])), red[0][i & 1] + group * warps, warp, warps, 1 + group), inv, p.eps));
      if (first == 0) o.post_rstd[n] = pr;
    }
    F2 t[2] = {f2(0.f), f2(0.f)};
    T* const out_s = static_cast<T*>(o.s) + static_cast<size_t>(n) * p.D + first * W;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      F2 x[H], c[H];
      read(0, k, p.x, p.x_stride, x);
      if (has_b && on(k)) {  // past the row's end there is no coefficient, and any in its place might be infinite
        if (keep)
          kept_vector<W>(kept, 0, units, first + k * width, c);
        else
          coefficient_vector<DT, W, AL>(p, f32, (first + k * width) * W, left(k), c);
#pragma unroll
        for (int j = 0; j < H; ++j) s[k][j] = mul2(mul2(s[k][j], f2(pr)), c[j]);
        if (ROWS) {
          F2 g[H];
          read(2, k, p.gate, p.gate_stride, g);
#pragma unroll
          for (int j = 0; j < H; ++j) s[k][j] = mul2(s[k][j], g[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < H; ++j) {
        s[k][j] = add2(s[k][j], x[j]);
        t[j & 1] = fma2(s[k][j], s[k][j], t[j & 1]);
      }
      if (o.s != nullptr && on(k)) S::store(out_s + k * width * W, pack2<DT, W>(s[k]), left(k));
    }
    if (p.weight == nullptr) continue;
    const float r = rsqrtf(fmaf(group_sum(sum2(add2(t[0], t[1])), red[1][i & 1] + group * warps, warp, warps, 1 + group), inv, p.eps));
    if (first == 0) o.rstd[n] = r;
    T* const out_h = static_cast<T*>(o.h) + static_cast<size_t>(n) * p.D + first * W;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (on(k)) {
        F2 w[H];
        if (keep)
          kept_vector<W>(kept, 1, units, first + k * width, w);
        else
          param_vector<DT, W, AL>(p.weight, f32, (first + k * width) * W, left(k), w);
#pragma unroll
        for (int j = 0; j < H; ++j) s[k][j] = mul2(mul2(s[k][j], f2(r)), w[j]);
        S::store(out_h + k * width * W, pack2<DT, W>(s[k]), left(k));
      }
    }
  }
}

// ---------------------------------------------------------------- wide rows

constexpr int kWideThreads = 512;

template <int DT, int PT>
__global__ void __launch_bounds__(kWideThreads) residual_norm_fwd_wide_kernel(ResidualNormParams p, ResidualNormOut o) {
  using E = Elem<DT>;
  using T = typename E::T;
  using P = Elem<PT>;
  using PE = typename P::T;
  __shared__ float sm[kWideThreads / 32];
  const long long n = blockIdx.x;
  const T* const x = static_cast<const T*>(p.x) + n * p.x_stride;
  const T* const b = p.branch == nullptr ? nullptr : static_cast<const T*>(p.branch) + n * p.b_stride;
  const T* const gr = p.gate_kind == kGateRows ? static_cast<const T*>(p.gate) + n * p.gate_stride : nullptr;
  const PE* const gc = p.gate_kind == kGateColumns ? static_cast<const PE*>(p.gate) : nullptr;
  const PE* const pw = static_cast<const PE*>(p.post_weight);
  const PE* const w = static_cast<const PE*>(p.weight);
  const float inv = 1.f / static_cast<float>(p.D);
  float pr = 1.f;
  if (pw != nullptr) {
    float t = 0.f;
#pragma unroll 8
    for (int c = threadIdx.x; c < p.D; c += kWideThreads) {
      const float v = E::get(__ldg(b + c));
      t = fmaf(v, v, t);
    }
    pr = rsqrtf(fmaf(cta_sum<kWideThreads>(t, sm), inv, p.eps));
    if (threadIdx.x == 0) o.post_rstd[n] = pr;
  }
  auto stream = [&](int c) {
    float v = E::get(__ldg(x + c));
    if (b != nullptr) {
      float m = E::get(__ldg(b + c)) * pr * p.scale;
      if (pw != nullptr) m *= P::get(__ldg(pw + c));
      if (gc != nullptr) m *= P::get(__ldg(gc + c));
      if (gr != nullptr) m *= E::get(__ldg(gr + c));
      v += m;
    }
    return v;
  };
  T* const s = static_cast<T*>(o.s) + n * p.D;
  T* const h = static_cast<T*>(o.h) + n * p.D;
  if (w == nullptr) {
#pragma unroll 4
    for (int c = threadIdx.x; c < p.D; c += kWideThreads) s[c] = E::put(stream(c));
    return;
  }
  float t = 0.f;
#pragma unroll 4
  for (int c = threadIdx.x; c < p.D; c += kWideThreads) {
    const float v = stream(c);
    t = fmaf(v, v, t);
  }
  const float r = rsqrtf(fmaf(cta_sum<kWideThreads>(t, sm), inv, p.eps));
  if (threadIdx.x == 0) o.rstd[n] = r;
#pragma unroll 4
  for (int c = threadIdx.x; c < p.D; c += kWideThreads) {
    const float v = stream(c);
    if (o.s != nullptr) s[c] = E::put(v);
    h[c] = E::put(v * r * P::get(__ldg(w + c)));
  }
}

// ---------------------------------------------------------------- launches

template <int DT, int K, bool ROWS>
cudaError_t rows(const ResidualNormParams& p, const ResidualNormOut& o, int warps, bool al, cudaStream_t s) {
  constexpr int W = Elem<DT>::W;
  const int units = (p.D + W - 1) / W, groups = kResThreads / 32 / warps;
  const size_t per_stage = static_cast<size_t>(ROWS ? 3 : 2) * K * kResThreads * (al ? 16 : Slot<DT, false>::BYTES);
  size_t kept = static_cast<size_t>(2) * units * W * sizeof(float);
  const bool keep = K < 4 || res_keep(per_stage, kept);
  if (!keep) kept = 0;
  const int stages = res_stages(per_stage, kept);
  const long long want = (static_cast<long long>(p.N) + groups - 1) / groups;
  const int grid = static_cast<int>(want < kPipeSMs ? want : kPipeSMs);
  const auto kernel = al ? residual_norm_fwd_kernel<DT, K, true, ROWS> : residual_norm_fwd_kernel<DT, K, false, ROWS>;
  kernel<<<grid, kResThreads, stages * per_stage + kept, s>>>(p, o, warps, stages, keep);
  return launch_result();
}

template <int DT, bool ROWS>
cudaError_t run(const ResidualNormParams& p, const ResidualNormOut& o, cudaStream_t s) {
  constexpr int W = Elem<DT>::W;
  const int units = (p.D + W - 1) / W, es = elem_bytes(DT);
  if (units > 2 * kPipeUnits) {
    const auto kernel = p.param_dtype == kDtypeF32 ? residual_norm_fwd_wide_kernel<DT, kDtypeF32>
                                                   : residual_norm_fwd_wide_kernel<DT, DT>;
    kernel<<<p.N, kWideThreads, 0, s>>>(p, o);
    return launch_result();
  }
  auto row_ok = [&](const void* base, long long stride) {
    return base == nullptr || (aligned16(base) && (stride * es) % 16 == 0);
  };
  const bool al = p.D % W == 0 && row_ok(p.x, p.x_stride) && row_ok(p.branch, p.b_stride) &&
                  (p.gate_kind == kGateRows ? row_ok(p.gate, p.gate_stride) : aligned16(p.gate)) &&
                  aligned16(p.post_weight) && aligned16(p.weight) && aligned16(o.s) && aligned16(o.h);
  if (units > kPipeUnits) return rows<DT, 4, ROWS>(p, o, 16, al, s);
  // three vectors per thread, two where ragged rows' slots take a fifth more room
  const ResShape q = res_shape(units, p.D % W == 0 ? 3 : 2);
  if (q.K == 1) return rows<DT, 1, ROWS>(p, o, q.warps, al, s);
  if (q.K == 2) return rows<DT, 2, ROWS>(p, o, q.warps, al, s);
  return rows<DT, 3, ROWS>(p, o, q.warps, al, s);
}

template <int DT, int K>
cudaError_t allow() {
  cudaError_t e = cudaSuccess;
  const void* const kernels[4] = {
      reinterpret_cast<const void*>(residual_norm_fwd_kernel<DT, K, true, false>),
      reinterpret_cast<const void*>(residual_norm_fwd_kernel<DT, K, false, false>),
      reinterpret_cast<const void*>(residual_norm_fwd_kernel<DT, K, true, true>),
      reinterpret_cast<const void*>(residual_norm_fwd_kernel<DT, K, false, true>)};
  for (const void* k : kernels)
    if (e == cudaSuccess) e = note_cuda(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kResSmem));
  return e;
}

template <int DT>
cudaError_t setup() {
  cudaError_t e = allow<DT, 1>();
  if (e == cudaSuccess) e = allow<DT, 2>();
  if (e == cudaSuccess) e = allow<DT, 3>();
  if (e == cudaSuccess) e = allow<DT, 4>();
  return e;
}

}  // namespace

cudaError_t residual_norm_fwd_setup() {
  cudaError_t e = setup<kDtypeF32>();
  if (e == cudaSuccess) e = setup<kDtypeBF16>();
  if (e == cudaSuccess) e = setup<kDtypeF16>();
  return e;
}

cudaError_t launch_residual_norm_fwd(const ResidualNormParams& p, const ResidualNormOut& o, cudaStream_t s) {
  const bool rows = p.gate_kind == kGateRows;
  if (p.dtype == kDtypeF32) return rows ? run<kDtypeF32, true>(p, o, s) : run<kDtypeF32, false>(p, o, s);
  if (p.dtype == kDtypeBF16) return rows ? run<kDtypeBF16, true>(p, o, s) : run<kDtypeBF16, false>(p, o, s);
  return rows ? run<kDtypeF16, true>(p, o, s) : run<kDtypeF16, false>(p, o, s);
}

}  // namespace llp
