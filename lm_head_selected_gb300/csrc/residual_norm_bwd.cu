// Gradient of the RMS norms around a block.  With c = s * rstd, a = grad_h * weight, k = branch * post_rstd:
//
//   G = grad_s + rstd * (a - c * sum(a c) / D)                    grad_x
//   e = scale * gate * G * post_weight,  grad_branch = post_rstd * (e - k * sum(e k) / D)
//   sums over rows: grad_h * c for the weight, and S = scale * G * k (times the row's own gate), of which
//   the gradients of post_weight and of a gate per column are multiples: gate * S and post_weight * S.
//
// One pass over the rows gives all of them.  A group of warps owns a row at a time, up to three vectors per
// thread, which it copies itself into a ring of rows, so that the rows to come are in flight.  The row is
// read from the ring twice: for sum(a c), and for G, whose products stay in registers while sum(e k) is
// joined.  As a thread's columns are the same in every row, it keeps their sums in registers; a second
// launch joins the CTAs' sums in ascending order.  Rows of 1025 to 2048 vectors take four vectors per
// thread and a third reading in place of the registers; wider ones take plain kernels: one CTA per row,
// one thread per column over a range of rows.
//
// Bound by memory: four tensors read (five with a gate of the rows' own) and two (three) written.  Measured in
// a captured graph: 16384 x 4096 bf16 134 us (6.0 TB/s, 89% of the measured copy peak; plain kernels 1047);
// 2049 x 1001 fp32 with a gate of the rows' own 23.4 us (2.8 TB/s: odd rows come in 4-byte copies, whose
// accesses to shared memory, not HBM, are the bound).
#include "residual_norm.cuh"

namespace llp {

namespace {

// part: [gridDim.x][2][D], the CTA's sums of grad_h * c and of S over its rows; null to skip them.
// Vectors per lane: K = ceil(units / (32 * warps)); those from kFull<K> on may lie past the row's end.
// What no copy writes stays 0 in the ring and adds nothing to any sum; so do inputs that are not there.
template <int DT, int K, bool AL, bool ROWS>
__global__ void __launch_bounds__(kResThreads, 1) residual_norm_bwd_kernel(const ResidualNormParams p,
                                                                           const ResidualNormGrads o, int warps,
                                                                           int stages, bool keep_wide,
                                                                           float* __restrict__ part) {
  using T = typename Elem<DT>::T;
  constexpr int W = Elem<DT>::W, H = W / 2, N_IN = ROWS ? 5 : 4, threads = kResThreads;
  constexpr bool HOLD = K < 4;
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
  const bool f32 = p.param_dtype == kDtypeF32, post = p.post_weight != nullptr;
  const bool has_gs = p.gs != nullptr, has_w = p.weight != nullptr;
  const bool has_b = p.branch != nullptr && (post || p.gate_kind != kGateNone);  // else k is of no use
  for (int i = 0; i < stages * N_IN; ++i)
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int t = i % N_IN;
      const bool there = t == 0 ? has_gs : t <= 2 ? has_w : t == 3 ? has_b : true;
      if (!AL || !on(k) || !there) mine[(i * K + k) * threads] = make_uint4(0, 0, 0, 0);
      if (S::FIVE) fifth[(i * K + k) * threads] = 0;  // read wherever a row starts in the middle of a word
    }
  auto copy = [&](int t, const void* base, long long stride, unsigned n, int stage) {
    const T* const lo = static_cast<const T*>(base);
    const T* const src = lo + static_cast<long long>(n) * stride + first * W;
    const T* const hi = lo + static_cast<long long>(p.N - 1) * stride + p.D;
    const int at = stage * pitch + t * K * threads;
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (on(k)) S::copy(mine + at + k * threads, fifth + at + k * threads, src + k * width * W, left(k), lo, hi);
  };
  auto issue = [&](unsigned n, int stage) {  // row n, if there is one
    if (n < r1) {
      if (has_gs) copy(0, p.gs, p.gs_stride, n, stage);
      if (has_w) {
        copy(1, p.gh, p.gh_stride, n, stage);
        copy(2, p.x, p.x_stride, n, stage);
      }
      if (has_b) copy(3, p.branch, p.b_stride, n, stage);
      if (ROWS) copy(4, p.gate, p.gate_stride, n, stage);
    }
    copy_commit();
  };
  for (int s = 0; s < stages - 1; ++s) issue(r0 + s * step, s);
  if (keep) keep_coefficients<DT, AL>(kept, p);
  F2 aw[K][H], as[K][H];  // this thread's columns' sums
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int j = 0; j < H; ++j) aw[k][j] = as[k][j] = f2(0.f);
  __syncthreads();
  const float inv = 1.f / static_cast<float>(p.D);
  int stage = 0;
  unsigned i = 0;
  for (unsigned n = r0; n < r1; n += step, ++i) {
    const float r = has_w ? __ldg(o.rstd + n) : 0.f, pr = post ? __ldg(o.post_rstd + n) : 1.f;
    issue(n + (stages - 1) * step, stage == 0 ? stages - 1 : stage - 1);
    copies_left(stages - 1);
    const int at = stage * pitch;
    stage = stage + 1 == stages ? 0 : stage + 1;
    auto clear = [](F2 (&v)[H]) {
#pragma unroll
      for (int j = 0; j < H; ++j) v[j] = f2(0.f);
    };
    auto read = [&](int t, int k, const void* base, long long stride, F2 (&v)[H]) {
      const bool shift = S::shifted(static_cast<const T*>(base) + static_cast<long long>(n) * stride);
      const int slot = at + (t * K + k) * threads;
      unpack2<DT, W>(S::read(mine + slot, fifth + slot, shift, left(k)), v);
    };
    // Past the row's end coefficients are 0: the first vector's in their place might be infinite.  Up to three
    // vectors per thread the callers step over those; around four, loads from memory among them, a branch
    // for each cost a twentieth (4096 x 16384 bf16 264 us, 251 without).
    auto weight = [&](int k, F2 (&v)[H]) {
      const int u = HOLD || on(k) ? first + k * width : 0;
      if (keep)
        kept_vector<W>(kept, 1, units, u, v);
      else
        param_vector<DT, W, AL>(p.weight, f32, u * W, on(k) ? left(k) : min(p.D, W), v);
      if (!HOLD && !on(k)) clear(v);
    };
    auto coefficient = [&](int k, F2 (&v)[H]) {
      const int u = HOLD || on(k) ? first + k * width : 0;
      if (keep)
        kept_vector<W>(kept, 0, units, u, v);
      else
        coefficient_vector<DT, W, AL>(p, f32, u * W, on(k) ? left(k) : min(p.D, W), v);
      if (!HOLD && !on(k)) clear(v);
    };
    // sum(a c) / D, and the weight's columns
    float minus = 0.f;
    if (has_w) {
      F2 t = f2(0.f);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (HOLD && !on(k)) continue;
        F2 a[H], c[H], w[H];
        read(1, k, p.gh, p.gh_stride, a);
        read(2, k, p.x, p.x_stride, c);
        weight(k, w);
#pragma unroll
        for (int j = 0; j < H; ++j) {
          c[j] = mul2(c[j], f2(r));
          a[j] = mul2(a[j], c[j]);
          aw[k][j] = add2(aw[k][j], a[j]);
          t = fma2(a[j], w[j], t);
        }
      }
      minus = -group_sum(sum2(t), red[0][i & 1] + group * warps, warp, warps, 1 + group) * inv;
    }
    // G of a vector
    auto upstream = [&](int k, F2 (&G)[H]) {
      read(0, k, p.gs, p.gs_stride, G);
      if (!has_w) return;
      F2 a[H], c[H], w[H];
      read(1, k, p.gh, p.gh_stride, a);
      read(2, k, p.x, p.x_stride, c);
      weight(k, w);
#pragma unroll
      for (int j = 0; j < H; ++j)
        G[j] = fma2(fma2(mul2(c[j], f2(r)), f2(minus), mul2(a[j], w[j])), f2(r), G[j]);
    };
    // scale * gate * post_weight * G of a vector (held in G's place), k = branch * post_rstd
    auto scaled = [&](int k, F2 (&G)[H], F2 (&b)[H], bool columns) {
      read(3, k, p.branch, p.b_stride, b);
      F2 c[H], g[H];
      coefficient(k, c);
      if (ROWS) read(4, k, p.gate, p.gate_stride, g);
#pragma unroll
      for (int j = 0; j < H; ++j) {
        b[j] = mul2(b[j], f2(pr));
        if (columns) {
          const F2 u = mul2(G[j], b[j]);
          as[k][j] = ROWS ? fma2(u, g[j], as[k][j]) : add2(as[k][j], u);
        }
        G[j] = mul2(G[j], c[j]);
        if (ROWS) {
          c[j] = mul2(G[j], b[j]);  // the gate's own gradient
          G[j] = mul2(G[j], g[j]);
        }
      }
      if (ROWS && columns && o.ggate != nullptr && on(k))
        S::store(static_cast<T*>(o.ggate) + static_cast<size_t>(n) * p.D + (first + k * width) * W, pack2<DT, W>(c), left(k));
    };
    F2 e[HOLD ? K : 1][H], b[HOLD ? K : 1][H], t = f2(0.f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (HOLD && !on(k)) continue;
      F2(&ev)[H] = e[HOLD ? k : 0], (&bv)[H] = b[HOLD ? k : 0];
      upstream(k, ev);
      if (o.gx != nullptr && on(k))
        S::store(static_cast<T*>(o.gx) + static_cast<size_t>(n) * p.D + (first + k * width) * W, pack2<DT, W>(ev), left(k));
      if (p.branch == nullptr) continue;
      scaled(k, ev, bv, true);
#pragma unroll
      for (int j = 0; j < H; ++j) t = fma2(ev[j], bv[j], t);
    }
    if (o.gb == nullptr) continue;
    const float along = post ? -group_sum(sum2(t), red[1][i & 1] + group * warps, warp, warps, 1 + group) * inv : 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (!on(k)) continue;
      F2(&ev)[H] = e[HOLD ? k : 0], (&bv)[H] = b[HOLD ? k : 0];
      if (!HOLD) {
        upstream(k, ev);
        scaled(k, ev, bv, false);
      }
#pragma unroll
      for (int j = 0; j < H; ++j) ev[j] = mul2(fma2(bv[j], f2(along), ev[j]), f2(pr));
      S::store(static_cast<T*>(o.gb) + static_cast<size_t>(n) * p.D + (first + k * width) * W, pack2<DT, W>(ev), left(k));
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
      F2* const out = reinterpret_cast<F2*>(join + (group * 2 * units + first + k * width) * W);
#pragma unroll
      for (int j = 0; j < H; ++j) out[j] = aw[k][j], out[units * H + j] = mul2(as[k][j], f2(p.scale));
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

// ---------------------------------------------------------------- wide rows

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

template <int PT>
cudaError_t join(const ResidualNormParams& p, const ResidualNormGrads& o, const float* part, int parts, cudaStream_t s) {
  residual_norm_join_kernel<PT><<<(2 * p.D + 31) / 32, 32 * kJoinWarps, 0, s>>>(p, o, part, parts);
  return launch_result();
}

// Bytes of a row of the ring, for all threads.
size_t res_bwd_stage(int K, bool rows, int slot) { return static_cast<size_t>(rows ? 5 : 4) * K * kResThreads * slot; }

template <int DT, int PT>
cudaError_t wide(const ResidualNormParams& p, const ResidualNormGrads& o, bool columns, float* part, cudaStream_t s) {
  float* const means = part + static_cast<size_t>(p.N < kParts ? p.N : kParts) * 2 * p.D;
  residual_norm_bwd_wide_x_kernel<DT, PT><<<p.N, kWideThreads, 0, s>>>(p, o, means);
  cudaError_t e = launch_result();
  if (e != cudaSuccess || !columns) return e;
  const int parts = p.N < 64 ? 1 : p.N < 1024 ? p.N / 32 : 32;
  residual_norm_bwd_wide_columns_kernel<DT, PT><<<dim3((p.D + 255) / 256, parts), 256, 0, s>>>(p, o, means, part);
  if ((e = launch_result()) != cudaSuccess) return e;
  return join<PT>(p, o, part, parts, s);
}

template <int DT, int K, bool ROWS>
cudaError_t rows(const ResidualNormParams& p, const ResidualNormGrads& o, int warps, bool al, bool columns, float* part,
                 cudaStream_t s) {
  constexpr int W = Elem<DT>::W;
  const int units = (p.D + W - 1) / W, groups = kResThreads / 32 / warps;
  const size_t per_stage = res_bwd_stage(K, ROWS, al ? 16 : Slot<DT, false>::BYTES);
  size_t kept = static_cast<size_t>(2) * units * W * sizeof(float);
  const bool keep = K < 4 || res_keep(per_stage, kept);
  if (!keep) kept = 0;
  const int stages = res_stages(per_stage, kept);
  const long long want = (static_cast<long long>(p.N) + groups - 1) / groups;
  const int grid = static_cast<int>(want < kPipeSMs ? want : kPipeSMs);
  const auto kernel = al ? residual_norm_bwd_kernel<DT, K, true, ROWS> : residual_norm_bwd_kernel<DT, K, false, ROWS>;
  kernel<<<grid, kResThreads, stages * per_stage + kept, s>>>(p, o, warps, stages, keep, columns ? part : nullptr);
  const cudaError_t e = launch_result();
  if (e != cudaSuccess || !columns) return e;
  return p.param_dtype == kDtypeF32 ? join<kDtypeF32>(p, o, part, grid, s) : join<DT>(p, o, part, grid, s);
}

template <int DT, bool ROWS>
cudaError_t run(const ResidualNormParams& p, const ResidualNormGrads& o, cudaStream_t s) {
  constexpr int W = Elem<DT>::W;
  const int units = (p.D + W - 1) / W, es = elem_bytes(DT);
  float* const part = static_cast<float*>(o.workspace);
  const bool columns = o.gweight != nullptr || o.gpost != nullptr || (o.ggate != nullptr && !ROWS);
  if (units > 2 * kPipeUnits)
    return p.param_dtype == kDtypeF32 ? wide<DT, kDtypeF32>(p, o, columns, part, s) : wide<DT, DT>(p, o, columns, part, s);
  auto row_ok = [&](const void* base, long long stride) {
    return base == nullptr || (aligned16(base) && (stride * es) % 16 == 0);
  };
  const bool al = p.D % W == 0 && row_ok(p.gs, p.gs_stride) && row_ok(p.gh, p.gh_stride) && row_ok(p.x, p.x_stride) &&
                  row_ok(p.branch, p.b_stride) && (ROWS ? row_ok(p.gate, p.gate_stride) : aligned16(p.gate)) &&
                  aligned16(p.post_weight) && aligned16(p.weight) && aligned16(o.gx) && aligned16(o.gb) &&
                  (!ROWS || aligned16(o.ggate));
  if (units > kPipeUnits) return rows<DT, 4, ROWS>(p, o, 16, al, columns, part, s);
  // three vectors per thread where two rows of the ring still fit beside the coefficients, else two
  const size_t kept = static_cast<size_t>(2) * units * W * sizeof(float);
  const bool three = p.D % W == 0 && kept + 2 * res_bwd_stage(3, ROWS, 16) <= static_cast<size_t>(kResSmem);
  const ResShape q = res_shape(units, three ? 3 : 2);
  if (q.K == 1) return rows<DT, 1, ROWS>(p, o, q.warps, al, columns, part, s);
  if (q.K == 2) return rows<DT, 2, ROWS>(p, o, q.warps, al, columns, part, s);
  return rows<DT, 3, ROWS>(p, o, q.warps, al, columns, part, s);
}

template <int DT, int K>
cudaError_t allow() {
  cudaError_t e = cudaSuccess;
  const void* const kernels[4] = {
      reinterpret_cast<const void*>(residual_norm_bwd_kernel<DT, K, true, false>),
      reinterpret_cast<const void*>(residual_norm_bwd_kernel<DT, K, false, false>),
      reinterpret_cast<const void*>(residual_norm_bwd_kernel<DT, K, true, true>),
      reinterpret_cast<const void*>(residual_norm_bwd_kernel<DT, K, false, true>)};
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

cudaError_t residual_norm_bwd_setup() {
  cudaError_t e = setup<kDtypeF32>();
  if (e == cudaSuccess) e = setup<kDtypeBF16>();
  if (e == cudaSuccess) e = setup<kDtypeF16>();
  return e;
}

size_t residual_norm_bwd_workspace(long long N, long long D) {
  const long long parts = N < kParts ? N : kParts;
  return (static_cast<size_t>(parts) * 2 * D + N) * sizeof(float);
}

cudaError_t launch_residual_norm_bwd(const ResidualNormParams& p, const ResidualNormGrads& o, cudaStream_t s) {
  const bool rows = p.gate_kind == kGateRows;
  if (p.dtype == kDtypeF32) return rows ? run<kDtypeF32, true>(p, o, s) : run<kDtypeF32, false>(p, o, s);
  if (p.dtype == kDtypeBF16) return rows ? run<kDtypeBF16, true>(p, o, s) : run<kDtypeBF16, false>(p, o, s);
  return rows ? run<kDtypeF16, true>(p, o, s) : run<kDtypeF16, false>(p, o, s);
}

}  // namespace llp
