// Token embedding: lookup with scaling, and its gradient.
//
//   out[n, :]         = scale * weight[t_n, :]
//   grad_weight[v, :] = scale * sum over n with t_n = v, ascending, of grad_out[n, :]
//
// The gradient is two launches:
//   sort    every CTA owns a range of table rows.  It scans all tokens (in L2)
//           and counts, per warp and row, those in its range; the ones below it
//           give the place of its first token in the sorted order, so the CTAs
//           need nothing from one another.  A second scan puts each token at its
//           place: sorted by row, ascending within a row.
//   reduce  CTAs take 32 places of the sorted order and a slice of the columns,
//           stream those rows of grad_out with eight loads in flight per thread,
//           and write a table row whenever its tokens end.  A row of more than
//           64 tokens is cut into chunks whose length depends on its count
//           alone; the CTA that finishes the last chunk of a row joins them in
//           ascending order.  Other CTAs of the same launch write the zero rows.
#include "elem.cuh"

namespace llp {

namespace {

__device__ __forceinline__ bool token_ok(long long t, long long V, long long ignore_index) {
  return t != ignore_index && t >= 0 && t < V;
}

// ---------------------------------------------------------------- lookup

constexpr int kFwdWarps = 8;
constexpr int kFwdLoads = 4;  // units per lane, all in flight together

// One warp per row and chunk of 32 * kFwdLoads units (2 KB of vectors).
template <int DT, bool VEC>
__global__ void __launch_bounds__(32 * kFwdWarps) embedding_fwd_kernel(const long long* __restrict__ tokens,
                                                                       const typename Elem<DT>::T* __restrict__ weight,
                                                                       int N, int V, int D, int chunk_units,
                                                                       float scale, long long ignore_index,
                                                                       typename Elem<DT>::T* __restrict__ out) {
  using U = Unit<DT, VEC>;
  const long long n = static_cast<long long>(blockIdx.x) * kFwdWarps + (threadIdx.x >> 5);
  if (n >= N) return;
  const int units = D / U::W;
  const int u0 = blockIdx.y * chunk_units;
  const int u1 = min(u0 + chunk_units, units);
  const long long t = __ldg(tokens + n);
  const bool ok = token_ok(t, V, ignore_index);
  const typename U::T* w = weight + (ok ? static_cast<size_t>(t) * D : 0);
  typename U::T* o = out + static_cast<size_t>(n) * D;
  typename U::Raw r[kFwdLoads];
#pragma unroll
  for (int k = 0; k < kFwdLoads; ++k) {
    const int u = u0 + 32 * k + (threadIdx.x & 31);
    r[k] = (ok && u < u1) ? U::load(w + static_cast<size_t>(u) * U::W) : U::zero();
  }
#pragma unroll
  for (int k = 0; k < kFwdLoads; ++k) {
    const int u = u0 + 32 * k + (threadIdx.x & 31);
    if (u >= u1) break;
    float v[U::W];
    U::unpack(r[k], v);
#pragma unroll
    for (int i = 0; i < U::W; ++i) v[i] = ok ? v[i] * scale : 0.f;
    U::store(o + static_cast<size_t>(u) * U::W, v);
  }
}

// ---------------------------------------------------------------- gradient: sort

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortOwners = 152;      // CTAs that share the table's rows, one per SM
constexpr int kSortMaxRange = 1536;   // rows of one CTA: 32 warps x 1536 counters fill its shared memory
constexpr int kSortLoads = 8;         // tokens per lane in flight
constexpr int kWindow = 64;           // shortest chunk of a long row

// A place of the sorted order: the token n, its row v, and the places [begin, end) of that row.
using Place = int4;

struct SortPlan {
  int owners, range, warps, span;  // CTAs; rows per CTA (multiple of 32); scanning warps; tokens per warp
  size_t smem;
};

SortPlan sort_plan(long long N, long long V) {
  SortPlan p;
  long long range = ((V + kSortOwners - 1) / kSortOwners + 31) / 32 * 32;
  if (range > kSortMaxRange) range = kSortMaxRange;
  p.range = static_cast<int>(range);
  p.owners = static_cast<int>((V + range - 1) / range);
  const long long w = (N + 255) / 256;  // at least 256 tokens per warp
  p.warps = static_cast<int>(w < kSortWarps ? w : kSortWarps);
  p.span = static_cast<int>(((N + p.warps - 1) / p.warps + 31) / 32 * 32);
  p.smem = static_cast<size_t>(p.range) * (p.warps + 2) * sizeof(int);
  return p;
}

// First place of the chunk arithmetic: chunks of 64 * 2^s places, at most 64 of them.
__device__ __forceinline__ int chunk_of(int count) {
  return kWindow << (count > 4096 ? 32 - __clz((count - 1) >> 12) : 0);
}

__global__ void __launch_bounds__(kSortThreads, 1) embedding_sort_kernel(const long long* __restrict__ tokens, int N,
                                                                         int V, long long ignore_index, int range,
                                                                         int warps, int span, Place* __restrict__ places,
                                                                         unsigned* __restrict__ named,
                                                                         int* __restrict__ arrivals, int num_arrivals,
                                                                         int* __restrict__ total) {
  extern __shared__ int sm[];
  int* count = sm;                       // [warps][range]
  int* first = count + warps * range;    // [range] first place of each row
  int* last = first + range;             // [range] one past its last place
  __shared__ int warp_sum[kSortWarps], warp_low[kSortWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long lo = static_cast<long long>(blockIdx.x) * range;
  const long long hi = min(lo + range, static_cast<long long>(V));
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int i = blockIdx.x * kSortThreads + tid; i < num_arrivals; i += gridDim.x * kSortThreads) arrivals[i] = 0;
  for (int i = tid; i < warps * range; i += kSortThreads) count[i] = 0;
  __syncthreads();

  // this warp's tokens, in ascending order
  const long long t0 = static_cast<long long>(warp) * span;
  const long long t1 = min(t0 + span, static_cast<long long>(N));
  int* mine = count + warp * range;
  int low = 0;
  if (warp < warps) {
    for (long long b = t0; b < t1; b += 32 * kSortLoads) {
      long long t[kSortLoads];
#pragma unroll
      for (int k = 0; k < kSortLoads; ++k) {
        const long long n = b + 32 * k + lane;
        t[k] = n < t1 ? __ldg(tokens + n) : -1;
      }
#pragma unroll
      for (int k = 0; k < kSortLoads; ++k) {
        const bool ok = t[k] >= 0 && t[k] < hi && t[k] != ignore_index;
        if (ok && t[k] >= lo) atomicAdd(mine + static_cast<int>(t[k] - lo), 1);
        low += ok && t[k] < lo;
      }
    }
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) low += __shfl_xor_sync(0xffffffffu, low, off);
  if (lane == 0) warp_low[warp] = low;
  __syncthreads();

  // per row: exclusive prefix over the warps; over the rows: exclusive scan
  const int per = (range + kSortThreads - 1) / kSortThreads;  // 1 or 2 rows per thread
  int own = 0;
  for (int i = 0; i < per; ++i) {
    const int r = tid * per + i;
    if (r < range) {
      int run = 0;
      for (int w = 0; w < warps; ++w) {
        const int c = count[w * range + r];
        count[w * range + r] = run;
        run += c;
      }
      last[r] = run;  // the row's count for now
      own += run;
    }
  }
  int incl = own;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += o;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int base = 0;
  for (int w = 0; w < kSortWarps; ++w) base += warp_low[w] + (w < warp ? warp_sum[w] : 0);
  int at = base + incl - own;
  for (int i = 0; i < per; ++i) {
    const int r = tid * per + i;
    if (r < range) {
      const int c = last[r];
      first[r] = at;
      at += c;
      last[r] = at;
    }
  }
  if (blockIdx.x == gridDim.x - 1 && tid == kSortThreads - 1) *total = at;
  __syncthreads();
  for (int r = tid; r < range; r += kSortThreads) {  // range and kSortThreads are multiples of 32
    const unsigned m = __ballot_sync(0xffffffffu, last[r] > first[r]);
    if (lane == 0) named[(lo + r) >> 5] = m;
  }

  if (warp < warps) {
    const unsigned below = (1u << lane) - 1;
    for (long long b = t0; b < t1; b += 32 * kSortLoads) {
      long long t[kSortLoads];
#pragma unroll
      for (int k = 0; k < kSortLoads; ++k) {
        const long long n = b + 32 * k + lane;
        t[k] = n < t1 ? __ldg(tokens + n) : -1;
      }
#pragma unroll
      for (int k = 0; k < kSortLoads; ++k) {
        const bool in = t[k] >= lo && t[k] < hi && t[k] != ignore_index;
        const unsigned act = __ballot_sync(0xffffffffu, in);
        if (act == 0) continue;
        if (in) {
          const int r = static_cast<int>(t[k] - lo);
          const unsigned same = __match_any_sync(act, r);
          const int seen = mine[r];
          __syncwarp(act);
          if ((same & below) == 0) mine[r] = seen + __popc(same);
          const int begin = first[r];
          places[begin + seen + __popc(same & below)] =
              make_int4(static_cast<int>(b + 32 * k + lane), static_cast<int>(t[k]), begin, last[r]);
        }
        __syncwarp();
      }
    }
  }
}

// ---------------------------------------------------------------- gradient: reduce

constexpr int kPlaces = 32;   // places whose chunks a CTA takes
constexpr int kTile = 64;     // places held in shared memory
constexpr int kDeep = 8;      // rows in flight

// Slot of a long row's chunk among the partial sums.  Two chunks of one row begin at
// least kWindow places apart, and two long rows' first chunks (or two later ones)
// never begin in the same window: a window holds one first and one later chunk at most.
__device__ __forceinline__ long long slot_of(unsigned place, bool is_first) {
  return 2ll * (place / kWindow) + (is_first ? 1 : 0);
}

struct ReduceParams {
  const Place* places;
  const int* total;
  const unsigned* named;
  int* arrivals;   // [windows][slices]
  float* part;     // [2 * windows][D]
  long long stride;
  int V, D;
  int slices, slice_units;
  int reduce_ctas;
  float scale;
};

template <int DT, bool VEC, bool ACC, int T>
__global__ void __launch_bounds__(T) embedding_reduce_kernel(ReduceParams p,
                                                             const typename Elem<DT>::T* __restrict__ grad_out,
                                                             typename Elem<DT>::T* __restrict__ grad_weight) {
  using U = Unit<DT, VEC>;
  constexpr int W = U::W;
  constexpr int K = VEC ? 1 : 4;  // units per thread
  __shared__ Place tile[kTile];
  __shared__ int is_last;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int units = p.D / W;

  if (static_cast<int>(blockIdx.x) >= p.reduce_ctas) {  // zero rows: 32 table rows, one warp per row
    const int block = blockIdx.x - p.reduce_ctas;
    const unsigned m = __ldg(p.named + block);
    for (int i = threadIdx.x >> 5; i < 32; i += T / 32) {
      const long long v = 32ll * block + i;
      if (v >= p.V || ((m >> i) & 1)) continue;
      typename U::T* o = grad_weight + static_cast<size_t>(v) * p.D;
      for (int u = threadIdx.x & 31; u < units; u += 32) U::store_raw(o + static_cast<size_t>(u) * W, U::zero());
    }
    return;
  }

  const int slice = blockIdx.x % p.slices;
  const unsigned p0 = static_cast<unsigned>(blockIdx.x / p.slices) * kPlaces;
  const unsigned M = __ldg(p.total);
  if (p0 >= M) return;
  unsigned tile0 = p0;
  auto fill = [&]() {
    for (unsigned i = threadIdx.x; i < kTile; i += T)
      if (tile0 + i < M) tile[i] = __ldg(p.places + tile0 + i);
    __syncthreads();
  };
  fill();
  // the chunks that begin in [p0, p0 + kPlaces): the places [h0, h1)
  unsigned h0 = p0, h1;
  {
    const Place e = tile[0];
    const unsigned C = chunk_of(e.w - e.z), off = (p0 - e.z) % C;
    if (off != 0) h0 = min(p0 - off + C, static_cast<unsigned>(e.w));
    const unsigned q = min(p0 + kPlaces, M) - 1;
    if (h0 > q) return;
    const Place f = tile[q - p0];
    const unsigned Cq = chunk_of(f.w - f.z);
    h1 = min(q - (q - f.z) % Cq + Cq, static_cast<unsigned>(f.w));
  }
  const int ubase = slice * p.slice_units;
  const int uend = min(ubase + p.slice_units, units);
  size_t col[K];
  bool on[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int u = ubase + k * T + static_cast<int>(threadIdx.x);
    on[k] = u < uend;
    col[k] = static_cast<size_t>(on[k] ? u : 0) * W;
  }
  float acc[K][W];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < W; ++i) acc[k][i] = 0.f;

  for (unsigned b = h0; b < h1; b += kDeep) {
    if (b + kDeep > tile0 + kTile) {
      __syncthreads();
      tile0 = b;
      fill();
    }
    typename U::Raw g[kDeep][K], old[ACC ? kDeep : 1][K];
#pragma unroll
    for (int j = 0; j < kDeep; ++j) {
      if (b + j < h1) {
        const Place e = tile[b + j - tile0];
        const typename U::T* row = grad_out + e.x * p.stride;
#pragma unroll
        for (int k = 0; k < K; ++k) g[j][k] = on[k] ? U::load(row + col[k]) : U::zero();
        if (ACC && b + j + 1 == static_cast<unsigned>(e.w) && e.w - e.z <= kWindow) {
          const typename U::T* o = grad_weight + static_cast<size_t>(e.y) * p.D;
#pragma unroll
          for (int k = 0; k < K; ++k)
            old[ACC ? j : 0][k] = on[k] ? *reinterpret_cast<const typename U::Raw*>(o + col[k]) : U::zero();
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kDeep; ++j) {
      const unsigned at = b + j;
      if (at >= h1) break;
      const Place e = tile[at - tile0];
      const unsigned begin = e.z, end = e.w;
      const unsigned C = chunk_of(e.w - e.z);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        float v[W];
        U::unpack(g[j][k], v);
#pragma unroll
        for (int i = 0; i < W; ++i) acc[k][i] += v[i];
      }
      const bool row_ends = at + 1 == end;
      if (!row_ends && (at + 1 - begin) % C != 0) continue;
      typename U::T* o = grad_weight + static_cast<size_t>(e.y) * p.D;
      bool write = end - begin <= C;
      if (!write) {  // a chunk of a long row
        const unsigned head = at - (at - begin) % C;
        float* part = p.part + slot_of(head, head == begin) * p.D;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int i = 0; i < W; ++i)
            if (on[k]) part[col[k] + i] = acc[k][i];
        const int chunks = (end - begin + C - 1) / C;
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0)
          is_last = atomicAdd(p.arrivals + static_cast<long long>(begin / kWindow) * p.slices + slice, 1) == chunks - 1;
        __syncthreads();
        write = is_last;
        if (write) {
          __threadfence();
#pragma unroll
          for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < W; ++i) acc[k][i] = 0.f;
          for (int c = 0; c < chunks; ++c) {
            const float* q = p.part + slot_of(begin + c * C, c == 0) * p.D;
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
              for (int i = 0; i < W; ++i)
                if (on[k]) acc[k][i] += __ldcg(q + col[k] + i);
          }
        }
      }
      if (write) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
          if (!on[k]) continue;
          float v[W];
          if (ACC) {
            U::unpack(end - begin <= C ? old[ACC ? j : 0][k] : *reinterpret_cast<const typename U::Raw*>(o + col[k]), v);
#pragma unroll
            for (int i = 0; i < W; ++i) v[i] = fmaf(p.scale, acc[k][i], v[i]);
          } else {
#pragma unroll
            for (int i = 0; i < W; ++i) v[i] = p.scale * acc[k][i];
          }
          U::store(o + col[k], v);
        }
      }
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < W; ++i) acc[k][i] = 0.f;
    }
  }
}

// ---------------------------------------------------------------- launches

inline size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Column slices of the reduce launch: T threads, one vector or four elements each.
int slices_of(int units, int per_cta) { return (units + per_cta - 1) / per_cta; }

struct BwdLayout {
  size_t places, named, total, arrivals, part, bytes;
  long long windows;
};

// Columns of the narrowest slice of any type and alignment (one slice when rows have fewer).
constexpr int kMinSlice = 512;

BwdLayout bwd_layout(long long N, long long V, long long D) {
  BwdLayout L;
  L.windows = (N + kWindow - 1) / kWindow;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t here = at;
    at += up256(n);
    return here;
  };
  L.places = take(static_cast<size_t>(N) * sizeof(Place));
  L.named = take((static_cast<size_t>(V) / 32 + kSortMaxRange) * sizeof(unsigned));
  L.total = take(sizeof(int));
  L.arrivals = take(static_cast<size_t>(L.windows) * ((D + kMinSlice - 1) / kMinSlice) * sizeof(int));
  L.part = take(static_cast<size_t>(L.windows) * 2 * D * sizeof(float));
  L.bytes = at;
  return L;
}

template <int DT, bool VEC>
cudaError_t fwd(const EmbeddingParams& p, const void* weight, void* out, cudaStream_t s) {
  using U = Unit<DT, VEC>;
  const int units = p.D / U::W;
  const int chunks = (units + 32 * kFwdLoads - 1) / (32 * kFwdLoads);
  const dim3 grid((p.N + kFwdWarps - 1) / kFwdWarps, chunks);
  embedding_fwd_kernel<DT, VEC><<<grid, 32 * kFwdWarps, 0, s>>>(
      p.tokens, static_cast<const typename U::T*>(weight), p.N, p.V, p.D, (units + chunks - 1) / chunks, p.scale,
      p.ignore_index, static_cast<typename U::T*>(out));
  return launch_result();
}

template <int DT, bool VEC, bool ACC, int T>
cudaError_t reduce(ReduceParams r, long long N, int units, const void* grad_out, void* grad_weight, cudaStream_t s) {
  using Te = typename Elem<DT>::T;
  r.slices = slices_of(units, VEC ? T : 4 * T);
  r.slice_units = (units + r.slices - 1) / r.slices;
  r.reduce_ctas = static_cast<int>((N + kPlaces - 1) / kPlaces * r.slices);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(r.reduce_ctas + (ACC ? 0 : (r.V + 31) / 32));
  cfg.blockDim = dim3(T);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return note_cuda(cudaLaunchKernelEx(&cfg, embedding_reduce_kernel<DT, VEC, ACC, T>, r,
                                      static_cast<const Te*>(grad_out), static_cast<Te*>(grad_weight)));
}

template <int DT, bool VEC>
cudaError_t reduce_any(const ReduceParams& r, long long N, bool accumulate, const void* grad_out, void* grad_weight,
                       cudaStream_t s) {
  const int units = r.D / Unit<DT, VEC>::W;
  // rows of few units take one-warp CTAs
  if (units <= (VEC ? 32 : 128))
    return accumulate ? reduce<DT, VEC, true, 32>(r, N, units, grad_out, grad_weight, s)
                      : reduce<DT, VEC, false, 32>(r, N, units, grad_out, grad_weight, s);
  return accumulate ? reduce<DT, VEC, true, 128>(r, N, units, grad_out, grad_weight, s)
                    : reduce<DT, VEC, false, 128>(r, N, units, grad_out, grad_weight, s);
}

}  // namespace

cudaError_t embedding_setup() {
  const int bytes = kSortMaxRange * (kSortWarps + 2) * static_cast<int>(sizeof(int));
  return note_cuda(cudaFuncSetAttribute(embedding_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
}

size_t embedding_bwd_workspace(long long N, long long V, long long D) { return bwd_layout(N, V, D).bytes; }

cudaError_t launch_embedding_fwd(const EmbeddingParams& p, const void* weight, void* out, cudaStream_t s) {
  const bool vec = aligned16(weight) && aligned16(out) && (static_cast<long long>(p.D) * elem_bytes(p.dtype)) % 16 == 0;
  if (p.dtype == kDtypeBF16) return vec ? fwd<kDtypeBF16, true>(p, weight, out, s) : fwd<kDtypeBF16, false>(p, weight, out, s);
  if (p.dtype == kDtypeF16) return vec ? fwd<kDtypeF16, true>(p, weight, out, s) : fwd<kDtypeF16, false>(p, weight, out, s);
  return vec ? fwd<kDtypeF32, true>(p, weight, out, s) : fwd<kDtypeF32, false>(p, weight, out, s);
}

cudaError_t launch_embedding_bwd(const EmbeddingParams& p, const void* grad_out, long long stride, int accumulate,
                                 void* grad_weight, void* workspace, cudaStream_t s) {
  const BwdLayout L = bwd_layout(p.N, p.V, p.D);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const int es = elem_bytes(p.dtype);
  const bool vec = aligned16(grad_out) && aligned16(grad_weight) && (static_cast<long long>(p.D) * es) % 16 == 0 &&
                   (stride * es) % 16 == 0;
  const SortPlan sp = sort_plan(p.N, p.V);
  ReduceParams r = {};
  r.places = reinterpret_cast<Place*>(ws + L.places);
  r.named = reinterpret_cast<unsigned*>(ws + L.named);
  r.total = reinterpret_cast<int*>(ws + L.total);
  r.arrivals = reinterpret_cast<int*>(ws + L.arrivals);
  r.part = reinterpret_cast<float*>(ws + L.part);
  r.stride = stride;
  r.V = p.V;
  r.D = p.D;
  r.scale = p.scale;
  const int num_arrivals = static_cast<int>(L.windows * ((p.D + kMinSlice - 1) / kMinSlice));
  embedding_sort_kernel<<<sp.owners, kSortThreads, sp.smem, s>>>(
      p.tokens, p.N, p.V, p.ignore_index, sp.range, sp.warps, sp.span, reinterpret_cast<Place*>(ws + L.places),
      reinterpret_cast<unsigned*>(ws + L.named), reinterpret_cast<int*>(ws + L.arrivals), num_arrivals,
      reinterpret_cast<int*>(ws + L.total));
  const cudaError_t e = launch_result();
  if (e != cudaSuccess) return e;
  const bool acc = accumulate != 0;
  if (p.dtype == kDtypeBF16)
    return vec ? reduce_any<kDtypeBF16, true>(r, p.N, acc, grad_out, grad_weight, s)
               : reduce_any<kDtypeBF16, false>(r, p.N, acc, grad_out, grad_weight, s);
  if (p.dtype == kDtypeF16)
    return vec ? reduce_any<kDtypeF16, true>(r, p.N, acc, grad_out, grad_weight, s)
               : reduce_any<kDtypeF16, false>(r, p.N, acc, grad_out, grad_weight, s);
  return vec ? reduce_any<kDtypeF32, true>(r, p.N, acc, grad_out, grad_weight, s)
             : reduce_any<kDtypeF32, false>(r, p.N, acc, grad_out, grad_weight, s);
}

}  // namespace llp
