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
//   reduce  a warp takes 8 or 16 places of the sorted order and 64 vectors of the columns.
//           It streams those rows of grad_out through its own ring in shared memory
//           (cp.async, 6 or 12 rows), and writes a table row whenever its tokens end.  A row
//           of more than 32 tokens is cut into chunks, and where it has more than 16, those
//           into groups, whose lengths depend on its count alone; the warp that finishes a
//           group's last chunk joins them in ascending order, and the one that finishes the
//           last group the groups.  Other CTAs of the same launch write the zero rows.
//
// Measured, bf16, tokens of a 1 / (id + 1) distribution: 16384 tokens x 2688 into 131072
// rows 115 us (6.9 TB/s, the measured copy peak); added to 128256 rows of 4096, 49 us
// (5.0 TB/s, 75%: 9.2 us are the sort, and the reduce launch runs at 94%); fp32, 2049 x
// 1001 into 50257 rows 38 us (82%; the sort 5.9).  Where the longest row decides, 65600 x
// 512 into 101 rows 46 us, of which 19 are the sort (checks at every place and chunks of
// the square root of the count, without groups: 75).  Rows of an odd number of 16-bit elements:
// 16384 x 1001 into 50257 rows 39.4 us, added 41.0 (x 1000: 30.1, 24.9).
#include "elem.cuh"

namespace llp {

namespace {

__device__ __forceinline__ bool token_ok(long long t, long long V, long long ignore_index) {
  return t != ignore_index && t >= 0 && t < V;
}

// ---------------------------------------------------------------- lookup

constexpr int kFwdWarps = 8;
constexpr int kFwdLoads = 4;  // vectors per lane, all in flight together

// One warp per row and chunk of at most 32 * kFwdLoads vectors (2 KB).  Bound by memory:
// 16384 rows of 2688 bf16 take 21.3 us, 87% of the measured copy peak on the rows written
// and the distinct ones read, 65600 rows 72.4 (94%); 32 rows 1.6 us, one launch.  Two vectors
// per lane 23.3 and 84.5; six, or a row's chunks side by side in the grid, 21.1 and 74.7.
// Odd rows of 16 bits: 16384 x 1001 19.0 us, x 1000 9.7.
template <int DT, bool AL>
__global__ void __launch_bounds__(32 * kFwdWarps) embedding_fwd_kernel(const long long* __restrict__ tokens,
                                                                       const typename Elem<DT>::T* __restrict__ weight,
                                                                       int N, int V, int D, int chunk, float scale,
                                                                       long long ignore_index,
                                                                       typename Elem<DT>::T* __restrict__ out) {
  using S = Slot<DT, AL>;
  constexpr int W = Elem<DT>::W;
  const long long n = static_cast<long long>(blockIdx.x) * kFwdWarps + (threadIdx.x >> 5);
  if (n >= N) return;
  const int u0 = blockIdx.y * chunk + (threadIdx.x & 31);
  const int u1 = min(static_cast<int>(blockIdx.y + 1) * chunk, (D + W - 1) / W);
  const long long t = __ldg(tokens + n);
  const bool ok = token_ok(t, V, ignore_index);
  const typename Elem<DT>::T* const row = weight + (ok ? static_cast<size_t>(t) * D : 0);
  typename Elem<DT>::T* const o = out + static_cast<size_t>(n) * D;
  uint4 r[kFwdLoads];
#pragma unroll
  for (int k = 0; k < kFwdLoads; ++k) {
    const int u = u0 + 32 * k;
    r[k] = make_uint4(0, 0, 0, 0);
    if (ok && u < u1) r[k] = S::load(row + u * W, min(D - u * W, W), weight, weight + static_cast<size_t>(V) * D);
  }
#pragma unroll
  for (int k = 0; k < kFwdLoads; ++k) {
    const int u = u0 + 32 * k;
    if (u >= u1) break;
    float v[W];
    Elem<DT>::unpack(r[k], v);
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = ok ? v[i] * scale : 0.f;
    S::store(o + u * W, Elem<DT>::pack(v), min(D - u * W, W));
  }
}

// ---------------------------------------------------------------- gradient: sort

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;  // each scans a span of the tokens
constexpr int kSortSets = kSortWarps / 2;      // two spans share a set of counters: fewer to clear and to add up
constexpr int kSortShift = 7;         // log2 of the CTAs that share the table's rows: 128, more for large tables
constexpr int kSortMaxRange = 2048;   // rows of one CTA
constexpr int kSortList = 512;        // tokens of its rows that a warp notes as it scans
constexpr int kSortLoads = 8;         // tokens per lane in flight
constexpr int kSortSmem = 224 * 1024;
constexpr int kWindowShift = 5;
constexpr int kWindow = 1 << kWindowShift;  // shortest chunk of a long row

// A place of the sorted order: the token n, its row v, and the places [begin, end) of that
// row.  The sign bits say, of n, that it is the row's last token, and of v, that the row has
// more than kWindow.
using Place = int4;
constexpr int kFlag = static_cast<int>(0x80000000u);

// CTA b owns the rows v with v mod owners = b: frequent tokens, whose ids often lie
// together, are spread over the CTAs (with contiguous ranges one of them had 57% of the
// tokens of a 1 / (id + 1) distribution, and the launch took 17 us where it then took 9.5).
// Above 262144 rows there are 256 CTAs, 512 above 524288, and one SM has room for one: 16384 x
// 2688 added takes 38.2 us at 131072 rows, 40.6 at 262144, 43.1 at 262145, 55.0 at 524289.
struct SortPlan {
  int shift, owners, range;  // log2 of the CTAs; rows of each, a multiple of 32
  int warps, span, list;     // scanning warps; tokens of each (a multiple of 32), tokens that it notes
  size_t smem;
};

SortPlan sort_plan(long long N, long long V) {
  SortPlan p;
  p.shift = kSortShift;
  while (((V - 1) >> p.shift) >= kSortMaxRange) ++p.shift;
  p.owners = 1 << p.shift;
  p.range = static_cast<int>((((V - 1) >> p.shift) + 32) / 32 * 32);
  const long long w = (N + 255) / 256;  // at least 256 tokens per warp
  p.warps = static_cast<int>(w < kSortWarps ? w : kSortWarps);
  p.span = static_cast<int>(((N + p.warps - 1) / p.warps + 31) / 32 * 32);
  const size_t counters = static_cast<size_t>(p.range) * ((p.warps + 1) / 2 + 2) * sizeof(int);
  const size_t room = (kSortSmem - counters) / (p.warps * sizeof(int));
  p.list = static_cast<int>(room < kSortList ? room : kSortList);
  if (p.list > p.span) p.list = p.span;
  p.smem = counters + static_cast<size_t>(p.list) * p.warps * sizeof(int);
  return p;
}

// Chunks of a row of `count` tokens: 32 * 2^s places for at most 2^14 * 8^s tokens.  A chunk's
// places are added one after another, so are the chunks of a group, and so are the groups:
// with about as many of each none is long.
__device__ __forceinline__ int chunk_shift(int count) {  // log2 of the places
  return kWindowShift + (32 - __clz((count - 1) >> 14) + 2) / 3;
}
// log2 of the chunks of a group: all of them, where they are few.
__device__ __forceinline__ int group_shift(int chunks) {
  return chunks <= 16 ? 4 : (32 - __clz(chunks - 1)) / 2;
}

// Measured, tokens of a 1 / (id + 1) distribution, 131072 rows: 16384 tokens 9.2 us, bound by
// latency: the scan is about 2 us of it, the counters and their sums 2, placing the tokens 1.5
// to 2.5, the launch the rest.  2049 tokens and 50257 rows: 5.9 us.  65600 tokens: 19 us, most
// of it the scan's instructions, every CTA's over all tokens.  Zeroing a part of the table, or
// fetching a part of grad_out into L2, while it waits: both measured, neither pays.
__global__ void __launch_bounds__(kSortThreads, 1) embedding_sort_kernel(const long long* __restrict__ tokens, int N,
                                                                         int V, long long ignore_index, int shift,
                                                                         int range, int warps, int span, int list,
                                                                         Place* __restrict__ places,
                                                                         unsigned* __restrict__ named,
                                                                         int* __restrict__ arrivals, int num_arrivals,
                                                                         int* __restrict__ total) {
  extern __shared__ int4 sm4[];
  const int sets = (warps + 1) / 2;
  int* const count = reinterpret_cast<int*>(sm4);  // [sets][range]
  int* const first = count + sets * range;         // [range] first place of each row
  int* const last = first + range;                 // [range] one past its last place
  unsigned* const noted = reinterpret_cast<unsigned*>(last + range);  // [warps][list]: place in the span, row in the range
  __shared__ int warp_sum[kSortWarps], warp_low[kSortWarps], warp_hits[kSortWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const unsigned self = blockIdx.x, mask = (1u << shift) - 1, below = (1u << lane) - 1;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int i = blockIdx.x * kSortThreads + tid; i < num_arrivals; i += gridDim.x * kSortThreads) arrivals[i] = 0;
  for (int i = tid; i < sets * range / 4; i += kSortThreads) sm4[i] = make_int4(0, 0, 0, 0);  // range % 32 == 0

  // Calls take(place in the span, valid, row) for the tokens of a span in ascending order, a warp's
  // 32 at a time.
  const unsigned skipped = ignore_index >= 0 && ignore_index < V ? static_cast<unsigned>(ignore_index) : ~0u;
  auto scan = [&](int which, auto&& take) {
    const unsigned t0 = static_cast<unsigned>(which) * span;
    const unsigned count_of = t0 < static_cast<unsigned>(N) ? min(static_cast<unsigned>(span), N - t0) : 0;
    const uint2* const src = reinterpret_cast<const uint2*>(tokens) + t0 + lane;  // low and high word
    auto one = [&](unsigned at, const uint2& t) {
      take(at, t.y == 0 && t.x < static_cast<unsigned>(V) && t.x != skipped, t.x);
    };
    unsigned b = 0;
    for (; b + 32 * kSortLoads <= count_of; b += 32 * kSortLoads) {
      uint2 t[kSortLoads];
#pragma unroll
      for (int k = 0; k < kSortLoads; ++k) t[k] = __ldg(src + b + 32 * k);
#pragma unroll
      for (int k = 0; k < kSortLoads; ++k) one(b + 32 * k + lane, t[k]);
    }
    if (b < count_of) {
      uint2 t[kSortLoads];
#pragma unroll
      for (int k = 0; k < kSortLoads; ++k)
        t[k] = b + 32 * k + lane < count_of ? __ldg(src + b + 32 * k) : make_uint2(~0u, ~0u);
#pragma unroll
      for (int k = 0; k < kSortLoads; ++k)
        if (b + 32 * k < count_of) one(b + 32 * k + lane, t[k]);
    }
  };

  int low = 0, hits = 0;
  if (warp < warps) {
    unsigned* const mine = noted + warp * list;
    scan(warp, [&](unsigned at, bool ok, unsigned v) {
      const unsigned owner = v & mask;
      const bool in = ok && owner == self;
      low += ok && owner < self;
      const unsigned act = __ballot_sync(0xffffffffu, in);
      if (act == 0) return;
      const int h = hits + __popc(act & below);
      if (in && h < list) mine[h] = at << 11 | v >> shift;  // used when all of them fit and at < 2^21
      hits += __popc(act);
    });
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) low += __shfl_xor_sync(0xffffffffu, low, off);
  if (lane == 0) {
    warp_low[warp] = low;
    warp_hits[warp] = hits;
  }
  __syncthreads();
  // Calls take(is one, token, row in the range) for this CTA's tokens in a set's spans, in ascending order.
  auto own_tokens = [&](int set, auto&& take) {
    for (int w = 2 * set; w < min(2 * set + 2, warps); ++w) {
      const int n = warp_hits[w];
      const unsigned t0 = static_cast<unsigned>(w) * span;
      if (n <= list && span <= (1 << 21)) {
        for (int h = 0; h < n; h += 32) {
          const unsigned e = h + lane < n ? noted[w * list + h + lane] : 0;
          take(h + lane < n, t0 + (e >> 11), e & 2047);
        }
      } else {  // more than were noted: scan again
        scan(w, [&](unsigned at, bool ok, unsigned v) { take(ok && (v & mask) == self, t0 + at, v >> shift); });
      }
    }
  };
  int* const mine = count + warp * range;
  if (warp < sets) {
    own_tokens(warp, [&](bool in, unsigned, unsigned r) {
      if (in) atomicAdd(mine + r, 1);
    });
  }
  __syncthreads();

  // per row: exclusive prefix over the sets; over the rows: exclusive scan
  const int per = (range + kSortThreads - 1) / kSortThreads;  // 1 or 2 rows per thread
  int own = 0;
  for (int i = 0; i < per; ++i) {
    const int r = tid * per + i;
    if (r < range) {
      int run = 0;
      for (int w0 = 0; w0 < sets; w0 += 8) {
        int c[8];
#pragma unroll
        for (int w = 0; w < 8; ++w) c[w] = w0 + w < sets ? count[(w0 + w) * range + r] : 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          if (w0 + w < sets) count[(w0 + w) * range + r] = run;
          run += c[w];
        }
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
  int base = warp_low[lane] + (lane < warp ? warp_sum[lane] : 0);
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) base += __shfl_xor_sync(0xffffffffu, base, off);
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
    if (lane == 0) named[(self * range + r) >> 5] = m;
  }

  // each token to its place: its row's, its set's, then its own among the set's
  if (warp >= sets) return;
  own_tokens(warp, [&](bool in, unsigned n, unsigned r) {
    const unsigned act = __ballot_sync(0xffffffffu, in);
    if (act == 0) return;
    unsigned same = act;  // the lanes with this lane's row, bit by bit
    for (int bit = 1; bit < range; bit <<= 1) {
      const bool set = (r & bit) != 0;
      const unsigned with = __ballot_sync(0xffffffffu, set);
      same &= set ? with : ~with;
    }
    const int seen = in ? mine[r] : 0;
    __syncwarp();
    if (in) {
      if ((same & below) == 0) mine[r] = seen + __popc(same);
      const int begin = first[r], end = last[r], at = begin + seen + __popc(same & below);
      places[at] = make_int4(static_cast<int>(n) | (at + 1 == end ? kFlag : 0),
                             static_cast<int>(r << shift | self) | (end - begin > kWindow ? kFlag : 0), begin, end);
    }
    __syncwarp();
  });
}

// ---------------------------------------------------------------- gradient: reduce

constexpr int kTile = 64;  // places that a warp holds in shared memory: place b at b % kTile
constexpr int kPer = 2;    // vectors per lane
constexpr int kJoin = 3;   // partial sums loaded together: two cost the join more, four the others registers

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
  int* arrivals;   // [2 * windows][slices] of a long row's groups of chunks, [windows][slices] of its groups
  float* part;     // [2 * windows][units * W]
  long long windows;
  int stride;
  int N, V, D;
  int slices, slice_units;  // vectors of a slice: at most kPer per lane
  int per_warp;             // places whose chunks a warp takes
  unsigned warps;           // that reduce; the CTAs behind them write the zero rows
  int shift, range;         // of the sort
  int zero_rows;            // table rows that a CTA of those looks after: 4, 8, 16 or 32
  float scale;
};

// ACC: grad_weight's row is added to.  Its vectors are fetched with the row's last token --
// EARLY, unless a vector's words can hold its neighbours' elements, which another thread
// may be writing: those are read element by element when they are needed.
template <int DT, bool AL, bool ACC>
struct ReduceShape {
  static constexpr bool EARLY = ACC && !Slot<DT, AL>::FIVE;
  static constexpr int KINDS = EARLY ? 2 : 1;   // vectors in a stage: grad_out's, grad_weight's
  static constexpr int STAGES = EARLY ? 6 : 12;  // tokens of the ring
  static constexpr int BATCH = EARLY ? 3 : 4;    // of a long run added together, the others in flight
  // Warps of a CTA, each working alone: one, so that none holds the room of the others that are
  // done; four where the CTAs behind write zero rows, of which one-warp CTAs are too many.
  static constexpr int WARPS = ACC ? 1 : 4;
  static constexpr int BYTES = STAGES * KINDS * kPer * Slot<DT, AL>::BYTES;  // of the ring per thread
};

template <int DT, bool AL, bool ACC>
__global__ void __launch_bounds__(32 * ReduceShape<DT, AL, ACC>::WARPS, 1) embedding_reduce_kernel(
    ReduceParams p, const typename Elem<DT>::T* __restrict__ grad_out, typename Elem<DT>::T* grad_weight) {
  using S = Slot<DT, AL>;
  using T = typename Elem<DT>::T;
  using Shape = ReduceShape<DT, AL, ACC>;
  constexpr int W = Elem<DT>::W, H = W / 2, STAGES = Shape::STAGES, KINDS = Shape::KINDS;
  constexpr int kWarps = Shape::WARPS, threads = 32 * kWarps;
  extern __shared__ uint4 ring[];  // [STAGES][KINDS][kPer][threads]; then the slots' fifth words
  __shared__ Place tiles[kWarps][kTile];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int units = (p.D + W - 1) / W;
  const unsigned reduce_ctas = (p.warps + kWarps - 1) / kWarps;

  if (blockIdx.x >= reduce_ctas) {  // zero rows, one warp per row
    const unsigned block = blockIdx.x - reduce_ctas;
    const unsigned owner = block & ((1u << p.shift) - 1), r0 = (block >> p.shift) * p.zero_rows;
    const unsigned m = load_written(p.named + (owner * p.range + r0) / 32) >> (r0 & 31);
    for (int i = warp; i < p.zero_rows; i += kWarps) {
      const long long v = static_cast<long long>(r0 + i) << p.shift | owner;
      if (v >= p.V || ((m >> i) & 1)) continue;
      T* const row = grad_weight + static_cast<size_t>(v) * p.D;
      // elements up to a 128-byte line, vectors, elements
      const int head = AL ? 0 : min(p.D, static_cast<int>((128 - (reinterpret_cast<uintptr_t>(row) & 127)) % 128 / sizeof(T)));
      const int body = (p.D - head) / W;
      for (int c = lane; c < head; c += 32) row[c] = Elem<DT>::put(0.f);
      for (int u = lane; u < body; u += 32) reinterpret_cast<uint4*>(row + head)[u] = make_uint4(0, 0, 0, 0);
      if (!AL && head + body * W + lane < p.D) row[head + body * W + lane] = Elem<DT>::put(0.f);
    }
    return;
  }

  const unsigned w = blockIdx.x * kWarps + warp;
  if (w >= p.warps) return;
  const unsigned block = w / p.slices, p0 = block * p.per_warp;
  const int slice = w - block * p.slices;
  // The first places, read without waiting for their number: those past it hold nothing yet.
  const unsigned M = load_written(p.total);
  auto raw_place = [&](unsigned b) {
    return b < static_cast<unsigned>(p.N) ? load_written(p.places + b) : make_int4(0, 0, 0, 0);
  };
  auto place = [&](unsigned b) { return b < M ? load_written(p.places + b) : make_int4(0, 0, 0, 0); };
  const Place first = raw_place(p0 + lane), second = raw_place(p0 + 32 + lane);
  Place coming = raw_place(p0 + kTile + lane);  // takes the room of the 32 places that are done with
  if (p0 >= M) return;
  Place* const tile = tiles[warp];
  tile[(p0 + lane) % kTile] = first;
  tile[(p0 + 32 + lane) % kTile] = second;
  // the chunks that begin in [p0, p0 + per_warp): the places [h0, h1)
  unsigned h0 = p0, h1;
  {
    const unsigned q = min(p0 + p.per_warp, M) - 1;
    const unsigned e_begin = __shfl_sync(0xffffffffu, first.z, 0), e_end = __shfl_sync(0xffffffffu, first.w, 0);
    const unsigned f_begin = __shfl_sync(0xffffffffu, first.z, q - p0), f_end = __shfl_sync(0xffffffffu, first.w, q - p0);
    const unsigned C = 1u << chunk_shift(e_end - e_begin), off = (p0 - e_begin) & (C - 1);
    if (off != 0) h0 = min(p0 - off + C, e_end);
    if (h0 > q) return;
    const unsigned Cq = 1u << chunk_shift(f_end - f_begin);
    h1 = min(q - ((q - f_begin) & (Cq - 1)) + Cq, f_end);
  }
  __syncwarp();
  // this lane's vectors
  int col[kPer], left[kPer];
  const int here = min(p.slice_units, units - slice * p.slice_units);
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int u = slice * p.slice_units + 32 * k + lane;
    const bool on = 32 * k + lane < here;
    col[k] = on ? u * W : 0;
    left[k] = on ? min(p.D - u * W, W) : 0;
  }
  const T* const ghi = grad_out + static_cast<long long>(p.N - 1) * p.stride + p.D;
  const T* const whi = grad_weight + static_cast<size_t>(p.V) * p.D;
  uint32_t* const fifth = reinterpret_cast<uint32_t*>(ring + STAGES * KINDS * kPer * threads);
  constexpr int STEP = KINDS * kPer * threads;  // of a stage
  auto row_of = [&](int n) { return grad_out + static_cast<long long>(n & ~kFlag) * p.stride; };
  auto table_row = [&](int v) { return grad_weight + static_cast<long long>(v & ~kFlag) * p.D; };
  auto issue = [&](unsigned b, int at) {
    if (b < h1) {
      const Place e = tile[b % kTile];
      const T* const g = row_of(e.x);
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (left[k] > 0) S::copy(ring + at + k * threads, fifth + at + k * threads, g + col[k], left[k], grad_out, ghi);
      if (Shape::EARLY && e.x < 0 && e.y >= 0) {
        const T* const o = table_row(e.y);
#pragma unroll
        for (int k = 0; k < kPer; ++k)
          if (left[k] > 0)
            S::copy(ring + at + (kPer + k) * threads, fifth + at + (kPer + k) * threads, o + col[k], left[k], grad_weight,
                    whi);
      }
    }
    copy_commit();
  };
#pragma unroll 1
  for (int s = 0; s < STAGES; ++s) issue(h0 + s, s * STEP + tid);
  int out = tid;       // the ring's place of b
  unsigned base = p0;  // places [base, base + kTile) are in the tile
  auto step = [&](int at) { return at + STEP < STAGES * STEP ? at + STEP : at + STEP - STAGES * STEP; };
  auto refill = [&](unsigned b) {
    if (b - base >= 32) {
      __syncwarp();
      tile[(base + kTile + lane) % kTile] = coming;
      base += 32;
      coming = place(base + kTile + lane);
      __syncwarp();
    }
  };
  F2 acc[kPer][H];
  auto add = [&](unsigned b, int at) {
    const bool gshift = S::FIVE && S::shifted(row_of(tile[b % kTile].x));
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      F2 v[H];
      unpack2<DT, W>(S::read(ring + at + k * threads, fifth + at + k * threads, gshift, left[k]), v);
#pragma unroll
      for (int i = 0; i < H; ++i) acc[k][i] = add2(acc[k][i], v[i]);
    }
  };

  // One run of places, a row's or a long row's chunk, at a time; h1 is the end of one.
  for (unsigned b = h0; b < h1;) {
    const Place e = tile[b % kTile];
    const unsigned head = b, begin = e.z, end = e.w;
    const bool cut = e.y < 0;
    const int cs = cut ? chunk_shift(end - begin) : 0;
    const unsigned stop = cut ? min(end, b + (1u << cs)) : end;
#pragma unroll
    for (int k = 0; k < kPer; ++k)
#pragma unroll
      for (int i = 0; i < H; ++i) acc[k][i] = f2(0.f);
    // several places together while there are: one after another, the instructions of a place
    // wait for one another
    while (b + Shape::BATCH < stop) {
      copy_wait<STAGES - Shape::BATCH>();
      int at = out;
#pragma unroll
      for (int j = 0; j < Shape::BATCH; ++j) {
        add(b + j, at);
        at = step(at);
      }
      at = out;
#pragma unroll
      for (int j = 0; j < Shape::BATCH; ++j) {
        issue(b + STAGES + j, at);
        at = step(at);
      }
      out = at;
      b += Shape::BATCH;
      refill(b);
    }
    uint4 old[kPer];
    for (; b < stop; ++b) {
      copy_wait<STAGES - 1>();
      add(b, out);
      if (Shape::EARLY && b + 1 == stop) {
#pragma unroll
        for (int k = 0; k < kPer; ++k)
          old[k] = S::read(ring + out + (kPer + k) * threads, fifth + out + (kPer + k) * threads, false, left[k]);
      }
      issue(b + STAGES, out);
      out = step(out);
      refill(b + 1);
    }
    if (__builtin_expect(cut, 0)) {
      // The chunks' sums meet in memory: the warp that comes last of a group adds its chunks, and
      // the last of those the groups, each in ascending order.
      const int chunks = ((end - begin - 1) >> cs) + 1, shift = group_shift(chunks);
      const int group = (head - begin) >> (cs + shift);
      const bool more = chunks > 1 << shift;
      unsigned from = begin + (group << (cs + shift)), own = head;
      int members = min(1 << shift, chunks - (group << shift)), apart = cs;
      int* arrivals = p.arrivals + slot_of(from, group == 0) * p.slices;
      bool joined;
      while (true) {
        float* const part = p.part + slot_of(own, own == begin) * units * W;
#pragma unroll
        for (int k = 0; k < kPer; ++k)
          if (left[k] > 0) {
#pragma unroll
            for (int i = 0; i < H; i += 2)
              reinterpret_cast<float4*>(part + col[k])[i / 2] =
                  make_float4(acc[k][i].x, acc[k][i].y, acc[k][i + 1].x, acc[k][i + 1].y);
          }
        __threadfence();
        __syncwarp();
        int before = 0;
        if (lane == 0) before = atomicAdd(arrivals + slice, 1);
        joined = __shfl_sync(0xffffffffu, before, 0) == members - 1;
        if (!joined) break;
        __threadfence();
#pragma unroll
        for (int k = 0; k < kPer; ++k)
#pragma unroll
          for (int i = 0; i < H; ++i) acc[k][i] = f2(0.f);
        for (int c0 = 0; c0 < members; c0 += kJoin) {
          float4 v[kJoin][kPer][H / 2];  // loaded together
#pragma unroll
          for (int c = 0; c < kJoin; ++c) {
            const unsigned at = from + (min(c0 + c, members - 1) << apart);
            const float* const q = p.part + slot_of(at, at == begin) * units * W;
#pragma unroll
            for (int k = 0; k < kPer; ++k)
#pragma unroll
              for (int i = 0; i < H / 2; ++i) v[c][k][i] = load_written(reinterpret_cast<const float4*>(q + col[k]) + i);
          }
#pragma unroll
          for (int c = 0; c < kJoin; ++c) {
            if (c0 + c < members) {
#pragma unroll
              for (int k = 0; k < kPer; ++k)
#pragma unroll
                for (int i = 0; i < H / 2; ++i) {
                  acc[k][2 * i] = add2(acc[k][2 * i], f2(v[c][k][i].x, v[c][k][i].y));
                  acc[k][2 * i + 1] = add2(acc[k][2 * i + 1], f2(v[c][k][i].z, v[c][k][i].w));
                }
            }
          }
        }
        if (!more || apart != cs) break;
        // the groups of the row
        own = from;
        from = begin;
        apart = cs + shift;
        members = ((chunks - 1) >> shift) + 1;
        arrivals = p.arrivals + (p.windows * 2 + begin / kWindow) * p.slices;
      }
      if (!joined) continue;
    }
    T* const o = table_row(e.y);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (left[k] <= 0) continue;
      F2 v[H];
#pragma unroll
      for (int i = 0; i < H; ++i) v[i] = f2(0.f);
      if (ACC) {
        if (!Shape::EARLY || cut) old[k] = S::load_changed(o + col[k], left[k]);
        unpack2<DT, W>(old[k], v);
      }
#pragma unroll
      for (int i = 0; i < H; ++i) v[i] = ACC ? fma2(acc[k][i], f2(p.scale), v[i]) : mul2(acc[k][i], f2(p.scale));
      S::store(o + col[k], pack2<DT, W>(v), left[k]);
    }
  }
  copy_wait<0>();
}

// ---------------------------------------------------------------- launches

inline size_t up256(size_t n) { return (n + 255) / 256 * 256; }

struct BwdLayout {
  size_t places, named, total, arrivals, part, bytes;
  long long windows, num_arrivals;
};

BwdLayout bwd_layout(long long N, long long V, long long D) {
  BwdLayout L;
  L.windows = (N + kWindow - 1) / kWindow;
  L.num_arrivals = L.windows * 3 * ((D + 255) / 256);  // slices have 256 columns (fp32) or 512
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t here = at;
    at += up256(n);
    return here;
  };
  L.places = take(static_cast<size_t>(N) * sizeof(Place));
  const SortPlan sp = sort_plan(N, V);
  L.named = take(static_cast<size_t>(sp.owners) * (sp.range / 32) * sizeof(unsigned));
  L.total = take(sizeof(int));
  L.arrivals = take(static_cast<size_t>(L.num_arrivals) * sizeof(int));
  L.part = take(static_cast<size_t>(L.windows) * 2 * ((D + 7) / 8 * 8) * sizeof(float));
  L.bytes = at;
  return L;
}

template <int DT, bool AL>
cudaError_t fwd(const EmbeddingParams& p, const void* weight, void* out, cudaStream_t s) {
  using T = typename Elem<DT>::T;
  const int units = (p.D + Elem<DT>::W - 1) / Elem<DT>::W;
  const int chunks = (units + 32 * kFwdLoads - 1) / (32 * kFwdLoads);
  const dim3 grid(static_cast<unsigned>((static_cast<long long>(p.N) + kFwdWarps - 1) / kFwdWarps), chunks);
  embedding_fwd_kernel<DT, AL><<<grid, 32 * kFwdWarps, 0, s>>>(p.tokens, static_cast<const T*>(weight), p.N, p.V, p.D,
                                                               (units + chunks - 1) / chunks, p.scale, p.ignore_index,
                                                               static_cast<T*>(out));
  return launch_result();
}

template <int DT, bool AL, bool ACC>
cudaError_t reduce(ReduceParams r, const void* grad_out, void* grad_weight, cudaStream_t s) {
  using T = typename Elem<DT>::T;
  const int units = (r.D + Elem<DT>::W - 1) / Elem<DT>::W;
  r.slices = (units + 32 * kPer - 1) / (32 * kPer);
  r.slice_units = (units + r.slices - 1) / r.slices;
  // Places per warp: 16, or 8 where that leaves too few warps (16384 x 4096, accumulating: 50.1
  // us with 8, 54 with 16; 65600 x 2688: 123 and 117).
  using Shape = ReduceShape<DT, AL, ACC>;
  r.per_warp = (static_cast<long long>(r.N) + 15) / 16 * r.slices < 152 * (ACC ? 64 : 32) ? 8 : 16;
  r.warps = static_cast<unsigned>((static_cast<long long>(r.N) + r.per_warp - 1) / r.per_warp * r.slices);
  // about 32 KB of zeros per CTA: with 128 KB the last of few CTAs had the GPU to themselves
  r.zero_rows = 32;
  while (r.zero_rows > 4 && static_cast<long long>(r.zero_rows) * r.D * elem_bytes(DT) > 48 * 1024) r.zero_rows /= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((r.warps + Shape::WARPS - 1) / Shape::WARPS + (ACC ? 0 : r.range / r.zero_rows << r.shift));
  cfg.blockDim = dim3(32 * Shape::WARPS);
  cfg.dynamicSmemBytes = static_cast<size_t>(32 * Shape::WARPS) * Shape::BYTES;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return note_cuda(cudaLaunchKernelEx(&cfg, embedding_reduce_kernel<DT, AL, ACC>, r, static_cast<const T*>(grad_out),
                                      static_cast<T*>(grad_weight)));
}

template <int DT>
cudaError_t reduce_any(const ReduceParams& r, bool al, bool accumulate, const void* grad_out, void* grad_weight,
                       cudaStream_t s) {
  if (al)
    return accumulate ? reduce<DT, true, true>(r, grad_out, grad_weight, s)
                      : reduce<DT, true, false>(r, grad_out, grad_weight, s);
  return accumulate ? reduce<DT, false, true>(r, grad_out, grad_weight, s)
                    : reduce<DT, false, false>(r, grad_out, grad_weight, s);
}

template <int DT>
cudaError_t allow() {
  const void* const kernels[4] = {reinterpret_cast<const void*>(embedding_reduce_kernel<DT, true, true>),
                                  reinterpret_cast<const void*>(embedding_reduce_kernel<DT, true, false>),
                                  reinterpret_cast<const void*>(embedding_reduce_kernel<DT, false, true>),
                                  reinterpret_cast<const void*>(embedding_reduce_kernel<DT, false, false>)};
  for (const void* k : kernels) {
    const cudaError_t e = note_cuda(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * 1024));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t embedding_setup() {
  cudaError_t e = note_cuda(cudaFuncSetAttribute(embedding_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 kSortSmem));
  if (e == cudaSuccess) e = allow<kDtypeBF16>();
  if (e == cudaSuccess) e = allow<kDtypeF32>();
  if (e == cudaSuccess) e = allow<kDtypeF16>();
  return e;
}

size_t embedding_bwd_workspace(long long N, long long V, long long D) { return bwd_layout(N, V, D).bytes; }

cudaError_t launch_embedding_fwd(const EmbeddingParams& p, const void* weight, void* out, cudaStream_t s) {
  const bool al = aligned16(weight) && aligned16(out) && (static_cast<long long>(p.D) * elem_bytes(p.dtype)) % 16 == 0;
  if (p.dtype == kDtypeBF16)
    return al ? fwd<kDtypeBF16, true>(p, weight, out, s) : fwd<kDtypeBF16, false>(p, weight, out, s);
  if (p.dtype == kDtypeF16)
    return al ? fwd<kDtypeF16, true>(p, weight, out, s) : fwd<kDtypeF16, false>(p, weight, out, s);
  return al ? fwd<kDtypeF32, true>(p, weight, out, s) : fwd<kDtypeF32, false>(p, weight, out, s);
}

cudaError_t launch_embedding_bwd(const EmbeddingParams& p, const void* grad_out, long long stride, int accumulate,
                                 void* grad_weight, void* workspace, cudaStream_t s) {
  const BwdLayout L = bwd_layout(p.N, p.V, p.D);
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  const int es = elem_bytes(p.dtype);
  const bool al = aligned16(grad_out) && aligned16(grad_weight) && (static_cast<long long>(p.D) * es) % 16 == 0 &&
                  (stride * es) % 16 == 0;
  const SortPlan sp = sort_plan(p.N, p.V);
  Place* const places = reinterpret_cast<Place*>(ws + L.places);
  unsigned* const named = reinterpret_cast<unsigned*>(ws + L.named);
  int* const total = reinterpret_cast<int*>(ws + L.total);
  int* const arrivals = reinterpret_cast<int*>(ws + L.arrivals);
  embedding_sort_kernel<<<sp.owners, kSortThreads, sp.smem, s>>>(p.tokens, p.N, p.V, p.ignore_index, sp.shift,
                                                                 sp.range, sp.warps, sp.span, sp.list, places, named, arrivals,
                                                                 static_cast<int>(L.num_arrivals), total);
  const cudaError_t e = launch_result();
  if (e != cudaSuccess) return e;
  ReduceParams r = {};
  r.places = places;
  r.total = total;
  r.named = named;
  r.arrivals = arrivals;
  r.part = reinterpret_cast<float*>(ws + L.part);
  r.windows = L.windows;
  r.stride = static_cast<int>(stride);
  r.N = p.N;
  r.V = p.V;
  r.D = p.D;
  r.shift = sp.shift;
  r.range = sp.range;
  r.scale = p.scale;
  if (p.dtype == kDtypeBF16) return reduce_any<kDtypeBF16>(r, al, accumulate != 0, grad_out, grad_weight, s);
  if (p.dtype == kDtypeF16) return reduce_any<kDtypeF16>(r, al, accumulate != 0, grad_out, grad_weight, s);
  return reduce_any<kDtypeF32>(r, al, accumulate != 0, grad_out, grad_weight, s);
}

}  // namespace llp
