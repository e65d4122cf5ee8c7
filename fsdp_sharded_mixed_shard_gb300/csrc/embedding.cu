/*
 * embedding.cu -- token lookup and the table's gradient (zero_train.h).
 *
 * Lookup: out[t, :] = round16(scale * table[id_t, :]). A warp moves a slice of
 * 256 columns of four tokens at a time: four independent row loads in flight
 * per warp. Bound by memory: 2 dim bytes read and written per token; 32768 x
 * 2048 takes 30 us (9.0 TB/s of tokens, frequent rows coming from L2), 1024 x
 * 768 4.0 us, the time of the call itself.
 *
 * Gradient: grad[v, :] = round16(scale * sum of dy[t, :] over id_t == v). The
 * whole table is written, so the bound is 2 (T + V) dim bytes. Two parts:
 *
 * 1. The ids are sorted, equal ids in the order of their positions, by stable
 *    counting passes over at most 9 bits each (17 bits of id: two passes).
 *    Ids of a warp are ranked by match.any, warps by a scan over their counts.
 *    Up to 8192 ids one cluster of eight CTAs does all passes in one launch
 *    (sort_kernel). Beyond, hist_kernel counts the first pass's digits per
 *    chunk of the ids and scatter_kernel places a chunk's ids and counts the
 *    next pass's digits at the chunk each place belongs to, so each further
 *    pass is one launch. Integer counts: the order of their atomics does not
 *    matter.
 * 2. rows_kernel merges the sorted ids with the table's rows into one list --
 *    token, token, "row done", "row done", token, ... -- and cuts it into
 *    runs of kRun items, so that a run costs the same whether it sums the
 *    tokens of one frequent id or clears rows: item i of the sorted ids is
 *    item i + id_i of the merged list, so a run finds its first token by one
 *    search of all lanes. A warp sums a run's 256-column slice in registers
 *    (eight tokens' loads in flight) and stores each row as it is done; rows
 *    without tokens follow one another in memory and are cleared in 16-byte
 *    blocks whatever their length. An id whose tokens span runs leaves fp32
 *    partial sums in the workspace, which join_kernel adds in run order. The
 *    runs' bounds depend on the ids alone, so the sums do not change from call
 *    to call.
 *    Measured: 16384 x 2048 into 128256 rows 115 us (5.2 TB/s of 592 MB;
 *    rows_kernel alone 96 us, 6.2 TB/s), 8192 x 768 into 50257 rows 36 us, of
 *    which the sort and the join, bound by latency, take about 15. Runs of 64
 *    items took 125 and 39 us; four tokens in flight 120 and 43 us; clearing
 *    the table in a kernel beside the sort 145 and 36 us.
 */
#include "train.cuh"

#include <algorithm>

namespace ze {

using namespace zt;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSlice = 256;    // columns per warp: eight per lane
constexpr int kLookup = 4;     // tokens per warp and step of the lookup
constexpr int kRun = 32;       // items of the merged list per run
constexpr int kBatch = 8;      // dy rows in flight per warp
static_assert(kRun % 32 == 0 && kRun <= 64 && 32 % kBatch == 0, "a run's tokens fit its lanes");

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kDigits = 512;   // 9 bits per pass, one thread per digit
constexpr int kTile = 1024;    // ids ranked at a time
constexpr int kMaxChunks = 64; // chunks (CTAs) per pass
constexpr int kMaxPasses = 3;
static_assert(kDigits == kSortThreads, "one thread per digit");
static_assert(kTile % kSortThreads == 0, "whole rounds");

// the buffers of a call, for their bounds
enum { kTable, kOut, kLookupBuffers };
enum { kDy, kGrad, kParts, kSpans, kGradBuffers };

// A lane's eight neighbouring columns [c, c + 8) of a row; columns past dim
// are 0 (loads) or left alone (stores). kVecRows: rows lie on the 16-byte grid
// and dim is a multiple of 8.
template <bool kVecRows>
__device__ __forceinline__ uint4 load8(const uint16_t* row, int64_t c, int64_t dim,
                                       const Bounds& in) {
  if (!in.holds(row + c, 2 * (dim - c < kVec ? dim - c : kVec), kSiteLoad))
    return make_uint4(0, 0, 0, 0);
  if constexpr (kVecRows)
    return c < dim ? __ldcs(reinterpret_cast<const uint4*>(row + c)) : make_uint4(0, 0, 0, 0);
  if (c + kVec <= dim) return load8_any<false>(row + c);
  uint32_t h[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) h[j] = c + j < dim ? row[c + j] : 0;
  return make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
}

// The warp's slice of a row from column c0 on; all lanes call it.
template <bool kVecRows>
__device__ __forceinline__ void store_slice(uint8_t* stage, uint16_t* row, int64_t c0, int lane,
                                            int64_t dim, const uint4& v, const Bounds& in) {
  if constexpr (kVecRows) {
    const int64_t c = c0 + lane * kVec;
    if (c < dim && in.holds(row + c, 16, kSiteStore))
      __stcs(reinterpret_cast<uint4*>(row + c), v);
  } else {
    const int64_t left = dim - c0;
    store_any(stage, row + c0, left < kSlice ? static_cast<int>(left) : kSlice, lane, v, in);
  }
}

// stages of the CTA's warps for store_slice
template <bool kVecRows>
struct Stages {
  __align__(16) uint8_t of_warp[kVecRows ? 1 : kWarps][kVecRows ? 16 : kStageWarp];
};

// ------------------------------------------------------------------ lookup ----

struct LookupArgs : Checked<kLookupBuffers> {
  const void* tokens;
  const uint16_t* table;
  uint16_t* out;
  int64_t n, vocab, dim, slices, units;
  int32_t token_bytes;
  float scale;
};

template <bool kBf16, bool kVecRows>
__global__ void __launch_bounds__(kThreads) lookup_kernel(const LookupArgs a) {
  pdl_begin();
  __shared__ Stages<kVecRows> stages;
  uint8_t* stage = stages.of_warp[kVecRows ? 0 : threadIdx.x >> 5];
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (unit >= a.units) return;
  const int64_t group = unit / a.slices;
  const int64_t c0 = (unit - group * a.slices) * kSlice;
  const int64_t t0 = group * kLookup;
  uint4 v[kLookup];
#pragma unroll
  for (int k = 0; k < kLookup; ++k) {
    const int64_t t = t0 + k;
    const int64_t id = t < a.n ? load_id(a.tokens, a.token_bytes, t, a.vocab) : -1;
    v[k] = id >= 0 ? load8<kVecRows>(a.table + id * a.dim, c0 + lane * kVec, a.dim,
                                     a.bounds(kTable))
                   : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int k = 0; k < kLookup; ++k) {
    const int64_t t = t0 + k;
    if (t >= a.n) break;
    float f[8];
    widen8<kBf16>(v[k], f);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] *= a.scale;
    store_slice<kVecRows>(stage, a.out + t * a.dim, c0, lane, a.dim, narrow8<kBf16>(f),
                          a.bounds(kOut));
  }
}

// -------------------------------------------------------------------- sort ----

struct SortArgs {
  const void* tokens;            // first pass reads the ids themselves
  const uint32_t* key_in;        // later passes: ids and positions of the pass before
  const uint32_t* pos_in;
  uint32_t* key_out;
  uint32_t* pos_out;
  uint32_t* hist;                // this pass: [kDigits][kMaxChunks]
  uint32_t* hist_next;           // next pass, or NULL
  uint32_t* n_spans;             // cleared for rows_kernel
  int64_t n, vocab, chunk;       // chunk: ids per CTA, a multiple of kTile
  int32_t token_bytes, shift, bits, n_chunks, n_hists;
};

// padding ids sort after the last row
__device__ __forceinline__ uint32_t first_key(const SortArgs& a, int64_t i) {
  const int64_t id = load_id(a.tokens, a.token_bytes, i, a.vocab);
  return static_cast<uint32_t>(id < 0 ? a.vocab : id);
}

// Digits of the first pass, counted per chunk; the other passes' counts are
// cleared for the scatter kernels to add to.
__global__ void __launch_bounds__(kSortThreads) hist_kernel(const SortArgs a) {
  pdl_begin();
  __shared__ uint32_t count[kDigits];
  count[threadIdx.x] = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.n_spans = 0;
  __syncthreads();
  const int64_t lo = blockIdx.x * a.chunk;
  const int64_t hi = lo + a.chunk < a.n ? lo + a.chunk : a.n;
  const uint32_t mask = (1u << a.bits) - 1;
  for (int64_t i = lo + threadIdx.x; i < hi; i += kSortThreads)
    atomicAdd(&count[first_key(a, i) & mask], 1u);
  __syncthreads();
  a.hist[threadIdx.x * kMaxChunks + blockIdx.x] = count[threadIdx.x];
  // the scatter kernels read counts in fours
  if (blockIdx.x == gridDim.x - 1)
    for (int g = gridDim.x; g < kMaxChunks && (g & 3); ++g)
      a.hist[threadIdx.x * kMaxChunks + g] = 0;
  const int total = (a.n_hists - 1) * kDigits * kMaxChunks;
  for (int i = blockIdx.x * kSortThreads + threadIdx.x; i < total; i += gridDim.x * kSortThreads)
    a.hist[kDigits * kMaxChunks + i] = 0;
}

__global__ void __launch_bounds__(kSortThreads) scatter_kernel(const SortArgs a) {
  pdl_begin();
  constexpr int kRounds = kTile / kSortThreads;
  __shared__ uint32_t base[kDigits];               // next free place of each digit
  __shared__ uint32_t of_warp[kSortWarps][kDigits];
  __shared__ uint32_t warp_sum[kSortWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t lo = blockIdx.x * a.chunk;
  const int64_t hi = lo + a.chunk < a.n ? lo + a.chunk : a.n;
  const uint32_t mask = (1u << a.bits) - 1;
  // warp w ranks ids [w, w + 1) * kTile / kSortWarps of a tile
  uint32_t key[kRounds], pos[kRounds], rank[kRounds];
  const auto load = [&](int64_t t0) {
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
      const int64_t i = t0 + (warp * kRounds + k) * 32 + lane;
      key[k] = i >= hi ? 0xFFFFFFFFu : a.key_in ? a.key_in[i] : first_key(a, i);
      pos[k] = i >= hi ? 0 : a.pos_in ? a.pos_in[i] : static_cast<uint32_t>(i);
    }
  };
  load(lo);
  {
    // digit tid: all its ids, and those in the chunks before this one
    const uint4* row = reinterpret_cast<const uint4*>(a.hist + tid * kMaxChunks);
    const int me = blockIdx.x;
    uint32_t all = 0, before = 0;
#pragma unroll 4
    for (int g = 0; g < a.n_chunks; g += 4) {  // counts past n_chunks are 0
      const uint4 c = row[g >> 2];
      all += (c.x + c.y) + (c.z + c.w);
      before += (g < me ? c.x : 0) + (g + 1 < me ? c.y : 0) + (g + 2 < me ? c.z : 0) +
                (g + 3 < me ? c.w : 0);
    }
    uint32_t inc = all;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += y;
    }
    if (lane == 31) warp_sum[warp] = inc;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) of_warp[w][tid] = 0;
    __syncthreads();
    uint32_t lower = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) lower += w < warp ? warp_sum[w] : 0;
    base[tid] = lower + inc - all + before;
  }
  for (int64_t t0 = lo; t0 < hi; t0 += kTile) {
    if (t0 > lo) {
      load(t0);
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) of_warp[w][tid] = 0;
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
      const bool on = t0 + (warp * kRounds + k) * 32 + lane < hi;
      const uint32_t d = (key[k] >> a.shift) & mask;
      const uint32_t same = __match_any_sync(0xffffffffu, on ? d : 0xFFFFFFFFu);
      const uint32_t ahead = __popc(same & ((1u << lane) - 1));
      const uint32_t seen = on ? of_warp[warp][d] : 0;
      __syncwarp();
      if (on && ahead == 0) of_warp[warp][d] = seen + __popc(same);
      __syncwarp();
      rank[k] = seen + ahead;
    }
    __syncthreads();
    {
      uint32_t c[kSortWarps], run = base[tid];
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) c[w] = of_warp[w][tid];
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) {
        of_warp[w][tid] = run;
        run += c[w];
      }
      base[tid] = run;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
      const int64_t i = t0 + (warp * kRounds + k) * 32 + lane;
      if (i >= hi) continue;
      const uint32_t to = of_warp[warp][(key[k] >> a.shift) & mask] + rank[k];
      if (!ZCHECK(to < a.n, kSiteStore, to)) continue;
      a.key_out[to] = key[k];
      a.pos_out[to] = pos[k];
      if (a.hist_next) {
        const uint32_t d = (key[k] >> (a.shift + a.bits)) & mask;
        atomicAdd(&a.hist_next[d * kMaxChunks + to / static_cast<uint32_t>(a.chunk)], 1u);
      }
    }
    __syncthreads();
  }
}

// The whole sort of up to kClusterMost ids by one cluster in one launch: each
// CTA ranks its eighth of the ids, the CTAs read each other's counts from
// shared memory, and the order between the passes goes through global memory.
// The whole gradient against the separate launches: 64 ids 16.9 us, 20.1; 4000
// ids 33.4, 35.1; 8192 ids the same; 16384 ids 118, 115 (more CTAs rank faster).
constexpr int kCluster = 8, kClusterRounds = 2;
constexpr int64_t kClusterMost = static_cast<int64_t>(kCluster) * kClusterRounds * kSortThreads;

struct ClusterArgs {
  const void* tokens;
  uint32_t* key[2];
  uint32_t* pos[2];
  uint32_t* n_spans;
  int64_t n, vocab;
  int32_t token_bytes, bits, passes;
};

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::
          : "memory");
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kSortThreads)
    sort_kernel(const ClusterArgs a) {
  pdl_begin();
  __shared__ uint32_t count[kDigits];              // this CTA's ids of each digit
  __shared__ uint32_t of_warp[kSortWarps][kDigits];
  __shared__ uint32_t warp_sum[kSortWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, me = blockIdx.x;
  // rounds of 32 ids per warp, the same for every CTA
  constexpr int kRoundIds = kCluster * kSortThreads;
  const int rounds = static_cast<int>((a.n + kRoundIds - 1) / kRoundIds);
  const uint32_t n = static_cast<uint32_t>(a.n), mask = (1u << a.bits) - 1;
  const uint32_t first = (me * kSortWarps + warp) * rounds * 32 + lane;
  if (me == 0 && tid == 0) *a.n_spans = 0;
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * a.bits, from = (pass - 1) & 1;
    uint32_t key[kClusterRounds], pos[kClusterRounds], rank[kClusterRounds];
#pragma unroll
    for (int k = 0; k < kClusterRounds; ++k) {
      const uint32_t i = first + k * 32;
      const bool on = k < rounds && i < n;
      pos[k] = on ? pass ? a.pos[from][i] : i : 0;
      key[k] = 0xFFFFFFFFu;
      if (on && pass) key[k] = a.key[from][i];
      if (on && !pass) {
        const int64_t id = load_id(a.tokens, a.token_bytes, i, a.vocab);
        key[k] = static_cast<uint32_t>(id < 0 ? a.vocab : id);  // padding sorts last
      }
    }
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) of_warp[w][tid] = 0;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kClusterRounds; ++k) {
      if (k >= rounds) break;
      const bool on = first + k * 32 < n;
      const uint32_t d = (key[k] >> shift) & mask;
      const uint32_t same = __match_any_sync(0xffffffffu, on ? d : 0xFFFFFFFFu);
      const uint32_t ahead = __popc(same & ((1u << lane) - 1));
      const uint32_t seen = on ? of_warp[warp][d] : 0;
      __syncwarp();
      if (on && ahead == 0) of_warp[warp][d] = seen + __popc(same);
      __syncwarp();
      rank[k] = seen + ahead;
    }
    __syncthreads();
    uint32_t c[kSortWarps], run = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) c[w] = of_warp[w][tid];
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      const uint32_t x = c[w];
      c[w] = run;
      run += x;
    }
    count[tid] = run;
    cluster_sync();
    uint32_t all = 0, before = 0;
#pragma unroll
    for (int g = 0; g < kCluster; ++g) {
      uint32_t remote, x;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                   : "=r"(remote)
                   : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(&count[tid]))), "r"(g));
      asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(remote) : "memory");
      all += x;
      before += g < me ? x : 0;
    }
    uint32_t inc = all;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += y;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    uint32_t base = inc - all + before;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) base += w < warp ? warp_sum[w] : 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) of_warp[w][tid] = base + c[w];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kClusterRounds; ++k) {
      if (k >= rounds || first + k * 32 >= n) break;
      const uint32_t to = of_warp[warp][(key[k] >> shift) & mask] + rank[k];
      if (!ZCHECK(to < n, kSiteStore, to)) continue;
      a.key[pass & 1][to] = key[k];
      a.pos[pass & 1][to] = pos[k];
    }
    // the next pass reads what all CTAs wrote, and no CTA's counts go (by the
    // next pass or its end) before all have read them
    cluster_sync();
  }
}

// -------------------------------------------------------------------- rows ----

struct RowsArgs : Checked<kGradBuffers> {
  const uint32_t* key;   // sorted ids; padding ids are vocab
  const uint32_t* pos;
  const uint16_t* dy;
  uint16_t* grad;
  uint32_t* n_spans;     // rows whose tokens span runs: how many,
  uint4* span;           // and row, first run, last run of each, in any order
  float* out_part;       // [n_runs][width] sums of a run's last row, not done there
  float* in_part;        // [n_runs][width] sums of a run's first row, begun before it
  int64_t n, vocab, dim, width;
  uint32_t slices, n_runs;
  float scale;
  int32_t accumulate;
};

// The slice of a run that a warp sums; run is n_runs or more for warps past
// the last.
struct Unit {
  uint32_t run, slice;
  int64_t c0;
};

__device__ __forceinline__ Unit unit_of(const RowsArgs& a, uint32_t unit) {
  const uint32_t run = unit / a.slices;
  const uint32_t slice = unit - run * a.slices;
  return Unit{run, slice, static_cast<int64_t>(slice) * kSlice};
}

// Number of tokens among the first `item` items of the merged list: the
// tokens with i + key_i < item. All lanes search together, 32 probes a step.
__device__ __forceinline__ int64_t tokens_before(const uint32_t* key, int64_t n, int64_t item,
                                                 int lane) {
  int64_t lo = 0, hi = n < item ? n : item;  // the answer is in [lo, hi]
  while (lo < hi) {
    const int64_t step = (hi - lo + 31) / 32;
    const int64_t i = lo + (lane + 1) * step - 1;
    const bool in = i < hi && i + key[i] < item;
    const int count = __popc(__ballot_sync(0xffffffffu, in));
    const int64_t new_lo = lo + count * step;
    const int64_t new_hi = lo + (count + 1) * step - 1;
    hi = new_hi < hi ? new_hi : hi;
    lo = new_lo < hi ? new_lo : hi;
  }
  return lo;
}

// First of the sorted ids [0, n) that is `row` or more; all lanes search.
__device__ __forceinline__ int64_t first_of(const uint32_t* key, int64_t n, int64_t row, int lane) {
  int64_t lo = 0, hi = n;
  while (lo < hi) {
    const int64_t step = (hi - lo + 31) / 32;
    const int64_t i = lo + (lane + 1) * step - 1;
    const int count = __popc(__ballot_sync(0xffffffffu, i < hi && key[i] < row));
    const int64_t new_hi = lo + (count + 1) * step - 1;
    hi = new_hi < hi ? new_hi : hi;
    lo = lo + count * step < hi ? lo + count * step : hi;
  }
  return lo;
}

template <bool kBf16, bool kVecRows>
__device__ __forceinline__ void store_row(const RowsArgs& a, uint8_t* stage, int64_t v,
                                          int64_t c0, int lane, const float (&sum)[8], bool hit) {
  if (a.accumulate && !hit) return;
  uint16_t* row = a.grad + v * a.dim;
  float f[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = sum[j] * a.scale;
  if (a.accumulate) {
    float old[8];
    widen8<kBf16>(load8<kVecRows>(row, c0 + lane * kVec, a.dim, a.bounds(kGrad)), old);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] += old[j];
  }
  store_slice<kVecRows>(stage, row, c0, lane, a.dim, narrow8<kBf16>(f), a.bounds(kGrad));
}

// fp32 partial sums sit lane by lane: lane l's eight columns at [l * 8, l * 8 + 8)
__device__ __forceinline__ void store_part(float* part, int64_t c0, int lane,
                                           const float (&s)[8], const Bounds& in) {
  float4* p = reinterpret_cast<float4*>(part + c0 + lane * kVec);
  if (!in.holds(p, 32, kSiteStore)) return;
  p[0] = make_float4(s[0], s[1], s[2], s[3]);
  p[1] = make_float4(s[4], s[5], s[6], s[7]);
}

// Zeros for the n elements from p on, rows that follow one another and so one
// piece of memory whatever their length: share `part` of `parts`, in 16-byte
// blocks but for the ends.
__device__ __forceinline__ void clear_share(uint16_t* p, int64_t n, uint32_t part, uint32_t parts,
                                            int lane, const Bounds& in) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p), hi = lo + 2 * static_cast<uintptr_t>(n);
  const uintptr_t in_lo = (lo + 15) & ~static_cast<uintptr_t>(15);
  const uintptr_t in_hi = hi & ~static_cast<uintptr_t>(15);
  if (part == 0) {  // at most seven elements before the first block and after the last
    const uintptr_t head = in_lo < hi ? in_lo : hi;
    uint16_t* end = reinterpret_cast<uint16_t*>(in_hi);
    if (lo + 2 * lane < head && in.holds(p + lane, 2, kSiteStore)) p[lane] = 0;
    if (in_hi >= in_lo && in_hi + 2 * lane < hi && in.holds(end + lane, 2, kSiteStore))
      end[lane] = 0;
  }
  if (in_hi <= in_lo) return;
  const uint32_t blocks = static_cast<uint32_t>((in_hi - in_lo) >> 4);
  const uint32_t per = (blocks + parts - 1) / parts;
  const uint32_t b0 = part * per, b1 = b0 + per < blocks ? b0 + per : blocks;
  uint4* q = reinterpret_cast<uint4*>(in_lo);
#pragma unroll 4
  for (uint32_t b = b0 + lane; b < b1; b += 32)
    if (in.holds(q + b, 16, kSiteStore)) __stcs(q + b, make_uint4(0, 0, 0, 0));
}

template <bool kBf16, bool kVecRows>
__global__ void __launch_bounds__(kThreads) rows_kernel(const RowsArgs a) {
  pdl_begin();
  __shared__ Stages<kVecRows> stages;
  uint8_t* stage = stages.of_warp[kVecRows ? 0 : threadIdx.x >> 5];
  const int lane = threadIdx.x & 31;
  const Unit u = unit_of(a, blockIdx.x * kWarps + (threadIdx.x >> 5));
  if (u.run >= a.n_runs) return;
  const int64_t run = u.run, c0 = u.c0, item0 = run * kRun;
  const int64_t item1 = item0 + kRun < a.n + a.vocab ? item0 + kRun : a.n + a.vocab;
  const int64_t i0 = tokens_before(a.key, a.n, item0, lane);
  // the run's tokens are among the next kRun: their ids and positions, one or
  // two per lane, and the id before them
  constexpr int kPer = kRun / 32;
  uint32_t key[kPer], pos[kPer];
  int count = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int64_t i = i0 + k * 32 + lane;
    key[k] = i < a.n ? a.key[i] : 0xFFFFFFFFu;
    pos[k] = i < a.n ? a.pos[i] : 0;
  }
  const uint32_t before = i0 > 0 ? a.key[i0 - 1] : 0xFFFFFFFFu;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int64_t i = i0 + k * 32 + lane;
    count += __popc(__ballot_sync(0xffffffffu, i < a.n && i + key[k] < item1));
  }
  int64_t row = item0 - i0;                      // rows done before this run
  const int64_t row_end = item1 - (i0 + count);  // and before the next
  // the first row's earlier tokens are in an earlier run
  bool begun = row < a.vocab && before == row;
  if (begun && row < row_end && c0 == 0) {
    // and its last in this one: join_kernel will add them up, from the run
    // that has the row's first token as an item of the merged list
    const int64_t first = (first_of(a.key, i0, row, lane) + row) / kRun;
    if (lane == 0) {
      uint4* to = a.span + atomicAdd(a.n_spans, 1u);
      if (a.bounds(kSpans).holds(to, 16, kSiteRecord))
        *to = make_uint4(static_cast<uint32_t>(row), static_cast<uint32_t>(first), u.run, 0);
    }
  }
  bool hit = false;
  float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  // rows up to `end` have all their tokens: the first the sum, the rest none
  const auto done_until = [&](int64_t end) {
    if (row >= end) return;
    if (begun) store_part(a.in_part + run * a.width, c0, lane, sum, a.bounds(kParts));
    else store_row<kBf16, kVecRows>(a, stage, row, c0, lane, sum, hit);
    begun = hit = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] = 0.f;
    ++row;
    if (!a.accumulate && row < end)
      clear_share(a.grad + row * a.dim, (end - row) * a.dim, u.slice, a.slices, lane,
                  a.bounds(kGrad));
    row = end;
  };
  for (int i = 0; i < count; i += kBatch) {
    uint4 v[kBatch];
    uint32_t id[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int at = i + k;  // kBatch divides 32: one register of the lanes' per batch
      const uint32_t p = __shfl_sync(0xffffffffu, at < 32 ? pos[0] : pos[kPer - 1], at & 31);
      id[k] = __shfl_sync(0xffffffffu, at < 32 ? key[0] : key[kPer - 1], at & 31);
      if (at >= count) id[k] = 0xFFFFFFFFu;
      if (id[k] < a.vocab)
        v[k] = load8<kVecRows>(a.dy + static_cast<int64_t>(p) * a.dim, c0 + lane * kVec, a.dim,
                               a.bounds(kDy));
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (id[k] >= a.vocab) break;
      done_until(id[k]);
      float f[8];
      widen8<kBf16>(v[k], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += f[j];
      hit = true;
    }
  }
  done_until(row_end);
  if (hit || begun) store_part(a.out_part + run * a.width, c0, lane, sum, a.bounds(kParts));
}

// Rows whose tokens span runs: the partial sums of the runs before the one
// that ends the row, in run order, then that run's own.
template <bool kBf16, bool kVecRows>
__global__ void __launch_bounds__(kThreads) join_kernel(const RowsArgs a) {
  pdl_begin();
  __shared__ Stages<kVecRows> stages;
  uint8_t* stage = stages.of_warp[kVecRows ? 0 : threadIdx.x >> 5];
  const int lane = threadIdx.x & 31;
  const uint32_t units = *a.n_spans * a.slices;
  for (uint32_t at = blockIdx.x * kWarps + (threadIdx.x >> 5); at < units;
       at += gridDim.x * kWarps) {
    const Unit u = unit_of(a, at);
    if (!a.bounds(kSpans).holds(a.span + u.run, 16, kSiteRecord)) continue;
    const uint4 span = a.span[u.run];
    const float* part = a.out_part + u.c0 + lane * kVec;
    float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 16
    for (uint32_t k = span.y; k <= span.z; ++k) {
      const float4* p = reinterpret_cast<const float4*>(
          (k < span.z ? part : a.in_part + u.c0 + lane * kVec) + static_cast<int64_t>(k) * a.width);
      if (!a.bounds(kParts).holds(p, 32, kSiteLoad)) continue;
      const float4 x = p[0], y = p[1];
      const float s[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += s[j];
    }
    store_row<kBf16, kVecRows>(a, stage, span.x, u.c0, lane, sum, true);
  }
}

// -------------------------------------------------------------------- host ----

struct Layout {
  int64_t n_runs, width;
  size_t hist, n_spans, key[2], pos[2], span, out_part, in_part, bytes;
};

Layout layout_of(int64_t n, int64_t vocab, int64_t dim) {
  Layout l = {};
  l.n_runs = ceil_div(n + vocab, kRun);
  l.width = ceil_div(dim, kSlice) * kSlice;
  size_t at = 0;
  const auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) & ~static_cast<size_t>(255);
    return here;
  };
  l.hist = take(sizeof(uint32_t) * kMaxPasses * kDigits * kMaxChunks);
  l.n_spans = take(sizeof(uint32_t));
  for (int k = 0; k < 2; ++k) {
    l.key[k] = take(sizeof(uint32_t) * static_cast<size_t>(n));
    l.pos[k] = take(sizeof(uint32_t) * static_cast<size_t>(n));
  }
  l.span = take(sizeof(uint4) * static_cast<size_t>(l.n_runs));
  l.out_part = take(sizeof(float) * static_cast<size_t>(l.n_runs * l.width));
  l.in_part = take(sizeof(float) * static_cast<size_t>(l.n_runs * l.width));
  l.bytes = at;
  return l;
}

constexpr int64_t kMaxTokens = int64_t{1} << 28;
constexpr int64_t kMaxVocab = int64_t{1} << 24;
constexpr int64_t kMaxGrid = 0x7fffffff;
constexpr unsigned kJoinGrid = 304;

template <bool kBf16, bool kVecRows>
int launch_rows(const RowsArgs& a, cudaStream_t st) {
  const unsigned grid =
      static_cast<unsigned>(ceil_div(static_cast<int64_t>(a.n_runs) * a.slices, kWarps));
  cudaError_t e = launch_pdl(rows_kernel<kBf16, kVecRows>, dim3(grid), dim3(kThreads), 0, st, a);
  // without tokens no row spans runs
  if (e == cudaSuccess && a.n > 0)
    e = launch_pdl(join_kernel<kBf16, kVecRows>, dim3(std::min(grid, kJoinGrid)), dim3(kThreads), 0,
                   st, a);
  return status_of(e);
}

}  // namespace ze

#ifdef ZERO_CHECKED
extern "C" int ze_collect_checks(unsigned long long* count, unsigned long long* first) {
  return collect_checks(count, first);
}
#endif

extern "C" {

ZERO_API int zero_embedding(const void* tokens, int32_t token_bytes, int64_t n_tokens,
                            const void* table, int64_t vocab, int64_t dim, float scale,
                            int32_t dtype, void* out, void* stream) {
  using namespace ze;
  if (n_tokens < 0 || vocab < 0 || dim < 0 || !is_dtype16(dtype) ||
      (token_bytes != 4 && token_bytes != 8))
    return ZERO_EINVAL;
  if (n_tokens > kMaxTokens || vocab > kMaxVocab || dim > kMaxTokens) return ZERO_ERANGE;
  if (n_tokens == 0 || dim == 0) return ZERO_OK;
  if (!tokens || !out || (!table && vocab)) return ZERO_EINVAL;
  if (!aligned(tokens, token_bytes) || !aligned(table, 2) || !aligned(out, 2)) return ZERO_EALIGN;
  LookupArgs a = new_args<LookupArgs>();
  a.tokens = tokens;
  a.table = static_cast<const uint16_t*>(table);
  a.out = static_cast<uint16_t*>(out);
  a.n = n_tokens;
  a.vocab = vocab;
  a.dim = dim;
  a.slices = ceil_div(dim, kSlice);
  a.units = ceil_div(n_tokens, kLookup) * a.slices;
  a.token_bytes = token_bytes;
  a.scale = scale;
  a.set_bounds(kTable, table, vocab, dim, dim, 2);
  a.set_bounds(kOut, out, n_tokens, dim, dim, 2);
  const int64_t grid = ceil_div(a.units, kWarps);
  if (grid > kMaxGrid) return ZERO_ERANGE;
  const bool vec = dim % kVec == 0 && aligned(table, 16) && aligned(out, 16);
  const auto fn = dtype == ZERO_BF16
                      ? (vec ? lookup_kernel<true, true> : lookup_kernel<true, false>)
                      : (vec ? lookup_kernel<false, true> : lookup_kernel<false, false>);
  return status_of(launch_pdl(fn, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0,
                              static_cast<cudaStream_t>(stream), a));
}

ZERO_API size_t zero_embedding_workspace_bytes(int64_t n_tokens, int64_t vocab, int64_t dim) {
  using namespace ze;
  if (n_tokens < 0 || vocab < 0 || dim < 0 || n_tokens > kMaxTokens || vocab > kMaxVocab ||
      dim > kMaxTokens)
    return 0;
  return layout_of(n_tokens, vocab, dim).bytes;
}

ZERO_API int zero_embedding_grad(const void* tokens, int32_t token_bytes, int64_t n_tokens,
                                 const void* dy, int64_t vocab, int64_t dim, float scale,
                                 int32_t dtype, int32_t accumulate, void* grad,
                                 void* workspace, void* stream) {
  using namespace ze;
  if (n_tokens < 0 || vocab < 0 || dim < 0 || !is_dtype16(dtype) ||
      (token_bytes != 4 && token_bytes != 8) || (accumulate != 0 && accumulate != 1))
    return ZERO_EINVAL;
  if (n_tokens > kMaxTokens || vocab > kMaxVocab || dim > kMaxTokens) return ZERO_ERANGE;
  if (vocab == 0 || dim == 0) return ZERO_OK;
  if (!grad || !workspace || (n_tokens && (!tokens || !dy))) return ZERO_EINVAL;
  if (!aligned(tokens, token_bytes) || !aligned(dy, 2) || !aligned(grad, 2) ||
      !aligned(workspace, 16))
    return ZERO_EALIGN;
  const Layout l = layout_of(n_tokens, vocab, dim);
  const int64_t slices = ceil_div(dim, kSlice);
  if (l.n_runs * slices > kMaxGrid) return ZERO_ERANGE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint32_t* key[2] = {reinterpret_cast<uint32_t*>(ws + l.key[0]),
                      reinterpret_cast<uint32_t*>(ws + l.key[1])};
  uint32_t* pos[2] = {reinterpret_cast<uint32_t*>(ws + l.pos[0]),
                      reinterpret_cast<uint32_t*>(ws + l.pos[1])};
  int last = 0;
  if (n_tokens > 0) {
    int width = 1;  // bits of the ids, vocab itself (padding) among them
    while ((vocab >> width) != 0) ++width;
    const int passes = static_cast<int>(ceil_div(width, 9));
    const int bits = static_cast<int>(ceil_div(width, passes));
    uint32_t* n_spans = reinterpret_cast<uint32_t*>(ws + l.n_spans);
    last = (passes - 1) & 1;
    cudaError_t e = cudaSuccess;
    if (n_tokens <= kClusterMost) {
      ClusterArgs c = {tokens, {key[0], key[1]}, {pos[0], pos[1]}, n_spans, n_tokens, vocab,
                       token_bytes, bits, passes};
      e = launch_pdl(sort_kernel, dim3(kCluster), dim3(kSortThreads), 0, st, c);
    } else {
      SortArgs s = {};
      s.tokens = tokens;
      s.token_bytes = token_bytes;
      s.n = n_tokens;
      s.vocab = vocab;
      s.chunk = ceil_div(ceil_div(n_tokens, kMaxChunks), kTile) * kTile;
      s.n_chunks = static_cast<int32_t>(ceil_div(n_tokens, s.chunk));
      s.bits = bits;
      s.n_hists = passes;
      s.n_spans = n_spans;
      uint32_t* hist = reinterpret_cast<uint32_t*>(ws + l.hist);
      s.hist = hist;
      e = launch_pdl(hist_kernel, dim3(s.n_chunks), dim3(kSortThreads), 0, st, s);
      for (int p = 0; p < passes && e == cudaSuccess; ++p) {
        s.key_in = p ? key[(p - 1) & 1] : nullptr;
        s.pos_in = p ? pos[(p - 1) & 1] : nullptr;
        s.key_out = key[p & 1];
        s.pos_out = pos[p & 1];
        s.hist = hist + static_cast<size_t>(p) * kDigits * kMaxChunks;
        s.hist_next = p + 1 < passes ? s.hist + kDigits * kMaxChunks : nullptr;
        s.shift = p * s.bits;
        e = launch_pdl(scatter_kernel, dim3(s.n_chunks), dim3(kSortThreads), 0, st, s);
      }
    }
    if (e != cudaSuccess) return ZERO_ECUDA;
  }
  RowsArgs a = new_args<RowsArgs>();
  a.key = key[last];
  a.pos = pos[last];
  a.dy = static_cast<const uint16_t*>(dy);
  a.grad = static_cast<uint16_t*>(grad);
  a.n_spans = reinterpret_cast<uint32_t*>(ws + l.n_spans);
  a.span = reinterpret_cast<uint4*>(ws + l.span);
  a.out_part = reinterpret_cast<float*>(ws + l.out_part);
  a.in_part = reinterpret_cast<float*>(ws + l.in_part);
  a.n = n_tokens;
  a.vocab = vocab;
  a.dim = dim;
  a.slices = static_cast<uint32_t>(slices);
  a.width = l.width;
  a.n_runs = static_cast<uint32_t>(l.n_runs);
  a.scale = scale;
  a.accumulate = accumulate;
  a.set_bounds(kDy, dy, n_tokens, dim, dim, 2);
  a.set_bounds(kGrad, grad, vocab, dim, dim, 2);
  // in_part follows out_part
  a.set_bounds(kParts, a.out_part, 1, 1, 0, static_cast<int64_t>(l.bytes - l.out_part));
  a.set_bounds(kSpans, a.span, 1, 1, 0, l.n_runs * static_cast<int64_t>(sizeof(uint4)));
  const bool vec = dim % kVec == 0 && aligned(dy, 16) && aligned(grad, 16);
  if (dtype == ZERO_BF16)
    return vec ? launch_rows<true, true>(a, st) : launch_rows<true, false>(a, st);
  return vec ? launch_rows<false, true>(a, st) : launch_rows<false, false>(a, st);
}

}  // extern "C"
