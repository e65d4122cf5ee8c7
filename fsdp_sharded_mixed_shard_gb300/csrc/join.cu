/*
 * join.cu -- where a block's output joins the residual stream: norms after the
 * block and before the next, gate, dropout and residual scale (zero_block.h).
 *
 * A team of warps holds a row in registers from the load to the last store:
 * forward 8 bytes per element, backward 12, and nothing is read twice. What a
 * norm needs of the whole row goes through shuffles and, where the team has
 * several warps, one exchange between them. These and a row's addresses cost
 * about as many instructions as a vector of eight elements does, so a thread
 * takes as many vectors as its registers hold beside the next row's loads: four
 * forward, two backward. (With one vector per thread the forward pass
 * was bound by instructions: 8192 x 2048 bf16 31 us, 360 instructions per 256
 * elements.)
 *
 * With m the dropout's factor (0 or its scale), c = branch_scale gate w_post and
 * d = branch_scale gate b_post, the forward pass is
 *   h_out = stream_scale h + m (c y^ + d)
 * and the backward pass, with g = dz w_pre, E = dh_out + r g and k = c m,
 *   D = E - r (c1 h^ + c2),  c1 = mean(g h^),  c2 = mean(g)
 *   dy = r' (k D - y^ mean(k D y^) - mean(k D)),
 * (the means without a square belong to ZERO_NORM_LAYER alone), where
 *   mean(k D y^) = mean(k y^ E) - r (c1 mean(k y^ h^) + c2 mean(k y^)),
 * and mean(k D) likewise: all of a row's sums are taken in one go, before D is
 * known. Of each column it needs, over the rows,
 *   P = sum dz h^,  Q = sum dz,  A = sum m D y^,  B = sum m D:
 *   dw_pre = P, db_pre = Q, dw_post = branch_scale gate A,
 *   db_post = branch_scale gate B, dgate = branch_scale (w_post A + b_post B).
 * A thread adds those of its own columns up. A CTA joins its teams' in order and
 * leaves one vector each in the workspace; a second kernel adds the (at most
 * kMaxParts) vectors in order.
 *
 * The row after the one at hand is on its way into shared memory meanwhile, as
 * the 16-byte blocks that hold it, so that memory is busy all the time and rows
 * off the 16-byte grid need no more registers (at Ahead). Measured, bf16,
 * ZERO_NORM_RMS with all parameters: 8192 x 2048 forward 20.5 to 22 us (91 % of copy
 * bandwidth), backward 39 (77 %), 4096 x 8192 47 to 49 and 71 (84 %); 8192 x 2047 41
 * and 67, where putting vectors together takes the time; 8192 x 2048 ZERO_NORM_LAYER
 * with dropout 34 and 57. With loads half a row's work ahead into registers the
 * backward pass took 46 and 102, rows off the grid 67 and 121. What bounds them now:
 * instructions and the latency of a row's sums (the issue slots are 40 to 60 % busy),
 * beside memory. The backward kernels with ZERO_NORM_LAYER on both sides and two
 * vectors per thread spill 44 to 72 bytes of their 128 registers.
 */
#include "draws.cuh"
#include "rows.cuh"

#include <algorithm>
#include <cfloat>
#include <cmath>

namespace zj {

using namespace zt;

constexpr int kMaxThreads = 512;  // of a CTA, one per SM, 128 registers each
constexpr int kMaxWarps = kMaxThreads / 32;
constexpr int kMaxParts = 152;    // CTAs
// vectors per thread at most
constexpr int kForwardVectors = 4, kBackVectors = 2;
static_assert(ZERO_MAX_JOIN_COLS <= kBackVectors * kMaxThreads * kVec, "a row fits a CTA");

enum { kWPost, kBPost, kGate, kWPre, kBPre, kParams };
// of a call, the parameters last
enum { kH, kY, kHOut, kZ, kStats, kDz, kDhOut, kDh, kDy, kParts, kParam0,
       kBuffers = kParam0 + kParams };
enum { kSumP, kSumA, kSumQ, kSumB, kSums };

struct Args : Checked<kBuffers> {
  const uint16_t *h, *y, *h_out, *dz, *dh_out;
  uint16_t *h_new, *z, *dh, *dy;
  float4* stats;
  const uint16_t* param[kParams];
  float* parts;          // [CTA][slot][pitch]
  int32_t slot[kSums];   // of a sum in parts, -1: not needed
  int32_t slots;
  int64_t rows, ld;
  int32_t cols, pitch;   // pitch: cols rounded up to whole vectors
  int32_t team_warps, teams, slots_of_row;  // vectors that a team has room for
  float eps, inv_cols, stream_scale, branch_scale;
  Drop drop;
};

// A thread's place: its team, its warp and lane there.
struct Place {
  int team, warp, lane;
  __device__ __forceinline__ Place(const Args& a)
      : team(static_cast<int>(threadIdx.x >> 5) / a.team_warps),
        warp(static_cast<int>(threadIdx.x >> 5) - team * a.team_warps),
        lane(threadIdx.x & 31) {}
  // first column of the warp's v-th 256
  __device__ __forceinline__ int first(const Args& a, int v) const {
    return (v * a.team_warps + warp) * kCols;
  }
};

// Eight values as four pairs (packed fp32 arithmetic).
struct Eight {
  Pair p[4];
};

__device__ __forceinline__ Pair both(float x) { return pair(x, x); }

__device__ __forceinline__ float sum_of(const Pair& p) {
  float a, b;
  unpair(p, a, b);
  return a + b;
}

template <bool kBf16>
__device__ __forceinline__ Eight widen_pairs(const uint4& v) {
  float f[8];
  widen8<kBf16>(v, f);
  Eight e;
#pragma unroll
  for (int j = 0; j < 4; ++j) e.p[j] = pair(f[2 * j], f[2 * j + 1]);
  return e;
}

template <bool kBf16>
__device__ __forceinline__ uint4 narrow_pairs(const Eight& e) {
  float f[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) unpair(e.p[j], f[2 * j], f[2 * j + 1]);
  return narrow8<kBf16>(f);
}

// Which of a row's eight columns from `col` on stay, a bit each.
__device__ __forceinline__ uint32_t kept(const Drop& d, uint32_t step, int64_t row, int col) {
  const uint4 w = draw8(d, step, static_cast<uint32_t>(row), static_cast<uint32_t>(col) / kVec);
  return keep8(d, w);
}

// what is left out becomes 0, whatever it was
__device__ __forceinline__ Eight kept_only(uint32_t keep, Eight e) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float a, b;
    unpair(e.p[j], a, b);
    e.p[j] = pair(keep >> (2 * j) & 1 ? a : 0.f, keep >> (2 * j + 1) & 1 ? b : 0.f);
  }
  return e;
}

__device__ __forceinline__ void drop_pairs(const Drop& d, uint32_t keep, Eight& e) {
#pragma unroll
  for (int j = 0; j < 4; ++j) e.p[j] = e.p[j] * both(d.scale);
  e = kept_only(keep, e);
}

// Eight floats in shared memory as two words of 16 bytes, `apart` words apart:
// neighbouring lanes' words lie side by side.
__device__ __forceinline__ Eight read_eight_at(const float4* at, int apart) {
  const float4 x = at[0], y = at[apart];
  return Eight{{pair(x.x, x.y), pair(x.z, x.w), pair(y.x, y.y), pair(y.z, y.w)}};
}

__device__ __forceinline__ void write_eight_at(float4* at, int apart, const Eight& e) {
  float f[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) unpair(e.p[j], f[2 * j], f[2 * j + 1]);
  at[0] = make_float4(f[0], f[1], f[2], f[3]);
  at[apart] = make_float4(f[4], f[5], f[6], f[7]);
}

// kGrid: rows lie on the 16-byte grid and consist of whole vectors.

// A row of kArrays arrays on its way into shared memory, the row after the one
// that is worked on: each warp its own kV times 256 columns, as the 16-byte blocks
// that hold them.
template <int kArrays, int kV, bool kGrid>
struct Ahead {
  static constexpr int kSpan = kGrid ? 32 : 34;  // blocks of 256 columns
  static constexpr int kBytes = kArrays * kV * kMaxWarps * kSpan * 16;
  uint4* own;  // the warp's
  int lane;
  __device__ __forceinline__ Ahead(void* smem)
      : own(static_cast<uint4*>(smem) + (threadIdx.x >> 5) * kSpan), lane(threadIdx.x & 31) {}
  // the lane's v-th vector lies past the last column, where nothing comes
  __device__ __forceinline__ void clear(int v) const {
#pragma unroll
    for (int k = 0; k < kArrays; ++k) at(k, v)[lane] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ uint4* at(int array, int v) const {
    return own + (array * kV + v) * (kMaxWarps * kSpan);
  }
  __device__ __forceinline__ static void copy(uint4* to, const uint4* from) {
    const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(to));
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
  }
  // columns [first, first + 256) of the row of x that starts at row_start
  __device__ __forceinline__ void start(int array, int v, const uint16_t* x, int64_t row_start,
                                        int first, int cols, const Bounds& in) const {
    const uint16_t* from = x + row_start + first;
    if constexpr (kGrid) {
      from += lane * kVec;
      if (first + lane * kVec < cols && in.holds(from, 16, kSiteLoad))
        copy(at(array, v) + lane, reinterpret_cast<const uint4*>(from));
    } else {
      const uintptr_t begin = reinterpret_cast<uintptr_t>(from);
      const int d = static_cast<int>(begin & 15), n = min(kCols, cols - first);
      const uint4* block = reinterpret_cast<const uint4*>(begin - d);
      const int blocks = n > 0 ? (d + 2 * n + 15) >> 4 : 0;
      if (lane < blocks && in.holds_blocks(block + lane, 16, kSiteLoad))
        copy(at(array, v) + lane, block + lane);
      if (blocks > 32 && lane == 0 && in.holds_blocks(block + 32, 16, kSiteLoad))
        copy(at(array, v) + 32, block + 32);
    }
  }
  // all that the warp has started is there
  __device__ __forceinline__ void wait() const {
    asm volatile("cp.async.wait_all;" ::: "memory");
    if constexpr (!kGrid) __syncwarp();
  }
  // the lane's eight columns, of which `there` are columns and the others 0
  __device__ __forceinline__ uint4 read(int array, int v, const uint16_t* x, int64_t row_start,
                                        int there) const {
    uint4 b = at(array, v)[lane];
    if constexpr (!kGrid) {
      const int d = static_cast<int>(reinterpret_cast<uintptr_t>(x + row_start) & 15);
      b = shifted_alike(b, at(array, v)[lane + 1], d);
    }
    if constexpr (!kGrid) b = first_of(b, there);
    return b;
  }
  // the warp has read all: the next row may come
  __device__ __forceinline__ void done() const { __syncwarp(); }
};

template <bool kGrid>
__device__ __forceinline__ void store_at(uint8_t* stage, uint16_t* x, int64_t row_start, int first,
                                         int lane, int cols, const uint4& v, const Bounds& in) {
  if constexpr (kGrid) {
    uint16_t* at = x + row_start + (first + lane * kVec);
    if (first + lane * kVec < cols && in.holds(at, 16, kSiteStore))
      __stcs(reinterpret_cast<uint4*>(at), v);
  } else {
    store_row<false>(stage, x + row_start, first, lane, cols, v, in);
  }
}

// A team's warps' sums, each team's padded with zeros to whole float4. Two sets
// in turn, so that one barrier each is enough: a warp that writes to one again
// has passed the other's barrier, before which all have read this one's.
constexpr int kMaxValues = 8;
struct Exchange {
  float4 sums[2][kMaxValues][8];  // [set][value]
};

// by every thread of the CTA, which waits for all others, before the first sum
__device__ __forceinline__ void clear(Exchange& ex) {
  for (int k = threadIdx.x; k < 2 * kMaxValues * 8; k += blockDim.x)
    (&ex.sums[0][0][0])[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  __syncthreads();
}

// Sums over the team, the same bits in all its threads.
template <int kValues>
__device__ __forceinline__ void team_sum(const Args& a, const Place& p, Exchange& ex, int& turn,
                                         float (&x)[kValues]) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
#pragma unroll
    for (int k = 0; k < kValues; ++k) x[k] += __shfl_xor_sync(0xffffffffu, x[k], d);
  if (a.team_warps == 1) return;
  const int fours = (a.team_warps + 3) >> 2;
  if (p.lane == 0)
#pragma unroll
    for (int k = 0; k < kValues; ++k)
      reinterpret_cast<float*>(&ex.sums[turn][k][p.team * fours])[p.warp] = x[k];
  asm volatile("bar.sync %0, %1;" ::"r"(1 + p.team), "r"(32 * a.team_warps) : "memory");
#pragma unroll
  for (int k = 0; k < kValues; ++k) x[k] = 0.f;
  for (int w = 0; w < fours; ++w)
#pragma unroll
    for (int k = 0; k < kValues; ++k) {
      const float4 s = ex.sums[turn][k][p.team * fours + w];
      x[k] += (s.x + s.y) + (s.z + s.w);
    }
  turn ^= 1;
}

__device__ __forceinline__ float inverse_root(float mean_square, float eps) {
  // NaN, not 0 or infinity, past fp32's range and below its normal numbers, where
  // squares (with eps 0) are lost; from 2^-126 on what single squares lose of a mean
  // is 2^-150 each, 2^-24 of it
  const float x = mean_square + eps;
  return x >= __uint_as_float(0x00800000u) && x < __uint_as_float(0x7F800000u)
             ? rsqrtf(x)
             : __uint_as_float(0x7FC00000u);
}

// Statistics (mean or 0, 1 / sqrt(mean square + eps)) of a row held by the team;
// past the last column it holds zeros. `there`: the thread's columns of each
// vector that are columns.
template <bool kBf16, bool kLayer, int kV>
__device__ __forceinline__ float2 row_stats(const Args& a, const Place& p, Exchange& ex, int& turn,
                                            const uint4 (&x)[kV], const int (&there)[kV]) {
  float mean = 0.f;
  if constexpr (kLayer) {
    Pair s = both(0.f);
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      const Eight e = widen_pairs<kBf16>(x[v]);
      s = s + ((e.p[0] + e.p[1]) + (e.p[2] + e.p[3]));
    }
    float sum[1] = {sum_of(s)};
    team_sum(a, p, ex, turn, sum);
    mean = sum[0] * a.inv_cols;
  }
  Pair s = both(0.f);
  float edge = 0.f;
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    const Eight e = widen_pairs<kBf16>(x[v]);
    if (!kLayer || there[v] == kVec) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const Pair d = kLayer ? e.p[j] + both(-mean) : e.p[j];
        s = fma2(d, d, s);
      }
    } else {  // past the last column 0 is not a value
      float f[8];
      widen8<kBf16>(x[v], f);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < there[v]) edge = __fmaf_rn(f[j] - mean, f[j] - mean, edge);
    }
  }
  float sum[1] = {sum_of(s) + edge};
  team_sum(a, p, ex, turn, sum);
  return make_float2(mean, inverse_root(sum[0] * a.inv_cols, a.eps));
}

// (x - mean) r
template <bool kLayer>
__device__ __forceinline__ Pair normed(const Pair& x, const float2& st) {
  return kLayer ? (x + both(-st.x)) * both(st.y) : x * both(st.y);
}

__device__ __forceinline__ Eight scaled(const Eight& x, const Eight& y, float s) {
  Eight e;
#pragma unroll
  for (int j = 0; j < 4; ++j) e.p[j] = x.p[j] * both(s) * y.p[j];
  return e;
}

// The numbers that the kernels need per column, in shared memory for all teams:
// kCount times as many vectors of eight floats as a row has.
enum { kC, kPre, kD, kBias };

template <bool kBf16, int kCount>
__device__ __forceinline__ void stage_columns(const Args& a, float4* w) {
  const int n = a.slots_of_row;
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int c = i * kVec;  // past the last column parameters count as 0
    Blocks b[kParams];  // all loads before the first use
#pragma unroll
    for (int k = 0; k < kParams; ++k)
      if (a.param[k]) b[k] = load_blocks(a.param[k], c, a.cols, a.bounds(kParam0 + k));
    const auto param = [&](int k, float none) {
      return a.param[k] ? widen_pairs<kBf16>(eight_of(b[k]))
                        : Eight{{both(none), both(none), both(none), both(none)}};
    };
    const auto put = [&](int k, const Eight& e) { write_eight_at(w + 2 * k * n + i, n, e); };
    const Eight gate = param(kGate, 1.f);
    put(kC, scaled(gate, param(kWPost, 1.f), a.branch_scale));
    put(kPre, param(kWPre, 0.f));
    if constexpr (kCount > 2) {
      // a bias that is not there adds nothing, also where the gate is infinite
      const Eight bias = param(kBPost, 0.f);
      put(kD, a.param[kBPost] ? scaled(gate, bias, a.branch_scale) : bias);
      put(kBias, param(kBPre, 0.f));
    }
  }
}

__device__ __forceinline__ Eight column(const Args& a, const float4* w, int k, int col) {
  return read_eight_at(w + 2 * k * a.slots_of_row + col / kVec, a.slots_of_row);
}

constexpr int kStagePitch = (kStageWarp + 15) & ~15;

template <bool kBf16, bool kGrid, bool kLayer, int kV>
__global__ void __launch_bounds__(kMaxThreads, 1) join_kernel(const Args a) {
  pdl_begin();
  extern __shared__ float4 smem[];
  __shared__ Exchange exchange;
  __shared__ __align__(16) uint8_t stages[kGrid ? 16 : kMaxWarps * kStagePitch];
  const Place p(a);
  uint8_t* stage = stages + (kGrid ? 0 : (threadIdx.x >> 5) * kStagePitch);
  int turn = 0;
  const bool post = a.param[kWPost] != nullptr, pre = a.param[kWPre] != nullptr;
  const uint32_t step = step_of(a.drop);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * a.teams;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * a.teams + p.team;
  int col[kV], there[kV];
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    col[v] = p.first(a, v) + p.lane * kVec;
    there[v] = max(0, min(kVec, a.cols - col[v]));
  }
  // behind the columns' numbers
  const Ahead<2, kV, kGrid> ahead(smem + 2 * (kLayer ? 4 : 2) * a.slots_of_row);
#pragma unroll
  for (int v = 0; v < kV; ++v)
    if (kGrid && there[v] == 0) ahead.clear(v);
  const auto start = [&](int64_t row) {
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      ahead.start(0, v, a.y, row * a.ld, p.first(a, v), a.cols, a.bounds(kY));
      ahead.start(1, v, a.h, row * a.ld, p.first(a, v), a.cols, a.bounds(kH));
    }
  };
  if (row0 < a.rows) start(row0);  // under way while the columns' numbers are set up
  stage_columns<kBf16, kLayer ? 4 : 2>(a, smem);
  clear(exchange);
  for (int64_t row = row0; row < a.rows; row += stride) {
    uint4 y[kV], h[kV];
    ahead.wait();
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      y[v] = ahead.read(0, v, a.y, row * a.ld, there[v]);
      h[v] = ahead.read(1, v, a.h, row * a.ld, there[v]);
    }
    ahead.done();
    if (row + stride < a.rows) start(row + stride);
    float2 sy = make_float2(0.f, 1.f), sh = make_float2(0.f, 0.f);
    if (post) sy = row_stats<kBf16, kLayer, kV>(a, p, exchange, turn, y, there);
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      Eight x = widen_pairs<kBf16>(y[v]);
      const Eight c = column(a, smem, kC, col[v]);
#pragma unroll
      for (int j = 0; j < 4; ++j) x.p[j] = normed<kLayer>(x.p[j], sy) * c.p[j];
      if constexpr (kLayer) {
        const Eight d = column(a, smem, kD, col[v]);
#pragma unroll
        for (int j = 0; j < 4; ++j) x.p[j] = x.p[j] + d.p[j];
      }
      if (a.drop.threshold) drop_pairs(a.drop, kept(a.drop, step, row, col[v]), x);
      const Eight s = widen_pairs<kBf16>(h[v]);
#pragma unroll
      for (int j = 0; j < 4; ++j) x.p[j] = fma2(s.p[j], both(a.stream_scale), x.p[j]);
      h[v] = narrow_pairs<kBf16>(x);
      store_at<kGrid>(stage, a.h_new, row * a.ld, p.first(a, v), p.lane, a.cols, h[v],
                      a.bounds(kHOut));
    }
    if (pre) {
      sh = row_stats<kBf16, kLayer, kV>(a, p, exchange, turn, h, there);
#pragma unroll
      for (int v = 0; v < kV; ++v) {
        Eight x = widen_pairs<kBf16>(h[v]);
        const Eight c = column(a, smem, kPre, col[v]);
#pragma unroll
        for (int j = 0; j < 4; ++j) x.p[j] = normed<kLayer>(x.p[j], sh) * c.p[j];
        if constexpr (kLayer) {
          const Eight d = column(a, smem, kBias, col[v]);
#pragma unroll
          for (int j = 0; j < 4; ++j) x.p[j] = x.p[j] + d.p[j];
        }
        store_at<kGrid>(stage, a.z, row * a.ld, p.first(a, v), p.lane, a.cols,
                        narrow_pairs<kBf16>(x), a.bounds(kZ));
      }
    }
    if (a.stats && p.warp == 0 && p.lane == 0 &&
        a.bounds(kStats).holds(a.stats + row, 16, kSiteStore))
      a.stats[row] = make_float4(post ? sy.x : 0.f, post ? sy.y : 0.f, sh.x, sh.y);
  }
}

// Sums over the rows of a thread's own columns. Two of them have room in registers
// until the rows are done: P and A or, with ZERO_NORM_LAYER, Q and B, while P and A
// then are in shared memory, eight floats for each sum and vector in the thread's
// own words.
template <bool kLayer, int kV>
struct ColumnSums {
  float4* own;
  Eight r[2][kV];
  __device__ __forceinline__ float4* at(int k, int v) const {
    return own + (k * kV + v) * 2 * kMaxThreads;
  }
  __device__ __forceinline__ explicit ColumnSums(float4* sums) : own(sums + threadIdx.x) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int v = 0; v < kV; ++v) {
        r[k][v] = Eight{{both(0.f), both(0.f), both(0.f), both(0.f)}};
        if constexpr (kLayer) put(k, v, r[k][v]);
      }
  }
  __device__ __forceinline__ void put(int k, int v, const Eight& e) const {
    write_eight_at(at(k, v), kMaxThreads, e);
  }
  // P (0) or A (1) += x y
  __device__ __forceinline__ void add(int k, int v, const Eight& x, const Eight& y) {
    Eight s = kLayer ? read_eight_at(at(k, v), kMaxThreads) : r[k][v];
#pragma unroll
    for (int j = 0; j < 4; ++j) s.p[j] = fma2(x.p[j], y.p[j], s.p[j]);
    if constexpr (kLayer) put(k, v, s);
    else r[k][v] = s;
  }
  // Q (0) or B (1) += x
  __device__ __forceinline__ void add(int k, int v, const Eight& x) {
#pragma unroll
    for (int j = 0; j < 4; ++j) r[k][v].p[j] = r[k][v].p[j] + x.p[j];
  }
  // those in registers into shared memory
  __device__ __forceinline__ void leave() const {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int v = 0; v < kV; ++v) put(k, v, r[k][v]);
  }
};

// a row's sums, by their place among the values that a team adds up: those for
// the norm before the next block (one, or two with ZERO_NORM_LAYER), then those
// for the norm after this one
enum { kGH, kG1, kRowSums = 8 };
template <bool kLayer>
struct Branch {
  static constexpr int kFirst = kLayer ? 2 : 1;
  static constexpr int kYE = kFirst, kYH = kYE + 1, kY1 = kYE + 2, kE1 = kYE + 3, kH1 = kYE + 4,
                       kK1 = kYE + 5;
};
static_assert(kRowSums <= kMaxValues, "exchange");

// kPost: there is a norm after the block.
template <bool kBf16, bool kGrid, bool kLayer, bool kPost, int kV>
__global__ void __launch_bounds__(kMaxThreads, 1) join_grad_kernel(const Args a) {
  using B = Branch<kLayer>;
  constexpr int kValues = !kPost ? B::kFirst : kLayer ? kRowSums : 3;
  pdl_begin();
  extern __shared__ float4 smem[];
  __shared__ Exchange exchange;
  __shared__ __align__(16) uint8_t stages[kGrid ? 16 : kMaxWarps * kStagePitch];
  float4* sums_smem = smem + 2 * 2 * a.slots_of_row;  // behind the columns' numbers
  const Place p(a);
  uint8_t* stage = stages + (kGrid ? 0 : (threadIdx.x >> 5) * kStagePitch);
  int turn = 0;
  const bool pre = a.param[kWPre] != nullptr;
  const bool need_y = kPost || a.param[kGate] != nullptr;
  const uint32_t step = step_of(a.drop);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * a.teams;
  int64_t row = static_cast<int64_t>(blockIdx.x) * a.teams + p.team;
  int col[kV], there[kV];
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    col[v] = p.first(a, v) + p.lane * kVec;
    there[v] = max(0, min(kVec, a.cols - col[v]));
  }
  float4 st = make_float4(0.f, 0.f, 0.f, 0.f);
  const Ahead<4, kV, kGrid> ahead(sums_smem + 2 * kV * 2 * kMaxThreads);
#pragma unroll
  for (int v = 0; v < kV; ++v)
    if (kGrid && there[v] == 0) ahead.clear(v);
  const auto start = [&](int64_t r) {
    const int64_t at = r * a.ld;
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      const int first = p.first(a, v);
      if (pre) ahead.start(0, v, a.dz, at, first, a.cols, a.bounds(kDz));
      if (pre) ahead.start(1, v, a.h_out, at, first, a.cols, a.bounds(kHOut));
      if (a.dh_out) ahead.start(2, v, a.dh_out, at, first, a.cols, a.bounds(kDhOut));
      if (need_y) ahead.start(3, v, a.y, at, first, a.cols, a.bounds(kY));
    }
    if ((kPost || pre) && a.bounds(kStats).holds(a.stats + r, 16, kSiteLoad)) st = a.stats[r];
  };
  if (row < a.rows) start(row);  // under way while the columns' numbers are set up
  stage_columns<kBf16, 2>(a, smem);
  ColumnSums<kLayer, kV> sums(sums_smem);
  clear(exchange);
  for (; row < a.rows; row += stride) {
    const float2 sy = make_float2(st.x, st.y);
    const float2 sh = pre ? make_float2(st.z, st.w) : make_float2(0.f, 0.f);
    const int64_t at = row * a.ld;
    const uint4 none = make_uint4(0, 0, 0, 0);
    uint4 y[kV], h[kV], dz[kV], up[kV];
    ahead.wait();
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      dz[v] = pre ? ahead.read(0, v, a.dz, at, there[v]) : none;
      h[v] = pre ? ahead.read(1, v, a.h_out, at, there[v]) : none;
      up[v] = a.dh_out ? ahead.read(2, v, a.dh_out, at, there[v]) : none;
      y[v] = need_y ? ahead.read(3, v, a.y, at, there[v]) : none;
    }
    ahead.done();
    if (row + stride < a.rows) start(row + stride);
    Eight d[kV], xh[kV], xy[kV];  // E, then D; h^; y^ (or y)
    uint32_t keep[kV];
    Pair part[kValues];
#pragma unroll
    for (int q = 0; q < kValues; ++q) part[q] = both(0.f);
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      const Eight w = column(a, smem, kPre, col[v]), g0 = widen_pairs<kBf16>(dz[v]);
      Eight g;
      xh[v] = widen_pairs<kBf16>(h[v]);
      xy[v] = widen_pairs<kBf16>(y[v]);
      d[v] = widen_pairs<kBf16>(up[v]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        xh[v].p[j] = normed<kLayer>(xh[v].p[j], sh);
        g.p[j] = g0.p[j] * w.p[j];
        part[kGH] = fma2(g.p[j], xh[v].p[j], part[kGH]);
        d[v].p[j] = fma2(g.p[j], both(sh.y), d[v].p[j]);
      }
      sums.add(0, v, g0, xh[v]);
      if constexpr (kLayer) {
        sums.add(0, v, g0);
#pragma unroll
        for (int j = 0; j < 4; ++j) part[kG1] = part[kG1] + g.p[j];
      }
      if (a.drop.threshold) keep[v] = kept(a.drop, step, row, col[v]);
      if constexpr (kPost) {
        Eight k = column(a, smem, kC, col[v]);
        if (a.drop.threshold) drop_pairs(a.drop, keep[v], k);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          xy[v].p[j] = normed<kLayer>(xy[v].p[j], sy);
          const Pair ky = k.p[j] * xy[v].p[j];
          part[B::kYE] = fma2(ky, d[v].p[j], part[B::kYE]);
          part[B::kYH] = fma2(ky, xh[v].p[j], part[B::kYH]);
          if constexpr (kLayer) {
            part[B::kY1] = part[B::kY1] + ky;
            part[B::kE1] = fma2(k.p[j], d[v].p[j], part[B::kE1]);
            part[B::kH1] = fma2(k.p[j], xh[v].p[j], part[B::kH1]);
            part[B::kK1] = part[B::kK1] + k.p[j];
          }
        }
      }
    }
    // r c1, r c2, mean(k D y^), mean(k D)
    float s[kValues];
#pragma unroll
    for (int q = 0; q < kValues; ++q) s[q] = sum_of(part[q]);
    team_sum(a, p, exchange, turn, s);
    const float c1 = sh.y * (s[kGH] * a.inv_cols);
    float c2 = 0.f, along = 0.f, flat = 0.f;
    if constexpr (kLayer) c2 = sh.y * (s[kG1] * a.inv_cols);
    if constexpr (kPost) {
      along = s[B::kYE] - c1 * s[B::kYH];
      if constexpr (kLayer) {
        along -= c2 * s[B::kY1];
        flat = (s[B::kE1] - (c1 * s[B::kH1] + c2 * s[B::kK1])) * a.inv_cols;
      }
      along *= a.inv_cols;
    }
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      Eight e;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        d[v].p[j] = fma2(xh[v].p[j], both(-c1), d[v].p[j]);
        if constexpr (kLayer) d[v].p[j] = d[v].p[j] + both(-c2);
        e.p[j] = d[v].p[j] * both(a.stream_scale);
      }
      store_at<kGrid>(stage, a.dh, row * a.ld, p.first(a, v), p.lane, a.cols,
                      narrow_pairs<kBf16>(e), a.bounds(kDh));
      if (a.drop.threshold) drop_pairs(a.drop, keep[v], d[v]);
      if (need_y) {
        // what was left out of y counts for nothing in the gate's gradient either
        if (!kPost && a.drop.threshold) xy[v] = kept_only(keep[v], xy[v]);
        sums.add(1, v, d[v], xy[v]);
        if constexpr (kLayer) sums.add(1, v, d[v]);
      }
      const Eight c = column(a, smem, kC, col[v]);
#pragma unroll
      for (int j = 0; j < 4; ++j) e.p[j] = d[v].p[j] * c.p[j];
      if constexpr (kPost)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          Pair t = fma2(xy[v].p[j], both(-along), e.p[j]);
          if constexpr (kLayer) t = t + both(-flat);
          e.p[j] = t * both(sy.y);
        }
      store_at<kGrid>(stage, a.dy, row * a.ld, p.first(a, v), p.lane, a.cols,
                      narrow_pairs<kBf16>(e), a.bounds(kDy));
    }
  }
  // this CTA's vectors: the teams' sums joined in order, P and A, then Q and B by
  // the same words
  if (a.slots == 0) return;
  const int team_threads = 32 * a.team_warps;
  float* part = a.parts + static_cast<int64_t>(blockIdx.x) * a.slots * a.pitch;
  for (int round = 0; round < (kLayer ? 2 : 1); ++round) {
    if (!kLayer || round) sums.leave();
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.slots_of_row; i += blockDim.x) {
      const int q = i / a.slots_of_row, vector = i - q * a.slots_of_row;
      const int v = vector / team_threads, t = vector - v * team_threads;
      const int slot = a.slot[2 * round + q], c = vector * kVec;
      if (slot < 0 || c >= a.pitch) continue;
      const float4* from = sums_smem + (q * kV + v) * 2 * kMaxThreads + t;
      Eight s = read_eight_at(from, kMaxThreads);
      for (int k = 1; k < a.teams; ++k) {
        const Eight x = read_eight_at(from + k * team_threads, kMaxThreads);
#pragma unroll
        for (int j = 0; j < 4; ++j) s.p[j] = s.p[j] + x.p[j];
      }
      float* to = part + static_cast<int64_t>(slot) * a.pitch + c;
      if (a.bounds(kParts).holds(to, 32, kSiteStore))
        write_eight_at(reinterpret_cast<float4*>(to), 1, s);
    }
    __syncthreads();
  }
}

// The vectors of all CTAs, in order, and the parameters' gradients from them. A
// CTA takes 32 columns of P and Q (blockIdx.y 0) or A and B (1); its 32 groups
// of eight lanes, four columns each, a share of the vectors.
struct JoinArgs : Checked<1> {
  const float* parts;
  const uint16_t* param[kParams];
  uint16_t* grad[kParams];
  int32_t slot[kSums];
  int32_t n_parts, slots, cols, pitch;
  float branch_scale;
};

constexpr int kJoinThreads = 256, kJoinGroups = kJoinThreads / 8;
constexpr int kJoinEach = (kMaxParts + kJoinGroups - 1) / kJoinGroups;  // vectors of a group

template <bool kBf16>
__global__ void __launch_bounds__(kJoinThreads) join_parts_kernel(const JoinArgs a) {
  pdl_begin();
  __shared__ float4 sums[2][kJoinThreads / 32][8];
  const int lane = threadIdx.x & 7, group = threadIdx.x >> 3;
  const bool branch = blockIdx.y != 0;
  const int c = (blockIdx.x * 8 + lane) * 4;
  const int64_t step = static_cast<int64_t>(a.slots) * a.pitch;
  // all loads before the first sum: a group's vectors are kJoinGroups apart
  float4 x[2][kJoinEach];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int slot = branch ? a.slot[k ? kSumB : kSumA] : a.slot[k ? kSumQ : kSumP];
#pragma unroll
    for (int q = 0; q < kJoinEach; ++q) {
      const int part = q * kJoinGroups + group;
      const float* from = a.parts + part * step + static_cast<int64_t>(slot) * a.pitch + c;
      x[k][q] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (slot >= 0 && c < a.pitch && part < a.n_parts && a.bounds(0).holds(from, 16, kSiteLoad))
        x[k][q] = *reinterpret_cast<const float4*>(from);
    }
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float4 s = x[k][0];
#pragma unroll
    for (int q = 1; q < kJoinEach; ++q)
      s.x += x[k][q].x, s.y += x[k][q].y, s.z += x[k][q].z, s.w += x[k][q].w;
#pragma unroll
    for (int d = 8; d < 32; d *= 2) {
      s.x += __shfl_xor_sync(0xffffffffu, s.x, d);
      s.y += __shfl_xor_sync(0xffffffffu, s.y, d);
      s.z += __shfl_xor_sync(0xffffffffu, s.z, d);
      s.w += __shfl_xor_sync(0xffffffffu, s.w, d);
    }
    if ((threadIdx.x & 31) < 8) sums[k][threadIdx.x >> 5][lane] = s;
  }
  __syncthreads();
  // a warp: one column per thread
  const int t = threadIdx.x, at = blockIdx.x * 32 + t;
  if (t >= 32 || at >= a.cols) return;
  float s[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    s[k] = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinThreads / 32; ++w)
      s[k] += reinterpret_cast<const float*>(&sums[k][w][0])[t];
  }
  const auto param = [&](int w, float none) {
    return a.param[w] ? widen<kBf16>(a.param[w][at]) : none;
  };
  if (!branch) {
    if (a.grad[kWPre]) a.grad[kWPre][at] = narrow<kBf16>(s[0]);
    if (a.grad[kBPre]) a.grad[kBPre][at] = narrow<kBf16>(s[1]);
  } else {
    const float scale = a.branch_scale * param(kGate, 1.f);
    if (a.grad[kWPost]) a.grad[kWPost][at] = narrow<kBf16>(scale * s[0]);
    if (a.grad[kBPost]) a.grad[kBPost][at] = narrow<kBf16>(scale * s[1]);
    if (a.grad[kGate])
      a.grad[kGate][at] = narrow<kBf16>(
          a.branch_scale * __fmaf_rn(param(kWPost, 1.f), s[0], param(kBPost, 0.f) * s[1]));
  }
}

// -------------------------------------------------------------------- host ----

int64_t pitch_of(int64_t cols) { return ceil_div(cols, kVec) * kVec; }

// A row's team of warps and a CTA's teams; returns the vectors per thread, which
// is the most that both the row and `most` allow. Where that leaves too few warps
// for the device (few rows: a call's latency counts), a thread takes fewer.
int set_teams(Args& a, int64_t rows, int64_t cols, int most) {
  const int64_t vectors = ceil_div(cols, kVec);
  int per = 1;
  while (per < most && 32 * per < vectors) per *= 2;
  while (per > 1 && ceil_div(vectors, 32 * per / 2) <= kMaxWarps &&
         rows * ceil_div(vectors, 32 * per) < kMaxParts * kMaxWarps / 2)
    per /= 2;
  // two vectors per thread leave up to half of a row's last warp idle: one, where
  // that fits a quarter tighter (8192 x 768 backward 25 us against 27). Forward a
  // team is as it comes, with up to 46 % of its places empty (1111 columns).
  const auto room = [&](int n) { return n * ceil_div(vectors, 32 * n); };
  if (most == kBackVectors && per == 2 && vectors <= kMaxThreads && 4 * room(2) > 5 * room(1))
    per = 1;
  a.team_warps = static_cast<int32_t>(ceil_div(vectors, 32 * per));
  a.teams = static_cast<int32_t>(std::min<int64_t>(
      kMaxWarps / a.team_warps, std::max<int64_t>(1, ceil_div(rows, kMaxParts))));
  a.slots_of_row = 32 * per * a.team_warps;
  a.pitch = static_cast<int32_t>(pitch_of(cols));
  return per;
}

int check(const zero_join_params* p, const zero_join_weights* w, int64_t rows, int64_t cols,
          int64_t ld, int32_t dtype) {
  if (!p || !w || rows < 0 || cols < 0 || ld < cols || !is_dtype16(dtype)) return ZERO_EINVAL;
  if (p->norm != ZERO_NORM_RMS && p->norm != ZERO_NORM_LAYER) return ZERO_EINVAL;
  // as the kernels have them, in fp32 (comparisons that a NaN fails)
  if (!(p->eps == 0.0 || (p->eps >= FLT_MIN && p->eps <= FLT_MAX)) ||
      !(std::fabs(p->stream_scale) <= FLT_MAX) || !(std::fabs(p->branch_scale) <= FLT_MAX))
    return ZERO_EINVAL;
  if (const int bad = check_drop(p->drop)) return bad;
  const bool layer = p->norm == ZERO_NORM_LAYER;
  if ((w->b_post && (!w->w_post || !layer)) || (w->b_pre && (!w->w_pre || !layer)))
    return ZERO_EINVAL;
  if (!aligned(w->w_post, 2) || !aligned(w->b_post, 2) || !aligned(w->gate, 2) ||
      !aligned(w->w_pre, 2) || !aligned(w->b_pre, 2))
    return ZERO_EALIGN;
  if (rows >= int64_t{1} << 31 || cols > ZERO_MAX_JOIN_COLS) return ZERO_ERANGE;
  return ZERO_OK;
}

void set_common(Args& a, const zero_join_params& p, const zero_join_weights& w, int64_t rows,
                int64_t cols, int64_t ld) {
  const void* params[kParams] = {w.w_post, w.b_post, w.gate, w.w_pre, w.b_pre};
  for (int k = 0; k < kParams; ++k) {
    a.param[k] = static_cast<const uint16_t*>(params[k]);
    a.set_bounds(kParam0 + k, params[k], 1, cols, 0, 2);
  }
  a.rows = rows, a.cols = static_cast<int32_t>(cols), a.ld = ld;
  a.eps = static_cast<float>(p.eps);
  a.inv_cols = static_cast<float>(1.0 / static_cast<double>(cols));
  a.stream_scale = static_cast<float>(p.stream_scale);
  a.branch_scale = static_cast<float>(p.branch_scale);
  a.drop = drop_of(p.drop);
}

// The widest row's vectors in a team of kV per thread.
template <int kV>
constexpr int kMostSlots = std::min(32 * kV * kMaxWarps, ZERO_MAX_JOIN_COLS / kVec);
static_assert(ZERO_MAX_JOIN_COLS / kVec % (32 * kForwardVectors) == 0, "whole warps");

// `columns` numbers per column and `more` bytes of shared memory. A kernel's limit
// is the same for every call, that of its widest row: all host threads share it, and
// one that set it for a row of its own would take it from another's launch.
template <int kV, class Kernel>
cudaError_t launch_with(Kernel fn, const Args& a, int columns, int more, cudaStream_t st) {
  const int bytes = 32 * columns * a.slots_of_row + more;
  if (bytes > 32 * 1024) {  // 48 KB with the kernels' own
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               32 * columns * kMostSlots<kV> + more);
    if (e != cudaSuccess) return e;
  }
  const int64_t ctas = std::min<int64_t>(kMaxParts, ceil_div(a.rows, a.teams));
  return launch_pdl(fn, dim3(static_cast<unsigned>(ctas)), dim3(32 * a.team_warps * a.teams),
                    bytes, st, a);
}

template <bool kBf16, bool kGrid, bool kLayer, int kV>
cudaError_t launch_join_of(const Args& a, cudaStream_t st) {
  return launch_with<kV>(join_kernel<kBf16, kGrid, kLayer, kV>, a, kLayer ? 4 : 2,
                         Ahead<2, kV, kGrid>::kBytes, st);
}

template <bool kBf16, bool kGrid, bool kLayer>
cudaError_t launch_join(const Args& a, int per, cudaStream_t st) {
  return per == 1   ? launch_join_of<kBf16, kGrid, kLayer, 1>(a, st)
         : per == 2 ? launch_join_of<kBf16, kGrid, kLayer, 2>(a, st)
                    : launch_join_of<kBf16, kGrid, kLayer, 4>(a, st);
}

template <bool kBf16, bool kGrid, bool kLayer, bool kPost, int kV>
cudaError_t launch_grad_of(const Args& a, cudaStream_t st) {
  return launch_with<kV>(join_grad_kernel<kBf16, kGrid, kLayer, kPost, kV>, a, 2,
                         2 * kV * 32 * kMaxThreads + Ahead<4, kV, kGrid>::kBytes, st);
}

template <bool kBf16, bool kGrid, bool kLayer>
cudaError_t launch_grad(const Args& a, int per, cudaStream_t st) {
  if (a.param[kWPost])
    return per == 1 ? launch_grad_of<kBf16, kGrid, kLayer, true, 1>(a, st)
                    : launch_grad_of<kBf16, kGrid, kLayer, true, 2>(a, st);
  return per == 1 ? launch_grad_of<kBf16, kGrid, kLayer, false, 1>(a, st)
                  : launch_grad_of<kBf16, kGrid, kLayer, false, 2>(a, st);
}

// fn<bf16, grid, layer>(...) for run-time values
#define ZJ_PICK(fn, bf16, grid, layer, ...)                                              \
  ((bf16) ? ((grid) ? ((layer) ? fn<true, true, true>(__VA_ARGS__)                       \
                               : fn<true, true, false>(__VA_ARGS__))                     \
                    : ((layer) ? fn<true, false, true>(__VA_ARGS__)                      \
                               : fn<true, false, false>(__VA_ARGS__)))                   \
          : ((grid) ? ((layer) ? fn<false, true, true>(__VA_ARGS__)                      \
                               : fn<false, true, false>(__VA_ARGS__))                    \
                    : ((layer) ? fn<false, false, true>(__VA_ARGS__)                     \
                               : fn<false, false, false>(__VA_ARGS__))))

}  // namespace zj

#ifdef ZERO_CHECKED
extern "C" int zj_collect_checks(unsigned long long* count, unsigned long long* first) {
  return collect_checks(count, first);
}
#endif

extern "C" {

ZERO_API int zero_block_join(const zero_join_params* params, const zero_join_weights* weights,
                             const void* h, const void* y, int64_t rows, int64_t cols, int64_t ld,
                             int32_t dtype, void* h_out, void* z, float* stats, void* stream) {
  using namespace zj;
  if (const int bad = check(params, weights, rows, cols, ld, dtype)) return bad;
  if ((z != nullptr) != (weights->w_pre != nullptr) && rows && cols) return ZERO_EINVAL;
  if (rows == 0 || cols == 0) return ZERO_OK;
  if (!h || !y || !h_out || z == h_out) return ZERO_EINVAL;
  if (!aligned(h, 2) || !aligned(y, 2) || !aligned(h_out, 2) || !aligned(z, 2) ||
      !aligned(stats, 16))
    return ZERO_EALIGN;
  Args a = new_args<Args>();
  set_common(a, *params, *weights, rows, cols, ld);
  a.h = static_cast<const uint16_t*>(h);
  a.y = static_cast<const uint16_t*>(y);
  a.h_new = static_cast<uint16_t*>(h_out);
  a.z = static_cast<uint16_t*>(z);
  a.stats = reinterpret_cast<float4*>(stats);
  a.set_bounds(kH, h, rows, cols, ld, 2);
  a.set_bounds(kY, y, rows, cols, ld, 2);
  a.set_bounds(kHOut, h_out, rows, cols, ld, 2);
  a.set_bounds(kZ, z, rows, cols, ld, 2);
  a.set_bounds(kStats, stats, 1, rows, rows, 16);
  const int per = set_teams(a, rows, cols, kForwardVectors);
  const bool grid = cols % kVec == 0 && on_grid(h, ld) && aligned(y, 16) && aligned(h_out, 16) &&
                    aligned(z, 16);
  return status_of(ZJ_PICK(launch_join, dtype == ZERO_BF16, grid, params->norm == ZERO_NORM_LAYER,
                           a, per, static_cast<cudaStream_t>(stream)));
}

ZERO_API size_t zero_block_join_workspace_bytes(int64_t rows, int64_t cols) {
  using namespace zj;
  if (rows < 0 || cols < 0 || rows >= int64_t{1} << 31 || cols > ZERO_MAX_JOIN_COLS) return 0;
  return static_cast<size_t>(std::min<int64_t>(rows, kMaxParts) * kSums * pitch_of(cols) * 4);
}

ZERO_API int zero_block_join_grad(const zero_join_params* params, const zero_join_weights* weights,
                                  const void* h_out, const void* y, const float* stats,
                                  const void* dz, const void* dh_out, int64_t rows, int64_t cols,
                                  int64_t ld, int32_t dtype, void* dh, void* dy,
                                  const zero_join_weights* grads, void* workspace, void* stream) {
  using namespace zj;
  if (const int bad = check(params, weights, rows, cols, ld, dtype)) return bad;
  if (!grads) return ZERO_EINVAL;
  const void* w[kParams] = {weights->w_post, weights->b_post, weights->gate, weights->w_pre,
                            weights->b_pre};
  void* g[kParams] = {grads->w_post, grads->b_post, grads->gate, grads->w_pre, grads->b_pre};
  for (int k = 0; k < kParams; ++k) {
    if ((w[k] != nullptr) != (g[k] != nullptr)) return ZERO_EINVAL;
    if (!aligned(g[k], 2)) return ZERO_EALIGN;
  }
  if (cols == 0) return ZERO_OK;
  JoinArgs j = new_args<JoinArgs>();
  Args a = new_args<Args>();
  const bool needed[kSums] = {g[kWPre] != nullptr, g[kWPost] || g[kGate], g[kBPre] != nullptr,
                              g[kBPost] != nullptr};
  for (int k = 0; k < kSums; ++k) a.slot[k] = j.slot[k] = needed[k] ? j.slots++ : -1;
  for (int k = 0; k < kParams; ++k) {
    j.param[k] = static_cast<const uint16_t*>(w[k]);
    j.grad[k] = static_cast<uint16_t*>(g[k]);
  }
  j.branch_scale = static_cast<float>(params->branch_scale);
  j.parts = static_cast<const float*>(workspace);
  j.cols = static_cast<int32_t>(cols), j.pitch = static_cast<int32_t>(pitch_of(cols));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf16 = dtype == ZERO_BF16;
  if (rows) {
    if (!dh || !dy || dh == dy || ((w[kWPost] || w[kWPre]) && !stats) ||
        (w[kWPre] && (!h_out || !dz)) || (!w[kWPre] && dz) || ((w[kWPost] || w[kGate]) && !y) ||
        (j.slots && !workspace))
      return ZERO_EINVAL;
    if (!aligned(h_out, 2) || !aligned(y, 2) || !aligned(dz, 2) || !aligned(dh_out, 2) ||
        !aligned(dh, 2) || !aligned(dy, 2) || !aligned(stats, 16) || !aligned(workspace, 16))
      return ZERO_EALIGN;
    set_common(a, *params, *weights, rows, cols, ld);
    a.h_out = static_cast<const uint16_t*>(h_out);
    a.y = static_cast<const uint16_t*>(y);
    a.dz = static_cast<const uint16_t*>(dz);
    a.dh_out = static_cast<const uint16_t*>(dh_out);
    a.dh = static_cast<uint16_t*>(dh);
    a.dy = static_cast<uint16_t*>(dy);
    a.stats = reinterpret_cast<float4*>(const_cast<float*>(stats));
    a.parts = static_cast<float*>(workspace);
    a.slots = j.slots;
    const int per = set_teams(a, rows, cols, kBackVectors);
    const int64_t ctas = std::min<int64_t>(kMaxParts, ceil_div(rows, a.teams));
    j.n_parts = static_cast<int32_t>(ctas);
    a.set_bounds(kHOut, h_out, rows, cols, ld, 2);
    a.set_bounds(kY, y, rows, cols, ld, 2);
    a.set_bounds(kStats, stats, 1, rows, rows, 16);
    a.set_bounds(kDz, dz, rows, cols, ld, 2);
    a.set_bounds(kDhOut, dh_out, rows, cols, ld, 2);
    a.set_bounds(kDh, dh, rows, cols, ld, 2);
    a.set_bounds(kDy, dy, rows, cols, ld, 2);
    a.set_bounds(kParts, workspace, 1, ctas * j.slots * j.pitch, 0, 4);
    const bool grid = cols % kVec == 0 && on_grid(dh, ld) && aligned(dy, 16) &&
                      aligned(h_out, 16) && aligned(y, 16) && aligned(dz, 16) && aligned(dh_out, 16);
    const int bad = status_of(ZJ_PICK(launch_grad, bf16, grid, params->norm == ZERO_NORM_LAYER, a,
                                      per, st));
    if (bad) return bad;
  }
  if (j.slots == 0) return ZERO_OK;
  j.set_bounds(0, workspace, 1, static_cast<int64_t>(j.n_parts) * j.slots * j.pitch, 0, 4);
  const dim3 blocks(static_cast<unsigned>(ceil_div(cols, 32)), 2);
  return status_of(launch_pdl(bf16 ? join_parts_kernel<true> : join_parts_kernel<false>, blocks,
                              dim3(kJoinThreads), 0, st, j));
}

}  // extern "C"
