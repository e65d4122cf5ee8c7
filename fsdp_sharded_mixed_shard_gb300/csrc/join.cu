/*
 * join.cu -- where a block's output joins the residual stream: norms after the
 * block and before the next, gate, dropout and residual scale (zero_block.h).
 *
 * A team of warps holds a row in registers, eight neighbouring columns per
 * thread (two times eight past 4096 columns), from the load to the last store:
 * forward 8 bytes per element, backward 12, and nothing is read twice. What a
 * norm needs of the whole row (a sum of squares; with ZERO_NORM_LAYER the mean
 * before it, from which the squares are then taken) goes through shuffles and,
 * past 256 columns, one exchange between the team's warps. Each team works
 * through rows of its own with the next row's loads under way.
 *
 * With m the dropout's factor (0 or its scale), c = branch_scale gate w_post and
 * d = branch_scale gate b_post, the forward pass is
 *   h_out = stream_scale h + m (c y^ + d)
 * and the backward pass needs, of each column, only
 *   P = sum dz h^,  Q = sum dz,  A = sum m D y^,  B = sum m D   over the rows:
 *   dw_pre = P, db_pre = Q, dw_post = branch_scale gate A,
 *   db_post = branch_scale gate B, dgate = branch_scale (w_post A + b_post B).
 * c, d and these sums are kept per thread, in fp32 registers (in shared memory
 * past 4096 columns). A CTA joins its teams' sums in order and leaves one vector
 * each in the workspace; a second kernel adds the (at most kMaxParts) vectors in
 * order.
 */
#include "draws.cuh"
#include "rows.cuh"

#include <algorithm>
#include <cmath>

namespace zj {

using namespace zt;

constexpr int kMaxThreads = 512;
constexpr int kMaxWarps = kMaxThreads / 32;
constexpr int kMaxParts = 152;  // CTAs of the backward pass: one per SM
static_assert(ZERO_MAX_JOIN_COLS == 2 * kMaxThreads * kVec, "two vectors per thread");

// threads per SM of the forward pass: 64 registers each, 96 with the means and
// biases of ZERO_NORM_LAYER
template <bool kLayer>
__device__ __host__ constexpr int resident_threads() { return kLayer ? 640 : 1024; }

enum { kH, kY, kHOut, kZ, kStats, kDz, kDhOut, kDh, kDy, kParts, kBuffers };  // of a call
enum { kWPost, kBPost, kGate, kWPre, kBPre, kParams };
enum { kSumP, kSumQ, kSumA, kSumB, kSums };

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
  int32_t team_warps, teams;
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

__device__ __forceinline__ void drop_pairs(const Drop& d, const uint4& draw, Eight& e) {
  float f[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) unpair(e.p[j], f[2 * j], f[2 * j + 1]);
  drop8(d, draw, f);
#pragma unroll
  for (int j = 0; j < 4; ++j) e.p[j] = pair(f[2 * j], f[2 * j + 1]);
}

// kCount numbers for each of a thread's columns: in registers, or, where it has
// two vectors, in shared memory (its own words, 16 bytes a lane).
template <int kV, int kCount>
struct Columns {
  Eight r[kCount];
  __device__ __forceinline__ explicit Columns(float4*) {}
  __device__ __forceinline__ Eight get(int k, int) const { return r[k]; }
  __device__ __forceinline__ void set(int k, int, const Eight& e) { r[k] = e; }
};

template <int kCount>
struct Columns<2, kCount> {
  float4* own;
  __device__ __forceinline__ explicit Columns(float4* smem) : own(smem + threadIdx.x) {}
  __device__ __forceinline__ float4* at(int k, int v) const {
    return own + (k * 2 + v) * 2 * kMaxThreads;
  }
  __device__ __forceinline__ Eight get(int k, int v) const {
    const float4 x = at(k, v)[0], y = at(k, v)[kMaxThreads];
    return Eight{{pair(x.x, x.y), pair(x.z, x.w), pair(y.x, y.y), pair(y.z, y.w)}};
  }
  __device__ __forceinline__ void set(int k, int v, const Eight& e) {
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) unpair(e.p[j], f[2 * j], f[2 * j + 1]);
    at(k, v)[0] = make_float4(f[0], f[1], f[2], f[3]);
    at(k, v)[kMaxThreads] = make_float4(f[4], f[5], f[6], f[7]);
  }
};

template <int kV>
constexpr int columns_bytes(int count) { return kV == 1 ? 0 : count * 2 * kMaxThreads * kVec * 4; }

// A team's warps' sums, each team's padded with zeros to whole float4. Two sets
// in turn, so that one barrier each is enough: a warp that writes to one again
// has passed the other's barrier, before which all have read this one's.
struct Exchange {
  float4 sums[2][2][8];  // [set][value]
};

// of every thread of the CTA, before the first sum
__device__ __forceinline__ void clear(Exchange& ex) {
  if (threadIdx.x < 32) (&ex.sums[0][0][0])[threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
  __syncthreads();
}

// Sums over the team, the same bits in all its threads.
template <int kValues>
__device__ __forceinline__ void team_sum(const Args& a, const Place& p, Exchange& ex, int& turn,
                                         float (&x)[kValues]) {
#pragma unroll
  for (int k = 0; k < kValues; ++k)
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x[k] += __shfl_xor_sync(0xffffffffu, x[k], d);
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
  // squares past fp32's range: NaN, not 0
  return mean_square < __uint_as_float(0x7F800000u) ? rsqrtf(mean_square + eps)
                                                    : __uint_as_float(0x7FC00000u);
}

// A row held by the team -> (x - mean) r in place; returns (mean or 0, r).
// `there`: how many of the thread's columns of each vector are columns.
template <bool kLayer, int kV>
__device__ __forceinline__ float2 normalise(const Args& a, const Place& p, Exchange& ex, int& turn,
                                            Eight (&x)[kV], const int (&there)[kV]) {
  float mean = 0.f;
  if constexpr (kLayer) {
    Pair s = both(0.f);
#pragma unroll
    for (int v = 0; v < kV; ++v)
      s = s + ((x[v].p[0] + x[v].p[1]) + (x[v].p[2] + x[v].p[3]));
    float sum[1] = {sum_of(s)};
    team_sum<1>(a, p, ex, turn, sum);
    mean = sum[0] * a.inv_cols;
#pragma unroll
    for (int v = 0; v < kV; ++v) {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[v].p[j] = x[v].p[j] + both(-mean);
      if (there[v] < kVec) {  // past the last column 0 is not a value
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float lo, hi;
          unpair(x[v].p[j], lo, hi);
          x[v].p[j] = pair(2 * j < there[v] ? lo : 0.f, 2 * j + 1 < there[v] ? hi : 0.f);
        }
      }
    }
  }
  Pair s = both(0.f);
#pragma unroll
  for (int v = 0; v < kV; ++v)
#pragma unroll
    for (int j = 0; j < 4; ++j) s = fma2(x[v].p[j], x[v].p[j], s);
  float sum[1] = {sum_of(s)};
  team_sum<1>(a, p, ex, turn, sum);
  const float r = inverse_root(sum[0] * a.inv_cols, a.eps);
#pragma unroll
  for (int v = 0; v < kV; ++v)
#pragma unroll
    for (int j = 0; j < 4; ++j) x[v].p[j] = x[v].p[j] * both(r);
  return make_float2(mean, r);
}

// (x - mean) r
template <bool kLayer>
__device__ __forceinline__ Pair normed(const Pair& x, const float2& st) {
  return kLayer ? (x + both(-st.x)) * both(st.y) : x * both(st.y);
}

// Eight of a parameter's elements, `none` where there is no parameter.
template <bool kBf16>
__device__ __forceinline__ Eight load_param(const uint16_t* w, int c, int cols, float none) {
  if (w) return widen_pairs<kBf16>(load8<false>(w, c, cols, Bounds{}));
  return Eight{{both(none), both(none), both(none), both(none)}};
}

__device__ __forceinline__ Eight scaled(const Eight& x, const Eight& y, float s) {
  Eight e;
#pragma unroll
  for (int j = 0; j < 4; ++j) e.p[j] = x.p[j] * both(s) * y.p[j];
  return e;
}

constexpr int kStagePitch = (kStageWarp + 15) & ~15;

enum { kC, kPre, kD, kBias };  // the forward pass's numbers per column

template <bool kBf16, bool kGrid, bool kLayer, int kV>
__global__ void __launch_bounds__(kV == 1 ? resident_threads<kLayer>() : kMaxThreads, 1)
    join_kernel(const Args a) {
  pdl_begin();
  extern __shared__ float4 smem_columns[];
  __shared__ Exchange exchange;
  __shared__ __align__(16) uint8_t stages[kGrid ? 16 : kMaxWarps * kStagePitch];
  const Place p(a);
  uint8_t* stage = stages + (kGrid ? 0 : (threadIdx.x >> 5) * kStagePitch);
  int turn = 0;
  const bool post = a.param[kWPost] != nullptr, pre = a.param[kWPre] != nullptr;
  Columns<kV, kLayer ? 4 : 2> w(smem_columns);
  int col[kV], there[kV];
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    col[v] = p.first(a, v) + p.lane * kVec;
    there[v] = max(0, min(kVec, a.cols - col[v]));
    const Eight gate = load_param<kBf16>(a.param[kGate], col[v], a.cols, 1.f);
    w.set(kC, v, scaled(gate, load_param<kBf16>(a.param[kWPost], col[v], a.cols, 1.f),
                        a.branch_scale));
    w.set(kPre, v, load_param<kBf16>(a.param[kWPre], col[v], a.cols, 0.f));
    if constexpr (kLayer) {
      w.set(kD, v, scaled(gate, load_param<kBf16>(a.param[kBPost], col[v], a.cols, 0.f),
                          a.branch_scale));
      w.set(kBias, v, load_param<kBf16>(a.param[kBPre], col[v], a.cols, 0.f));
    }
  }
  clear(exchange);
  const uint32_t step = step_of(a.drop);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * a.teams;
  int64_t row = static_cast<int64_t>(blockIdx.x) * a.teams + p.team;
  uint4 y[kV], h[kV];
  const auto load = [&](int64_t r) {
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      y[v] = load8<kGrid>(a.y + r * a.ld, col[v], a.cols, a.bounds(kY));
      h[v] = load8<kGrid>(a.h + r * a.ld, col[v], a.cols, a.bounds(kH));
    }
  };
  if (row < a.rows) load(row);
  for (; row < a.rows; row += stride) {
    float2 sy = make_float2(0.f, 0.f), sh = sy;
    Eight x[kV];
#pragma unroll
    for (int v = 0; v < kV; ++v) x[v] = widen_pairs<kBf16>(y[v]);
    if (post) sy = normalise<kLayer, kV>(a, p, exchange, turn, x, there);
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      const Eight c = w.get(kC, v);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[v].p[j] = x[v].p[j] * c.p[j];
      if constexpr (kLayer) {
        const Eight d = w.get(kD, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[v].p[j] = x[v].p[j] + d.p[j];
      }
      if (a.drop.threshold)
        drop_pairs(a.drop,
                   draw8(a.drop, step, static_cast<uint32_t>(row),
                         static_cast<uint32_t>(col[v]) / kVec), x[v]);
      const Eight s = widen_pairs<kBf16>(h[v]);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[v].p[j] = fma2(s.p[j], both(a.stream_scale), x[v].p[j]);
      const uint4 out = narrow_pairs<kBf16>(x[v]);
      store_row<kGrid>(stage, a.h_new + row * a.ld, p.first(a, v), p.lane, a.cols, out,
                       a.bounds(kHOut));
      x[v] = widen_pairs<kBf16>(out);
    }
    if (row + stride < a.rows) load(row + stride);
    if (pre) {
      sh = normalise<kLayer, kV>(a, p, exchange, turn, x, there);
#pragma unroll
      for (int v = 0; v < kV; ++v) {
        const Eight c = w.get(kPre, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[v].p[j] = x[v].p[j] * c.p[j];
        if constexpr (kLayer) {
          const Eight d = w.get(kBias, v);
#pragma unroll
          for (int j = 0; j < 4; ++j) x[v].p[j] = x[v].p[j] + d.p[j];
        }
        store_row<kGrid>(stage, a.z + row * a.ld, p.first(a, v), p.lane, a.cols,
                         narrow_pairs<kBf16>(x[v]), a.bounds(kZ));
      }
    }
    if (a.stats && p.warp == 0 && p.lane == 0 &&
        a.bounds(kStats).holds(a.stats + row, 16, kSiteStore))
      a.stats[row] = make_float4(sy.x, sy.y, sh.x, sh.y);
  }
}

// the backward pass's numbers per column: w_pre and c, then the sums
enum { kBackPre, kBackC, kBackSums };

template <bool kLayer>
__device__ __host__ constexpr int back_columns() { return kBackSums + (kLayer ? kSums : 2); }
// where a sum is among them (without ZERO_NORM_LAYER there are P and A)
template <bool kLayer>
__device__ __host__ constexpr int back_sum(int k) { return kBackSums + (kLayer ? k : k / 2); }

template <bool kBf16, bool kGrid, bool kLayer, int kV>
__global__ void __launch_bounds__(kMaxThreads, 1) join_grad_kernel(const Args a) {
  pdl_begin();
  extern __shared__ float4 smem_columns[];
  __shared__ Exchange exchange;
  __shared__ __align__(16) uint8_t stages[kGrid ? 16 : kMaxWarps * kStagePitch];
  const Place p(a);
  uint8_t* stage = stages + (kGrid ? 0 : (threadIdx.x >> 5) * kStagePitch);
  int turn = 0;
  const bool post = a.param[kWPost] != nullptr, pre = a.param[kWPre] != nullptr;
  const bool branch_sums = post || a.param[kGate] != nullptr;
  Columns<kV, back_columns<kLayer>()> w(smem_columns);
  int col[kV];
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    col[v] = p.first(a, v) + p.lane * kVec;
    w.set(kBackPre, v, load_param<kBf16>(a.param[kWPre], col[v], a.cols, 0.f));
    w.set(kBackC, v, scaled(load_param<kBf16>(a.param[kGate], col[v], a.cols, 1.f),
                            load_param<kBf16>(a.param[kWPost], col[v], a.cols, 1.f),
                            a.branch_scale));
#pragma unroll
    for (int k = kBackSums; k < back_columns<kLayer>(); ++k)
      w.set(k, v, Eight{{both(0.f), both(0.f), both(0.f), both(0.f)}});
  }
  // a sum += x y (or x)
  const auto add = [&](int sum, int v, const Eight& x, const Eight& y) {
    Eight s = w.get(back_sum<kLayer>(sum), v);
#pragma unroll
    for (int j = 0; j < 4; ++j) s.p[j] = fma2(x.p[j], y.p[j], s.p[j]);
    w.set(back_sum<kLayer>(sum), v, s);
  };
  const auto add_one = [&](int sum, int v, const Eight& x) {
    Eight s = w.get(back_sum<kLayer>(sum), v);
#pragma unroll
    for (int j = 0; j < 4; ++j) s.p[j] = s.p[j] + x.p[j];
    w.set(back_sum<kLayer>(sum), v, s);
  };
  clear(exchange);
  const uint32_t step = step_of(a.drop);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * a.teams;
  int64_t row = static_cast<int64_t>(blockIdx.x) * a.teams + p.team;
  const uint4 none = make_uint4(0, 0, 0, 0);
  uint4 y[kV], h[kV], dz[kV], dh[kV];
  float4 st = make_float4(0.f, 0.f, 0.f, 0.f);
  const auto load = [&](int64_t r) {
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      dz[v] = pre ? load8<kGrid>(a.dz + r * a.ld, col[v], a.cols, a.bounds(kDz)) : none;
      h[v] = pre ? load8<kGrid>(a.h_out + r * a.ld, col[v], a.cols, a.bounds(kHOut)) : none;
      dh[v] = a.dh_out ? load8<kGrid>(a.dh_out + r * a.ld, col[v], a.cols, a.bounds(kDhOut)) : none;
      y[v] = branch_sums ? load8<kGrid>(a.y + r * a.ld, col[v], a.cols, a.bounds(kY)) : none;
    }
    if (a.bounds(kStats).holds(a.stats + r, 16, kSiteLoad)) st = a.stats[r];
  };
  if (row < a.rows) load(row);
  for (; row < a.rows; row += stride) {
    const float2 sy = make_float2(st.x, st.y), sh = make_float2(st.z, st.w);
    // through the norm before the next block: D, the whole gradient of h_out
    Eight d[kV];
    if (pre) {
      Pair along = both(0.f), flat = both(0.f);
      Eight x[kV], g[kV];
#pragma unroll
      for (int v = 0; v < kV; ++v) {
        const Eight c = w.get(kBackPre, v);
        const Eight up = widen_pairs<kBf16>(dz[v]);
        x[v] = widen_pairs<kBf16>(h[v]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[v].p[j] = normed<kLayer>(x[v].p[j], sh);
          g[v].p[j] = up.p[j] * c.p[j];
          along = fma2(g[v].p[j], x[v].p[j], along);
          if constexpr (kLayer) flat = flat + g[v].p[j];
        }
        add(kSumP, v, up, x[v]);
        if constexpr (kLayer) add_one(kSumQ, v, up);
      }
      float s[kLayer ? 2 : 1];
      s[0] = sum_of(along);
      if constexpr (kLayer) s[1] = sum_of(flat);
      team_sum(a, p, exchange, turn, s);
      const Pair c1 = both(-s[0] * a.inv_cols), r = both(sh.y);
#pragma unroll
      for (int v = 0; v < kV; ++v) {
        const Eight up = widen_pairs<kBf16>(dh[v]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          Pair t = fma2(x[v].p[j], c1, g[v].p[j]);
          if constexpr (kLayer) t = t + both(-s[1] * a.inv_cols);
          d[v].p[j] = fma2(t, r, up.p[j]);
        }
      }
    } else {
#pragma unroll
      for (int v = 0; v < kV; ++v) d[v] = widen_pairs<kBf16>(dh[v]);
    }
    // through gate, dropout and the norm after the block
    Pair along = both(0.f), flat = both(0.f);
    Eight x[kV];
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      Eight e;
#pragma unroll
      for (int j = 0; j < 4; ++j) e.p[j] = d[v].p[j] * both(a.stream_scale);
      store_row<kGrid>(stage, a.dh + row * a.ld, p.first(a, v), p.lane, a.cols,
                       narrow_pairs<kBf16>(e), a.bounds(kDh));
      if (a.drop.threshold)
        drop_pairs(a.drop,
                   draw8(a.drop, step, static_cast<uint32_t>(row),
                         static_cast<uint32_t>(col[v]) / kVec), d[v]);
      x[v] = widen_pairs<kBf16>(y[v]);
      if (post) {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[v].p[j] = normed<kLayer>(x[v].p[j], sy);
      }
      add(kSumA, v, d[v], x[v]);
      if constexpr (kLayer) add_one(kSumB, v, d[v]);
      const Eight c = w.get(kBackC, v);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        d[v].p[j] = d[v].p[j] * c.p[j];
        along = fma2(d[v].p[j], x[v].p[j], along);
        if constexpr (kLayer) flat = flat + d[v].p[j];
      }
    }
    if (row + stride < a.rows) load(row + stride);
    if (post) {
      float s[kLayer ? 2 : 1];
      s[0] = sum_of(along);
      if constexpr (kLayer) s[1] = sum_of(flat);
      team_sum(a, p, exchange, turn, s);
      const Pair c1 = both(-s[0] * a.inv_cols), r = both(sy.y);
#pragma unroll
      for (int v = 0; v < kV; ++v)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          Pair t = fma2(x[v].p[j], c1, d[v].p[j]);
          if constexpr (kLayer) t = t + both(-s[1] * a.inv_cols);
          d[v].p[j] = t * r;
        }
    }
#pragma unroll
    for (int v = 0; v < kV; ++v)
      store_row<kGrid>(stage, a.dy + row * a.ld, p.first(a, v), p.lane, a.cols,
                       narrow_pairs<kBf16>(d[v]), a.bounds(kDy));
  }
  // this CTA's vectors: the teams' sums joined in order
  if (a.slots == 0) return;
  float* part = a.parts + static_cast<int64_t>(blockIdx.x) * a.slots * a.pitch;
  const auto leave = [&](int slot, int c, const float4& lo, const float4& hi) {
    float* to = part + static_cast<int64_t>(slot) * a.pitch + c;
    if (c >= a.pitch || !a.bounds(kParts).holds(to, 32, kSiteStore)) return;
    reinterpret_cast<float4*>(to)[0] = lo;
    reinterpret_cast<float4*>(to)[1] = hi;
  };
  if constexpr (kV == 1) {
    const int team_threads = 32 * a.team_warps, t = p.warp * 32 + p.lane;
    for (int k = 0; k < a.teams; ++k) {
      if (p.team == k) {
#pragma unroll
        for (int q = 0; q < kSums; q += kLayer ? 1 : 2) {
          float f[8];
          const Eight e = w.get(back_sum<kLayer>(q), 0);
#pragma unroll
          for (int j = 0; j < 4; ++j) unpair(e.p[j], f[2 * j], f[2 * j + 1]);
          float4 *lo = smem_columns + (2 * q) * team_threads + t, *hi = lo + team_threads;
          const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
          const float4 x = k ? *lo : z, y4 = k ? *hi : z;
          *lo = make_float4(x.x + f[0], x.y + f[1], x.z + f[2], x.w + f[3]);
          *hi = make_float4(y4.x + f[4], y4.y + f[5], y4.z + f[6], y4.w + f[7]);
        }
      }
      __syncthreads();
    }
    for (int q = p.team; q < kSums; q += a.teams)
      if (a.slot[q] >= 0)
        leave(a.slot[q], col[0], smem_columns[2 * q * team_threads + t],
              smem_columns[(2 * q + 1) * team_threads + t]);
  } else {
    for (int q = 0; q < kSums; ++q)
      if (a.slot[q] >= 0)
        for (int v = 0; v < kV; ++v) {
          const float4* at = w.at(back_sum<kLayer>(q), v);
          leave(a.slot[q], col[v], at[0], at[kMaxThreads]);
        }
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

template <bool kBf16>
__global__ void __launch_bounds__(kJoinThreads) join_parts_kernel(const JoinArgs a) {
  pdl_begin();
  __shared__ float4 sums[2][kJoinGroups][8];
  const int lane = threadIdx.x & 7, group = threadIdx.x >> 3;
  const bool branch = blockIdx.y != 0;
  const int c = (blockIdx.x * 8 + lane) * 4;
  const int64_t step = static_cast<int64_t>(a.slots) * a.pitch;
  const int lo = a.n_parts * group / kJoinGroups, hi = a.n_parts * (group + 1) / kJoinGroups;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int slot = branch ? a.slot[k ? kSumB : kSumA] : a.slot[k ? kSumQ : kSumP];
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (slot >= 0 && c < a.pitch) {
      const float* from = a.parts + static_cast<int64_t>(slot) * a.pitch + c;
#pragma unroll 5
      for (int q = lo; q < hi; ++q) {
        if (!a.bounds(0).holds(from + q * step, 16, kSiteLoad)) continue;
        const float4 x = *reinterpret_cast<const float4*>(from + q * step);
        s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
      }
    }
    sums[k][group][lane] = s;
  }
  __syncthreads();
  // a warp: one column per thread
  const int t = threadIdx.x, at = blockIdx.x * 32 + t;
  if (t >= 32 || at >= a.cols) return;
  float s[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    s[k] = 0.f;
    for (int g = 0; g < kJoinGroups; ++g)
      s[k] += reinterpret_cast<const float*>(&sums[k][g][0])[t];
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

// A row's team, and how many of at most `threads` together a CTA has: rows are
// spread over `sms` SMs first.
void set_teams(Args& a, int64_t rows, int64_t cols, int threads) {
  const int64_t vectors = ceil_div(cols, kVec), per = vectors > kMaxThreads ? 2 : 1;
  a.team_warps = static_cast<int32_t>(ceil_div(ceil_div(vectors, per), 32));
  const int64_t most = std::max(1, threads / 32 / a.team_warps);
  a.teams = static_cast<int32_t>(std::min(most, std::max<int64_t>(1, ceil_div(rows, kMaxParts))));
  a.pitch = static_cast<int32_t>(pitch_of(cols));
}

int check(const zero_join_params* p, const zero_join_weights* w, int64_t rows, int64_t cols,
          int64_t ld, int32_t dtype) {
  if (!p || !w || rows < 0 || cols < 0 || ld < cols || !is_dtype16(dtype)) return ZERO_EINVAL;
  if (p->norm != ZERO_NORM_RMS && p->norm != ZERO_NORM_LAYER) return ZERO_EINVAL;
  if (!(p->eps >= 0.0) || !std::isfinite(p->eps) || !std::isfinite(p->stream_scale) ||
      !std::isfinite(p->branch_scale))
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
  for (int k = 0; k < kParams; ++k) a.param[k] = static_cast<const uint16_t*>(params[k]);
  a.rows = rows, a.cols = static_cast<int32_t>(cols), a.ld = ld;
  a.eps = static_cast<float>(p.eps);
  a.inv_cols = static_cast<float>(1.0 / static_cast<double>(cols));
  a.stream_scale = static_cast<float>(p.stream_scale);
  a.branch_scale = static_cast<float>(p.branch_scale);
  a.drop = drop_of(p.drop);
}

template <class Kernel>
cudaError_t launch_with(Kernel fn, const Args& a, int64_t ctas, int bytes, cudaStream_t st) {
  if (bytes > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(fn, dim3(static_cast<unsigned>(ctas)), dim3(32 * a.team_warps * a.teams),
                    bytes, st, a);
}

template <bool kBf16, bool kGrid, bool kLayer>
cudaError_t launch_join(Args& a, cudaStream_t st) {
  constexpr int kThreads = resident_threads<kLayer>();
  set_teams(a, a.rows, a.cols, 256);
  const int per_sm = std::max(1, kThreads / (32 * a.team_warps * a.teams));
  const int64_t ctas = std::min<int64_t>(per_sm * kMaxParts, ceil_div(a.rows, a.teams));
  if (a.pitch <= kMaxThreads * kVec)
    return launch_with(join_kernel<kBf16, kGrid, kLayer, 1>, a, ctas, 0, st);
  return launch_with(join_kernel<kBf16, kGrid, kLayer, 2>, a,
                     std::min<int64_t>(kMaxParts, ctas), columns_bytes<2>(kLayer ? 4 : 2), st);
}

template <bool kBf16, bool kGrid, bool kLayer>
cudaError_t launch_grad(const Args& a, int64_t ctas, cudaStream_t st) {
  // one vector: room to join the teams' sums
  return a.pitch <= kMaxThreads * kVec
             ? launch_with(join_grad_kernel<kBf16, kGrid, kLayer, 1>, a, ctas,
                           kSums * 32 * a.team_warps * kVec * 4, st)
             : launch_with(join_grad_kernel<kBf16, kGrid, kLayer, 2>, a, ctas,
                           columns_bytes<2>(back_columns<kLayer>()), st);
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
  const bool grid = on_grid(h, ld) && aligned(y, 16) && aligned(h_out, 16) && aligned(z, 16);
  return status_of(ZJ_PICK(launch_join, dtype == ZERO_BF16, grid, params->norm == ZERO_NORM_LAYER,
                           a, static_cast<cudaStream_t>(stream)));
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
  const bool needed[kSums] = {g[kWPre] != nullptr, g[kBPre] != nullptr,
                              g[kWPost] || g[kGate], g[kBPost] != nullptr};
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
    if (!dh || !dy || !stats || dh == dy || (w[kWPre] && (!h_out || !dz)) || (!w[kWPre] && dz) ||
        ((w[kWPost] || w[kGate]) && !y) || (j.slots && !workspace))
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
    set_teams(a, rows, cols, kMaxThreads);
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
    const bool grid = on_grid(dh, ld) && aligned(dy, 16) && aligned(h_out, 16) && aligned(y, 16) &&
                      aligned(dz, 16) && aligned(dh_out, 16);
    const int bad = status_of(ZJ_PICK(launch_grad, bf16, grid, params->norm == ZERO_NORM_LAYER, a,
                                      ctas, st));
    if (bad) return bad;
  }
  if (j.slots == 0) return ZERO_OK;
  j.set_bounds(0, workspace, 1, static_cast<int64_t>(j.n_parts) * j.slots * j.pitch, 0, 4);
  const dim3 blocks(static_cast<unsigned>(ceil_div(cols, 32)), 2);
  return status_of(launch_pdl(bf16 ? join_parts_kernel<true> : join_parts_kernel<false>, blocks,
                              dim3(kJoinThreads), 0, st, j));
}

}  // extern "C"
