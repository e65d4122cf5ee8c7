/*
 * join.cu -- where a block's output joins the residual stream: norms after the
 * block and before the next, gate, dropout and residual scale (zero_block.h).
 *
 * A team of warps holds a row in registers, eight neighbouring columns per
 * thread (two times eight past 4096 columns), from the load to the last store:
 * forward 8 bytes per element, backward 12, and nothing is read twice. What a
 * norm needs of the whole row (a sum of squares; with ZERO_NORM_LAYER the mean
 * before it, from which the squares are then taken) goes through shuffles and,
 * past 256 columns, one exchange between the team's warps. A CTA has as many
 * teams as fit 512 threads, each with rows of its own and the next row's loads
 * under way while it works on one.
 *
 * The parameters' gradients are sums over the rows: each thread keeps those of
 * its own columns while its rows pass, a CTA joins its teams' in order and
 * leaves one partial vector per parameter in the workspace, and a second kernel
 * adds the (at most kMaxParts) vectors in order.
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
constexpr int kForwardCtas = 2; // of the forward pass per SM
static_assert(ZERO_MAX_JOIN_COLS == 2 * kMaxThreads * kVec, "two vectors per thread");

enum { kH, kY, kHOut, kZ, kStats, kDz, kDhOut, kDh, kDy, kParts, kBuffers };  // of a call
enum { kWPost, kBPost, kGate, kWPre, kBPre, kParams };

struct Args : Checked<kBuffers> {
  const uint16_t *h, *y, *h_out, *dz, *dh_out;
  uint16_t *h_new, *z, *dh, *dy;
  float4* stats;
  const uint16_t* param[kParams];
  float* parts;            // [CTA][slot][pitch]
  int32_t slot[kParams];   // of a parameter's gradient in parts, -1: none
  int32_t slots;
  int64_t rows, ld;
  int32_t cols, pitch;     // pitch: cols rounded up to whole vectors
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

__device__ __forceinline__ void team_sync(const Args& a, const Place& p) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + p.team), "r"(32 * a.team_warps) : "memory");
}

// Sums over the team, the same bits in all its threads. Two exchanges in turn,
// so that one barrier each is enough: a warp that writes to one again has
// passed the other's barrier, before which all have read this one's.
struct Exchange {
  float2 sums[2][kMaxWarps];
};

__device__ __forceinline__ float2 team_sum(const Args& a, const Place& p, Exchange& ex, int& turn,
                                           float x, float y) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    x += __shfl_xor_sync(0xffffffffu, x, d);
    y += __shfl_xor_sync(0xffffffffu, y, d);
  }
  if (a.team_warps == 1) return make_float2(x, y);
  float2* sums = ex.sums[turn] + p.team * a.team_warps;
  turn ^= 1;
  if (p.lane == 0) sums[p.warp] = make_float2(x, y);
  team_sync(a, p);
  float2 s = make_float2(0.f, 0.f);
  for (int w = 0; w < a.team_warps; ++w) {
    s.x += sums[w].x;
    s.y += sums[w].y;
  }
  return s;
}

__device__ __forceinline__ float inverse_root(float mean_square, float eps) {
  // squares past fp32's range: NaN, not 0
  return mean_square < __uint_as_float(0x7F800000u) ? rsqrtf(mean_square + eps)
                                                    : __uint_as_float(0x7FC00000u);
}

// Eight values as four pairs (packed fp32 arithmetic).
struct Eight {
  Pair p[4];
};

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

__device__ __forceinline__ Pair both(float x) { return pair(x, x); }

__device__ __forceinline__ float sum_of(const Pair& p) {
  float a, b;
  unpair(p, a, b);
  return a + b;
}

// Statistics of a row held by the team: (mean or 0, 1 / sqrt(mean square + eps)).
// `there`: how many of the thread's columns of each vector are columns.
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
    mean = team_sum(a, p, ex, turn, sum_of(s), 0.f).x * a.inv_cols;
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
        if (j < there[v]) edge += (f[j] - mean) * (f[j] - mean);
    }
  }
  const float square = team_sum(a, p, ex, turn, sum_of(s) + edge, 0.f).x * a.inv_cols;
  return make_float2(mean, inverse_root(square, a.eps));
}

// (x - mean) r
template <bool kLayer>
__device__ __forceinline__ Pair normed(const Pair& x, const float2& st) {
  return kLayer ? (x + both(-st.x)) * both(st.y) : x * both(st.y);
}

__device__ __forceinline__ uint4 load_param(const uint16_t* w, int c, int cols) {
  return w ? load8<false>(w, c, cols, Bounds{}) : make_uint4(0, 0, 0, 0);
}

constexpr int kStagePitch = (kStageWarp + 15) & ~15;

template <bool kBf16, bool kGrid, bool kLayer, int kV>
__global__ void __launch_bounds__(kMaxThreads, kV == 1 ? kForwardCtas : 1)
    join_kernel(const Args a) {
  pdl_begin();
  __shared__ Exchange exchange;
  __shared__ __align__(16) uint8_t stages[kGrid ? 16 : kMaxWarps * kStagePitch];
  const Place p(a);
  uint8_t* stage = stages + (kGrid ? 0 : (threadIdx.x >> 5) * kStagePitch);
  int turn = 0;
  uint4 w_post[kV], b_post[kV], gate[kV], w_pre[kV], b_pre[kV];
  int col[kV], there[kV];
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    col[v] = p.first(a, v) + p.lane * kVec;
    there[v] = max(0, min(kVec, a.cols - col[v]));
    w_post[v] = load_param(a.param[kWPost], col[v], a.cols);
    gate[v] = load_param(a.param[kGate], col[v], a.cols);
    w_pre[v] = load_param(a.param[kWPre], col[v], a.cols);
    if constexpr (kLayer) {
      b_post[v] = load_param(a.param[kBPost], col[v], a.cols);
      b_pre[v] = load_param(a.param[kBPre], col[v], a.cols);
    }
  }
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
    const bool post = a.param[kWPost] != nullptr;
    if (post) sy = row_stats<kBf16, kLayer, kV>(a, p, exchange, turn, y, there);
    uint4 out[kV];
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      Eight b = widen_pairs<kBf16>(y[v]);
      if (post) {
        const Eight w = widen_pairs<kBf16>(w_post[v]);
#pragma unroll
        for (int j = 0; j < 4; ++j) b.p[j] = normed<kLayer>(b.p[j], sy) * w.p[j];
        if constexpr (kLayer) {
          const Eight add = widen_pairs<kBf16>(b_post[v]);
#pragma unroll
          for (int j = 0; j < 4; ++j) b.p[j] = b.p[j] + add.p[j];
        }
      }
      if (a.drop.threshold)
        drop_pairs(a.drop,
                   draw8(a.drop, step, static_cast<uint32_t>(row),
                         static_cast<uint32_t>(col[v]) / kVec), b);
      const Pair s = both(a.branch_scale);
#pragma unroll
      for (int j = 0; j < 4; ++j) b.p[j] = b.p[j] * s;
      if (a.param[kGate]) {
        const Eight g = widen_pairs<kBf16>(gate[v]);
#pragma unroll
        for (int j = 0; j < 4; ++j) b.p[j] = b.p[j] * g.p[j];
      }
      const Eight x = widen_pairs<kBf16>(h[v]);
#pragma unroll
      for (int j = 0; j < 4; ++j) b.p[j] = fma2(x.p[j], both(a.stream_scale), b.p[j]);
      out[v] = narrow_pairs<kBf16>(b);
      store_row<kGrid>(stage, a.h_new + row * a.ld, p.first(a, v), p.lane, a.cols, out[v],
                       a.bounds(kHOut));
    }
    if (row + stride < a.rows) load(row + stride);
    if (a.param[kWPre]) {
      sh = row_stats<kBf16, kLayer, kV>(a, p, exchange, turn, out, there);
#pragma unroll
      for (int v = 0; v < kV; ++v) {
        Eight x = widen_pairs<kBf16>(out[v]);
        const Eight w = widen_pairs<kBf16>(w_pre[v]);
#pragma unroll
        for (int j = 0; j < 4; ++j) x.p[j] = normed<kLayer>(x.p[j], sh) * w.p[j];
        if constexpr (kLayer) {
          const Eight add = widen_pairs<kBf16>(b_pre[v]);
#pragma unroll
          for (int j = 0; j < 4; ++j) x.p[j] = x.p[j] + add.p[j];
        }
        store_row<kGrid>(stage, a.z + row * a.ld, p.first(a, v), p.lane, a.cols,
                         narrow_pairs<kBf16>(x), a.bounds(kZ));
      }
    }
    if (a.stats && p.warp == 0 && p.lane == 0 &&
        a.bounds(kStats).holds(a.stats + row, 16, kSiteStore))
      a.stats[row] = make_float4(sy.x, sy.y, sh.x, sh.y);
  }
}

// Sums over the rows of a thread's own columns: in registers, or, where a
// thread has two vectors, in shared memory (its own words, 16 bytes a lane).
template <int kV>
struct ColumnSums {
  Eight r[kParams];
  __device__ __forceinline__ void clear(float4*, int) {
#pragma unroll
    for (int k = 0; k < kParams; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) r[k].p[j] = both(0.f);
  }
  __device__ __forceinline__ void add(int k, int, const Eight& e) {
#pragma unroll
    for (int j = 0; j < 4; ++j) r[k].p[j] = r[k].p[j] + e.p[j];
  }
  // += x y
  __device__ __forceinline__ void add(int k, int, const Eight& x, const Eight& y) {
#pragma unroll
    for (int j = 0; j < 4; ++j) r[k].p[j] = fma2(x.p[j], y.p[j], r[k].p[j]);
  }
};

template <>
struct ColumnSums<2> {
  float4* own;
  __device__ __forceinline__ float4* at(int k, int v) const {
    return own + (k * 2 + v) * 2 * kMaxThreads;
  }
  __device__ __forceinline__ void clear(float4* smem, int thread) {
    own = smem + thread;
    for (int k = 0; k < 2 * kParams; ++k) {
      own[2 * k * kMaxThreads] = make_float4(0.f, 0.f, 0.f, 0.f);
      own[(2 * k + 1) * kMaxThreads] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  __device__ __forceinline__ void add(int k, int v, const Eight& e) {
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) unpair(e.p[j], f[2 * j], f[2 * j + 1]);
    float4 *lo = at(k, v), *hi = lo + kMaxThreads;
    float4 x = *lo, y = *hi;
    x.x += f[0], x.y += f[1], x.z += f[2], x.w += f[3];
    y.x += f[4], y.y += f[5], y.z += f[6], y.w += f[7];
    *lo = x, *hi = y;
  }
  __device__ __forceinline__ void add(int k, int v, const Eight& x, const Eight& y) {
    Eight e;
#pragma unroll
    for (int j = 0; j < 4; ++j) e.p[j] = x.p[j] * y.p[j];
    add(k, v, e);
  }
};

// shared memory of the backward kernel's column sums
template <int kV>
constexpr int sums_bytes() { return kParams * kV * kMaxThreads * kVec * 4; }

template <bool kBf16, bool kGrid, bool kLayer, int kV>
__global__ void __launch_bounds__(kMaxThreads, 1) join_grad_kernel(const Args a) {
  pdl_begin();
  extern __shared__ float4 smem_sums[];
  __shared__ Exchange exchange;
  __shared__ __align__(16) uint8_t stages[kGrid ? 16 : kMaxWarps * kStagePitch];
  const Place p(a);
  uint8_t* stage = stages + (kGrid ? 0 : (threadIdx.x >> 5) * kStagePitch);
  int turn = 0;
  ColumnSums<kV> sums;
  sums.clear(smem_sums, threadIdx.x);
  uint4 w_post[kV], b_post[kV], gate[kV], w_pre[kV];
  int col[kV];
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    col[v] = p.first(a, v) + p.lane * kVec;
    w_post[v] = load_param(a.param[kWPost], col[v], a.cols);
    gate[v] = load_param(a.param[kGate], col[v], a.cols);
    w_pre[v] = load_param(a.param[kWPre], col[v], a.cols);
    if constexpr (kLayer) b_post[v] = load_param(a.param[kBPost], col[v], a.cols);
  }
  const uint32_t step = step_of(a.drop);
  const bool post = a.param[kWPost] != nullptr, gated = a.param[kGate] != nullptr;
  const bool pre = a.param[kWPre] != nullptr;
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
      y[v] = post || gated ? load8<kGrid>(a.y + r * a.ld, col[v], a.cols, a.bounds(kY)) : none;
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
#pragma unroll
      for (int v = 0; v < kV; ++v) {
        const Eight g0 = widen_pairs<kBf16>(dz[v]), w = widen_pairs<kBf16>(w_pre[v]);
        Eight x = widen_pairs<kBf16>(h[v]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x.p[j] = normed<kLayer>(x.p[j], sh);
          const Pair g = g0.p[j] * w.p[j];
          along = fma2(g, x.p[j], along);
          if constexpr (kLayer) flat = flat + g;
        }
        sums.add(kWPre, v, g0, x);
        if constexpr (kLayer) sums.add(kBPre, v, g0);
      }
      const float2 s = team_sum(a, p, exchange, turn, sum_of(along), kLayer ? sum_of(flat) : 0.f);
      const Pair c1 = both(-s.x * a.inv_cols), c2 = both(-s.y * a.inv_cols), r = both(sh.y);
#pragma unroll
      for (int v = 0; v < kV; ++v) {
        const Eight g0 = widen_pairs<kBf16>(dz[v]), w = widen_pairs<kBf16>(w_pre[v]);
        const Eight x = widen_pairs<kBf16>(h[v]), up = widen_pairs<kBf16>(dh[v]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          Pair g = fma2(normed<kLayer>(x.p[j], sh), c1, g0.p[j] * w.p[j]);
          if constexpr (kLayer) g = g + c2;
          d[v].p[j] = fma2(g, r, up.p[j]);
        }
      }
    } else {
#pragma unroll
      for (int v = 0; v < kV; ++v) d[v] = widen_pairs<kBf16>(dh[v]);
    }
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      Eight e;
#pragma unroll
      for (int j = 0; j < 4; ++j) e.p[j] = d[v].p[j] * both(a.stream_scale);
      store_row<kGrid>(stage, a.dh + row * a.ld, p.first(a, v), p.lane, a.cols,
                       narrow_pairs<kBf16>(e), a.bounds(kDh));
    }
    // through gate, dropout and the norm after the block
    Pair along = both(0.f), flat = both(0.f);
    uint4 yy[kV];
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      yy[v] = y[v];
      uint4 draw = none;
      if (a.drop.threshold)
        draw = draw8(a.drop, step, static_cast<uint32_t>(row),
                     static_cast<uint32_t>(col[v]) / kVec);
#pragma unroll
      for (int j = 0; j < 4; ++j) d[v].p[j] = d[v].p[j] * both(a.branch_scale);
      if (a.drop.threshold) drop_pairs(a.drop, draw, d[v]);
      if (post || gated) {
        Eight x = widen_pairs<kBf16>(yy[v]);
        const Eight w = widen_pairs<kBf16>(w_post[v]);
        if (post) {
#pragma unroll
          for (int j = 0; j < 4; ++j) x.p[j] = normed<kLayer>(x.p[j], sy);
        }
        if (gated) {
          Eight n = x;
          if (post) {
#pragma unroll
            for (int j = 0; j < 4; ++j) n.p[j] = x.p[j] * w.p[j];
            if constexpr (kLayer) {
              const Eight b = widen_pairs<kBf16>(b_post[v]);
#pragma unroll
              for (int j = 0; j < 4; ++j) n.p[j] = n.p[j] + b.p[j];
            }
          }
          sums.add(kGate, v, d[v], n);
          const Eight g = widen_pairs<kBf16>(gate[v]);
#pragma unroll
          for (int j = 0; j < 4; ++j) d[v].p[j] = d[v].p[j] * g.p[j];
        }
        if (post) {
          sums.add(kWPost, v, d[v], x);
          if constexpr (kLayer) sums.add(kBPost, v, d[v]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            d[v].p[j] = d[v].p[j] * w.p[j];
            along = fma2(d[v].p[j], x.p[j], along);
            if constexpr (kLayer) flat = flat + d[v].p[j];
          }
        }
      }
    }
    if (row + stride < a.rows) load(row + stride);
    if (post) {
      const float2 s = team_sum(a, p, exchange, turn, sum_of(along), kLayer ? sum_of(flat) : 0.f);
      const Pair c1 = both(-s.x * a.inv_cols), c2 = both(-s.y * a.inv_cols), r = both(sy.y);
#pragma unroll
      for (int v = 0; v < kV; ++v) {
        const Eight x = widen_pairs<kBf16>(yy[v]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          Pair g = fma2(normed<kLayer>(x.p[j], sy), c1, d[v].p[j]);
          if constexpr (kLayer) g = g + c2;
          d[v].p[j] = g * r;
        }
      }
    }
#pragma unroll
    for (int v = 0; v < kV; ++v)
      store_row<kGrid>(stage, a.dy + row * a.ld, p.first(a, v), p.lane, a.cols,
                       narrow_pairs<kBf16>(d[v]), a.bounds(kDy));
  }
  // this CTA's vectors: the teams' sums joined in order
  if (a.slots == 0) return;
  const int team_threads = 32 * a.team_warps, t = p.warp * 32 + p.lane;
  float* part = a.parts + static_cast<int64_t>(blockIdx.x) * a.slots * a.pitch;
  const auto leave = [&](int slot, int c, const float4& lo, const float4& hi) {
    float* to = part + static_cast<int64_t>(slot) * a.pitch + c;
    if (c >= a.pitch || !a.bounds(kParts).holds(to, 32, kSiteStore)) return;
    reinterpret_cast<float4*>(to)[0] = lo;
    reinterpret_cast<float4*>(to)[1] = hi;
  };
  if constexpr (kV == 1) {
    for (int k = 0; k < a.teams; ++k) {
      if (p.team == k) {
#pragma unroll
        for (int w = 0; w < kParams; ++w) {
          float f[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) unpair(sums.r[w].p[j], f[2 * j], f[2 * j + 1]);
          float4 *lo = smem_sums + (2 * w) * team_threads + t, *hi = lo + team_threads;
          const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
          const float4 x = k ? *lo : z, y4 = k ? *hi : z;
          *lo = make_float4(x.x + f[0], x.y + f[1], x.z + f[2], x.w + f[3]);
          *hi = make_float4(y4.x + f[4], y4.y + f[5], y4.z + f[6], y4.w + f[7]);
        }
      }
      __syncthreads();
    }
    for (int w = p.team; w < kParams; w += a.teams)
      if (a.slot[w] >= 0)
        leave(a.slot[w], col[0], smem_sums[2 * w * team_threads + t],
              smem_sums[(2 * w + 1) * team_threads + t]);
  } else {
    for (int w = 0; w < kParams; ++w)
      if (a.slot[w] >= 0)
        for (int v = 0; v < kV; ++v) leave(a.slot[w], col[v], *sums.at(w, v), sums.at(w, v)[kMaxThreads]);
  }
}

// The vectors of all CTAs, in order: 128 columns of one parameter per CTA, its
// eight warps an eighth of the vectors each.
struct JoinArgs : Checked<1> {
  const float* parts;
  uint16_t* grad[kParams];  // by slot
  int32_t n_parts, slots, cols, pitch;
};

constexpr int kJoinWarps = 8;

template <bool kBf16>
__global__ void __launch_bounds__(32 * kJoinWarps) join_parts_kernel(const JoinArgs a) {
  pdl_begin();
  __shared__ float4 sums[kJoinWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, slot = blockIdx.y;
  const int c = (blockIdx.x * 32 + lane) * 4;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < a.pitch) {
    const int64_t step = static_cast<int64_t>(a.slots) * a.pitch;
    const float* from = a.parts + static_cast<int64_t>(slot) * a.pitch + c;
    const int lo = a.n_parts * warp / kJoinWarps, hi = a.n_parts * (warp + 1) / kJoinWarps;
#pragma unroll 8
    for (int k = lo; k < hi; ++k) {
      if (!a.bounds(0).holds(from + k * step, 16, kSiteLoad)) continue;
      const float4 x = *reinterpret_cast<const float4*>(from + k * step);
      s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
    }
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp) return;
  for (int w = 1; w < kJoinWarps; ++w) {
    const float4 x = sums[w][lane];
    s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
  }
  uint16_t* grad = a.grad[slot];
  const float f[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (c + j < a.cols) grad[c + j] = narrow<kBf16>(f[j]);
}

// -------------------------------------------------------------------- host ----

int64_t pitch_of(int64_t cols) { return ceil_div(cols, kVec) * kVec; }

// teams of a CTA: rows are spread over `ctas` first
void set_teams(Args& a, int64_t rows, int64_t cols, int64_t ctas) {
  const int64_t vectors = ceil_div(cols, kVec), per = vectors > kMaxThreads ? 2 : 1;
  a.team_warps = static_cast<int32_t>(ceil_div(ceil_div(vectors, per), 32));
  const int64_t most = kMaxWarps / a.team_warps;
  a.teams = static_cast<int32_t>(std::min(most, std::max<int64_t>(1, ceil_div(rows, ctas))));
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

template <bool kBf16, bool kGrid, bool kLayer>
cudaError_t launch_join(const Args& a, int64_t ctas, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(ctas)), block(32 * a.team_warps * a.teams);
  return a.pitch > kMaxThreads * kVec
             ? launch_pdl(join_kernel<kBf16, kGrid, kLayer, 2>, grid, block, 0, st, a)
             : launch_pdl(join_kernel<kBf16, kGrid, kLayer, 1>, grid, block, 0, st, a);
}

template <bool kBf16, bool kGrid, bool kLayer, int kV>
cudaError_t launch_grad_of(const Args& a, int64_t ctas, cudaStream_t st) {
  const auto fn = join_grad_kernel<kBf16, kGrid, kLayer, kV>;
  const int bytes = kV == 1 ? kParams * 32 * a.team_warps * kVec * 4 : sums_bytes<kV>();
  const cudaError_t e =
      cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, sums_bytes<kV>());
  if (e != cudaSuccess) return e;
  return launch_pdl(fn, dim3(static_cast<unsigned>(ctas)), dim3(32 * a.team_warps * a.teams),
                    bytes, st, a);
}

template <bool kBf16, bool kGrid, bool kLayer>
cudaError_t launch_grad(const Args& a, int64_t ctas, cudaStream_t st) {
  return a.pitch > kMaxThreads * kVec ? launch_grad_of<kBf16, kGrid, kLayer, 2>(a, ctas, st)
                                      : launch_grad_of<kBf16, kGrid, kLayer, 1>(a, ctas, st);
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
  const int64_t most = kForwardCtas * kMaxParts;
  set_teams(a, rows, cols, most);
  const int64_t ctas = std::min(most, ceil_div(rows, a.teams));
  const bool grid = on_grid(h, ld) && aligned(y, 16) && aligned(h_out, 16) && aligned(z, 16);
  return status_of(ZJ_PICK(launch_join, dtype == ZERO_BF16, grid, params->norm == ZERO_NORM_LAYER,
                           a, ctas, static_cast<cudaStream_t>(stream)));
}

ZERO_API size_t zero_block_join_workspace_bytes(int64_t rows, int64_t cols) {
  using namespace zj;
  if (rows < 0 || cols < 0 || rows >= int64_t{1} << 31 || cols > ZERO_MAX_JOIN_COLS) return 0;
  return static_cast<size_t>(std::min<int64_t>(rows, kMaxParts) * kParams * pitch_of(cols) * 4);
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
  for (int k = 0; k < kParams; ++k) {
    a.slot[k] = g[k] ? j.slots : -1;
    if (g[k]) j.grad[j.slots++] = static_cast<uint16_t*>(g[k]);
  }
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
    set_teams(a, rows, cols, kMaxParts);
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
  const dim3 blocks(static_cast<unsigned>(ceil_div(j.pitch, 128)), j.slots);
  return status_of(launch_pdl(bf16 ? join_parts_kernel<true> : join_parts_kernel<false>, blocks,
                              dim3(32 * kJoinWarps), 0, st, j));
}

}  // extern "C"
