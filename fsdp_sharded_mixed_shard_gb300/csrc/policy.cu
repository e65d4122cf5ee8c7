/*
 * policy.cu -- token log-probabilities and the clipped policy loss with its
 * gradient (zero_train.h).
 *
 * A row's softmax needs its maximum and sum before its gradient can be
 * written, so the row is read once into the shared memory of a cluster of 1
 * to 8 CTAs and the gradient is formed from there: rows * vocab elements read
 * and as many written, nothing in between. Each lane keeps a running maximum
 * m and sum s of exp(x - m) over its vectors (a new maximum rescales s), the
 * CTA joins its lanes' pairs, and every CTA sends its pair to all others of
 * the cluster over distributed shared memory; all join them in rank order, so
 * all hold the same bits.
 *
 * The row is cut into parts, kParts per warp and the same number of blocks
 * (+-1) each. A part belongs to one warp from its bulk copy to its gradient:
 * the warp waits for the copy, sums, later forms the gradient from the same
 * bytes, and at once starts the copy of the next row's part into their place,
 * so the next row arrives while this one's gradient leaves, and no barrier of
 * the CTA stands between them.
 *
 * A row of an odd vocabulary starts anywhere. It is numbered in the 16-byte
 * blocks of its addresses; the first and last may hold elements of other
 * rows, which are read as -inf and not written.
 *
 * Bound by memory once the exponentials (two per element) are cheap: packed
 * fp32 arithmetic, four blocks per lane and step, and the row's scalars by one
 * warp. Measured: 4096 x 128256 bf16, a quarter of the rows left out, 297 us
 * (91 % of copy bandwidth; ncu on 1024 rows: 400 MB moved for 394), 2048 x 50257
 * 73 us (73 %: 6 or 7 rows per cluster), 16 x 50257 8.2 us. Log-probabilities
 * alone stream the row through registers: 2048 x 128256 fp32 150 us (7.0 TB/s
 * read; the copy that is measured against also writes).
 *
 * Every wait is bounded (2 s). One that expires ends the work of its CTA and,
 * as the others' waits for it expire, of its cluster: the rows left are NaN, and
 * no CTA ends before what is on its way to it has landed.
 */
#include "train.cuh"

#include <algorithm>
#include <cmath>
#include <map>
#include <mutex>
#include <tuple>

namespace zp {

using namespace zt;

constexpr int kMaxWarps = 8;   // per CTA; 1, 2, 4 or 8 by the row's length
constexpr int kMaxCluster = 8;
constexpr int kParts = 2;      // parts of a row per warp
constexpr int kBatch = 4;      // blocks per lane and step
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

enum { kLogits, kDlogits, kBuffers };  // of a call, for their bounds

struct Args : Checked<kBuffers> {
  const uint8_t* logits;
  uint8_t* dlogits;
  const void* actions;
  const float *old_logp, *ref_logp, *advantage, *weight;
  const zero_scaler* scaler;
  float *logp, *loss, *stats;
  int64_t rows, vocab, ld;
  int32_t action_bytes;
  float lo, hi, beta;
};

// exp(x - m) is formed as 2^(x c - m c) with c = log2 e: one fused
// multiply-add per element, and what m c loses in rounding is the same for
// every element and cancels. It is a factor of at most 2^64 (half an ulp of
// m c) below |m| = kFar, and would pass fp32's range soon after. From there on
// every other logit is at least 64 away from m, so that 2^(x - m) and
// exp(x - m) alike are nothing beside the 1 of m itself: c = 1, whose products
// are exact.
constexpr float kFar = 0x1p30f;

struct Base {
  float c, mc;
};

__device__ __forceinline__ Base base_of(float m) {
  const float at = m == -INFINITY ? 0.f : m;  // nothing but -inf so far
  const float c = fabsf(at) < kFar ? kLog2e : 1.f;
  return Base{c, at * c};
}

// softmax statistics: largest value and sum of exp(x - m); (-inf, 0) for none
struct Stat {
  float m, s;
};

// a's sum over another, not smaller, maximum. Maxima on two sides of kFar are
// so far apart that nothing of the smaller one's sum is left.
__device__ __forceinline__ float moved(const Stat& a, float m) {
  const Base from = base_of(a.m), to = base_of(m);
  // a side with nothing adds nothing; NaN goes on into the sum
  return a.s == 0.f ? 0.f : a.s * (from.c == to.c ? exp2_fast(from.mc - to.mc) : 0.f);
}

// the pairs of a warp's lanes; all lanes hold the same bits afterwards
__device__ __forceinline__ Stat join_lanes(Stat t) {
  float m = t.m;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  float s = moved(t, m);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  return Stat{m, s};
}

// A 16-byte block of logits.
template <int kType>
struct Block {
  static constexpr bool kBf16 = kType == ZERO_BF16;
  static constexpr int kElems = 8;
  static constexpr int kBytes = 2;
  static constexpr uint32_t kNone = kBf16 ? 0xFF80FF80u : 0xFC00FC00u;  // -inf, -inf
  __device__ static __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (kBf16) asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  // two running maxima; top() joins them
  __device__ static __forceinline__ uint32_t max_of(const uint4& v, uint32_t so_far) {
    return max2(so_far, max2(max2(v.x, v.y), max2(v.z, v.w)));
  }
  __device__ static __forceinline__ float top(uint32_t w) {
    float a, b;
    widen2<kBf16>(w, a, b);
    return fmaxf(a, b);
  }
  __device__ static __forceinline__ void get(const uint4& v, Pair (&f)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float x, y;
      widen2<kBf16>(w[j], x, y);
      f[j] = pair(x, y);
    }
  }
  __device__ static __forceinline__ uint4 put(const float (&f)[8]) { return narrow8<kBf16>(f); }
  __device__ static __forceinline__ float one(const uint8_t* p) {
    return widen<kBf16>(*reinterpret_cast<const uint16_t*>(p));
  }
  __device__ static __forceinline__ void set(uint8_t* p, float x) {
    *reinterpret_cast<uint16_t*>(p) = narrow<kBf16>(x);
  }
};

template <>
struct Block<ZERO_FP32> {
  static constexpr int kElems = 4;
  static constexpr int kBytes = 4;
  static constexpr uint32_t kNone = 0xFF800000u;
  __device__ static __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }
  __device__ static __forceinline__ uint32_t max_of(const uint4& v, uint32_t so_far) {
    return max2(so_far, max2(max2(v.x, v.y), max2(v.z, v.w)));
  }
  __device__ static __forceinline__ float top(uint32_t w) { return __uint_as_float(w); }
  __device__ static __forceinline__ void get(const uint4& v, Pair (&f)[2]) {
    f[0] = pair(__uint_as_float(v.x), __uint_as_float(v.y));
    f[1] = pair(__uint_as_float(v.z), __uint_as_float(v.w));
  }
  __device__ static __forceinline__ uint4 put(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
  __device__ static __forceinline__ float one(const uint8_t* p) {
    return *reinterpret_cast<const float*>(p);
  }
  __device__ static __forceinline__ void set(uint8_t* p, float x) {
    *reinterpret_cast<float*>(p) = x;
  }
};

template <int kType>
__device__ __forceinline__ uint4 no_block() {
  constexpr uint32_t w = Block<kType>::kNone;
  return make_uint4(w, w, w, w);
}

// exp(x - m) of a block's elements
template <int kType>
__device__ __forceinline__ void exp_block(const uint4& v, const Pair& c, const Pair& minus_mc,
                                          Pair (&e)[Block<kType>::kElems / 2]) {
  Block<kType>::get(v, e);
#pragma unroll
  for (int j = 0; j < Block<kType>::kElems / 2; ++j) {
    float x, y;
    unpair(fma2(e[j], c, minus_mc), x, y);
    e[j] = pair(exp2_fast(x), exp2_fast(y));
  }
}

// kBatch blocks into a lane's statistics: one rescaling for all of them
template <int kType>
__device__ __forceinline__ void add_blocks(Stat& t, const uint4 (&v)[kBatch]) {
  using B = Block<kType>;
  uint32_t w = B::max_of(v[0], B::kNone);
#pragma unroll
  for (int k = 1; k < kBatch; ++k) w = B::max_of(v[k], w);
  const float top = B::top(w);
  if (top > t.m) {
    t.s = moved(t, top);
    t.m = top;
  }
  const Base b = base_of(t.m);
  const Pair c = pair(b.c, b.c), minus_mc = pair(-b.mc, -b.mc);
  Pair sum[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
#pragma unroll
  for (int k = 0; k < kBatch; ++k) {
    Pair e[B::kElems / 2];
    exp_block<kType>(v[k], c, minus_mc, e);
#pragma unroll
    for (int j = 0; j < B::kElems / 2; ++j) sum[j & 1] = sum[j & 1] + e[j];
  }
  float x, y;
  unpair(sum[0] + sum[1], x, y);
  t.s += x + y;
}

// log(exp(x - m) / s). The products x c and m c leave fp32 where x is a type's
// lowest value (a masked token taken); the difference itself is the result there.
__device__ __forceinline__ float log_share(float x, const Stat& t) {
  const Base b = base_of(t.m);
  const bool plain = b.c == 1.f || !(fabsf(x) < 0x1p126f);
  return (plain ? x - t.m : __fmaf_rn(x, b.c, -b.mc) * kLn2) - logf(t.s);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::
          : "memory");
}

// every thread of the cluster is here; nothing is said about memory
__device__ __forceinline__ void cluster_meet() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n barrier.cluster.wait.aligned;" ::
                   : "memory");
}

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// Bulk copy of whole 16-byte blocks (possibly none) that completes one phase
// of `bar`.
__device__ __forceinline__ void copy_blocks(void* dst, const uint8_t* src, uint32_t bytes,
                                            uint64_t* bar) {
  asm volatile(
      "{\n .reg .b64 st;\n mbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n}" ::"r"(
          smem_u32(bar)),
      "r"(bytes)
      : "memory");
  if (bytes)
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
            "r"(smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}

// Acquires at cluster scope: what it waits for may be another CTA's sums. The
// first tries come one after another, as a copy or the sums are mostly there.
__device__ __forceinline__ bool bar_try(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ bool is_set(const int* flag) {
  return *static_cast<const volatile int*>(flag) != 0;
}

// true when the phase has completed; false once *lost is set or the limit has
// passed, which sets it. A CTA that has lost a wait neither copies nor sends any
// more, as its barriers may be a turn off, and its rows are NaN from then on; the
// waits of the cluster's other CTAs for it expire in their turn.
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, uint64_t limit,
                                         int* lost) {
  for (int k = 0; k < 64; ++k)
    if (bar_try(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  for (;;) {
    if (bar_try(bar, parity)) return true;
    if (is_set(lost)) return false;
    if (global_ns() - t0 > limit) {
      *static_cast<volatile int*>(lost) = 1;
      return false;
    }
  }
}

// A row as 16-byte blocks.
struct Row {
  const uint8_t* base;  // block 0; the row starts `head` bytes into it
  int32_t head, n_blk;
  int32_t end;          // head + the row's bytes
  int32_t action;       // -1: left out
  float weight;
  __device__ __forceinline__ bool on() const { return action >= 0 && weight != 0.f; }
};

template <int kBytes, bool kGrad>
__device__ __forceinline__ Row row_of(const Args& a, int64_t row) {
  Row r;
  const uint8_t* x = a.logits + row * a.ld * kBytes;
  r.head = static_cast<int32_t>(reinterpret_cast<uintptr_t>(x) & 15);
  r.base = x - r.head;
  r.end = r.head + static_cast<int32_t>(a.vocab) * kBytes;
  r.n_blk = (r.end + 15) >> 4;
  r.action = static_cast<int32_t>(load_id(a.actions, a.action_bytes, row, a.vocab));
  r.weight = kGrad ? a.weight[row] : 1.f;
  return r;
}

// Block b of the row with -inf in place of what it holds of other rows (the
// first and the last block may).
template <int kType>
__device__ __forceinline__ uint4 own_part(const Row& r, int32_t b, const uint4& v) {
  using B = Block<kType>;
  if (b != 0 && b != r.n_blk - 1) return v;
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
  const int lo = b == 0 ? r.head : 0;
  const int hi = b == r.n_blk - 1 ? r.end - b * 16 : 16;
#pragma unroll
  for (int j = 0; j < B::kElems; ++j) {
    const int at = j * B::kBytes;
    if (at >= lo && at < hi) continue;
    const uint32_t keep = B::kBytes == 4 ? 0u : (at & 2) ? 0x0000FFFFu : 0xFFFF0000u;
    w[at >> 2] = (w[at >> 2] & keep) | (B::kNone & ~keep);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The pairs of a CTA's warps, of the cluster's CTAs, and the barrier that
// counts the latter's arrival. Two of them in turn: a CTA sends for the row
// after next only once every CTA has sent for the next row, hence read this
// one.
struct Exchange {
  Stat of_warp[kMaxWarps];
  Stat of_cta[kMaxCluster];
  uint64_t arrived;
};

__device__ __forceinline__ void bar_init(uint64_t* bar) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_u32(bar)) : "memory");
}

// Store v into *to of CTA `rank`, counted by that CTA's barrier. (A cluster
// barrier would also wait for this CTA's stores to dlogits, of no interest
// here: 1 us and more per row.)
__device__ __forceinline__ void send(Stat* to, uint64_t* bar, uint32_t rank, const Stat& v) {
  uint32_t remote, remote_bar;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(remote)
               : "r"(smem_u32(to)), "r"(rank));
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(remote_bar)
               : "r"(smem_u32(bar)), "r"(rank));
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::"r"(
          remote),
      "r"(__float_as_uint(v.m)), "r"(__float_as_uint(v.s)), "r"(remote_bar)
      : "memory");
}

// The statistics of a row from its warps' pairs, by warp 0 of every CTA of
// the cluster; its lanes hold the same bits afterwards. `use` counts the calls.
template <int kWarps>
__device__ __forceinline__ Stat join_all(Exchange (&x)[2], uint32_t rank, uint32_t n_cta,
                                         uint32_t use, const Args& a, int64_t row, int* lost) {
  const uint32_t lane = threadIdx.x & 31;
  Exchange& e = x[use & 1];
  const Stat none = {-INFINITY, 0.f}, nan = {0.f, __uint_as_float(0x7FC00000u)};
  const bool gone = is_set(lost);  // by a warp before the CTA's barrier, or this one earlier
  const Stat t = join_lanes(gone ? nan : lane < kWarps ? e.of_warp[lane] : none);
  if (n_cta == 1 || gone) return t;
  if (lane < n_cta) {
    if (lane == 0)
      asm volatile(
          "{\n .reg .b64 st;\n mbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n}" ::"r"(
              smem_u32(&e.arrived)),
          "r"(n_cta * static_cast<uint32_t>(sizeof(Stat)))
          : "memory");
    if (!(rank == 1 && a.holds(ZERO_PLANT_NO_SEND, row)))
      send(&e.of_cta[rank], &e.arrived, lane, t);
  }
  const bool ok = bar_wait(&e.arrived, (use >> 1) & 1, a.limit(), lost);
  return join_lanes(!ok ? nan : lane < n_cta ? e.of_cta[lane] : none);
}

// The end of a CTA: no other sends to it any more, and where a wait expired,
// what is still on its way (microseconds) lands.
__device__ __forceinline__ void leave(uint32_t n_cta, int* lost) {
  if (n_cta > 1) cluster_meet();
  if (is_set(lost)) drain();
}

// The row's logits as a single stream: statistics only.
template <int kType, int kWarps>
__global__ void __launch_bounds__(32 * kWarps) logp_kernel(const Args a) {
  pdl_begin();
  constexpr int kThreads = 32 * kWarps;
  using B = Block<kType>;
  __shared__ Exchange exchange[2];
  const int tid = threadIdx.x;
  const uint32_t rank = cluster_rank(), n_cta = cluster_size();
  __shared__ int lost;
  uint32_t use = 0;
  if (tid == 0) {
    lost = 0;
    bar_init(&exchange[0].arrived);
    bar_init(&exchange[1].arrived);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();
  if (n_cta > 1) cluster_sync();  // every CTA of the cluster is ready before any sends to it
  else __syncthreads();
  for (int64_t row = blockIdx.x / n_cta; row < a.rows; row += gridDim.x / n_cta) {
    const Row r = row_of<B::kBytes, false>(a, row);
    float lp = 0.f;
    if (r.on()) {
      const uint8_t* at_action = r.base + r.head + r.action * B::kBytes;
      const float picked =
          a.bounds(kLogits).holds(at_action, B::kBytes, kSiteLoad) ? B::one(at_action) : 0.f;
      const int32_t b0 = static_cast<int64_t>(r.n_blk) * rank / n_cta;
      const int32_t b1 = static_cast<int64_t>(r.n_blk) * (rank + 1) / n_cta;
      const uint4* blocks = reinterpret_cast<const uint4*>(r.base);
      Stat t = {-INFINITY, 0.f};
      for (int32_t b = b0 + tid; b < b1; b += kThreads * kBatch) {
        uint4 v[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const int32_t at = b + k * kThreads;
          v[k] = at < b1 && a.bounds(kLogits).holds_blocks(blocks + at, 16, kSiteLoad)
                     ? __ldcs(blocks + at)
                     : no_block<kType>();
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) v[k] = own_part<kType>(r, b + k * kThreads, v[k]);
        add_blocks<kType>(t, v);
      }
      t = join_lanes(t);
      if ((tid & 31) == 0) exchange[use & 1].of_warp[tid >> 5] = t;
      __syncthreads();
      if (tid < 32)
        lp = log_share(picked,
                       join_all<kWarps>(exchange, rank, n_cta, use, a, row, &lost));
      ++use;
    }
    if (rank == 0 && tid == 0) a.logp[row] = lp;
  }
  leave(n_cta, &lost);
}

// What warp 0 tells the others between a row's sums and its gradient.
struct Turn {
  Row next;
  Base base;
  float slope, inv;  // dloss/dlogp with its factors, and -slope / sum
};

template <int kType, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, 24 / kWarps)
    policy_kernel(const Args a, const int32_t part_cap) {
  pdl_begin();
  using B = Block<kType>;
  extern __shared__ __align__(16) uint8_t stage[];
  __shared__ Exchange exchange[2];
  __shared__ uint64_t landed[kWarps][kParts];
  __shared__ Turn turn;
  __shared__ float taken;
  __shared__ int lost;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank(), n_cta = cluster_size();
  const int64_t n_clusters = gridDim.x / n_cta;
  const float scale = a.scaler ? a.scaler->scale : 1.f;
  const bool kl = a.ref_logp && a.beta != 0.f;
  // the row is cut into n_cta kWarps kParts = 2^cut parts of equal size (+-1 block)
  const int cut = __ffs(n_cta * kWarps * kParts) - 1;
  const int32_t part0 = (rank * kWarps + warp) * kParts;
  uint8_t* mine = stage + static_cast<int64_t>(warp) * kParts * part_cap * 16;
  if (lane == 0) {
    for (int p = 0; p < kParts; ++p) bar_init(&landed[warp][p]);
    if (warp == 0) {
      lost = 0;
      bar_init(&exchange[0].arrived);
      bar_init(&exchange[1].arrived);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();
  if (n_cta > 1) cluster_sync();  // every CTA of the cluster is ready before any sends to it
  else __syncthreads();
  const auto block_of = [&](const Row& r, int p) {
    return (r.n_blk * (part0 + p)) >> cut;
  };
  const auto part_at = [&](int p) {
    return reinterpret_cast<uint4*>(mine + static_cast<int64_t>(p) * part_cap * 16);
  };
  const auto fetch = [&](const Row& r, int64_t row, int p) {  // one lane
    if (part0 + p == 0 && a.holds(ZERO_PLANT_NO_COPY, row)) return;
    const int32_t b0 = block_of(r, p), n = block_of(r, p + 1) - b0;
    const uint8_t* from = r.base + static_cast<int64_t>(b0) * 16;
    const bool in = ZCHECK(n <= part_cap, kSiteStageBytes, n) &&
                    a.bounds(kLogits).holds_blocks(from, n * 16, kSiteLoad);
    copy_blocks(part_at(p), from, in ? n * 16 : 0, &landed[warp][p]);
  };
  uint32_t use = 0, phase = 0;
  int64_t row = blockIdx.x / n_cta;
  Row r = {};
  if (row < a.rows) r = row_of<B::kBytes, true>(a, row);
  bool fetched = false;  // this row's parts are on their way
  while (row < a.rows) {
    const int64_t next_row = row + n_clusters;
    const bool on = r.on();
    // what warp 0 needs after the sums, asked for before them
    float picked = 0.f, old = 0.f, adv = 0.f, ref = 0.f;
    Row next = {};
    next.action = -1;
    if (warp == 0) {
      if (on) {
        const uint8_t* at = r.base + r.head + r.action * B::kBytes;
        if (a.bounds(kLogits).holds(at, B::kBytes, kSiteLoad)) picked = B::one(at);
        old = a.old_logp[row];
        adv = a.advantage[row];
        if (kl) ref = a.ref_logp[row];
      }
      if (next_row < a.rows) next = row_of<B::kBytes, true>(a, next_row);
    }
    if (on) {
      if (!fetched && lane == 0 && !is_set(&lost)) {
#pragma unroll
        for (int p = 0; p < kParts; ++p) fetch(r, row, p);
      }
      Stat t = {-INFINITY, 0.f};
#pragma unroll 1
      for (int p = 0; p < kParts; ++p) {
        const int32_t b0 = block_of(r, p), n = block_of(r, p + 1) - b0;
        const uint4* part = part_at(p);
        bar_wait(&landed[warp][p], phase, a.limit(), &lost);  // expired: join_all sees `lost`
        const bool edge = b0 == 0 || b0 + n == r.n_blk;
        for (int32_t k0 = 0; k0 < n; k0 += 32 * kBatch) {
          uint4 v[kBatch];
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            const int32_t k = k0 + 32 * j + lane;
            v[j] = k < n ? part[k] : no_block<kType>();
            if (edge) v[j] = own_part<kType>(r, b0 + k, v[j]);
          }
          add_blocks<kType>(t, v);
        }
      }
      phase ^= 1;
      t = join_lanes(t);
      if (lane == 0) exchange[use & 1].of_warp[warp] = t;
    }
    // stored, so read: once this CTA has sent its sums, another may write the
    // gradient over this logit (dlogits in the logits' place)
    if (tid == 0) taken = picked;
    __syncthreads();
    if (warp == 0) {
      Turn n = {};
      n.next = next;
      float lp = 0.f, loss = 0.f;
      if (on) {
        const Stat t = join_all<kWarps>(exchange, rank, n_cta, use, a, row, &lost);
        lp = log_share(taken, t);
        const float ratio = expf(lp - old);
        const float plain = ratio * adv, held = fminf(fmaxf(ratio, a.lo), a.hi) * adv;
        const bool cut = held < plain;
        loss = -(cut ? held : plain);
        float slope = cut ? 0.f : -plain;
        if (kl) {
          const float d = ref - lp, e = expm1f(d);
          loss = __fmaf_rn(a.beta, e - d, loss);
          slope = __fmaf_rn(a.beta, -e, slope);
        }
        slope *= scale * r.weight;
        n.base = base_of(t.m);
        n.slope = slope;
        n.inv = -slope / t.s;
      }
      if (lane == 0) {
        turn = n;
        if (rank == 0) {
          a.logp[row] = lp;
          a.loss[row] = loss;
        }
      }
    }
    if (on) ++use;
    __syncthreads();
    next = turn.next;
    // the next row's parts follow this row's gradient out of the same place
    const bool follow = on && next.on() && !is_set(&lost);
    uint8_t* dx = a.dlogits ? a.dlogits + row * a.ld * B::kBytes - r.head : nullptr;
    // whole blocks when dlogits lies on the 16-byte grid as the logits do
    const bool same = (reinterpret_cast<uintptr_t>(dx) & 15) == 0;
    const Base base = turn.base;
    const Pair c = pair(base.c, base.c), minus_mc = pair(-base.mc, -base.mc);
    const Pair by = pair(turn.inv, turn.inv);
    const float slope = turn.slope;
    const int32_t action_at = r.head + r.action * B::kBytes;
    const Bounds out = a.bounds(kDlogits);
#pragma unroll 1
    for (int p = 0; p < kParts; ++p) {
      const int32_t b0 = block_of(r, p), n = dx ? block_of(r, p + 1) - b0 : 0;
      const uint4* part = part_at(p);
      const bool plain = same && b0 != 0 && b0 + n != r.n_blk;
      const int32_t special = (action_at >> 4) - b0;  // the block with the action, if in this part
      uint4* to = reinterpret_cast<uint4*>(dx + static_cast<int64_t>(b0) * 16);
      // loops of the warp, not of the lane: lanes past the end sit a turn out
      if (plain && !on) {
        for (int32_t k = lane; k < n; k += 32)
          if (out.holds(to + k, 16, kSiteStore)) __stcs(to + k, make_uint4(0, 0, 0, 0));
      } else if (plain && (special < 0 || special >= n)) {
        for (int32_t k0 = 0; k0 < n; k0 += 32 * kBatch) {
          uint4 v[kBatch];
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            const int32_t k = k0 + 32 * j + lane;
            if (k < n) v[j] = part[k];
          }
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            Pair e[B::kElems / 2];
            exp_block<kType>(v[j], c, minus_mc, e);
            float f[B::kElems];
#pragma unroll
            for (int i = 0; i < B::kElems / 2; ++i) unpair(e[i] * by, f[2 * i], f[2 * i + 1]);
            const int32_t k = k0 + 32 * j + lane;
            if (k < n && out.holds(to + k, 16, kSiteStore)) __stcs(to + k, B::put(f));
          }
        }
      } else {
#pragma unroll 1
        for (int32_t k = lane; k < n; k += 32) {
          const int32_t b = b0 + k;
          float f[B::kElems];
#pragma unroll
          for (int j = 0; j < B::kElems; ++j) f[j] = 0.f;
          if (on) {
            Pair e[B::kElems / 2];
            exp_block<kType>(part[k], c, minus_mc, e);
#pragma unroll
            for (int j = 0; j < B::kElems / 2; ++j) unpair(e[j] * by, f[2 * j], f[2 * j + 1]);
#pragma unroll
            for (int j = 0; j < B::kElems; ++j)
              if (b * 16 + j * B::kBytes == action_at) f[j] += slope;
          }
          if (same && b * 16 >= r.head && b * 16 + 16 <= r.end) {
            if (out.holds(to + k, 16, kSiteStore)) __stcs(to + k, B::put(f));
          } else {
#pragma unroll
            for (int j = 0; j < B::kElems; ++j) {
              const int32_t at = b * 16 + j * B::kBytes;
              if (at >= r.head && at < r.end && out.holds(dx + at, B::kBytes, kSiteStore))
                B::set(dx + at, f[j]);
            }
          }
        }
      }
      __syncwarp();
      if (follow && lane == 0) fetch(next, next_row, p);
    }
    fetched = follow;
    r = next;
    row = next_row;
  }
  leave(n_cta, &lost);
}

// Sum with what each addition lost beside it (the file is built without
// contraction and reassociation). Beside an infinite sum `lo` holds inf - inf.
struct Sum {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float x) {
    const float t = hi + x, b = t - hi;
    lo += (hi - (t - b)) + (x - b);
    hi = t;
  }
  __device__ __forceinline__ float value() const { return fabsf(hi) < INFINITY ? hi + lo : hi; }
};

// The four sums over the rows that are not left out, by one CTA: each thread
// its rows in order, then a tree. fp64 would take most of this kernel's time
// (15 us of 16 at 2048 rows); two fp32 words carry as much as a result holds.
__global__ void __launch_bounds__(1024) stats_kernel(const Args a) {
  pdl_begin();
  __shared__ Sum part[4][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Sum s[4];
#pragma unroll 2
  for (int64_t row = tid; row < a.rows; row += 1024) {
    const float w = a.weight[row], lp = a.logp[row], old = a.old_logp[row];
    const float adv = a.advantage[row], loss = a.loss[row];
    const float ref = a.ref_logp ? a.ref_logp[row] : lp;
    if (w == 0.f || load_id(a.actions, a.action_bytes, row, a.vocab) < 0) continue;
    const float r = expf(lp - old), d = ref - lp;
    s[0].add(w * loss);
    s[1].add(w * (expm1f(d) - d));
    if (fminf(fmaxf(r, a.lo), a.hi) * adv < r * adv) s[2].add(w);
    s[3].add(w);
  }
  if (!a.ref_logp) s[1] = Sum();  // no KL term, also where lp - lp is not 0
  const auto tree = [](Sum& v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const float hi = __shfl_down_sync(0xffffffffu, v.hi, d);
      const float lo = __shfl_down_sync(0xffffffffu, v.lo, d);
      v.add(hi);
      v.lo += lo;
    }
  };
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    tree(s[k]);
    if (lane == 0) part[k][warp] = s[k];
  }
  __syncthreads();
  if (warp < 4) {
    Sum v = part[warp][lane];
    tree(v);
    if (lane == 0) a.stats[warp] = v.value();
  }
}

constexpr int kLaneBlocks = 16;
constexpr int kStageCap = 196 * 1024;  // a CTA's share of a row, at most
// the longest row off the 16-byte grid has a block more; whole blocks per part
static_assert(((ZERO_MAX_LOGIT_ROW_BYTES / 16 + 1) / (kMaxCluster * kMaxWarps * kParts) + 1) *
                      (16 * kMaxWarps * kParts) <= kStageCap,
              "a cluster holds the longest row");
constexpr int kStageGoal = 72 * 1024;  // three CTAs per SM

// bytes of shared memory per CTA for rows of at most `blocks` blocks
int64_t stage_bytes(int64_t blocks, int n_cta, int warps, int32_t* part_cap) {
  const int64_t cap = ceil_div(blocks, static_cast<int64_t>(n_cta) * warps * kParts);
  *part_cap = static_cast<int32_t>(cap);
  return cap * 16 * warps * kParts;
}

struct Launch {
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  Launch(int64_t clusters, int n_cta, int warps, size_t smem, cudaStream_t st) : cfg(), attr() {
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * n_cta));
    cfg.blockDim = dim3(32 * warps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = n_cta;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = kProgrammaticLaunch ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
  }
};

// Clusters of `fn` the device holds at once (0 on error). One more would
// wait for a whole row of rows: the grid is exactly these.
int resident_clusters(const void* fn, int n_cta, int warps, size_t smem) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  try {
    static std::mutex mu;
    static std::map<std::tuple<const void*, int, int, size_t>, int> known;
    std::lock_guard<std::mutex> lock(mu);
    int& n = known[std::make_tuple(fn, dev, n_cta, smem)];
    if (n == 0) {
      Launch l(1, n_cta, warps, smem, nullptr);
      if ((smem && cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        kStageCap) != cudaSuccess) ||
          cudaOccupancyMaxActiveClusters(&n, fn, &l.cfg) != cudaSuccess)
        n = 0;
    }
    return n;
  } catch (...) {  // no exception leaves a C call
    return 0;
  }
}

template <int kType, bool kGrad, int kWarps>
int launch_warps(const Args& a, int n_cta, size_t smem, int32_t cap, cudaStream_t st) {
  const void* fn = kGrad ? reinterpret_cast<const void*>(policy_kernel<kType, kWarps>)
                         : reinterpret_cast<const void*>(logp_kernel<kType, kWarps>);
  const int most = resident_clusters(fn, n_cta, kWarps, smem);
  if (most <= 0) return ZERO_ECUDA;
  Launch l(std::min<int64_t>(a.rows, most), n_cta, kWarps, smem, st);
  return status_of(kGrad ? cudaLaunchKernelEx(&l.cfg, policy_kernel<kType, kWarps>, a, cap)
                         : cudaLaunchKernelEx(&l.cfg, logp_kernel<kType, kWarps>, a));
}

template <int kType, bool kGrad>
int launch(const Args& a, cudaStream_t st) {
  const int64_t blocks = (a.vocab * Block<kType>::kBytes + 15 + 15) / 16;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return ZERO_ECUDA;
  // Warps per CTA: up to kLaneBlocks blocks per lane, so that short rows run
  // many to an SM (2000 rows of 1111: 8 warps 23.4 us, 1 warp 12.6 us); more
  // warps, then more CTAs, while few rows would leave SMs idle and each lane
  // keeps two blocks.
  int warps = 1, n_cta = 1;
  int32_t cap = 0;
  while (warps < kMaxWarps && blocks > kLaneBlocks * 32 * warps) warps *= 2;
  while (warps < kMaxWarps && a.rows * warps < 8 * sms && blocks > 2 * 2 * 32 * warps) warps *= 2;
  while (n_cta < kMaxCluster && kGrad && stage_bytes(blocks, n_cta, warps, &cap) > kStageGoal)
    n_cta *= 2;
  while (n_cta < kMaxCluster && a.rows * n_cta < 2 * sms && blocks > 2 * 2 * 32 * warps * n_cta)
    n_cta *= 2;
  const int64_t smem = kGrad ? stage_bytes(blocks, n_cta, warps, &cap) : 0;
  if (smem > kStageCap) return ZERO_ERANGE;
  const size_t bytes = static_cast<size_t>(smem);
  switch (warps) {
    case 1: return launch_warps<kType, kGrad, 1>(a, n_cta, bytes, cap, st);
    case 2: return launch_warps<kType, kGrad, 2>(a, n_cta, bytes, cap, st);
    case 4: return launch_warps<kType, kGrad, 4>(a, n_cta, bytes, cap, st);
    default: return launch_warps<kType, kGrad, 8>(a, n_cta, bytes, cap, st);
  }
}

template <bool kGrad>
int launch_type(const Args& a, int32_t dtype, cudaStream_t st) {
  switch (dtype) {
    case ZERO_BF16: return launch<ZERO_BF16, kGrad>(a, st);
    case ZERO_FP16: return launch<ZERO_FP16, kGrad>(a, st);
    default: return launch<ZERO_FP32, kGrad>(a, st);
  }
}

int check(const void* logits, int64_t rows, int64_t vocab, int64_t ld, int32_t dtype,
          const void* actions, int32_t action_bytes, const float* logp) {
  if (rows < 0 || vocab < 1 || ld < vocab || !(is_dtype16(dtype) || dtype == ZERO_FP32) ||
      (action_bytes != 4 && action_bytes != 8))
    return ZERO_EINVAL;
  const size_t size = dtype == ZERO_FP32 ? 4 : 2;
  constexpr int64_t kMost = int64_t{1} << 31;
  if (vocab > kMost || vocab * static_cast<int64_t>(size) > (int64_t{1} << 30) || rows > kMost ||
      ld > kMost)
    return ZERO_ERANGE;
  if (rows == 0) return ZERO_OK;
  if (!logits || !actions || !logp) return ZERO_EINVAL;
  if (!aligned(logits, size) || !aligned(actions, action_bytes) || !aligned(logp, 4))
    return ZERO_EALIGN;
  return ZERO_OK;
}

}  // namespace zp

#ifdef ZERO_CHECKED
extern "C" int zp_collect_checks(unsigned long long* count, unsigned long long* first) {
  return collect_checks(count, first);
}
#endif

extern "C" {

ZERO_API int zero_token_logp(const void* logits, int64_t rows, int64_t vocab, int64_t ld,
                             int32_t dtype, const void* actions, int32_t action_bytes,
                             float* logp, void* stream) {
  using namespace zp;
  const int rc = check(logits, rows, vocab, ld, dtype, actions, action_bytes, logp);
  if (rc != ZERO_OK || rows == 0) return rc;
  Args a = new_args<Args>();
  a.logits = static_cast<const uint8_t*>(logits);
  a.set_bounds(kLogits, logits, rows, vocab, ld, dtype == ZERO_FP32 ? 4 : 2);
  a.actions = actions;
  a.action_bytes = action_bytes;
  a.rows = rows, a.vocab = vocab, a.ld = ld;
  a.logp = logp;
  return launch_type<false>(a, dtype, static_cast<cudaStream_t>(stream));
}

ZERO_API int zero_policy_loss(const void* logits, int64_t rows, int64_t vocab, int64_t ld,
                              int32_t dtype, const void* actions, int32_t action_bytes,
                              const float* old_logp, const float* ref_logp,
                              const float* advantage, const float* weight,
                              const zero_policy_params* params, const zero_scaler* d_scaler,
                              float* logp, float* loss, float* stats, void* dlogits,
                              void* stream) {
  using namespace zp;
  const int rc = check(logits, rows, vocab, ld, dtype, actions, action_bytes, logp);
  if (rc != ZERO_OK) return rc;
  if (!params || !(params->clip_lo >= 0 && params->clip_lo < 1) || !(params->clip_hi >= 0) ||
      !(params->kl_coef >= 0) || std::isinf(params->clip_hi) || std::isinf(params->kl_coef))
    return ZERO_EINVAL;
  const size_t size = dtype == ZERO_FP32 ? 4 : 2;
  if (vocab * static_cast<int64_t>(size) > ZERO_MAX_LOGIT_ROW_BYTES) return ZERO_ERANGE;
  if (rows && (!old_logp || !advantage || !weight || !loss)) return ZERO_EINVAL;
  if (!aligned(old_logp, 4) || !aligned(ref_logp, 4) || !aligned(advantage, 4) ||
      !aligned(weight, 4) || !aligned(loss, 4) || !aligned(stats, 4) || !aligned(dlogits, size) ||
      !aligned(d_scaler, 16))
    return ZERO_EALIGN;
  Args a = new_args<Args>();
  a.logits = static_cast<const uint8_t*>(logits);
  a.set_bounds(kLogits, logits, rows, vocab, ld, dtype == ZERO_FP32 ? 4 : 2);
  a.dlogits = static_cast<uint8_t*>(dlogits);
  a.set_bounds(kDlogits, dlogits, rows, vocab, ld, static_cast<int64_t>(size));
  a.actions = actions;
  a.action_bytes = action_bytes;
  a.old_logp = old_logp, a.ref_logp = ref_logp, a.advantage = advantage, a.weight = weight;
  a.scaler = d_scaler;
  a.logp = logp, a.loss = loss, a.stats = stats;
  a.rows = rows, a.vocab = vocab, a.ld = ld;
  a.lo = static_cast<float>(1.0 - params->clip_lo);
  a.hi = static_cast<float>(1.0 + params->clip_hi);
  a.beta = static_cast<float>(params->kl_coef);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rows) {
    const int e = launch_type<true>(a, dtype, st);
    if (e != ZERO_OK) return e;
  }
  if (stats) return status_of(launch_pdl(stats_kernel, dim3(1), dim3(1024), 0, st, a));
  return ZERO_OK;
}

}  // extern "C"
