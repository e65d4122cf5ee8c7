/*
 * policy.cu -- token log-probabilities and the clipped policy loss with its
 * gradient (zero_train.h).
 *
 * A row's softmax needs its maximum and sum before its gradient can be
 * written, so the row is read once into the shared memory of a cluster of 1
 * to 8 CTAs and the gradient is formed from there: rows * vocab elements read
 * and as many written, nothing in between. Each thread keeps a running
 * maximum m and sum s of exp(x - m) over its vectors (a new maximum rescales
 * s), the CTA joins its threads' pairs, and every CTA sends its pair to all
 * others of the cluster over distributed shared memory; all join them in rank
 * order, so all hold the same bits.
 *
 * A row of an odd vocabulary starts anywhere. It is numbered in the 16-byte
 * blocks of its addresses: whole blocks move as blocks, the elements of the
 * first and last partial block one by one, and in shared memory the parts of
 * those blocks outside the row hold -inf, so the arithmetic sees whole blocks.
 */
#include "train.cuh"

#include <algorithm>
#include <cmath>

namespace zp {

using namespace zt;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr float kLog2e = 1.4426950408889634f;

struct Args {
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

// softmax statistics: largest value and sum of exp(x - m); (-inf, 0) for none
struct Stat {
  float m, s;
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// exp(x - m) for m >= x; m finite
__device__ __forceinline__ float exp_below(float x, float m) {
  return exp2_fast((x - m) * kLog2e);
}

__device__ __forceinline__ Stat join(const Stat& a, const Stat& b) {
  const float m = fmaxf(a.m, b.m);
  // a side with nothing adds nothing; inf and NaN go on into the sum
  const float sa = a.s == 0.f ? 0.f : a.s * exp_below(a.m, m);
  const float sb = b.s == 0.f ? 0.f : b.s * exp_below(b.m, m);
  return Stat{m, sa + sb};
}

// elements of a 16-byte block as fp32
template <int kType>
struct Block {
  static constexpr int kElems = 8;
  static constexpr int kBytes = 2;
  __device__ static __forceinline__ void get(const uint4& v, float (&f)[8]) {
    widen8<kType == ZERO_BF16>(v, f);
  }
  __device__ static __forceinline__ uint4 put(const float (&f)[8]) {
    return narrow8<kType == ZERO_BF16>(f);
  }
  __device__ static __forceinline__ float one(const uint8_t* p) {
    return widen<kType == ZERO_BF16>(*reinterpret_cast<const uint16_t*>(p));
  }
  __device__ static __forceinline__ void set(uint8_t* p, float x) {
    *reinterpret_cast<uint16_t*>(p) = narrow<kType == ZERO_BF16>(x);
  }
};

template <>
struct Block<ZERO_FP32> {
  static constexpr int kElems = 4;
  static constexpr int kBytes = 4;
  __device__ static __forceinline__ void get(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
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

template <int kElems>
__device__ __forceinline__ void add_block(Stat& t, const float (&f)[kElems]) {
  float top = f[0];
#pragma unroll
  for (int j = 1; j < kElems; ++j) top = fmaxf(top, f[j]);
  if (top > t.m) {
    t.s = t.s == 0.f ? 0.f : t.s * exp_below(t.m, top);
    t.m = top;
  }
  // nothing but -inf so far: no sum to form (a NaN beside it still counts)
  const float m = t.m == -INFINITY ? 0.f : t.m;
#pragma unroll
  for (int j = 0; j < kElems; ++j) t.s += exp_below(f[j], m);
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

// store one Stat into the same shared variable of CTA `rank` of the cluster
__device__ __forceinline__ void send(Stat* local, uint32_t rank, const Stat& v) {
  const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(local));
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(at), "r"(rank));
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(remote), "f"(v.m), "f"(v.s)
               : "memory");
}

template <int kType, bool kGrad>
__global__ void __launch_bounds__(kThreads) policy_kernel(const Args a) {
  pdl_begin();
  using B = Block<kType>;
  extern __shared__ __align__(16) uint8_t stage[];
  __shared__ Stat of_warp[kWarps];
  __shared__ Stat of_cta[2][kMaxCluster];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank(), n_cta = cluster_size();
  const int64_t first = blockIdx.x / n_cta, step = gridDim.x / n_cta;
  const float scale = kGrad && a.scaler ? a.scaler->scale : 1.f;
  int parity = 0;
  cluster_sync();  // every CTA of the cluster runs before any sends to it
  for (int64_t row = first; row < a.rows; row += step) {
    const uint8_t* x = a.logits + row * a.ld * B::kBytes;
    uint8_t* dx = kGrad && a.dlogits ? a.dlogits + row * a.ld * B::kBytes : nullptr;
    // this CTA's blocks [b0, b1) of the row's n_blk; block 0 starts `head`
    // bytes before the row
    const int64_t bytes = a.vocab * B::kBytes;
    const int64_t head = static_cast<int64_t>(reinterpret_cast<uintptr_t>(x) & 15);
    const int64_t n_blk = (head + bytes + 15) / 16;
    const int64_t b0 = n_blk * rank / n_cta, b1 = n_blk * (rank + 1) / n_cta;
    const int64_t action = load_id(a.actions, a.action_bytes, row, a.vocab);
    const float w = kGrad ? a.weight[row] : 1.f;
    const bool on = action >= 0 && w != 0.f;
    Stat t = {-INFINITY, 0.f};
    float picked = 0.f;
    if (on) {
      if (tid == 0) picked = B::one(x + action * B::kBytes);
      for (int64_t b = b0 + tid; b < b1; b += kThreads) {
        const int64_t at = b * 16 - head;  // byte of the row
        uint4 v;
        if (at >= 0 && at + 16 <= bytes) {
          v = __ldcs(reinterpret_cast<const uint4*>(x + at));
        } else {
          float f[B::kElems];
#pragma unroll
          for (int j = 0; j < B::kElems; ++j) {
            const int64_t e = at + j * B::kBytes;
            f[j] = e >= 0 && e < bytes ? B::one(x + e) : -INFINITY;
          }
          v = B::put(f);
        }
        if constexpr (kGrad) *reinterpret_cast<uint4*>(stage + (b - b0) * 16) = v;
        float f[B::kElems];
        B::get(v, f);
        add_block(t, f);
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) {
        const Stat o = {__shfl_xor_sync(0xffffffffu, t.m, d), __shfl_xor_sync(0xffffffffu, t.s, d)};
        // the same operands in the same order on both lanes
        t = (lane & d) ? join(o, t) : join(t, o);
      }
      if (lane == 0) of_warp[warp] = t;
      __syncthreads();
      if (tid < static_cast<int>(n_cta)) {
        Stat c = of_warp[0];
        for (int k = 1; k < kWarps; ++k) c = join(c, of_warp[k]);
        send(&of_cta[parity][rank], tid, c);
      }
      __syncwarp();
      cluster_sync();
      t = of_cta[parity][0];
      for (uint32_t k = 1; k < n_cta; ++k) t = join(t, of_cta[parity][k]);
      parity ^= 1;
    }
    const float log_s = on ? logf(t.s) : 0.f;
    float slope = 0.f;
    __shared__ float shared_slope;
    if (tid == 0) {
      float lp = 0.f, loss = 0.f;
      if (on) {
        lp = (picked - t.m) - log_s;
        if constexpr (kGrad) {
          const float r = expf(lp - a.old_logp[row]), adv = a.advantage[row];
          const float plain = r * adv, held = fminf(fmaxf(r, a.lo), a.hi) * adv;
          const bool cut = held < plain;
          loss = -(cut ? held : plain);
          slope = cut ? 0.f : -plain;
          if (a.ref_logp && a.beta != 0.f) {
            const float d = a.ref_logp[row] - lp, e = expm1f(d);
            loss = __fmaf_rn(a.beta, e - d, loss);
            slope = __fmaf_rn(a.beta, -e, slope);
          }
          slope *= scale * w;
        }
      }
      if (rank == 0) {
        a.logp[row] = lp;
        if constexpr (kGrad) a.loss[row] = loss;
      }
      if constexpr (kGrad) shared_slope = slope;
    }
    if constexpr (kGrad) {
      if (!dx) {
        __syncthreads();  // of_warp is free again
        continue;
      }
      __syncthreads();
      slope = shared_slope;
      // dlogits = slope ([j == a] - p); the row's own blocks when it lies on
      // the 16-byte grid as the logits do, else element by element
      const bool same = (reinterpret_cast<uintptr_t>(dx) & 15) == static_cast<uintptr_t>(head);
      const float m = t.m, inv = on ? -slope / t.s : 0.f;
      for (int64_t b = b0 + tid; b < b1; b += kThreads) {
        const int64_t at = b * 16 - head;
        float f[B::kElems];
        if (on) {
          B::get(*reinterpret_cast<const uint4*>(stage + (b - b0) * 16), f);
#pragma unroll
          for (int j = 0; j < B::kElems; ++j) {
            f[j] = exp_below(f[j], m) * inv;
            if (at + j * B::kBytes == action * B::kBytes) f[j] += slope;
          }
        } else {
#pragma unroll
          for (int j = 0; j < B::kElems; ++j) f[j] = 0.f;
        }
        if (same && at >= 0 && at + 16 <= bytes) {
          __stcs(reinterpret_cast<uint4*>(dx + at), B::put(f));
        } else {
#pragma unroll
          for (int j = 0; j < B::kElems; ++j) {
            const int64_t e = at + j * B::kBytes;
            if (e >= 0 && e < bytes) B::set(dx + e, f[j]);
          }
        }
      }
      __syncthreads();  // stage, of_warp and shared_slope are free again
    } else {
      __syncthreads();
    }
  }
}

// The four sums over the rows that are not left out, by one CTA: each thread
// its rows in order, then a tree.
__global__ void __launch_bounds__(1024) stats_kernel(const Args a) {
  pdl_begin();
  __shared__ double part[4][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  double s[4] = {0, 0, 0, 0};
  for (int64_t row = tid; row < a.rows; row += 1024) {
    const float w = a.weight[row];
    if (w == 0.f || load_id(a.actions, a.action_bytes, row, a.vocab) < 0) continue;
    const float lp = a.logp[row], r = expf(lp - a.old_logp[row]), adv = a.advantage[row];
    s[0] += static_cast<double>(w) * a.loss[row];
    if (a.ref_logp) {
      const float d = a.ref_logp[row] - lp;
      s[1] += static_cast<double>(w) * (expm1f(d) - d);
    }
    if (fminf(fmaxf(r, a.lo), a.hi) * adv < r * adv) s[2] += w;
    s[3] += w;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s[k] += __shfl_xor_sync(0xffffffffu, s[k], d);
    if (lane == 0) part[k][warp] = s[k];
  }
  __syncthreads();
  if (warp < 4) {
    double v = part[warp][lane];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    if (lane == 0) a.stats[warp] = static_cast<float>(v);
  }
}

constexpr int kStageCap = 192 * 1024;  // a CTA's share of a row, at most
constexpr int kStageGoal = 72 * 1024;  // three CTAs per SM

template <int kType, bool kGrad>
int launch(const Args& a, cudaStream_t st) {
  const int64_t blocks = (a.vocab * Block<kType>::kBytes + 15 + 15) / 16;
  int n_cta = 1;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return ZERO_ECUDA;
  while (n_cta < kMaxCluster && kGrad && ceil_div(blocks, n_cta) * 16 > kStageGoal) n_cta *= 2;
  while (n_cta < kMaxCluster && a.rows * n_cta < 2 * sms && blocks / n_cta > 2 * kThreads) n_cta *= 2;
  const size_t smem = kGrad ? static_cast<size_t>(ceil_div(blocks, n_cta) * 16) : 0;
  if (smem > kStageCap) return ZERO_ERANGE;
  const void* fn = reinterpret_cast<const void*>(policy_kernel<kType, kGrad>);
  if (smem > 48 * 1024 && cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kStageCap) != cudaSuccess)
    return ZERO_ECUDA;
  const int per_sm = kGrad ? std::max<int>(1, std::min<int>(8, 220 * 1024 / static_cast<int>(smem + 1280))) : 8;
  const int64_t clusters = std::min<int64_t>(a.rows, std::max<int64_t>(1, static_cast<int64_t>(sms) * per_sm / n_cta));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * n_cta));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = n_cta;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = kProgrammaticLaunch ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return status_of(cudaLaunchKernelEx(&cfg, policy_kernel<kType, kGrad>, a));
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
  if (vocab > (int64_t{1} << 30) || rows > (int64_t{1} << 31) || ld > (int64_t{1} << 31))
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
  Args a = {};
  a.logits = static_cast<const uint8_t*>(logits);
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
  if (vocab * static_cast<int64_t>(size) > ZERO_MAX_LOGIT_ROW_BYTES - 16 * kMaxCluster)
    return ZERO_ERANGE;
  if (rows && (!old_logp || !advantage || !weight || !loss)) return ZERO_EINVAL;
  if (!aligned(old_logp, 4) || !aligned(ref_logp, 4) || !aligned(advantage, 4) ||
      !aligned(weight, 4) || !aligned(loss, 4) || !aligned(stats, 4) || !aligned(dlogits, size) ||
      !aligned(d_scaler, 16))
    return ZERO_EALIGN;
  Args a = {};
  a.logits = static_cast<const uint8_t*>(logits);
  a.dlogits = static_cast<uint8_t*>(dlogits);
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
