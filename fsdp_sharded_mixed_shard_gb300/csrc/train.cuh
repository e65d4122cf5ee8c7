// train.cuh -- what the kernels behind zero_train.h share: the element types,
// 16-byte vectors of eight 16-bit elements, launch helpers and host checks.
#ifndef ZERO_TRAIN_CUH
#define ZERO_TRAIN_CUH

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

// this unit's violations are collected by the unit that owns the status call
#define ZERO_CHECKED_LEAF
#include "checked.cuh"
#include "pdl.cuh"
#include "zero_train.h"

namespace zt {

constexpr int kVec = 8;  // 16-bit elements per 16-byte vector

// Two fp32 values as one operand: sm_100's packed fp32 arithmetic does both
// in one instruction, each rounded to nearest even.
struct Pair {
  uint64_t v;
};

__device__ __forceinline__ Pair pair(float x, float y) {
  Pair p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p.v) : "f"(x), "f"(y));
  return p;
}

__device__ __forceinline__ void unpair(const Pair& p, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p.v));
}

__device__ __forceinline__ Pair operator*(const Pair& a, const Pair& b) {
  Pair p;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(p.v) : "l"(a.v), "l"(b.v));
  return p;
}

__device__ __forceinline__ Pair fma2(const Pair& a, const Pair& b, const Pair& c) {
  Pair p;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(p.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return p;
}

__device__ __forceinline__ Pair operator+(const Pair& a, const Pair& b) {
  Pair p;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(p.v) : "l"(a.v), "l"(b.v));
  return p;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// One 16-bit element (its bits) to fp32, exactly.
template <bool kBf16>
__device__ __forceinline__ float widen(uint32_t bits) {
  if constexpr (kBf16) return __uint_as_float(bits << 16);
  else return __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
}

// Both halves of a word to fp32, exactly.
template <bool kBf16>
__device__ __forceinline__ void widen2(uint32_t w, float& a, float& b) {
  if constexpr (kBf16) {
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xFFFF0000u);
  } else {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    a = f.x;
    b = f.y;
  }
}

// fp32 to one 16-bit element, to nearest even.
template <bool kBf16>
__device__ __forceinline__ uint16_t narrow(float a) {
  if constexpr (kBf16) return __bfloat16_as_ushort(__float2bfloat16_rn(a));
  else return __half_as_ushort(__float2half_rn(a));
}

template <bool kBf16>
__device__ __forceinline__ uint32_t narrow2(float a, float b) {
  uint32_t w;
  if constexpr (kBf16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
  return w;
}

template <bool kBf16>
__device__ __forceinline__ void widen8(const uint4& v, float (&f)[8]) {
  widen2<kBf16>(v.x, f[0], f[1]);
  widen2<kBf16>(v.y, f[2], f[3]);
  widen2<kBf16>(v.z, f[4], f[5]);
  widen2<kBf16>(v.w, f[6], f[7]);
}

template <bool kBf16>
__device__ __forceinline__ uint4 narrow8(const float (&f)[8]) {
  return make_uint4(narrow2<kBf16>(f[0], f[1]), narrow2<kBf16>(f[2], f[3]),
                    narrow2<kBf16>(f[4], f[5]), narrow2<kBf16>(f[6], f[7]));
}

// The 16 bytes that start kDistance bytes (even, below 16) into x and run on
// into y, the block after it.
template <int kDistance>
__device__ __forceinline__ uint4 shifted_by(const uint4& x, const uint4& y) {
  constexpr int kWord = kDistance / 4;
  const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    o[j] = kDistance & 2 ? __funnelshift_r(w[kWord + j], w[kWord + j + 1], 16) : w[kWord + j];
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// The same for a distance d in 0..16 that all lanes share (rows of a warp's
// own): a branch and at most four shifts, where selects by d take 15 (SwiGLU
// both ways, 8000 x 8001 bf16: 264 us against 276; the table gradient, which
// loads many rows at once, 101 against 90 at 16384 x 1111).
__device__ __forceinline__ uint4 shifted_alike(const uint4& x, const uint4& y, int d) {
  switch (d >> 1) {
    case 0: return x;
    case 1: return shifted_by<2>(x, y);
    case 2: return shifted_by<4>(x, y);
    case 3: return shifted_by<6>(x, y);
    case 4: return shifted_by<8>(x, y);
    case 5: return shifted_by<10>(x, y);
    case 6: return shifted_by<12>(x, y);
    case 7: return shifted_by<14>(x, y);
    default: return y;
  }
}

// The same for d below 16 that may differ between lanes, or where a branch
// would keep the loads behind it waiting: words and halfword picked in steps.
__device__ __forceinline__ uint4 shifted(const uint4& x, const uint4& y, int d) {
  const uint32_t c[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
  uint32_t t[6], w[5], o[4];
#pragma unroll
  for (int j = 0; j < 6; ++j) t[j] = d & 8 ? c[j + 2] : c[j];
#pragma unroll
  for (int j = 0; j < 5; ++j) w[j] = d & 4 ? t[j + 1] : t[j];
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = __funnelshift_r(w[j], w[j + 1], (d & 2) * 8);
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// The 16 bytes that end d bytes (even, below 16) before the end of y.
__device__ __forceinline__ uint4 shifted_back(const uint4& x, const uint4& y, int d) {
  return d ? shifted(x, y, 16 - d) : y;
}

// Eight 16-bit elements at any element address, from the one or two 16-byte
// blocks that hold them; the caller knows that all eight lie in its buffer.
// kAlike: the warp's lanes load one row, nothing else is loaded meanwhile.
template <bool kAlike>
__device__ __forceinline__ uint4 load8_any(const uint16_t* p) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  const uint4* block = reinterpret_cast<const uint4*>(at & ~static_cast<uintptr_t>(15));
  const uint4 x = *block;
  const int d = static_cast<int>(at & 15);
  if (d == 0) return x;
  return kAlike ? shifted_alike(x, block[1], d) : shifted(x, block[1], d);
}

__device__ __forceinline__ uint64_t global_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

// given up: lets the copies and products in flight (microseconds) land
__device__ __forceinline__ void drain() {
  constexpr uint64_t kDrainNs = 1000000;
  const uint64_t t0 = global_ns();
  while (global_ns() - t0 < kDrainNs) {
  }
}

constexpr uint64_t kWaitLimitNs = 2000000000ull;

// A mistake to make on purpose (zero_selftest_plant), and how long a wait may
// take: a base of the kernels' arguments, with nothing in it in the release
// build. (An empty member changed the policy kernel's code: 72.8 to 73.5 us at
// 2048 x 50257.)
struct Plant {
#ifdef ZERO_CHECKED
  int32_t what;
  int64_t at;
  uint64_t limit_ns;
  __device__ __forceinline__ bool holds(int32_t kind, int64_t where) const {
    return what == kind && at == where;
  }
  __device__ __forceinline__ uint64_t limit() const { return limit_ns; }
#else
  __device__ __forceinline__ bool holds(int32_t, int64_t) const { return false; }
  __device__ __forceinline__ uint64_t limit() const { return kWaitLimitNs; }
#endif
};

// The bytes a call may touch of one of its buffers. The checked build tests
// every element that a kernel is about to load or store against them, from the
// address itself, and leaves out what lies outside; the release build has
// neither the bytes nor the tests.
struct Bounds {
#ifdef ZERO_CHECKED
  uintptr_t lo, hi;
#endif
  __device__ __forceinline__ bool holds(const void* p, int64_t bytes, int site) const {
#ifdef ZERO_CHECKED
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    return bytes <= 0 || ZCHECK(at >= lo && at + bytes <= hi, site,
                                static_cast<int64_t>(at - lo));
#else
    (void)p, (void)bytes, (void)site;
    return true;
#endif
  }
  // whole 16-byte blocks, the first and last of which may be the buffer's in part
  __device__ __forceinline__ bool holds_blocks(const void* p, int64_t bytes, int site) const {
#ifdef ZERO_CHECKED
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    return bytes <= 0 || ZCHECK(at + 16 > lo && at + bytes < hi + 16, site,
                                static_cast<int64_t>(at - lo));
#else
    (void)p, (void)bytes, (void)site;
    return true;
#endif
  }
};

// What the arguments of all kernels begin with: the plant and the bounds of the
// call's kBuffers buffers.
template <int kBuffers>
struct Checked : Plant {
#ifdef ZERO_CHECKED
  Bounds buffers[kBuffers];
  __device__ __forceinline__ Bounds bounds(int k) const { return buffers[k]; }
#else
  __device__ __forceinline__ Bounds bounds(int) const { return Bounds{}; }
#endif
  // host: buffer k is `rows` rows of `cols` elements of `size` bytes, ld apart
  void set_bounds(int k, const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t size) {
#ifdef ZERO_CHECKED
    Bounds& b = buffers[k];
    b.lo = b.hi = reinterpret_cast<uintptr_t>(p);
    if (!p || rows <= 0 || cols <= 0) return;
    b.hi += ((rows - 1) * ld + cols) * size;
    if (what == ZERO_PLANT_SHORT && at == k) b.hi -= size;
#else
    (void)k, (void)p, (void)rows, (void)cols, (void)ld, (void)size;
#endif
  }
};

// arguments of a launch with the plant that holds for it, all else 0
#ifdef ZERO_CHECKED
Plant planted();
template <class Args>
Args new_args() {
  Args a = {};
  static_cast<Plant&>(a) = planted();
  return a;
}
#else
template <class Args>
Args new_args() { return Args{}; }
#endif

// A warp's store of up to 256 neighbouring elements to any element address,
// eight per lane (v), `count` of them in all: through shared memory, so that
// whole 16-byte blocks of the destination leave as such and only the elements
// before the first and after the last go one by one. All lanes call it; stage
// is the warp's own kStageWarp bytes, 16-byte aligned.
constexpr int kStageWarp = 16 + 512 + 16;

__device__ __forceinline__ void store_any(uint8_t* stage, uint16_t* to, int count, int lane,
                                          const uint4& v, const Bounds& in) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(to);
  const int d = static_cast<int>(at & 15);
  uint4* mine = reinterpret_cast<uint4*>(stage + 16);
  __syncwarp();  // the stage's last use is read
  mine[lane] = v;
  __syncwarp();
  // destination block k: bytes [16 k - d, 16 k - d + 16) of the run
  uint8_t* blocks = reinterpret_cast<uint8_t*>(at - d);
  const int bytes = 2 * count;
  const auto block = [&](int k) {
    if (16 * k - d < 0 || 16 * k - d + 16 > bytes) return;
    if (!in.holds(blocks + 16 * k, 16, kSiteStore)) return;
    const uint4 x = mine[k - 1];
    const uint4 y = mine[k];
    __stcs(reinterpret_cast<uint4*>(blocks + 16 * k), shifted_alike(x, y, 16 - d));
  };
  block(lane);  // block 32 is never whole unless d is 0, and then it is past the run
  // at most seven elements before the first whole block and after the last
  const uint16_t* elems = reinterpret_cast<const uint16_t*>(stage + 16);
  const int head = d ? min((16 - d) >> 1, count) : 0;
  const int tail = max(head, (((bytes + d) & ~15) - d) >> 1);
  if (lane < head && in.holds(to + lane, 2, kSiteStore)) to[lane] = elems[lane];
  if (tail + lane < count && in.holds(to + tail + lane, 2, kSiteStore))
    to[tail + lane] = elems[tail + lane];
}

// Token ids are int32 or int64; an id outside [0, limit) becomes -1.
__device__ __forceinline__ int64_t load_id(const void* ids, int32_t bytes, int64_t i,
                                           int64_t limit) {
  const int64_t v = bytes == 4 ? static_cast<int64_t>(static_cast<const int32_t*>(ids)[i])
                               : static_cast<const int64_t*>(ids)[i];
  return v >= 0 && v < limit ? v : -1;
}

inline bool aligned(const void* p, size_t n) {
  return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline bool is_dtype16(int32_t d) { return d == ZERO_BF16 || d == ZERO_FP16; }

inline int status_of(cudaError_t e) { return e == cudaSuccess ? ZERO_OK : ZERO_ECUDA; }

}  // namespace zt

#endif
