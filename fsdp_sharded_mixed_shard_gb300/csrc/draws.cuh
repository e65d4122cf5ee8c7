// draws.cuh -- dropout's random bits (zero_block.h), drawn where they are used.
//
// Philox 4x32 with 7 rounds (Salmon, Moraes, Dror and Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", 2011: 7 are the fewest that passed all their
// tests): one counter gives 128 bits, 16 for each of a lane's eight columns,
// so an element costs about nine instructions; 32 bits each would double that
// and make dropout's passes arithmetic-bound.
#ifndef ZERO_DRAWS_CUH
#define ZERO_DRAWS_CUH

#include "train.cuh"
#include "zero_block.h"

namespace zt {

// A call's dropout as its kernels take it: nothing is left out where
// threshold is 0.
struct Drop {
  uint32_t key0, key1, call;
  uint32_t threshold;  // T << 16
  const uint32_t* d_step;
  float scale;         // 65536 / (65536 - T)
};

__device__ __forceinline__ uint32_t step_of(const Drop& d) {
  return d.threshold && d.d_step ? *d.d_step : 0;
}

// The eight random halves of columns [8 group, 8 group + 8) of a row.
__device__ __forceinline__ uint4 draw8(const Drop& d, uint32_t step, uint32_t row,
                                       uint32_t group) {
  uint32_t c0 = group, c1 = row, c2 = d.call, c3 = step, k0 = d.key0, k1 = d.key1;
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    const uint64_t a = static_cast<uint64_t>(0xD2511F53u) * c0;
    const uint64_t b = static_cast<uint64_t>(0xCD9E8D57u) * c2;
    c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0;
    c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
    c1 = static_cast<uint32_t>(b);
    c3 = static_cast<uint32_t>(a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// The factor of each of the eight elements is 0 or the scale; what is left out
// is chosen, not multiplied, so that infinities and NaN go too.
__device__ __forceinline__ void drop8(const Drop& d, const uint4& draw, float (&f)[8]) {
  const uint32_t w[4] = {draw.x, draw.y, draw.z, draw.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = (w[j] << 16) >= d.threshold ? f[2 * j] * d.scale : 0.f;
    f[2 * j + 1] = w[j] >= d.threshold ? f[2 * j + 1] * d.scale : 0.f;
  }
}

// Which of the eight stay, a bit each.
__device__ __forceinline__ uint32_t keep8(const Drop& d, const uint4& draw) {
  const uint32_t w[4] = {draw.x, draw.y, draw.z, draw.w};
  uint32_t keep = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    keep |= (w[j] << 16) >= d.threshold ? 1u << (2 * j) : 0;
    keep |= w[j] >= d.threshold ? 2u << (2 * j) : 0;
  }
  return keep;
}

// 0 <= p < 1, aligned pointers
inline int check_drop(const zero_dropout_params& p) {
  if (!(p.p >= 0.0 && p.p < 1.0)) return ZERO_EINVAL;
  return aligned(p.d_step, 4) ? ZERO_OK : ZERO_EALIGN;
}

inline Drop drop_of(const zero_dropout_params& p) {
  const int t = static_cast<int>(p.p * 65536.0 + 0.5);
  const uint32_t threshold = t < 65535 ? t : 65535;
  Drop d = {};
  d.key0 = static_cast<uint32_t>(p.seed);
  d.key1 = static_cast<uint32_t>(p.seed >> 32);
  d.call = p.call;
  d.threshold = threshold << 16;
  d.d_step = p.d_step;
  d.scale = static_cast<float>(65536.0 / (65536 - threshold));
  return d;
}

}  // namespace zt

#endif
