/*
 * wgrad.cu -- weight gradient of a linear layer from its input's 8-bit
 * checkpoint (zero_train.h): dw[i, j] = sum over t of x^[t, i] dy[t, j].
 *
 * A CTA forms a 64 x 64 tile of dw, 16 tokens at a time through shared
 * memory, each thread 4 x 4 sums in fp32.
 */
#include "train.cuh"

namespace zw {

using namespace zt;

constexpr int kThreads = 256;
constexpr int kTile = 64;
constexpr int kStep = 16;

struct Args {
  const int8_t* q;
  const uint8_t* scale;
  const uint16_t* dy;
  uint16_t* dw;
  int64_t rows, cols, pitch, n, ld;
};

template <bool kBf16>
__global__ void __launch_bounds__(kThreads) wgrad_kernel(const Args a) {
  pdl_begin();
  __shared__ float xs[kStep][kTile], ys[kStep][kTile];
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kTile;
  const int64_t j0 = static_cast<int64_t>(blockIdx.y) * kTile;
  const int ti = threadIdx.x / 16, tj = threadIdx.x % 16;
  float sum[4][4] = {};
  for (int64_t t0 = 0; t0 < a.rows; t0 += kStep) {
    for (int k = threadIdx.x; k < kStep * kTile; k += kThreads) {
      const int64_t t = t0 + k / kTile, i = i0 + k % kTile, j = j0 + k % kTile;
      float x = 0.f, y = 0.f;
      if (t < a.rows && i < a.cols) {
        const uint32_t s = a.scale[t * (a.pitch / ZERO_CKPT_BLOCK) + i / ZERO_CKPT_BLOCK];
        x = static_cast<float>(a.q[t * a.pitch + i]) *
            (s == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float(s << 23));
      }
      if (t < a.rows && j < a.n) y = widen<kBf16>(a.dy[t * a.ld + j]);
      xs[k / kTile][k % kTile] = x;
      ys[k / kTile][k % kTile] = y;
    }
    __syncthreads();
    for (int k = 0; k < kStep; ++k) {
#pragma unroll
      for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          sum[p][q] = __fmaf_rn(xs[k][ti * 4 + p], ys[k][tj * 4 + q], sum[p][q]);
    }
    __syncthreads();
  }
  for (int p = 0; p < 4; ++p)
    for (int q = 0; q < 4; ++q) {
      const int64_t i = i0 + ti * 4 + p, j = j0 + tj * 4 + q;
      if (i < a.cols && j < a.n && ZCHECK(i * a.n + j < a.cols * a.n, kSiteStore, i))
        a.dw[i * a.n + j] = narrow<kBf16>(sum[p][q]);
    }
}

}  // namespace zw

#ifdef ZERO_CHECKED
extern "C" int zw_collect_checks(unsigned long long* count, unsigned long long* first) {
  return collect_checks(count, first);
}
#endif

extern "C" {

ZERO_API int zero_ckpt_wgrad(const void* ckpt, int64_t rows, int64_t cols, const void* dy,
                             int64_t n, int64_t ld, int32_t dtype, void* dw,
                             zero_scaler* d_scaler, void* stream) {
  using namespace zw;
  if (rows < 0 || cols < 0 || n < 0 || ld < n || !is_dtype16(dtype)) return ZERO_EINVAL;
  constexpr int64_t kMost = int64_t{1} << 31;
  if (rows >= kMost || cols >= kMost || n >= kMost) return ZERO_ERANGE;
  if (cols == 0 || n == 0) return ZERO_OK;
  if (!dw || (rows && (!ckpt || !dy))) return ZERO_EINVAL;
  if (!aligned(ckpt, 16) || !aligned(dy, 2) || !aligned(dw, 2) || !aligned(d_scaler, 16))
    return ZERO_EALIGN;
  Args a = {};
  a.q = static_cast<const int8_t*>(ckpt);
  a.pitch = ceil_div(cols, ZERO_CKPT_PAD) * ZERO_CKPT_PAD;
  a.scale = static_cast<const uint8_t*>(ckpt) + rows * a.pitch;
  a.dy = static_cast<const uint16_t*>(dy);
  a.dw = static_cast<uint16_t*>(dw);
  a.rows = rows, a.cols = cols, a.n = n, a.ld = ld;
  const dim3 grid(static_cast<unsigned>(ceil_div(cols, kTile)),
                  static_cast<unsigned>(ceil_div(n, kTile)));
  if (grid.y > 65535) return ZERO_ERANGE;
  return status_of(launch_pdl(dtype == ZERO_BF16 ? wgrad_kernel<true> : wgrad_kernel<false>, grid,
                              dim3(kThreads), 0, static_cast<cudaStream_t>(stream), a));
}

}  // extern "C"
