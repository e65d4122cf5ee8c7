/*
 * dropout.cu -- dropout whose mask is never stored (zero_block.h).
 *
 * A thread takes two times 8 neighbouring elements of a row, 8 of which share
 * one draw of the generator (draws.cuh); a warp 512 columns, the warps of a CTA
 * running on into the next row. Bound by memory with a residual (8192 x 8192
 * bf16, p = 0.25: 59 us, 100 % of copy bandwidth) and nearly so without (46 us,
 * 85 %; 39 without the generator, whose multiplications take the rest). One piece
 * per warp took 66 and 53. Off the 16-byte grid 92 and 71 (8192 x 8191), putting
 * vectors together on both sides.
 */
#include "draws.cuh"
#include "rows.cuh"

#include <algorithm>

namespace zd {

using namespace zt;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kPieces = 2;  // of 256 columns per warp

enum { kX, kResidual, kOut, kBuffers };  // a call's buffers, for their bounds

struct Args : Checked<kBuffers> {
  const uint16_t *x, *residual;
  uint16_t* out;
  int64_t rows, cols, ld, ld_out;
  uint32_t col_tiles;
  Drop drop;
};

template <bool kBf16, bool kGrid>
__global__ void __launch_bounds__(kThreads, kGrid ? 6 : 5) dropout_kernel(const Args a) {
  pdl_begin();
  __shared__ __align__(16) uint8_t stages[kGrid ? 1 : kWarps][kGrid ? 16 : kStageWarp];
  uint8_t* stage = stages[kGrid ? 0 : threadIdx.x >> 5];
  const int lane = threadIdx.x & 31;
  const uint32_t tile = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const uint32_t row = tile / a.col_tiles;
  const int64_t r = row;
  if (r >= a.rows) return;
  const int64_t c0 = static_cast<int64_t>(tile - row * a.col_tiles) * (kPieces * kCols);
  const uint32_t step = step_of(a.drop);
  uint4 vx[kPieces], vr[kPieces];
  const auto column = [&](int k) { return c0 + k * kCols + lane * kVec; };
  if constexpr (kGrid) {
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      vx[k] = load8<true>(a.x + r * a.ld, column(k), a.cols, a.bounds(kX));
      vr[k] = make_uint4(0, 0, 0, 0);
      if (a.residual)
        vr[k] = load8<true>(a.residual + r * a.ld_out, column(k), a.cols, a.bounds(kResidual));
    }
  } else {
    if (a.residual)
      load_all<false>(vr, [&](int) { return a.residual + r * a.ld_out; }, column, a.cols,
                      a.bounds(kResidual));
    load_all<false>(vx, [&](int) { return a.x + r * a.ld; }, column, a.cols, a.bounds(kX));
  }
#pragma unroll
  for (int k = 0; k < kPieces; ++k) {
    const int64_t c = c0 + k * kCols;
    if (c >= a.cols) break;
    float x[8], s[8];
    widen8<kBf16>(vx[k], x);
    if (a.drop.threshold)
      drop8(a.drop, draw8(a.drop, step, row, static_cast<uint32_t>(c >> 3) + lane), x);
    if (a.residual) {
      widen8<kBf16>(vr[k], s);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] += s[j];
    }
    store_row<kGrid>(stage, a.out + r * a.ld_out, c, lane, a.cols, narrow8<kBf16>(x),
                     a.bounds(kOut));
  }
}

}  // namespace zd

#ifdef ZERO_CHECKED
extern "C" int zd_collect_checks(unsigned long long* count, unsigned long long* first) {
  return collect_checks(count, first);
}
#endif

extern "C" ZERO_API int zero_dropout(const zero_dropout_params* params, const void* x,
                                     const void* residual, int64_t rows, int64_t cols, int64_t ld,
                                     int32_t dtype, void* out, int64_t ld_out, void* stream) {
  using namespace zd;
  if (!params || rows < 0 || cols < 0 || ld < cols || ld_out < cols || !is_dtype16(dtype))
    return ZERO_EINVAL;
  if (const int bad = check_drop(*params)) return bad;
  constexpr int64_t kMost = int64_t{1} << 31;
  if (rows >= kMost || cols >= kMost || rows * ceil_div(cols, kCols) >= kMost) return ZERO_ERANGE;
  const bool grid = on_grid(x, ld) && on_grid(out, ld_out) && aligned(residual, 16);
  const int64_t col_tiles = ceil_div(cols, kPieces * kCols);
  if (rows == 0 || cols == 0) return ZERO_OK;
  if (!x || !out || (x == out && ld != ld_out)) return ZERO_EINVAL;
  if (!aligned(x, 2) || !aligned(residual, 2) || !aligned(out, 2)) return ZERO_EALIGN;
  Args a = new_args<Args>();
  a.x = static_cast<const uint16_t*>(x);
  a.residual = static_cast<const uint16_t*>(residual);
  a.out = static_cast<uint16_t*>(out);
  a.rows = rows, a.cols = cols, a.ld = ld, a.ld_out = ld_out;
  a.col_tiles = static_cast<uint32_t>(col_tiles);
  a.drop = drop_of(*params);
  a.set_bounds(kX, x, rows, cols, ld, 2);
  a.set_bounds(kResidual, residual, rows, cols, ld_out, 2);
  a.set_bounds(kOut, out, rows, cols, ld_out, 2);
  const auto fn = dtype == ZERO_BF16
                      ? (grid ? dropout_kernel<true, true> : dropout_kernel<true, false>)
                      : (grid ? dropout_kernel<false, true> : dropout_kernel<false, false>);
  return status_of(launch_pdl(fn, dim3(static_cast<unsigned>(ceil_div(rows * col_tiles, kWarps))),
                              dim3(kThreads), 0, static_cast<cudaStream_t>(stream), a));
}
