// rows.cuh -- a warp's part of a row of 16-bit elements, at any alignment:
// 256 neighbouring columns, eight per lane.
#ifndef ZERO_ROWS_CUH
#define ZERO_ROWS_CUH

#include "train.cuh"

namespace zt {

constexpr int kCols = 32 * kVec;

// Eight elements of a row of 16-bit elements starting at column c; those at
// or past `cols` are 0. kGrid: rows lie on the 16-byte grid.
template <bool kGrid>
__device__ __forceinline__ uint4 load8(const uint16_t* row, int64_t c, int64_t cols,
                                       const Bounds& in) {
  if (!in.holds(row + c, 2 * (cols - c < kVec ? cols - c : kVec), kSiteLoad))
    return make_uint4(0, 0, 0, 0);
  if (c + kVec <= cols)
    return kGrid ? __ldcs(reinterpret_cast<const uint4*>(row + c)) : load8_any<true>(row + c);
  uint32_t h[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) h[j] = c + j < cols ? row[c + j] : 0;
  return make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
}

// The same in two steps, so that several loads off the grid are under way
// together: the one or two 16-byte blocks that hold the elements, then the
// elements. All lanes of the warp take vectors of one row.
struct Blocks {
  uint4 x, y;
  int distance, count;
};

__device__ __forceinline__ Blocks load_blocks(const uint16_t* row, int64_t c, int64_t cols,
                                              const Bounds& in) {
  Blocks b;
  const uintptr_t at = reinterpret_cast<uintptr_t>(row + c);
  const uint4* block = reinterpret_cast<const uint4*>(at & ~static_cast<uintptr_t>(15));
  b.distance = static_cast<int>(at & 15);
  b.count = c < cols ? static_cast<int>(cols - c < kVec ? cols - c : kVec) : 0;
  b.x = b.y = make_uint4(0, 0, 0, 0);
  if (b.count > 0 && in.holds_blocks(block, 16, kSiteLoad)) b.x = block[0];
  if (b.distance + 2 * b.count > 16 && in.holds_blocks(block + 1, 16, kSiteLoad)) b.y = block[1];
  return b;
}

// the first `there` of eight elements, the others 0
__device__ __forceinline__ uint4 first_of(uint4 v, int there) {
  if (there >= kVec) return v;
  const uint32_t low = 0xFFFFu;
  v.x = there > 1 ? v.x : there == 1 ? v.x & low : 0;
  v.y = there > 3 ? v.y : there == 3 ? v.y & low : 0;
  v.z = there > 5 ? v.z : there == 5 ? v.z & low : 0;
  v.w = there == 7 ? v.w & low : 0;
  return v;
}

__device__ __forceinline__ uint4 eight_of(const Blocks& b) {
  return first_of(shifted_alike(b.x, b.y, b.distance), b.count);
}

// kCount vectors of eight, by a grid's rows or off it; row(k), column(k)
template <bool kGrid, int kCount, class Row, class Column>
__device__ __forceinline__ void load_all(uint4 (&v)[kCount], Row row, Column column, int64_t cols,
                                         const Bounds& in) {
  if constexpr (kGrid) {
#pragma unroll
    for (int k = 0; k < kCount; ++k) v[k] = load8<true>(row(k), column(k), cols, in);
  } else {
    Blocks b[kCount];
#pragma unroll
    for (int k = 0; k < kCount; ++k) b[k] = load_blocks(row(k), column(k), cols, in);
#pragma unroll
    for (int k = 0; k < kCount; ++k) v[k] = eight_of(b[k]);
  }
}

// A warp's 256 columns of a row from c0 on, those before `cols`; all lanes
// call it.
template <bool kGrid>
__device__ __forceinline__ void store_row(uint8_t* stage, uint16_t* row, int64_t c0, int lane,
                                          int64_t cols, const uint4& v, const Bounds& in) {
  const int64_t c = c0 + lane * kVec;
  if constexpr (kGrid) {
    if (!in.holds(row + c, 2 * (cols - c < kVec ? cols - c : kVec), kSiteStore)) return;
    if (c + kVec <= cols) {
      __stcs(reinterpret_cast<uint4*>(row + c), v);
      return;
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j < cols) row[c + j] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
  } else {
    const int64_t left = cols - c0;
    if (left > 0)
      store_any(stage, row + c0, left < kCols ? static_cast<int>(left) : kCols, lane, v, in);
  }
}

// Two 16-bit magnitudes at once: as integers they are ordered like the values,
// infinity and NaN above all numbers.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// whether every row start of a [.., ld] array of 16-bit elements lies on the
// 16-byte grid
inline bool on_grid(const void* p, int64_t ld) { return aligned(p, 16) && ld % 8 == 0; }

}  // namespace zt

#endif
