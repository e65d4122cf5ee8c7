/*
 * fp8.cu -- linear layers in 8-bit floating point with one power-of-two scale
 * per block of 128 (zero_block.h): the 8-bit copies, and the products that read
 * them on the 5th-generation tensor cores.
 *
 * Copies. With m the block's largest magnitude and 1.75 2^t the format's
 * largest number, 2^k is m's power of two over 2^t, one more where m's mantissa
 * passes 1.75; x / 2^k is exact, its rounding to the format the only one. The
 * scale bytes are the tensor cores' own scale type (UE8M0) and lie in the tiles
 * that go to tensor memory as they are: 128 rows by four blocks, 512 bytes.
 *
 * Products. out[i, j] = sum over b of 2^(ka + kb) sum of a[i, .] b[., j] over
 * block b of the reduction; the tensor core applies both scales, so the sums
 * stay in tensor memory (fp32) from the first block to the last. (With scales
 * that are not powers of two every block's sums would have to be read back and
 * scaled in registers.) A weight's copy serves both directions: x W reduces over
 * its rows (the operand's slow axis), dy W^T over its columns.
 *
 * A pair of CTAs (one tcgen05.mma over two SMs) forms a tile of 256 rows by up
 * to 256 columns, 128 reduction steps at a time: each CTA brings 128 rows of
 * the left operand, half of the right one and the scale tiles through a ring of
 * stages. Warps by role: copies, products, four for the output, which read a
 * finished tile while the next one's sums form elsewhere in tensor memory. Two
 * tiles of 256 columns and the scales do not fit there, so that two such tiles
 * share 32 columns: those are read first, and the next tile's products wait for
 * them alone.
 *
 * One lane issues, but the whole warp with it (at copy_box2). 8192 x 2048 x 8192
 * takes 83 us for x W and 84 for dy W^T (3.3 PFLOP/s; 8192^3 305 to 312 us, 3.6).
 * Time is cycles over a clock that power holds down: 159,000 cycles each way
 * on random numbers as on zeros, 97 us at 1.63 GHz after seconds on end and 77 at
 * the full 2.07 (8192^3: 506,000 at 1.39 GHz, 537,000 at 2.07). The tensor cores
 * are busy for 110,000 of them (72 and 70 %; 8192^3 87 %). At 2.07 GHz a block costs
 * 562 cycles, 512 of them products, and each of the 14 turns of tiles 2,400 more, for
 * its start and end, the pairs without a tile in the last turn and the launch; dy W^T
 * has 3.4 turns' tiles in four. The right operand brought for two pairs at once by
 * multicast was no faster (84 to 86; 322).
 *
 * Few tiles and a long reduction: a cluster of 2, 4 or 8 pairs shares a tile,
 * each pair a part of the reduction; the sums meet in shared memory and every
 * CTA adds its share of the rows over the cluster in rank order. Split and tile
 * width depend on the sizes and the device alone.
 *
 * Every wait is bounded (2 s); one that expires ends the work of its cluster,
 * whose tiles left become NaN, and raises the scaler's error word.
 */
#include "rows.cuh"
#include "tensor.cuh"
#include "zero_block.h"

#include <algorithm>
#include <atomic>

namespace zf {

using namespace zt;

constexpr int kBlock = ZERO_FP8_BLOCK;
constexpr int kTileBytes = 512;  // scales of 128 rows x 4 blocks

int64_t blocks_of(int64_t n) { return ceil_div(n, kBlock); }
int64_t groups_of(int64_t n) { return ceil_div(n, 4 * kBlock); }

// ------------------------------------------------------------------ copies ----

__device__ __forceinline__ int64_t scale_at(uint32_t row, uint32_t block, uint32_t groups) {
  return (static_cast<int64_t>(row / 128) * groups + block / 4) * kTileBytes +
         (16 * (row % 32) + 4 * (row % 128 / 32) + block % 4);
}

// The scale byte of a block from its largest magnitude (16-bit pattern).
template <bool kBf16>
__device__ __forceinline__ uint32_t scale_of(uint32_t top, int32_t format) {
  if (top >= (kBf16 ? 0x7F80u : 0x7C00u)) return 255;
  if (top == 0) return 127;
  const uint32_t bits = __float_as_uint(widen<kBf16>(top));
  const int k = static_cast<int>(bits >> 23) - (format == ZERO_E4M3 ? 8 : 15) +
                ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return max(k, 1);
}

// Eight elements over 2^k, to the format (ties to even); NaN where the block is
// not finite.
template <bool kBf16>
__device__ __forceinline__ uint2 narrow_fp8(const uint4& v, uint32_t scale, int32_t format) {
  if (scale == 255) return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
  const float inv = __uint_as_float((254 - scale) << 23);
  float f[8];
  widen8<kBf16>(v, f);
  uint32_t h[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint16_t w;
    const float a = f[2 * j] * inv, b = f[2 * j + 1] * inv;
    if (format == ZERO_E4M3)
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(w) : "f"(b), "f"(a));
    else
      asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(w) : "f"(b), "f"(a));
    h[j] = w;
  }
  return make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
}

__device__ __forceinline__ uint32_t top_of(const uint4& v) {
  constexpr uint32_t kAbs = 0x7FFF7FFFu;
  return max_u16x2(max_u16x2(v.x & kAbs, v.y & kAbs), max_u16x2(v.z & kAbs, v.w & kAbs));
}

enum { kX, kCopy, kQuantBuffers };

struct QuantArgs : Checked<kQuantBuffers> {
  const uint16_t* x;
  uint8_t *q, *scale, *scale_t;  // scale_t: a weight's second set
  int64_t rows, cols, pitch, ld;
  uint32_t col_tiles;
  int32_t format;
};

constexpr int kQuantWarps = 8;

// A warp takes 512 columns of a row, 16 a lane and so eight lanes a block: 32
// bytes in flight per thread (8192 x 8192: 46 us with 8 columns a lane).
constexpr int kQuantCols = 512;

template <bool kBf16, bool kGrid>
__global__ void __launch_bounds__(32 * kQuantWarps) quant_kernel(const QuantArgs a) {
  pdl_begin();
  const int lane = threadIdx.x & 31;
  const uint32_t tile = blockIdx.x * kQuantWarps + (threadIdx.x >> 5);
  const uint32_t row = tile / a.col_tiles;
  const int64_t r = row;
  if (r >= a.rows) return;
  const int64_t c = static_cast<int64_t>(tile - row * a.col_tiles) * kQuantCols + lane * 16;
  uint4 v[2];
  load_all<kGrid>(v, [&](int) { return a.x + r * a.ld; }, [&](int k) { return c + 8 * k; }, a.cols,
                  a.bounds(kX));
  uint32_t top = max_u16x2(top_of(v[0]), top_of(v[1]));
#pragma unroll
  for (int d = 1; d < 8; d *= 2) top = max_u16x2(top, __shfl_xor_sync(0xffffffffu, top, d));
  top = max(top & 0xFFFFu, top >> 16);
  if (c >= a.pitch) return;
  const uint32_t scale = scale_of<kBf16>(top, a.format);
  uint8_t* q = a.q + r * a.pitch + c;
  if (a.bounds(kCopy).holds(q, 16, kSiteStore)) {
    const uint2 lo = narrow_fp8<kBf16>(v[0], scale, a.format);
    const uint2 hi = narrow_fp8<kBf16>(v[1], scale, a.format);
    *reinterpret_cast<uint4*>(q) = make_uint4(lo.x, lo.y, hi.x, hi.y);
    // NaN, but past the last column zeros as everywhere. A loop that stays one, for 32
    // registers: with 34 a CTA less fits (8192 x 8191 41 us, 38 so)
    if (scale == 255) {
#pragma unroll 1
      for (int64_t j = max(c, a.cols); j < c + 16; ++j) a.q[r * a.pitch + j] = 0;
    }
  }
  if ((lane & 7) == 0) {
    uint8_t* s = a.scale + scale_at(row, static_cast<uint32_t>(c) / kBlock,
                                    static_cast<uint32_t>(a.pitch + 4 * kBlock - 1) / (4 * kBlock));
    if (a.bounds(kCopy).holds(s, 1, kSiteStore)) *s = static_cast<uint8_t>(scale);
  }
}

// A CTA takes two neighbouring 128 x 128 blocks of a weight, a warp 16 rows of
// 256 columns in registers, so that it is read once and in runs of 512 bytes.
// (Single blocks, runs of 256 bytes: 2048 x 8192 15 us.)
constexpr int kWeightRows = 16;

template <bool kBf16, bool kGrid>
__global__ void __launch_bounds__(256) quant_weight_kernel(const QuantArgs a) {
  pdl_begin();
  __shared__ uint32_t tops[2][8];
  const int64_t kb = blockIdx.x / a.col_tiles, nt = blockIdx.x - kb * a.col_tiles;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, side = lane >> 4;
  const int64_t c = nt * kCols + lane * kVec, r0 = kb * kBlock + warp * kWeightRows;
  uint4 v[kWeightRows];
  uint32_t top = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {  // two halves: off the grid a row takes twice the registers
    uint4 w[kWeightRows / 2];
    const auto row = [&](int i) { return r0 + h * (kWeightRows / 2) + i; };
    load_all<kGrid>(w, [&](int i) { return a.x + row(i) * a.cols; },
                    [&](int i) { return row(i) < a.rows ? c : a.cols; }, a.cols, a.bounds(kX));
#pragma unroll
    for (int i = 0; i < kWeightRows / 2; ++i) v[h * (kWeightRows / 2) + i] = w[i];
  }
#pragma unroll
  for (int i = 0; i < kWeightRows; ++i) top = max_u16x2(top, top_of(v[i]));
#pragma unroll
  for (int d = 1; d < 16; d *= 2) top = max_u16x2(top, __shfl_xor_sync(0xffffffffu, top, d));
  if ((lane & 15) == 0) tops[side][warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) top = max_u16x2(top, tops[side][w]);
  const uint32_t scale = scale_of<kBf16>(max(top & 0xFFFFu, top >> 16), ZERO_E4M3);
  // zeros past the last column, also where the block is not finite
  const int64_t left = a.cols - c;
  const uint64_t all = ~0ull, bits = left >= kVec ? all : left > 0 ? all >> (8 * (kVec - left)) : 0;
  const uint2 columns = make_uint2(static_cast<uint32_t>(bits), static_cast<uint32_t>(bits >> 32));
#pragma unroll
  for (int i = 0; i < kWeightRows; ++i) {
    uint8_t* q = a.q + (r0 + i) * a.pitch + c;
    const uint2 n = narrow_fp8<kBf16>(v[i], scale, ZERO_E4M3);
    if (r0 + i < a.rows && c < a.pitch && a.bounds(kCopy).holds(q, kVec, kSiteStore))
      *reinterpret_cast<uint2*>(q) = make_uint2(n.x & columns.x, n.y & columns.y);
  }
  // the scale of each of a block's 128 columns and rows
  const int64_t nb = 2 * nt + side;
  if (nb * kBlock >= a.cols) return;
  const int m = warp * 16 + (lane & 15);
  uint8_t* by_column = a.scale + scale_at(nb * 128 + m, kb, (a.rows + 511) / 512);
  uint8_t* by_row = a.scale_t + scale_at(kb * 128 + m, nb, (a.cols + 511) / 512);
  if (a.bounds(kCopy).holds(by_column, 1, kSiteStore)) *by_column = static_cast<uint8_t>(scale);
  if (a.bounds(kCopy).holds(by_row, 1, kSiteStore)) *by_row = static_cast<uint8_t>(scale);
}

// ---------------------------------------------------------------- products ----

constexpr int kM = 128, kN = 256, kK = kBlock;  // rows per CTA, columns at most, steps per stage
constexpr int kOutWarps = 4;
constexpr int kCopyWarp = 0, kProductWarp = 1, kOutWarp0 = 2, kWarps = kOutWarp0 + kOutWarps;
constexpr int kThreads = 32 * kWarps;
constexpr int kBytesA = kM * kK, kBytesB = kK * 128, kScaleTiles = 2;  // of the right operand
constexpr int kBytesScales = 2048;
constexpr int kStageBytes = kBytesA + kBytesB + kBytesScales, kStages = 6;
constexpr int kRing = kStages * kStageBytes;
constexpr int kOutBytes = 5 * 1024;  // an output warp's stage: 32 rows of 64 columns
constexpr int kSmem = kRing + kOutWarps * kOutBytes + 1024;
constexpr int kJoinPitch = kN + 4;  // fp32 row of a tile in shared memory
constexpr int kMaxSplit = 8, kJoinAhead = 4;
// tensor memory: two tiles' sums, the second from kSecond on, then scales in two
// sets of 16 columns (4 of the left operand, up to 8 of the right one). Copies of
// scales and products run in the order in which one thread issues them, so that a
// set is not written before the products that were to read it.
constexpr int kTensorColumns = 512, kSecond = 224, kScaleColumn = 480, kScaleSets = 2;
static_assert(kSecond + kN <= kScaleColumn && kN - kSecond == 32, "the tiles share 32 columns");
static_assert(kScaleColumn + 16 * kScaleSets <= kTensorColumns, "tensor memory");
static_assert(32 * kOutPitch <= kOutBytes && 32 * 128 <= kOutBytes, "output stage");
static_assert((1 + kScaleTiles) * kTileBytes <= kBytesScales && kStageBytes % 1024 == 0, "stages");
static_assert(kM * kJoinPitch * 4 <= kRing, "the tile fits the stages");
// costs in cycles: a block, and its thirds per column (128, 192 and 256 columns
// took 484, 595 to 625 and 661 to 717 at 8192 x 2048 x 8192 and 8192^3, what a tile
// costs beside its blocks shared out among them; the products alone are 256, 384
// and 512); a column put out; the join of a split, by rows per
// warp (600 x 512 x 512 4.8 us, split in two 10.1; 16 x 8192 x 256 16 us, split in
// two, four and eight 11.4, 8.0 and 7.2); clusters of 16 CTAs
constexpr int kBlockCycles = 340, kColumnThirds = 4;
constexpr int kOutCycles = 14, kJoinCycles = 1500, kJoinRowCycles = 900, kBigClusterCycles = 4000;

enum { kOut, kBuffers };

struct Args : Checked<kBuffers> {
  uint16_t* out;
  zero_scaler* scaler;
  int64_t rows, n, ld;
  int32_t blocks;  // of the reduction
  int32_t split, tma_out, bn, m_tiles, tiles, scale_tiles, a_format;
};

struct Maps {
  CUtensorMap a, b, scale_a, scale_b, out;
};

// What one lane starts (copies, products, commits) is issued by the whole warp
// with one lane elected in the instruction itself: the operands then are the
// warp's, in uniform registers. Behind a branch on the lane each operand goes
// there lane by lane, and the issuing thread, not the tensor core, is the bound
// (four products of 256 x 192 x 32 and their commit took 413 cycles, 384 so).
__device__ __forceinline__ void copy_box2(void* dst, const CUtensorMap* map, int32_t x, int32_t y,
                                          uint32_t cluster_bar) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%2, %3}], [%4];\n}" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(cluster_bar)
      : "memory");
}

__device__ __forceinline__ void copy_box3(void* dst, const CUtensorMap* map, int32_t x, int32_t y,
                                          int32_t z, uint32_t cluster_bar) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%2, %3, %4}], [%5];\n}" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(cluster_bar)
      : "memory");
}

__device__ __forceinline__ void expect_bytes(uint64_t* bar, uint32_t bytes) {
  asm volatile(
      "{\n .reg .pred e;\n .reg .b64 st;\n elect.sync _|e, 0xffffffff;\n"
      " @e mbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n}" ::"r"(smem_u32(bar)),
      "r"(bytes)
      : "memory");
}

// arrive at `bar` of both CTAs of the pair once the products issued so far are done
__device__ __forceinline__ void commit_pair(uint64_t* bar, uint16_t pair_mask) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster"
      ".b64 [%0], %1;\n}" ::"r"(smem_u32(bar)),
      "h"(pair_mask)
      : "memory");
}

// the stage's 32 rows of 64 columns to the output; rows and columns past its
// ends stay away
__device__ __forceinline__ void store_box(const CUtensorMap* map, const void* src, int32_t x,
                                          int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];\n"
      "cp.async.bulk.commit_group;" ::"l"(map),
      "r"(smem_u32(src)), "r"(x), "r"(y)
      : "memory");
}

// the warp waits together and has one verdict
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* failed,
                                          uint64_t limit) {
  return __all_sync(0xffffffffu, bar_wait(bar, parity, failed, limit));
}

// Shared-memory operands with 128-byte swizzle: rows of 128 bytes, eight rows
// per 1024-byte atom. The reduction runs along the rows (32 steps are 32 bytes
// on) or, for a weight's slow axis, over them (32 steps are 4096 bytes on).
constexpr uint32_t kOperandHigh = (1024 >> 4) | 1u << 14 | 2u << 29;
// scale tiles: 32 rows of 16 bytes, eight rows per 128 bytes
constexpr uint32_t kScaleHigh = (128 >> 4) | 1u << 14;

__device__ __forceinline__ uint32_t operand_low(uint32_t addr) {
  return (addr & 0x3FFFF) >> 4 | 1u << 16;
}

__device__ __forceinline__ uint32_t scale_low(uint32_t addr) {
  return (addr & 0x3FFFF) >> 4 | static_cast<uint32_t>(128 >> 4) << 16;
}

// fp32 sums of 256 x bn, UE8M0 scales; `slow`: the right operand's slow axis
// is reduced. The block's scales are byte `b` of their words.
__device__ __forceinline__ uint32_t product_desc(int a_format, bool slow, int bn) {
  return static_cast<uint32_t>(a_format) << 7 | (slow ? 1u << 16 : 0u) |
         static_cast<uint32_t>(bn >> 3) << 17 | 1u << 23 | static_cast<uint32_t>(2 * kM >> 4) << 24;
}

__device__ __forceinline__ void product(uint32_t d, uint32_t a_low, uint32_t b_low, uint32_t desc,
                                        uint32_t scale_a, uint32_t scale_b, uint32_t add) {
  asm volatile(
      "{\n .reg .pred p, e;\n .reg .b64 da, db;\n setp.ne.b32 p, %4, 0;\n"
      " elect.sync _|e, 0xffffffff;\n"
      " mov.b64 da, {%1, %5};\n mov.b64 db, {%2, %5};\n"
      " @e tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], da, db, %3, "
      "[%6], [%7], p;\n}" ::"r"(d),
      "r"(a_low), "r"(b_low), "r"(desc), "r"(add), "r"(kOperandHigh), "r"(scale_a), "r"(scale_b)
      : "memory");
}

// a scale tile of each CTA of the pair into its tensor memory, all four quarters
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint32_t low) {
  asm volatile(
      "{\n .reg .pred e;\n .reg .b64 s;\n elect.sync _|e, 0xffffffff;\n mov.b64 s, {%1, %2};\n"
      " @e tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], s;\n}" ::"r"(tmem),
      "r"(low), "r"(kScaleHigh)
      : "memory");
}

// kSlow: the right operand's reduction axis is its slow one (x W).
template <bool kBf16, bool kSlow>
__global__ void __launch_bounds__(kThreads, 1)
    product_kernel(const __grid_constant__ Maps maps, const Args a) {
  extern __shared__ uint8_t raw[];
  uint8_t* stages = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  // full: in the pair's first CTA, counted by both; empty and done: in each
  __shared__ uint64_t full[kStages], empty[kStages], done[2], freed[2];
  __shared__ uint32_t tmem_base;
  __shared__ int failed;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // the warp's, not the lane's
  const uint64_t limit = a.limit();
  const int n_cta = 2 * a.split;
  const int rank = static_cast<int>(blockIdx.x) % n_cta;
  const int half = rank & 1, part = rank >> 1, leader = rank & ~1;
  const int tile0 = static_cast<int>(blockIdx.x) / n_cta;
  const int tile_stride = static_cast<int>(gridDim.x) / n_cta;
  const int my_tiles = tile0 < a.tiles ? (a.tiles - tile0 + tile_stride - 1) / tile_stride : 0;
  // this pair's blocks of the reduction
  const int s0 = static_cast<int>(static_cast<int64_t>(a.blocks) * part / a.split);
  const int s1 = static_cast<int>(static_cast<int64_t>(a.blocks) * (part + 1) / a.split);
  const auto row_of = [&](int tile) {  // first row of this CTA's part of the tile
    return static_cast<int64_t>(tile % a.m_tiles) * (2 * kM) + half * kM;
  };
  const auto column_of = [&](int tile) { return static_cast<int64_t>(tile / a.m_tiles) * a.bn; };
  const bool shared_columns = a.bn > kSecond;

  if (warp == kProductWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&tmem_base)),
                 "n"(kTensorColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      bar_init(&full[s], 1);
      bar_init(&empty[s], 1);
    }
    for (int k = 0; k < 2; ++k) {
      bar_init(&done[k], 1);
      bar_init(&freed[k], 2 * kOutWarps);
    }
    failed = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  cluster_sync();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = tmem_base;
  // all up to here touches only this cluster's own memory and may run beside
  // the kernel before this one
  pdl_begin();

  if (warp == kCopyWarp) {
    const uint32_t full_at = in_cta(full, leader);
    const int b_rows = kSlow ? kK : a.bn / 2;
    const uint32_t bytes = 2 * (kBytesA + b_rows * 128);
    const uint32_t scale_bytes = 2 * (1 + a.scale_tiles) * kTileBytes;
    Ring<kStages> ring;
    bool ok = true;
    int left_fresh = kStages;
    for (int k = 0; k < my_tiles && ok; ++k) {
      const int tile = tile0 + k * tile_stride;
      const int32_t i = static_cast<int32_t>(row_of(tile));
      const int32_t j = static_cast<int32_t>(column_of(tile));
      const int32_t jb = j + half * (a.bn / 2);
      for (int b = s0; b < s1; ++b) {
        const int s = ring.stage;
        if (left_fresh > 0) --left_fresh;
        else if (!warp_wait(&empty[s], ring.parity ^ 1, &failed, limit)) {
          ok = false;
          break;
        }
        if (blockIdx.x == 0 &&
            a.holds(ZERO_PLANT_NO_COPY, static_cast<int64_t>(k) * (s1 - s0) + b - s0)) {
          ring.advance(1);
          continue;
        }
        uint8_t* to = stages + s * kStageBytes;
        const bool scales = b == s0 || b % 4 == 0;
        if (half == 0) expect_bytes(&full[s], bytes + (scales ? scale_bytes : 0));
        const uint32_t bar = full_at + s * 8;
        copy_box2(to, &maps.a, b * kK, i, bar);
        if (kSlow) copy_box2(to + kBytesA, &maps.b, jb, b * kK, bar);
        else copy_box2(to + kBytesA, &maps.b, b * kK, jb, bar);
        if (scales) {
          copy_box3(to + kBytesA + kBytesB, &maps.scale_a, 0, b / 4, i / 128, bar);
          copy_box3(to + kBytesA + kBytesB + kTileBytes, &maps.scale_b, 0, b / 4, j / 128, bar);
        }
        ring.advance(1);
      }
    }
  } else if (warp == kProductWarp) {
    if (half == 0) {
      const uint16_t pair_mask = static_cast<uint16_t>(3u << leader);
      const uint32_t desc = product_desc(a.a_format, kSlow, a.bn);
      const uint32_t at0 = smem_u32(stages);
      constexpr uint32_t kNextA = 32 >> 4, kNextB = kSlow ? 32 * 128 >> 4 : 32 >> 4;
      Ring<kStages> ring;
      bool ok = true;
      uint32_t set = 0;
      for (int k = 0; k < my_tiles && ok && s1 > s0; ++k) {
        const int buf = k & 1;
        const uint32_t sums = tmem + buf * kSecond;
        // where in its scale tile the first column's scales are: a tensor memory
        // column per 32 of them
        const uint32_t shift =
            static_cast<uint32_t>(column_of(tile0 + k * tile_stride) % 128) / 32;
        // the tile before the last one is read whole or, where it is not in the
        // way, the last one's shared columns are (and with them all of that)
        const int after = k - (shared_columns ? 1 : 2);
        ok = after < 0 || warp_wait(&freed[after & 1], (after >> 1) & 1, &failed, limit);
        uint32_t scales = 0;
        for (int b = s0; b < s1 && ok; ++b) {
          const int s = ring.stage;
          ok = warp_wait(&full[s], ring.parity, &failed, limit);
          if (!ok) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint32_t at = at0 + s * kStageBytes;
          if (b == s0 || b % 4 == 0) {
            scales = tmem + kScaleColumn + 16 * set;
            set = (set + 1) % kScaleSets;
            const uint32_t low = scale_low(at + kBytesA + kBytesB);
            for (int t = 0; t <= a.scale_tiles; ++t)
              copy_scales(scales + 4 * t, low + t * (kTileBytes >> 4));
          }
          const uint32_t low_a = operand_low(at), low_b = operand_low(at + kBytesA);
          const uint32_t id = static_cast<uint32_t>(b % 4);
#pragma unroll
          for (int q = 0; q < kK / 32; ++q)
            product(sums, low_a + q * kNextA, low_b + q * kNextB, desc | id << 4 | id << 29, scales,
                    scales + 4 + shift, q > 0 || b > s0 ? 1u : 0u);
          commit_pair(&empty[s], pair_mask);
          ring.advance(1);
        }
        if (ok) commit_pair(&done[buf], pair_mask);  // whole sums only
      }
    }
  } else {
    // this warp's quarter of tensor memory's lanes
    const int row0 = (warp & 3) * 32;
    uint8_t* stage = stages + kRing + (warp - kOutWarp0) * kOutBytes;
    const int chunks = a.bn / kOutCols;
    bool ok = true;
    for (int k = 0; k < my_tiles; ++k) {
      const int tile = tile0 + k * tile_stride;
      const int buf = k & 1, use = k >> 1;
      if (s1 > s0 && ok) ok = warp_wait(&done[buf], use & 1, &failed, limit);
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t sums = tmem + (static_cast<uint32_t>(row0) << 16) + buf * kSecond;
      const int64_t i0 = row_of(tile) + row0, j = column_of(tile);
      // given up: the sums stay taken, others may still read theirs
      const auto free_sums = [&]() {
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (ok && lane == 0) bar_arrive_at(in_cta(&freed[buf], leader));
      };
#pragma unroll 1
      for (int m = 0; m < chunks; ++m) {
        // the first tile's shared columns are its last ones
        const int c = (!shared_columns || buf ? m : (m ? m - 1 : chunks - 1)) * kOutCols;
        float f[2][32];
        if (ok && s1 > s0) {
          read_sums(sums + c, f[0]);
          read_sums(sums + c + 32, f[1]);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) f[0][e] = f[1][e] = ok ? 0.f : __uint_as_float(0x7FC00000u);
        }
        // the eight columns before, for stores off the grid
        float before[8] = {f[0][0], f[0][0], f[0][0], f[0][0], f[0][0], f[0][0], f[0][0], f[0][0]};
        if (!a.tma_out && a.split == 1 && c && ok) read_eight(sums + c - 8, before);
        if (m == (shared_columns ? 0 : chunks - 1)) free_sums();
        if (a.split > 1) {
          float4* p = reinterpret_cast<float4*>(
              reinterpret_cast<float*>(stages) + (row0 + lane) * kJoinPitch + c);
#pragma unroll
          for (int e = 0; e < 16; ++e)
            p[e] = make_float4(f[e / 8][4 * e % 32], f[e / 8][4 * e % 32 + 1],
                               f[e / 8][4 * e % 32 + 2], f[e / 8][4 * e % 32 + 3]);
          continue;
        }
        uint4 v[2][4];
        narrow32<kBf16>(f[0], v[0]);
        narrow32<kBf16>(f[1], v[1]);
        if (a.tma_out) {
          // the store before has read the stage
          if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          __syncwarp();
          uint4* row = reinterpret_cast<uint4*>(stage + lane * 128);
#pragma unroll
          for (int e = 0; e < 8; ++e) row[e ^ (lane & 7)] = v[e / 4][e % 4];
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0 && i0 < a.rows && j + c < a.n)
            store_box(&maps.out, stage, static_cast<int32_t>(j + c), static_cast<int32_t>(i0));
        } else if (j + c < a.n) {
          uint16_t* to = a.out + i0 * a.ld + j;  // the tile's columns of this warp's first row
          uint4* row = reinterpret_cast<uint4*>(stage + lane * kOutPitch);
          const int count = static_cast<int>(min(a.n - j, static_cast<int64_t>(a.bn)));
          row[0] = narrow8<kBf16>(before);
#pragma unroll
          for (int e = 0; e < 8; ++e) row[1 + e] = v[e / 4][e % 4];
          __syncwarp();
          store_staged<4>(stage, to, a.ld, a.rows - i0, c, kOutCols, count, lane, a.bounds(kOut));
          __syncwarp();
        }
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  __syncthreads();
  cluster_sync();
  // no thread of the cluster starts a copy or a product any more, and all its
  // CTAs know if one gave up
  const bool gave_up = *static_cast<volatile int*>(&failed) != 0;
  if (gave_up) {
    drain();
    if (tid == 0 && a.scaler) atomicCAS(&a.scaler->error, 0, ZERO_DEVERR_TIMEOUT);
  }
  if (a.split > 1) {
    // one tile per cluster: this CTA's share of its rows, a warp per row and
    // eight columns per lane
    const float* tile_sums = reinterpret_cast<const float*>(stages);
    const int share = kM / a.split;
    const int64_t j = column_of(tile0);
    // the output warps' stages as one, a row's worth for each warp
    uint8_t* stage = stages + kRing + warp * ((kStageWarp + 15) & ~15);
    for (int m = warp; m < share; m += kWarps) {
      // rows dealt out in turn, so that a short tile's are shared too
      const int row = m * a.split + part;
      const int64_t i = row_of(tile0) + row;
      if (i >= a.rows) break;
      float f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (lane * 8 < a.bn) {
        for (int k0 = 0; k0 < a.split; k0 += kJoinAhead) {
          float4 x[kJoinAhead], y[kJoinAhead];
#pragma unroll
          for (int k = 0; k < kJoinAhead; ++k) {
            if (k0 + k >= a.split) break;
            const uint32_t remote =
                in_cta(tile_sums + row * kJoinPitch + lane * 8, 2 * (k0 + k) + half);
            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(x[k].x), "=f"(x[k].y), "=f"(x[k].z), "=f"(x[k].w)
                         : "r"(remote));
            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(y[k].x), "=f"(y[k].y), "=f"(y[k].z), "=f"(y[k].w)
                         : "r"(remote + 16));
          }
#pragma unroll
          for (int k = 0; k < kJoinAhead; ++k) {
            if (k0 + k >= a.split) break;
            f[0] += x[k].x, f[1] += x[k].y, f[2] += x[k].z, f[3] += x[k].w;
            f[4] += y[k].x, f[5] += y[k].y, f[6] += y[k].z, f[7] += y[k].w;
          }
        }
      }
      if (gave_up) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(0x7FC00000u);
      }
      const int64_t left = a.n - j;
      const int count = left < a.bn ? static_cast<int>(left) : a.bn;
      store_any(stage, a.out + i * a.ld + j, count, lane, narrow8<kBf16>(f), a.bounds(kOut));
    }
    cluster_sync();  // no CTA ends while another reads its sums
  }
  if (warp == kProductWarp) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "n"(kTensorColumns));
  }
}

// -------------------------------------------------------------------- host ----

// A map of bytes, 128 of a row and `box_rows` rows to a box, 128-byte swizzle.
bool encode_bytes(CUtensorMap* map, const uint8_t* base, int64_t pitch, int64_t rows,
                  uint32_t box_rows) {
  const EncodeTiled encode = encode_tiled();
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(pitch), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch)};
  const cuuint32_t box[2] = {128, box_rows}, unit[2] = {1, 1};
  return encode && encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(base), dims,
                          strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A map of scale tiles [row tiles][groups], `tiles` row tiles to a box.
bool encode_scales(CUtensorMap* map, const uint8_t* base, int64_t row_tiles, int64_t groups,
                   uint32_t tiles) {
  const EncodeTiled encode = encode_tiled();
  const cuuint64_t dims[3] = {kTileBytes / 4, static_cast<cuuint64_t>(groups),
                              static_cast<cuuint64_t>(row_tiles)};
  const cuuint64_t strides[2] = {kTileBytes, static_cast<cuuint64_t>(groups) * kTileBytes};
  const cuuint32_t box[3] = {kTileBytes / 4, 1, tiles}, unit[3] = {1, 1, 1};
  return encode && encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<uint8_t*>(base), dims,
                          strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A map of the output, a warp's 32 rows of 64 columns to a box.
bool encode_out(CUtensorMap* map, void* base, int64_t n, int64_t rows, int64_t ld) {
  const EncodeTiled encode = encode_tiled();
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(n), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
  const cuuint32_t box[2] = {kOutCols, 32}, unit[2] = {1, 1};
  return encode && encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, base, dims, strides, box, unit,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_NONE,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Launch {
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  Launch(int clusters, int split, cudaStream_t st) : cfg(), attr() {
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * 2 * split));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = kProgrammaticLaunch ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2 * split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
  }
};

// the kernel's shared memory, and clusters of 16 CTAs
template <class Kernel>
bool prepare(Kernel fn) {
  return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) ==
             cudaSuccess &&
         cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) ==
             cudaSuccess;
}

// Devices whose answers are kept (a call's checks cost about as much host time
// as its launch otherwise). A kernel's attributes hold in every context of its
// device, also after a reset: the runtime sets them again where it loads the kernel.
constexpr int kDevices = 64;

// the current device, -1 on error or past those
int current_device() {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < kDevices ? dev : -1;
}

template <bool kBf16, bool kSlow>
int launch(const Maps& maps, const Args& a, int clusters, int dev, cudaStream_t st) {
  const auto fn = product_kernel<kBf16, kSlow>;
  static std::atomic<bool> prepared[kDevices];
  if (!prepared[dev].load(std::memory_order_relaxed)) {
    if (!prepare(fn)) return ZERO_ECUDA;
    prepared[dev].store(true, std::memory_order_relaxed);
  }
  Launch l(clusters, a.split, st);
  return status_of(cudaLaunchKernelEx(&l.cfg, fn, maps, a));
}

// Clusters of `split` pairs that the device holds at once (0 on error).
int resident_clusters(int dev, int split) {
  static std::atomic<int> known[kDevices][kMaxSplit + 1];
  int n = known[dev][split].load(std::memory_order_relaxed);
  if (n == 0) {
    const auto fn = product_kernel<true, true>;
    Launch l(1, split, nullptr);
    if (!prepare(fn) || cudaOccupancyMaxActiveClusters(&n, fn, &l.cfg) != cudaSuccess) return 0;
    known[dev][split].store(n, std::memory_order_relaxed);
  }
  return n;
}

bool known_format(int32_t f) { return f == ZERO_E4M3 || f == ZERO_E5M2; }

constexpr int64_t kMost = int64_t{1} << 31;
constexpr int64_t kMostProduct = int64_t{1} << 30;  // tiles' ends stay below 2^31

// out[rows, n] from the left copy [rows, k] and the weight's copy [w_rows, w_cols]
template <bool kSlow>
int multiply(const void* copy, int32_t format, int64_t rows, const void* w_copy, int64_t w_rows,
             int64_t w_cols, int32_t dtype, void* out, int64_t ld, zero_scaler* d_scaler,
             void* stream) {
  if (rows < 0 || w_rows < 0 || w_cols < 0 || !known_format(format) || !is_dtype16(dtype))
    return ZERO_EINVAL;
  const int64_t n = kSlow ? w_cols : w_rows, k = kSlow ? w_rows : w_cols;
  if (ld < n) return ZERO_EINVAL;
  if (rows >= kMostProduct || w_rows >= kMostProduct || w_cols >= kMostProduct) return ZERO_ERANGE;
  if (rows == 0 || n == 0) return ZERO_OK;
  if (!out || (k && (!copy || !w_copy))) return ZERO_EINVAL;
  if (!aligned(copy, 16) || !aligned(w_copy, 16) || !aligned(out, 2) || !aligned(d_scaler, 16))
    return ZERO_EALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (k == 0) return status_of(cudaMemset2DAsync(out, 2 * ld, 0, 2 * n, rows, st));
  Args a = new_args<Args>();
  a.out = static_cast<uint16_t*>(out);
  a.scaler = d_scaler;
  a.rows = rows, a.n = n, a.ld = ld;
  a.blocks = static_cast<int32_t>(blocks_of(k));
  a.a_format = format;
  // TMA stores whole 16-byte blocks on their grid, row distances below 2^40 bytes
  a.tma_out = n % kVec == 0 && ld % kVec == 0 && aligned(out, 16) && ld < int64_t{1} << 39;
  a.set_bounds(kOut, out, rows, n, ld, 2);
  const int dev = current_device();
  if (dev < 0) return ZERO_ECUDA;
  int fit[kMaxSplit + 1];
  for (int split = 1; split <= kMaxSplit; split *= 2) fit[split] = resident_clusters(dev, split);
  if (fit[1] <= 0) return ZERO_ECUDA;
  const int64_t pairs = fit[1], m_tiles = ceil_div(rows, 2 * kM);
  // Tile width and split of the reduction by the cycles they take: turns of all
  // pairs times their blocks, a tile put out alone at the end, and the join of a
  // split, which needs room for all its clusters at once.
  const auto join_rows = [&](int split) {  // of a warp
    return ceil_div(ceil_div(std::min<int64_t>(rows, kM), split), kWarps);
  };
  int64_t best = 0;
  for (int bn = kN; bn >= 128; bn -= 64)
    for (int split = 1; split <= kMaxSplit; split *= 2) {
      const int64_t all = m_tiles * ceil_div(n, bn), turns = ceil_div(all, pairs);
      if (split > 1 && (all > fit[split] || a.blocks < 2 * split)) break;
      const int64_t cost = turns * ceil_div(a.blocks, split) *
                               (kBlockCycles + kColumnThirds * bn / 3) + kOutCycles * bn +
                           (split > 1 ? kJoinCycles + join_rows(split) * kJoinRowCycles : 0) +
                           (split == kMaxSplit ? kBigClusterCycles : 0);
      if (best == 0 || cost < best) {
        best = cost;
        a.bn = bn;
        a.split = split;
      }
    }
  const int64_t tiles = m_tiles * ceil_div(n, a.bn);
  if (tiles > 0x3fffffff) return ZERO_ERANGE;
  a.m_tiles = static_cast<int32_t>(m_tiles);
  a.tiles = static_cast<int32_t>(tiles);
  // row tiles of scales that a tile's columns may touch
  a.scale_tiles = ceil_div(a.bn, 128);
  const int clusters = static_cast<int>(std::min(tiles, a.split > 1 ? tiles : pairs));
  const int64_t pitch = blocks_of(k) * kBlock, w_pitch = blocks_of(w_cols) * kBlock;
  const uint8_t *left = static_cast<const uint8_t*>(copy),
                *right = static_cast<const uint8_t*>(w_copy);
  const uint8_t* scales = right + w_rows * w_pitch;
  if (!kSlow) scales += blocks_of(w_cols) * groups_of(w_rows) * kTileBytes;
  Maps maps = {};
  if (!encode_bytes(&maps.a, left, pitch, rows, kM) ||
      !encode_bytes(&maps.b, right, w_pitch, w_rows, kSlow ? kK : a.bn / 2) ||
      !encode_scales(&maps.scale_a, left + rows * pitch, blocks_of(rows), groups_of(k), 1) ||
      !encode_scales(&maps.scale_b, scales, blocks_of(n), groups_of(k), a.scale_tiles) ||
      (a.tma_out && !encode_out(&maps.out, out, n, rows, ld)))
    return ZERO_ECUDA;
  return dtype == ZERO_BF16 ? launch<true, kSlow>(maps, a, clusters, dev, st)
                            : launch<false, kSlow>(maps, a, clusters, dev, st);
}

}  // namespace zf

#ifdef ZERO_CHECKED
extern "C" int zf_collect_checks(unsigned long long* count, unsigned long long* first) {
  return collect_checks(count, first);
}
#endif

extern "C" {

ZERO_API size_t zero_fp8_bytes(int64_t rows, int64_t cols) {
  using namespace zf;
  if (rows < 0 || cols < 0 || rows >= kMost || cols >= kMost) return 0;
  return static_cast<size_t>(rows * blocks_of(cols) * kBlock +
                             blocks_of(rows) * groups_of(cols) * kTileBytes);
}

ZERO_API int zero_fp8_quant(const void* x, int64_t rows, int64_t cols, int64_t ld, int32_t dtype,
                            int32_t format, void* copy, void* stream) {
  using namespace zf;
  if (rows < 0 || cols < 0 || ld < cols || !is_dtype16(dtype) || !known_format(format))
    return ZERO_EINVAL;
  if (rows >= kMost || cols >= kMost || rows * ceil_div(cols, kCols) >= kMost) return ZERO_ERANGE;
  const int64_t col_tiles = ceil_div(cols, kQuantCols);
  if (rows == 0 || cols == 0) return ZERO_OK;
  if (!x || !copy) return ZERO_EINVAL;
  if (!aligned(x, 2) || !aligned(copy, 16)) return ZERO_EALIGN;
  QuantArgs a = new_args<QuantArgs>();
  a.x = static_cast<const uint16_t*>(x);
  a.rows = rows, a.cols = cols, a.ld = ld, a.pitch = blocks_of(cols) * kBlock;
  a.q = static_cast<uint8_t*>(copy);
  a.scale = a.q + rows * a.pitch;
  a.col_tiles = static_cast<uint32_t>(col_tiles);
  a.format = format;
  a.set_bounds(kX, x, rows, cols, ld, 2);
  a.set_bounds(kCopy, copy, 1, static_cast<int64_t>(zero_fp8_bytes(rows, cols)), 0, 1);
  const bool grid = on_grid(x, ld);
  const auto fn = dtype == ZERO_BF16
                      ? (grid ? quant_kernel<true, true> : quant_kernel<true, false>)
                      : (grid ? quant_kernel<false, true> : quant_kernel<false, false>);
  const dim3 ctas(static_cast<unsigned>(ceil_div(rows * col_tiles, kQuantWarps)));
  return status_of(launch_pdl(fn, ctas, dim3(32 * kQuantWarps), 0,
                              static_cast<cudaStream_t>(stream), a));
}

ZERO_API size_t zero_fp8_weight_bytes(int64_t k, int64_t n) {
  using namespace zf;
  if (k < 0 || n < 0 || k >= kMost || n >= kMost) return 0;
  return static_cast<size_t>(k * blocks_of(n) * kBlock +
                             (blocks_of(n) * groups_of(k) + blocks_of(k) * groups_of(n)) *
                                 kTileBytes);
}

ZERO_API int zero_fp8_quant_weight(const void* w, int64_t k, int64_t n, int32_t dtype, void* copy,
                                   void* stream) {
  using namespace zf;
  if (k < 0 || n < 0 || !is_dtype16(dtype)) return ZERO_EINVAL;
  if (k >= kMost || n >= kMost || blocks_of(k) * blocks_of(n) >= kMost) return ZERO_ERANGE;
  if (k == 0 || n == 0) return ZERO_OK;
  if (!w || !copy) return ZERO_EINVAL;
  if (!aligned(w, 2) || !aligned(copy, 16)) return ZERO_EALIGN;
  QuantArgs a = new_args<QuantArgs>();
  a.x = static_cast<const uint16_t*>(w);
  a.rows = k, a.cols = a.ld = n, a.pitch = blocks_of(n) * kBlock;
  a.q = static_cast<uint8_t*>(copy);
  a.scale = a.q + k * a.pitch;
  a.scale_t = a.scale + blocks_of(n) * groups_of(k) * kTileBytes;
  a.col_tiles = static_cast<uint32_t>(ceil_div(n, kCols));
  a.format = ZERO_E4M3;
  a.set_bounds(kX, w, k, n, n, 2);
  a.set_bounds(kCopy, copy, 1, static_cast<int64_t>(zero_fp8_weight_bytes(k, n)), 0, 1);
  const bool grid = on_grid(w, n);
  const bool bf16 = dtype == ZERO_BF16;
  const auto fn =
      grid ? (bf16 ? quant_weight_kernel<true, true> : quant_weight_kernel<false, true>)
           : (bf16 ? quant_weight_kernel<true, false> : quant_weight_kernel<false, false>);
  return status_of(launch_pdl(fn, dim3(static_cast<unsigned>(blocks_of(k) * ceil_div(n, kCols))),
                              dim3(256), 0, static_cast<cudaStream_t>(stream), a));
}

ZERO_API int zero_fp8_linear(const void* x_copy, int32_t x_format, int64_t rows,
                             const void* w_copy, int64_t k, int64_t n, int32_t dtype, void* y,
                             int64_t ld, zero_scaler* d_scaler, void* stream) {
  return zf::multiply<true>(x_copy, x_format, rows, w_copy, k, n, dtype, y, ld, d_scaler, stream);
}

ZERO_API int zero_fp8_linear_dgrad(const void* dy_copy, int32_t dy_format, int64_t rows,
                                   const void* w_copy, int64_t k, int64_t n, int32_t dtype,
                                   void* dx, int64_t ld, zero_scaler* d_scaler, void* stream) {
  return zf::multiply<false>(dy_copy, dy_format, rows, w_copy, k, n, dtype, dx, ld, d_scaler,
                             stream);
}

}  // extern "C"
