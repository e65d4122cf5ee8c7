/*
 * wgrad.cu -- weight gradient of a linear layer from its input's 8-bit
 * checkpoint (zero_train.h): dw[i, j] = sum over t of x^[t, i] dy[t, j].
 *
 * A matrix product whose reduction runs over the tokens, the slow axis of
 * both operands, on the 5th-generation tensor cores. A pair of CTAs (one
 * tcgen05.mma over two SMs) forms a tile of dw of 256 rows and one or two
 * groups of up to 256 columns in tensor memory (fp32), 64 tokens per step:
 * each CTA holds 128 rows of the tile, 128 of the checkpoint's columns and half
 * of dy's. (One CTA per 128 x 256 tile took in 40 KB per step against 24, and
 * the whole product 307 us against 255.) Per CTA, through a ring of stages:
 *   copy warp       brings its half of dy's tile by TMA (128-byte swizzle, rows
 *                   of 64 columns: the tensor core's layout for an operand
 *                   whose slow axis is the reduction);
 *   16 value warps  in two groups, each every other step: read the
 *                   checkpoint's 64 x 128 tile into registers two of its steps
 *                   ahead (eight lanes a row), turn it into 16-bit values and
 *                   store them in the same layout. q * 2^k is exact in the
 *                   16-bit type, so the operand is the checkpoint itself,
 *                   without a rounding;
 *   product warp    (first CTA of the pair) one thread issues four products of
 *                   16 tokens per column group and stage;
 *   4 output warps  read a finished tile from tensor memory, round once and
 *                   store. With one column group the next tile's sums form in
 *                   the other half of tensor memory meanwhile; two groups fill
 *                   it, and halve the value warps' work per product.
 * A step's values take about 850 cycles, 256 columns' products 512, so two
 * groups are what feeds the tensor cores: 8192 x 2048 x 8192 bf16 takes 157 to
 * 179 us by the card and its power cap (cuBLAS on bf16 operands 162 to 167 where
 * this takes 176 to 179) against 240 us with one group. Its 152 tiles are two
 * whole turns of the 76 pairs, which suits it best. Where tiles fill the turns
 * less or only one column group fits them, the tensor cores wait: 8192 x 2048 x
 * 5632 156 us (97 at their rate), x 2048 70 (35), 1024 x 4096 71 (35), 768 x 2304
 * 41 (15). 1024 tokens x 768 x 2304 takes 13.5 us, of which 8 are set-up, the
 * first copies' latency and the output.
 *
 * Few tiles and many tokens: a cluster of 2, 4 or 8 pairs shares a tile, each
 * pair a part of the tokens; the sums meet in shared memory and every CTA adds
 * its share of the rows over the cluster in rank order. Split and tile width
 * depend on the sizes and the device alone, so results do not change from call
 * to call.
 *
 * A dy whose rows do not start on 16-byte boundaries comes as the 16-byte
 * blocks that hold it, and three groups of warps move it to its places beside
 * the values (at Maps; 8000 x 2000 x 5555: 236 us against 150 at 5552. One
 * group for dy and two for the values took 416).
 *
 * Every wait is bounded (2 s). One that expires ends the work of its cluster:
 * the sums of a tile are given out only when all its products were issued, the
 * tiles left become NaN, copies and products in flight land before the CTAs
 * end, and the scaler's error word is raised.
 */
#include <cuda.h>

#include "train.cuh"

#include <algorithm>
#include <atomic>

namespace zw {

using namespace zt;

constexpr int kGroupWarps = 8;
constexpr int kGroupThreads = 32 * kGroupWarps;
constexpr int kOutWarps = 4;
// warps by role: groups that fill stages, copies, products, output. Groups that
// also place dy take longer over a step, so there is one more.
template <bool kTma>
struct Roles {
  static constexpr int kGroups = kTma ? 2 : 3;
  static constexpr int kCopyWarp = kGroups * kGroupWarps, kProductWarp = kCopyWarp + 1;
  static constexpr int kOutWarp0 = kProductWarp + 1, kWarps = kOutWarp0 + kOutWarps;
  static constexpr int kThreads = 32 * kWarps;
};
constexpr int kM = 128, kN = 256, kK = 64;     // rows per CTA, columns at most, tokens per stage
constexpr int kAhead = 2;                       // a value thread's steps loaded ahead
constexpr int kChunk = kK * 128;               // 64 tokens x 64 columns of 16 bits
constexpr int kBytesA = kM / 64 * kChunk, kBytesB = kN / 2 / 64 * kChunk;
constexpr int kRing = 198 * 1024;              // shared memory for stages
constexpr int kJoinPitch = kN + 4;             // fp32 row of a tile in shared memory
constexpr int kSmem = kRing + 1024;
constexpr int kMaxSplit = 8, kJoinAhead = 4;
// costs in cycles, from times at 768 x 2304 and 2048 x 8192 over 1 to 8192 tokens:
// a step's values, a column put out, the join of a split
constexpr int kValueCycles = 850, kOutCycles = 28, kJoinCycles = 3500;
// clusters of 16 CTAs, beside that: together and each. Only for the narrowest
// tiles (8192 x 256 x 256: two clusters of 128 columns 21.9 us, one of 256
// columns 29.3, smaller clusters 26.2; 8192 x 100 x 101: 24 against 32).
constexpr int kBigClusterCycles = 4000, kPerBigCluster = 1000;
// a step's values and one or two column groups of dy off the grid, from 8192 x
// 2048 x 8191 (341 us with one group per tile, 313 with two)
constexpr int kPlaceCycles[2] = {1250, 2200};
static_assert(kM * kJoinPitch * 4 <= kRing, "the tile fits the stages");
static_assert(kM == ZERO_CKPT_PAD, "a checkpoint row is whole CTA tiles");

enum { kCkpt, kDw, kBuffers };  // of a call, for their bounds

struct Args : Checked<kBuffers> {
  const int8_t* q;
  const uint8_t* scale;
  const uint16_t* dy;
  uint16_t* dw;
  zero_scaler* scaler;
  int64_t rows, cols, pitch, n, ld;
  int32_t split, vec_out, bn, m_tiles, tiles;
};

// ------------------------------------------------------------- primitives ----

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void bar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count)
               : "memory");
}

__device__ __forceinline__ void bar_expect(uint64_t* bar, uint32_t bytes) {
  asm volatile(
      "{\n .reg .b64 st;\n mbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n}" ::"r"(
          smem_u32(bar)),
      "r"(bytes)
      : "memory");
}

// the same variable in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t in_cta(const void* p, uint32_t rank) {
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(p)), "r"(rank));
  return remote;
}

// CTA-scope release: what it publishes is this CTA's own shared or tensor
// memory, read by this SM's tensor core after the proxy fence that precedes it
// (a cluster-scope release would wait for this thread's loads ahead as well:
// 224 us against 179 at 8192 x 2048 x 8192). The waits need no wider scope for
// the same reason; no thread reads through them what another CTA wrote.
__device__ __forceinline__ void bar_arrive_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}

// One try; the thread sleeps in it until the phase completes, at most about a
// millisecond (22 warps that asked in turn would slow what they wait for).
__device__ __forceinline__ bool bar_try(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000000;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Sets *failed in every CTA of the cluster (each stays until all have ended).
__device__ __forceinline__ void give_up(int* failed) {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
  for (uint32_t r = 0; r < n; ++r)
    asm volatile("st.relaxed.cluster.shared::cluster.u32 [%0], 1;" ::"r"(in_cta(failed, r))
                 : "memory");
}

// true when the phase has completed; false once *failed is set or the limit
// has passed (which sets it)
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, int* failed,
                                         uint64_t limit) {
  if (bar_try(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  for (;;) {
    if (bar_try(bar, parity)) return true;
    if (*static_cast<volatile int*>(failed)) return false;
    if (global_ns() - t0 > limit) {
      give_up(failed);
      return false;
    }
  }
}

// all threads of a value group
__device__ __forceinline__ void group_sync(int group) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(kGroupThreads) : "memory");
}

// A box of dy into this CTA; its bytes are counted by the barrier at
// `cluster_bar`, in this CTA or the other of the pair.
__device__ __forceinline__ void copy_box(void* dst, const CUtensorMap* map, int32_t x, int32_t y,
                                         uint32_t cluster_bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(cluster_bar)
      : "memory");
}

// Shared-memory operand whose reduction axis is the slow one, 128-byte
// swizzle: rows of 64 elements (128 bytes), eight rows per 1024-byte atom
// (the next eight reduction steps), the next 64 elements kChunk bytes on. The
// low word holds the address in 16-byte units and the chunk distance; stages
// and reduction steps are added to it.
constexpr uint32_t kOperandHigh = (1024 >> 4) | 1u << 14 | 2u << 29;

__device__ __forceinline__ uint32_t operand_low(uint32_t addr) {
  return (addr & 0x3FFFF) >> 4 | static_cast<uint32_t>(kChunk >> 4) << 16;
}

// fp32 sums; both operands of the 16-bit type, slow axis reduced; 256 x bn
template <bool kBf16>
__device__ __forceinline__ uint32_t product_desc(int bn) {
  return 1u << 4 | (kBf16 ? 1u : 0u) << 7 | (kBf16 ? 1u : 0u) << 10 | 1u << 15 | 1u << 16 |
         static_cast<uint32_t>(bn >> 3) << 17 | static_cast<uint32_t>(2 * kM >> 4) << 24;
}

__device__ __forceinline__ void product(uint32_t d, uint32_t a_low, uint32_t b_low, uint32_t desc,
                                        uint32_t add) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 da, db;\n setp.ne.b32 p, %4, 0;\n"
      " mov.b64 da, {%1, %5};\n mov.b64 db, {%2, %5};\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %3, p;\n}" ::"r"(d),
      "r"(a_low), "r"(b_low), "r"(desc), "r"(add), "r"(kOperandHigh)
      : "memory");
}

// arrive at `bar` of both CTAs of the pair once the products issued so far are done
__device__ __forceinline__ void commit(uint64_t* bar, uint16_t pair_mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(smem_u32(bar)),
      "h"(pair_mask)
      : "memory");
}

// 32 lanes x 32 columns of tensor memory
__device__ __forceinline__ void read_sums(uint32_t addr, float (&f)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
#pragma unroll
  for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(r[j]);
}

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::
          : "memory");
}

// ------------------------------------------------------------------ values ----

// One block's step 2^k in both halves of a word. 255 (not finite) becomes an
// infinity or NaN that turns the block's zeros into NaN.
template <bool kBf16>
__device__ __forceinline__ uint32_t step_pair(uint32_t s) {
  uint32_t h;
  if constexpr (kBf16) h = s << 7;
  else h = s == 255 ? 0x7E00u : s >= 113 ? (s - 112) << 10 : 1u << (s - 103);
  return h * 0x10001u;
}

// Two of a word's four int8 values (bytes 0 and 1, or 2 and 3) as a pair of
// 16-bit floats times `step`: the byte's bits are put under the exponent of a
// number whose last place is 1, and that number is taken off again.
template <bool kBf16, int kHalf>
__device__ __forceinline__ uint32_t value_pair(uint32_t w, uint32_t step) {
  uint32_t r;
  if constexpr (kBf16) {
    // 128 + low seven bits, less 128 or (sign bit set) 256
    const uint32_t p = __byte_perm(w, 0, kHalf ? 0x4342 : 0x4140);
    const uint32_t lo = (p & 0x007F007Fu) | 0x43004300u, hi = (p & 0x00800080u) | 0x43004300u;
    asm("{\n .reg .b32 d;\n sub.rn.bf16x2 d, %1, %2;\n mul.rn.bf16x2 %0, d, %3;\n}"
        : "=r"(r)
        : "r"(lo), "r"(hi), "r"(step));
  } else {
    // w holds value + 128: 1024 + (value + 128), less 1152
    const uint32_t u = __byte_perm(w, 0x64646464u, kHalf ? 0x4342 : 0x4140);
    asm("{\n .reg .b32 d;\n sub.rn.f16x2 d, %1, %2;\n mul.rn.f16x2 %0, d, %3;\n}"
        : "=r"(r)
        : "r"(u), "r"(0x64806480u), "r"(step));
  }
  return r;
}

// A thread's part of a step: 16 checkpointed values of each of two tokens,
// four rows apart. Eight lanes read a row's 128 bytes together.
struct Piece {
  uint4 q[2];
  uint32_t scale[2];
};

// Where a thread's values of one tile are: q and scale of its first token of
// the next step to load; left: tokens from there on (0 or less: none, or the
// tile's columns lie past the checkpoint's).
struct Source {
  const int8_t* q;
  const uint8_t* scale;
  int32_t left;
};

// Ordinary loads: the kernel before may have written the checkpoint while this
// one was already resident, which the read-only path does not allow for.
__device__ __forceinline__ Piece load_piece(const Args& a, const Source& s, int64_t q_step,
                                            int64_t scale_step) {
  Piece b;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    b.q[k] = make_uint4(0, 0, 0, 0);
    b.scale[k] = 127;
    if (s.left > 4 * k && a.bounds(kCkpt).holds(s.q + k * q_step, 16, kSiteLoad) &&
        a.bounds(kCkpt).holds(s.scale + k * scale_step, 1, kSiteLoad)) {
      b.q[k] = *reinterpret_cast<const uint4*>(s.q + k * q_step);
      b.scale[k] = s.scale[k * scale_step];
    }
  }
  return b;
}

// Token row r's 16 values of columns [16 p, 16 p + 16) of the A tile: two
// 16-byte pieces. The upper four of eight lanes take theirs in the other
// order, so that the eight lanes of a store phase fall on eight different
// pieces of the 128-byte rows.
struct Values {
  uint4 v[2];
};

template <bool kBf16>
__device__ __forceinline__ Values values_of(const uint4& q, uint32_t scale, int p) {
  const uint32_t s = step_pair<kBf16>(scale);
  const bool swap = p >= 4;
  const uint32_t w[4] = {swap ? q.z : q.x, swap ? q.w : q.y, swap ? q.x : q.z, swap ? q.y : q.w};
  Values out;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint32_t x0 = w[2 * j], x1 = w[2 * j + 1];
    if constexpr (!kBf16) x0 ^= 0x80808080u, x1 ^= 0x80808080u;
    out.v[j] = make_uint4(value_pair<kBf16, 0>(x0, s), value_pair<kBf16, 1>(x0, s),
                          value_pair<kBf16, 0>(x1, s), value_pair<kBf16, 1>(x1, s));
  }
  return out;
}

__device__ __forceinline__ void store_values(uint8_t* stage_a, const Values& x, int r, int p) {
  uint8_t* row = stage_a + (p >> 2) * kChunk + r * 128;
  const int at = (((p & 3) << 1 | (p >> 2)) ^ (r & 7)) << 4;
  *reinterpret_cast<uint4*>(row + at) = x.v[0];
  *reinterpret_cast<uint4*>(row + (at ^ 16)) = x.v[1];
}

// dy's half tile when its rows do not start on 16-byte boundaries, where no one
// TMA map covers it: eight rows are 16 ld bytes, so each class of every eighth
// token has a map of its own, from the boundary at or before its first element.
// The copy warp brings a step's 64 tokens class by class into the stage, eight
// boxes of the blocks that hold 128 columns (17 where they do not start on one),
// and a group moves them to their places there: every piece is in a register
// before the first is put back. (Slots for the raw rows beside fewer stages spare
// that wait; the same time, and no room for two column groups.) A step is 64 rows
// and a tile's columns are whole blocks, so the distance d of a row's first
// column from its block is its class's in every step and tile. Shared memory's
// pipe is 56 % busy then, the integer pipe 59, the tensor cores 38.
constexpr int kClasses = 8, kRawColumns = 128 + 8;
constexpr int kRawPitch = kRawColumns * 2, kRawBytes = kK * kRawPitch;
static_assert(kRawBytes >= kBytesB && kRawBytes % 1024 == 0, "a stage of raw rows");
static_assert(kGroupWarps == kClasses && kK == 64, "a warp places eight rows of 16 pieces");

template <bool kAligned>
struct Maps {
  CUtensorMap of[kAligned ? 1 : kClasses];
};

// A warp moves its class: pieces of eight columns, eight of a row by eight
// lanes, which meet no bank twice, in the raw rows or the placed ones. from: the
// first of the lane's four pieces (rows 4 i apart, then 64 columns on). The
// distance is the warp's own, so that a piece costs at most four shifts (picked
// by selects from a distance per lane, 15: 309 us against 251). Columns past
// dy's end are whatever lies there: no column of dw that is stored depends on
// them.
struct Pieces {
  uint4 v[4];
};

template <int kDistance>
__device__ __forceinline__ Pieces take_pieces(const uint8_t* from) {
  Pieces p;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint4* block =
        reinterpret_cast<const uint4*>(from + (k & 1) * (4 * kRawPitch) + (k >> 1) * 128);
    const uint4 x = block[0];
    p.v[k] = kDistance ? shifted_by<kDistance>(x, block[1]) : x;
  }
  return p;
}

// r: the warp's class, d: its distance
__device__ __forceinline__ Pieces take_raw(const uint8_t* raw, int r, int lane, int d) {
  const uint8_t* from = raw + (r * (kK / kClasses) + (lane >> 3)) * kRawPitch + (lane & 7) * 16;
  switch (d >> 1) {
    case 0: return take_pieces<0>(from);
    case 1: return take_pieces<2>(from);
    case 2: return take_pieces<4>(from);
    case 3: return take_pieces<6>(from);
    case 4: return take_pieces<8>(from);
    case 5: return take_pieces<10>(from);
    case 6: return take_pieces<12>(from);
    default: return take_pieces<14>(from);
  }
}

__device__ __forceinline__ void place(uint8_t* stage_b, const Pieces& p, int r, int lane) {
  uint8_t* to = stage_b + (8 * (lane >> 3) + r) * 128 + (((lane & 7) ^ r) << 4);
#pragma unroll
  for (int k = 0; k < 4; ++k)
    *reinterpret_cast<uint4*>(to + (k & 1) * (4 * 1024) + (k >> 1) * kChunk) = p.v[k];
}

// An output warp's 32 columns of its lanes' rows, in the 16-bit type.
template <bool kBf16>
__device__ __forceinline__ void narrow32(const float (&f)[32], uint4 (&v)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k)
    v[k] = make_uint4(
        narrow2<kBf16>(f[8 * k], f[8 * k + 1]), narrow2<kBf16>(f[8 * k + 2], f[8 * k + 3]),
        narrow2<kBf16>(f[8 * k + 4], f[8 * k + 5]), narrow2<kBf16>(f[8 * k + 6], f[8 * k + 7]));
}

// Rows of dw off the 16-byte grid leave through shared memory, kOutCols columns
// of 32 rows at a time and eight lanes per row, in the whole blocks of their
// addresses (a lane storing its own row element by element wrote every 32-byte
// sector 16 times). A block may begin in the columns before: each row's stage
// starts with its last eight of those. Only the elements before a tile's first
// block and after its last go one by one.
constexpr int kOutCols = 64, kOutPitch = 16 + kOutCols * 2;

// columns [c, c + width) of the tile's row that starts at `to`, which has
// `count` columns
__device__ __forceinline__ void store_staged(uint8_t* stage, uint16_t* to, int64_t n, int64_t rows,
                                             int c, int width, int count, int lane,
                                             const Bounds& in) {
  const int k = lane & 7, row0 = lane >> 3;
  const int end = c + width < count ? c + width : count;  // columns there are so far
#pragma unroll 1
  for (int pass = 0; pass < 8; ++pass) {
    const int row = pass * 4 + row0;
    if (row >= rows) continue;
    uint16_t* at = to + row * n;
    const int d = static_cast<int>(reinterpret_cast<uintptr_t>(at) & 15);
    const uint4* block = reinterpret_cast<const uint4*>(stage + row * kOutPitch + 16) + k;
    const int begin = 2 * c + 16 * k - d;  // byte of the row the block starts at
    uint8_t* whole = reinterpret_cast<uint8_t*>(at) + begin;
    if (begin >= 0 && begin + 16 <= 2 * end && in.holds(whole, 16, kSiteStore))
      *reinterpret_cast<uint4*>(whole) = shifted_back(block[-1], block[0], d);
    if (c == 0 || end == count) {
      const uint16_t* elems = reinterpret_cast<const uint16_t*>(stage + row * kOutPitch + 16);
      const int head = d ? min((16 - d) >> 1, end) : 0;
      if (c == 0 && k < head && in.holds(at + k, 2, kSiteStore)) at[k] = elems[k];
      // elements of the block that no later columns complete
      const int tail = max(c == 0 ? head : 0, (((2 * end + d) & ~15) - d) >> 1);
      if (end == count && tail + k < end && in.holds(at + tail + k, 2, kSiteStore))
        at[tail + k] = elems[tail + k - c];
    }
  }
}

// ------------------------------------------------------------------ kernel ----

// A step of this pair's work: token block `step` of tile `tile`.
struct Cursor {
  int32_t tile, step;
  __device__ __forceinline__ void advance(int by, int steps, int tile_stride) {
    step += by;
    while (step >= steps) {
      step -= steps;
      tile += tile_stride;
    }
  }
};

template <int kStages>
struct Ring {  // stage and the parity of its current use
  int32_t stage = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void advance(int by) {
    stage += by;
    if (stage >= kStages) {
      stage -= kStages;
      parity ^= 1;
    }
  }
};

// kWide: column groups of bn per tile (1 or 2), which share the checkpoint's
// stage.
template <bool kBf16, bool kTma, int kWide>
__global__ void __launch_bounds__(Roles<kTma>::kThreads, 1)
    wgrad_kernel(const __grid_constant__ Maps<kTma> maps, const Args a) {
  constexpr int kStageB = kTma ? kBytesB : kRawBytes;  // a column group's dy
  constexpr int kStageBytes = kBytesA + kWide * kStageB;
  constexpr int kStages = kRing / kStageBytes;
  using R = Roles<kTma>;
  constexpr int kCopyWarp = R::kCopyWarp, kProductWarp = R::kProductWarp;
  constexpr int kOutWarp0 = R::kOutWarp0, kGroups = R::kGroups;
  extern __shared__ uint8_t raw[];
  uint8_t* stages = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  // full: in the pair's first CTA, counted by both (off the grid full_b in each,
  // for its own groups); empty and done: in each
  __shared__ uint64_t full_a[kStages], full_b[kStages], empty[kStages], done[2], free_sums[2];
  __shared__ uint32_t tmem_base;
  __shared__ int failed, group_ok[kGroups];
  __shared__ __align__(16) uint8_t out_stage[kOutWarps][32 * kOutPitch];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint64_t limit = a.limit();
  const int n_cta = 2 * a.split;
  const int rank = static_cast<int>(blockIdx.x) % n_cta;
  const int half = rank & 1, part = rank >> 1, leader = rank & ~1;
  const int tile0 = static_cast<int>(blockIdx.x) / n_cta;
  const int tile_stride = static_cast<int>(gridDim.x) / n_cta;
  const int my_tiles = tile0 < a.tiles ? (a.tiles - tile0 + tile_stride - 1) / tile_stride : 0;
  // this pair's tokens: whole steps
  const int64_t all_steps = (a.rows + kK - 1) / kK;
  const int64_t s0 = all_steps * part / a.split, s1 = all_steps * (part + 1) / a.split;
  const int steps = static_cast<int>(s1 - s0);
  const int64_t total = static_cast<int64_t>(steps) * my_tiles;
  const int64_t t_begin = s0 * kK, t_end = s1 * kK < a.rows ? s1 * kK : a.rows;
  const auto row_of = [&](int tile) {  // first row of dw of this CTA's part of the tile
    return static_cast<int64_t>(tile % a.m_tiles) * (2 * kM) + half * kM;
  };
  const auto column_of = [&](int tile) {
    return static_cast<int64_t>(tile / a.m_tiles) * (kWide * a.bn);
  };

  if (warp == kProductWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&tmem_base)),
                 "n"(2 * kN)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      bar_init(&full_a[s], 2);
      bar_init(&full_b[s], 1);
      bar_init(&empty[s], 1);
    }
    for (int k = 0; k < 2; ++k) {
      bar_init(&done[k], 1);
      bar_init(&free_sums[k], 2 * kOutWarps);
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

  if (warp < kCopyWarp) {
    // value warps: thread -> tokens r and r + 4 of a step, columns [16 p, 16 p + 16)
    const int group = warp / kGroupWarps, r = (warp % kGroupWarps) * 8 + (lane >> 3), p = lane & 7;
    const uint32_t arrive_at = in_cta(full_a, leader);
    const int64_t blocks = a.pitch / ZERO_CKPT_BLOCK;
    const int tokens = static_cast<int>(t_end - t_begin);
    const auto source_of = [&](const Cursor& c) {
      const int64_t i = row_of(c.tile) + p * 16;
      const int32_t t = c.step * kK + r;
      return Source{a.q + (t_begin + t) * a.pitch + i, a.scale + (t_begin + t) * blocks + (i >> 5),
                    c.tile < a.tiles && i < a.pitch ? tokens - t : 0};
    };
    Cursor ahead = {tile0, 0};
    Ring<kStages> ring;
    ring.advance(group);
    Piece next[kAhead];
    Source src = {};
    const auto load = [&]() {
      const Piece b = load_piece(a, src, 4 * a.pitch, 4 * blocks);
      ahead.step += kGroups;
      if (ahead.step < steps) {
        src.q += kGroups * kK * a.pitch;
        src.scale += kGroups * kK * blocks;
        src.left -= src.left > 0 ? kGroups * kK : 0;
      } else {
        ahead.advance(0, steps, tile_stride);
        src = source_of(ahead);
      }
      return b;
    };
    bool ok = true;
    // off the grid: the class this warp places
    const int place_class = warp % kGroupWarps;
    const int distance =
        static_cast<int>((reinterpret_cast<uintptr_t>(a.dy) + 2 * place_class * a.ld) & 15);
    // the stage of the step at hand once it is free (off the grid: has its dy),
    // or NULL: given up. One warp of the group asks (many that poll slow what
    // they wait for).
    const auto free_stage = [&](int64_t at) -> uint8_t* {
      if (!kTma || at >= kStages) {
        if (warp % kGroupWarps == 0) {
          const bool free = kTma ? bar_wait(&empty[ring.stage], ring.parity ^ 1, &failed, limit)
                                 : bar_wait(&full_b[ring.stage], ring.parity, &failed, limit);
          if (lane == 0) group_ok[group] = free;
        }
        group_sync(group);
        ok = *static_cast<volatile int*>(&group_ok[group]) != 0;
      }
      return ok ? stages + ring.stage * kStageBytes : nullptr;
    };
    const auto stored = [&]() {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      group_sync(group);
      if (tid % kGroupThreads == 0) bar_arrive_at(arrive_at + ring.stage * 8);
      ring.advance(kGroups);
    };
    if (total > 0) {
      ahead.advance(group, steps, tile_stride);
      src = source_of(ahead);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) next[k] = load();
    }
    for (int64_t it = group; it < total && ok; it += kAhead * kGroups) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int64_t at = it + k * kGroups;
        if (at >= total || !ok) break;
        // worked out before the stage is free: only the stores stand between
        // that and the products
        const Values v0 = values_of<kBf16>(next[k].q[0], next[k].scale[0], p);
        const Values v1 = values_of<kBf16>(next[k].q[1], next[k].scale[1], p);
        uint8_t* stage = free_stage(at);
        if (!stage) break;
        store_values(stage, v0, r, p);
        store_values(stage, v1, r + 4, p);
        if constexpr (!kTma) {
#pragma unroll 1
          for (uint8_t* b = stage + kBytesA; b < stage + kStageBytes; b += kStageB) {
            const Pieces pieces = take_raw(b, place_class, lane, distance);
            group_sync(group);
            place(b, pieces, place_class, lane);
          }
        }
        stored();
        next[k] = load();  // not before: the proxy fence would wait for it
      }
    }
  } else if (warp == kCopyWarp) {
    if (lane == 0) {
      // one thread's dependent instructions are slow beside 22 warps: what
      // does not change from step to step is worked out before
      const int chunks = (a.bn / 2 + 63) / 64;
      const uint32_t full_at = in_cta(full_b, kTma ? leader : rank);
      Ring<kStages> ring;
      bool ok = true;
      int left_fresh = kStages;
      for (int k = 0; k < my_tiles && ok; ++k) {
        const int32_t x =
            static_cast<int32_t>(column_of(tile0 + k * tile_stride) + half * (a.bn / 2));
        int32_t y = static_cast<int32_t>(t_begin);
        for (int step = 0; step < steps; ++step, y += kK) {
          const int s = ring.stage;
          if (left_fresh > 0) --left_fresh;
          else if (!bar_wait(&empty[s], ring.parity ^ 1, &failed, limit)) {
            ok = false;
            break;
          }
          if (blockIdx.x == 0 &&
              a.holds(ZERO_PLANT_NO_COPY, static_cast<int64_t>(k) * steps + step)) {
            ring.advance(1);
            continue;
          }
          uint8_t* b = stages + s * kStageBytes + kBytesA;
          if constexpr (kTma) {
            if (half == 0) bar_expect(&full_b[s], 2 * kWide * chunks * kChunk);
#pragma unroll
            for (int w = 0; w < kWide; ++w) {
              copy_box(b + w * kStageB, &maps.of[0], x + w * a.bn, y, full_at + s * 8);
              if (chunks > 1)
                copy_box(b + w * kStageB + kChunk, &maps.of[0], x + w * a.bn + 64, y,
                         full_at + s * 8);
            }
          } else {
            bar_expect(&full_b[s], kWide * kRawBytes);
#pragma unroll
            for (int c = 0; c < kClasses; ++c)
#pragma unroll
              for (int w = 0; w < kWide; ++w)  // no tokens: past the end of another class
                copy_box(b + w * kStageB + c * (kRawBytes / kClasses), &maps.of[c], x + w * a.bn,
                         y / kClasses + (c < a.rows ? 0 : 1), full_at + s * 8);
          }
          ring.advance(1);
        }
      }
    }
  } else if (warp == kProductWarp) {
    if (half == 0 && lane == 0) {
      const uint16_t pair_mask = static_cast<uint16_t>(3u << leader);
      const uint32_t desc = product_desc<kBf16>(a.bn);
      const uint32_t base = operand_low(smem_u32(stages));
      Ring<kStages> ring;
      bool ok = true;
      for (int k = 0; k < my_tiles && ok && steps > 0; ++k) {
        // one group per tile: two tiles' sums in turn; two groups fill tensor memory
        const int buf = kWide == 1 ? k & 1 : 0, use = kWide == 1 ? k >> 1 : k;
        const uint32_t sums = tmem + buf * kN;
        ok = use == 0 || bar_wait(&free_sums[buf], (use - 1) & 1, &failed, limit);
        for (int step = 0; step < steps && ok; ++step) {
          const int s = ring.stage;
          ok = bar_wait(&full_a[s], ring.parity, &failed, limit) &&
               (!kTma || bar_wait(&full_b[s], ring.parity, &failed, limit));
          if (!ok) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint32_t at = base + s * (kStageBytes >> 4);
#pragma unroll
          for (int q = 0; q < kK / 16; ++q)
#pragma unroll
            for (int w = 0; w < kWide; ++w)
              product(sums + w * kN, at + q * (2048 >> 4),
                      at + ((kBytesA + w * kStageB) >> 4) + q * (2048 >> 4), desc,
                      q > 0 ? 1u : step);
          commit(&empty[s], pair_mask);
          ring.advance(1);
        }
        if (ok) commit(&done[buf], pair_mask);  // whole sums only
      }
    }
  } else if (warp >= kOutWarp0) {
    // this warp's quarter of tensor memory's lanes
    const int row0 = (warp & 3) * 32;
    bool ok = true;
    for (int k = 0; k < my_tiles; ++k) {
      const int tile = tile0 + k * tile_stride;
      const int buf = kWide == 1 ? k & 1 : 0, use = kWide == 1 ? k >> 1 : k;
      // the warp's verdict: its lanes read tensor memory together
      if (steps > 0 && ok)
        ok = __all_sync(0xffffffffu, bar_wait(&done[buf], use & 1, &failed, limit));
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t sums = tmem + (static_cast<uint32_t>(row0) << 16) + buf * kN;
      const int64_t i0 = row_of(tile) + row0, j = column_of(tile);
      uint4 last = make_uint4(0, 0, 0, 0);  // the eight columns before, of this lane's row
#pragma unroll 1
      for (int c = 0; c < kWide * a.bn; c += 32) {
        float f[32];
        if (ok && steps > 0) {
          read_sums(sums + (kWide == 2 && c >= a.bn ? kN - a.bn : 0) + c, f);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) f[e] = ok ? 0.f : __uint_as_float(0x7FC00000u);
        }
        if (a.split == 1) {
          uint4 v[4];
          narrow32<kBf16>(f, v);
          uint16_t* to = a.dw + i0 * a.n + j;  // the tile's columns of this warp's first row
          if (a.vec_out) {
            uint4* row = reinterpret_cast<uint4*>(to + lane * a.n + c);
#pragma unroll
            for (int e = 0; e < 4; ++e)  // n is a multiple of 8
              if (i0 + lane < a.cols && j + c + 8 * e < a.n &&
                  a.bounds(kDw).holds(row + e, 16, kSiteStore))
                row[e] = v[e];
          } else if (j + (c & ~(kOutCols - 1)) < a.n) {
            uint8_t* stage = out_stage[warp - kOutWarp0];
            uint4* row = reinterpret_cast<uint4*>(stage + lane * kOutPitch);
            const int within = c & (kOutCols - 1);
            const int count =
                static_cast<int>(min(a.n - j, static_cast<int64_t>(kWide * a.bn)));
            if (within == 0) row[0] = last;
#pragma unroll
            for (int e = 0; e < 4; ++e) row[1 + within / 8 + e] = v[e];
            last = v[3];
            if (within || c + 32 == kWide * a.bn) {
              __syncwarp();
              store_staged(stage, to, a.n, a.cols - i0, c - within, within + 32, count, lane,
                           a.bounds(kDw));
              __syncwarp();
            }
          }
        } else {
          float4* p = reinterpret_cast<float4*>(
              reinterpret_cast<float*>(stages) + (row0 + lane) * kJoinPitch + c);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            p[e] = make_float4(f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3]);
        }
      }
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      // given up: the sums stay taken, others may still read theirs
      if (ok && lane == 0) bar_arrive_at(in_cta(&free_sums[buf], leader));
    }
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
    uint8_t* stage = &out_stage[0][0] + warp * ((kStageWarp + 15) & ~15);
    for (int m = warp; m < share; m += R::kWarps) {
      const int row = part * share + m;
      const int64_t i = row_of(tile0) + row;
      if (i >= a.cols) break;
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
      uint16_t* to = a.dw + i * a.n + j;
      if (a.vec_out) {
        if (lane * 8 < count && a.bounds(kDw).holds(to + lane * 8, 16, kSiteStore))
          *reinterpret_cast<uint4*>(to + lane * 8) = narrow8<kBf16>(f);
      } else {
        store_any(stage, to, count, lane, narrow8<kBf16>(f), a.bounds(kDw));
      }
    }
    cluster_sync();  // no CTA ends while another reads its sums
  }
  if (warp == kProductWarp) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(2 * kN));
  }
}

// -------------------------------------------------------------------- host ----

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// Map of `rows` rows of n elements, ld apart; boxes of 64 columns go to swizzled
// stages, wider ones as they lie.
bool encode_rows(CUtensorMap* map, uintptr_t base, int64_t n, int64_t rows, int64_t ld,
                 uint32_t box_columns, uint32_t box_rows, bool bf16) {
  const EncodeTiled encode = encode_tiled();
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(n), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
  const cuuint32_t box[2] = {box_columns, box_rows}, unit[2] = {1, 1};
  return encode &&
         encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                reinterpret_cast<void*>(base), dims, strides, box, unit,
                CU_TENSOR_MAP_INTERLEAVE_NONE,
                box_columns == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Launch {
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  Launch(int clusters, int split, int threads, cudaStream_t st) : cfg(), attr() {
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * 2 * split));
    cfg.blockDim = dim3(threads);
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

template <bool kBf16, bool kTma, int kWide>
int launch(const Maps<kTma>& maps, const Args& a, int clusters, cudaStream_t st) {
  const auto fn = wgrad_kernel<kBf16, kTma, kWide>;
  if (!prepare(fn)) return ZERO_ECUDA;
  Launch l(clusters, a.split, Roles<kTma>::kThreads, st);
  return status_of(cudaLaunchKernelEx(&l.cfg, fn, maps, a));
}

// Clusters of `split` pairs that the device holds at once (0 on error): SMs
// come in groups that a cluster does not leave, so clusters of eight use fewer
// of them than pairs do.
int resident_clusters(int split) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices][kMaxSplit + 1];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return 0;
  int n = known[dev][split].load(std::memory_order_relaxed);
  if (n == 0) {
    const auto fn = wgrad_kernel<true, true, 1>;
    Launch l(1, split, Roles<true>::kThreads, nullptr);
    if (!prepare(fn) || cudaOccupancyMaxActiveClusters(&n, fn, &l.cfg) != cudaSuccess)
      return 0;
    known[dev][split].store(n, std::memory_order_relaxed);
  }
  return n;
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
  // TMA takes row distances below 2^40 bytes; off the grid eight rows are one
  constexpr int64_t kMostLd = int64_t{1} << 36;
  if (rows >= kMost || cols >= kMost || n >= kMost || ld >= kMostLd) return ZERO_ERANGE;
  if (cols == 0 || n == 0) return ZERO_OK;
  if (!dw || (rows && (!ckpt || !dy))) return ZERO_EINVAL;
  if (!aligned(ckpt, 16) || !aligned(dy, 2) || !aligned(dw, 2) || !aligned(d_scaler, 16))
    return ZERO_EALIGN;
  Args a = new_args<Args>();
  a.q = static_cast<const int8_t*>(ckpt);
  a.pitch = ceil_div(cols, ZERO_CKPT_PAD) * ZERO_CKPT_PAD;
  a.scale = static_cast<const uint8_t*>(ckpt) + rows * a.pitch;
  a.dy = static_cast<const uint16_t*>(dy);
  a.dw = static_cast<uint16_t*>(dw);
  a.scaler = d_scaler;
  a.rows = rows, a.cols = cols, a.n = n, a.ld = ld;
  a.vec_out = n % kVec == 0 && aligned(dw, 16);
  a.set_bounds(kCkpt, ckpt, 1, rows * (a.pitch + a.pitch / ZERO_CKPT_BLOCK), 0, 1);
  a.set_bounds(kDw, dw, cols, n, n, 2);
  int fit[kMaxSplit + 1];
  for (int split = 1; split <= kMaxSplit; split *= 2)
    fit[split] = resident_clusters(split);
  if (fit[1] <= 0) return ZERO_ECUDA;
  const int64_t pairs = fit[1], m_tiles = ceil_div(a.pitch, 2 * kM);
  const bool tma = rows > 0 && ld % kVec == 0 && aligned(dy, 16);
  // Tile width, column groups and split of the tokens by the cycles they take:
  // turns of all pairs times steps of 2 cycles per column, at least what filling
  // a stage takes; a tile put out alone at the end (two groups: every tile), and
  // the join of a split. A split needs room for all its clusters at once and
  // four steps in each part.
  const int64_t steps = ceil_div(rows, kK);
  int wide = 1;
  int64_t best = 0;
  for (int w = 1; w <= 2; ++w)
    for (int bn = kN; bn >= 128; bn -= 32)
      for (int split = 1; split <= (w == 1 ? kMaxSplit : 1); split *= 2) {
        const int64_t all = m_tiles * ceil_div(n, w * bn), turns = ceil_div(all, pairs);
        if (split > 1 && (all > fit[split] || steps < 4 * split)) break;
        if (split == kMaxSplit && bn > kM) break;
        const int64_t fill = tma ? kValueCycles : kPlaceCycles[w - 1];
        const int64_t cost =
            turns * ceil_div(steps, split) * std::max<int64_t>(2 * w * bn, fill) +
            (w == 2 ? turns : 1) * kOutCycles * w * bn + (split > 1 ? kJoinCycles : 0) +
            (split == kMaxSplit ? kBigClusterCycles + kPerBigCluster * all : 0);
        if (best == 0 || cost < best) {
          best = cost;
          a.bn = bn;
          a.split = split;
          wide = w;
        }
      }
  const int64_t tiles = m_tiles * ceil_div(n, wide * a.bn);
  if (tiles > 0x3fffffff) return ZERO_ERANGE;
  a.m_tiles = static_cast<int32_t>(m_tiles);
  a.tiles = static_cast<int32_t>(tiles);
  const int clusters = static_cast<int>(std::min(tiles, a.split > 1 ? tiles : pairs));
  const bool bf16 = dtype == ZERO_BF16;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const uintptr_t at = reinterpret_cast<uintptr_t>(dy);
  if (!tma) {
    Maps<false> maps = {};
    for (int64_t c = 0; c < kClasses && rows > 0; ++c) {
      const int64_t first = c < rows ? c : 0;
      const uintptr_t row = at + 2 * first * ld;
      if (!encode_rows(&maps.of[c], row & ~static_cast<uintptr_t>(15),
                       n + static_cast<int64_t>(row & 15) / 2, ceil_div(rows - first, kClasses),
                       kClasses * ld, kRawColumns, kK / kClasses, bf16))
        return ZERO_ECUDA;
    }
    if (wide == 2) return bf16 ? launch<true, false, 2>(maps, a, clusters, st)
                               : launch<false, false, 2>(maps, a, clusters, st);
    return bf16 ? launch<true, false, 1>(maps, a, clusters, st)
                : launch<false, false, 1>(maps, a, clusters, st);
  }
  Maps<true> maps = {};
  if (!encode_rows(&maps.of[0], at, n, rows, ld, 64, kK, bf16)) return ZERO_ECUDA;
  if (wide == 2) return bf16 ? launch<true, true, 2>(maps, a, clusters, st)
                             : launch<false, true, 2>(maps, a, clusters, st);
  return bf16 ? launch<true, true, 1>(maps, a, clusters, st)
              : launch<false, true, 1>(maps, a, clusters, st);
}

}  // extern "C"
