// tensor.cuh -- what the kernels on the 5th-generation tensor cores share:
// barriers with bounded waits, copies by TMA, sums out of tensor memory.
#ifndef ZERO_TENSOR_CUH
#define ZERO_TENSOR_CUH

#include <cuda.h>

#include "train.cuh"

namespace zt {

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

// A box of a 2-d map into this CTA; its bytes are counted by the barrier at
// `cluster_bar`, in this CTA or the other of the pair.
__device__ __forceinline__ void copy_box(void* dst, const CUtensorMap* map, int32_t x, int32_t y,
                                         uint32_t cluster_bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(cluster_bar)
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

// 32 lanes x 8 columns of tensor memory
__device__ __forceinline__ void read_eight(uint32_t addr, float (&f)[8]) {
  uint32_t r[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(addr)
      : "memory");
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(r[j]);
}

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::
          : "memory");
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

// Output rows off the 16-byte grid leave through shared memory, kOutCols columns
// of 32 rows at a time and eight lanes per row, in the whole blocks of their
// addresses (a lane storing its own row element by element wrote every 32-byte
// sector 16 times). A block may begin in the columns before: each row's stage
// starts with its last eight of those. Only the elements before a tile's first
// block and after its last go one by one.
constexpr int kOutCols = 64, kOutPitch = 16 + kOutCols * 2;

// columns [c, c + width) of the tile's row that starts at `to`, which has
// `count` columns; kTogether passes of four rows at a time
template <int kTogether>
__device__ __forceinline__ void store_staged(uint8_t* stage, uint16_t* to, int64_t n, int64_t rows,
                                             int c, int width, int count, int lane,
                                             const Bounds& in) {
  const int k = lane & 7, row0 = lane >> 3;
  const int end = c + width < count ? c + width : count;  // columns there are so far
#pragma unroll kTogether
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

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled encode_tiled() {
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

}  // namespace zt

#endif
