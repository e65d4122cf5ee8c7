/*
 * ckpt.cu -- 8-bit activation checkpoints: writing, reading back, and the
 * activation functions that make and use them (zero_train.h).
 *
 * One value in 32 shares a power-of-two step 2^k with its block: with
 * 2^E <= max|x| < 2^(E+1), k = E - 6, so |x| / 2^k < 128 and q = rint(x / 2^k)
 * fits 8 bits (127.5 and more is held at 127). Multiplying by a power of two
 * is exact, so q * 2^k is exact in bf16 (8 significant bits) and fp16, and no
 * reader of a checkpoint rounds it.
 *
 * All kernels here are bound by memory. A thread moves 8 neighbouring elements
 * (16 bytes of the 16-bit side, 8 of the checkpoint), so four lanes share a
 * block and its maximum takes two shuffles; a warp covers 256 columns of a
 * row, the warps of a CTA neighbouring columns, running on into the next row.
 * Measured on SwiGLU both ways, 8192 x 8192: 201 us, 89 % of copy bandwidth; a
 * CTA of eight rows by 256 columns took 206, two rows per warp 204.
 */
#include "rows.cuh"

#include <algorithm>

namespace zc {

using namespace zt;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

// a call's buffers, for their bounds
enum { kX, kU, kDy, kY, kDx, kDu, kCkptX, kCkptU, kBuffers };

struct Ckpt {
  int8_t* q;       // [rows][pitch]
  uint8_t* scale;  // [rows][pitch / 32]
};

// x held in [-limit, limit], pairs of 16-bit values
template <bool kBf16>
__device__ __forceinline__ uint32_t hold2(uint32_t x, uint32_t limit, uint32_t minus_limit) {
  if constexpr (kBf16)
    asm("{\n .reg .b32 t;\n min.bf16x2 t, %1, %2;\n max.bf16x2 %0, t, %3;\n}"
        : "=r"(x)
        : "r"(x), "r"(limit), "r"(minus_limit));
  else
    asm("{\n .reg .b32 t;\n min.f16x2 t, %1, %2;\n max.f16x2 %0, t, %3;\n}"
        : "=r"(x)
        : "r"(x), "r"(limit), "r"(minus_limit));
  return x;
}

// Quantise the lane's eight values v with its block's other three lanes and
// store them; all lanes of the warp call it. `in` is false past the pitch.
// q = rint(x / 2^k) falls out of one fused multiply-add: added to 1.5 2^23, the
// quotient is rounded to a whole number, ties to even, in the sum's last bits.
template <bool kBf16>
__device__ __forceinline__ void save8(const Ckpt& k, int64_t row, int64_t c, int64_t pitch,
                                      bool in, const uint4& v, const Bounds& bounds) {
  constexpr uint32_t kAbs = 0x7FFF7FFFu;
  uint32_t top = max_u16x2(max_u16x2(v.x & kAbs, v.y & kAbs), max_u16x2(v.z & kAbs, v.w & kAbs));
  top = max_u16x2(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max_u16x2(top, __shfl_xor_sync(0xffffffffu, top, 2));
  top = max(top & 0xFFFFu, top >> 16);
  const bool finite = top < (kBf16 ? 0x7F80u : 0x7C00u);
  // biased exponent of 2^k, from that of the maximum (0 for zero and, in bf16,
  // the subnormals), and of the largest magnitude kept, 127 2^k = 2^(k+6) 1.984375
  uint32_t step, limit;
  if constexpr (kBf16) {
    step = max(static_cast<int>(top >> 7) - 6, 1);
    limit = ((step + 6) << 7 | 0x7Eu) * 0x10001u;
  } else {
    step = max(static_cast<int>(__float_as_uint(widen<false>(top)) >> 23) - 6, 103);
    const float most = __uint_as_float((step + 6) << 23 | 0x7E0000u);
    limit = narrow2<false>(most, most);
  }
  const uint32_t minus = limit | 0x80008000u;
  const float inv = __uint_as_float((254 - step) << 23);
  const Pair inv2 = pair(inv, inv), magic = pair(12582912.f, 12582912.f);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t q[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float a, b;
    widen2<kBf16>(hold2<kBf16>(w[j], limit, minus), a, b);
    unpair(fma2(pair(a, b), inv2, magic), a, b);
    q[2 * j] = __float_as_uint(a);
    q[2 * j + 1] = __float_as_uint(b);
  }
  if (!in) return;
  const auto low_bytes = [](uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
  };
  uint2 out = make_uint2(low_bytes(q[0], q[1], q[2], q[3]), low_bytes(q[4], q[5], q[6], q[7]));
  if (!finite) out = make_uint2(0, 0);
  if (bounds.holds(k.q + row * pitch + c, kVec, kSiteStore))
    __stcs(reinterpret_cast<uint2*>(k.q + row * pitch + c), out);
  if ((threadIdx.x & 3) == 0) {
    uint8_t* scale = k.scale + row * (pitch / ZERO_CKPT_BLOCK) + c / ZERO_CKPT_BLOCK;
    if (bounds.holds(scale, 1, kSiteStore)) *scale = static_cast<uint8_t>(finite ? step : 255);
  }
}

// The lane's eight checkpointed values. A byte with its sign bit
// turned over is value + 128; under the exponent of 2^23 it is that much more
// than 2^23, which one addition takes off.
__device__ __forceinline__ void unpack8(const uint2& w, uint32_t scale, float (&f)[8]) {
  const float s = scale == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float(scale << 23);
  const Pair step = pair(s, s), bias = pair(-8388736.f, -8388736.f);
  const uint32_t x[2] = {w.x ^ 0x80808080u, w.y ^ 0x80808080u};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t at = x[j >> 1];
    const float a = __uint_as_float(__byte_perm(at, 0x4B000000u, j & 1 ? 0x7442 : 0x7440));
    const float b = __uint_as_float(__byte_perm(at, 0x4B000000u, j & 1 ? 0x7443 : 0x7441));
    unpair((pair(a, b) + bias) * step, f[2 * j], f[2 * j + 1]);
  }
}

// p = 1 / (1 + exp(-z)) and q = 1 - p, from exp(-|z|): nothing overflows, and
// both keep their relative accuracy down into the subnormal numbers.
struct Gate {
  float p, q;
};

__device__ __forceinline__ Gate sigmoid(float z) {
  // exp(-|z|) as a square: its root stays normal down to |z| = 174
  const float root = exp2_fast(fabsf(z) * -0.72134752044f);  // -log2(e) / 2
  const float t = root * root, sum = 1.f + t;
  float big;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(big) : "f"(sum));  // sum in [1, 2]
  const float small = t * big;
  return z >= 0.f ? Gate{big, small} : Gate{small, big};
}

// GELU's tanh form is x p(z) with z = 2 sqrt(2/pi) (x + 0.044715 x^3).
constexpr float kGeluC = 1.5957691216057308f;  // 2 sqrt(2/pi)
constexpr float kGeluA = 0.044715f;

// held below overflow, so that p q z' is 0 and not 0 * inf far out
__device__ __forceinline__ float square(float x) { return fminf(x * x, 1e30f); }

__device__ __forceinline__ Gate gelu_gate(float x) {
  return sigmoid(kGeluC * __fmaf_rn(kGeluA * square(x), x, x));
}

struct Args : Checked<kBuffers> {
  const uint16_t *x, *u, *dy;
  uint16_t *y, *dx, *du;
  Ckpt kx, ku;
  int64_t rows, cols, pitch, ld, ld_y;  // ld: x, u (forward), dx, du, y (backward)
  uint32_t col_tiles;
};

enum Op { kSave, kLoad, kGelu, kSwiglu, kGeluGrad, kSwigluGrad };

template <int kOp, bool kBf16, bool kGrid>
__global__ void __launch_bounds__(kThreads) ckpt_kernel(const Args a) {
  pdl_begin();
  __shared__ __align__(16) uint8_t stages[kGrid ? 1 : kWarps][kGrid ? 16 : kStageWarp];
  uint8_t* stage = stages[kGrid ? 0 : threadIdx.x >> 5];
  const int lane = threadIdx.x & 31;
  // the CTA's warps take neighbouring column tiles, running on into the next rows
  const uint32_t tile = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const uint32_t row = tile / a.col_tiles;
  const int64_t c0 = static_cast<int64_t>(tile - row * a.col_tiles) * kCols, c = c0 + lane * kVec;
  const int64_t r = row;
  if (r >= a.rows) return;
  const bool in = c < a.pitch;
  if constexpr (kOp == kSave || kOp == kGelu || kOp == kSwiglu) {
    const uint4 vx = load8<kGrid>(a.x + r * a.ld, c, a.cols, a.bounds(kX));
    uint4 vu = make_uint4(0, 0, 0, 0);
    if constexpr (kOp == kSwiglu) vu = load8<kGrid>(a.u + r * a.ld, c, a.cols, a.bounds(kU));
    save8<kBf16>(a.kx, r, c, a.pitch, in, vx, a.bounds(kCkptX));
    if constexpr (kOp == kSwiglu)
      save8<kBf16>(a.ku, r, c, a.pitch, in, vu, a.bounds(kCkptU));
    if constexpr (kOp != kSave) {
      float x[8], u[8], y[8];
      widen8<kBf16>(vx, x);
      if constexpr (kOp == kSwiglu) widen8<kBf16>(vu, u);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        y[j] = kOp == kSwiglu ? x[j] * sigmoid(x[j]).p * u[j] : x[j] * gelu_gate(x[j]).p;
      store_row<kGrid>(stage, a.y + r * a.ld_y, c0, lane, a.cols, narrow8<kBf16>(y),
                       a.bounds(kY));
    }
  } else {
    const int64_t blk = a.pitch / ZERO_CKPT_BLOCK;
    uint2 qx = make_uint2(0, 0), qu = qx;
    uint32_t sx = 1, su = 1;
    uint4 vd = make_uint4(0, 0, 0, 0);
    if (in) {
      const uint8_t* scale = a.kx.scale + r * blk + c / ZERO_CKPT_BLOCK;
      if (a.bounds(kCkptX).holds(a.kx.q + r * a.pitch + c, kVec, kSiteLoad) &&
          a.bounds(kCkptX).holds(scale, 1, kSiteLoad)) {
        qx = __ldcs(reinterpret_cast<const uint2*>(a.kx.q + r * a.pitch + c));
        sx = a.kx.scale[r * blk + c / ZERO_CKPT_BLOCK];
      }
      if constexpr (kOp == kSwigluGrad) {
        scale = a.ku.scale + r * blk + c / ZERO_CKPT_BLOCK;
        if (a.bounds(kCkptU).holds(a.ku.q + r * a.pitch + c, kVec, kSiteLoad) &&
            a.bounds(kCkptU).holds(scale, 1, kSiteLoad)) {
          qu = __ldcs(reinterpret_cast<const uint2*>(a.ku.q + r * a.pitch + c));
          su = a.ku.scale[r * blk + c / ZERO_CKPT_BLOCK];
        }
      }
      if constexpr (kOp != kLoad)
        vd = load8<kGrid>(a.dy + r * a.ld_y, c, a.cols, a.bounds(kDy));
    }
    float x[8], u[8], d[8], y[8], gx[8], gu[8];
    unpack8(qx, sx, x);
    if constexpr (kOp == kLoad) {
      store_row<kGrid>(stage, a.y + r * a.ld, c0, lane, a.cols, narrow8<kBf16>(x), a.bounds(kY));
    } else {
      if constexpr (kOp == kSwigluGrad) unpack8(qu, su, u);
      widen8<kBf16>(vd, d);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (kOp == kSwigluGrad) {
          // y = x p u, p = p(x): dy/dx = u p (1 + x q), dy/du = x p
          const Gate g = sigmoid(x[j]);
          const float xp = x[j] * g.p;
          y[j] = xp * u[j];
          gu[j] = d[j] * xp;
          gx[j] = d[j] * u[j] * (g.p * __fmaf_rn(x[j], g.q, 1.f));
        } else {
          // y = x p(z), z' = c (1 + 3 a x^2): dy/dx = p + x p q z'
          const Gate g = gelu_gate(x[j]);
          y[j] = x[j] * g.p;
          const float z1 = kGeluC * __fmaf_rn(3.f * kGeluA, square(x[j]), 1.f);
          gx[j] = d[j] * __fmaf_rn(y[j] * g.q, z1, g.p);
        }
      }
      store_row<kGrid>(stage, a.dx + r * a.ld, c0, lane, a.cols, narrow8<kBf16>(gx),
                       a.bounds(kDx));
      if constexpr (kOp == kSwigluGrad)
        store_row<kGrid>(stage, a.du + r * a.ld, c0, lane, a.cols, narrow8<kBf16>(gu),
                         a.bounds(kDu));
      if (a.y)
        store_row<kGrid>(stage, a.y + r * a.ld, c0, lane, a.cols, narrow8<kBf16>(y),
                         a.bounds(kY));
    }
  }
}

constexpr int64_t kMaxTiles = 0x7fffffff;  // rows x column tiles
constexpr int64_t kMaxBytes = int64_t{1} << 62;

int64_t pitch_of(int64_t cols) { return ceil_div(cols, ZERO_CKPT_PAD) * ZERO_CKPT_PAD; }

bool sizes_ok(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0 || cols > kMaxBytes / 4) return false;
  const int64_t p = pitch_of(cols);
  return p == 0 || rows <= kMaxBytes / 2 / p;
}

Ckpt ckpt_of(const void* p, int64_t rows, int64_t pitch) {
  int8_t* q = static_cast<int8_t*>(const_cast<void*>(p));
  return Ckpt{q, reinterpret_cast<uint8_t*>(q) + rows * pitch};
}

// ld: of all 16-bit arrays but ld_y's, y's (forward) or dy's (backward)
template <int kOp>
void bound_buffers(Args& a) {
  constexpr bool kBack = kOp == kGeluGrad || kOp == kSwigluGrad;
  const auto array = [&](int k, const void* p, int64_t ld) {
    a.set_bounds(k, p, a.rows, a.cols, ld, 2);
  };
  array(kX, a.x, a.ld), array(kU, a.u, a.ld), array(kDy, a.dy, a.ld_y);
  array(kY, a.y, kBack || kOp == kLoad ? a.ld : a.ld_y), array(kDx, a.dx, a.ld);
  array(kDu, a.du, a.ld);
  const int64_t bytes = a.rows * (a.pitch + a.pitch / ZERO_CKPT_BLOCK);
  a.set_bounds(kCkptX, a.kx.q, 1, bytes, 0, 1);
  a.set_bounds(kCkptU, a.ku.q, 1, bytes, 0, 1);
}

template <int kOp>
int launch(Args& a, int32_t dtype, bool on_grid, void* stream) {
  bound_buffers<kOp>(a);
  const int64_t col_tiles = ceil_div(a.pitch, kCols);
  if (col_tiles > kMaxTiles || a.rows > kMaxTiles / col_tiles) return ZERO_ERANGE;
  a.col_tiles = static_cast<uint32_t>(col_tiles);
  const auto fn = dtype == ZERO_BF16
                      ? (on_grid ? ckpt_kernel<kOp, true, true> : ckpt_kernel<kOp, true, false>)
                      : (on_grid ? ckpt_kernel<kOp, false, true> : ckpt_kernel<kOp, false, false>);
  return status_of(launch_pdl(fn, dim3(static_cast<unsigned>(ceil_div(a.rows * col_tiles, kWarps))),
                              dim3(kThreads), 0, static_cast<cudaStream_t>(stream), a));
}

}  // namespace zc

#ifdef ZERO_CHECKED
namespace zt {
static Plant g_plant = {ZERO_PLANT_NOTHING, 0, kWaitLimitNs};
Plant planted() { return g_plant; }
}  // namespace zt

extern "C" int zc_collect_checks(unsigned long long* count, unsigned long long* first) {
  return collect_checks(count, first);
}
#endif

extern "C" {

ZERO_API size_t zero_ckpt_bytes(int64_t rows, int64_t cols) {
  if (!zc::sizes_ok(rows, cols)) return 0;
  const int64_t p = zc::pitch_of(cols);
  return static_cast<size_t>(rows * (p + p / ZERO_CKPT_BLOCK));
}

ZERO_API int zero_ckpt_save(const void* x, int64_t rows, int64_t cols, int64_t ld, int32_t dtype,
                            void* ckpt, void* stream) {
  using namespace zc;
  if (!sizes_ok(rows, cols) || !is_dtype16(dtype) || ld < cols) return ZERO_EINVAL;
  if (rows == 0 || cols == 0) return ZERO_OK;
  if (!x || !ckpt) return ZERO_EINVAL;
  if (!aligned(x, 2) || !aligned(ckpt, 16)) return ZERO_EALIGN;
  Args a = new_args<Args>();
  a.x = static_cast<const uint16_t*>(x);
  a.rows = rows, a.cols = cols, a.pitch = pitch_of(cols), a.ld = ld;
  a.kx = ckpt_of(ckpt, rows, a.pitch);
  return launch<kSave>(a, dtype, on_grid(x, ld), stream);
}

ZERO_API int zero_ckpt_load(const void* ckpt, int64_t rows, int64_t cols, int32_t dtype,
                            void* out, int64_t ld, void* stream) {
  using namespace zc;
  if (!sizes_ok(rows, cols) || !is_dtype16(dtype) || ld < cols) return ZERO_EINVAL;
  if (rows == 0 || cols == 0) return ZERO_OK;
  if (!out || !ckpt) return ZERO_EINVAL;
  if (!aligned(out, 2) || !aligned(ckpt, 16)) return ZERO_EALIGN;
  Args a = new_args<Args>();
  a.y = static_cast<uint16_t*>(out);
  a.rows = rows, a.cols = cols, a.pitch = pitch_of(cols), a.ld = ld;
  a.kx = ckpt_of(ckpt, rows, a.pitch);
  return launch<kLoad>(a, dtype, on_grid(out, ld), stream);
}

ZERO_API int zero_ckpt_act(int32_t act, const void* x, const void* u, int64_t rows, int64_t cols,
                           int64_t ld, int32_t dtype, void* y, int64_t ld_y, void* ckpt_x,
                           void* ckpt_u, void* stream) {
  using namespace zc;
  if (act != ZERO_ACT_GELU && act != ZERO_ACT_SWIGLU) return ZERO_EINVAL;
  if (!sizes_ok(rows, cols) || !is_dtype16(dtype) || ld < cols || ld_y < cols) return ZERO_EINVAL;
  const bool gated = act == ZERO_ACT_SWIGLU;
  if (!gated && (u || ckpt_u)) return ZERO_EINVAL;
  if (rows == 0 || cols == 0) return ZERO_OK;
  if (!x || !y || !ckpt_x || (gated && (!u || !ckpt_u))) return ZERO_EINVAL;
  if (!aligned(x, 2) || !aligned(u, 2) || !aligned(y, 2) || !aligned(ckpt_x, 16) ||
      !aligned(ckpt_u, 16))
    return ZERO_EALIGN;
  Args a = new_args<Args>();
  a.x = static_cast<const uint16_t*>(x);
  a.u = static_cast<const uint16_t*>(u);
  a.y = static_cast<uint16_t*>(y);
  a.rows = rows, a.cols = cols, a.pitch = pitch_of(cols), a.ld = ld, a.ld_y = ld_y;
  a.kx = ckpt_of(ckpt_x, rows, a.pitch);
  if (gated) a.ku = ckpt_of(ckpt_u, rows, a.pitch);
  const bool align = on_grid(x, ld) && on_grid(u, ld) && on_grid(y, ld_y);
  return gated ? launch<kSwiglu>(a, dtype, align, stream) : launch<kGelu>(a, dtype, align, stream);
}

ZERO_API int zero_ckpt_act_grad(int32_t act, const void* ckpt_x, const void* ckpt_u,
                                const void* dy, int64_t rows, int64_t cols, int64_t ld_dy,
                                int32_t dtype, void* dx, void* du, void* y, int64_t ld,
                                void* stream) {
  using namespace zc;
  if (act != ZERO_ACT_GELU && act != ZERO_ACT_SWIGLU) return ZERO_EINVAL;
  if (!sizes_ok(rows, cols) || !is_dtype16(dtype) || ld < cols || ld_dy < cols) return ZERO_EINVAL;
  const bool gated = act == ZERO_ACT_SWIGLU;
  if (!gated && (du || ckpt_u)) return ZERO_EINVAL;
  if (rows == 0 || cols == 0) return ZERO_OK;
  if (!ckpt_x || !dy || !dx || (gated && (!ckpt_u || !du))) return ZERO_EINVAL;
  if ((dx == dy || du == dy) && ld != ld_dy) return ZERO_EINVAL;
  if (!aligned(dy, 2) || !aligned(dx, 2) || !aligned(du, 2) || !aligned(y, 2) ||
      !aligned(ckpt_x, 16) || !aligned(ckpt_u, 16))
    return ZERO_EALIGN;
  Args a = new_args<Args>();
  a.dy = static_cast<const uint16_t*>(dy);
  a.dx = static_cast<uint16_t*>(dx);
  a.du = static_cast<uint16_t*>(du);
  a.y = static_cast<uint16_t*>(y);
  a.rows = rows, a.cols = cols, a.pitch = pitch_of(cols), a.ld = ld, a.ld_y = ld_dy;
  a.kx = ckpt_of(ckpt_x, rows, a.pitch);
  if (gated) a.ku = ckpt_of(ckpt_u, rows, a.pitch);
  const bool align =
      on_grid(dy, ld_dy) && on_grid(dx, ld) && on_grid(du, ld) && on_grid(y, ld);
  return gated ? launch<kSwigluGrad>(a, dtype, align, stream)
               : launch<kGeluGrad>(a, dtype, align, stream);
}

ZERO_API int zero_selftest_plant(int32_t what, int64_t at, int64_t limit_ns) {
  if (what < ZERO_PLANT_NOTHING || what > ZERO_PLANT_SHORT || limit_ns < 1 ||
      limit_ns > 1000000000)
    return ZERO_EINVAL;
#ifdef ZERO_CHECKED
  const bool wait = what == ZERO_PLANT_NO_COPY || what == ZERO_PLANT_NO_SEND;
  zt::g_plant = {what, at, wait ? static_cast<uint64_t>(limit_ns) : zt::kWaitLimitNs};
  return ZERO_OK;
#else
  (void)at;
  return ZERO_ESTATE;
#endif
}

}  // extern "C"
