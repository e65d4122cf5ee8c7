/*
 * zero_block.h -- operators of a block of a trained model, next to those of
 * zero_train.h: dropout, the place where a block's output joins the residual
 * stream, and linear layers in 8-bit floating point.
 *
 *   dropout    from a counter: the mask is drawn again in the backward pass
 *              and never stored;
 *   join       norms after a block and before the next one, with the block's
 *              gate, dropout and residual scale between them, in one pass
 *              over the rows; its gradient, and those of the norms' and the
 *              gate's parameters into a gradient replica;
 *   fp8        forward product and input gradient of a linear layer on the
 *              tensor cores, with one power-of-two scale per block of 128
 *              (zero_ckpt_wgrad has the weight gradient).
 *
 * Why they are here: activations stay whole on every rank, so what a block
 * keeps of them counts; the norms' and gates' parameters lie in flat_params,
 * their gradients in a replica, like any other tensor's.
 *
 * Conventions are those of zero_train.h: int status, caller-owned memory,
 * asynchronous calls on the given stream, no device allocation; 16-bit arrays
 * need their element's alignment only, workspaces and 8-bit copies 16 bytes
 * (ZERO_EALIGN otherwise); `ld` is a row distance in elements, at least the row
 * length (ZERO_EINVAL); calls with no rows or no columns return ZERO_OK and
 * write only what is still defined (zeros for parameter gradients); buffers
 * must not overlap unless stated. Computed in fp32, rounded once per result;
 * the same bits every time.
 */
#ifndef ZERO_BLOCK_H
#define ZERO_BLOCK_H

#include "zero_train.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ----------------------------------------------------------------- dropout --
 *
 * Each element has 16 random bits r of its own, and stays where r >= T, with
 * T = min(floor(65536 p + 1/2), 65535): p counts in steps of 2^-16. What stays
 * is multiplied by 65536 / (65536 - T) (in fp32), so that the mean is kept
 * whatever p was rounded to; what does not stay is 0, infinities and NaN too.
 * The bits come from Philox 4x32 with 7 rounds (Salmon, Moraes, Dror and Shaw
 * 2011), key = seed (low word first), counter = (column / 8, row, call, step):
 * word (column % 8) / 2 of the result, its low half for even columns. They
 * depend on nothing else: not on ld, the type, the launch or the device.
 * step is read from d_step when the kernel runs (0 when NULL): a captured graph
 * that is replayed takes new masks as the word it points to (the scaler's t,
 * say) moves on. */
typedef struct zero_dropout_params {
  double p;               /* share of the elements left out, 0 <= p < 1 */
  uint64_t seed;
  uint32_t call;          /* which dropout of the step: layer, place, micro-batch, rank */
  const uint32_t* d_step; /* device memory, or NULL */
} zero_dropout_params;

/* out = round16(residual + dropout(x)); residual may be NULL (then nothing is
 * added). x has row distance ld; residual and out ld_out. out may be residual
 * itself, or x itself where ld equals ld_out. The gradient of x is this call on the
 * gradient of out, with the same params, without residual.
 * rows, cols < 2^31, rows times the row's blocks of 256 columns < 2^31
 * (ZERO_ERANGE). */
ZERO_API int zero_dropout(const zero_dropout_params* params, const void* x, const void* residual,
                          int64_t rows, int64_t cols, int64_t ld, int32_t dtype, void* out,
                          int64_t ld_out, void* stream);

/* -------------------------------------------------------------------- join --
 *
 * With norm(x) = x / sqrt(mean(x^2) + eps) (ZERO_NORM_RMS), or the same of
 * x - mean(x) (ZERO_NORM_LAYER), over the columns of a row:
 *
 *   n     = norm(y) * w_post + b_post   (y itself where w_post is NULL)
 *   b     = dropout(n)
 *   h_out = round16(stream_scale * h + branch_scale * gate * b)
 *   z     = round16(norm(h_out) * w_pre + b_pre)
 *
 * y is the block's output, h the residual stream, z what the next block reads.
 * Parameters are 16-bit vectors of cols elements (tensors in flat_params), each
 * NULL where it is not used: no gate is a gate of ones, b_post and b_pre belong
 * to ZERO_NORM_LAYER and need their w (ZERO_EINVAL otherwise). w_pre NULL: no z
 * (z must be NULL). Statistics are those of the stored h_out, so that the
 * gradient is that of what was computed. Sums are fp32: a row that is normalised
 * and holds an infinity or a NaN, or whose mean square plus eps passes fp32's range
 * (values past about 1e18; with eps 0 also a mean square below 2^-126, values
 * below about 1e-19, zeros among them), comes out NaN throughout (but for what
 * dropout leaves out of n), so that its step is skipped. A gate that is not finite
 * makes h_out infinite or NaN where dropout keeps n, and stream_scale * h where not.
 * rows < 2^31, cols <= ZERO_MAX_JOIN_COLS (ZERO_ERANGE). */
#define ZERO_MAX_JOIN_COLS 8192

typedef enum zero_norm { ZERO_NORM_RMS = 0, ZERO_NORM_LAYER = 1 } zero_norm;

typedef struct zero_join_params {
  int32_t norm;
  double eps;           /* 0, or a normal number of fp32 (2^-126 and more) */
  double stream_scale;  /* in fp32's range, as branch_scale */
  double branch_scale;
  zero_dropout_params drop; /* p = 0: none */
} zero_join_params;

/* For zero_block_join_grad's grads: where each gradient goes. */
typedef struct zero_join_weights {
  void* w_post;
  void* b_post;
  void* gate;
  void* w_pre;
  void* b_pre;
} zero_join_weights;

/* h, y, h_out, z: [rows, cols] with row distance ld. stats: fp32 [rows][4],
 * 16-byte aligned: mean and 1 / sqrt(.) of y, then of h_out (0 for what is not
 * there), for the gradient; may be NULL. h_out may be h or y itself, z y
 * itself (not both in one buffer). */
ZERO_API int zero_block_join(const zero_join_params* params, const zero_join_weights* weights,
                             const void* h, const void* y, int64_t rows, int64_t cols, int64_t ld,
                             int32_t dtype, void* h_out, void* z, float* stats, void* stream);

/* Bytes of the workspace zero_block_join_grad needs (0 on bad arguments, or
 * when there is nothing to do). Its contents mean nothing between calls; calls
 * that may run at the same time need one each. */
ZERO_API size_t zero_block_join_workspace_bytes(int64_t rows, int64_t cols);

/* The join's gradient, from h_out, y and stats of the forward call and the
 * gradients dz of z and dh_out of h_out (the stream's later uses; NULL: zero):
 *   D  = dh_out + d norm(h_out)/dh_out applied to dz * w_pre
 *   dh = round16(stream_scale * D)
 *   dy = round16(norm's gradient of dropout(branch_scale * gate * D) * w_post)
 * and, summed over the rows in fp32 and rounded once, the gradient of each
 * parameter given in weights, written to its place in grads (which is NULL
 * exactly where weights is; ZERO_EINVAL otherwise). dz is NULL exactly where
 * w_pre is. h_out may be NULL where w_pre is not given, y where neither w_post nor
 * gate is, stats where neither w_post nor w_pre is, workspace where no parameter is.
 * All [rows, cols] arrays have row distance ld. dh may be dh_out itself, dy dz
 * itself, or the other way round. */
ZERO_API int zero_block_join_grad(const zero_join_params* params, const zero_join_weights* weights,
                                  const void* h_out, const void* y, const float* stats,
                                  const void* dz, const void* dh_out, int64_t rows, int64_t cols,
                                  int64_t ld, int32_t dtype, void* dh, void* dy,
                                  const zero_join_weights* grads, void* workspace, void* stream);

/* --------------------------------------------------------------------- fp8 --
 *
 * An 8-bit copy holds numbers of the formats E4M3 (largest magnitude 448) or
 * E5M2 (57344), one power-of-two scale 2^k per block of ZERO_FP8_BLOCK: with
 * m the block's largest magnitude, k is the least whole number with
 * m <= largest * 2^k, at least -126 (0 for a block of zeros), and the element
 * x is held as x / 2^k rounded to the format, ties to even. Scale byte k + 127;
 * 255 for a block that holds an infinity or a NaN, which then stands for NaN
 * throughout. Blocks of activations and gradients are 128 columns of one row,
 * those of a weight 128 x 128, so that one copy serves both products.
 * The products' sums run over the exact products of what the copies stand for,
 * in fp32; where a factor's block is not finite, sums that it enters are NaN. */
#define ZERO_FP8_BLOCK 128

typedef enum zero_fp8_format { ZERO_E4M3 = 0, ZERO_E5M2 = 1 } zero_fp8_format;

/* Bytes of the copy of x [rows, cols]: rows of P = cols rounded up to 128 bytes
 * (zeros past cols), then the scale bytes in tiles of 512 bytes: tile
 * (r / 128) * ceil(P / 512) + b / 4 for row r and block b of the row, byte
 * 16 (r % 32) + 4 ((r % 128) / 32) + b % 4 of it. The rest of a tile is not
 * written. 0 on bad arguments (negative, or past 2^31). */
ZERO_API size_t zero_fp8_bytes(int64_t rows, int64_t cols);

/* x: 16-bit elements of type dtype, row distance ld. rows, cols < 2^31, rows
 * times the row's blocks of 256 columns < 2^31 (ZERO_ERANGE). */
ZERO_API int zero_fp8_quant(const void* x, int64_t rows, int64_t cols, int64_t ld, int32_t dtype,
                            int32_t format, void* copy, void* stream);

/* Bytes of the E4M3 copy of a weight [k, n]: k rows of P = n rounded up to 128
 * bytes (zeros past n), then two sets of scale tiles as above: one for the
 * columns as rows (n of them, blocks along k), one for the rows (k of them,
 * blocks along n). */
ZERO_API size_t zero_fp8_weight_bytes(int64_t k, int64_t n);

/* w: [k, n] 16-bit elements, rows contiguous (a tensor's place in flat_params). */
ZERO_API int zero_fp8_quant_weight(const void* w, int64_t k, int64_t n, int32_t dtype, void* copy,
                                   void* stream);

/* y = round16(x W) [rows, n] from x's copy [rows, k] and W's [k, n];
 * dx = round16(dy W^T) [rows, k] from dy's copy [rows, n] and W's. Sizes and
 * formats are those that the copies were made with. ld is the row distance of y, dx. Zeros
 * where the reduction is empty. A pipeline wait that expires (2 s) fills the
 * tiles that its cluster of CTAs had left with NaN and, when d_scaler is not
 * NULL, raises ZERO_DEVERR_TIMEOUT there.
 * Sums past the smallest normal fp32 number (2^-126) may come out 0.
 * rows, k, n < 2^30 (ZERO_ERANGE). */
ZERO_API int zero_fp8_linear(const void* x_copy, int32_t x_format, int64_t rows,
                             const void* w_copy, int64_t k, int64_t n, int32_t dtype, void* y,
                             int64_t ld, zero_scaler* d_scaler, void* stream);
ZERO_API int zero_fp8_linear_dgrad(const void* dy_copy, int32_t dy_format, int64_t rows,
                                   const void* w_copy, int64_t k, int64_t n, int32_t dtype,
                                   void* dx, int64_t ld, zero_scaler* d_scaler, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* ZERO_BLOCK_H */
