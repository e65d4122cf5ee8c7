/*
 * zero_train.h -- operators of a micro-batch's forward and backward pass that
 * stand next to the sharded step: what reads the 16-bit working parameters
 * (zero.h's flat_params) and what fills a gradient replica.
 *
 *   embedding   the lookup of token rows in a table inside flat_params, and
 *               the table's dense gradient written into its place in a
 *               gradient replica;
 *   checkpoints activations kept between the passes in 8 bits: written as
 *               they are made (alone or with the activation function), read
 *               back, and used in the backward pass by the activation's
 *               gradient and by a linear layer's weight gradient;
 *   loss        token log-probabilities, and the clipped policy loss with a
 *               KL term, with the gradient of the logits under the loss scale
 *               that zero_step divides out again.
 *
 * Why they are here: ZeRO divides the 16 bytes per parameter of model states
 * by N ("ZeRO stages 1, 2 and 3"); activations, the first and last layer's
 * gradients and the logits stay whole on every rank.
 *
 * Conventions are those of zero.h (int status, caller-owned memory,
 * asynchronous calls on the given stream, no device allocation), except that a
 * tensor inside a flat buffer starts at any element: pointers to 16-bit and
 * 32-bit elements need their element's alignment only, checkpoint buffers and
 * workspaces 16 bytes (ZERO_EALIGN otherwise). Rows that start on 16-byte
 * boundaries are moved as they are, others through 16-byte blocks that may
 * hold neighbouring elements, with the same results: a call may read the rest
 * of the block that holds a buffer's first or last element (any cudaMalloc'd
 * buffer covers it), and writes its own elements only. (The one exception:
 * dlogits whose rows lie otherwise on the 16-byte grid than the logits' are
 * written element by element.)
 * `ld` is the distance between the starts of two rows, in elements, at least
 * the row length (ZERO_EINVAL). Calls with no rows (or no elements) return
 * ZERO_OK and write only what the call still defines (the whole table's
 * gradient, the four statistics). Input and output buffers must not overlap
 * unless stated. Sums, softmax statistics and activation functions are
 * computed in fp32 and each result is rounded once to its type, to nearest
 * even. Results do not depend on the run: no floating-point atomics, sums in a
 * fixed order.
 */
#ifndef ZERO_TRAIN_H
#define ZERO_TRAIN_H

#include "zero.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Third element type, for logits (zero_dtype has the two 16-bit ones). */
#define ZERO_FP32 2

/* Largest vocabulary row the policy loss takes, in bytes: eight CTAs of a
 * cluster keep it in shared memory. */
#define ZERO_MAX_LOGIT_ROW_BYTES (8 * 192 * 1024)

/* --------------------------------------------------------------- embedding --
 *
 * tokens: n_tokens token ids, int32 or int64 (token_bytes 4 or 8). An id
 * outside [0, vocab) is padding: its output row is zeros and it takes no part
 * in the gradient. n_tokens <= 2^28, vocab <= 2^24, dim <= 2^28 (ZERO_ERANGE).
 * table: [vocab, dim] 16-bit elements, rows contiguous.
 *   out[t, :] = round16(scale * table[tokens[t], :])                          */
ZERO_API int zero_embedding(const void* tokens, int32_t token_bytes, int64_t n_tokens,
                            const void* table, int64_t vocab, int64_t dim, float scale,
                            int32_t dtype, void* out, void* stream);

/* Bytes of the workspace zero_embedding_grad needs (0 on bad arguments). Its
 * contents need no initialisation and mean nothing between calls. */
ZERO_API size_t zero_embedding_workspace_bytes(int64_t n_tokens, int64_t vocab, int64_t dim);

/* Gradient of the table from the gradient dy [n_tokens, dim] of the lookup's
 * output:
 *   grad[v, :] = round16(scale * sum over t with tokens[t] == v of dy[t, :])
 * accumulate = 0: every row of grad [vocab, dim] is written, zeros where no
 *   token names it (a replica is dense);
 * accumulate = 1: the sum is added to the row's present value in fp32 and
 *   rounded once; rows that no token names are left alone (a table tied to the
 *   output layer, whose gradient is already there).
 * Tokens are sorted by id first, equal ids in the order of their positions;
 * the rows of dy are summed in that order, in runs whose bounds depend on the
 * ids alone. The workspace holds two fp32 rows for every 32 rows of the table
 * and tokens together, whether or not tokens fall there. */
ZERO_API int zero_embedding_grad(const void* tokens, int32_t token_bytes, int64_t n_tokens,
                                 const void* dy, int64_t vocab, int64_t dim, float scale,
                                 int32_t dtype, int32_t accumulate, void* grad,
                                 void* workspace, void* stream);

/* ------------------------------------------------------------- checkpoints --
 *
 * A checkpoint of x [rows, cols] is one buffer of zero_ckpt_bytes(rows, cols)
 * bytes: rows of P = cols rounded up to ZERO_CKPT_PAD int8 values (zeros past
 * cols), then rows of P / ZERO_CKPT_BLOCK scale bytes. Each block of
 * ZERO_CKPT_BLOCK values along a row has one power-of-two step 2^k:
 *   k = max(floor(log2(max |x|)) - 6, k_min), k_min = -24 (fp16), -126 (bf16);
 *   q = min(max(round(x / 2^k), -127), 127), ties to even;
 *   scale byte = k + 127; a block of zeros has k = k_min.
 * A block that holds an infinity or a NaN has scale byte 255 and reads back
 * as NaN throughout, so an overflowed activation still ends in a skipped step.
 * The value it stands for, q * 2^k, is exact in the 16-bit type: reading it
 * back never rounds. The error is at most half a step, a full one where
 * |x| > 127 steps: 2^-7 of the block's largest magnitude.
 * rows times the row's blocks of 256 columns < 2^31 (ZERO_ERANGE), but for the
 * weight gradient.                                                           */
#define ZERO_CKPT_BLOCK 32
#define ZERO_CKPT_PAD 128

/* 0 on bad arguments (rows or cols negative, or a size past 2^62). */
ZERO_API size_t zero_ckpt_bytes(int64_t rows, int64_t cols);

/* Write the checkpoint of x (16-bit elements of type dtype). */
ZERO_API int zero_ckpt_save(const void* x, int64_t rows, int64_t cols, int64_t ld, int32_t dtype,
                            void* ckpt, void* stream);

/* Read a checkpoint back into 16-bit elements. dtype is the type it was saved
 * from. */
ZERO_API int zero_ckpt_load(const void* ckpt, int64_t rows, int64_t cols, int32_t dtype,
                            void* out, int64_t ld, void* stream);

typedef enum zero_act {
  ZERO_ACT_GELU = 0,   /* x/2 (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3))) */
  ZERO_ACT_SWIGLU = 1  /* x / (1 + exp(-x)) * u */
} zero_act;

/* Activation function and checkpoint of its inputs in one pass: y = f(x) (or
 * f(x, u)), from the inputs themselves; ckpt_x (and ckpt_u) as zero_ckpt_save
 * writes them. x, u: [rows, cols] with row distance ld; y with ld_y. u and
 * ckpt_u are NULL for ZERO_ACT_GELU (ZERO_EINVAL otherwise). */
ZERO_API int zero_ckpt_act(int32_t act, const void* x, const void* u, int64_t rows, int64_t cols,
                           int64_t ld, int32_t dtype, void* y, int64_t ld_y, void* ckpt_x,
                           void* ckpt_u, void* stream);

/* The activation's gradient from the checkpoints, with dy [rows, cols] (row
 * distance ld_dy): dx = dy * df/dx, du = dy * df/du (NULL for ZERO_ACT_GELU)
 * at the checkpointed values. y, when not NULL, receives f of the checkpointed
 * values again (the next linear layer's weight gradient needs it). dx, du and
 * y have row distance ld; dx or du may be dy itself (with ld equal to ld_dy). */
ZERO_API int zero_ckpt_act_grad(int32_t act, const void* ckpt_x, const void* ckpt_u,
                                const void* dy, int64_t rows, int64_t cols, int64_t ld_dy,
                                int32_t dtype, void* dx, void* du, void* y, int64_t ld,
                                void* stream);

/* Weight gradient of a linear layer y = x W, W [cols, n], from x's checkpoint
 * and dy [rows, n] (row distance ld):
 *   dw[i, j] = round16(sum over t of x^[t, i] * dy[t, j])
 * on the tensor cores, accumulated in fp32; dw is [cols, n] contiguous (a
 * tensor's place in a gradient replica) and written whole (zeros when rows is
 * 0). A pipeline wait that expires (2 s) fills the tiles that its cluster of
 * CTAs had left with NaN and, when d_scaler is not NULL, raises
 * ZERO_DEVERR_TIMEOUT there.
 * rows, cols, n < 2^31, ld < 2^36 (ZERO_ERANGE). */
ZERO_API int zero_ckpt_wgrad(const void* ckpt, int64_t rows, int64_t cols, const void* dy,
                             int64_t n, int64_t ld, int32_t dtype, void* dw,
                             zero_scaler* d_scaler, void* stream);

/* -------------------------------------------------------------------- loss --
 *
 * A pipeline wait that expires (2 s) makes the rows that its CTAs had left
 * NaN; it raises no error word.
 *
 * logits: [rows, vocab], row distance ld, of type dtype (ZERO_BF16, ZERO_FP16
 * or ZERO_FP32), rows and ld <= 2^31 (ZERO_ERANGE). -inf entries are tokens
 * ruled out (probability 0); a row of nothing but -inf, or one with a NaN or
 * +inf, has logp NaN. Finite values of any size are logits like others (a mask
 * of the type's lowest value among them).
 * actions: the tokens taken, int32 or int64 (action_bytes 4 or 8).
 *   logp[t] = logits[t, a_t] - log(sum over j of exp(logits[t, j]))
 * An action outside [0, vocab) leaves its row out: logp 0. A row may have at
 * most 2^30 bytes (ZERO_ERANGE).                                             */
ZERO_API int zero_token_logp(const void* logits, int64_t rows, int64_t vocab, int64_t ld,
                             int32_t dtype, const void* actions, int32_t action_bytes,
                             float* logp, void* stream);

typedef struct zero_policy_params {
  double clip_lo;  /* ratio is clipped to [1 - clip_lo, 1 + clip_hi], 0 <= clip_lo < 1 */
  double clip_hi;  /* >= 0 */
  double kl_coef;  /* beta >= 0 */
} zero_policy_params;

/* Clipped policy loss with a KL term, and its gradient, in one pass over the
 * logits. Per token, with lp = logp[t], A = advantage[t], w = weight[t]:
 *   r = exp(lp - old_logp[t]),   d = ref_logp[t] - lp
 *   loss[t] = -min(r A, clip(r) A) + beta (exp(d) - d - 1)
 *   dloss/dlp = -r A where r A <= clip(r) A, else 0;  + beta (1 - exp(d))
 *   dlogits[t, j] = S w dloss/dlp ([j == a_t] - exp(logits[t, j] - lse_t))
 * S is the loss scale in d_scaler (1 when d_scaler is NULL), so that the
 * gradient replicas hold S times the gradient as zero_step expects. A weight
 * of 0 (a prompt token, padding) or an action outside [0, vocab) leaves the
 * row out: its logits are not read, logp and loss are 0 and dlogits are 0.
 * ref_logp may be NULL: no KL term, its sum in stats is 0 (with kl_coef 0 it
 * is only reported there). dlogits may be the logits buffer itself.
 * logp, loss (fp32 [rows]) are always written; dlogits [rows, vocab] with the
 * logits' type and row distance; stats, when not NULL, receives
 *   { sum w loss, sum w (exp(d) - d - 1), sum w [clipped], sum w }
 * over the rows that are not left out.
 * A row may have at most ZERO_MAX_LOGIT_ROW_BYTES (ZERO_ERANGE). */
ZERO_API int zero_policy_loss(const void* logits, int64_t rows, int64_t vocab, int64_t ld,
                              int32_t dtype, const void* actions, int32_t action_bytes,
                              const float* old_logp, const float* ref_logp,
                              const float* advantage, const float* weight,
                              const zero_policy_params* params, const zero_scaler* d_scaler,
                              float* logp, float* loss, float* stats, void* dlogits,
                              void* stream);

/* --------------------------------------------------------------- self-test --
 *
 * Checked build (libzero_checked.so) only; ZERO_ESTATE in the release build.
 * Plants a mistake in the calls that follow in this process, until it is
 * called with ZERO_PLANT_NOTHING; a wait then expires after limit_ns (1 to
 * 10^9, ZERO_EINVAL otherwise) in place of 2 s. Nothing faults or hangs: the
 * kernels give up as they do after any wait that expires.
 *   ZERO_PLANT_NO_COPY  zero_ckpt_wgrad: the first CTA leaves out the copy of
 *                       its step `at`; zero_policy_loss: the first part of
 *                       row `at` is not copied
 *   ZERO_PLANT_NO_SEND  zero_token_logp, zero_policy_loss: the second CTA of
 *                       a cluster does not send its sums of row `at`
 *   ZERO_PLANT_SHORT    the range checks take buffer `at` of a call for one
 *                       element shorter than it is, so that the access to its
 *                       last element is a violation (zero_checked_status) and
 *                       left out. Buffers by call: zero_embedding table, out;
 *                       zero_embedding_grad dy, grad, partial sums, rows that
 *                       span runs (the last two: taken for empty); zero_ckpt_* but wgrad x, u, dy, y (out of
 *                       load), dx, du, ckpt_x, ckpt_u; zero_ckpt_wgrad ckpt,
 *                       dw; loss logits, dlogits */
typedef enum zero_plant {
  ZERO_PLANT_NOTHING = 0,
  ZERO_PLANT_NO_COPY = 1,
  ZERO_PLANT_NO_SEND = 2,
  ZERO_PLANT_SHORT = 3
} zero_plant;
ZERO_API int zero_selftest_plant(int32_t what, int64_t at, int64_t limit_ns);

#ifdef __cplusplus
}
#endif
#endif /* ZERO_TRAIN_H */
