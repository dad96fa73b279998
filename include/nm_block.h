/*
 * nm_block.h -- C ABI of libnmsparse.so for what a transformer block does around its sparse
 * products on AMD Instinct MI355X (gfx950): the products with their bias, activation, scale and
 * residual, the gated feed-forward's two products as one, the norms before and after a block
 * with the residual addition between them, and the log probabilities of its answers.
 *
 * A block: nm_block_norm joins the last branch to the residual stream and normalises it;
 * nm_linear gives q, k and v (nm_decode.h turns, caches and attends); nm_linear projects the
 * attention's output; nm_block_norm; nm_gated; nm_linear. After the last block's norm and the
 * vocabulary's product, nm_logprobs scores given tokens.
 *
 * Conventions: those of nm_sparse.h (device pointers owned by the caller, work enqueued on
 * `stream`, arguments checked before any HIP call, status codes, no allocation, copy or
 * synchronisation in the library). fp16 is passed as its raw bit pattern (uint16_t). Sums,
 * statistics and the arithmetic between them are in 32 bits, with one rounding where a result
 * is stored. NaN and infinities go through by the formulas as they stand, but where a call says
 * otherwise. An output may be the same array as an input only where a call says so; other
 * overlaps of outputs with inputs or with each other give unspecified values.
 */
#ifndef NM_BLOCK_H
#define NM_BLOCK_H

#include <stddef.h>
#include <stdint.h>

#include "nm_sparse.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Unknown activation, norm kind or element type: NM_ERR_FORMAT (nm_decode.h) = 8. */

/* silu: x / (1 + exp(-x)); gelu: x Phi(x); gelu_tanh: x / (1 + exp(-2 u)), u = sqrt(2/pi)
 * (x + 0.044715 x^3). */
enum { NM_ACT_NONE = 0, NM_ACT_RELU = 1, NM_ACT_SILU = 2, NM_ACT_GELU = 3, NM_ACT_GELU_TANH = 4 };

/* Y = scale * act(X W'^T + bias) + residual, as nm_spmm_ws with this end.
 *   values, masks, X, Y, rows, cols, batch, N, M, workspace  as nm_spmm_ws (every pattern and
 *             batch that it takes; nm_spmm_workspace_bytes says how much workspace it can use)
 *   bias      fp16 [rows], or NULL (none)
 *   residual  fp16 [batch][rows], or NULL (none); may be Y
 * Errors as nm_spmm_ws; NM_ERR_SHAPE also for rows above 2^26 - 64 or rows * batch above 2^35;
 * NM_ERR_FORMAT: unknown activation; NM_ERR_ALIGN also for bias or residual not 2-byte aligned. (Y,
 * bias and residual that are 16-byte aligned, with rows a multiple of 8, are moved 8 rows at a time.)
 * One workspace serves these calls and nm_spmm_ws's in stream order, but not nm_logprobs's. */
int nm_linear(const uint16_t* values, const uint32_t* masks, const uint16_t* X, uint16_t* Y, int64_t rows,
              int64_t cols, int64_t batch, int N, int M, const uint16_t* bias, int activation, float scale,
              const uint16_t* residual, void* workspace, size_t workspace_bytes, void* stream);

/* Y = act(X Wg'^T + gate_bias) * (X Wu'^T + up_bias), both matrices rows x cols and of one
 * pattern, read once in one launch where nm_spmm takes one.
 *   gate_values, up_values, gate_masks, up_masks  as values and masks of nm_spmm_ws
 *   gate_bias, up_bias  fp16 [rows], or NULL
 *   workspace  as nm_spmm_ws's, of nm_gated_workspace_bytes or more (NULL, or less: columns are
 *              not split)
 * Errors as nm_linear, whose limits here are 2 * rows'. */
int nm_gated(const uint16_t* gate_values, const uint32_t* gate_masks, const uint16_t* up_values,
             const uint32_t* up_masks, const uint16_t* X, uint16_t* Y, int64_t rows, int64_t cols, int64_t batch,
             int N, int M, const uint16_t* gate_bias, const uint16_t* up_bias, int activation, void* workspace,
             size_t workspace_bytes, void* stream);

/* Workspace bytes nm_gated can use (0: none, or bad arguments). */
size_t nm_gated_workspace_bytes(int64_t rows, int64_t cols, int64_t batch, int N, int M);

/* Norms of a row v: rms: v / sqrt(mean(v^2) + eps) * (offset + weight) + bias; layer: the same of
 * v - mean(v). A weight of NULL stands for one without offset (factor 1), a bias of NULL for 0. */
enum { NM_NORM_RMS = 0, NM_NORM_LAYER = 1 };

/* y = norm(x) for `heads` rows of `width` elements a token.
 *   x        fp16 or (fp32_input) fp32, token t's row h at [t * x_stride + h * width]
 *   y        fp16, likewise; may be x (fp16, same stride)
 *   weight, bias  fp16 [width], or NULL
 * NM_ERR_SHAPE: tokens or heads below 1, width outside 1 .. 32768, tokens * heads * (width, or 128 if
 * that is more) above 2^33, a stride below heads * width or above 2^40, eps negative or not finite;
 * NM_ERR_FORMAT: unknown kind; NM_ERR_ALIGN: a pointer not aligned to its elements. */
int nm_norm(const void* x, uint16_t* y, const uint16_t* weight, const uint16_t* bias, int64_t tokens,
            int64_t heads, int64_t width, int64_t x_stride, int64_t y_stride, int fp32_input, int kind, float offset,
            float eps, void* stream);

/* Between two blocks: h = x + scale * gate * post(branch), y = norm(h), of rows of `width`.
 *   x, h       the residual stream before and after, fp16 or fp32 (fp32_stream); h may be x, or
 *              NULL (not stored)
 *   branch, y  fp16; y may be branch
 *   post       fp16 [width], the weight of the norm after the branch (same kind, offset and eps,
 *              no bias), or NULL: the branch as it is
 *   gate       fp16, row r's at [r * gate_stride]; a gate_stride of 0 is one gate [width] for all
 *              rows; NULL: 1
 *   weight, bias  fp16 [width] or NULL, of the norm before the next block
 * y is the norm of h in 32 bits, before h is rounded to its type. Strides count elements between
 * rows. Errors as nm_norm. */
int nm_block_norm(const void* x, const uint16_t* branch, void* h, uint16_t* y, const uint16_t* post,
                  const uint16_t* gate, const uint16_t* weight, const uint16_t* bias, int64_t rows, int64_t width,
                  int64_t x_stride, int64_t branch_stride, int64_t h_stride, int64_t y_stride, int64_t gate_stride,
                  int fp32_stream, int kind, float scale, float offset, float eps, void* stream);

#define NM_MAX_TOP 64

/* Of each row of logits, with z = scale * logits and p = softmax(z):
 *   logprob[r]   log p at tokens[r]; 0 for a negative token (padding), NaN for one past the
 *                vocabulary. tokens and logprob may both be NULL
 *   entropy[r]   -sum p log p; may be NULL
 *   top_tokens, top_logprobs [rows][top]   the `top` most likely tokens, best first, ties to the
 *                lower one, and their log p; NULL where top is 0
 *   logits       fp32, or fp16 (fp16_logits), row r at [r * stride], any alignment of its elements
 *   workspace    nm_logprobs_workspace_bytes of zeroed memory, 16-byte aligned, or NULL (with that,
 *                or less, rows are not split); a call leaves its counters at zero, so one serves any
 *                sequence of these calls and those of nm_decode.h in stream order (not the products',
 *                whose counters lie otherwise)
 * Logits of -infinity have no probability and are never listed: entries past the last token with
 * one are -1 and -infinity. A row without any has log probabilities of -infinity and an entropy of
 * 0. A row with a NaN or +infinity has NaN for each number and -1 for each top token. Logits of the
 * type's lowest value are numbers like others, and so are those of any other finite mask, at any scale (beside
 * one that leaves fewer than `top` tokens, alternatives take many times as long as beside -infinity). Sums over
 * the row hold the largest term apart, so that log p near 0 and small entropies keep their digits.
 * NM_ERR_NULL; NM_ERR_SHAPE: rows outside 1 .. 2^23, vocab outside 1 .. 2^24, top outside 0 .. 64 or
 * above vocab, a stride below vocab or above 2^40, scale not positive and finite; NM_ERR_ALIGN. */
int nm_logprobs(const void* logits, const int32_t* tokens, float* logprob, float* entropy, int32_t* top_tokens,
                float* top_logprobs, int64_t rows, int64_t vocab, int64_t stride, int64_t top, int fp16_logits,
                float scale, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes nm_logprobs can use for these sizes, or for fewer rows (0: none). */
size_t nm_logprobs_workspace_bytes(int64_t rows, int64_t vocab);

#ifdef __cplusplus
}
#endif

#endif
