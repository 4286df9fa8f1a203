/*
 * cbk_nn.h -- C ABI of libcbk, continued: the operators with which a model whose weights stay
 * codebook-compressed (cbk.h) is run over any number of tokens, scored and tuned: products for any
 * number of tokens, the gated feed-forward block and the softmax cross entropy of a compressed
 * output head, each with its gradient.
 *
 * The weights are a lossless code of fixed values, so a backward pass gives the gradients of the
 * activations (and, for the feed-forward block, those at the two projections' outputs, which an
 * adapter beside a projection needs), never of the weights.  Nothing of the weights' uncompressed
 * size is kept: weights are decoded tile by tile, or a piece of a tensor at a time into the
 * workspace.
 *
 * Notation: T tokens; a tensor W is [rows][cols]; every matrix of activations is row-major with a
 * leading dimension in elements, [T][ld], and BF16; products and sums are fp32, rounded once (to
 * nearest even) where a BF16 output is written.
 *
 * Conventions: as in cbk.h (status codes, arguments validated on the host before any HIP call, the
 * caller's stream, no allocation, no state kept between calls, outputs must not alias inputs,
 * corrupt indices read as 0x7FC0).  In addition:
 *  - tokens == 0 is a no-op.  Rows past the last token are neither read nor written, and neither
 *    are columns past the last one of any row.
 *  - workspace: device scratch of at least the bytes that the operator's _workspace_bytes call
 *    gives for the same tensors and tokens, 256-byte aligned, owned by the caller; its contents on
 *    entry do not matter.  Calls that may overlap (two streams, two captured graphs that are
 *    replayed side by side) need separate workspaces.  workspace_bytes is its size;
 *    CBK_E_CAPACITY when that is too small.  A workspace may be NULL only when 0 bytes are needed.
 *  - BF16 pointers must be 2-byte aligned.  Matrices that are 16-byte aligned with a leading
 *    dimension that is a multiple of 8 are read and written 16 bytes at a time; others give the same
 *    bits, more slowly.  X and dY may be copied into the workspace first.
 *  - results do not depend on timing: equal inputs give equal bits.
 *  - limits: cols <= 2^20, rows < 2^31, tokens < 2^31, leading dimensions < 2^32;
 *    CBK_E_UNSUPPORTED beyond.
 */
#ifndef CBK_NN_H
#define CBK_NN_H

#include "cbk.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * cbk_linear -- GPU.  Y[t][r] = sum_k X[t][k] W[r][k] for any number of tokens (cbk_gemm_small
 * stops at 16 and writes fp32).
 *   X   device, [tokens][ldx] BF16, ldx >= cols.
 *   Y   device, [tokens][ldy] BF16, ldy >= rows; Y[t][0..rows) is overwritten (zeros when cols == 0).
 * cbk_linear_dx -- GPU.  Its gradient: dX[t][k] = sum_r dY[t][r] W[r][k].
 *   dY  device, [tokens][lddy] BF16, lddy >= rows.
 *   dX  device, [tokens][lddx] BF16, lddx >= cols; overwritten (zeros when rows == 0).
 * Both take cbk_linear_workspace_bytes(t, tokens) bytes of workspace.
 */
size_t cbk_linear_workspace_bytes(const cbk_tensor *t, uint64_t tokens);
cbk_status cbk_linear(const cbk_tensor *t, const uint16_t *X, uint64_t ldx, uint64_t tokens, uint16_t *Y,
                      uint64_t ldy, void *workspace, size_t workspace_bytes, void *stream);
cbk_status cbk_linear_dx(const cbk_tensor *t, const uint16_t *dY, uint64_t lddy, uint64_t tokens, uint16_t *dX,
                         uint64_t lddx, void *workspace, size_t workspace_bytes, void *stream);

/* Activations of the gated feed-forward block. */
typedef enum {
    CBK_ACT_SILU = 0,      /* z / (1 + exp(-z))                                               */
    CBK_ACT_GELU = 1,      /* z Phi(z), Phi the normal distribution function                  */
    CBK_ACT_GELU_TANH = 2  /* z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2               */
} cbk_act;

/*
 * cbk_ffn_gated -- GPU.  The gated feed-forward block up to its down projection:
 * H[t][f] = act(g) u with g = sum_k X[t][k] Wg[f][k] and u = sum_k X[t][k] Wu[f][k]; g and u stay
 * in fp32 and are not written.
 *   gate, up  tensors of equal rows and cols (their U and b may differ).
 *   X   device, [tokens][ldx] BF16, ldx >= cols.
 *   H   device, [tokens][ldh] BF16, ldh >= rows; overwritten.
 * cbk_ffn_gated_bwd -- GPU.  Its gradient.  g and u are computed again from X; with dH the
 * gradient of H: dG = dH u act'(g), dU = dH act(g), dX[t][k] = sum_f dG[t][f] Wg[f][k] +
 * dU[t][f] Wu[f][k].  The products that give dX take dG and dU as rounded to BF16.
 *   dH  device, [tokens][lddh] BF16, lddh >= rows.
 *   dX  device, [tokens][lddx] BF16, lddx >= cols; overwritten.
 *   dG, dU  device, [tokens][ldg] BF16, ldg >= rows, overwritten; either may be NULL where it is
 *       not wanted.
 * Both take cbk_ffn_workspace_bytes(gate, up, tokens) bytes of workspace.
 */
size_t cbk_ffn_workspace_bytes(const cbk_tensor *gate, const cbk_tensor *up, uint64_t tokens);
cbk_status cbk_ffn_gated(const cbk_tensor *gate, const cbk_tensor *up, int act, const uint16_t *X, uint64_t ldx,
                         uint64_t tokens, uint16_t *H, uint64_t ldh, void *workspace, size_t workspace_bytes,
                         void *stream);
cbk_status cbk_ffn_gated_bwd(const cbk_tensor *gate, const cbk_tensor *up, int act, const uint16_t *X, uint64_t ldx,
                             const uint16_t *dH, uint64_t lddh, uint64_t tokens, uint16_t *dX, uint64_t lddx,
                             uint16_t *dG, uint16_t *dU, uint64_t ldg, void *workspace, size_t workspace_bytes,
                             void *stream);

/*
 * cbk_xent -- GPU.  Softmax cross entropy over the head's rows (the vocabulary), without keeping
 * the logits z[t][v] = sum_k X[t][k] W[v][k]:
 *   lse[t]  = log sum_v exp z[t][v]
 *   loss[t] = lse[t] - z[t][labels[t]], or 0 where labels[t] == ignore_index.
 * A label that is neither ignore_index nor in [0, rows) gives a loss of NaN (it is known only on
 * the device, and nothing is read or written out of range).
 *   head    rows >= 1 (CBK_E_INVALID otherwise).
 *   X       device, [tokens][ldx] BF16, ldx >= cols.
 *   labels  device, tokens int64, 8-byte aligned.
 *   loss, lse  device, tokens fp32 each, 4-byte aligned; overwritten.
 * cbk_xent_bwd -- GPU.  Its gradient.  The logits are computed again; with dloss the gradient of
 * loss: dX[t][k] = dloss[t] sum_v (exp(z[t][v] - lse[t]) - [v == labels[t]]) W[v][k], where the
 * bracketed differences are rounded to BF16 for the product.  Rows whose label is ignore_index
 * are zero whatever their X, lse and dloss hold; rows of an out-of-range label are NaN.
 *   lse     device, tokens fp32, as cbk_xent gave it for the same head and X.
 *   dloss   device, tokens fp32, 4-byte aligned.
 *   dX      device, [tokens][lddx] BF16, lddx >= cols; overwritten.
 * Both take cbk_xent_workspace_bytes(head, tokens) bytes of workspace.
 */
size_t cbk_xent_workspace_bytes(const cbk_tensor *head, uint64_t tokens);
cbk_status cbk_xent(const cbk_tensor *head, const uint16_t *X, uint64_t ldx, const int64_t *labels, uint64_t tokens,
                    int64_t ignore_index, float *loss, float *lse, void *workspace, size_t workspace_bytes,
                    void *stream);
cbk_status cbk_xent_bwd(const cbk_tensor *head, const uint16_t *X, uint64_t ldx, const int64_t *labels,
                        const float *lse, const float *dloss, uint64_t tokens, int64_t ignore_index, uint16_t *dX,
                        uint64_t lddx, void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* CBK_NN_H */
