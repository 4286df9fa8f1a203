/*
 * cbk_moe.h -- C ABI of libcbk, continued: feed-forward blocks of experts whose weights stay
 * codebook-compressed (cbk.h), from the scores that route a token to its experts to the weighted sum of
 * what they give, each with its gradient.
 *
 * Conventions: as in cbk_nn.h (status codes, arguments validated on the host before any HIP call, the
 * caller's stream and workspace, no state kept between calls, outputs must not alias inputs, corrupt
 * indices read as 0x7FC0, equal inputs give equal bits, tokens == 0 is a no-op, gradients of the
 * activations and never of the weights).  What a call does depends on device data alone, nothing is read
 * back to the host, and every call can be captured into a graph.  A call of fewer tokens may need more
 * workspace than one of more tokens (its reductions are shared out).
 *
 * Notation: T tokens, E experts, k of them for a token.  A token's k places are its slots.
 */
#ifndef CBK_MOE_H
#define CBK_MOE_H

#include "cbk_nn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { CBK_SCORE_SOFTMAX = 0, CBK_SCORE_SIGMOID = 1 } cbk_score;
typedef enum { CBK_F32 = 0, CBK_BF16 = 1 } cbk_dtype;

/* How tokens are routed. */
typedef struct {
    uint32_t experts;     /* E, 1..1024                                                          */
    uint32_t k;           /* experts of a token, 1..min(E, 64)                                   */
    int32_t score;        /* cbk_score                                                           */
    int32_t renormalise;  /* nonzero: a token's weights are divided by their sum                 */
    float scale;          /* factor of every weight                                              */
    uint32_t groups;      /* E is a multiple of it; 1: no groups                                 */
    uint32_t top_groups;  /* groups that experts are chosen from, 1..groups                      */
    uint32_t group_top;   /* 1 or 2: a group's mark is its best expert's score, or its two best's sum */
} cbk_router;

/*
 * cbk_route -- GPU.  Chooses a token's experts.  With logits z:
 *   s = softmax(z) or 1 / (1 + exp(-z)),  c = s + bias (bias may be NULL: c = s);
 *   of the groups of E / groups neighbouring experts the top_groups with the highest mark, the sum of
 *   their group_top largest c, are kept; of the kept groups' experts the k with the largest c are
 *   chosen, in falling order; equal ones go by the lower index, groups as well as experts;
 *   weights = scale * s, or scale * s / (sum of the chosen s).  The bias only steers the choice.
 * An expert whose logit or bias is -inf is never chosen and is left out of its group's mark; slots that
 * no expert is left for get -1 and a weight of 0 (all of them where a row is all -inf: padding).  A row that
 * holds a NaN, or a +inf logit, or whose biased scores hold a NaN, gets experts 0..k-1 and NaN weights.
 * Scores are compared in 64 bits (without a bias and sums of two, the logits themselves are); weights
 * are rounded to fp32.
 *   logits   device, [tokens][ld] fp32 (4-byte aligned) or BF16 (2-byte aligned), ld >= E, < 2^32.
 *   bias     device, E fp32, 4-byte aligned, or NULL.
 *   experts  device, [tokens][k] int32; weights  device, [tokens][k] fp32; 4-byte aligned; overwritten.
 */
cbk_status cbk_route(const cbk_router *r, const void *logits, int dtype, uint64_t ld, uint64_t tokens, const float *bias,
                     int32_t *experts, float *weights, void *stream);

/*
 * cbk_route_bwd -- GPU.  The gradient of the logits, for the experts that cbk_route chose and the gradient
 * dweights of their weights: through the chosen experts' scores (and, for softmax, the others'); choosing
 * has no gradient, and bias and groups play no part.  A slot whose expert is outside [0, E) gets none.
 * An expert that stands in two slots of a token counts with the sum of both; when renormalised, its score
 * counts twice in the sum, as the forward formula has it.
 *   dlogits  device, [tokens][ldd] of the logits' type, ldd >= E; overwritten.  Rows that are all -inf are zero.
 */
cbk_status cbk_route_bwd(const cbk_router *r, const void *logits, int dtype, uint64_t ld, uint64_t tokens,
                         const int32_t *experts, const float *dweights, void *dlogits, uint64_t ldd, void *stream);

/*
 * The experts of a layer: a table of their tensors in device memory, made once.  gate and up are
 * [rows][cols], down is [out][rows]; all experts' shapes are alike, U and b may differ from tensor to
 * tensor.
 */
typedef struct {
    void *buffer;     /* device, cbk_experts_bytes(count) bytes, the caller's                       */
    uint64_t rows;    /* the hidden width                                                          */
    uint64_t cols;    /* columns of X                                                              */
    uint64_t out;     /* columns of Y                                                              */
    uint32_t count;
    uint32_t b;       /* the widest index of gate and up                                           */
    uint32_t b_down;  /* and of down                                                               */
    uint32_t device;
} cbk_experts;

/*
 * cbk_experts_init -- GPU.  Fills `ex` and copies the table to `buffer` (256-byte aligned, at least
 * cbk_experts_bytes(count)) on the current device; returns when it is there (not for capture).  The
 * tensors' codebooks and words, and the buffer, have to live as long as `ex` is used.
 * 1 <= count <= 1024 and rows, cols, out >= 1 (CBK_E_INVALID otherwise); all three <= 2^20
 * (CBK_E_UNSUPPORTED).
 */
size_t cbk_experts_bytes(uint32_t count);
cbk_status cbk_experts_init(const cbk_tensor *gate, const cbk_tensor *up, const cbk_tensor *down, uint32_t count,
                            void *buffer, size_t bytes, cbk_experts *ex);

/*
 * cbk_ffn_experts -- GPU.  Y[t] = sum_j weights[t][j] Wd_e H, H = act(Wg_e X[t]) (Wu_e X[t]), e = experts[t][j].
 * A slot whose expert is outside [0, count) contributes nothing (unused, or another device's).  H is rounded
 * to BF16 for the second product; weights, sums over experts and both products' sums are fp32.
 *   X        device, [tokens][ldx] BF16, ldx >= cols.
 *   experts  device, [tokens][k] int32; weights  device, [tokens][k] fp32; 4-byte aligned; 1 <= k <= 64.
 *   Y        device, [tokens][ldy] BF16, ldy >= out; overwritten.
 * cbk_ffn_experts_bwd -- GPU.  Its gradient; g, u and H are computed again from X.  With D = Wd_e^T dY[t]:
 * dweights[t][j] = <H, D> (with H not rounded; 0 for unused slots), dH = weights[t][j] D,
 * dG = dH u act'(g), dU = dH act(g), dX[t] = sum_j Wg_e^T dG + Wu_e^T dU; dG and dU are rounded to BF16 for
 * these products.
 *   dY       device, [tokens][lddy] BF16, lddy >= out.
 *   dX       device, [tokens][lddx] BF16, lddx >= cols; overwritten.
 *   dweights device, [tokens][k] fp32, 4-byte aligned; overwritten; NULL where it is not wanted.
 * Both run on the device that `ex` was made on (CBK_E_INVALID where another is current), with
 * cbk_experts_workspace_bytes(ex, tokens, k, backward) bytes of workspace.
 */
size_t cbk_experts_workspace_bytes(const cbk_experts *ex, uint64_t tokens, uint32_t k, int backward);
cbk_status cbk_ffn_experts(const cbk_experts *ex, int act, const uint16_t *X, uint64_t ldx, uint64_t tokens,
                           const int32_t *experts, const float *weights, uint32_t k, uint16_t *Y, uint64_t ldy,
                           void *workspace, size_t workspace_bytes, void *stream);
cbk_status cbk_ffn_experts_bwd(const cbk_experts *ex, int act, const uint16_t *X, uint64_t ldx, uint64_t tokens,
                               const int32_t *experts, const float *weights, uint32_t k, const uint16_t *dY,
                               uint64_t lddy, uint16_t *dX, uint64_t lddx, float *dweights, void *workspace,
                               size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* CBK_MOE_H */
