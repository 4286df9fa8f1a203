/*
 * cbk_sample.h -- C ABI of libcbk, continued: drawing the next token from a head's logits, as cbk_gemv and
 * cbk_gemm_small (fp32) or cbk_linear (BF16) of the compressed head give them.
 *
 * Conventions: as in cbk_nn.h (status codes, validation before any HIP call, the caller's stream and
 * workspace, no allocation, no state kept between calls, tokens == 0 is a no-op).
 */
#ifndef CBK_SAMPLE_H
#define CBK_SAMPLE_H

#include "cbk_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Settings of a draw.  Each is a number for all rows, or, where the pointer is not NULL, a device vector
 * with one of each row (4-byte aligned). */
typedef struct {
    float temperature, top_p, min_p;
    int32_t top_k;
    const float *temperatures, *top_ps, *min_ps;
    const int32_t *top_ks;
} cbk_sampling;

/*
 * cbk_sample -- GPU.  Draws one of a row's V entries.  With x = logits / temperature and p = softmax(x),
 * entries in falling order of their logits, equal ones by index:
 *   top_k > 0        the first top_k are kept (all, where top_k <= 0 or >= V);
 *   min_p > 0        of these, those with p >= min(min_p, 1) * (the largest p);
 *   top_p < 1        of these, the fewest first ones whose p sum to at least top_p of the sum of all that
 *                    the other two keep, at least one (all, where top_p >= 1 or is a NaN).
 * The token is the first kept entry, by index, at which the running sum of the kept p exceeds uniform times
 * their whole sum (the last kept one where rounding leaves none, or uniform >= 1; the first where it is
 * negative or a NaN).  temperature <= 0 takes the row's first entry in that order.
 *   logprob = log of the probability with which it was drawn: p over the sum of the kept p (0 if greedy).
 * An entry of -inf is never drawn.  A row that is all -inf, or holds a NaN, gives token -1 and a logprob of
 * NaN; entries of +inf share the draw with equal parts.  A NaN temperature gives -1 and NaN as well.
 * Probabilities and their sums are formed in 64 bits, so that the token is the one that the formula names
 * unless uniform falls within some 1e-12 of the border of two.
 *   logits    device, [tokens][ld] fp32 (4-byte aligned) or BF16 (2-byte aligned); 1 <= V <= 2^20
 *             (CBK_E_INVALID for 0, CBK_E_UNSUPPORTED beyond), V <= ld < 2^32.
 *   uniform   device, tokens fp32 in [0, 1), 4-byte aligned.
 *   token     device, tokens int64, 8-byte aligned; logprob  device, tokens fp32, 4-byte aligned, or NULL;
 *             overwritten.
 *   workspace cbk_sample_workspace_bytes(p, V, tokens) bytes: up to 64 MB, by V and by whether p has filters, 0 for some.
 */
size_t cbk_sample_workspace_bytes(const cbk_sampling *p, uint64_t V, uint64_t tokens);
cbk_status cbk_sample(const cbk_sampling *p, const void *logits, int dtype, uint64_t ld, uint64_t V, uint64_t tokens,
                      const float *uniform, int64_t *token, float *logprob, void *workspace, size_t workspace_bytes,
                      void *stream);

#ifdef __cplusplus
}
#endif

#endif /* CBK_SAMPLE_H */
