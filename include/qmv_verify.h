/*
 * qmv_verify.h -- C ABI of the verification of drafted tokens: which drafts of a
 * speculative step stand, and the token that follows them.
 *
 * The conventions of qmv.h hold: device pointers, asynchronous work on `stream`,
 * arguments checked on the host before any HIP call, the same bits from run to
 * run. Calls may run at the same time on different streams, may be captured into
 * a HIP graph and hold no state; only a workspace must not be shared by calls
 * that overlap in time.
 */
#ifndef QMV_VERIFY_H
#define QMV_VERIFY_H

#include "qmm_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- limits (QMV_ERR_RANGE above) ---------------------------------------- */
#define QMV_MAX_DRAFTS   32          /* of a request                             */
#define QMV_MAX_REQUESTS 65535       /* of a call                                */
#define QMV_MAX_VOCAB    (1 << 22)

/*
 * Distribution-exact acceptance of drafted tokens, from given random numbers.
 *   p        [requests][drafts + 1][vocab] of `type` (QMM_F32 or QMM_BF16),
 *            16-byte aligned: the target's probabilities, row i after i drafts
 *   q        [requests][drafts][vocab] of the same type, 16-byte aligned: those
 *            the drafts were drawn from; NULL: each draft had all of them (a
 *            drafter that takes its likeliest token)
 *   tokens   int32 [requests][drafts], the drafts
 *   lengths  int32 [requests] or NULL: a request has lengths[r] drafts (clamped
 *            to [0, drafts]; the rows behind are not read); NULL: all
 *   u        fp32 [requests][drafts + 1], uniform in [0, 1): u[r][i] decides on
 *            draft i, u[r][drafts] picks the token that follows
 *   accepted int32 [requests]: the drafts that stand
 *   out      int32 [requests][drafts + 1]: these, the token that follows, and -1s
 *   ws       device memory of ws_bytes >= qmv_verify_drafts_workspace(requests, vocab),
 *            256-byte aligned (its contents do not matter); may be NULL when
 *            that size is 0, else QMV_ERR_WORKSPACE
 *   requests >= 0 (0: nothing is done), 0 <= drafts <= QMV_MAX_DRAFTS, vocab >= 1;
 *   the small arrays 4-byte aligned; with drafts = 0 q and tokens are not read
 *
 * Draft i stands when all before it do and u[i] * q_i[d] < p_i[d] (the product is
 * taken exactly; a token outside the vocabulary or a NaN does not stand). The
 * token that follows is picked by the weights max(p_i - q_i, 0) of the first
 * draft that does not stand, or by p of the row behind the last one that does:
 * the first token whose running sum of weights, in 64 bits, lies above u[drafts]
 * times their whole sum. A weight that is negative or not finite counts as 0.
 * Where no weight of a refused draft is positive, p_i itself picks; where p_i
 * has none either, the token is -1. A u[drafts] of 1 or more (or NaN) picks the
 * last token with a weight, a negative one the first.
 */
size_t qmv_verify_drafts_workspace(int requests, int vocab);
int qmv_verify_drafts(const void *p, const void *q, int type, const int32_t *tokens, const int32_t *lengths,
                      const float *u, int32_t *accepted, int32_t *out, int requests, int drafts, int vocab, void *ws,
                      size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QMV_VERIFY_H */
