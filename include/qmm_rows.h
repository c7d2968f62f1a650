/*
 * qmm_rows.h -- C ABI of what stands around the grouped products: rows sorted by
 * the matrix they go through and summed back, with the gradient of that, and
 * low-rank adapters added to a shared projection.
 *
 * The conventions of qmm_fp8.h hold for every entry point here (its types and
 * limits too): device pointers, asynchronous work on `stream`, arguments checked
 * on the host before any HIP call, the same bits from run to run. All calls may
 * run at the same time on different streams, may be captured into a HIP graph
 * and hold no state between calls; only a workspace must not be shared by calls
 * that overlap in time.
 *
 * A routed layer by these calls, for `tokens` rows x and their choices ids and
 * weights w (top_k a token):
 *   qmm_rows_sort(ids)                     -> offsets, row_index, places
 *   qmm_fp8_quant(x), qmm_fp8_grouped(.., offsets, row_index, ..),
 *   qmm_fp8_quant_silu_mul, qmm_fp8_grouped(.., offsets, NULL, ..) -> z
 *   qmm_rows_combine(z, places, w)         -> y
 */
#ifndef QMM_ROWS_H
#define QMM_ROWS_H

#include "qmm_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- limits (QMV_ERR_RANGE above) ---------------------------------------- */
#define QMM_MAX_TOP_K 32    /* choices of a token; tokens * top_k <= QMM_MAX_ROWS */
#define QMM_MAX_RANK  128   /* of an adapter                                      */

/*
 * Choices sorted by expert (or by any other key below QMM_MAX_EXPERTS, such as a
 * request's adapter with top_k = 1).
 *   ids        int32 [tokens][top_k]; a value outside [0, n_experts) is no
 *              choice (padding, an expert held elsewhere). A token may name one
 *              expert twice: two rows.
 *   offsets    int32 [n_experts + 1]: rows offsets[e] .. offsets[e+1] - 1 are
 *              expert e's, in the order of (token, choice)
 *   row_index  int32 [tokens * top_k]: the token of each row; -1 from
 *              offsets[n_experts] on. May be NULL.
 *   places     int32 [tokens][top_k]: the row of each choice, -1 where there is
 *              none. May be NULL.
 *   ws         device memory of ws_bytes >= qmm_rows_sort_workspace(tokens, top_k,
 *              n_experts), 256-byte aligned (its contents do not matter); may
 *              be NULL when that size is 0, else QMV_ERR_WORKSPACE
 *   tokens >= 0 (0: offsets are zeros), 1 <= top_k <= QMM_MAX_TOP_K,
 *   1 <= n_experts <= QMM_MAX_EXPERTS; all arrays 4-byte aligned
 */
size_t qmm_rows_sort_workspace(int tokens, int top_k, int n_experts);
int qmm_rows_sort(const int32_t *ids, int32_t *offsets, int32_t *row_index, int32_t *places, int tokens, int top_k,
                  int n_experts, void *ws, size_t ws_bytes, void *stream);

/*
 * Tokens' rows written where their choices stand: out[places[t][j]] = x[t].
 *   x       [tokens][h] of `type` (QMM_F32 or QMM_BF16), 16-byte aligned
 *   places  int32 [tokens][top_k], 4-byte aligned; outside [0, rows): not written
 *   out     [rows][h] of the same type, 16-byte aligned; rows that no place names
 *           are left as they were
 *   tokens >= 0, rows >= 0 (0: nothing is done), 1 <= h <= QMM_MAX_K
 * A row that several places name gets values of any of their tokens, in no
 * defined mix. The gradient by x is qmm_rows_combine on out's, without weights.
 */
int qmm_rows_spread(const void *x, int type, const int32_t *places, void *out, int tokens, int top_k, int h, int rows,
                    void *stream);

/*
 * Rows summed back: y[t] = sum_j w[t][j] * z[places[t][j]], in fp32, in the order
 * of j, rounded once to y's type (nearest even).
 *   z       [rows][h] of z_type, 16-byte aligned
 *   places  as above; a choice outside [0, rows) adds nothing, whatever its
 *           weight, and a token without one gets zeros
 *   w       fp32 [tokens][top_k], 4-byte aligned, or NULL: weights of one
 *   y       [tokens][h] of y_type, 16-byte aligned
 *   tokens >= 0 (0: nothing is done), rows >= 0, 1 <= h <= QMM_MAX_K
 */
int qmm_rows_combine(const void *z, int z_type, const int32_t *places, const float *w, void *y, int y_type, int tokens,
                     int top_k, int h, int rows, void *stream);

/*
 * The gradient of qmm_rows_combine, from dy [tokens][h]:
 *   dz[places[t][j]] = w[t][j] * dy[t], in fp32, rounded once
 *   dw[t][j]         = sum_h dy[t] * z[places[t][j]], fp32 sums; 0 where a choice has no place
 *   dy, z, dz  of one `type`, 16-byte aligned; rows of dz that no place names
 *              are left as they were; one that several name is not defined
 *   w          as above (NULL: weights of one)
 *   dw         fp32 [tokens][top_k], 4-byte aligned
 *   z and dw may both be NULL: dz alone
 */
int qmm_rows_combine_grad(const void *dy, const void *z, int type, const int32_t *places, const float *w, void *dz,
                          float *dw, int tokens, int top_k, int h, int rows, void *stream);

/*
 * Workspace bytes qmm_lora needs (0 if an argument is out of range). It depends
 * on the shape alone.
 */
size_t qmm_lora_workspace(int rows, int n, int k, int rank, int n_adapters);

/*
 * Low-rank adapters of many requests beside a shared projection:
 *   y[r] = base[r] + scale[e] * B_e (A_e x[r])
 * for the rows r of adapter e's run, with fp32 sums (A_e x[r] included; bits of
 * scale[e] * (A_e x[r]) below 2^-133 are cut), rounded once to y's type. With
 * base == y the projection's result is added to in place.
 *   a          bf16 [n_adapters][rank][k], 16-byte aligned, a_bytes == 2*n_adapters*rank*k
 *   b          bf16 [n_adapters][n][rank], 16-byte aligned, b_bytes == 2*n_adapters*n*rank
 *   scale      fp32 [n_adapters] or NULL (ones)
 *   ranks      int32 [n_adapters] or NULL: adapter e uses the first ranks[e] rows
 *              of A_e and columns of B_e (clamped to [0, rank]); what lies behind
 *              them does not matter
 *   x          bf16 [x_rows][k], 16-byte aligned
 *   offsets    int32 [n_adapters + 1], row_index int32 [rows] or NULL, as
 *              qmm_rows_sort (top_k = 1) gives them: row row_index[r] of x, base
 *              and y for r in offsets[e] .. offsets[e+1] - 1. An index outside
 *              [0, x_rows) is passed over. NULL: row r, and x_rows must equal
 *              rows. A row of x that stands in the runs twice gets values of no
 *              defined sum in y.
 *   base, y    [x_rows][n] of y_type (QMM_F32 or QMM_BF16), 16-byte aligned; the
 *              same array or two without a shared byte. Rows in no run are left
 *              as they were in y.
 *   ws         as in qmm_rows_sort, of qmm_lora_workspace(...) bytes
 *   rows >= 0 (0: nothing is done), n >= 1, k >= 8 and k % 8 == 0,
 *   rank >= 8 and rank % 8 == 0, 1 <= n_adapters <= QMM_MAX_EXPERTS,
 *   (rows / 16 + min(rows, n_adapters)) * ceil(n / 256) <= 2^28
 * Offsets are clamped to [0, rows]; where they decrease, which rows are written
 * is not defined, but no memory outside the arguments is touched. The order of
 * the sums depends on the sizes alone; for rows <= QMM_SAME_ROWS a row's bits
 * depend on its adapter alone, whatever rows stand beside it. A NaN or an
 * infinity in x[r], A_e or B_e makes the sums it enters not finite and touches
 * no other.
 */
int qmm_lora(const uint16_t *a, size_t a_bytes, const uint16_t *b, size_t b_bytes, const float *scale,
             const int32_t *ranks, const uint16_t *x, const int32_t *offsets, const int32_t *row_index,
             const void *base, void *y, int y_type, int rows, int x_rows, int n, int k, int rank, int n_adapters,
             void *ws, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QMM_ROWS_H */
