/*
 * qmm_fp8.h -- C ABI of the 8-bit floating point and grouped matrix products.
 *
 * The conventions of qmv.h hold for every entry point here: device pointers of
 * the current device, caller-owned buffers, asynchronous work on `stream`
 * (NULL = the null stream), every argument checked on the host before any HIP
 * call, QMV_ERR_* status codes with qmv_strerror() and qmv_last_error(),
 * results that are the same bits from run to run. All calls may run at the
 * same time on different streams, may be captured into a HIP graph and hold no
 * state between calls; only a workspace must not be shared by calls that
 * overlap in time.
 *
 * The e4m3 format
 * ---------------
 * One byte: sign, four exponent bits (bias 7), three mantissa bits; the largest
 * value is 448, there is no infinity, and 0x7F / 0xFF are NaN. A matrix comes
 * with fp32 scales, one for each block of 128 along k (the last block of a row
 * is shorter when k is not a multiple of 128):
 *  - activations: one scale per row and block, stored block by block:
 *    x_scale[b * rows + r] belongs to x[r][128 b .. 128 b + 127];
 *  - weights: one scale per 128 x 128 block, w_scale[j * ceil(k/128) + b]
 *    belongs to w[128 j .. 128 j + 127][128 b .. 128 b + 127].
 * The products below are
 *   y[r][i] = sum_b x_scale[b][r] * w_scale[i/128][b] *
 *             sum_{k in block b} x[r][k] * w[i][k],
 * with fp32 sums, y rounded once to its type (nearest even). The product of the
 * two scales is formed first, in fp32. The codes go through the matrix cores as
 * bf16, which holds them exactly: every product is exact, and the sums lose what
 * fp32 additions lose.
 *
 * QMM_FAST_SUMS, with y in bf16, lets a call take the e4m3 matrix instruction
 * instead, at about twice the rate for many rows. It aligns each eight
 * neighbouring products along k to the largest of them and cuts what lies 13
 * bits below: a result is off by up to 7 * 2^-13 * sum |x w| before it is rounded
 * (eight products that cancel can lose their sum), on normal data by 1.5e-5 and
 * with a few strong channels by 4e-5 of the results' norm.
 *
 * Values that are not finite go through as arithmetic has them: a NaN code or a
 * NaN or infinite scale makes the sums it enters NaN or infinite and touches no
 * other.
 */
#ifndef QMM_FP8_H
#define QMM_FP8_H

#include "qmv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- types of y, and of the rows given to the quantisers ---------------- */
#define QMM_F32   0
#define QMM_BF16  1
#define QMM_FAST_SUMS 16   /* QMM_BF16 | QMM_FAST_SUMS: a y_type of qmm_fp8,
                              qmm_fp8_workspace and qmm_fp8_grouped        */

/* ---- limits (QMV_ERR_RANGE above) ---------------------------------------- */
#define QMM_MAX_ROWS    (1 << 24)   /* rows of x or y of one call               */
#define QMM_MAX_N       (1 << 20)   /* rows of one weight matrix                */
#define QMM_MAX_K       (1 << 20)   /* values per row                           */
#define QMM_MAX_EXPERTS 1024
#define QMM_SAME_ROWS   16          /* qmm_fp8: rows whose bits do not depend on m */

/*
 * Rows of activations to e4m3 with one scale per 128 values.
 *   x        [m][k], fp32 (x_type QMM_F32) or bf16 (QMM_BF16), 16-byte aligned
 *   xq       e4m3 [m][k], 16-byte aligned
 *   xs       fp32 [ceil(k/128)][m], 4-byte aligned
 *   m >= 0 (0: nothing is done), k >= 8 and k % 8 == 0 (the products take
 *   rows of a multiple of 16)
 * With a the largest |x| of a block of 128: scale = max(a / 448, 2^-126) in
 * fp32 (so a block of zeros has codes 0), code = x / scale in fp32 rounded to
 * the nearest e4m3 value, ties to even. A block that holds an infinity or a NaN
 * gets that as its scale: every product of that row is then not finite.
 */
int qmm_fp8_quant(const void *x, int x_type, uint8_t *xq, float *xs, int m, int k, void *stream);

/*
 * The gated form, between the two products of a feed-forward layer:
 *   x        [m][2 k]: row r holds gate[r][0 .. k) and then up[r][0 .. k)
 * h = gate / (1 + exp(-gate)) * up in fp32, then as qmm_fp8_quant on h [m][k].
 */
int qmm_fp8_quant_silu_mul(const void *x, int x_type, uint8_t *xq, float *xs, int m, int k, void *stream);

/*
 * Workspace bytes qmm_fp8 needs for m x n x k (0 if none, or if an argument is
 * out of range). It depends on the shape and y_type alone.
 */
size_t qmm_fp8_workspace(int m, int n, int k, int y_type);

/*
 * Y = X W^T, both e4m3 with scales as above.
 *   w, w_scale   e4m3 [n][k], 16-byte aligned, w_bytes == n*k;
 *                fp32 [ceil(n/128)][ceil(k/128)], 4-byte aligned
 *   x, x_scale   e4m3 [m][k], 16-byte aligned; fp32 [ceil(k/128)][m]
 *   y            [m][n] of y_type (QMM_F32, QMM_BF16 or QMM_BF16 |
 *                QMM_FAST_SUMS), 16-byte aligned
 *   ws           device memory of ws_bytes >= qmm_fp8_workspace(m, n, k, y_type),
 *                256-byte aligned (its contents do not matter); may be NULL
 *                when that size is 0, else QMV_ERR_WORKSPACE
 *   m >= 1, n >= 1, k >= 16 and k % 16 == 0
 * The order of the sums depends on m, n, k and QMM_FAST_SUMS alone; for m <=
 * QMM_SAME_ROWS it depends on (n, k) alone, so a row has the same bits whatever m
 * is (plain decode and speculative verify run one numerical program; fast sums
 * have no effect there). From more rows on the order of a row's sums may change
 * with m.
 */
int qmm_fp8(const void *w, size_t w_bytes, const float *w_scale, const void *x, const float *x_scale,
            void *y, int y_type, int m, int n, int k, void *ws, size_t ws_bytes, void *stream);

/*
 * The same product with one weight matrix per expert over runs of rows.
 *   w, w_scale   n_experts matrices as in qmm_fp8, one after the other;
 *                w_bytes == n_experts*n*k
 *   x, x_scale   e4m3 [x_rows][k]; fp32 [ceil(k/128)][x_rows]
 *   offsets      int32 [n_experts + 1], 4-byte aligned: rows offsets[e] ..
 *                offsets[e+1] - 1 of y belong to expert e; nondecreasing,
 *                within [0, rows]. An expert may have no row.
 *   row_index    int32 [rows] or NULL: row r of y takes row row_index[r] of x
 *                (a token's row may serve several experts); an index outside
 *                [0, x_rows) stands for a row of zeros. NULL: row r of x, and
 *                x_rows must equal rows.
 *   y            [rows][n] of y_type, 16-byte aligned; rows in no run (before
 *                offsets[0], from offsets[n_experts] on) are left as they were
 *   rows >= 0 (0: nothing is done), n, k as in qmm_fp8, 1 <= n_experts <= QMM_MAX_EXPERTS;
 *   with row_index, x must be under 4 GiB (QMV_ERR_RANGE)
 * offsets and row_index are read on the device. Offsets are clamped to
 * [0, rows]; where they decrease, which rows are written is not defined, but no
 * memory outside the arguments is touched. Needs no workspace.
 */
int qmm_fp8_grouped(const void *w, size_t w_bytes, const float *w_scale, const void *x, const float *x_scale,
                    const int32_t *offsets, const int32_t *row_index, void *y, int y_type,
                    int rows, int x_rows, int n, int k, int n_experts, void *stream);

/*
 * The grouped product on bf16 weights and rows (fp32 sums), arguments as in
 * qmm_fp8_grouped without the scales: w bf16 [n_experts][n][k], x bf16
 * [x_rows][k], 16-byte aligned, w_bytes == 2*n_experts*n*k; k >= 8 and k % 8 == 0.
 */
int qmm_bf16_grouped(const uint16_t *w_bf16, size_t w_bytes, const uint16_t *x_bf16, const int32_t *offsets,
                     const int32_t *row_index, void *y, int y_type,
                     int rows, int x_rows, int n, int k, int n_experts, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QMM_FP8_H */
