// C ABI of the e4m3 and grouped products: argument validation and dispatch.
// Pure host code: it calls no HIP function and reads no device property. See
// include/qmm_fp8.h for the contract of each entry point.
#include "../../include/qmm_fp8.h"

#include <stdint.h>

#include "fp8_internal.h"
#include "fp8_layout.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// [p, p+pb) and [q, q+qb) share a byte.
bool overlap(const void *p, size_t pb, const void *q, size_t qb) {
  if (pb == 0 || qb == 0) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + qb && b < a + pb;
}

bool type_ok(int t) { return t == QMM_F32 || t == QMM_BF16; }
size_t type_bytes(int t) { return t == QMM_F32 ? 4 : 2; }

// Takes QMM_FAST_SUMS off the y_type of an e4m3 product; what is left of a
// value it cannot stand with is no type.
bool take_fast(int *y_type) {
  if (*y_type != (QMM_BF16 | QMM_FAST_SUMS)) return false;
  *y_type = QMM_BF16;
  return true;
}

// k: a positive multiple of `step`, within range. n likewise without the step.
int check_nk(int n, int k, int step) {
  if (n < 1 || k < step || k % step) return QMV_ERR_SHAPE;
  if (n > QMM_MAX_N || k > QMM_MAX_K) return QMV_ERR_RANGE;
  return QMV_OK;
}

int quant(const void *x, int x_type, bool gated, uint8_t *xq, float *xs, int m, int k, void *stream) {
  if (!type_ok(x_type)) return QMV_ERR_RANGE;
  if (m < 0 || m > QMM_MAX_ROWS) return QMV_ERR_RANGE;
  const int rc = check_nk(1, k, 8);
  if (rc) return rc;
  if (m == 0) return QMV_OK;
  if (!x || !xq || !xs) return QMV_ERR_NULL;
  if (!aligned(x, 16) || !aligned(xq, 16) || !aligned(xs, 4)) return QMV_ERR_ALIGN;
  const size_t xb = (size_t)m * k * type_bytes(x_type) * (gated ? 2 : 1), qb = (size_t)m * k;
  const size_t sb = (size_t)m * qmv::fp8::blocks_of(k) * 4;
  if (overlap(xq, qb, x, xb) || overlap(xs, sb, x, xb) || overlap(xq, qb, xs, sb)) return QMV_ERR_ALIAS;
  return qmv::launch_fp8_quant(x, x_type == QMM_F32, gated, xq, xs, m, k, stream);
}

// The checks the two grouped products share; value_bytes: 1 (e4m3) or 2 (bf16).
int grouped(const void *w, size_t w_bytes, const float *w_scale, const void *x, const float *x_scale,
            const int32_t *offsets, const int32_t *row_index, void *y, int y_type, int rows, int x_rows, int n, int k,
            int n_experts, int value_bytes, void *stream) {
  const bool e4m3 = value_bytes == 1, fast = e4m3 && take_fast(&y_type), exact = e4m3 && !fast;
  if (!type_ok(y_type)) return QMV_ERR_RANGE;
  if (rows < 0 || rows > QMM_MAX_ROWS || x_rows < 0 || x_rows > QMM_MAX_ROWS || n_experts < 1 ||
      n_experts > QMM_MAX_EXPERTS)
    return QMV_ERR_RANGE;
  const int rc = check_nk(n, k, 16 / value_bytes);
  if (rc) return rc;
  if (!row_index && x_rows != rows) return QMV_ERR_SHAPE;
  if (!w || !offsets || (e4m3 && !w_scale)) return QMV_ERR_NULL;
  const size_t wb = (size_t)n_experts * n * k * value_bytes;   // <= 2^51
  if (w_bytes != wb) return QMV_ERR_SIZE;
  if (rows == 0) return QMV_OK;
  if (!qmv::fp8::grouped_in_grid(rows, n_experts, n, qmv::fp8::blocks_of(k * value_bytes), exact)) return QMV_ERR_RANGE;
  // rows are gathered by 32-bit byte offsets
  if (row_index && (size_t)x_rows * k * value_bytes > UINT32_MAX) return QMV_ERR_RANGE;
  // with no row of x every index is out of range, and x itself may be null
  if (!y || (x_rows > 0 && (!x || (e4m3 && !x_scale)))) return QMV_ERR_NULL;
  if (!aligned(w, 16) || !aligned(x, 16) || !aligned(y, 16) || !aligned(w_scale, 4) || !aligned(x_scale, 4) ||
      !aligned(offsets, 4) || !aligned(row_index, 4))
    return QMV_ERR_ALIGN;
  const size_t nb = (size_t)qmv::fp8::blocks_of(k);
  const size_t yb = (size_t)rows * n * type_bytes(y_type);
  const void *in_p[] = {w, w_scale, x, x_scale, offsets, row_index};
  const size_t in_b[] = {wb, e4m3 ? (size_t)n_experts * qmv::fp8::blocks_of(n) * nb * 4 : 0,
                         (size_t)x_rows * k * value_bytes, e4m3 ? (size_t)x_rows * nb * 4 : 0,
                         ((size_t)n_experts + 1) * 4, row_index ? (size_t)rows * 4 : 0};
  for (int i = 0; i < 6; ++i)
    if (overlap(y, yb, in_p[i], in_b[i])) return QMV_ERR_ALIAS;
  qmv::ProductArgs a{};
  a.w = static_cast<const uint8_t *>(w);
  a.w_scale = w_scale;
  a.x = static_cast<const uint8_t *>(x);
  a.x_scale = x_scale;
  a.offsets = offsets;
  a.index = row_index;
  a.y = y;
  a.rows = rows;
  a.x_rows = x_rows;
  a.n = n;
  a.k_bytes = k * value_bytes;
  a.nb = qmv::fp8::blocks_of(a.k_bytes);
  a.n_experts = n_experts;
  a.y_bf16 = y_type == QMM_BF16;
  a.fast = fast;
  return e4m3 ? qmv::launch_fp8_grouped(a, stream) : qmv::launch_bf16_grouped(a, stream);
}

bool dense_in_range(int m, int n, int k) {
  return m >= 1 && m <= QMM_MAX_ROWS && check_nk(n, k, 16) == QMV_OK && qmv::fp8::dense_in_grid(m, n);
}

}  // namespace

extern "C" {

int qmm_fp8_quant(const void *x, int x_type, uint8_t *xq, float *xs, int m, int k, void *stream) {
  return quant(x, x_type, false, xq, xs, m, k, stream);
}

int qmm_fp8_quant_silu_mul(const void *x, int x_type, uint8_t *xq, float *xs, int m, int k, void *stream) {
  return quant(x, x_type, true, xq, xs, m, k, stream);
}

size_t qmm_fp8_workspace(int m, int n, int k, int y_type) {
  const bool fast = take_fast(&y_type);
  if (!type_ok(y_type) || !dense_in_range(m, n, k)) return 0;
  return qmv::fp8::dense_workspace(m, n, k, fast);
}

int qmm_fp8(const void *w, size_t w_bytes, const float *w_scale, const void *x, const float *x_scale, void *y,
            int y_type, int m, int n, int k, void *ws, size_t ws_bytes, void *stream) {
  if (!w || !w_scale || !x || !x_scale || !y) return QMV_ERR_NULL;
  const bool fast = take_fast(&y_type);
  if (!type_ok(y_type)) return QMV_ERR_RANGE;
  if (m < 1 || m > QMM_MAX_ROWS) return QMV_ERR_RANGE;
  const int rc = check_nk(n, k, 16);
  if (rc) return rc;
  if (!dense_in_range(m, n, k)) return QMV_ERR_RANGE;
  const size_t wb = (size_t)n * k;
  if (w_bytes != wb) return QMV_ERR_SIZE;
  if (!aligned(w, 16) || !aligned(x, 16) || !aligned(y, 16) || !aligned(w_scale, 4) || !aligned(x_scale, 4) ||
      !aligned(ws, 256))
    return QMV_ERR_ALIGN;
  const size_t nb = (size_t)qmv::fp8::blocks_of(k);
  const size_t yb = (size_t)m * n * type_bytes(y_type), need = qmv::fp8::dense_workspace(m, n, k, fast);
  const void *in_p[] = {w, w_scale, x, x_scale};
  const size_t in_b[] = {wb, (size_t)qmv::fp8::blocks_of(n) * nb * 4, (size_t)m * k, (size_t)m * nb * 4};
  for (int i = 0; i < 4; ++i)
    if (overlap(y, yb, in_p[i], in_b[i])) return QMV_ERR_ALIAS;
  if (need) {
    if (!ws || ws_bytes < need) return QMV_ERR_WORKSPACE;
    if (overlap(ws, need, y, yb)) return QMV_ERR_ALIAS;
    for (int i = 0; i < 4; ++i)
      if (overlap(ws, need, in_p[i], in_b[i])) return QMV_ERR_ALIAS;
  }
  qmv::ProductArgs a{};
  a.w = static_cast<const uint8_t *>(w);
  a.w_scale = w_scale;
  a.x = static_cast<const uint8_t *>(x);
  a.x_scale = x_scale;
  a.y = y;
  a.part = need ? static_cast<float *>(ws) : nullptr;
  a.rows = m;
  a.x_rows = m;
  a.n = n;
  a.k_bytes = k;
  a.nb = qmv::fp8::blocks_of(k);
  a.n_experts = 1;
  a.y_bf16 = y_type == QMM_BF16;
  a.fast = fast;
  return qmv::launch_fp8_dense(a, stream);
}

int qmm_fp8_grouped(const void *w, size_t w_bytes, const float *w_scale, const void *x, const float *x_scale,
                    const int32_t *offsets, const int32_t *row_index, void *y, int y_type, int rows, int x_rows,
                    int n, int k, int n_experts, void *stream) {
  return grouped(w, w_bytes, w_scale, x, x_scale, offsets, row_index, y, y_type, rows, x_rows, n, k, n_experts, 1,
                 stream);
}

int qmm_bf16_grouped(const uint16_t *w_bf16, size_t w_bytes, const uint16_t *x_bf16, const int32_t *offsets,
                     const int32_t *row_index, void *y, int y_type, int rows, int x_rows, int n, int k, int n_experts,
                     void *stream) {
  return grouped(w_bf16, w_bytes, nullptr, x_bf16, nullptr, offsets, row_index, y, y_type, rows, x_rows, n, k,
                 n_experts, 2, stream);
}

}  // extern "C"
