// Launch interface between fp8_api.cpp (pure host code) and the HIP files of
// the e4m3 and grouped products. Arguments are validated when these are called;
// each returns QMV_OK or QMV_ERR_HIP.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace qmv {

// One product call. Bytes, not values, along k: k_bytes is the length of a row
// of x and of w, nb its blocks of 128 bytes.
struct ProductArgs {
  const uint8_t *w;
  const float *w_scale;    // null: bf16
  const uint8_t *x;
  const float *x_scale;
  const int32_t *offsets;  // null: dense
  const int32_t *index;    // null: row r of x
  void *y;
  float *part;             // the workspace of a dense plan with parts
  int rows, x_rows, n, k_bytes, nb, n_experts, y_bf16;
  int fast;                // e4m3: QMM_FAST_SUMS
};

int launch_fp8_quant(const void *x, bool x_f32, bool gated, uint8_t *xq, float *xs, int m, int k, void *stream);
int launch_fp8_dense(const ProductArgs &a, void *stream);
int launch_fp8_grouped(const ProductArgs &a, void *stream);
int launch_bf16_grouped(const ProductArgs &a, void *stream);

}  // namespace qmv
