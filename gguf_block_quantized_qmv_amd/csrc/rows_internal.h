// Launch interface between rows_api.cpp (pure host code) and the HIP files of
// the rows' operators and of the verification of drafts. Arguments are
// validated when these are called; each returns QMV_OK or QMV_ERR_HIP.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace qmv {

struct SortArgs {
  const int32_t *ids;
  int32_t *offsets, *row_index, *places;   // the last two may be null
  int32_t *counts;                         // the workspace, where the plan has parts
  int choices, top_k, n_experts;
};

// Rows of `width` fp32 or bf16 values, choices [tokens][top_k].
struct MoveArgs {
  const void *x;           // spread: x; combine: z; gradient: dy
  const void *z;           // gradient: z, or null
  const int32_t *places;
  const float *w;          // or null
  void *out;               // spread: out; combine: y; gradient: dz
  float *dw;               // gradient, or null
  int tokens, top_k, width, rows, in_f32, out_f32;
};

struct LoraArgs {
  const uint16_t *a, *b, *x;
  const float *scale;             // or null
  const int32_t *ranks;           // or null
  const int32_t *offsets, *index; // index: or null
  const void *base;
  void *y;
  float *part;
  int y_f32, rows, x_rows, n, k, rank, n_adapters;
};

struct VerifyArgs {
  const void *p, *q;              // q: or null
  const int32_t *tokens, *lengths;
  const float *u;
  int32_t *accepted, *out;
  double *sums;
  int f32, requests, drafts, vocab;
};

int launch_rows_sort(const SortArgs &a, void *stream);
int launch_rows_spread(const MoveArgs &a, void *stream);
int launch_rows_combine(const MoveArgs &a, void *stream);
int launch_rows_combine_grad(const MoveArgs &a, void *stream);
int launch_lora(const LoraArgs &a, void *stream);
int launch_verify_drafts(const VerifyArgs &a, void *stream);

}  // namespace qmv
