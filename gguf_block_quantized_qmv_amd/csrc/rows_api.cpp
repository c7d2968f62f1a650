// C ABI of the rows' operators and of the verification of drafts: argument
// validation and dispatch. Pure host code: it calls no HIP function and reads no
// device property. See include/qmm_rows.h and include/qmv_verify.h for the
// contract of each entry point.
#include <stdint.h>

#include "rows_internal.h"
#include "rows_layout.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct Span {
  const void *p;
  size_t bytes;
};

// The two share a byte.
bool overlap(const Span &s, const Span &t) {
  if (!s.p || !t.p || s.bytes == 0 || t.bytes == 0) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(s.p), b = reinterpret_cast<uintptr_t>(t.p);
  return a < b + t.bytes && b < a + s.bytes;
}

// Any of the first `outs` arrays shares a byte with another array.
template <size_t N>
bool any_overlap(const Span (&s)[N], size_t outs) {
  for (size_t i = 0; i < outs; ++i)
    for (size_t j = i + 1; j < N; ++j)
      if (overlap(s[i], s[j])) return true;
  return false;
}

bool type_ok(int t) { return t == QMM_F32 || t == QMM_BF16; }
size_t type_bytes(int t) { return t == QMM_F32 ? 4 : 2; }

// tokens >= 0 and 1 <= top_k, both and their product within range.
bool choices_ok(int tokens, int top_k) {
  return tokens >= 0 && top_k >= 1 && top_k <= QMM_MAX_TOP_K && (int64_t)tokens * top_k <= QMM_MAX_ROWS;
}

int check_move(int tokens, int top_k, int h, int rows) {
  if (!choices_ok(tokens, top_k) || rows < 0 || rows > QMM_MAX_ROWS) return QMV_ERR_RANGE;
  if (h < 1) return QMV_ERR_SHAPE;
  return h > QMM_MAX_K ? QMV_ERR_RANGE : QMV_OK;
}

int check_lora(int rows, int n, int k, int rank, int n_adapters) {
  if (rows < 0 || rows > QMM_MAX_ROWS || n_adapters < 1 || n_adapters > QMM_MAX_EXPERTS) return QMV_ERR_RANGE;
  if (n < 1 || k < 8 || k % 8 || rank < 8 || rank % 8) return QMV_ERR_SHAPE;
  if (n > QMM_MAX_N || k > QMM_MAX_K || rank > QMM_MAX_RANK) return QMV_ERR_RANGE;
  return qmv::rows::lora_in_grid(rows, n, n_adapters) ? QMV_OK : QMV_ERR_RANGE;
}

bool verify_ok(int requests, int vocab) {
  return requests >= 0 && requests <= QMV_MAX_REQUESTS && vocab >= 1 && vocab <= QMV_MAX_VOCAB;
}

}  // namespace

extern "C" {

size_t qmm_rows_sort_workspace(int tokens, int top_k, int n_experts) {
  if (!choices_ok(tokens, top_k) || n_experts < 1 || n_experts > QMM_MAX_EXPERTS) return 0;
  return qmv::rows::sort_workspace(tokens * top_k, n_experts);
}

int qmm_rows_sort(const int32_t *ids, int32_t *offsets, int32_t *row_index, int32_t *places, int tokens, int top_k,
                  int n_experts, void *ws, size_t ws_bytes, void *stream) {
  if (!choices_ok(tokens, top_k) || n_experts < 1 || n_experts > QMM_MAX_EXPERTS) return QMV_ERR_RANGE;
  const int choices = tokens * top_k;
  if (!offsets || (choices > 0 && !ids)) return QMV_ERR_NULL;
  if (!aligned(ids, 4) || !aligned(offsets, 4) || !aligned(row_index, 4) || !aligned(places, 4) || !aligned(ws, 256))
    return QMV_ERR_ALIGN;
  const size_t need = qmv::rows::sort_workspace(choices, n_experts), cb = (size_t)choices * 4;
  if (need && (!ws || ws_bytes < need)) return QMV_ERR_WORKSPACE;
  const Span all[] = {{offsets, ((size_t)n_experts + 1) * 4}, {row_index, cb}, {places, cb}, {ws, need}, {ids, cb}};
  if (any_overlap(all, 4)) return QMV_ERR_ALIAS;
  qmv::SortArgs a{};
  a.ids = ids;
  a.offsets = offsets;
  a.row_index = row_index;
  a.places = places;
  a.counts = need ? static_cast<int32_t *>(ws) : nullptr;
  a.choices = choices;
  a.top_k = top_k;
  a.n_experts = n_experts;
  return qmv::launch_rows_sort(a, stream);
}

int qmm_rows_spread(const void *x, int type, const int32_t *places, void *out, int tokens, int top_k, int h, int rows,
                    void *stream) {
  if (!type_ok(type)) return QMV_ERR_RANGE;
  const int rc = check_move(tokens, top_k, h, rows);
  if (rc) return rc;
  if (tokens == 0 || rows == 0) return QMV_OK;
  if (!x || !places || !out) return QMV_ERR_NULL;
  if (!aligned(x, 16) || !aligned(out, 16) || !aligned(places, 4)) return QMV_ERR_ALIGN;
  const size_t row = (size_t)h * type_bytes(type);
  const Span all[] = {{out, rows * row}, {x, tokens * row}, {places, (size_t)tokens * top_k * 4}};
  if (any_overlap(all, 1)) return QMV_ERR_ALIAS;
  qmv::MoveArgs a{};
  a.x = x;
  a.places = places;
  a.out = out;
  a.tokens = tokens;
  a.top_k = top_k;
  a.width = h;
  a.rows = rows;
  a.in_f32 = a.out_f32 = type == QMM_F32;
  return qmv::launch_rows_spread(a, stream);
}

int qmm_rows_combine(const void *z, int z_type, const int32_t *places, const float *w, void *y, int y_type, int tokens,
                     int top_k, int h, int rows, void *stream) {
  if (!type_ok(z_type) || !type_ok(y_type)) return QMV_ERR_RANGE;
  const int rc = check_move(tokens, top_k, h, rows);
  if (rc) return rc;
  if (tokens == 0) return QMV_OK;
  if (!places || !y || (rows > 0 && !z)) return QMV_ERR_NULL;   // without a row every choice adds nothing
  if (!aligned(z, 16) || !aligned(y, 16) || !aligned(places, 4) || !aligned(w, 4)) return QMV_ERR_ALIGN;
  const size_t choices = (size_t)tokens * top_k * 4;
  const Span all[] = {{y, (size_t)tokens * h * type_bytes(y_type)},
                      {z, (size_t)rows * h * type_bytes(z_type)},
                      {places, choices},
                      {w, choices}};
  if (any_overlap(all, 1)) return QMV_ERR_ALIAS;
  qmv::MoveArgs a{};
  a.x = z;
  a.places = places;
  a.w = w;
  a.out = y;
  a.tokens = tokens;
  a.top_k = top_k;
  a.width = h;
  a.rows = rows;
  a.in_f32 = z_type == QMM_F32;
  a.out_f32 = y_type == QMM_F32;
  return qmv::launch_rows_combine(a, stream);
}

int qmm_rows_combine_grad(const void *dy, const void *z, int type, const int32_t *places, const float *w, void *dz,
                          float *dw, int tokens, int top_k, int h, int rows, void *stream) {
  if (!type_ok(type)) return QMV_ERR_RANGE;
  const int rc = check_move(tokens, top_k, h, rows);
  if (rc) return rc;
  if (tokens == 0) return QMV_OK;
  if (!dy || !places || (rows > 0 && (!dz || !z != !dw))) return QMV_ERR_NULL;
  if (!aligned(dy, 16) || !aligned(z, 16) || !aligned(dz, 16) || !aligned(places, 4) || !aligned(w, 4) || !aligned(dw, 4))
    return QMV_ERR_ALIGN;
  const size_t row = (size_t)h * type_bytes(type), choices = (size_t)tokens * top_k * 4;
  const Span all[] = {{dz, rows * row}, {dw, choices}, {dy, tokens * row}, {z, rows * row}, {places, choices}, {w, choices}};
  if (any_overlap(all, 2)) return QMV_ERR_ALIAS;
  if (rows == 0 && !dw) return QMV_OK;
  qmv::MoveArgs a{};
  a.x = dy;
  a.z = z;
  a.places = places;
  a.w = w;
  a.out = dz;
  a.dw = dw;
  a.tokens = tokens;
  a.top_k = top_k;
  a.width = h;
  a.rows = rows;
  a.in_f32 = a.out_f32 = type == QMM_F32;
  return qmv::launch_rows_combine_grad(a, stream);
}

size_t qmm_lora_workspace(int rows, int n, int k, int rank, int n_adapters) {
  if (check_lora(rows, n, k, rank, n_adapters) || rows == 0) return 0;
  return qmv::rows::lora_workspace(rows, n, k, rank, n_adapters);
}

int qmm_lora(const uint16_t *a, size_t a_bytes, const uint16_t *b, size_t b_bytes, const float *scale,
             const int32_t *ranks, const uint16_t *x, const int32_t *offsets, const int32_t *row_index,
             const void *base, void *y, int y_type, int rows, int x_rows, int n, int k, int rank, int n_adapters,
             void *ws, size_t ws_bytes, void *stream) {
  if (!type_ok(y_type) || x_rows < 0 || x_rows > QMM_MAX_ROWS) return QMV_ERR_RANGE;
  const int rc = check_lora(rows, n, k, rank, n_adapters);
  if (rc) return rc;
  if (!row_index && x_rows != rows) return QMV_ERR_SHAPE;
  if (!a || !b || !offsets) return QMV_ERR_NULL;
  const size_t ab = (size_t)n_adapters * rank * k * 2, bb = (size_t)n_adapters * n * rank * 2;
  if (a_bytes != ab || b_bytes != bb) return QMV_ERR_SIZE;
  if (rows == 0 || x_rows == 0) return QMV_OK;   // no row of x: every index is passed over
  if (!x || !base || !y) return QMV_ERR_NULL;
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(x, 16) || !aligned(base, 16) || !aligned(y, 16) ||
      !aligned(scale, 4) || !aligned(ranks, 4) || !aligned(offsets, 4) || !aligned(row_index, 4) || !aligned(ws, 256))
    return QMV_ERR_ALIGN;
  const size_t need = qmv::rows::lora_workspace(rows, n, k, rank, n_adapters);
  if (need && (!ws || ws_bytes < need)) return QMV_ERR_WORKSPACE;
  const size_t yb = (size_t)x_rows * n * type_bytes(y_type), eb = (size_t)n_adapters * 4;
  const Span all[] = {{y, yb},      {ws, need},   {a, ab},
                      {b, bb},      {scale, eb},  {ranks, eb},
                      {x, (size_t)x_rows * k * 2}, {offsets, eb + 4}, {row_index, (size_t)rows * 4},
                      {base == y ? nullptr : base, yb}};
  if (any_overlap(all, 2)) return QMV_ERR_ALIAS;
  qmv::LoraArgs v{};
  v.a = a;
  v.b = b;
  v.x = x;
  v.scale = scale;
  v.ranks = ranks;
  v.offsets = offsets;
  v.index = row_index;
  v.base = base;
  v.y = y;
  v.part = static_cast<float *>(ws);
  v.y_f32 = y_type == QMM_F32;
  v.rows = rows;
  v.x_rows = x_rows;
  v.n = n;
  v.k = k;
  v.rank = rank;
  v.n_adapters = n_adapters;
  return qmv::launch_lora(v, stream);
}

size_t qmv_verify_drafts_workspace(int requests, int vocab) {
  return verify_ok(requests, vocab) ? qmv::rows::verify_workspace(requests, vocab) : 0;
}

int qmv_verify_drafts(const void *p, const void *q, int type, const int32_t *tokens, const int32_t *lengths,
                      const float *u, int32_t *accepted, int32_t *out, int requests, int drafts, int vocab, void *ws,
                      size_t ws_bytes, void *stream) {
  if (!type_ok(type) || drafts < 0 || drafts > QMV_MAX_DRAFTS || requests < 0 || requests > QMV_MAX_REQUESTS)
    return QMV_ERR_RANGE;
  if (vocab < 1) return QMV_ERR_SHAPE;
  if (vocab > QMV_MAX_VOCAB) return QMV_ERR_RANGE;
  if (requests == 0) return QMV_OK;
  if (!p || !u || !accepted || !out || (drafts > 0 && !tokens)) return QMV_ERR_NULL;
  if (!aligned(p, 16) || !aligned(q, 16) || !aligned(tokens, 4) || !aligned(lengths, 4) || !aligned(u, 4) ||
      !aligned(accepted, 4) || !aligned(out, 4) || !aligned(ws, 256))
    return QMV_ERR_ALIGN;
  const size_t need = qmv::rows::verify_workspace(requests, vocab);
  if (need && (!ws || ws_bytes < need)) return QMV_ERR_WORKSPACE;
  const size_t r = (size_t)requests, row = (size_t)vocab * type_bytes(type);
  const Span all[] = {{accepted, r * 4}, {out, r * (drafts + 1) * 4}, {ws, need}, {p, r * (drafts + 1) * row},
                      {q, r * drafts * row}, {tokens, r * drafts * 4}, {lengths, r * 4}, {u, r * (drafts + 1) * 4}};
  if (any_overlap(all, 3)) return QMV_ERR_ALIAS;
  qmv::VerifyArgs v{};
  v.p = p;
  v.q = q;
  v.tokens = tokens;
  v.lengths = lengths;
  v.u = u;
  v.accepted = accepted;
  v.out = out;
  v.sums = need ? static_cast<double *>(ws) : nullptr;
  v.f32 = type == QMM_F32;
  v.requests = requests;
  v.drafts = drafts;
  v.vocab = vocab;
  return qmv::launch_verify_drafts(v, stream);
}

}  // extern "C"
