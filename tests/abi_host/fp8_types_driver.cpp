// Every y_type with every product, QMM_FAST_SUMS among them, in a host-only
// build (fp8_api.cpp + stand-in launchers, no HIP runtime) under the address and
// undefined-behaviour sanitizers: what is refused, what reaches a launcher, and
// the plan that an accepted call takes. Pointers are fake. Exit status 0: every
// expectation held.
#include <initializer_list>
#include <limits.h>
#include <stdint.h>
#include <stdio.h>

#include "../../gguf_block_quantized_qmv_amd/csrc/fp8_internal.h"
#include "../../gguf_block_quantized_qmv_amd/csrc/fp8_layout.h"
#include "../../include/qmm_fp8.h"

namespace stub {
extern int launches;
extern qmv::ProductArgs last;
}  // namespace stub

namespace {

namespace fp8 = qmv::fp8;
int failures = 0;
#define EXPECT(cond)                                                                \
  do {                                                                              \
    if (!(cond)) {                                                                  \
      if (++failures < 20) fprintf(stderr, "%s:%d: failed: %s\n", __FILE__, __LINE__, #cond); \
    }                                                                               \
  } while (0)

// Regions of 4 PiB: no argument reaches the next one.
void *at(int region) { return reinterpret_cast<void *>((uintptr_t)(region + 1) << 52); }

const int kRows[] = {1, 2, 15, 16, 17, 31, 32, 33, 64, 65, 127, 128, 129, 256, 257, 768, 1000, 2064, 17408, 65536, 65537, 1 << 20, 1 << 24};
const int kCols[] = {1, 16, 63, 64, 65, 127, 128, 129, 257, 1000, 5120, 17408, 65537, 1 << 20};
const int kDepth[] = {16, 48, 128, 144, 768, 2064, 5120, 17408, 1 << 20};
const int kExperts[] = {1, 2, 63, 64, 65, 128, 1024};
const int kFast = QMM_BF16 | QMM_FAST_SUMS;

void dense_plan_holds(int m, int n, int k, bool fast, size_t need) {
  const int nb = fp8::blocks_of(k);
  const fp8::DensePlan p = fp8::dense_plan(m, n, k, fast);
  EXPECT(m > QMM_SAME_ROWS || p.stream);
  if (p.stream) {
    EXPECT(need == 0);
    return;
  }
  EXPECT(p.tile >= fp8::kTile32 && p.tile <= (fast ? fp8::kTile256Wide : fp8::kTile256));
  EXPECT((int64_t)p.t_main + p.r_tiles ==
         (int64_t)fp8::ceil_div(m, fp8::tile_rows(p.tile)) * fp8::ceil_div(n, fp8::tile_cols(p.tile)));
  EXPECT(p.splits >= 1 && p.splits <= 16 && (p.splits > 1) == (p.r_tiles > 0));
  EXPECT(p.splits == 1 || (nb / p.splits >= 4 && (int64_t)p.r_tiles * p.splits <= fp8::kSlots));
  EXPECT(need == (size_t)(p.splits > 1 ? p.r_tiles * p.splits : 0) * fp8::tile_rows(p.tile) * fp8::tile_cols(p.tile) * 4);
}

void dense() {
  const float *ws = static_cast<const float *>(at(1)), *xs = static_cast<const float *>(at(3));
  const int types[] = {QMM_F32, QMM_BF16, kFast, QMM_F32 | QMM_FAST_SUMS, QMM_FAST_SUMS << 1 | QMM_BF16, 2, -1, INT_MIN, INT_MAX};
  for (int m : kRows)
    for (int n : kCols)
      for (int k : kDepth)
        for (int t : types) {
          const bool good = t == QMM_F32 || t == QMM_BF16 || t == kFast;
          const size_t need = qmm_fp8_workspace(m, n, k, t);
          const int before = stub::launches;
          const int rc = qmm_fp8(at(0), (size_t)n * k, ws, at(2), xs, at(9), t, m, n, k, need ? at(4) : nullptr, need, nullptr);
          EXPECT((rc == QMV_OK) == (good && fp8::dense_in_grid(m, n)));
          EXPECT(rc == QMV_OK || rc == QMV_ERR_RANGE);
          EXPECT(stub::launches == before + (rc == QMV_OK));
          if (rc != QMV_OK) {
            EXPECT(need == 0);
            continue;
          }
          EXPECT(stub::last.y_bf16 == (t != QMM_F32) && stub::last.fast == (t == kFast));
          EXPECT((stub::last.part != nullptr) == (need > 0));
          dense_plan_holds(m, n, k, t == kFast, need);
          // results of either type under fp32 sums take one plan
          EXPECT(t != QMM_BF16 || need == qmm_fp8_workspace(m, n, k, QMM_F32));
        }
}

void grouped() {
  const float *ws = static_cast<const float *>(at(1)), *xs = static_cast<const float *>(at(3));
  const int32_t *off = static_cast<const int32_t *>(at(5)), *idx = static_cast<const int32_t *>(at(6));
  for (int rows : kRows)
    for (int n : kCols)
      for (int k : kDepth)
        for (int e : kExperts)
          for (int t : {QMM_F32, QMM_BF16, kFast, QMM_F32 | QMM_FAST_SUMS})
            for (int vb = 1; vb <= 2; ++vb) {
              const size_t bytes = (size_t)e * n * k * vb;
              const bool good = t == QMM_F32 || t == QMM_BF16 || (t == kFast && vb == 1), exact = vb == 1 && t != kFast;
              const int before = stub::launches, nb = fp8::blocks_of(k * vb);
              const int rc = vb == 2 ? qmm_bf16_grouped(static_cast<const uint16_t *>(at(0)), bytes,
                                                        static_cast<const uint16_t *>(at(2)), off, idx, at(9), t, rows, 100, n, k, e, nullptr)
                                     : qmm_fp8_grouped(at(0), bytes, ws, at(2), xs, off, idx, at(9), t, rows, 100, n, k, e, nullptr);
              EXPECT((rc == QMV_OK) == (good && fp8::grouped_in_grid(rows, e, n, nb, exact)));
              EXPECT(rc == QMV_OK || rc == QMV_ERR_RANGE);
              EXPECT(stub::launches == before + (rc == QMV_OK));
              if (rc != QMV_OK) continue;
              EXPECT(stub::last.y_bf16 == (t != QMM_F32) && stub::last.fast == (t == kFast));
              const int tile = fp8::grouped_tile(rows, e, n, nb, exact);
              EXPECT(tile == fp8::kTile32 || tile == fp8::kTile64 || tile == (exact ? fp8::kTile256 : fp8::kTile256Wide) ||
                     (!exact && tile == fp8::kTile128));
              EXPECT(fp8::grouped_row_tiles(rows, e, fp8::tile_rows(tile)) * fp8::ceil_div(n, fp8::tile_cols(tile)) <= fp8::kMaxTiles);
              EXPECT((int64_t)fp8::tile_rows(tile) * k * vb <= (int64_t)UINT32_MAX && (int64_t)fp8::tile_cols(tile) * k * vb <= (int64_t)UINT32_MAX);
            }
}

void quant() {
  uint8_t *xq = static_cast<uint8_t *>(at(2));
  float *xs = static_cast<float *>(at(3));
  for (int t : {QMM_F32 | QMM_FAST_SUMS, kFast, 2, INT_MAX}) {
    EXPECT(qmm_fp8_quant(at(0), t, xq, xs, 4, 128, nullptr) == QMV_ERR_RANGE);
    EXPECT(qmm_fp8_quant_silu_mul(at(0), t, xq, xs, 4, 128, nullptr) == QMV_ERR_RANGE);
  }
}

}  // namespace

int main() {
  dense();
  grouped();
  quant();
  printf("%d failures, %d launches\n", failures, stub::launches);
  return failures ? 1 : 0;
}
