// Drives the argument checks and plans of the rows' operators and of the
// verification of drafts in a host-only build (rows_api.cpp + stand-in launchers,
// no HIP runtime) under the address and undefined-behaviour sanitizers. Pointers
// are fake: a call is refused or reaches a stand-in. Exit status 0: every
// expectation held.
#include <limits.h>
#include <stdint.h>
#include <stdio.h>

#include <initializer_list>

#include "../../gguf_block_quantized_qmv_amd/csrc/rows_internal.h"
#include "../../gguf_block_quantized_qmv_amd/csrc/rows_layout.h"

namespace stub {
extern int launches;
extern qmv::SortArgs sort;
extern qmv::MoveArgs move;
extern qmv::LoraArgs lora;
extern qmv::VerifyArgs verify;
}  // namespace stub

namespace {

int failures = 0;
#define EXPECT(cond)                                                                \
  do {                                                                              \
    if (!(cond)) {                                                                  \
      if (++failures < 20) fprintf(stderr, "%s:%d: failed: %s\n", __FILE__, __LINE__, #cond); \
    }                                                                               \
  } while (0)

// 16 regions of 2^47 bytes each would not fit an address: the largest arrays are 2^46.
template <class T = void>
T *at(int region) {
  return reinterpret_cast<T *>((uintptr_t)0x1000000 + ((uintptr_t)region << 50));
}

const int kInts[] = {INT_MIN, -257, -1, 0, 1, 2, 7, 8, 16, 17, 31, 32, 33, 64, 100, 128, 129, 136, 1000, 1023, 1024, 1025, 4096,
                     4097, 16384, 16385, 65535, 65536, 1 << 20, (1 << 20) + 8, 1 << 22, (1 << 22) + 1, 1 << 24, (1 << 24) + 1, INT_MAX};

bool is_code(int rc) { return rc <= 0 && rc >= QMV_ERR_HIP; }

void sort() {
  for (int t : kInts)
    for (int k : kInts)
      for (int e : kInts) {
        const size_t need = qmm_rows_sort_workspace(t, k, e);
        const int before = stub::launches;
        const int rc = qmm_rows_sort(at<int32_t>(0), at<int32_t>(1), at<int32_t>(2), at<int32_t>(3), t, k, e,
                                     need ? at<>(4) : nullptr, need, nullptr);
        EXPECT(is_code(rc) && (rc == QMV_OK) == (stub::launches == before + 1));
        if (rc != QMV_OK) {
          EXPECT(need == 0);
          continue;
        }
        EXPECT(t >= 0 && k >= 1 && k <= 32 && e >= 1 && e <= 1024 && (int64_t)t * k <= QMM_MAX_ROWS);
        EXPECT(stub::sort.choices == t * k && (stub::sort.counts != nullptr) == (need > 0));
        const qmv::rows::SortPlan p = qmv::rows::sort_plan(t * k);
        EXPECT(p.parts >= 1 && p.parts <= qmv::rows::kSortParts && p.chunk % qmv::rows::kSortTile == 0);
        EXPECT((int64_t)p.parts * p.chunk >= t * k && (p.parts == 1 || (int64_t)(p.parts - 1) * p.chunk < t * k));
        EXPECT(need == (t * k > qmv::rows::kSortCounts ? (size_t)p.parts * e * 4 : 0));
        if (need) {
          EXPECT(qmm_rows_sort(at<int32_t>(0), at<int32_t>(1), nullptr, nullptr, t, k, e, nullptr, 0, nullptr) == QMV_ERR_WORKSPACE);
          EXPECT(qmm_rows_sort(at<int32_t>(0), at<int32_t>(1), nullptr, nullptr, t, k, e, at<>(4), need - 1, nullptr) == QMV_ERR_WORKSPACE);
        }
      }
}

void move() {
  for (int t : kInts)
    for (int k : {-1, 0, 1, 2, 8, 32, 33, INT_MAX})
      for (int h : kInts)
        for (int rows : kInts)
          for (int ty = -1; ty <= 2; ++ty) {
            int before = stub::launches;
            int rc = qmm_rows_spread(at<>(0), ty, at<int32_t>(1), at<>(2), t, k, h, rows, nullptr);
            EXPECT(is_code(rc));
            EXPECT(stub::launches == before + (rc == QMV_OK && t > 0 && rows > 0 ? 1 : 0));
            before = stub::launches;
            rc = qmm_rows_combine(at<>(0), ty, at<int32_t>(1), at<float>(3), at<>(2), QMM_BF16, t, k, h, rows, nullptr);
            EXPECT(is_code(rc));
            EXPECT(stub::launches == before + (rc == QMV_OK && t > 0 ? 1 : 0));
            before = stub::launches;
            rc = qmm_rows_combine_grad(at<>(0), at<>(4), ty, at<int32_t>(1), nullptr, at<>(2), at<float>(5), t, k, h, rows, nullptr);
            EXPECT(is_code(rc));
            EXPECT(stub::launches == before + (rc == QMV_OK && t > 0 ? 1 : 0));
            if (rc != QMV_OK || t == 0) continue;
            EXPECT(k >= 1 && k <= 32 && (int64_t)t * k <= QMM_MAX_ROWS && h >= 1 && h <= QMM_MAX_K && rows >= 0 && rows <= QMM_MAX_ROWS);
            // the grids' second dimension, pieces of 16 bytes by at least eight lanes
            EXPECT(qmv::rows::ceil_div(qmv::rows::ceil_div(h, 4), 8) <= 65535);
          }
}

void lora() {
  for (int rows : kInts)
    for (int n : kInts)
      for (int k : {0, 8, 12, 64, 72, 640, 5120, 17408, 1 << 20, (1 << 20) + 8, INT_MAX / 8 * 8})
        for (int rank : {-8, 0, 8, 12, 16, 24, 32, 64, 72, 128, 136, INT_MAX / 8 * 8})
          for (int e : {INT_MIN, 0, 1, 3, 64, 65, 1024, 1025}) {
            const size_t ab = e > 0 && rank > 0 && k > 0 ? (size_t)e * rank * k * 2 : 1;
            const size_t bb = e > 0 && rank > 0 && n > 0 ? (size_t)e * rank * n * 2 : 1;
            const size_t need = qmm_lora_workspace(rows, n, k, rank, e);
            for (int gather = 0; gather < 2; ++gather) {
              const int before = stub::launches, x_rows = gather ? 100 : rows;
              const int rc = qmm_lora(at<uint16_t>(0), ab, at<uint16_t>(1), bb, at<float>(2), at<int32_t>(3), at<uint16_t>(4),
                                      at<int32_t>(5), gather ? at<int32_t>(6) : nullptr, at<>(7), at<>(8), QMM_BF16, rows,
                                      x_rows, n, k, rank, e, need ? at<>(9) : nullptr, need, nullptr);
              EXPECT(is_code(rc));
              EXPECT(stub::launches == before + (rc == QMV_OK && rows > 0 ? 1 : 0));
              if (rc != QMV_OK || rows == 0) continue;
              EXPECT(rows <= QMM_MAX_ROWS && n >= 1 && k % 8 == 0 && rank % 8 == 0 && rank <= 128 && e <= 1024);
              for (int f32 = 0; f32 < 2; ++f32) {
                const qmv::rows::LoraPlan p = qmv::rows::lora_plan(rows, n, k, rank, e, x_rows, f32);
                EXPECT((p.tile == 16 || p.tile == 32) && p.splits >= 0 && p.splits <= 16);
                EXPECT(p.splits > 0 || (rank <= 32 && p.tile == 16 && (16 + rank) * (int64_t)k <= 160 << 10));
                EXPECT(p.splits <= 1 || p.splits <= qmv::rows::ceil_div(k, qmv::rows::kKBlock) / 10);
                EXPECT(p.columns >= 256 && p.columns % 256 == 0 && qmv::rows::ceil_div(n, p.columns) <= 65535);
                EXPECT(need == (size_t)p.splits * rows * rank * 4);
                EXPECT(((int64_t)qmv::rows::lora_tiles(rows, e, p.tile) + 7) * 256 <= (int64_t)UINT32_MAX);
                if (rows <= QMM_SAME_ROWS) EXPECT(p.tile == 16 && p.splits == qmv::rows::lora_plan(1, n, k, rank, 1, 1, f32).splits);
              }
              EXPECT(need == 0 || qmm_lora(at<uint16_t>(0), ab, at<uint16_t>(1), bb, nullptr, nullptr, at<uint16_t>(4), at<int32_t>(5),
                              gather ? at<int32_t>(6) : nullptr, at<>(8), at<>(8), QMM_F32, rows, x_rows, n, k, rank, e,
                              at<>(9), need - 1, nullptr) == QMV_ERR_WORKSPACE);
            }
          }
  for (int c = 1; c <= 16; ++c)   // chunks of a row of B, found without a division
    for (int q = 0; q < 1024; ++q) EXPECT((q * (65536 / c + 1)) >> 16 == q / c);
}

void verify() {
  for (int r : kInts)
    for (int d : kInts)
      for (int v : kInts)
        for (int ty = -1; ty <= 2; ++ty) {
          const size_t need = qmv_verify_drafts_workspace(r, v);
          const int before = stub::launches;
          const int rc = qmv_verify_drafts(at<>(0), at<>(1), ty, at<int32_t>(2), nullptr, at<float>(3), at<int32_t>(4),
                                           at<int32_t>(5), r, d, v, need ? at<>(6) : nullptr, need, nullptr);
          EXPECT(is_code(rc));
          EXPECT(stub::launches == before + (rc == QMV_OK && r > 0 ? 1 : 0));
          if (rc != QMV_OK || r == 0) continue;
          EXPECT(r <= QMV_MAX_REQUESTS && d >= 0 && d <= 32 && v >= 1 && v <= QMV_MAX_VOCAB);
          EXPECT((stub::verify.sums != nullptr) == (need > 0) && (need > 0) == (v > 16 * 1024));
          EXPECT(need == 0 || need == (size_t)r * qmv::rows::ceil_div(v, 1024) * 16);
        }
}

}  // namespace

int main() {
  sort();
  move();
  lora();
  verify();
  printf("%d failures, %d launches\n", failures, stub::launches);
  return failures ? 1 : 0;
}
