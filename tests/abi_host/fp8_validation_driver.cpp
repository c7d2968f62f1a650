// Drives the argument checks and plans of the e4m3 and grouped entry points in
// a host-only build (fp8_api.cpp + stand-in launchers, no HIP runtime) under
// the address and undefined-behaviour sanitizers. Pointers are fake: a call is
// refused or reaches a stand-in. Exit status 0: every expectation held.
#include <limits.h>
#include <stdint.h>
#include <stdio.h>

#include "../../gguf_block_quantized_qmv_amd/csrc/fp8_internal.h"
#include "../../gguf_block_quantized_qmv_amd/csrc/fp8_layout.h"
#include "../../include/qmm_fp8.h"

namespace stub {
extern int launches;
extern qmv::ProductArgs last;
extern int last_m, last_k;
}  // namespace stub

namespace {

int failures = 0;
#define EXPECT(cond)                                                                \
  do {                                                                              \
    if (!(cond)) {                                                                  \
      if (++failures < 20) fprintf(stderr, "%s:%d: failed: %s\n", __FILE__, __LINE__, #cond); \
    }                                                                               \
  } while (0)

void *at(int region) { return reinterpret_cast<void *>((uintptr_t)0x100000000000ull + ((uintptr_t)region << 40)); }

const int kInts[] = {INT_MIN, -257, -1, 0, 1, 2, 7, 8, 15, 16, 17, 31, 32, 33, 64, 65, 127, 128, 129, 130, 256, 257, 768,
                     1000, 2064, 5120, 17408, 65536, 65537, 1 << 20, (1 << 20) + 16, 1 << 24, (1 << 24) + 1,
                     INT_MAX / 16 * 16, INT_MAX};

bool is_code(int rc) { return rc <= 0 && rc >= QMV_ERR_HIP; }

namespace fp8 = qmv::fp8;

// What the kernels assume of a plan.
void plan_holds(int m, int n, int k, bool bf16) {
  const int nb = fp8::blocks_of(k);
  const fp8::DensePlan p = fp8::dense_plan(m, n, k, bf16);
  EXPECT(m > QMM_SAME_ROWS || p.stream);
  if (p.stream) {
    const fp8::StreamPlan s = fp8::stream_plan(m, n, nb);
    EXPECT(s.tile >= 4 && s.tile <= 32 && s.tile % 4 == 0);
    EXPECT(s.waves == 4 || s.waves == 8 || s.waves == 16);
    EXPECT((int64_t)fp8::ceil_div(n, s.tile) * s.waves * 64 <= (int64_t)UINT32_MAX);
    EXPECT(fp8::ceil_div(m, 16) <= 65535);                    // the grid's second dimension
    EXPECT((int64_t)32 * k <= (int64_t)UINT32_MAX);           // a tile's rows by 32-bit offsets
    if (m <= QMM_SAME_ROWS) {
      const fp8::StreamPlan one = fp8::stream_plan(1, n, nb);
      EXPECT(one.tile == s.tile && one.waves == s.waves);
    }
    EXPECT(fp8::dense_workspace(m, n, k, bf16) == 0);
    return;
  }
  EXPECT(p.tile >= fp8::kTile32 && p.tile <= (bf16 ? fp8::kTile256Wide : fp8::kTile256));
  const int64_t tiles = (int64_t)fp8::ceil_div(m, fp8::tile_rows(p.tile)) * fp8::ceil_div(n, fp8::tile_cols(p.tile));
  EXPECT((int64_t)p.t_main + p.r_tiles == tiles);
  EXPECT(p.splits >= 1 && p.splits <= 16 && (p.splits > 1) == (p.r_tiles > 0));
  EXPECT(p.splits == 1 || (nb / p.splits >= 4 && (int64_t)p.r_tiles * p.splits <= fp8::kSlots));
  EXPECT((int64_t)tiles + 256 <= INT_MAX);
  EXPECT((int64_t)fp8::tile_cols(p.tile) * k <= (int64_t)UINT32_MAX && (int64_t)fp8::tile_rows(p.tile) * k <= (int64_t)UINT32_MAX);
  EXPECT(fp8::dense_workspace(m, n, k, bf16) ==
         (p.splits > 1 ? (size_t)p.r_tiles * p.splits * fp8::tile_rows(p.tile) * fp8::tile_cols(p.tile) * 4 : 0));
}

void dense() {
  const float *ws = static_cast<const float *>(at(1)), *xs = static_cast<const float *>(at(3));
  for (int m : kInts)
    for (int n : kInts)
      for (int k : kInts)
        for (int t = -1; t <= 2; ++t) {
          const size_t bytes = n > 0 && k > 0 ? (size_t)n * k : 1;
          const size_t need = qmm_fp8_workspace(m, n, k, t);
          const int before = stub::launches;
          // y may be as large as 2^46 bytes: its region is the last one
          const int rc = qmm_fp8(at(0), bytes, ws, at(2), xs, at(9), t, m, n, k, need ? at(4) : nullptr, need, nullptr);
          EXPECT(is_code(rc));
          EXPECT((rc == QMV_OK) == (stub::launches == before + 1));
          if (rc != QMV_OK) continue;
          EXPECT(m >= 1 && n >= 1 && k >= 16 && k % 16 == 0 && (t == QMM_F32 || t == QMM_BF16));
          EXPECT(stub::last.rows == m && stub::last.n == n && stub::last.k_bytes == k && stub::last.nb == (k + 127) / 128);
          EXPECT((stub::last.part != nullptr) == (need > 0));
          plan_holds(m, n, k, t == QMM_BF16);
          if (need) {
            EXPECT(qmm_fp8(at(0), bytes, ws, at(2), xs, at(9), t, m, n, k, nullptr, 0, nullptr) == QMV_ERR_WORKSPACE);
            EXPECT(qmm_fp8(at(0), bytes, ws, at(2), xs, at(9), t, m, n, k, at(4), need - 1, nullptr) == QMV_ERR_WORKSPACE);
          }
        }
  const size_t full = 64 * 256;
  for (size_t b = 0; b < 2 * full; ++b)
    if (b != full) EXPECT(qmm_fp8(at(0), b, ws, at(2), xs, at(9), QMM_F32, 1, 64, 256, nullptr, 0, nullptr) == QMV_ERR_SIZE);
}

void grouped() {
  const float *ws = static_cast<const float *>(at(1)), *xs = static_cast<const float *>(at(3));
  const int32_t *off = static_cast<const int32_t *>(at(5)), *idx = static_cast<const int32_t *>(at(6));
  const int experts[] = {INT_MIN, 0, 1, 2, 63, 64, 65, 128, 1024, 1025};
  for (int rows : kInts)
    for (int n : kInts)
      for (int k : kInts)
        for (int e : experts)
          for (int kind = 0; kind < 2; ++kind) {
            const int vb = kind ? 2 : 1;
            const size_t bytes = n > 0 && k > 0 && e > 0 ? (size_t)e * n * k * vb : 1;
            for (int gather = 0; gather < 2; ++gather) {
              const int before = stub::launches, x_rows = gather ? 100 : rows;
              const int rc = kind ? qmm_bf16_grouped(static_cast<const uint16_t *>(at(0)), bytes,
                                                     static_cast<const uint16_t *>(at(2)), off, gather ? idx : nullptr,
                                                     at(9), QMM_BF16, rows, x_rows, n, k, e, nullptr)
                                  : qmm_fp8_grouped(at(0), bytes, ws, at(2), xs, off, gather ? idx : nullptr, at(9),
                                                    QMM_F32, rows, x_rows, n, k, e, nullptr);
              EXPECT(is_code(rc));
              EXPECT(stub::launches == before + (rc == QMV_OK && rows > 0 ? 1 : 0));
              if (rc != QMV_OK || rows == 0) continue;
              EXPECT(rows >= 1 && n >= 1 && e >= 1 && e <= 1024 && k % (16 / vb) == 0);
              EXPECT(stub::last.n_experts == e && stub::last.k_bytes == k * vb);
              const int tile = fp8::grouped_tile(rows, e, n, fp8::blocks_of(k * vb), kind == 0);
              EXPECT(tile >= fp8::kTile32 && tile <= (kind == 0 ? fp8::kTile256 : fp8::kTile256Wide));
              EXPECT(fp8::grouped_row_tiles(rows, e, fp8::tile_rows(tile)) * fp8::ceil_div(n, fp8::tile_cols(tile)) <= fp8::kMaxTiles);
            }
          }
}

void quant() {
  for (int m : kInts)
    for (int k : kInts)
      for (int t = -1; t <= 2; ++t)
        for (int gated = 0; gated < 2; ++gated) {
          const int before = stub::launches;
          uint8_t *xq = static_cast<uint8_t *>(at(2));
          float *xs = static_cast<float *>(at(3));
          const int rc = gated ? qmm_fp8_quant_silu_mul(at(0), t, xq, xs, m, k, nullptr)
                               : qmm_fp8_quant(at(0), t, xq, xs, m, k, nullptr);
          EXPECT(is_code(rc));
          EXPECT(stub::launches == before + (rc == QMV_OK && m > 0 ? 1 : 0));
          if (rc == QMV_OK) EXPECT(m >= 0 && m <= QMM_MAX_ROWS && k >= 8 && k % 8 == 0 && k <= QMM_MAX_K);
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
