// Sizes and launch plans of the rows' operators (include/qmm_rows.h) and of the
// verification of drafts (include/qmv_verify.h). Plain C++ with no HIP
// dependency: the argument checks (rows_api.cpp, built with g++) and the kernel
// files use the same arithmetic. Everything depends on the arguments only.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/qmm_rows.h"
#include "../../include/qmv_verify.h"

namespace qmv {
namespace rows {

constexpr int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// ---- sort ----------------------------------------------------------------------

// Up to kSortOne choices one workgroup of 16 waves sorts alone. More are cut
// into parts of whole tiles of kSortTile for a workgroup of four waves each, at
// most kSortParts: a first launch counts every part's choices by expert into the
// workspace, a second adds up the counts before its part and places them.
constexpr int kSortOne = 4096;
constexpr int kSortTile = 1024;
constexpr int kSortParts = 256;

struct SortPlan {
  int parts, chunk;   // parts == 1: one launch, no workspace
};

inline SortPlan sort_plan(int choices) {
  if (choices <= kSortOne) return SortPlan{1, kSortOne};
  const int tiles = ceil_div(choices, kSortTile), per = ceil_div(tiles, kSortParts);
  return SortPlan{ceil_div(tiles, per), per * kSortTile};
}

inline size_t sort_workspace(int choices, int n_experts) {
  const SortPlan p = sort_plan(choices);
  return p.parts == 1 ? 0 : (size_t)p.parts * n_experts * 4;
}

// ---- adapters --------------------------------------------------------------------

constexpr int kKBlock = 64;   // values of k a wave takes at a time

// Rows of one tile (one adapter's), the parts of k of the first product and the
// columns of y of one workgroup of the second. Up to QMM_SAME_ROWS rows all of
// it goes by (n, k, rank) alone.
struct LoraPlan {
  int tile, splits, columns;
};

inline int lora_tiles(int rows, int n_adapters, int tile) {
  return rows / tile + (rows < n_adapters ? rows : n_adapters);
}

inline LoraPlan lora_plan(int rows, int n, int k, int rank, int n_adapters) {
  (void)n;
  const int blocks = ceil_div(k, kKBlock);
  int most = blocks / 4 < 1 ? 1 : blocks / 4 > 16 ? 16 : blocks / 4;   // a block for each of four waves
  if (rows <= QMM_SAME_ROWS) return LoraPlan{16, most, 256};
  const bool many = rows / n_adapters >= 64;
  const int tile = !many ? 16 : rank <= 64 ? 64 : 32;
  const int tiles = lora_tiles(rows, n_adapters, tile);
  int splits = ceil_div(512, tiles);
  if (splits > most) splits = most;
  return LoraPlan{tile, splits, many ? 1024 : 256};
}

// The first product's sums, fp32 [splits][rows][rank].
inline size_t lora_workspace(int rows, int n, int k, int rank, int n_adapters) {
  return (size_t)lora_plan(rows, n, k, rank, n_adapters).splits * rows * rank * 4;
}

// ---- verification ------------------------------------------------------------------

// Tokens of one workgroup: 256 threads of 16.
constexpr int kVerifyChunk = 4096;

// Two fp64 sums for each request and chunk.
inline size_t verify_workspace(int requests, int vocab) {
  return (size_t)requests * ceil_div(vocab, kVerifyChunk) * 16;
}

}  // namespace rows
}  // namespace qmv
