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

// Up to kSortTile choices one workgroup sorts alone, of as many waves as these
// need. More are cut into parts of whole tiles for a workgroup of 16 waves each,
// at most kSortParts. Up to kSortCounts every workgroup counts all choices by
// expert for itself; above, a first launch counts every part's into the workspace.
constexpr int kSortTile = 4096;
constexpr int kSortParts = 256;
constexpr int kSortCounts = 16384;   // 16384 choices of 128 experts 10.5 us so, 11.4 by two launches; 32768 13.4 and 11.6

struct SortPlan {
  int parts, chunk;
};

inline SortPlan sort_plan(int choices) {
  const int tiles = ceil_div(choices, kSortTile), per = ceil_div(tiles, kSortParts);
  return tiles <= 1 ? SortPlan{1, kSortTile} : SortPlan{ceil_div(tiles, per), per * kSortTile};
}

inline size_t sort_workspace(int choices, int n_experts) {
  return choices <= kSortCounts ? 0 : (size_t)sort_plan(choices).parts * n_experts * 4;
}

// ---- spread, combine, gradient ----------------------------------------------------

// The rows are read or written past the caches: from 64 MiB on, where what is
// written would not wait in the last-level cache for its reader. 65536 rows of 2048
// bf16 spread 52 us against 61, summed back 52 against 61, their gradient from
// 32768 rows 56 against 62; 8192 rows the same either way.
inline bool past_caches(int rows, int width, bool f32) {
  return (int64_t)rows * width * (f32 ? 4 : 2) >= (int64_t)64 << 20;
}

// ---- adapters --------------------------------------------------------------------

constexpr int kKBlock = 64;   // values of k a wave takes at a time
constexpr int kCus = 256;     // compute units

// Rows of one tile (one adapter's), the parts of k of the first product (0: both
// products in one launch), the columns of y of one workgroup of the second, and
// whether y goes past the caches. The sums of a row go by the parts alone, and up
// to QMM_SAME_ROWS rows these go by n, k and rank.
struct LoraPlan {
  int tile, splits, columns;
  bool far;
};

inline int lora_tiles(int rows, int n_adapters, int tile) {
  return rows / tile + (rows < n_adapters ? rows : n_adapters);
}

inline LoraPlan lora_plan(int rows, int n, int k, int rank, int n_adapters, int x_rows, bool y_f32) {
  LoraPlan p{};
  // One launch, in which every workgroup of a tile takes all of A x for itself, where that
  // is few bytes for one CU and all workgroups run at once. A CU gets some 115 GB/s of
  // the lines of x and A (A's by 16 rows: ranks 8 and 16 take the same time, 24 and 32 too).
  // One launch against two, us, one row of one of 8 adapters, 5120 columns, in a graph of
  // twelve calls, k 2048, 4096, 5120, 6144, 8192: rank 16 7.0 and 7.8, 8.2 and 7.8, 8.8 and 7.8,
  // 9.4 and 8.2, 10.6 and 8.3; rank 32 7.4 and 8.2, 9.2 and 8.2, 10.1 and 8.2, 10.9 and 8.6, 12.5 and 8.7.
  // Launched from the host one takes 10.1 and two 12.8, whatever k up to 5120.
  // So up to QMM_SAME_ROWS rows, a decode step, which is launched either way, one launch goes
  // on to 340 KiB, where a graph loses 1 us (16 rows of 16 adapters 1.8) and the host
  // saves 2.7. More rows go by the graph: 64 of 5 adapters, 5120 columns, rank 16, k 2048 8.0
  // and 8.4, 4096 10.3 and 8.5; 300 of 2048 columns 8.9 and 9.2, 10.9 and 9.8; 1000 of 1024
  // 9.7 and 11.0, 11.3 and 12.1.
  // More workgroups than CUs run in two rounds (64 rows of 64 adapters each once, rank 16, k
  // 2048: 256 workgroups 8.8 and 11.1, 320 14.2 and 11.7). How many have rows only the device knows:
  // an adapter's last tile is taken for half full (64 rows of 64 adapters drawn at random,
  // 5120 columns: 340 could be, 200 are, 8.5 and 11.1), and up to QMM_SAME_ROWS rows, where the
  // choice must not go by them, 14 tiles are taken: with 17408 columns 16 rows of an adapter
  // each lose (13.9 and 11.2, at k 5120 18.6 and 11.5), 12 gain (7.5 and 10.3, 9.9 and 10.1).
  p.tile = 16;
  p.columns = 1024;
  const bool few = rows <= QMM_SAME_ROWS;
  const int some16 = few ? 14 : rows / 16 + (lora_tiles(rows, n_adapters, 16) - rows / 16) / 2;
  if (rank <= 32 && (16 + ceil_div(rank, 16) * 16) * (int64_t)k * 2 <= (few ? 340 << 10 : 192 << 10) &&
      some16 * (int64_t)ceil_div(n, p.columns) <= kCus)
    return p;
  // Long runs take tiles of 32 rows, which read A and B half as often: 8192 rows
  // of 5 adapters of 5120 x 5120, rank 64: 67 us against 90; 205 rows of each 22
  // against 24.4, 51 of each 19 against 16.4. Above rank 64 such a tile leaves one
  // wave a SIMD: 4096 rows at rank 128 67 us either way, 2048 55 against 51.
  p.tile = rows >= 128 * (rank > 64 ? 4 : 1) * (int64_t)n_adapters ? 32 : 16;
  const int tiles = lora_tiles(rows, n_adapters, p.tile), blocks = ceil_div(k, kKBlock);
  // Ten blocks of k a part, for four waves: one row of 5120 in 8 parts 9.1 us, in
  // 4 9.4, in 16 9.3; 64 rows of 17408 in 16 parts 14.4, in 8 15.7. Fewer where
  // tiles fill the CUs (512 rows of rank 128: 4 parts 28.7, 8 33.7).
  p.splits = blocks / 10 < ceil_div(kCus, tiles) ? blocks / 10 : ceil_div(kCus, tiles);
  p.splits = p.splits < 1 ? 1 : p.splits > 16 ? 16 : p.splits;
  // One more where that takes a fifth off the CU with the most: of 4096 rows of 5
  // adapters, rank 64, some 130 tiles, 3 parts 40.0 us, 2 42.7, 1 46.2, 4 41.1; of 3000
  // 4 parts 37.2, 3 39.4. An adapter's last tile is taken for half full.
  const int some = rows / p.tile + (tiles - rows / p.tile) / 2, more = p.splits + 1;
  const int64_t most_now = ceil_div((int64_t)some * p.splits, kCus), most_then = ceil_div((int64_t)some * more, kCus);
  if (rows > QMM_SAME_ROWS && more <= 16 && more <= blocks / 10 && most_then * p.splits * 5 <= most_now * more * 4)
    p.splits = more;
  // As many columns' shares as let all workgroups run at once, but for an eighth:
  // `waves` a SIMD is what the second kernel's registers allow. 64 rows of 24
  // adapters by 512 of 17408 columns 15.6 us, by 256 17.6; 4096 rows of rank 64 by
  // 1280 of 5120 42, by 1024 49, by 2560 54.
  const int waves = p.tile == 16 ? (rank <= 32 ? 4 : rank <= 64 ? 3 : 2) : rank <= 32 && !y_f32 ? 3 : rank <= 64 ? 2 : 1;
  const int shares = 288 * waves / tiles < 1 ? 1 : 288 * waves / tiles;
  p.columns = ceil_div(ceil_div(n, shares), 256) * 256;
  // y larger than all L2s (4096 x 5120 bf16: 34 us against 38, 1024 x 5120 fp32,
  // which stays in them, 23 against 20).
  p.far = (int64_t)x_rows * n * (y_f32 ? 4 : 2) >= (int64_t)32 << 20;
  return p;
}

// Workgroups of the second launch stay far inside 32 bits.
inline bool lora_in_grid(int rows, int n, int n_adapters) {
  return (int64_t)lora_tiles(rows, n_adapters, 16) * ceil_div(n, 256) <= (int64_t)1 << 28;
}

// The first product's sums, fp32 [splits][rows][rank].
inline size_t lora_workspace(int rows, int n, int k, int rank, int n_adapters) {
  return (size_t)lora_plan(rows, n, k, rank, n_adapters, 0, false).splits * rows * rank * 4;
}

// ---- verification ------------------------------------------------------------------

constexpr int kVerifyChunk = 1024;   // tokens of one wave: 64 lanes of 16

// A workgroup a request, in one launch and without a workspace, where its 16 waves
// have a chunk each. One launch against two, us, fp32, in a graph of twelve calls: one
// request of 8192 tokens 6.3 and 7.7, 16384 7.5 and 7.9, 24576 8.2 and 7.9, 32768 9.7 and 7.9;
// 16 of 24576 8.4 and 8.3; 256 of 16384 10.4 and 13.2, of 32768 15.1 and 16.9, 131072 46.0 and
// 45.4: with a request for each CU the change would come later. A workspace goes by the vocabulary.
inline bool verify_whole(int vocab) { return vocab <= 16 * kVerifyChunk; }

// Two fp64 sums for each request and chunk.
inline size_t verify_workspace(int requests, int vocab) {
  return verify_whole(vocab) ? 0 : (size_t)requests * ceil_div(vocab, kVerifyChunk) * 16;
}

}  // namespace rows
}  // namespace qmv
