// Sizes and launch plans of the e4m3 and grouped products (include/qmm_fp8.h).
// Plain C++ with no HIP dependency: the argument checks (fp8_api.cpp, built
// with g++) and the kernel files use the same arithmetic. Everything depends on
// the arguments only, never on the device, so a call's numerical program is
// fixed by its shape.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/qmm_fp8.h"

namespace qmv {
namespace fp8 {

constexpr int kBlock = 128;   // values of k under one scale
constexpr int kSlots = 256;   // compute units a plan fills (a 256-CU MI355X)

constexpr int blocks_of(int k) { return (k + kBlock - 1) / kBlock; }
constexpr int ceil_div(int a, int b) { return (a + b - 1) / b; }

constexpr int kLdsPerCu = 160 * 1024;

// ---- tile shapes (rows of x by rows of w of one workgroup) -------------------

enum Tile { kTile32 = 0, kTile64 = 1, kTile128 = 2, kTile256 = 3, kTile256Wide = 4 };
constexpr int tile_rows(int t) { return t == kTile32 ? 32 : t == kTile64 ? 64 : t == kTile128 ? 128 : 256; }
constexpr int tile_cols(int t) { return t == kTile32 ? 64 : t == kTile256Wide ? 256 : 128; }

// ---- dense -------------------------------------------------------------------

// A few rows of x against a matrix that is soon read: `stream`, the kernel that
// takes the weights straight into registers, every wave a share of k. Else
// tiles: t_main whole ones (a multiple of the CUs, or all), and r_tiles that
// are cut into `splits` parts of k so that the last round fills the CUs; the
// parts' fp32 sums go to the workspace and a second launch adds them in order.
struct DensePlan {
  bool stream;
  int tile, t_main, r_tiles, splits;
};

// The streaming kernel reads the weights once per 16 rows of x, from the L2
// after the first. Up to 16 rows it always wins (1 x 17408 x 5120: 22.9 us
// against 26.9 by tiles of 32 rows); with more of them while the weights are
// small (77 x 1000 x 2064: 8 us against 14; 32 x 17408 x 5120: 56 against 33).
constexpr int64_t kStreamBytes = (int64_t)32 << 20;
constexpr int kStreamRows = 2048;   // 512 x 1024 x 1024: 15.4 us against 16.7

inline DensePlan split_plan(int tile, int m, int n, int nb) {
  DensePlan p{false, tile, 0, 0, 1};
  const int64_t tiles = (int64_t)ceil_div(m, tile_rows(tile)) * ceil_div(n, tile_cols(tile));
  // small tiles share a CU: a second round of them costs little
  const int64_t rest = tile <= kTile64 && tiles >= kSlots ? 0 : tiles % kSlots;
  int64_t s = rest ? kSlots / rest : 1;
  if (s > nb / 4) s = nb / 4;      // at least four blocks a part
  if (s > 16) s = 16;
  p.splits = s < 1 ? 1 : (int)s;
  p.r_tiles = p.splits > 1 ? (int)rest : 0;
  p.t_main = (int)(tiles < INT32_MAX ? tiles : INT32_MAX) - p.r_tiles;
  return p;
}

inline size_t split_bytes(const DensePlan &p) {
  return p.splits > 1 ? (size_t)p.r_tiles * p.splits * tile_rows(p.tile) * tile_cols(p.tile) * 4 : 0;
}

// fast: QMM_FAST_SUMS is asked for.
inline DensePlan dense_plan(int m, int n, int k, bool fast) {
  const int nb = blocks_of(k);
  if (m <= QMM_SAME_ROWS || (m <= kStreamRows && (int64_t)n * k * ceil_div(m, 16) < kStreamBytes))
    return DensePlan{true, kTile32, 0, 0, 1};
  if (m <= 128) return split_plan(m <= 32 ? kTile32 : m <= 64 ? kTile64 : kTile128, m, n, nb);
  // Of the large tiles the one with the least time by this model, in ns: a step
  // of one block of k takes, with every CU at work, 2200 (256 x 128) and 1300
  // (128 x 128), with fast sums 1150, 750 and 1800 (256 x 256); a tile
  // starts and ends in 8000; parts are written and read at 5 bytes a ps.
  DensePlan best{};
  int64_t least = INT64_MAX;
  for (int tile = kTile128; tile <= (fast ? kTile256Wide : kTile256); ++tile) {
    const DensePlan p = split_plan(tile, m, n, nb);
    const int64_t step = tile == kTile256Wide ? 1800 : tile == kTile256 ? (fast ? 1150 : 2200) : fast ? 750 : 1300;
    const int64_t rounds = (p.t_main + kSlots - 1) / kSlots;
    int64_t cost = rounds * (nb * step + 8000);
    if (p.r_tiles) cost += ceil_div(nb, p.splits) * step + 8000 + 3000 + (int64_t)split_bytes(p) * 2 / 5000;
    if (cost < least) {
      least = cost;
      best = p;
    }
  }
  return best;
}

inline size_t dense_workspace(int m, int n, int k, bool fast) { return split_bytes(dense_plan(m, n, k, fast)); }

// The streaming kernel: `tile` weight rows (a multiple of four, so that a
// lane's four results lie under one scale; above 16, two fragments a wave) and
// `waves` waves a workgroup, one workgroup for each 16 rows of x. The tile is
// the one of 8 to 32 rows that spreads the workgroups most evenly over the CUs
// (a longer one unless a shorter is 5 % better); with few rows, shorter tiles
// keep every CU at work.
struct StreamPlan {
  int tile, waves;
};

inline StreamPlan stream_plan(int m, int n, int nb) {
  const int chunks = ceil_div(m, 16);   // one for every m that shares its bits
  int tile = 4;
  int64_t best_num = 0, best_den = 1, per_cu = 1;
  for (int t = 32; t >= 8; t -= 4) {
    const int64_t groups = (int64_t)ceil_div(n, t) * chunks, rounds = (groups + kSlots - 1) / kSlots;
    if (groups * best_den * 20 > best_num * rounds * kSlots * 21) {   // share of the CUs' rounds that has work
      best_num = groups;
      best_den = rounds * kSlots;
      per_cu = rounds;
      tile = t;
    }
  }
  if (best_num * 2 <= kSlots) tile = 4;   // fewer than half the CUs even with tiles of 8
  int waves = per_cu <= 1 ? 16 : per_cu <= 2 ? 8 : 4;
  while (waves > 4 && waves > nb) waves >>= 1;
  return StreamPlan{tile, waves};
}

// ---- grouped -----------------------------------------------------------------

// Host code cannot see the offsets: rows are taken as spread evenly, half a
// tile lost at the end of each expert's run. Of the tiles the one with the
// least time by this model, in ns: a step of one block of k takes 700 (32 x 64,
// four workgroups a CU), 900 (64 x 128, two), 750 (128 x 128) and 1800 (256 x
// 256), for codes widened to bf16 (`exact`: e4m3 without fast sums) 900, 1200
// and 2200 (256 x 128); a tile starts and ends in 6000. Measured, in us: with
// fast sums 8 rows, 8 of 128 experts of 1536 x 2048, 8.5 by 32 x 64, 11.4 by 64 x
// 128, 10.1 by 128 x 128, and 4096 rows 102, 84, 88; widened 8 rows 10 by 32 x
// 64, 17 by 64 x 128, 20 by 256 x 128, 4096 rows 106, 104, 131, and 65536 rows of
// 2048 x 768 480, 321, 282.
inline int grouped_tile(int rows, int n_experts, int n, int nb, bool exact) {
  const int busy = rows < n_experts ? rows : n_experts;
  int best = kTile32;
  int64_t least = INT64_MAX;
  for (int tile = kTile32; tile <= (exact ? kTile256 : kTile256Wide); ++tile) {
    if (tile == (exact ? kTile128 : kTile256)) continue;   // 64 x 128 and 256 x 256 do better
    const int bm = tile_rows(tile), per_cu = tile == kTile32 ? 4 : tile == kTile64 ? 2 : 1;
    int64_t row_tiles = ((int64_t)rows + (int64_t)busy * bm / 2) / bm;
    if (row_tiles < busy) row_tiles = busy;
    const int64_t tiles = row_tiles * ceil_div(n, tile_cols(tile));
    const int64_t rounds = (tiles + per_cu * kSlots - 1) / (per_cu * kSlots);
    const int64_t step = tile == kTile32 ? (exact ? 900 : 700) : tile == kTile64 ? (exact ? 1200 : 900)
                         : tile == kTile128 ? 750 : tile == kTile256 ? 2200 : 1800;
    const int64_t cost = rounds * (nb * step + 6000);
    if (cost < least) {
      least = cost;
      best = tile;
    }
  }
  return best;
}

// Row tiles a grouped launch can need: every expert with rows may have one
// partial tile.
inline int64_t grouped_row_tiles(int rows, int n_experts, int bm) {
  return (int64_t)rows / bm + (rows < n_experts ? rows : n_experts);
}

// Tiles of a launch stay far inside 32 bits.
constexpr int64_t kMaxTiles = (int64_t)1 << 28;

inline bool dense_in_grid(int m, int n) { return (int64_t)ceil_div(m, 128) * ceil_div(n, 64) <= kMaxTiles; }

inline bool grouped_in_grid(int rows, int n_experts, int n, int nb, bool exact) {
  const int t = grouped_tile(rows, n_experts, n, nb, exact);
  return grouped_row_tiles(rows, n_experts, tile_rows(t)) * ceil_div(n, tile_cols(t)) <= kMaxTiles;
}

}  // namespace fp8
}  // namespace qmv
