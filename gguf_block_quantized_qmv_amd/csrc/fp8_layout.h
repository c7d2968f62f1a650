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

struct DensePlan {
  bool stream;   // the weight-streaming kernel (m <= QMM_SAME_ROWS), no workspace
  int tile;      // else a Tile
  int splits;    // parts of k, summed by a second launch when more than one
};

// The weight-streaming kernel: `tile` weight rows (a multiple of four, so that
// a lane's four results lie under one scale) and `waves` waves a workgroup.
// The tile is the one of 16, 12 and 8 rows that spreads the workgroups most
// evenly over the CUs; with few rows, shorter tiles keep every CU at work.
// About sixteen waves a CU keep the memory busy.
struct StreamPlan {
  int tile, waves;
};

inline StreamPlan stream_plan(int n, int nb, int slots) {
  int tile = 4;
  int64_t best_num = 0, best_den = 1, per_cu = 1;
  for (int t = 16; t >= 8; t -= 4) {
    const int64_t groups = (int64_t)ceil_div(n, t) * slots, rounds = (groups + kSlots - 1) / kSlots;
    if (groups * best_den > best_num * rounds * kSlots) {   // share of the CUs' rounds that has work
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

inline DensePlan dense_plan(int m, int n, int k, bool y_bf16) {
  DensePlan p{false, kTile128, 1};
  const int nb = blocks_of(k);
  if (m <= 32) {
    // by (n, k) alone
    p.tile = kTile32;
    p.stream = (int64_t)n * k < (int64_t)32 << 20;
    if (p.stream) return p;
  } else {
    p.tile = m <= 64 ? kTile64 : m <= 128 ? kTile128 : kTile256;
    const int64_t wide = (int64_t)ceil_div(m, 256) * ceil_div(n, 256);
    if (y_bf16 && m > 128 && wide >= kSlots) p.tile = kTile256Wide;
  }
  const int64_t tiles = (int64_t)(m <= 32 ? 1 : ceil_div(m, tile_rows(p.tile))) * ceil_div(n, tile_cols(p.tile));
  int64_t s = kSlots / tiles;
  if (s > nb / 4) s = nb / 4;      // at least four blocks a part
  if (s > 16) s = 16;
  p.splits = s < 1 ? 1 : (int)s;
  return p;
}

inline size_t dense_workspace(int m, int n, int k, bool y_bf16) {
  const DensePlan p = dense_plan(m, n, k, y_bf16);
  return p.splits > 1 ? (size_t)p.splits * (size_t)m * (size_t)n * 4 : 0;
}

// ---- grouped -----------------------------------------------------------------

// Expected rows of an expert that has any: host code cannot see the offsets, so
// the tile goes by rows spread evenly.
struct GroupedPlan {
  bool stream;
  int tile;
};

inline GroupedPlan grouped_plan(int rows, int n_experts, bool exact) {
  const int avg = rows / (n_experts < 1 ? 1 : n_experts);
#ifndef GSTREAM
#define GSTREAM 0
#endif
#ifndef GBIG
#define GBIG kTile256
#endif
  GroupedPlan p{rows <= GSTREAM, kTile32};
  p.tile = avg <= 24 ? kTile32 : avg <= 64 ? kTile64 : avg <= 128 ? kTile128 : exact ? kTile256 : GBIG;
  return p;
}

// Row tiles a grouped launch can need: every expert with rows may have one
// partial tile.
inline int64_t grouped_row_tiles(int rows, int n_experts, int bm) {
  return (int64_t)rows / bm + (rows < n_experts ? rows : n_experts);
}

// Workgroups of a launch: 2^22 of up to 512 threads keep a grid inside 32 bits.
constexpr int64_t kMaxWorkgroups = (int64_t)1 << 22;

inline bool dense_fits_grid(int m, int n, int k, bool y_bf16) {
  const DensePlan p = dense_plan(m, n, k, y_bf16);
  return p.stream || (int64_t)ceil_div(m, tile_rows(p.tile)) * ceil_div(n, tile_cols(p.tile)) * p.splits <= kMaxWorkgroups;
}

inline bool grouped_fits_grid(int rows, int n, int n_experts, bool exact) {
  const GroupedPlan p = grouped_plan(rows, n_experts, exact);
  return p.stream || grouped_row_tiles(rows, n_experts, tile_rows(p.tile)) * ceil_div(n, tile_cols(p.tile)) <= kMaxWorkgroups;
}

}  // namespace fp8
}  // namespace qmv
