// Choices sorted by expert: a stable counting sort of int32 ids below 1024; gfx950.
//
// A wave takes 64 consecutive choices at a time. Lanes of one id find each other
// by one ballot for each bit of the id (the machine has no match instruction):
// what is left of the mask is the lanes of that id, the bits below a lane's own
// its rank among them. Every wave counts in its own LDS row, so nothing is
// atomic and the order is that of the choices. The rows' columns are then summed
// over the waves, the totals scanned over the experts, and a choice's row is
// its expert's start, its wave's share and its rank.
//
// Bound by latency: a chain of loads, ballots and barriers, a few us whatever the
// bytes. 32 choices of 128 experts by one wave 2.6 us (a replay 4.7, by 16 waves 5.7), 65536 by 16
// workgroups in two launches 4.6 and 7.6 us, where 0.8 MB at a copy's 5.2 TB/s would
// be 0.2; 16384 in one launch 10.5 us, launch included.
#include "rows_device.h"
#include "rows_internal.h"
#include "rows_layout.h"

namespace qmv {
namespace {

constexpr int kRounds = 4;   // of 64 choices: a wave's share of a tile, ranks in registers

// One tile of NW * kRounds * 64 choices from `first` on: ids and ranks of this
// lane's choices, counts by wave and expert in `hist` (cleared here).
template <int NW>
struct Tile {
  int id[kRounds], rank[kRounds];   // id: -1 where there is no choice

  __device__ __forceinline__ int choice(int r, int first) const {
    return first + (((int)threadIdx.x >> 6) * kRounds + r) * 64 + ((int)threadIdx.x & 63);
  }

  __device__ __forceinline__ void load(const SortArgs &p, int first, int last) {
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const int c = choice(r, first), v = c < last ? p.ids[c] : -1;
      id[r] = (unsigned)v < (unsigned)p.n_experts ? v : -1;
    }
  }

  __device__ __forceinline__ void count(const SortArgs &p, int bits, uint16_t *hist) {
    for (int i = (int)threadIdx.x; i < NW * p.n_experts; i += NW * 64) hist[i] = 0;
    __syncthreads();
    uint16_t *mine = hist + ((int)threadIdx.x >> 6) * p.n_experts;
    const int lane = (int)threadIdx.x & 63;
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      uint64_t same = __ballot(id[r] >= 0);
      if (same == 0) {
        rank[r] = 0;
        continue;
      }
      for (int b = 0; b < bits; ++b) {
        const bool set = (id[r] >> b) & 1;
        const uint64_t with = __ballot(set);
        same &= set ? with : ~with;
      }
      // the lanes of an id read its count together, then its first lane writes
      const uint64_t below = same & (((uint64_t)1 << lane) - 1);
      int before = 0;
      if (id[r] >= 0) before = mine[id[r]];
      in_order();
      if (id[r] >= 0 && below == 0) mine[id[r]] = (uint16_t)(before + __popcll(same));
      in_order();
      rank[r] = before + __popcll(below);
    }
    __syncthreads();
  }

  // hist: the rows that each wave's first choices of an expert get, from start[expert] on
  __device__ __forceinline__ void place(const SortArgs &p, int first, int last, const uint16_t *hist, const int *start) const {
    const uint16_t *mine = hist + ((int)threadIdx.x >> 6) * p.n_experts;
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const int c = choice(r, first);
      if (c >= last) continue;
      const int row = id[r] < 0 ? -1 : start[id[r]] + mine[id[r]] + rank[r];
      if (p.places) p.places[c] = row;
      if (p.row_index && row >= 0) p.row_index[row] = c / p.top_k;
    }
  }
};

// Each wave's count of expert e becomes the sum of those before it; all of them come back.
template <int NW>
__device__ __forceinline__ int sum_waves(uint16_t *hist, int n_experts, int e) {
  int c[NW], sum = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) c[w] = hist[w * n_experts + e];
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    hist[w * n_experts + e] = (uint16_t)sum;
    sum += c[w];
  }
  return sum;
}

// Exclusive sum over the workgroup's threads; `all` gets the whole sum.
template <int NW>
__device__ __forceinline__ int scan(int v, int *waves, int &all) {
  const int wave = (int)threadIdx.x >> 6, upto = wave_upto(v);
  if constexpr (NW == 1) {
    all = __builtin_amdgcn_readlane(upto, 63);
    return upto - v;
  }
  if (((int)threadIdx.x & 63) == 63) waves[wave] = upto;
  __syncthreads();
  int before = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const int s = waves[w];
    before += w < wave ? s : 0;
    all += s;
  }
  return before + upto - v;
}

// The rows from `total` on, in shares of the grid's workgroups.
__device__ __forceinline__ void clear_rest(const SortArgs &p, int total) {
  if (!p.row_index) return;
  for (int r = total + (int)(blockIdx.x * blockDim.x + threadIdx.x); r < p.choices; r += (int)(gridDim.x * blockDim.x))
    p.row_index[r] = -1;
}

// Up to one tile: everything in one workgroup.
template <int NW>
__global__ __launch_bounds__(NW * 64) void rows_sort_one_kernel(const SortArgs p, const int bits) {
  extern __shared__ uint16_t hist[];   // [NW][experts]
  __shared__ int waves[NW], start[QMM_MAX_EXPERTS];
  Tile<NW> t;
  t.load(p, 0, p.choices);
  t.count(p, bits, hist);
  const int per = rows::ceil_div(p.n_experts, NW * 64), e0 = (int)threadIdx.x * per;   // neighbouring experts a thread
  int sum = 0;
  for (int e = e0; e < e0 + per && e < p.n_experts; ++e) {
    start[e] = sum;
    sum += sum_waves<NW>(hist, p.n_experts, e);
  }
  int total;
  const int before = scan<NW>(sum, waves, total);
  for (int e = e0; e < e0 + per && e < p.n_experts; ++e) p.offsets[e] = start[e] += before;
  if (threadIdx.x == 0) p.offsets[p.n_experts] = total;
  __syncthreads();
  t.place(p, 0, p.choices, hist, start);
  clear_rest(p, total);
}

// A part's choices by expert: counts[part][expert].
__global__ __launch_bounds__(1024) void rows_sort_count_kernel(const SortArgs p, const int chunk) {
  __shared__ int sums[QMM_MAX_EXPERTS];
  if ((int)threadIdx.x < p.n_experts) sums[threadIdx.x] = 0;   // at most 1024 experts: one a thread
  __syncthreads();
  const int first = (int)blockIdx.x * chunk, last = first + chunk < p.choices ? first + chunk : p.choices;
  for (int f = first; f < last; f += rows::kSortTile) {
    Tile<16> t;
    t.load(p, f, last);
#pragma unroll
    for (int r = 0; r < kRounds; ++r)
      if (t.id[r] >= 0) atomicAdd(&sums[t.id[r]], 1);   // whole numbers: any order gives the same
  }
  __syncthreads();
  if ((int)threadIdx.x < p.n_experts) p.counts[(size_t)blockIdx.x * p.n_experts + threadIdx.x] = sums[threadIdx.x];
}

// A part's rows: its expert's start is the choices of that expert before the part
// and those of the experts before. Every workgroup adds these up for itself, from
// the counts of the first launch or, COUNTS, from the choices themselves; then its
// tiles go one by one.
template <bool COUNTS>
__global__ __launch_bounds__(1024) void rows_sort_place_kernel(const SortArgs p, const int chunk, const int bits) {
  constexpr int NW = 16;
  extern __shared__ uint16_t hist[];
  __shared__ int waves[NW];
  __shared__ int start[QMM_MAX_EXPERTS], total_of[QMM_MAX_EXPERTS];
  const int part = (int)blockIdx.x, parts = (int)gridDim.x, tid = (int)threadIdx.x;
  const int first = part * chunk, last = first + chunk < p.choices ? first + chunk : p.choices;
  Tile<NW> t;
  t.load(p, first, last);
  if (tid < p.n_experts) start[tid] = total_of[tid] = 0;
  __syncthreads();
  if constexpr (COUNTS) {
    for (int f = 0; f < p.choices; f += rows::kSortTile) {
      Tile<NW> all;
      all.load(p, f, p.choices);
#pragma unroll
      for (int r = 0; r < kRounds; ++r)
        if (all.id[r] >= 0) {   // whole numbers: any order gives the same; a part is whole tiles
          atomicAdd(&total_of[all.id[r]], 1);
          if (f < first) atomicAdd(&start[all.id[r]], 1);
        }
    }
  } else {
    // threads of one expert take turns over the parts
    const int turns = 1024 / p.n_experts, turn = tid / p.n_experts, of = tid - turn * p.n_experts;
    if (turn < turns) {
      int before = 0, all = 0;
#pragma unroll 4
      for (int b = turn; b < parts; b += turns) {
        const int c = p.counts[(size_t)b * p.n_experts + of];
        before += b < part ? c : 0;
        all += c;
      }
      atomicAdd(&start[of], before);
      atomicAdd(&total_of[of], all);
    }
  }
  __syncthreads();
  int total;
  const int at = scan<NW>(tid < p.n_experts ? total_of[tid] : 0, waves, total);
  if (tid < p.n_experts) {
    if (part == 0) p.offsets[tid] = at;
    start[tid] += at;
  }
  if (part == 0 && tid == 0) p.offsets[p.n_experts] = total;
  for (int f = first; f < last; f += rows::kSortTile) {
    if (f > first) t.load(p, f, last);
    t.count(p, bits, hist);   // its first barrier is behind the last tile's reads of hist
    const int sum = tid < p.n_experts ? sum_waves<NW>(hist, p.n_experts, tid) : 0;
    __syncthreads();
    t.place(p, f, last, hist, start);
    __syncthreads();
    if (tid < p.n_experts) start[tid] += sum;
  }
  clear_rest(p, total);
}

template <int NW>
int one(const SortArgs &a, int bits, hipStream_t s) {
  return launch_kernel("rows_sort_one_kernel", rows_sort_one_kernel<NW>, dim3(1), dim3(NW * 64), (size_t)NW * a.n_experts * 2,
                       s, a, bits);
}

}  // namespace

int launch_rows_sort(const SortArgs &a, void *stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  int bits = 0;
  while ((1 << bits) < a.n_experts) ++bits;
  const rows::SortPlan plan = rows::sort_plan(a.choices);
  if (plan.parts == 1)
    return a.choices <= kRounds * 64 ? one<1>(a, bits, s) : a.choices <= kRounds * 256 ? one<4>(a, bits, s) : one<16>(a, bits, s);
  const dim3 grid((unsigned)plan.parts), block(1024);
  const size_t lds = (size_t)16 * a.n_experts * 2;
  if (!a.counts)
    return launch_kernel("rows_sort_place_kernel", rows_sort_place_kernel<true>, grid, block, lds, s, a, plan.chunk, bits);
  const int rc = launch_kernel("rows_sort_count_kernel", rows_sort_count_kernel, grid, block, 0, s, a, plan.chunk);
  if (rc) return rc;
  return launch_kernel("rows_sort_place_kernel", rows_sort_place_kernel<false>, grid, block, lds, s, a, plan.chunk, bits);
}

}  // namespace qmv
