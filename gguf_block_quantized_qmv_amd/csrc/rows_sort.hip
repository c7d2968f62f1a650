// Choices sorted by expert: a stable counting sort of int32 ids below 1024; gfx950.
//
// A wave takes 64 consecutive choices at a time. Lanes of one id find each other
// by one ballot for each bit of the id (the machine has no match instruction):
// what is left of the mask is the lanes of that id, the bits below a lane's own
// its rank among them. Every wave counts in its own LDS row, so nothing is
// atomic and the order is that of the choices. The rows' columns are then summed
// over the waves, the totals scanned over the experts, and a choice's row is
// its expert's start, its wave's share and its rank.
#include "qmv_device.h"
#include "rows_internal.h"
#include "rows_layout.h"

namespace qmv {
namespace {

constexpr int kRounds = 4;   // of 64 choices, a wave's share of a tile, ranks in registers

// One tile of 64 * kRounds * NW choices from `first` on: ids and ranks of this
// lane's choices, counts by wave and expert in `hist` (cleared here). COUNT holds
// a tile's counts and the rows that become of them.
template <int NW, class COUNT>
struct Tile {
  int id[kRounds], rank[kRounds];   // id: -1 where there is no choice

  __device__ __forceinline__ int choice(int r, int first) const {
    return first + (((int)threadIdx.x >> 6) * kRounds + r) * 64 + ((int)threadIdx.x & 63);
  }

  __device__ void count(const SortArgs &p, int first, int last, int bits, COUNT *hist) {
    for (int i = (int)threadIdx.x; i < NW * p.n_experts; i += NW * 64) hist[i] = 0;
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const int c = choice(r, first), v = c < last ? p.ids[c] : -1;
      id[r] = (unsigned)v < (unsigned)p.n_experts ? v : -1;
    }
    __syncthreads();
    COUNT *mine = hist + ((int)threadIdx.x >> 6) * p.n_experts;
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
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      if (id[r] >= 0 && below == 0) mine[id[r]] = (COUNT)(before + __popcll(same));
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      rank[r] = before + __popcll(below);
    }
    __syncthreads();
  }

  // hist: the row that each wave's first choice of an expert gets
  __device__ void place(const SortArgs &p, int first, int last, const COUNT *hist) const {
    const COUNT *mine = hist + ((int)threadIdx.x >> 6) * p.n_experts;
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const int c = choice(r, first);
      if (c >= last) continue;
      const int row = id[r] < 0 ? -1 : mine[id[r]] + rank[r];
      if (p.places) p.places[c] = row;
      if (p.row_index && row >= 0) p.row_index[row] = c / p.top_k;
    }
  }
};

// Exclusive sum over the workgroup's threads; `all` gets the whole sum.
template <int NW>
__device__ __forceinline__ int scan(int v, int *waves, int &all) {
  const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
  int upto = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(upto, d);
    if (lane >= d) upto += o;
  }
  if (lane == 63) waves[wave] = upto;
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

// Up to 4096 choices: everything in one workgroup. A thread owns the columns of
// `per` neighbouring experts.
__global__ __launch_bounds__(1024) void rows_sort_one_kernel(const SortArgs p, const int bits) {
  constexpr int NW = 16;
  extern __shared__ uint16_t few[];   // rows up to 4096 fit: 32 KiB at most
  __shared__ int waves[NW];
  uint16_t *hist = few;
  Tile<NW, uint16_t> t;
  t.count(p, 0, p.choices, bits, hist);
  const int e = (int)threadIdx.x;   // at most 1024 experts: one a thread
  int sum = 0;
  if (e < p.n_experts)
#pragma unroll
    for (int w = 0; w < NW; ++w) sum += hist[w * p.n_experts + e];
  int total;
  int start = scan<NW>(sum, waves, total);
  if (e < p.n_experts) {
    p.offsets[e] = start;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const int c = hist[w * p.n_experts + e];
      hist[w * p.n_experts + e] = (uint16_t)start;
      start += c;
    }
  }
  if (e == 0) p.offsets[p.n_experts] = total;
  __syncthreads();
  t.place(p, 0, p.choices, hist);
  clear_rest(p, total);
}

// A part's choices by expert: counts[part][expert].
__global__ __launch_bounds__(256) void rows_sort_count_kernel(const SortArgs p, const int chunk) {
  __shared__ int sums[QMM_MAX_EXPERTS];
  for (int e = (int)threadIdx.x; e < p.n_experts; e += 256) sums[e] = 0;
  __syncthreads();
  const int first = (int)blockIdx.x * chunk, last = first + chunk < p.choices ? first + chunk : p.choices;
  for (int c = first + (int)threadIdx.x; c < last; c += 256) {
    const int v = p.ids[c];
    if ((unsigned)v < (unsigned)p.n_experts) atomicAdd(&sums[v], 1);   // whole numbers: any order gives the same
  }
  __syncthreads();
  for (int e = (int)threadIdx.x; e < p.n_experts; e += 256) p.counts[(size_t)blockIdx.x * p.n_experts + e] = sums[e];
}

// A part's rows: the counts of the parts before it and of all are added up by
// every workgroup for itself (from the L2), then its tiles go one by one.
__global__ __launch_bounds__(256) void rows_sort_place_kernel(const SortArgs p, const int chunk, const int bits) {
  constexpr int NW = 4;
  extern __shared__ int hist[];
  __shared__ int waves[NW];
  __shared__ int start[QMM_MAX_EXPERTS], total_of[QMM_MAX_EXPERTS];
  const int part = (int)blockIdx.x, parts = (int)gridDim.x, tid = (int)threadIdx.x;
  for (int e = tid; e < p.n_experts; e += 256) start[e] = total_of[e] = 0;
  __syncthreads();
  // threads of one expert take turns over the parts
  const int lanes = p.n_experts >= 256 ? 256 : p.n_experts, turns = 256 / lanes;
  if (tid < lanes * turns) {
    const int turn = tid / lanes;
    for (int e = tid % lanes; e < p.n_experts; e += lanes) {
      int before = 0, all = 0;
#pragma unroll 8
      for (int b = turn; b < parts; b += turns) {
        const int c = p.counts[(size_t)b * p.n_experts + e];
        before += b < part ? c : 0;
        all += c;
      }
      atomicAdd(&start[e], before);   // whole numbers
      atomicAdd(&total_of[e], all);
    }
  }
  __syncthreads();
  const int per = rows::ceil_div(p.n_experts, 256), e0 = tid * per;
  int sum = 0;
  for (int e = e0; e < e0 + per && e < p.n_experts; ++e) sum += total_of[e];
  int total;
  int at = scan<NW>(sum, waves, total);
  for (int e = e0; e < e0 + per && e < p.n_experts; ++e) {
    if (part == 0) p.offsets[e] = at;
    start[e] += at;
    at += total_of[e];
  }
  if (part == 0 && tid == 0) p.offsets[p.n_experts] = total;
  const int first = part * chunk, last = first + chunk < p.choices ? first + chunk : p.choices;
  for (int f = first; f < last; f += rows::kSortTile) {
    Tile<NW, int> t;
    t.count(p, f, last, bits, hist);   // its first barrier also closes the last tile's reads of hist
    for (int e = tid; e < p.n_experts; e += 256) {
      int s = start[e];
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const int c = hist[w * p.n_experts + e];
        hist[w * p.n_experts + e] = s;
        s += c;
      }
      start[e] = s;
    }
    __syncthreads();
    t.place(p, f, last, hist);
    __syncthreads();
  }
  clear_rest(p, total);
}

}  // namespace

int launch_rows_sort(const SortArgs &a, void *stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  int bits = 0;
  while ((1 << bits) < a.n_experts) ++bits;
  const rows::SortPlan plan = rows::sort_plan(a.choices);
  if (plan.parts == 1)
    return launch_kernel("rows_sort_one_kernel", rows_sort_one_kernel, dim3(1), dim3(1024), (size_t)16 * a.n_experts * 2,
                         s, a, bits);
  const int rc = launch_kernel("rows_sort_count_kernel", rows_sort_count_kernel, dim3((unsigned)plan.parts), dim3(256), 0,
                               s, a, plan.chunk);
  if (rc) return rc;
  return launch_kernel("rows_sort_place_kernel", rows_sort_place_kernel, dim3((unsigned)plan.parts), dim3(256),
                       (size_t)4 * a.n_experts * 4, s, a, plan.chunk, bits);
}

}  // namespace qmv
