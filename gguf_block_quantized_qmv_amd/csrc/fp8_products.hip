// Products of e4m3 rows with block-scaled e4m3 weights, dense and grouped by
// expert, and the grouped product on bf16; gfx950 matrix cores.
//
// Along k everything is counted in blocks of 128 bytes: 128 e4m3 values under
// one scale, or 64 bf16 values. The weights are the A operand (16 rows of w),
// the activations the B operand (16 rows of x), so a lane's four results are
// four neighbouring columns of one row of y. An MFMA takes k in any order as
// long as both operands agree: lane l of a fragment holds the 16-byte chunks
// l / 16 and l / 16 + 4 of row l % 16.
//
// e4m3: the scales vary from block to block, so a block's product starts from
// zero and enters the sum by one fma per result, y += (xs * ws) * d, in fp32.
// Two ways to a block's product:
//  * kExact, the codes as bf16 (exact, two by one v_cvt_scalef32_pk_bf16_fp8)
//    through four v_mfma_f32_16x16x32_bf16, whose sums keep fp32: 1e-8 to 8e-8
//    of the result's norm over a block, and a block's integers under 2^24 come
//    out as they are. Results of both types are made so.
//  * kNative, one v_mfma_f32_16x16x128_f8f6f4 at twice the rate, where the
//    caller asks for fast sums (tiles only). Every e4m3 instruction aligns each
//    eight neighbouring products to the largest of them and cuts what lies 13
//    bits below (2^16 + 2^2 in one group of eight gives 2^16, in two groups
//    2^16 + 2^2; v_mfma_f32_16x16x32_fp8_fp8 the same). Measured over a block:
//    1.5e-5 of the norm on normal data, 4e-5 with a few strong channels, 5e-5 on
//    uniform codes; a group that cancels (448^2 - 448^2 + 6 * 4) loses all.
//    But for such groups that is less than a rounding to bf16, so it goes with
//    bf16 results alone.
// bf16 operands (kBf16) take two v_mfma_f32_16x16x32_bf16 a block.
// The rates that bound them on this card, with random operands from registers:
// kNative 3.65 PFLOP/s with the fma beside it, bf16 instructions 1.8 to 1.9.
#include <type_traits>

#include "fp8_internal.h"
#include "fp8_layout.h"
#include "qmv_device.h"
#include "../../include/qmm_fp8.h"

namespace qmv {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// One block's chunk pair of one lane.
struct Frag {
  v4i lo, hi;
};

enum Kind { kNative, kExact, kBf16 };
constexpr bool is_e4m3(Kind kind) { return kind != kBf16; }

// Eight e4m3 codes as a bf16 MFMA operand (exact; NaN stays NaN).
__device__ __forceinline__ bf16x8 widen(const int c0, const int c1) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)c0, 1.0f, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)c0, 1.0f, true);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)c1, 1.0f, false);
  const bf16x2 e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)c1, 1.0f, true);
  return bf16x8{a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
}

// A block's operand in the form its instructions take.
template <Kind KIND>
struct Operand {
  v8i v;
  __device__ __forceinline__ void set(const Frag &f) { v = __builtin_shufflevector(f.lo, f.hi, 0, 1, 2, 3, 4, 5, 6, 7); }
};
template <>
struct Operand<kExact> {
  bf16x8 v[4];
  // part h of the block
  __device__ __forceinline__ void set(int h, const Frag &f) {
    const v4i c = h < 2 ? f.lo : f.hi;
    v[h] = h % 2 == 0 ? widen(c[0], c[1]) : widen(c[2], c[3]);
  }
  __device__ __forceinline__ void set(const Frag &f) {
#pragma unroll
    for (int h = 0; h < 4; ++h) set(h, f);
  }
};
template <>
struct Operand<kBf16> {
  bf16x8 v[2];
  __device__ __forceinline__ void set(const Frag &f) {
    v[0] = __builtin_bit_cast(bf16x8, f.lo);
    v[1] = __builtin_bit_cast(bf16x8, f.hi);
  }
};

// d = from + A B over one block.
template <Kind KIND>
__device__ __forceinline__ v4f mma_block(const Operand<KIND> &a, const Operand<KIND> &b, v4f d) {
  if constexpr (KIND == kNative) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, d, 0, 0, 0, 0, 0, 0);
  } else {
    constexpr int kParts = KIND == kExact ? 4 : 2;
#pragma unroll
    for (int h = 0; h < kParts; ++h) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[h], b.v[h], d, 0, 0, 0);
    return d;
  }
}

// acc += scale * d
__device__ __forceinline__ void scaled_add(const float scale, const v4f d, v4f &acc) {
#pragma unroll
  for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(scale, d[e], acc[e]);
}

constexpr v4f kZero4 = {0.0f, 0.0f, 0.0f, 0.0f};

__device__ const uint4 g_zeros[8] = {};   // what loads past the end of a row read: one block

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

// Rows of expert e, clamped to y.
__device__ __forceinline__ void expert_rows(const int32_t *__restrict__ offsets, int e, int rows, int &begin,
                                            int &end) {
  begin = clampi(offsets[e], 0, rows);
  end = clampi(offsets[e + 1], begin, rows);
}

// ---- a few rows: stream the weights ---------------------------------------------
//
// A workgroup owns `tile` <= 16 MW rows of w and 16 rows of x; wave v takes
// blocks v, v + NW, ... of k straight from memory into MFMA fragments (no LDS),
// DEPTH blocks in flight, and the waves' sums are added in wave order: no
// second launch. The host chooses the tile so that every CU gets the same number
// of workgroups (a fragment of fewer than 16 rows repeats its last row: matrix
// work, no memory traffic). The order of the sums goes by (n, k) alone and the columns
// of an MFMA do not mix, so a row of x has the same bits in any company.
//
// Bound by the weight stream: 1 x 17408 x 5120 takes 17.5 us with the weights
// partly in the last-level cache (5.1 TB/s; a plain read of as many bytes 17.6
// us from HBM) and 21.4 to 23 us from HBM. What counted: two fragments of w for one
// of x (MW = 1 reads as many bytes of x as of w through the L2: 26.5 us), and
// plain loads (a fragment takes a 128-byte line in two halves: with
// non-temporal loads each half fetched the line, 23.7 us). Matrices of less
// than 32 rows a CU take MW = 1 and shorter tiles: 1 x 4096 x 4096 8 us.
template <int NW, int MW, int DEPTH>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(4))) void fp8_stream_kernel(
    const ProductArgs p, const int tile) {
  __shared__ float red[NW][MW * 256];
  const int lane = (int)threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int n0 = (int)blockIdx.x * tile, n1 = n0 + tile < p.n ? n0 + tile : p.n;
  const int m0 = (int)blockIdx.y * 16, m1 = m0 + 16 < p.rows ? m0 + 16 : p.rows;
  // Lane offsets from scalar addresses. They are hidden from the optimiser at
  // every use, which would otherwise keep one 64-bit address per block alive.
  const uint8_t *wbase = p.w + (size_t)n0 * p.k_bytes, *xbase = p.x + (size_t)m0 * p.k_bytes;
  uint32_t wlane[MW], wslane[MW];
#pragma unroll
  for (int i = 0; i < MW; ++i) {
    const int row = n0 + i * 16 + r, srow = n0 + i * 16 + g * 4;
    wlane[i] = (uint32_t)((row < n1 ? row : n1 - 1) - n0) * (uint32_t)p.k_bytes + g * 16;
    // tiles are multiples of four rows: a lane's four results share a scale
    wslane[i] = (uint32_t)((srow < p.n ? srow : p.n - 1) >> 7) * (uint32_t)p.nb;
  }
  uint32_t xlane = (uint32_t)(m0 + r < m1 ? r : m1 - 1 - m0) * (uint32_t)p.k_bytes + g * 16;
  uint32_t xslane = (uint32_t)(m0 + r < m1 ? m0 + r : m1 - 1);
  const int whole = p.k_bytes >> 7, tail = p.k_bytes & 127;

  Frag wf[DEPTH][MW], xf[DEPTH];
  float xs[DEPTH], ws[DEPTH][MW];
  // Block b (past the last whole one: zeros, so that every pass of the loop
  // sends the same loads and each wait counts exactly those behind it).
  auto load_scales = [&](int b, int u, bool ok) {
    const float *zeros = reinterpret_cast<const float *>(g_zeros);
    asm("" : "+v"(xslane));
    xs[u] = (ok ? p.x_scale + (size_t)b * p.x_rows : zeros)[ok ? xslane : 0];
#pragma unroll
    for (int i = 0; i < MW; ++i) {
      asm("" : "+v"(wslane[i]));
      ws[u][i] = (ok ? p.w_scale + b : zeros)[ok ? wslane[i] : 0];
    }
  };
  auto load = [&](int b, int u) {
    const bool ok = b < whole;
    const uint8_t *zeros = reinterpret_cast<const uint8_t *>(g_zeros);
#pragma unroll
    for (int i = 0; i < MW; ++i) {
      asm("" : "+v"(wlane[i]));
      const uint8_t *w = (ok ? wbase + (size_t)b * 128 : zeros) + (ok ? wlane[i] : 0);
      wf[u][i].lo = *reinterpret_cast<const v4i *>(w);
      wf[u][i].hi = *reinterpret_cast<const v4i *>(w + 64);
    }
    asm("" : "+v"(xlane));
    const uint8_t *x = (ok ? xbase + (size_t)b * 128 : zeros) + (ok ? xlane : 0);
    xf[u].lo = *reinterpret_cast<const v4i *>(x);
    xf[u].hi = *reinterpret_cast<const v4i *>(x + 64);
    load_scales(b, u, ok);
  };
  v4f acc[MW];
#pragma unroll
  for (int i = 0; i < MW; ++i) acc[i] = kZero4;
  auto use = [&](int u) {
    Operand<kExact> c;
    c.set(xf[u]);
#pragma unroll
    for (int i = 0; i < MW; ++i) {
      Operand<kExact> a;
      a.set(wf[u][i]);
      scaled_add(xs[u] * ws[u][i], mma_block<kExact>(a, c, kZero4), acc[i]);
    }
  };
#pragma unroll
  for (int u = 0; u < DEPTH; ++u) load(wave + u * NW, u);
  for (int b = wave; b < whole; b += DEPTH * NW)
#pragma unroll
    for (int u = 0; u < DEPTH; ++u) {
      use(u);
      load(b + (u + DEPTH) * NW, u);
      __builtin_amdgcn_sched_barrier(0);   // one block's widened operands at a time
    }
  if (tail && wave == whole % NW) {   // the partial last block: zeros past the row
    const v4i none = {0, 0, 0, 0};
    const uint8_t *x = xbase + (size_t)whole * 128 + xlane;
    xf[0].lo = xf[0].hi = none;
    if (g * 16 < tail) xf[0].lo = *reinterpret_cast<const v4i *>(x);
    if (g * 16 + 64 < tail) xf[0].hi = *reinterpret_cast<const v4i *>(x + 64);
#pragma unroll
    for (int i = 0; i < MW; ++i) {
      const uint8_t *w = wbase + (size_t)whole * 128 + wlane[i];
      wf[0][i].lo = wf[0][i].hi = none;
      if (g * 16 < tail) wf[0][i].lo = *reinterpret_cast<const v4i *>(w);
      if (g * 16 + 64 < tail) wf[0][i].hi = *reinterpret_cast<const v4i *>(w + 64);
    }
    load_scales(whole, 0, true);
    use(0);
  }
  // lane l holds columns 4 g .. 4 g + 3 of each 16 of row r of x
#pragma unroll
  for (int i = 0; i < MW; ++i) *reinterpret_cast<v4f *>(&red[wave][(r * MW + i) * 16 + g * 4]) = acc[i];
  __syncthreads();
  for (int at = (int)threadIdx.x; at < MW * 256; at += NW * 64) {
    const int row = m0 + at / (MW * 16), col = n0 + at % (MW * 16);
    float sum = red[0][at];
#pragma unroll
    for (int v = 1; v < NW; ++v) sum += red[v][at];
    if (row < m1 && col < n1) {
      const size_t to = (size_t)row * p.n + col;
      if (p.y_bf16)
        static_cast<__bf16 *>(p.y)[to] = (__bf16)sum;
      else
        static_cast<float *>(p.y)[to] = sum;
    }
  }
}

// ---- many rows: tiles through LDS --------------------------------------------------
//
// A workgroup computes BM x BN tiles of y (rows of x by rows of w), one after
// the other. Each step moves one block of k of both into an LDS stage by
// direct-to-LDS loads, kStages - 1 blocks ahead of the waves, which multiply
// the oldest stage; one barrier a step hands the stages on. The first blocks of
// the next tile are sent before the results of a tile are stored, so that the
// memory works through the stores.
//
// A stage row is 128 bytes, eight 16-byte chunks. A fragment read takes one
// chunk of 16 rows; it is free of bank conflicts when the eight even and the
// eight odd rows each find the chunk in eight different slots: chunk c of row r
// sits at slot c ^ f(r). The direct loads write LDS in lane order, so the
// permutation is applied to the global address each lane reads.
//  * rows of x: a fragment is 16 consecutive rows, f(r) = r / 2 % 8;
//  * rows of w, where a wave has an even number of column tiles: two tiles share
//    32 rows in alternating fours, so that a lane's two results of four columns
//    are eight neighbouring ones (one 16-byte store in bf16); f(r) takes bits
//    1, 3 and 4 of r.
//
// What bounds it, and why these shapes:
//  * Long products: the conversions. 4096 x 17408 x 5120 takes 600 to 633 us,
//    1.15 to 1.2 PFLOP/s, the matrix cores 58 % busy: two conversions for each of
//    their instructions share the issue slots with the fma. A widened operand
//    takes twice the registers, so 256 x 128 is the largest tile.
//  * With fast sums, the matrix cores and their power: 309 to 336 us, 2.2 to 2.4
//    PFLOP/s, 59 % busy; on zeros a fifth less. Of the shapes only 256 x 256
//    (waves of 128 x 64) asks LDS for no more than it gives beside the matrix
//    instructions; a step of it takes 1.8 us, two of 256 x 128 (waves of
//    64 x 64) take 2.3. Its sums fill the registers at two waves a SIMD, and two
//    stages fill LDS.
//  * Few steps a tile (k of 768): the stores beside them. 65536 rows over 128
//    experts, n 2048, bf16 results: 281 to 289 us, with fast sums 182 to 190, of
//    which 50 are the 268 MB of y at the card's write rate; the loads of a
//    following tile beyond its first blocks queue behind them. Smaller tiles, two
//    workgroups a CU, overlap them and lose more to LDS (64 x 128: 321 us; fast
//    sums by 128 x 128: 224 us).
//  * Few rows: the weight stream. 512 tokens to 8 of 128 experts of 1536 x
//    2048: 89 us for 417 MB, by 64 x 128 tiles, two workgroups a CU.
// Without effect or slower: weight scales through LDS, a rotated first block
// per workgroup, other places for the loads in a step, non-temporal loads or
// stores, a wait that leaves the stores of the tile before under way.
constexpr int kStageRow = 128;

template <int BM_, int BN_, int WM_, int WN_, int STAGES_>
struct Shape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;   // waves along rows of x, of w
  static constexpr int kStages = STAGES_;
  static constexpr int kWaves = WM * WN, kThreads = kWaves * 64;
  static constexpr int TM = BM / WM / 16, TN = BN / WN / 16;     // MFMA tiles of a wave
  static constexpr bool kPairs = TN % 2 == 0;
  static constexpr int kLoads = (BM + BN) / 8 / kWaves;          // 1 KiB direct loads of a wave and step
  static constexpr int kStageBytes = (BM + BN) * kStageRow;
  static constexpr int kScales = (BM + 63) / 64 * 64;
  static constexpr int kLdsBytes = kStages * (kStageBytes + kScales * 4);
  static constexpr int kPerCu = fp8::kLdsPerCu / kLdsBytes;      // workgroups a CU holds
  static_assert((BM + BN) % (8 * kWaves) == 0 && TM * WM * 16 == BM && TN * WN * 16 == BN, "whole tiles and loads");
  static_assert(BN / WN <= 128 && 128 % (BN / WN) == 0, "a wave's columns lie under one weight scale");
  static_assert(TM % 2 == 0, "tiles alternate between two registers");
  static_assert(kStages >= 2 && kStages <= 4 && kPerCu >= 1, "the arrays below");
};

// Buffer form of the direct load: LDS at `to` + 16 (or 4) bytes a lane gets
// the bytes at base + at + step; at or beyond `size` it gets zeros. (Unlike the
// global form it does not make the compiler drain the LDS reads in flight.)
typedef __amdgpu_buffer_rsrc_t Buffer;
__device__ __forceinline__ Buffer buffer_of(const void *base, uint32_t size) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, (int)size, 0x00020000);
}
constexpr uint32_t kOutside = 0xFFFFFFF0u;   // an offset past every buffer
__device__ __forceinline__ void load_lds16(Buffer from, uint32_t at, uint32_t step, void *to) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void *)to, 16, (int)at, (int)step,
                                           0, 0);
}
__device__ __forceinline__ void load_lds4(Buffer from, uint32_t at, void *to) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void *)to, 4, (int)at, 0, 0, 0);
}

// All but the last `AFTER` memory operations of this wave are done and every
// LDS read has returned, then all waves meet. (Loads and stores of a wave are
// counted off in order.)
template <int AFTER>
__device__ __forceinline__ void stage_barrier() {
  static_assert(AFTER < 64, "the counter's range");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((AFTER & 15) | (AFTER >> 4) << 14 | 0x0070);   // vmcnt(AFTER) lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// First row and column of tile id: bands of eight row tiles, rows first within a band.
template <class S>
__device__ __forceinline__ void tile_place(int id, int rows, int n_tiles, int &m0, int &n0) {
  const int m_tiles = fp8::ceil_div(rows, S::BM);
  const int band = uniform(id / (8 * n_tiles)), in = id - band * 8 * n_tiles;
  const int high = m_tiles - band * 8 < 8 ? m_tiles - band * 8 : 8;
  const int nt = uniform(in / high);
  n0 = nt * S::BN;
  m0 = (band * 8 + in - nt * high) * S::BM;
}

template <class S, Kind KIND, bool GROUPED>
__global__ __launch_bounds__(S::kThreads) void product_tile_kernel(const ProductArgs p, const int t_main,
                                                                    const int r_tiles, const int splits) {
  constexpr bool FP8 = is_e4m3(KIND);
  // one array a stage, each named in the unrolled loop below: the compiler then
  // knows which reads a load in flight cannot touch
  __shared__ __attribute__((aligned(1024))) uint8_t stage0[S::kStageBytes], stage1[S::kStageBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t stage2[S::kStages > 2 ? S::kStageBytes : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t stage3[S::kStages > 3 ? S::kStageBytes : 16];
  __shared__ float scale0[S::kScales], scale1[S::kScales], scale2[S::kStages > 2 ? S::kScales : 1],
      scale3[S::kStages > 3 ? S::kScales : 1];
  const int lane = (int)threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6);
  const int n_tiles = fp8::ceil_div(p.n, S::BN);

  // tiles in all; grouped: the row tiles of each lane's run of experts, and
  // their running sum over the lanes
  const int per = fp8::ceil_div(p.n_experts, 64);
  int total, mine = 0, upto = 0;
  if constexpr (GROUPED) {
    for (int e = lane * per; e < lane * per + per && e < p.n_experts; ++e) {
      int b0, b1;
      expert_rows(p.offsets, e, p.rows, b0, b1);
      mine += fp8::ceil_div(b1 - b0, S::BM);
    }
    upto = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(upto, d);
      if (lane >= d) upto += o;
    }
    // decreasing offsets can give more row tiles than rows and experts allow:
    // the host has checked n_tiles times this bound
    const int rows_most = p.rows / S::BM + (p.rows < p.n_experts ? p.rows : p.n_experts);
    const int sum = uniform(__shfl(upto, 63));
    total = (sum < rows_most ? sum : rows_most) * n_tiles;
  } else {
    total = t_main;
  }
  // Workgroups are dealt to the eight XCDs in turn. Each XCD takes one
  // contiguous run of the whole tiles and one of the parts, its workgroups side
  // by side in it, so that neighbouring tiles share rows of x and w in the
  // XCD's cache.
  const int xcd = (int)blockIdx.x & 7, parts = r_tiles * splits;
  auto run_of = [&](int all, int &start, int &length) {
    const int share = all >> 3, rest = all & 7;
    start = xcd * share + (xcd < rest ? xcd : rest);
    length = share + (xcd < rest);
  };
  int first, count, first_part, part_count;
  run_of(total, first, count);
  run_of(parts, first_part, part_count);
  const int stride = ((int)gridDim.x - xcd + 7) >> 3, all_count = count + part_count;
  int at = (int)blockIdx.x >> 3;
  if (at >= all_count) return;
  auto id_of = [&](int at) { return at < count ? first + at : total + first_part + at - count; };

  struct Tile {
    int expert, m0, end, n0, part, blk0, blk1;   // part: its slot in the workspace, -1 for a whole tile
  };
  auto locate = [&](int id) {
    Tile t{0, 0, p.rows, 0, -1, 0, p.nb};
    if constexpr (GROUPED) {
      const int mt = uniform(id / n_tiles);
      t.n0 = (id - mt * n_tiles) * S::BN;
      const int owner = uniform(__ffsll((unsigned long long)__ballot(upto > mt)) - 1);
      int left = mt - uniform(__shfl(upto - mine, owner)), begin;
      int e = owner * per;
      for (;; ++e) {
        expert_rows(p.offsets, e, p.rows, begin, t.end);
        const int tiles = fp8::ceil_div(t.end - begin, S::BM);
        if (left < tiles || e + 1 >= p.n_experts) break;
        left -= tiles;
      }
      t.expert = uniform(e);
      t.m0 = uniform(begin + left * S::BM);
      t.end = uniform(t.end);
    } else {
      if (id >= total) {   // part q of tile total + r sits at slot q * r_tiles + r
        t.part = id - total;
        const int q = uniform(t.part / r_tiles);
        id = total + t.part - q * r_tiles;
        t.blk0 = uniform((int)((int64_t)p.nb * q / splits));
        t.blk1 = uniform((int)((int64_t)p.nb * (q + 1) / splits));
      }
      tile_place<S>(id, p.rows, n_tiles, t.m0, t.n0);
    }
    return t;
  };

  // This lane's direct loads of a tile's block: row q * 8 + lane / 8 of the
  // stage, chunk by the slot, as an offset from a scalar base: the tile's first
  // row of w, and of x unless its rows are gathered (from all of x, which the
  // host then keeps under 4 GiB). Rows past a tile's end lie outside the buffers
  // and are zeros that nothing has to be read for, and so is a gathered row
  // outside x.
  struct Loads {
    Buffer x, w;
    uint32_t from[S::kLoads];
    uint32_t scale_from;
  };
  const bool gather = GROUPED && p.index;
  auto chunk_of = [&](int i) {
    const int q = wave * S::kLoads + i, row = q * 8 + (lane >> 3), wrow = row - S::BM;
    const int f = q < S::BM / 8 || !S::kPairs ? row >> 1 & 7 : (wrow >> 1 & 1) | (wrow >> 3 & 3) << 1;
    return ((lane & 7) ^ f) * 16;
  };
  constexpr int kScaleWaves = S::kScales / 64;   // waves past these bring the same scales again: no branch in the loop
  const int scale_to = wave % kScaleWaves * 64;
  auto loads_of = [&](const Tile &t) {
    Loads l;
    l.w = buffer_of(p.w + ((size_t)t.expert * p.n + t.n0) * p.k_bytes,
                    (uint32_t)(p.n - t.n0 < S::BN ? p.n - t.n0 : S::BN) * (uint32_t)p.k_bytes);
    const int x_first = gather ? 0 : t.m0, x_count = gather ? p.x_rows : t.end - t.m0 < S::BM ? t.end - t.m0 : S::BM;
    l.x = buffer_of(p.x + (size_t)x_first * p.k_bytes, (uint32_t)x_count * (uint32_t)p.k_bytes);
    int row[S::kLoads + 1];
#pragma unroll
    for (int i = 0; i < S::kLoads; ++i) {
      const int q = wave * S::kLoads + i, r = q * 8 + (lane >> 3);
      row[i] = q < S::BM / 8 ? t.m0 + r - x_first : r - S::BM;
    }
    row[S::kLoads] = t.m0 + scale_to + lane < t.end ? t.m0 + scale_to + lane : t.end - 1;
    if (gather) {   // all index loads before the first use
      int found[S::kLoads + 1];
#pragma unroll
      for (int i = 0; i <= S::kLoads; ++i)
        found[i] = p.index[i < S::kLoads && wave * S::kLoads + i >= S::BM / 8 ? t.m0 : row[i] < t.end ? row[i] : t.m0];
#pragma unroll
      for (int i = 0; i <= S::kLoads; ++i)
        if (i == S::kLoads || wave * S::kLoads + i < S::BM / 8) row[i] = row[i] < t.end ? found[i] : -1;
    }
#pragma unroll
    for (int i = 0; i < S::kLoads; ++i) {
      l.from[i] = (uint32_t)row[i] * (uint32_t)p.k_bytes + (uint32_t)chunk_of(i);
      if (gather && wave * S::kLoads + i < S::BM / 8 && (unsigned)row[i] >= (unsigned)p.x_rows) l.from[i] = kOutside;
    }
    l.scale_from = (unsigned)row[S::kLoads] < (unsigned)p.x_rows ? (uint32_t)row[S::kLoads] * 4 : kOutside;
    return l;
  };
  const int tail = p.k_bytes & 127;   // bytes of a partial last block
  // one of the wave's direct loads of block b
  auto load_piece = [&](const Loads &l, int i, int b, uint8_t *stage, bool last) {
    const uint32_t from = last && chunk_of(i) >= tail ? kOutside : l.from[i];
    uint8_t *to = stage + (wave * S::kLoads + i) * 1024;
    // kOutside stays outside: the hardware compares the offset without the scalar step
    if (wave * S::kLoads + i < S::BM / 8)
      load_lds16(l.x, from, (uint32_t)b * 128, to);
    else
      load_lds16(l.w, from, (uint32_t)b * 128, to);
  };
  auto load_scales = [&](const Loads &l, int b, float *scale) {
    if constexpr (FP8)
      load_lds4(buffer_of(p.x_scale + (size_t)b * p.x_rows, (uint32_t)p.x_rows * 4), l.scale_from, scale + scale_to);
  };
  // all loads of block b, which may be the partial last one
  auto issue = [&](const Loads &l, int b, uint8_t *stage, float *scale) {
    const bool partial = tail != 0 && b == p.nb - 1;
#pragma unroll
    for (int i = 0; i < S::kLoads; ++i) load_piece(l, i, b, stage, partial);
    load_scales(l, b, scale);
  };
  // Block b of a tile in stage (b - blk0) % kStages; the loads of kAhead blocks
  // are under way.
  constexpr int kAhead = S::kStages - 1;
  constexpr int kAfter = (kAhead - 1) * (S::kLoads + (FP8 ? 1 : 0));   // direct loads sent after a block's own
  auto issue_first = [&](const Loads &l, const Tile &t) {
    issue(l, t.blk0, stage0, scale0);
    if constexpr (kAhead > 1) {
      if (t.blk0 + 1 < t.blk1) issue(l, t.blk0 + 1, stage1, scale1);
    }
    if constexpr (kAhead > 2) {
      if (t.blk0 + 2 < t.blk1) issue(l, t.blk0 + 2, stage2, scale2);
    }
  };
  auto stage_of = [&](auto u) {
    constexpr int v = decltype(u)::value % S::kStages;
    if constexpr (v == 0) return stage0;
    else if constexpr (v == 1) return stage1;
    else if constexpr (v == 2) return stage2;
    else return stage3;
  };
  auto scale_at = [&](auto u) {
    constexpr int v = decltype(u)::value % S::kStages;
    if constexpr (v == 0) return scale0;
    else if constexpr (v == 1) return scale1;
    else if constexpr (v == 2) return scale2;
    else return scale3;
  };

  auto stage_in = [&](int v) {
    return v == 0 ? stage0 : v == 1 ? stage1 : S::kStages > 2 && v == 2 ? stage2 : S::kStages > 3 ? stage3 : stage0;
  };
  auto scale_in = [&](int v) {
    return v == 0 ? scale0 : v == 1 ? scale1 : S::kStages > 2 && v == 2 ? scale2 : S::kStages > 3 ? scale3 : scale0;
  };

  // fragment addresses in a stage; chunk g + 4 is 64 bytes on or back
  const int wm = wave / S::WN, wn = wave % S::WN;
  const int r = lane & 15, g = lane >> 4;
  const int x_at = (wm * S::TM * 16 + r) * kStageRow + ((g ^ (r >> 1 & 7)) << 4);
  const int w_row = S::kPairs ? (r >> 2) * 8 + (r & 3) : r;
  const int w_f = S::kPairs ? (r >> 1 & 1) | (r >> 2) << 1 : r >> 1 & 7;
  const int w_at = (S::BM + wn * S::TN * 16 + w_row) * kStageRow + ((g ^ w_f) << 4);
  auto w_tile = [](int j) { return S::kPairs ? (j >> 1) * 32 * kStageRow + (j & 1) * 4 * kStageRow : j * 16 * kStageRow; };

  Tile t = locate(id_of(at));
  Loads loads = loads_of(t);
  issue_first(loads, t);
  for (;;) {
    // A wave whose rows all lie behind the tile's last one brings its share of
    // the stages and multiplies nothing: the matrix cores of its SIMD are the
    // other wave's (65536 rows over 128 experts, n 2048, k 768, fast
    // sums: 193 us, 189).
    if (GROUPED && S::WM > 1 && t.m0 + wm * S::TM * 16 >= t.end) {
      for (int b = t.blk0; b < t.blk1; ++b) {
        if (b + kAhead < t.blk1) {
          stage_barrier<kAfter>();
          issue(loads, b + kAhead, stage_in((b + kAhead - t.blk0) % S::kStages), scale_in((b + kAhead - t.blk0) % S::kStages));
        } else {
          stage_barrier<0>();
        }
      }
      at += stride;
      stage_barrier<63>();
      if (at >= all_count) return;
      t = locate(id_of(at));
      loads = loads_of(t);
      issue_first(loads, t);
      continue;
    }
    const int col0 = t.n0 + wn * S::TN * 16;
    // the scale of this wave's columns, read a block ahead (a vector load: a scalar
    // one would make every wait for an LDS read of its block a full one)
    const float *wsp = nullptr;
    if constexpr (FP8)
      wsp = p.w_scale + ((size_t)t.expert * fp8::ceil_div(p.n, 128) + ((col0 < p.n ? col0 : p.n - 1) >> 7)) * p.nb;
    auto scale_of = [&](int b) { return FP8 ? wsp[b < p.nb ? b : p.nb - 1] : 0.0f; };

    // The wave's weight operands stay in registers, the rows of x pass one
    // 16-row tile after the other, and a tile's products are added one tile
    // later, so that the fma run beside the matrix instructions. The last tile
    // of a block is multiplied after the barrier, each weight operand making
    // room for the next block's as it is used: the matrix cores have work while
    // the first reads of a stage are under way.
    v4f acc[S::TM][S::TN];
    Operand<KIND> wf[S::TN], xf[2];   // xf[1] between blocks: the last tile of the block before
    v4f d[2][S::TN];                  // d[0] between blocks: the products of the tile before that
    float s[2] = {0.0f, 0.0f};        // scales of the tiles in xf[1] and d[0]: s[1], s[0]
    float ws_before = 0.0f;
    {
      const Frag none = {{0, 0, 0, 0}, {0, 0, 0, 0}};
      xf[1].set(none);
#pragma unroll
      for (int j = 0; j < S::TN; ++j) {
        wf[j].set(none);
        d[0][j] = kZero4;
#pragma unroll
        for (int i = 0; i < S::TM; ++i) acc[i][j] = kZero4;
      }
    }
    // One block. With next_too the loads of block `sent` (a whole one) go out
    // over the first half.
    auto compute = [&](auto next_too, int sent, float ws, const uint8_t *stage, const float *scale, uint8_t *next,
                       float *next_scale) {
      constexpr int kEvery = (S::kLoads + (S::TM + 1) / 2 - 1) / ((S::TM + 1) / 2);
      auto fragment = [&](int lo, int more) {
        Frag f;
        f.lo = *reinterpret_cast<const v4i *>(stage + lo + more);
        f.hi = *reinterpret_cast<const v4i *>(stage + (lo ^ 64) + more);
        return f;
      };
#pragma unroll
      for (int i = -1; i < S::TM - 1; ++i) {
        // i = -1: the last tile of the block before
        constexpr int kLast = S::TM - 1;
        const int now = i & 1, then = now ^ 1;                 // buffers of this tile and of its neighbours
        const int tile = i < 0 ? kLast : i, back = i < 0 ? kLast - 1 : i == 0 ? kLast : i - 1;
        const float before = s[then] * (i <= 0 ? ws_before : ws);
        if constexpr (FP8) s[then] = scale[(wm * S::TM + i + 1) * 16 + r];
        const Frag x_next = fragment(x_at, (i + 1) * 16 * kStageRow);
        if constexpr (KIND != kExact) xf[then].set(x_next);
        if constexpr (decltype(next_too)::value) {
          if (i < 0) load_scales(loads, sent, next_scale);
#pragma unroll
          for (int l = (i + 1) * kEvery; l < (i + 2) * kEvery && l < S::kLoads; ++l) load_piece(loads, l, sent, next, false);
        }
        if constexpr (KIND == kExact) {
          // part by part of the block, so that four columns' sums take turns in
          // the matrix cores; the codes read above are widened behind them, each
          // part of the old operand being done with by then
          Frag w_next[S::TN];
          if (i < 0) {
#pragma unroll
            for (int j = 0; j < S::TN; ++j) w_next[j] = fragment(w_at, w_tile(j));
          }
#pragma unroll
          for (int h = 0; h < 4; ++h) {
#pragma unroll
            for (int j = 0; j < S::TN; ++j)
              d[now][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[j].v[h], xf[now].v[h], h ? d[now][j] : kZero4, 0, 0, 0);
#pragma unroll
            for (int j = h * S::TN / 4; j < (h + 1) * S::TN / 4; ++j) scaled_add(before, d[then][j], acc[back][j]);
            if (h >= 2) {
#pragma unroll
              for (int q = 2 * h - 4; q < 2 * h - 2; ++q) {
                xf[then].set(q, x_next);
                if (i < 0) {
#pragma unroll
                  for (int j = 0; j < S::TN; ++j) wf[j].set(q, w_next[j]);
                }
              }
            }
            __builtin_amdgcn_sched_barrier(0);
          }
        } else {
#pragma unroll
          for (int j = 0; j < S::TN; ++j) {
            if constexpr (FP8) {
              d[now][j] = mma_block<KIND>(wf[j], xf[now], kZero4);
              scaled_add(before, d[then][j], acc[back][j]);
            } else {
              acc[tile][j] = mma_block<KIND>(wf[j], xf[now], acc[tile][j]);
            }
            if (i < 0) wf[j].set(fragment(w_at, w_tile(j)));
            // keeps the fma of a result TN matrix instructions behind it
            if (KIND == kNative) __builtin_amdgcn_sched_barrier(0);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      ws_before = ws;
    };

    int b = t.blk0;
    float ws = scale_of(b);
    // one step of the steady loop: block b + u, sending b + u + kAhead (a whole one)
    auto step = [&](auto u) {
      constexpr int v = decltype(u)::value;
      using Next = std::integral_constant<int, v + kAhead>;
      stage_barrier<kAfter>();
      const float ws_next = scale_of(b + v + 1);
      compute(std::true_type{}, b + v + kAhead, ws, stage_of(u), scale_at(u), stage_of(Next{}), scale_at(Next{}));
      ws = ws_next;
    };
    // one of the last blocks: block b + u of `left`, sending b + u + kAhead if there is one
    auto last_step = [&](auto u, int left) {
      constexpr int v = decltype(u)::value;
      using Next = std::integral_constant<int, v + kAhead>;
      if (v >= left) return;
      stage_barrier<0>();
      const float ws_next = scale_of(b + v + 1);
      if (v + kAhead < left) issue(loads, b + v + kAhead, stage_of(Next{}), scale_at(Next{}));
      compute(std::false_type{}, 0, ws, stage_of(u), scale_at(u), nullptr, nullptr);
      ws = ws_next;
    };
    using U0 = std::integral_constant<int, 0>;
    using U1 = std::integral_constant<int, 1>;
    using U2 = std::integral_constant<int, 2>;
    using U3 = std::integral_constant<int, 3>;
    using U4 = std::integral_constant<int, 4>;
    using U5 = std::integral_constant<int, 5>;
    using U6 = std::integral_constant<int, 6>;
    for (; b + 2 * S::kStages - 1 < t.blk1; b += S::kStages) {
      step(U0{});
      step(U1{});
      if constexpr (S::kStages > 2) step(U2{});
      if constexpr (S::kStages > 3) step(U3{});
    }
    const int left = t.blk1 - b;   // 1 to 2 kStages - 1
    last_step(U0{}, left);
    last_step(U1{}, left);
    last_step(U2{}, left);
    if constexpr (S::kStages > 2) {
      last_step(U3{}, left);
      last_step(U4{}, left);
    }
    if constexpr (S::kStages > 3) {
      last_step(U5{}, left);
      last_step(U6{}, left);
    }

    // all waves are through with the stages: the next tile's loads may go
    at += stride;
    const bool more = at < all_count;
    const Tile done = t;
    stage_barrier<63>();
    if (more) {
      t = locate(id_of(at));
      loads = loads_of(t);
      issue_first(loads, t);
    }

    // the last tile of the last block
#pragma unroll
    for (int j = 0; j < S::TN; ++j) {
      if constexpr (FP8) {
        scaled_add(s[0] * ws_before, d[0][j], acc[S::TM - 2][j]);
        scaled_add(s[1] * ws_before, mma_block<KIND>(wf[j], xf[1], kZero4), acc[S::TM - 1][j]);
      } else {
        acc[S::TM - 1][j] = mma_block<KIND>(wf[j], xf[1], acc[S::TM - 1][j]);
      }
    }

    // A lane holds, of row r of each 16 rows of x, columns 8 g .. 8 g + 7 of each
    // 32 (from two tiles), or 4 g .. 4 g + 3 of each 16.
    constexpr int kWide = S::kPairs ? 8 : 4;
    if (!GROUPED && done.part >= 0) {
      // a part keeps the order of the registers: 1 KiB a store, in one piece
      float *to = p.part + (size_t)done.part * (S::BM * S::BN) + (size_t)wave * (S::TM * S::TN * 256) + lane * 4;
#pragma unroll
      for (int i = 0; i < S::TM; ++i)
#pragma unroll
        for (int j = 0; j < S::TN; ++j) *reinterpret_cast<v4f *>(to + (i * S::TN + j) * 256) = acc[i][j];
      if (!more) return;
      continue;
    }
    const bool bf16 = p.y_bf16;
    uint8_t *to = static_cast<uint8_t *>(p.y);
    // vector stores to any element's address: rows of y of odd lengths keep no alignment
    typedef __bf16 RowBf16 __attribute__((ext_vector_type(kWide), aligned(2)));
    typedef float RowF32 __attribute__((ext_vector_type(4), aligned(4)));
#pragma unroll
    for (int i = 0; i < S::TM; ++i) {
      const int row = done.m0 + (wm * S::TM + i) * 16 + r;
      if (row >= done.end) continue;
#pragma unroll
      for (int j = 0; j < S::TN; j += S::kPairs ? 2 : 1) {
        const int col = col0 + j * 16 + g * kWide;
        float v[kWide];
#pragma unroll
        for (int e = 0; e < kWide; ++e) v[e] = acc[i][j + e / 4][e % 4];
        const size_t place = (size_t)row * p.n + col;
        if (col + kWide > p.n) {
#pragma unroll
          for (int e = 0; e < kWide; ++e)
            if (col + e < p.n) {
              if (bf16)
                reinterpret_cast<__bf16 *>(to)[place + e] = (__bf16)v[e];
              else
                reinterpret_cast<float *>(to)[place + e] = v[e];
            }
        } else if (bf16) {
          RowBf16 o;
#pragma unroll
          for (int e = 0; e < kWide; ++e) o[e] = (__bf16)v[e];
          *reinterpret_cast<RowBf16 *>(reinterpret_cast<__bf16 *>(to) + place) = o;
        } else {
#pragma unroll
          for (int e = 0; e < kWide; e += 4)
            *reinterpret_cast<RowF32 *>(reinterpret_cast<float *>(to) + place + e) = RowF32{v[e], v[e + 1], v[e + 2], v[e + 3]};
        }
      }
    }
    if (!more) return;
  }
}

// y of the tiles that were cut along k: the parts in the order of k, a lane's
// four or eight neighbouring columns a thread. Bound by the parts' bytes, read
// once and past the caches that the next call's operands use (512 x 5120 x
// 17408, fast sums: the whole call 58.7 us with plain loads, 57.1 so).
template <class S>
__global__ __launch_bounds__(256) void product_sum_kernel(const ProductArgs p, const int t_main, const int r_tiles,
                                                          const int splits) {
  constexpr int kQuads = S::kPairs ? 2 : 1, kWide = 4 * kQuads, kRow = S::TN / kQuads;
  constexpr int kThreads = S::BM * S::BN / kWide;   // of a tile, whole blocks
  const int at = (int)blockIdx.x * 256 + (int)threadIdx.x, in = at % kThreads, tile = uniform(at / kThreads);
  const int lane = in & 63, j = in / 64 % kRow * kQuads, i = in / (64 * kRow) % S::TM, wave = in / (64 * kRow * S::TM);
  int m0, n0;
  tile_place<S>(t_main + tile, p.rows, fp8::ceil_div(p.n, S::BN), m0, n0);
  const int row = m0 + (wave / S::WN * S::TM + i) * 16 + (lane & 15);
  const int col = n0 + (wave % S::WN * S::TN + j) * 16 + (lane >> 4) * kWide;
  if (row >= p.rows || col >= p.n) return;
  const float *from = p.part + (size_t)tile * (S::BM * S::BN) + ((wave * S::TM + i) * S::TN + j) * 256 + lane * 4;
  v4f v[kQuads];
#pragma unroll
  for (int h = 0; h < kQuads; ++h) v[h] = __builtin_nontemporal_load(reinterpret_cast<const v4f *>(from + h * 256));
#pragma unroll 4
  for (int s = 1; s < splits; ++s)
#pragma unroll
    for (int h = 0; h < kQuads; ++h)
      v[h] += __builtin_nontemporal_load(
          reinterpret_cast<const v4f *>(from + (size_t)s * r_tiles * (S::BM * S::BN) + h * 256));
  const size_t place = (size_t)row * p.n + col;
  typedef __bf16 RowBf16 __attribute__((ext_vector_type(kWide), aligned(2)));
  typedef float RowF32 __attribute__((ext_vector_type(4), aligned(4)));
  if (col + kWide > p.n) {
#pragma unroll
    for (int e = 0; e < kWide; ++e)
      if (col + e < p.n) {
        if (p.y_bf16)
          static_cast<__bf16 *>(p.y)[place + e] = (__bf16)v[e / 4][e % 4];
        else
          static_cast<float *>(p.y)[place + e] = v[e / 4][e % 4];
      }
  } else if (p.y_bf16) {
    RowBf16 o;
#pragma unroll
    for (int e = 0; e < kWide; ++e) o[e] = (__bf16)v[e / 4][e % 4];
    *reinterpret_cast<RowBf16 *>(static_cast<__bf16 *>(p.y) + place) = o;
  } else {
#pragma unroll
    for (int h = 0; h < kQuads; ++h)
      *reinterpret_cast<RowF32 *>(static_cast<float *>(p.y) + place + h * 4) = RowF32{v[h][0], v[h][1], v[h][2], v[h][3]};
  }
}

using Tile32 = Shape<32, 64, 1, 4, 3>;
using Tile64 = Shape<64, 128, 1, 4, 3>;
using Tile128 = Shape<128, 128, 4, 2, 4>;
using Tile256 = Shape<256, 128, 4, 2, 3>;
using Tile256Wide = Shape<256, 256, 2, 4, 2>;

template <class S>
unsigned grid_of(int64_t tiles) {
  const int64_t most = (int64_t)S::kPerCu * fp8::kSlots;
  return (unsigned)(tiles < most ? tiles : most);
}

template <class S, Kind KIND>
int launch_dense(const ProductArgs &a, const fp8::DensePlan &plan, hipStream_t s) {
  const int rc = launch_kernel("product_tile_kernel", product_tile_kernel<S, KIND, false>,
                               dim3(grid_of<S>((int64_t)plan.t_main + (int64_t)plan.r_tiles * plan.splits)),
                               dim3(S::kThreads), 0, s, a, plan.t_main, plan.r_tiles, plan.splits);
  if (rc || plan.r_tiles == 0) return rc;
  return launch_kernel("product_sum_kernel", product_sum_kernel<S>, dim3((unsigned)(plan.r_tiles * (S::BM * S::BN / (S::kPairs ? 2048 : 1024)))),
                       dim3(256), 0, s, a, plan.t_main, plan.r_tiles, plan.splits);
}

template <class S, Kind KIND>
int launch_grouped(const ProductArgs &a, hipStream_t s) {
  const int64_t tiles = fp8::grouped_row_tiles(a.rows, a.n_experts, S::BM) * fp8::ceil_div(a.n, S::BN);
  return launch_kernel("product_tile_kernel", product_tile_kernel<S, KIND, true>, dim3(grid_of<S>(tiles)),
                       dim3(S::kThreads), 0, s, a, 0, 0, 1);
}

template <Kind KIND>
int launch_grouped(int tile, const ProductArgs &a, hipStream_t s) {
  if (tile == fp8::kTile32) return launch_grouped<Tile32, KIND>(a, s);
  if (tile == fp8::kTile64) return launch_grouped<Tile64, KIND>(a, s);
  if constexpr (KIND == kExact) {
    return launch_grouped<Tile256, KIND>(a, s);
  } else {
    return tile == fp8::kTile128 ? launch_grouped<Tile128, KIND>(a, s) : launch_grouped<Tile256Wide, KIND>(a, s);
  }
}

template <int MW>
int launch_stream(const ProductArgs &a, const fp8::StreamPlan &plan, hipStream_t s) {
  const dim3 grid((unsigned)fp8::ceil_div(a.n, plan.tile), (unsigned)fp8::ceil_div(a.rows, 16));
  constexpr int kDepth = MW == 1 ? 3 : 2;
  switch (plan.waves) {
    case 16: return launch_kernel("fp8_stream_kernel", fp8_stream_kernel<16, MW, kDepth>, grid, dim3(1024), 0, s, a, plan.tile);
    case 8: return launch_kernel("fp8_stream_kernel", fp8_stream_kernel<8, MW, kDepth>, grid, dim3(512), 0, s, a, plan.tile);
    default: return launch_kernel("fp8_stream_kernel", fp8_stream_kernel<4, MW, kDepth>, grid, dim3(256), 0, s, a, plan.tile);
  }
}

int launch_stream(const ProductArgs &a, hipStream_t s) {
  const fp8::StreamPlan plan = fp8::stream_plan(a.rows, a.n, a.nb);
  return plan.tile > 16 ? launch_stream<2>(a, plan, s) : launch_stream<1>(a, plan, s);
}

}  // namespace

int launch_fp8_dense(const ProductArgs &a, void *stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const fp8::DensePlan plan = fp8::dense_plan(a.rows, a.n, a.k_bytes, a.fast);
  if (plan.stream) return launch_stream(a, s);
  switch (plan.tile) {
    case fp8::kTile32:
      return a.fast ? launch_dense<Tile32, kNative>(a, plan, s) : launch_dense<Tile32, kExact>(a, plan, s);
    case fp8::kTile64:
      return a.fast ? launch_dense<Tile64, kNative>(a, plan, s) : launch_dense<Tile64, kExact>(a, plan, s);
    case fp8::kTile128:
      return a.fast ? launch_dense<Tile128, kNative>(a, plan, s) : launch_dense<Tile128, kExact>(a, plan, s);
    case fp8::kTile256:
      return a.fast ? launch_dense<Tile256, kNative>(a, plan, s) : launch_dense<Tile256, kExact>(a, plan, s);
    default: return launch_dense<Tile256Wide, kNative>(a, plan, s);
  }
}

int launch_fp8_grouped(const ProductArgs &a, void *stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int tile = fp8::grouped_tile(a.rows, a.n_experts, a.n, a.nb, !a.fast);
  return a.fast ? launch_grouped<kNative>(tile, a, s) : launch_grouped<kExact>(tile, a, s);
}

int launch_bf16_grouped(const ProductArgs &a, void *stream) {
  return launch_grouped<kBf16>(fp8::grouped_tile(a.rows, a.n_experts, a.n, a.nb, false), a, static_cast<hipStream_t>(stream));
}

}  // namespace qmv
