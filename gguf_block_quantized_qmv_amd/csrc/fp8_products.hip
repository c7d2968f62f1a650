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
//  * kNative, one v_mfma_f32_16x16x128_f8f6f4. The instruction aligns each
//    eight neighbouring products to the largest of them and cuts what lies 13
//    bits below (measured: 2^16 + 2^2 in one group of eight gives 2^16, in two
//    groups 2^16 + 2^2); on normal data that is 1.6e-5 of the result's norm.
//  * kExact, the codes as bf16 (exact, two by one v_cvt_scalef32_pk_bf16_fp8)
//    through four v_mfma_f32_16x16x32_bf16, whose sums keep fp32 (5e-8), at
//    half the matrix rate.
// Results in fp32 are kExact. Results in bf16, whose rounding (2^-9 on average
// of its value) is a hundred times the native sums' error, are kNative where
// the matrix cores bound the product and kExact where the weight stream does.
// bf16 operands (kBf16) take two v_mfma_f32_16x16x32_bf16 a block.
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

// Sixteen e4m3 codes as two bf16 MFMA operands (exact; NaN stays NaN).
__device__ __forceinline__ void widen(const v4i c, bf16x8 &lo, bf16x8 &hi) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)c[i], 1.0f, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)c[i], 1.0f, true);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)c[2 + i], 1.0f, false);
    const bf16x2 e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)c[2 + i], 1.0f, true);
    lo[4 * i] = a[0]; lo[4 * i + 1] = a[1]; lo[4 * i + 2] = b[0]; lo[4 * i + 3] = b[1];
    hi[4 * i] = d[0]; hi[4 * i + 1] = d[1]; hi[4 * i + 2] = e[0]; hi[4 * i + 3] = e[1];
  }
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
  __device__ __forceinline__ void set(const Frag &f) {
    widen(f.lo, v[0], v[1]);
    widen(f.hi, v[2], v[3]);
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

// Row of x behind row `row` of y; false (and row 0) for an index outside x.
__device__ __forceinline__ bool source_row(const ProductArgs &p, int row, int &src) {
  src = p.index ? p.index[row] : row;
  const bool ok = (unsigned)src < (unsigned)p.x_rows;
  src = ok ? src : 0;
  return ok;
}

__device__ __forceinline__ void store_y(const ProductArgs &p, int row, int col, float v) {
  const size_t at = (size_t)row * p.n + col;
  if (p.y_bf16)
    static_cast<__bf16 *>(p.y)[at] = (__bf16)v;
  else
    static_cast<float *>(p.y)[at] = v;
}

// ---- a few rows: stream the weights ---------------------------------------------
//
// A workgroup owns `tile` <= 16 rows of one weight matrix and up to 16 rows of
// x at a time; wave v takes blocks v, v + NW, ... of k straight from memory
// into MFMA fragments (no LDS), kDepth blocks in flight, and the waves' sums
// are added in wave order. Bound by the weight stream. The host chooses the
// tile so that every CU gets the same number of workgroups (a tile shorter
// than 16 rows repeats its last row: matrix work, no memory traffic). The order
// of the sums goes by (n, k) alone and the columns of an MFMA do not mix, so a
// row of x has the same bits in any company. Grouped: workgroup (t, s) serves
// the s-th expert that has rows, and takes 16 of its rows at a time.
constexpr int kDepth = 3;

template <Kind KIND, bool GROUPED, int NW>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(4))) void product_stream_kernel(
    const ProductArgs p, const int tile) {
  constexpr bool FP8 = is_e4m3(KIND);
  __shared__ float red[NW][256];
  const int lane = (int)threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int n0 = (int)blockIdx.x * tile;
  const int n1 = n0 + tile < p.n ? n0 + tile : p.n;
  int expert = 0, begin = 0, end = p.rows;
  if constexpr (GROUPED) {
    int want = (int)blockIdx.y, found = -1;
    for (int base = 0; base < p.n_experts && found < 0; base += 64) {
      int b0 = 0, b1 = 0;
      if (base + lane < p.n_experts) expert_rows(p.offsets, base + lane, p.rows, b0, b1);
      uint64_t mask = __ballot(b1 > b0);
      const int have = __popcll(mask);
      if (want < have) {
        for (int i = 0; i < want; ++i) mask &= mask - 1;
        found = base + __ffsll((unsigned long long)mask) - 1;
      }
      want -= have;
    }
    if (found < 0) return;
    expert = uniform(found);
    expert_rows(p.offsets, expert, p.rows, begin, end);
  }
  // Lane offsets from scalar addresses. They are hidden from the optimiser at
  // every use, which would otherwise keep one 64-bit address per block alive.
  const uint8_t *wbase = p.w + ((size_t)expert * p.n + n0) * p.k_bytes;
  uint32_t wlane = (uint32_t)(n0 + r < n1 ? r : n1 - 1 - n0) * (uint32_t)p.k_bytes + g * 16;
  // tiles are multiples of four rows: a lane's four results share a scale
  const float *wsbase = FP8 ? p.w_scale + (size_t)expert * fp8::ceil_div(p.n, 128) * p.nb : nullptr;
  const int srow = n0 + g * 4 < p.n ? n0 + g * 4 : p.n - 1;
  uint32_t wslane = FP8 ? (uint32_t)(srow >> 7) * (uint32_t)p.nb : 0;
  const int whole = p.k_bytes >> 7, tail = p.k_bytes & 127;

  for (int t0 = begin; t0 < end; t0 += 16) {
    int src;
    source_row(p, t0 + r < end ? t0 + r : end - 1, src);
    using Offset = std::conditional_t<GROUPED, uint64_t, uint32_t>;   // dense: within 16 rows
    Offset xlane = (Offset)src * (Offset)p.k_bytes + (Offset)(g * 16);
    uint32_t xslane = (uint32_t)src;

    Frag wf[kDepth], xf[kDepth];
    float xs[kDepth], ws[kDepth];
    // Block b (past the last whole one: zeros, so that every pass of the loop
    // sends the same loads and each wait counts exactly those behind it).
    auto load_scales = [&](int b, int u, bool ok) {
      if constexpr (FP8) {
        asm("" : "+v"(xslane), "+v"(wslane));
        const float *zeros = reinterpret_cast<const float *>(g_zeros);
        xs[u] = (ok ? p.x_scale + (size_t)b * p.x_rows : zeros)[ok ? xslane : 0];
        ws[u] = (ok ? wsbase + b : zeros)[ok ? wslane : 0];
      }
    };
    auto load = [&](int b, int u) {
      asm("" : "+v"(wlane), "+v"(xlane));
      const bool ok = b < whole;
      const uint8_t *zeros = reinterpret_cast<const uint8_t *>(g_zeros);
      const uint8_t *w = (ok ? wbase + (size_t)b * 128 : zeros) + (ok ? wlane : 0);
      const uint8_t *x = (ok ? p.x + (size_t)b * 128 : zeros) + (ok ? xlane : 0);
      wf[u].lo = __builtin_nontemporal_load(reinterpret_cast<const v4i *>(w));
      wf[u].hi = __builtin_nontemporal_load(reinterpret_cast<const v4i *>(w + 64));
      xf[u].lo = *reinterpret_cast<const v4i *>(x);
      xf[u].hi = *reinterpret_cast<const v4i *>(x + 64);
      load_scales(b, u, ok);
    };
    v4f acc = kZero4;
    auto use = [&](int u) {
      Operand<KIND> a, c;
      a.set(wf[u]);
      c.set(xf[u]);
      if constexpr (FP8)
        scaled_add(xs[u] * ws[u], mma_block<KIND>(a, c, kZero4), acc);
      else
        acc = mma_block<KIND>(a, c, acc);
    };
#pragma unroll
    for (int u = 0; u < kDepth; ++u) load(wave + u * NW, u);
    for (int b = wave; b < whole; b += kDepth * NW)
#pragma unroll
      for (int u = 0; u < kDepth; ++u) {
        use(u);
        load(b + (u + kDepth) * NW, u);
        __builtin_amdgcn_sched_barrier(0);   // one block's widened operands at a time
      }
    if (tail && wave == whole % NW) {   // the partial last block: zeros past the row
      const v4i none = {0, 0, 0, 0};
      wf[0].lo = wf[0].hi = xf[0].lo = xf[0].hi = none;
      const uint8_t *w = wbase + (size_t)whole * 128 + wlane, *x = p.x + (size_t)whole * 128 + xlane;
      if (g * 16 < tail) {
        wf[0].lo = *reinterpret_cast<const v4i *>(w);
        xf[0].lo = *reinterpret_cast<const v4i *>(x);
      }
      if (g * 16 + 64 < tail) {
        wf[0].hi = *reinterpret_cast<const v4i *>(w + 64);
        xf[0].hi = *reinterpret_cast<const v4i *>(x + 64);
      }
      load_scales(whole, 0, true);
      use(0);
    }
    // lane l holds columns 4 g .. 4 g + 3 of row r of x
    *reinterpret_cast<v4f *>(&red[wave][r * 16 + g * 4]) = acc;
    __syncthreads();
    if ((int)threadIdx.x < 256) {
      const int row = t0 + ((int)threadIdx.x >> 4), col = n0 + ((int)threadIdx.x & 15);
      float sum = red[0][threadIdx.x];
#pragma unroll
      for (int v = 1; v < NW; ++v) sum += red[v][threadIdx.x];
      if (row < end && col < n1) {
        int at;
        store_y(p, row, col, source_row(p, row, at) ? sum : 0.0f);
      }
    }
    __syncthreads();
  }
}

// ---- many rows: tiles through LDS --------------------------------------------------
//
// A workgroup owns BM rows of x by BN rows of w. Each step moves one block of
// k of both into one of two LDS stages by direct-to-LDS loads while the waves
// multiply the other stage; one barrier a step hands the stages over. A stage
// row is 128 bytes, eight 16-byte chunks; chunk c of row r sits at slot
// c ^ ((r / 2) % 8), which leaves the fragment reads (16 consecutive rows, one
// chunk) free of bank conflicts. The direct loads write LDS in lane order, so
// the permutation is applied to the global address each lane reads.
constexpr int kStageRow = 128;

template <int BM_, int BN_, int WM_, int WN_>
struct Shape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;   // waves along rows of x, of w
  static constexpr int kWaves = WM * WN, kThreads = kWaves * 64;
  static constexpr int TM = BM / WM / 16, TN = BN / WN / 16;     // MFMA tiles of a wave
  static constexpr int kLoads = (BM + BN) / 8 / kWaves;          // 1 KiB direct loads of a wave and step
  static constexpr int kStageBytes = (BM + BN) * kStageRow;
  static_assert((BM + BN) % (8 * kWaves) == 0 && TM * WM * 16 == BM && TN * WN * 16 == BN, "whole tiles and loads");
  static_assert(BN / WN <= 128 && 128 % (BN / WN) == 0, "a wave's columns lie under one weight scale");
};

// Buffer form of the direct load: LDS at `to` + 16 (or 4) bytes a lane gets
// the bytes at base + at + step; at or beyond `size` it gets zeros. (Unlike the
// global form it does not make the compiler drain the LDS reads in flight.)
typedef __amdgpu_buffer_rsrc_t Buffer;
__device__ __forceinline__ Buffer buffer_of(const void *base, uint32_t size) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, (int)size, 0x00020000);
}
constexpr uint32_t kOutside = 0xFFFFFFFFu;   // an offset past every buffer
__device__ __forceinline__ void load_lds16(Buffer from, uint32_t at, uint32_t step, void *to) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void *)to, 16, (int)at, (int)step,
                                           0, 0);
}
__device__ __forceinline__ void load_lds4(Buffer from, uint32_t at, uint32_t step, void *to) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void *)to, 4, (int)at, (int)step,
                                           0, 0);
}

// Every direct load of this wave has landed and every LDS read has returned,
// then all waves meet.
__device__ __forceinline__ void stage_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070);   // vmcnt(0) lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// id -> position in an order that gives each of the eight XCDs (workgroups are
// dealt to them in turn) one contiguous run of [0, total).
__device__ __forceinline__ int xcd_order(int id, int total) {
  const int q = total >> 3, rest = total & 7, x = id & 7;
  return x * q + (x < rest ? x : rest) + (id >> 3);
}

template <class S, Kind KIND, bool GROUPED>
__global__ __launch_bounds__(S::kThreads) void product_tile_kernel(const ProductArgs p) {
  constexpr bool FP8 = is_e4m3(KIND);
  __shared__ __attribute__((aligned(1024))) uint8_t stage0[S::kStageBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t stage1[S::kStageBytes];
  __shared__ float scale0[(S::BM + 63) / 64 * 64], scale1[(S::BM + 63) / 64 * 64];
  const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int n_tiles = fp8::ceil_div(p.n, S::BN);

  // this workgroup's tile
  int expert = 0, m0, begin = 0, end = p.rows, nt, part = 0;
  if constexpr (GROUPED) {
    // row tiles of each lane's run of experts, and their running sum over the lanes
    const int per = fp8::ceil_div(p.n_experts, 64), e0 = lane * per;
    int mine = 0;
    for (int e = e0; e < e0 + per && e < p.n_experts; ++e) {
      int b0, b1;
      expert_rows(p.offsets, e, p.rows, b0, b1);
      mine += fp8::ceil_div(b1 - b0, S::BM);
    }
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(upto, d);
      if (lane >= d) upto += o;
    }
    const int total = __builtin_amdgcn_readfirstlane(__shfl(upto, 63));
    // decreasing offsets can give more tiles than the grid holds: they are not done
    const int all = total < (int)gridDim.x / n_tiles ? total * n_tiles : (int)gridDim.x;
    if ((int)blockIdx.x >= all) return;
    const int id = xcd_order((int)blockIdx.x, all);
    const int mt = id / n_tiles;
    nt = id - mt * n_tiles;
    const int owner = __ffsll((unsigned long long)__ballot(upto > mt)) - 1;
    int left = mt - __builtin_amdgcn_readfirstlane(__shfl(upto - mine, owner));
    expert = owner * per;
    for (;;) {
      expert_rows(p.offsets, expert, p.rows, begin, end);
      const int t = fp8::ceil_div(end - begin, S::BM);
      if (left < t) break;
      left -= t;
      ++expert;
    }
    expert = __builtin_amdgcn_readfirstlane(expert);
    m0 = begin + left * S::BM;
  } else {
    const int m_tiles = fp8::ceil_div(p.rows, S::BM);
    const int tiles = m_tiles * n_tiles;
    int id = xcd_order((int)blockIdx.x, tiles * p.splits);
    part = id / tiles;
    id -= part * tiles;
    // bands of eight row tiles, rows first within a band
    const int band = id / (8 * n_tiles), in = id - band * 8 * n_tiles;
    const int high = m_tiles - band * 8 < 8 ? m_tiles - band * 8 : 8;
    nt = in / high;
    m0 = (band * 8 + in - nt * high) * S::BM;
  }
  // uniform, but divided on vector lanes: into scalar registers
  m0 = uniform(m0);
  nt = uniform(nt);
  begin = uniform(begin);
  end = uniform(end);
  const int n0 = nt * S::BN;
  const int blk0 = GROUPED ? 0 : uniform((int)((int64_t)p.nb * part / p.splits));
  const int blk1 = GROUPED ? p.nb : uniform((int)((int64_t)p.nb * (part + 1) / p.splits));

  // This lane's direct loads: row q * 8 + lane / 8 of the stage, chunk by the
  // slot, as an offset from a scalar base: the tile's first row of w, and of x
  // unless its rows are gathered (from all of x, which the host then keeps under
  // 4 GiB).
  const bool gather = GROUPED && p.index;
  const Buffer wbuf = buffer_of(p.w + ((size_t)expert * p.n + n0) * p.k_bytes,
                                (uint32_t)(p.n - n0 < S::BN ? p.n - n0 : S::BN) * (uint32_t)p.k_bytes);
  const int x_first = gather ? 0 : m0, x_count = gather ? p.x_rows : end - m0 < S::BM ? end - m0 : S::BM;
  const Buffer xbuf = buffer_of(p.x + (size_t)x_first * p.k_bytes, (uint32_t)x_count * (uint32_t)p.k_bytes);
  uint32_t from[S::kLoads];
  int chunk_at[S::kLoads];
  int src[S::kLoads];
#pragma unroll
  for (int i = 0; i < S::kLoads; ++i) {
    const int row = (wave * S::kLoads + i) * 8 + (lane >> 3);
    chunk_at[i] = ((lane & 7) ^ ((row >> 1) & 7)) * 16;
    if (wave * S::kLoads + i < S::BM / 8)
      src[i] = (m0 + row < end ? m0 + row : end - 1) - x_first;
    else
      src[i] = n0 + row - S::BM < p.n ? row - S::BM : p.n - 1 - n0;
  }
  if (gather) {   // all index loads before the first use
    int found[S::kLoads];
#pragma unroll
    for (int i = 0; i < S::kLoads; ++i) found[i] = p.index[wave * S::kLoads + i < S::BM / 8 ? src[i] : m0];
#pragma unroll
    for (int i = 0; i < S::kLoads; ++i)
      if (wave * S::kLoads + i < S::BM / 8) src[i] = (unsigned)found[i] < (unsigned)p.x_rows ? found[i] : 0;
  }
#pragma unroll
  for (int i = 0; i < S::kLoads; ++i) from[i] = (uint32_t)src[i] * (uint32_t)p.k_bytes + (uint32_t)chunk_at[i];
  // the scales of x, 64 rows a wave (waves past the tile's rows bring the same
  // values again: no branch in the loop)
  constexpr int kScaleRows = (S::BM + 63) / 64 * 64;
  const int scale_to = wave * 64 % kScaleRows;
  uint32_t scale_from = 0;
  if constexpr (FP8) {
    const int row = m0 + scale_to + lane;
    int at;
    source_row(p, row < end ? row : end - 1, at);
    scale_from = (uint32_t)at * 4;
  }
  const int tail = p.k_bytes & 127;   // bytes of a partial last block
  // one of the wave's direct loads of block b
  auto load_piece = [&](int i, int b, uint8_t *stage, bool last) {
    const uint32_t at = last && chunk_at[i] >= tail ? kOutside : from[i];
    uint8_t *to = stage + (wave * S::kLoads + i) * 1024;
    if (wave * S::kLoads + i < S::BM / 8)
      load_lds16(xbuf, at, (uint32_t)b * 128, to);
    else
      load_lds16(wbuf, at, (uint32_t)b * 128, to);
  };
  auto load_scales = [&](int b, float *scale) {
    if constexpr (FP8)
      load_lds4(buffer_of(p.x_scale + (size_t)b * p.x_rows, (uint32_t)p.x_rows * 4), scale_from, 0, scale + scale_to);
  };
  // all loads of block b, which may be the partial last one
  auto issue = [&](int b, uint8_t *stage, float *scale) {
    const bool partial = tail != 0 && b == p.nb - 1;
#pragma unroll
    for (int i = 0; i < S::kLoads; ++i) load_piece(i, b, stage, partial);
    load_scales(b, scale);
  };

  const int wm = wave / S::WN, wn = wave % S::WN;
  const int r = lane & 15, g = lane >> 4;
  const int frag_at = r * kStageRow + ((g ^ ((r >> 1) & 7)) << 4);   // chunk g of row r; chunk g + 4 is 64 bytes on or back
  const int x_at = wm * S::TM * 16 * kStageRow + frag_at;
  const int w_at = (S::BM + wn * S::TN * 16) * kStageRow + frag_at;
  const int col0 = n0 + wn * S::TN * 16;
  const int sblk = (col0 < p.n ? col0 : p.n - 1) >> 7;
  // the scale of this wave's columns, read a block ahead (a vector load: a scalar
  // one would make every wait for an LDS read of its block a full one)
  const float *wsp = FP8 ? p.w_scale + ((size_t)expert * fp8::ceil_div(p.n, 128) + uniform(sblk)) * p.nb : nullptr;
  auto scale_of = [&](int b) { return FP8 ? wsp[b < p.nb ? b : p.nb - 1] : 0.0f; };

  v4f acc[S::TM][S::TN];
#pragma unroll
  for (int i = 0; i < S::TM; ++i)
#pragma unroll
    for (int j = 0; j < S::TN; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  // One block: the wave's weight operands stay in registers, the rows of x pass
  // one 16-row tile after the other, and a tile's products are added one tile
  // later, so that the fma run beside the matrix instructions. The last tile of
  // a block is multiplied after the barrier, each weight operand making room for
  // the next block's as it is used: the matrix cores have work while the first
  // reads of a stage are under way. With next_too the loads of the next block (a
  // whole one) go out over the first half.
  Operand<KIND> wf[S::TN], xf[2];   // xf[1] between blocks: the last tile of the block before
  v4f d[2][S::TN];                  // d[0] between blocks: the products of the tile before that
  float s[2] = {0.0f, 0.0f};        // scales of the tiles in xf[1] and d[0]: s[1], s[0]
  float ws_before = 0.0f;
  static_assert(S::TM % 2 == 0, "tiles alternate between two registers");
  {
    const Frag none = {{0, 0, 0, 0}, {0, 0, 0, 0}};
    xf[1].set(none);
#pragma unroll
    for (int j = 0; j < S::TN; ++j) {
      wf[j].set(none);
      d[0][j] = kZero4;
    }
  }
  auto compute = [&](auto next_too, int b, float ws, const uint8_t *stage, const float *scale, uint8_t *next, float *next_scale) {
    constexpr int kEvery = (S::kLoads + (S::TM + 1) / 2 - 1) / ((S::TM + 1) / 2);
    auto read = [&](int lo, int hi, int rows16, Operand<KIND> &to) {
      Frag f;
      f.lo = *reinterpret_cast<const v4i *>(stage + lo + rows16 * 2048);
      f.hi = *reinterpret_cast<const v4i *>(stage + hi + rows16 * 2048);
      to.set(f);
    };
#pragma unroll
    for (int i = -1; i < S::TM - 1; ++i) {
      // i = -1: the last tile of the block before
      constexpr int kLast = S::TM - 1;
      const int now = i & 1, then = now ^ 1;                 // buffers of this tile and of its neighbours
      const int tile = i < 0 ? kLast : i, back = i < 0 ? kLast - 1 : i == 0 ? kLast : i - 1;
      const float before = s[then] * (i <= 0 ? ws_before : ws);
      if constexpr (FP8) s[then] = scale[(wm * S::TM + i + 1) * 16 + r];
      read(x_at, x_at ^ 64, i + 1, xf[then]);
      if constexpr (decltype(next_too)::value) {
        if (i < 0) load_scales(b + 1, next_scale);
#pragma unroll
        for (int l = (i + 1) * kEvery; l < (i + 2) * kEvery && l < S::kLoads; ++l) load_piece(l, b + 1, next, false);
      }
#pragma unroll
      for (int j = 0; j < S::TN; ++j) {
        if constexpr (FP8) {
          d[now][j] = mma_block<KIND>(wf[j], xf[now], kZero4);
          scaled_add(before, d[then][j], acc[back][j]);
        } else {
          acc[tile][j] = mma_block<KIND>(wf[j], xf[now], acc[tile][j]);
        }
        if (i < 0) read(w_at, w_at ^ 64, j, wf[j]);
        // keeps the fma of a result TN matrix instructions behind it
        if (KIND == kNative) __builtin_amdgcn_sched_barrier(0);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    ws_before = ws;
  };

  issue(blk0, stage0, scale0);
  int b = blk0;
  float ws = scale_of(b);
  for (; b + 3 < blk1; b += 2) {   // the loads sent here are all of whole blocks
    stage_barrier();
    const float ws1 = scale_of(b + 1);
    compute(std::true_type{}, b, ws, stage0, scale0, stage1, scale1);
    stage_barrier();
    ws = scale_of(b + 2);
    compute(std::true_type{}, b + 1, ws1, stage1, scale1, stage0, scale0);
  }
  const int left = blk1 - b;       // one to three blocks, the first of them on its way
  const float ws1 = scale_of(b + 1), ws2 = scale_of(b + 2);
  stage_barrier();
  if (left > 1) issue(b + 1, stage1, scale1);
  compute(std::false_type{}, b, ws, stage0, scale0, nullptr, nullptr);
  if (left > 1) {
    stage_barrier();
    if (left > 2) issue(b + 2, stage0, scale0);
    compute(std::false_type{}, b + 1, ws1, stage1, scale1, nullptr, nullptr);
    if (left > 2) {
      stage_barrier();
      compute(std::false_type{}, b + 2, ws2, stage0, scale0, nullptr, nullptr);
    }
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

  // lane: columns 4 g .. 4 g + 3 of row r of each 16 x 16 tile
#pragma unroll
  for (int i = 0; i < S::TM; ++i) {
    const int row = m0 + (wm * S::TM + i) * 16 + r;
    if (row >= end) continue;
    bool ok = true;
    if constexpr (GROUPED) {
      int src;
      ok = source_row(p, row, src);
    }
#pragma unroll
    for (int j = 0; j < S::TN; ++j) {
      const int col = col0 + j * 16 + g * 4;
      const v4f zero = {0.0f, 0.0f, 0.0f, 0.0f};
      const v4f v = ok ? acc[i][j] : zero;
      if (!GROUPED && p.splits > 1) {
        float *to = p.part + ((size_t)part * p.rows + row) * p.n + col;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (col + e < p.n) to[e] = v[e];
        continue;
      }
      if ((p.n & 3) == 0) {   // four columns at once: rows of y keep the alignment of y
        if (col >= p.n) continue;
        const size_t at = (size_t)row * p.n + col;
        if (p.y_bf16) {
          typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
          *reinterpret_cast<bf16x4 *>(static_cast<__bf16 *>(p.y) + at) =
              bf16x4{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
        } else {
          *reinterpret_cast<v4f *>(static_cast<float *>(p.y) + at) = v;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (col + e < p.n) store_y(p, row, col + e, v[e]);
      }
    }
  }
}

// y of a product split along k: the parts in the order of k.
__global__ __launch_bounds__(256) void product_sum_kernel(const float *__restrict__ part, const ProductArgs p) {
  const size_t count = (size_t)p.rows * p.n;
  const size_t at = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= count) return;
  float v = part[at];
  for (int s = 1; s < p.splits; ++s) v += part[(size_t)s * count + at];
  if (p.y_bf16)
    static_cast<__bf16 *>(p.y)[at] = (__bf16)v;
  else
    static_cast<float *>(p.y)[at] = v;
}

using Tile32 = Shape<32, 128, 1, 4>;
using Tile64 = Shape<64, 128, 1, 4>;
using Tile128 = Shape<128, 128, 2, 2>;
using Tile256 = Shape<256, 256, 2, 4>;

template <class S, Kind KIND, bool GROUPED>
int launch_tile(const ProductArgs &a, unsigned grid, hipStream_t s) {
  return launch_kernel("product_tile_kernel", product_tile_kernel<S, KIND, GROUPED>, dim3(grid), dim3(S::kThreads), 0,
                       s, a);
}

template <Kind KIND, bool GROUPED>
int launch_tiles(int tile, const ProductArgs &a, hipStream_t s) {
  const int bm = fp8::tile_rows(tile), bn = fp8::tile_cols(tile);
  const int64_t row_tiles = GROUPED ? fp8::grouped_row_tiles(a.rows, a.n_experts, bm) : fp8::ceil_div(a.rows, bm);
  const unsigned grid = (unsigned)(row_tiles * fp8::ceil_div(a.n, bn) * a.splits);
  switch (tile) {
    case fp8::kTile32: return launch_tile<Tile32, KIND, GROUPED>(a, grid, s);
    case fp8::kTile64: return launch_tile<Tile64, KIND, GROUPED>(a, grid, s);
    case fp8::kTile128: return launch_tile<Tile128, KIND, GROUPED>(a, grid, s);
    default:
      if constexpr (KIND == kNative && !GROUPED) return launch_tile<Tile256, KIND, GROUPED>(a, grid, s);
      set_error_detail("product_tile_kernel", 0, "no such tile");
      return QMV_ERR_HIP;
  }
}

template <Kind KIND, bool GROUPED>
int launch_stream(const ProductArgs &a, hipStream_t s) {
  const int slots = GROUPED ? (a.rows < a.n_experts ? a.rows : a.n_experts) : 1;
  const fp8::StreamPlan plan = fp8::stream_plan(a.n, a.nb, slots);
  const dim3 grid((unsigned)fp8::ceil_div(a.n, plan.tile), (unsigned)slots);
  switch (plan.waves) {
    case 16: return launch_kernel("product_stream_kernel", product_stream_kernel<KIND, GROUPED, 16>, grid, dim3(1024), 0, s, a, plan.tile);
    case 8: return launch_kernel("product_stream_kernel", product_stream_kernel<KIND, GROUPED, 8>, grid, dim3(512), 0, s, a, plan.tile);
    default: return launch_kernel("product_stream_kernel", product_stream_kernel<KIND, GROUPED, 4>, grid, dim3(256), 0, s, a, plan.tile);
  }
}

}  // namespace

int launch_fp8_dense(const ProductArgs &a, void *stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const fp8::DensePlan plan = fp8::dense_plan(a.rows, a.n, a.k_bytes, a.y_bf16);
  if (plan.stream) return launch_stream<kExact, false>(a, s);
  const int rc = a.y_bf16 ? launch_tiles<kNative, false>(plan.tile, a, s) : launch_tiles<kExact, false>(plan.tile, a, s);
  if (rc || a.splits == 1) return rc;
  const unsigned grid = (unsigned)(((size_t)a.rows * a.n + 255) / 256);
  return launch_kernel("product_sum_kernel", product_sum_kernel, dim3(grid), dim3(256), 0, s,
                       static_cast<const float *>(a.part), a);
}

int launch_fp8_grouped(const ProductArgs &a, void *stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const fp8::GroupedPlan plan = fp8::grouped_plan(a.rows, a.n_experts);
  if (plan.stream) return launch_stream<kExact, true>(a, s);
  return a.y_bf16 ? launch_tiles<kNative, true>(plan.tile, a, s) : launch_tiles<kExact, true>(plan.tile, a, s);
}

int launch_bf16_grouped(const ProductArgs &a, void *stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const fp8::GroupedPlan plan = fp8::grouped_plan(a.rows, a.n_experts);
  return plan.stream ? launch_stream<kBf16, true>(a, s) : launch_tiles<kBf16, true>(plan.tile, a, s);
}

}  // namespace qmv
