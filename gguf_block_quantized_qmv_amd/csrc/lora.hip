// Low-rank adapters of many requests beside a shared projection; gfx950 matrix
// cores.
//
//   y[r] = base[r] + B_e h[r],  h[r] = scale_e A_e x[r]
//
// by two launches over tiles of one adapter's rows. The first takes A as the A
// operand of v_mfma_f32_16x16x32_bf16 and x as its B operand, cuts k into parts
// for workgroups and those into blocks of 64 for their four waves, and leaves
// fp32 sums by part. The second adds the parts, scales them and multiplies by B.
//
// h keeps its 24 bits through the matrix cores: cut into three bf16 values of
// eight bits each, hi + mid + lo == h, three instructions for one. The products
// are exact in fp32, so y loses what fp32 additions lose.
#include "qmv_device.h"
#include "rows_internal.h"
#include "rows_layout.h"
#include "../../include/qmm_rows.h"

namespace qmv {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr v4f kZero4 = {0.0f, 0.0f, 0.0f, 0.0f};
constexpr u4 kNone = {0, 0, 0, 0};

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

__device__ __forceinline__ v4f mma(u4 a, u4 b, v4f d) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), d, 0, 0, 0);
}

__device__ __forceinline__ void run_of(const LoraArgs &p, int e, int &begin, int &end) {
  begin = clampi(p.offsets[e], 0, p.rows);
  end = clampi(p.offsets[e + 1], begin, p.rows);
}

// Rows m0 .. end - 1 of one adapter's run, its rank.
struct Run {
  int e, m0, end, rank;
};

// Tile `tile` of `size` rows: every wave scans the runs for itself, 64 lanes by
// n_adapters / 64 of them. False behind the last one.
__device__ __forceinline__ bool find_run(const LoraArgs &p, int tile, int size, Run &t) {
  const int lane = (int)threadIdx.x & 63, per = rows::ceil_div(p.n_adapters, 64);
  int mine = 0;
  for (int e = lane * per; e < lane * per + per && e < p.n_adapters; ++e) {
    int b0, b1;
    run_of(p, e, b0, b1);
    mine += rows::ceil_div(b1 - b0, size);
  }
  int upto = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(upto, d);
    if (lane >= d) upto += o;
  }
  const uint64_t past = __ballot(upto > tile);
  if (past == 0) return false;
  const int owner = uniform(__ffsll((unsigned long long)past) - 1);
  int left = tile - uniform(__shfl(upto - mine, owner)), begin, end;
  int e = owner * per;
  for (;; ++e) {
    run_of(p, e, begin, end);
    const int tiles = rows::ceil_div(end - begin, size);
    if (left < tiles || e + 1 >= p.n_adapters) break;
    left -= tiles;
  }
  t.e = uniform(e);
  t.m0 = uniform(begin + left * size);
  t.end = uniform(end);
  t.rank = uniform(p.ranks ? clampi(p.ranks[e], 0, p.rank) : p.rank);
  return t.m0 < t.end;
}

// Row of x and y behind place r of the runs, -1 where there is none.
__device__ __forceinline__ int row_at(const LoraArgs &p, int r) {
  if (!p.index) return r;
  const int v = p.index[r];
  return (unsigned)v < (unsigned)p.x_rows ? v : -1;
}

// h by part: part[s][r][i]. MT * 16 rows, RT * 16 dimensions.
template <int MT, int RT>
__global__ __launch_bounds__(256) void lora_down_kernel(const LoraArgs p, const int splits) {
  __shared__ v4f sums[4][MT * RT][64];
  Run t;
  if (!find_run(p, (int)blockIdx.x, MT * 16, t) || t.rank == 0) return;
  const int lane = (int)threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), col = lane & 15, group = lane >> 4;
  const uint16_t *x[MT], *a[RT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {   // rows past the end repeat the last one: matrix work, no memory traffic
    const int r = t.m0 + m * 16 + col, from = row_at(p, r < t.end ? r : t.end - 1);
    x[m] = p.x + (size_t)(from < 0 ? 0 : from) * p.k;
  }
#pragma unroll
  for (int c = 0; c < RT; ++c) {
    const int i = c * 16 + col;
    a[c] = p.a + ((size_t)t.e * p.rank + (i < t.rank ? i : t.rank - 1)) * p.k;
  }
  const int blocks = rows::ceil_div(p.k, rows::kKBlock), s = (int)blockIdx.y;
  const int b0 = (int)((int64_t)blocks * s / splits), b1 = (int)((int64_t)blocks * (s + 1) / splits);
  v4f acc[MT][RT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int c = 0; c < RT; ++c) acc[m][c] = kZero4;
  for (int b = b0 + wave; b < b1; b += 4) {
    u4 fx[2][MT], fa[2][RT];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = b * rows::kKBlock + h * 32 + group * 8;
      const bool in = at < p.k;   // k is a multiple of 8
#pragma unroll
      for (int m = 0; m < MT; ++m) fx[h][m] = in ? *reinterpret_cast<const u4 *>(x[m] + at) : kNone;
#pragma unroll
      for (int c = 0; c < RT; ++c) fa[h][c] = in ? *reinterpret_cast<const u4 *>(a[c] + at) : kNone;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int c = 0; c < RT; ++c) acc[m][c] = mma(fa[h][c], fx[h][m], acc[m][c]);
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int c = 0; c < RT; ++c) sums[wave][m * RT + c][lane] = acc[m][c];
  __syncthreads();
  for (int i = wave; i < MT * RT; i += 4) {
    const int r = t.m0 + i / RT * 16 + col, at = i % RT * 16 + group * 4;
    if (r < t.end && at < p.rank)   // the rank is a multiple of 8: four dimensions are all in or all out
      *reinterpret_cast<v4f *>(p.part + ((size_t)s * p.rows + r) * p.rank + at) =
          (sums[0][i][lane] + sums[1][i][lane]) + (sums[2][i][lane] + sums[3][i][lane]);
  }
}

// The upper eight significant bits of v, which is left with the rest (exact).
// What is not finite goes whole, and nothing is left.
__device__ __forceinline__ uint32_t take_bf16(float &v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  if ((u & 0x7F800000u) == 0x7F800000u) {
    v = 0.0f;
    return u & 0x007FFFFFu ? 0x7FC0u : u >> 16;
  }
  v -= __builtin_bit_cast(float, u & 0xFFFF0000u);
  return u >> 16;
}

// y of MT * 16 rows by `columns` columns: a wave takes 64 of them at a time. The
// rows of B stand in its four fragments so that a lane's 16 results are 16
// neighbouring columns of one row: fragment f's row i is column
// 16 (i / 4) + 4 f + i % 4.
template <int MT, bool F32>
__global__ __launch_bounds__(256) void lora_up_kernel(const LoraArgs p, const int splits, const int columns) {
  extern __shared__ uint16_t parts[];   // [3][MT * 16][pitch]
  Run t;
  if (!find_run(p, (int)blockIdx.x, MT * 16, t)) return;
  const int lane = (int)threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), col = lane & 15, group = lane >> 4;
  const int steps = rows::ceil_div(t.rank, 32), pitch = rows::ceil_div(p.rank, 32) * 32 + 8;
  const float scale = p.scale ? p.scale[t.e] : 1.0f;
  const int quads = steps * 8;   // of dimensions in a row
  for (int i = (int)threadIdx.x; i < MT * 16 * quads; i += 256) {
    const int r = i / quads, at = (i - r * quads) * 4;
    v4f h = kZero4;
    if (t.m0 + r < t.end && at < t.rank)
      for (int s = 0; s < splits; ++s)
        h += *reinterpret_cast<const v4f *>(p.part + ((size_t)s * p.rows + t.m0 + r) * p.rank + at);
    uint32_t cut[3][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float v = at + e < t.rank ? scale * h[e] : 0.0f;
#pragma unroll
      for (int q = 0; q < 3; ++q) cut[q][e] = take_bf16(v);
    }
#pragma unroll
    for (int q = 0; q < 3; ++q)
      *reinterpret_cast<uint2 *>(parts + (q * MT * 16 + r) * pitch + at) =
          make_uint2(cut[q][0] | cut[q][1] << 16, cut[q][2] | cut[q][3] << 16);
  }
  __syncthreads();
  int to[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int r = t.m0 + m * 16 + col;
    to[m] = r < t.end ? row_at(p, r) : -1;
  }
  const uint16_t *b = p.b + (size_t)t.e * p.n * p.rank;
  const int first = (int)blockIdx.y * columns, last = first + columns < p.n ? first + columns : p.n;
  for (int n0 = first + wave * 64; n0 < last; n0 += 256) {
    v4f acc[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int f = 0; f < 4; ++f) acc[m][f] = kZero4;
    for (int k = 0; k < steps; ++k) {
      const int at = k * 32 + group * 8;
      u4 fb[4];
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const int n = n0 + (col >> 2) * 16 + f * 4 + (col & 3);
        fb[f] = at < t.rank ? *reinterpret_cast<const u4 *>(b + (size_t)(n < p.n ? n : p.n - 1) * p.rank + at) : kNone;
#pragma unroll
        for (int d = 0; d < 4; ++d) {   // columns of B behind the adapter's own rank may hold anything
          const int own = t.rank - at - 2 * d;
          fb[f][d] &= own >= 2 ? 0xFFFFFFFFu : own == 1 ? 0xFFFFu : 0u;
        }
      }
#pragma unroll
      for (int q = 2; q >= 0; --q)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const u4 fh = *reinterpret_cast<const u4 *>(parts + (q * MT * 16 + m * 16 + col) * pitch + at);
#pragma unroll
          for (int f = 0; f < 4; ++f) acc[m][f] = mma(fb[f], fh, acc[m][f]);
        }
    }
    const int c0 = n0 + group * 16;
    typedef float RowF32 __attribute__((ext_vector_type(4), aligned(4)));
    typedef __bf16 RowBf16 __attribute__((ext_vector_type(8), aligned(2)));
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (to[m] < 0) continue;
      const size_t place = (size_t)to[m] * p.n + c0;
      if (c0 + 16 <= p.n) {
        if constexpr (F32) {
          const float *from = static_cast<const float *>(p.base) + place;
          float *y = static_cast<float *>(p.y) + place;
          RowF32 v[4];
#pragma unroll
          for (int f = 0; f < 4; ++f) v[f] = *reinterpret_cast<const RowF32 *>(from + f * 4);
#pragma unroll
          for (int f = 0; f < 4; ++f) *reinterpret_cast<RowF32 *>(y + f * 4) = v[f] + (RowF32)acc[m][f];
        } else {
          const __bf16 *from = static_cast<const __bf16 *>(p.base) + place;
          __bf16 *y = static_cast<__bf16 *>(p.y) + place;
          RowBf16 v[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) v[h] = *reinterpret_cast<const RowBf16 *>(from + h * 8);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[h][e] = (__bf16)((float)v[h][e] + acc[m][h * 2 + e / 4][e % 4]);
            *reinterpret_cast<RowBf16 *>(y + h * 8) = v[h];
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (c0 + e < p.n) {
            if constexpr (F32)
              static_cast<float *>(p.y)[place + e] = static_cast<const float *>(p.base)[place + e] + acc[m][e / 4][e % 4];
            else
              static_cast<__bf16 *>(p.y)[place + e] =
                  (__bf16)((float)static_cast<const __bf16 *>(p.base)[place + e] + acc[m][e / 4][e % 4]);
          }
      }
    }
  }
}

template <int MT, int RT>
int down(const LoraArgs &a, const rows::LoraPlan &plan, hipStream_t s) {
  return launch_kernel("lora_down_kernel", lora_down_kernel<MT, RT>,
                       dim3((unsigned)rows::lora_tiles(a.rows, a.n_adapters, MT * 16), (unsigned)plan.splits), dim3(256), 0,
                       s, a, plan.splits);
}

template <int MT>
int both(const LoraArgs &a, const rows::LoraPlan &plan, hipStream_t s) {
  int rc;
  if (a.rank <= 16) rc = down<MT, 1>(a, plan, s);
  else if (a.rank <= 32) rc = down<MT, 2>(a, plan, s);
  else if constexpr (MT == 4) rc = down<MT, 4>(a, plan, s);   // the plan takes these tiles up to rank 64
  else rc = a.rank <= 64 ? down<MT, 4>(a, plan, s) : down<MT, 8>(a, plan, s);
  if (rc) return rc;
  const dim3 grid((unsigned)rows::lora_tiles(a.rows, a.n_adapters, MT * 16), (unsigned)rows::ceil_div(a.n, plan.columns));
  const size_t lds = (size_t)3 * MT * 16 * (rows::ceil_div(a.rank, 32) * 32 + 8) * 2;
  return a.y_f32 ? launch_kernel("lora_up_kernel", lora_up_kernel<MT, true>, grid, dim3(256), lds, s, a, plan.splits, plan.columns)
                 : launch_kernel("lora_up_kernel", lora_up_kernel<MT, false>, grid, dim3(256), lds, s, a, plan.splits, plan.columns);
}

}  // namespace

int launch_lora(const LoraArgs &a, void *stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const rows::LoraPlan plan = rows::lora_plan(a.rows, a.n, a.k, a.rank, a.n_adapters);
  return plan.tile == 16 ? both<1>(a, plan, s) : plan.tile == 32 ? both<2>(a, plan, s) : both<4>(a, plan, s);
}

}  // namespace qmv
