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
#include "rows_device.h"
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

// Rows m0 .. end - 1 of adapter e's run, its rank and scale, and this workgroup's
// part of k or of the columns.
struct Run {
  int e, m0, end, rank, part;
  float scale;
};

// This workgroup's tile of `size` rows and its part: every wave scans the runs for
// itself, lane i the runs of n_adapters / 64 neighbouring adapters from i of those
// on. What a lane has read of its first adapter goes to the others from its
// registers, so up to 64 adapters cost one trip to memory. Workgroups are dealt to
// the eight XCDs in turn and the grid is a multiple of eight wide: with LONG runs
// each XCD gets one contiguous run of the tiles, for few adapters in its cache, and
// without, adapters of any rank are spread over all. False behind the last tile.
template <bool LONG>
__device__ __forceinline__ bool find_run(const LoraArgs &p, int size, Run &t) {
  const int lane = (int)threadIdx.x & 63, per = rows::ceil_div(p.n_adapters, 64), e0 = lane * per;
  int begin = 0, end = 0, rank = p.rank, mine = 0;
  float scale = 1.0f;
  if (e0 < p.n_adapters) {
    run_of(p, e0, begin, end);
    if (p.ranks) rank = p.ranks[e0];
    if (p.scale) scale = p.scale[e0];
    mine = rows::ceil_div(end - begin, size);
  }
  for (int e = e0 + 1; e < e0 + per && e < p.n_adapters; ++e) {
    int b0, b1;
    run_of(p, e, b0, b1);
    mine += rows::ceil_div(b1 - b0, size);
  }
  const int upto = wave_upto(mine);
  int tile = (int)blockIdx.x;
  const int tiles = __builtin_amdgcn_readlane(upto, 63);
  if constexpr (LONG) {
    const int share = tiles >> 3, spare = tiles & 7, xcd = tile & 7, at = tile >> 3;
    if (at >= share + (xcd < spare)) return false;
    tile = xcd * share + (xcd < spare ? xcd : spare) + at;
  } else if (tile >= tiles) {
    return false;
  }
  t.part = (int)blockIdx.y;
  const uint64_t past = __ballot(upto > tile);
  const int owner = uniform(__ffsll((unsigned long long)past) - 1);
  int left = tile - __builtin_amdgcn_readlane(upto - mine, owner);
  t.e = owner * per;
  begin = __builtin_amdgcn_readlane(begin, owner);
  end = __builtin_amdgcn_readlane(end, owner);
  rank = __builtin_amdgcn_readlane(rank, owner);
  scale = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, scale), owner));
  while (left >= rows::ceil_div(end - begin, size) && t.e + 1 < owner * per + per && t.e + 1 < p.n_adapters) {
    left -= rows::ceil_div(end - begin, size);
    ++t.e;
    run_of(p, t.e, begin, end);
    if (p.ranks) rank = p.ranks[t.e];
    if (p.scale) scale = p.scale[t.e];
  }
  t.e = uniform(t.e);
  t.m0 = uniform(begin + left * size);
  t.end = uniform(end);
  t.rank = uniform(clampi(rank, 0, p.rank));
  t.scale = scale;
  return t.m0 < t.end;
}

// Row of x and y behind place r of the runs, -1 where there is none.
__device__ __forceinline__ int row_at(const LoraArgs &p, int r) {
  if (!p.index) return r;
  const int v = p.index[r];
  return (unsigned)v < (unsigned)p.x_rows ? v : -1;
}

// h by part: part[s][r][i], of MT * 16 rows and RT * 16 dimensions.
//
// A fragment of a matrix instruction takes a row a lane, and 64 lanes of 16 bytes
// in 16 rows cost the address unit 64 cycles instead of 16. So a wave loads whole
// lines, eight lanes a row, a block of k ahead, and takes the fragments from a
// buffer of its own in LDS. Slots of 16 bytes are swapped by the lower bits of
// their row, so that eight lanes never meet in a bank.
template <int MT, int RT>
__global__ __launch_bounds__(256) void lora_down_kernel(const LoraArgs p, const int splits) {
  constexpr int kLines = (MT + RT) * 2;   // loads of a block, of 8 rows by 128 bytes
  __shared__ u4 slots[4][(MT * RT > kLines ? MT * RT : kLines) * 64];   // a block of k, and in the end the wave's sums
  Run t;
  if (!find_run<(MT > 1)>(p, MT * 16, t) || t.rank == 0) return;
  const int lane = (int)threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), col = lane & 15, group = lane >> 4;
  const int line = lane >> 3, chunk = lane & 7;
  u4 *const mine = slots[wave];
  const uint16_t *from[kLines];
#pragma unroll
  for (int i = 0; i < kLines; ++i) {   // rows past the end repeat the last one: matrix work, no memory traffic
    if (i < MT * 2) {
      const int r = t.m0 + i * 8 + line, row = row_at(p, r < t.end ? r : t.end - 1);
      from[i] = p.x + (size_t)(row < 0 ? 0 : row) * p.k + chunk * 8;
    } else {
      const int r = (i - MT * 2) * 8 + line;
      from[i] = p.a + ((size_t)t.e * p.rank + (r < t.rank ? r : t.rank - 1)) * p.k + chunk * 8;
    }
  }
  const int blocks = rows::ceil_div(p.k, rows::kKBlock), s = t.part;
  const int b0 = (int)((int64_t)blocks * s / splits), b1 = (int)((int64_t)blocks * (s + 1) / splits);
  u4 f[kLines];
  auto fetch = [&](int b) {
    const int k0 = b * rows::kKBlock;
    const bool in = k0 + chunk * 8 < p.k;   // k is a multiple of 8
#pragma unroll
    for (int i = 0; i < kLines; ++i) f[i] = in ? *reinterpret_cast<const u4 *>(from[i] + k0) : kNone;
  };
  v4f acc[MT][RT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int c = 0; c < RT; ++c) acc[m][c] = kZero4;
  if (b0 + wave < b1) fetch(b0 + wave);
  for (int b = b0 + wave; b < b1; b += 4) {
#pragma unroll
    for (int i = 0; i < kLines; ++i) mine[(i * 8 + line) * 8 + (chunk ^ line)] = f[i];
    in_order();
    if (b + 4 < b1) fetch(b + 4);
    auto fragment = [&](int r, int h) {   // rows 16 r .., values 32 h ..
      return mine[(r * 16 + col) * 8 + ((h * 4 + group) ^ (col & 7))];
    };
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      u4 fx[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) fx[m] = fragment(m, h);
#pragma unroll
      for (int c = 0; c < RT; ++c) {
        const u4 fa = fragment(MT + c, h);
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[m][c] = mma(fa, fx[m], acc[m][c]);
      }
    }
    in_order();
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int c = 0; c < RT; ++c) mine[(m * RT + c) * 64 + lane] = __builtin_bit_cast(u4, acc[m][c]);
  __syncthreads();
  for (int i = wave; i < MT * RT; i += 4) {
    const int r = t.m0 + i / RT * 16 + col, at = i % RT * 16 + group * 4;
    if (r < t.end && at < p.rank) {   // the rank is a multiple of 8: four dimensions are all in or all out
      v4f v[4];
#pragma unroll
      for (int w = 0; w < 4; ++w) v[w] = __builtin_bit_cast(v4f, slots[w][i * 64 + lane]);
      *reinterpret_cast<v4f *>(p.part + ((size_t)s * p.rows + r) * p.rank + at) = (v[0] + v[1]) + (v[2] + v[3]);
    }
  }
}

// v as three bf16 values of eight significant bits each that add up to it exactly.
// What is not finite goes whole into the first.
__device__ __forceinline__ void cut_in_three(float v, uint32_t (&out)[3]) {
  const bool finite = (__builtin_bit_cast(uint32_t, v) & 0x7F800000u) != 0x7F800000u;
  const __bf16 whole = (__bf16)v;
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v) & 0xFFFF0000u;
    out[q] = finite ? u >> 16 : 0u;
    v -= __builtin_bit_cast(float, u);
  }
  if (!finite) out[0] = __builtin_bit_cast(uint16_t, whole);   // a NaN stays one
}

// y of MT * 16 rows by `columns` columns, STEPS of 32 dimensions: a wave takes 64
// columns at a time. B comes as A does above, and the results go through the same
// buffer on their way to y. What a pass needs from memory is sent before the last
// one's, or the parts of h, are waited for. FAR: base and y past the caches.
template <int MT, int STEPS, bool F32, bool FAR>
__global__ __launch_bounds__(256) void lora_up_kernel(const LoraArgs p, const int splits, const int columns,
                                                      const int inverse) {
  constexpr int kPitch = STEPS * 32 + 8, kWide = STEPS * 4;   // kWide: slots of a row of B
  constexpr int kSize = F32 ? 4 : 2, kPer = F32 ? 4 : 8;   // values of a load or store of y
  // of 16 rows: kOut loads, each of kOutRows rows by kOutLanes lanes
  constexpr int kOut = F32 ? 4 : 2, kOutRows = 16 / kOut, kOutLanes = 64 / kOutRows;
  __shared__ u4 slots[4][64 * kWide];   // 64 rows of B, then 16 x 64 results at a time
  __shared__ __attribute__((aligned(16))) uint16_t parts[3][MT * 16][kPitch];
  Run t;
  if (!find_run<(MT > 1)>(p, MT * 16, t)) return;
  const int lane = (int)threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), col = lane & 15, group = lane >> 4;
  u4 *const mine = slots[wave];
  // 64 rows of B are `chunks` whole instructions, one after the other in memory. A column's chunk c goes to slot c of row
  // 16 f + 4 a + b for column 16 a + 4 f + b, so that a lane's results of fragment f are neighbours of those of f + 1;
  // slots behind B's row, or the adapter's own rank, get zeros: `own` of a chunk's values are its.
  const int chunks = p.rank >> 3;   // q * inverse >> 16 == q / chunks for q < 1024
  int put[kWide];   // the slot, and from bit 16 on `own`
#pragma unroll
  for (int j = 0; j < kWide; ++j) {
    const int q = j * 64 + lane, n = j < chunks ? q * inverse >> 16 : lane, c = j < chunks ? q - n * chunks : j;
    const int row = (n >> 2 & 3) * 16 + (n >> 4) * 4 + (n & 3), own = clampi(t.rank - c * 8, 0, 8);
    put[j] = (row * kWide + (c ^ (kWide == 4 ? row >> 2 & 3 : row & 7))) | own << 16;
  }
  int to[MT * kOut];
#pragma unroll
  for (int i = 0; i < MT * kOut; ++i) {
    const int r = t.m0 + i * kOutRows + lane / kOutLanes;
    to[i] = r < t.end ? row_at(p, r) : -1;
  }
  typedef uint32_t RowVec __attribute__((ext_vector_type(4), aligned(2)));
  const int part = lane % kOutLanes * kPer;   // of a pass's columns
  const int first = t.part * columns, last = first + columns < p.n ? first + columns : p.n;
  const u4 *bank = reinterpret_cast<const u4 *>(p.b + (size_t)t.e * p.n * p.rank);
  u4 fb[kWide];
  RowVec base[MT * kOut];
  auto send = [&](int n0) {
    const size_t here = (size_t)n0 * chunks + lane, all = (size_t)p.n * chunks;
#pragma unroll
    for (int j = 0; j < kWide; ++j) fb[j] = put[j] >> 16 && here + j * 64 < all ? bank[here + j * 64] : kNone;
    if (n0 + part + kPer <= p.n)
#pragma unroll
      for (int i = 0; i < MT * kOut; ++i)
        if (to[i] >= 0) {
          const RowVec *at = reinterpret_cast<const RowVec *>(static_cast<const char *>(p.base) +
                                                              ((size_t)to[i] * p.n + n0 + part) * kSize);
          if constexpr (FAR) base[i] = __builtin_nontemporal_load(at);
          else base[i] = *at;
        }
  };
  int n0 = first + wave * 64;
  if (n0 < last) send(n0);

  constexpr int kQuads = MT * 16 * STEPS * 8, kTurns = (kQuads + 255) / 256;
  constexpr int kGroup = kTurns == 1 ? 8 : 4;   // parts whose loads are sent together
  v4f hs[kTurns];
#pragma unroll
  for (int i = 0; i < kTurns; ++i) hs[i] = kZero4;
  for (int s0 = 0; s0 < splits; s0 += kGroup) {
    v4f v[kTurns][kGroup];
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
      const int q = i * 256 + (int)threadIdx.x, r = q / (STEPS * 8), at = q % (STEPS * 8) * 4;
      const bool in = q < kQuads && t.m0 + r < t.end && at < t.rank;
      const float *from = p.part + ((size_t)s0 * p.rows + t.m0 + r) * p.rank + at;
#pragma unroll
      for (int s = 0; s < kGroup; ++s)
        v[i][s] = in && s0 + s < splits ? *reinterpret_cast<const v4f *>(from + (size_t)s * p.rows * p.rank) : kZero4;
    }
#pragma unroll
    for (int i = 0; i < kTurns; ++i)
#pragma unroll
      for (int s = 0; s < kGroup; ++s) hs[i] += v[i][s];
  }
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const int q = i * 256 + (int)threadIdx.x, r = q / (STEPS * 8), at = q % (STEPS * 8) * 4;
    if (q >= kQuads) break;
    uint32_t cut[4][3];
#pragma unroll
    for (int e = 0; e < 4; ++e) cut_in_three(at + e < t.rank ? t.scale * hs[i][e] : 0.0f, cut[e]);
#pragma unroll
    for (int c = 0; c < 3; ++c)
      *reinterpret_cast<uint2 *>(&parts[c][r][at]) = make_uint2(cut[0][c] | cut[1][c] << 16, cut[2][c] | cut[3][c] << 16);
  }
  __syncthreads();

  for (; n0 < last; n0 += 256) {
#pragma unroll
    for (int j = 0; j < kWide; ++j) {
      if (t.rank & 7) {   // what lies behind the adapter's own rank may be anything
        const int own = put[j] >> 16;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (own < e * 2 + 2) fb[j][e] = own == e * 2 + 1 ? fb[j][e] & 0xFFFFu : 0u;
      }
      mine[put[j] & 0xFFFF] = fb[j];
    }
    in_order();
    RowVec was[MT * kOut];
#pragma unroll
    for (int i = 0; i < MT * kOut; ++i) was[i] = base[i];
    if (n0 + 256 < last) send(n0 + 256);
    v4f acc[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int f = 0; f < 4; ++f) acc[m][f] = kZero4;
    const int swap = kWide == 4 ? col >> 2 & 3 : col & 7;
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
      u4 w[4];
#pragma unroll
      for (int f = 0; f < 4; ++f) w[f] = mine[(f * 16 + col) * kWide + ((k * 4 + group) ^ swap)];
#pragma unroll
      for (int c = 2; c >= 0; --c)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const u4 h = *reinterpret_cast<const u4 *>(&parts[c][m * 16 + col][k * 32 + group * 8]);
#pragma unroll
          for (int f = 0; f < 4; ++f) acc[m][f] = mma(w[f], h, acc[m][f]);
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      in_order();
#pragma unroll
      for (int f = 0; f < 4; ++f) mine[col * 16 + ((group * 4 + f) ^ (col & 7))] = __builtin_bit_cast(u4, acc[m][f]);
      in_order();
#pragma unroll
      for (int i = 0; i < kOut; ++i) {
        const int r = i * kOutRows + lane / kOutLanes, row = to[m * kOut + i], c0 = n0 + part, s = part / 4;
        const v4f lo = __builtin_bit_cast(v4f, mine[r * 16 + (s ^ (r & 7))]);
        v4f hi = kZero4;
        if constexpr (!F32) hi = __builtin_bit_cast(v4f, mine[r * 16 + ((s + 1) ^ (r & 7))]);
        if (row < 0) continue;
        const size_t place = (size_t)row * p.n + c0;
        if (c0 + kPer <= p.n) {
          RowVec o;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t u = was[m * kOut + i][e];
            if constexpr (F32) {
              o[e] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, u) + lo[e]);
            } else {
              const v4f v = e < 2 ? lo : hi;
              const bf16x2 pair = {(__bf16)(__builtin_bit_cast(float, u << 16) + v[e % 2 * 2]),
                                   (__bf16)(__builtin_bit_cast(float, u & 0xFFFF0000u) + v[e % 2 * 2 + 1])};
              o[e] = __builtin_bit_cast(uint32_t, pair);
            }
          }
          RowVec *at = reinterpret_cast<RowVec *>(static_cast<char *>(p.y) + place * kSize);
          if constexpr (FAR) __builtin_nontemporal_store(o, at);
          else *at = o;
        } else {
#pragma unroll 1
          for (int e = 0; e < kPer && c0 + e < p.n; ++e) {
            const v4f from = e < 4 ? lo : hi;
            const float v = e % 4 < 2 ? (e % 2 ? from[1] : from[0]) : e % 2 ? from[3] : from[2];
            if constexpr (F32)
              static_cast<float *>(p.y)[place + e] = static_cast<const float *>(p.base)[place + e] + v;
            else
              static_cast<__bf16 *>(p.y)[place + e] = (__bf16)((float)static_cast<const __bf16 *>(p.base)[place + e] + v);
          }
        }
      }
    }
    in_order();
  }
}

template <int MT>
unsigned grid_of(const LoraArgs &a) {
  const unsigned tiles = (unsigned)rows::lora_tiles(a.rows, a.n_adapters, MT * 16);
  return MT > 1 ? (tiles + 7) / 8 * 8 : tiles;
}

template <int MT, int RT>
int down(const LoraArgs &a, const rows::LoraPlan &plan, hipStream_t s) {
  return launch_kernel("lora_down_kernel", lora_down_kernel<MT, RT>, dim3(grid_of<MT>(a), (unsigned)plan.splits), dim3(256), 0,
                       s, a, plan.splits);
}

template <int MT, int STEPS>
int up(const LoraArgs &a, const rows::LoraPlan &plan, hipStream_t s) {
  return launch_kernel("lora_up_kernel",
                       plan.far ? (a.y_f32 ? lora_up_kernel<MT, STEPS, true, true> : lora_up_kernel<MT, STEPS, false, true>)
                                : (a.y_f32 ? lora_up_kernel<MT, STEPS, true, false> : lora_up_kernel<MT, STEPS, false, false>),
                       dim3(grid_of<MT>(a), (unsigned)rows::ceil_div(a.n, plan.columns)), dim3(256), 0, s, a, plan.splits,
                       plan.columns, 65536 / (a.rank >> 3) + 1);
}

template <int MT>
int both(const LoraArgs &a, const rows::LoraPlan &plan, hipStream_t s) {
  const int rc = a.rank <= 16   ? down<MT, 1>(a, plan, s)
                 : a.rank <= 32 ? down<MT, 2>(a, plan, s)
                 : a.rank <= 64 ? down<MT, 4>(a, plan, s)
                                : down<MT, 8>(a, plan, s);
  if (rc) return rc;
  return a.rank <= 32 ? up<MT, 1>(a, plan, s) : a.rank <= 64 ? up<MT, 2>(a, plan, s) : up<MT, 4>(a, plan, s);
}

}  // namespace

int launch_lora(const LoraArgs &a, void *stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const rows::LoraPlan plan = rows::lora_plan(a.rows, a.n, a.k, a.rank, a.n_adapters, a.x_rows, a.y_f32);
  return plan.tile == 32 ? both<2>(a, plan, s) : both<1>(a, plan, s);
}

}  // namespace qmv
