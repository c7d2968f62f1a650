// Low-rank adapters of many requests beside a shared projection; gfx950 matrix
// cores.
//
//   y[r] = base[r] + B_e h[r],  h[r] = scale_e A_e x[r]
//
// by two launches over tiles of one adapter's rows. The first takes A as the A
// operand of v_mfma_f32_16x16x32_bf16 and x as its B operand, cuts k into parts
// for workgroups and those into blocks of 64 for their four waves, and leaves
// fp32 sums by part. The second adds the parts, scales them and multiplies by B.
// With a small A and workgroups that should have a CU each both are one launch (lora_plan).
//
// h keeps its 24 bits through the matrix cores: cut into three bf16 values of
// eight bits each, hi + mid + lo == h but for bits below 2^-133, the smallest bf16
// value, three instructions for one. The products are exact in fp32, so y loses
// what fp32 additions lose.
//
// What bounds it. Few rows: a launch and trips to memory one behind the other, the
// run's offsets, its index, A and x, then B (one row, rank 16, 5120 x 5120: 8.8 us in
// a graph of many calls, 10.1 launched from the host; 64 rows of 24 adapters, rank 32, k 5120,
// 17408 columns: 5.1 and 9.4 us, where a large copy would take 4.6 for the bytes). Long runs: the L2, of which a CU
// gets some 24 bytes a cycle, since each tile of 32 rows reads all of A and B (4096
// rows of 5 adapters, rank 64, 5120 x 5120, bf16: 13.5 and 24.3 us, 42 MB read and
// 84 MB read and written, 3.1 and 3.5 TB/s of a large copy's 5.2; the products alone
// would be 2 and 7 us at a large library product's rate). Both products of 16 rows in
// one workgroup read A and B twice as often and took 51 us; tiles of 64 rows, with
// A and B through registers as here, gained nothing over 32.
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

// The first product over blocks b0 .. b1 - 1 of k, for one wave of NW: its share of
// A x for MT * 16 rows and RT * 16 dimensions.
//
// A fragment of a matrix instruction takes a row a lane, and 64 lanes of 16 bytes
// in 16 rows cost the address unit 64 cycles instead of 16. So a wave loads whole
// lines, eight lanes a row, AHEAD blocks of k ahead, and takes the fragments from a
// buffer of its own in LDS (`mine`, kSlots). Slots of 16 bytes are swapped by the
// lower bits of their row, so that eight lanes never meet in a bank.
template <int MT, int RT, int NW, int AHEAD>
struct Down {
  static constexpr int kLines = (MT + RT) * 2;   // loads of a block, of 8 rows by 128 bytes
  static constexpr int kSlots = kLines * 64;
  v4f acc[MT][RT];

  __device__ __forceinline__ Down(const LoraArgs &p, const Run &t, int b0, int b1, u4 *mine) {
    const int lane = (int)threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), col = lane & 15, group = lane >> 4;
    const int line = lane >> 3, chunk = lane & 7;
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
    u4 f[AHEAD][kLines];
    auto fetch = [&](u4(&f)[kLines], int b) {
      const int k0 = b * rows::kKBlock;
      const bool in = k0 + chunk * 8 < p.k;   // k is a multiple of 8
#pragma unroll
      for (int i = 0; i < kLines; ++i) f[i] = in ? *reinterpret_cast<const u4 *>(from[i] + k0) : kNone;
    };
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int c = 0; c < RT; ++c) acc[m][c] = kZero4;
#pragma unroll
    for (int n = 0; n < AHEAD; ++n)
      if (b0 + wave + n * NW < b1) fetch(f[n], b0 + wave + n * NW);
    for (int at = b0 + wave; at < b1; at += AHEAD * NW)
#pragma unroll
      for (int n = 0; n < AHEAD; ++n) {
        const int b = at + n * NW;
        if (b >= b1) break;
#pragma unroll
        for (int i = 0; i < kLines; ++i) mine[(i * 8 + line) * 8 + (chunk ^ line)] = f[n][i];
        in_order();
        if (b + AHEAD * NW < b1) fetch(f[n], b + AHEAD * NW);
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
  }

  __device__ __forceinline__ void leave(u4 *mine) const {   // MT * RT * 64 slots
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int c = 0; c < RT; ++c) mine[(m * RT + c) * 64 + ((int)threadIdx.x & 63)] = __builtin_bit_cast(u4, acc[m][c]);
  }
};

// v as three bf16 values of eight significant bits each that add up to it exactly,
// but for bits below 2^-133. What is not finite goes whole into the first.
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

// h = scale times four dimensions from `at` on, of the adapter's own rank, in three parts.
template <class ROWS>
__device__ __forceinline__ void put_h(const Run &t, v4f h, int r, int at, ROWS &parts) {
  uint32_t cut[4][3];
#pragma unroll
  for (int e = 0; e < 4; ++e) cut_in_three(at + e < t.rank ? t.scale * h[e] : 0.0f, cut[e]);
#pragma unroll
  for (int c = 0; c < 3; ++c)
    *reinterpret_cast<uint2 *>(&parts[c][r][at]) = make_uint2(cut[0][c] | cut[1][c] << 16, cut[2][c] | cut[3][c] << 16);
}

// The second product, for one wave of NW: y of MT * 16 rows, 64 columns at a time,
// STEPS of 32 dimensions, h in `parts`. B comes as A does above, and the results go
// through the same buffer (kSlots) on their way to y. What a pass needs from memory
// is sent before the last one's, or h, is waited for. FAR: base and y past the caches.
template <int MT, int STEPS, bool F32, bool FAR, int NW>
struct Up {
  static constexpr int kPitch = STEPS * 32 + 8, kWide = STEPS * 4, kSlots = 64 * kWide;   // kWide: slots of a row of B
  static constexpr int kSize = F32 ? 4 : 2, kPer = F32 ? 4 : 8;   // values of a load or store of y
  // of 16 rows: kOut loads, each of kOutRows rows by kOutLanes lanes
  static constexpr int kOut = F32 ? 4 : 2, kOutRows = 16 / kOut, kOutLanes = 64 / kOutRows;
  typedef uint16_t Parts[3][MT * 16][kPitch];
  typedef uint32_t RowVec __attribute__((ext_vector_type(4), aligned(2)));

  const LoraArgs &p;
  const Run &t;
  const u4 *bank;
  int chunks, first, last, part;   // chunks of a row of B; this workgroup's columns; a lane's place in a pass's
  int put[kWide];                  // slots, and from bit 16 on the chunk's values within the adapter's own rank
  int to[MT * kOut];
  u4 fb[kWide];
  RowVec base[MT * kOut];

  // 64 rows of B are `chunks` whole instructions, one after the other in memory. A column's chunk c goes to slot c of row
  // 16 f + 4 a + b for column 16 a + 4 f + b, so that a lane's results of fragment f are neighbours of those of f + 1;
  // slots behind B's row, or the adapter's own rank, get zeros. q * inverse >> 16 == q / chunks for q < 1024.
  __device__ __forceinline__ Up(const LoraArgs &p, const Run &t, int columns, int inverse) : p(p), t(t) {
    const int lane = (int)threadIdx.x & 63;
    chunks = p.rank >> 3;
#pragma unroll
    for (int j = 0; j < kWide; ++j) {
      const int q = j * 64 + lane, n = j < chunks ? q * inverse >> 16 : lane, c = j < chunks ? q - n * chunks : j;
      const int row = (n >> 2 & 3) * 16 + (n >> 4) * 4 + (n & 3), own = clampi(t.rank - c * 8, 0, 8);
      put[j] = (row * kWide + (c ^ (kWide == 4 ? row >> 2 & 3 : row & 7))) | own << 16;
    }
#pragma unroll
    for (int i = 0; i < MT * kOut; ++i) {
      const int r = t.m0 + i * kOutRows + lane / kOutLanes;
      to[i] = r < t.end ? row_at(p, r) : -1;
    }
    part = lane % kOutLanes * kPer;
    first = t.part * columns;
    last = first + columns < p.n ? first + columns : p.n;
    bank = reinterpret_cast<const u4 *>(p.b + (size_t)t.e * p.n * p.rank);
  }

  __device__ __forceinline__ void send(int n0) {
    const size_t here = (size_t)n0 * chunks + ((int)threadIdx.x & 63), all = (size_t)p.n * chunks;
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
  }

  // The wave's first columns are sent already.
  __device__ __forceinline__ void passes(const Parts &parts, u4 *mine) {
    const int lane = (int)threadIdx.x & 63, col = lane & 15, group = lane >> 4;
    const int swap = kWide == 4 ? col >> 2 & 3 : col & 7;
    for (int n0 = first + uniform((int)threadIdx.x >> 6) * 64; n0 < last; n0 += NW * 64) {
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
      if (n0 + NW * 64 < last) send(n0 + NW * 64);
      v4f acc[MT][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int f = 0; f < 4; ++f) acc[m][f] = kZero4;
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
        for (int i = 0; i < kOut; ++i) finish(i, to[m * kOut + i], was[m * kOut + i], n0 + part, mine);
      }
      in_order();
    }
  }

  // Load or store i of 16 rows.
  __device__ __forceinline__ void finish(int i, int row, RowVec was, int c0, const u4 *mine) const {
    const int r = i * kOutRows + ((int)threadIdx.x & 63) / kOutLanes, s = part / 4;
    const v4f lo = __builtin_bit_cast(v4f, mine[r * 16 + (s ^ (r & 7))]);
    v4f hi = kZero4;
    if constexpr (!F32) hi = __builtin_bit_cast(v4f, mine[r * 16 + ((s + 1) ^ (r & 7))]);
    if (row < 0) return;
    const size_t place = (size_t)row * p.n + c0;
    if (c0 + kPer <= p.n) {
      RowVec o;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t u = was[e];
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
};

// The first launch of two: h by part, part[s][r][i], without the scale.
template <int MT, int RT>
__global__ __launch_bounds__(256) void lora_down_kernel(const LoraArgs p, const int splits) {
  typedef Down<MT, RT, 4, 1> D;
  __shared__ u4 slots[4][D::kSlots > MT * RT * 64 ? D::kSlots : MT * RT * 64];   // in the end the wave's sums
  Run t;
  if (!find_run<(MT > 1)>(p, MT * 16, t) || t.rank == 0) return;
  const int lane = (int)threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), col = lane & 15, group = lane >> 4;
  const int blocks = rows::ceil_div(p.k, rows::kKBlock), s = t.part;
  const D d(p, t, (int)((int64_t)blocks * s / splits), (int)((int64_t)blocks * (s + 1) / splits), slots[wave]);
  d.leave(slots[wave]);
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

// The second: adds h's parts, in order, and multiplies by B.
template <int MT, int STEPS, bool F32, bool FAR>
__global__ __launch_bounds__(256) void lora_up_kernel(const LoraArgs p, const int splits, const int columns,
                                                      const int inverse) {
  typedef Up<MT, STEPS, F32, FAR, 4> U;
  __shared__ u4 slots[4][U::kSlots];
  __shared__ __attribute__((aligned(16))) typename U::Parts parts;
  Run t;
  if (!find_run<(MT > 1)>(p, MT * 16, t)) return;
  const int wave = uniform((int)threadIdx.x >> 6);
  U u(p, t, columns, inverse);
  if (u.first + wave * 64 < u.last) u.send(u.first + wave * 64);

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
    const int q = i * 256 + (int)threadIdx.x;
    if (q < kQuads) put_h(t, hs[i], q / (STEPS * 8), q % (STEPS * 8) * 4, parts);
  }
  __syncthreads();
  u.passes(parts, slots[wave]);
}

// Both in one launch, for few tiles of 16 rows and a small A: every workgroup of a
// tile takes all of A x for itself, its 16 waves a share of k each.
template <int RT, bool F32>
__global__ __launch_bounds__(1024) void lora_whole_kernel(const LoraArgs p, const int columns, const int inverse) {
  constexpr int NW = 16;
  typedef Down<1, RT, NW, RT == 1 ? 3 : 2> D;
  typedef Up<1, 1, F32, false, NW> U;
  __shared__ u4 slots[NW][D::kSlots > U::kSlots ? D::kSlots : U::kSlots];
  __shared__ __attribute__((aligned(16))) typename U::Parts parts;
  Run t;
  if (!find_run<false>(p, 16, t)) return;
  const int wave = uniform((int)threadIdx.x >> 6);
  const D d(p, t, 0, t.rank > 0 ? rows::ceil_div(p.k, rows::kKBlock) : 0, slots[wave]);   // no rank: base as it is
  U u(p, t, columns, inverse);
  if (u.first + wave * 64 < u.last) u.send(u.first + wave * 64);
  d.leave(slots[wave]);
  __syncthreads();
  if (threadIdx.x < 128) {   // four dimensions a thread, 32 of them: behind A's are zeros
    const int c = (int)threadIdx.x >> 6, l = (int)threadIdx.x & 63;
    v4f h = kZero4;
    if (c < RT)
#pragma unroll
      for (int w = 0; w < NW; ++w) h += __builtin_bit_cast(v4f, slots[w][c * 64 + l]);
    put_h(t, h, l & 15, c * 16 + (l >> 4) * 4, parts);
  }
  __syncthreads();
  u.passes(parts, slots[wave]);
}

template <int MT>
unsigned grid_of(const LoraArgs &a) {
  const unsigned tiles = (unsigned)rows::lora_tiles(a.rows, a.n_adapters, MT * 16);
  return MT > 1 ? (tiles + 7) / 8 * 8 : tiles;
}

template <int RT>
int whole(const LoraArgs &a, const rows::LoraPlan &plan, hipStream_t s) {
  return launch_kernel("lora_whole_kernel", a.y_f32 ? lora_whole_kernel<RT, true> : lora_whole_kernel<RT, false>,
                       dim3(grid_of<1>(a), (unsigned)rows::ceil_div(a.n, plan.columns)), dim3(1024), 0, s, a, plan.columns,
                       65536 / (a.rank >> 3) + 1);
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
  if (plan.splits == 0) return a.rank <= 16 ? whole<1>(a, plan, s) : whole<2>(a, plan, s);
  return plan.tile == 32 ? both<2>(a, plan, s) : both<1>(a, plan, s);
}

}  // namespace qmv
