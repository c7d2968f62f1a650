// Rows spread to the places of their choices, summed back with weights, and the
// gradient of that; gfx950.
//
// All three are bound by memory: a row is read or written in pieces of 16 bytes,
// one a lane, every byte once. Rows of any length and start are taken by the
// same 16-byte instructions (the machine allows them at any address of the
// element's own alignment), the last piece of a row by elements. A thread keeps one
// piece of a token for all its choices, so x is read once for top_k rows written,
// and what a sum or a gradient needs of a token stays in registers.
//
// Rows of 2048 bf16, top 8: 8192 tokens spread 53 us (302 MB, 5.7 TB/s) and summed
// back 51.5 us (302 MB, 5.9 TB/s), the gradient of 4096 tokens 55.5 us (285 MB, 5.1
// TB/s); a large copy reaches 5.2 TB/s, a fill 6.8. Four tokens: 3 us, a launch.
#include "qmv_device.h"
#include "rows_internal.h"
#include "rows_layout.h"

namespace qmv {
namespace {

// 16 bytes at the alignment A of an element or of a whole piece.
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef uint32_t u4_at4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u4_at2 __attribute__((ext_vector_type(4), aligned(2)));
template <int A>
struct Piece {
  typedef u4 type;
};
template <>
struct Piece<4> {
  typedef u4_at4 type;
};
template <>
struct Piece<2> {
  typedef u4_at2 type;
};

// Values of one piece.
template <bool F32>
constexpr int kValues = F32 ? 4 : 8;

// Piece c of a row of `width` values; behind the end: zeros. FAR (whole pieces):
// past the caches.
template <bool F32, int A, bool FAR = false>
__device__ __forceinline__ u4 load_piece(const void *rows, size_t row, int c, int width) {
  constexpr int V = kValues<F32>;
  const char *at = static_cast<const char *>(rows) + (row * width + (size_t)c * V) * (F32 ? 4 : 2);
  if constexpr (FAR) return __builtin_nontemporal_load(reinterpret_cast<const u4 *>(at));
  if (A == 16 || (c + 1) * V <= width) return *reinterpret_cast<const typename Piece<A>::type *>(at);
  u4 v = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < V - 1; ++i)
    if (c * V + i < width) {
      if constexpr (F32)
        v[i] = reinterpret_cast<const uint32_t *>(at)[i];
      else
        v[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(at)[i] << (i % 2 * 16);
    }
  return v;
}

template <bool F32, int A, bool FAR = false>
__device__ __forceinline__ void store_piece(void *rows, size_t row, int c, int width, u4 v) {
  constexpr int V = kValues<F32>;
  char *at = static_cast<char *>(rows) + (row * width + (size_t)c * V) * (F32 ? 4 : 2);
  if constexpr (FAR) {
    __builtin_nontemporal_store(v, reinterpret_cast<u4 *>(at));
    return;
  }
  if (A == 16 || (c + 1) * V <= width) {
    *reinterpret_cast<typename Piece<A>::type *>(at) = v;
    return;
  }
#pragma unroll
  for (int i = 0; i < V - 1; ++i)
    if (c * V + i < width) {
      if constexpr (F32)
        reinterpret_cast<uint32_t *>(at)[i] = v[i];
      else
        reinterpret_cast<uint16_t *>(at)[i] = (uint16_t)(v[i / 2] >> (i % 2 * 16));
    }
}

template <bool F32>
__device__ __forceinline__ float value(u4 v, int i) {
  if constexpr (F32) return __builtin_bit_cast(float, (uint32_t)v[i]);
  else return __builtin_bit_cast(float, i % 2 ? v[i / 2] & 0xFFFF0000u : v[i / 2] << 16);
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const bf16x2 v = {(__bf16)lo, (__bf16)hi};   // to nearest even, a NaN stays one
  return __builtin_bit_cast(uint32_t, v);
}

template <bool F32>
__device__ __forceinline__ u4 pack(const float (&f)[kValues<F32>]) {
  u4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (F32) v[i] = __builtin_bit_cast(uint32_t, f[i]);
    else v[i] = bf16_pair(f[2 * i], f[2 * i + 1]);
  }
  return v;
}

// The places of choices j0 .. j0 + G - 1 of token t; -1 where none is.
template <int G>
__device__ __forceinline__ void load_places(const MoveArgs &p, int t, int j0, int (&at)[G]) {
#pragma unroll
  for (int j = 0; j < G; ++j) {
    const int v = j0 + j < p.top_k ? p.places[(size_t)t * p.top_k + j0 + j] : -1;
    at[j] = (unsigned)v < (unsigned)p.rows ? v : -1;
  }
}

// A workgroup is 256 / lanes tokens by `lanes` pieces, blockIdx.y the piece's group.
__device__ __forceinline__ bool own_piece(const MoveArgs &p, int shift, int pieces, int &t, int &step, int &c) {
  t = (int)((blockIdx.x * 256 + threadIdx.x) >> shift);
  step = (int)((gridDim.x * 256) >> shift);
  c = (int)(blockIdx.y << shift) + (int)(threadIdx.x & ((1u << shift) - 1));
  return c < pieces;
}

template <bool F32, int A, bool FAR>
__global__ __launch_bounds__(256) void rows_spread_kernel(const MoveArgs p, const int shift, const int pieces) {
  int t, step, c;
  if (!own_piece(p, shift, pieces, t, step, c)) return;
  for (; t < p.tokens; t += step) {
    const u4 v = load_piece<F32, A>(p.x, t, c, p.width);
    for (int j0 = 0; j0 < p.top_k; j0 += 8) {
      int at[8];
      load_places(p, t, j0, at);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (at[j] >= 0) store_piece<F32, A, FAR>(p.out, at[j], c, p.width, v);
    }
  }
}

// The rows of G choices are sent for together: with room for 8 of which top 2 has
// two, six loads of eight are of row 0, so G is 2, 4 or 8 by top_k.
template <bool ZF32, bool YF32, int A, int G, bool FAR>
__global__ __launch_bounds__(256) void rows_combine_kernel(const MoveArgs p, const int shift, const int pieces) {
  constexpr int V = kValues<ZF32>;
  int t, step, c;
  if (!own_piece(p, shift, pieces, t, step, c)) return;
  for (; t < p.tokens; t += step) {
    float sum[V];
#pragma unroll
    for (int i = 0; i < V; ++i) sum[i] = 0.0f;
    for (int j0 = 0; j0 < p.top_k && p.rows > 0; j0 += G) {
      int at[G];
      float w[G];
      u4 v[G];
      load_places(p, t, j0, at);
#pragma unroll
      for (int j = 0; j < G; ++j) {   // without a place: row 0 is read and not added
        v[j] = load_piece<ZF32, A, FAR>(p.x, at[j] < 0 ? 0 : at[j], c, p.width);
        w[j] = p.w && j0 + j < p.top_k ? p.w[(size_t)t * p.top_k + j0 + j] : 1.0f;
      }
#pragma unroll
      for (int j = 0; j < G; ++j)
        if (at[j] >= 0)
#pragma unroll
          for (int i = 0; i < V; ++i) sum[i] = __builtin_fmaf(w[j], value<ZF32>(v[j], i), sum[i]);
    }
    if constexpr (ZF32 == YF32) {
      store_piece<YF32, A, FAR>(p.out, t, c, p.width, pack<YF32>(sum));
    } else if constexpr (YF32) {   // a piece of z is two of y
      const float lo[4] = {sum[0], sum[1], sum[2], sum[3]}, hi[4] = {sum[4], sum[5], sum[6], sum[7]};
      store_piece<true, A == 2 ? 4 : A>(p.out, t, 2 * c, p.width, pack<true>(lo));
      if (A == 16 || (2 * c + 1) * 4 < p.width)
        store_piece<true, A == 2 ? 4 : A>(p.out, t, 2 * c + 1, p.width, pack<true>(hi));
    } else {                       // half of one
      uint16_t *to = static_cast<uint16_t *>(p.out) + (size_t)t * p.width + c * 4;
      const uint32_t v[2] = {bf16_pair(sum[0], sum[1]), bf16_pair(sum[2], sum[3])};
      if (A == 16) {
        *reinterpret_cast<uint2 *>(to) = make_uint2(v[0], v[1]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c * 4 + i < p.width) to[i] = (uint16_t)(v[i / 2] >> (i % 2 * 16));
      }
    }
  }
}

// LANES lanes a token (a wave, or the whole workgroup), which keep the dot
// products of G choices in registers and add them up at the end, in an order that
// goes by the width alone; dy is read again for each G of them, once up to top 8.
// The whole workgroup where a row has more pieces than a wave: 4096 tokens of 2048
// bf16, top 8, 62 us against a wave's 74. Groups of G choices by top_k as above:
// 16384 tokens of top 2 54 us, with groups of 8 73.
template <bool F32, int A, int LANES, int G, bool FAR>
__global__ __launch_bounds__(256) void rows_combine_grad_kernel(const MoveArgs p, const int pieces) {
  constexpr int V = kValues<F32>;
  __shared__ float waves[4][G];
  const int lane = (int)threadIdx.x & (LANES - 1), step = (int)(gridDim.x * 256) / LANES;
  for (int t = (int)(blockIdx.x * 256 + threadIdx.x) / LANES; t < p.tokens; t += step) {
    for (int j0 = 0; j0 < p.top_k; j0 += G) {
      int at[G];
      float w[G], dot[G];
      load_places(p, t, j0, at);
#pragma unroll
      for (int j = 0; j < G; ++j) {
        w[j] = p.w && j0 + j < p.top_k ? p.w[(size_t)t * p.top_k + j0 + j] : 1.0f;
        dot[j] = 0.0f;
      }
      for (int c = lane; c < pieces && p.rows > 0; c += LANES) {
        const u4 dy = load_piece<F32, A>(p.x, t, c, p.width);
        if (p.z) {
          u4 z[G];
#pragma unroll
          for (int j = 0; j < G; ++j) z[j] = load_piece<F32, A, FAR>(p.z, at[j] < 0 ? 0 : at[j], c, p.width);
#pragma unroll
          for (int j = 0; j < G; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) dot[j] = __builtin_fmaf(value<F32>(dy, i), value<F32>(z[j], i), dot[j]);
        }
#pragma unroll
        for (int j = 0; j < G; ++j) {
          if (at[j] < 0) continue;
          float f[V];
#pragma unroll
          for (int i = 0; i < V; ++i) f[i] = w[j] * value<F32>(dy, i);
          store_piece<F32, A, FAR>(p.out, at[j], c, p.width, pack<F32>(f));
        }
      }
      if (!p.dw) continue;
#pragma unroll
      for (int j = 0; j < G; ++j) dot[j] = group_sum<64>(dot[j]);
      if constexpr (LANES == 256) {
        __syncthreads();
        if ((threadIdx.x & 63) == 0)
#pragma unroll
          for (int j = 0; j < G; ++j) waves[threadIdx.x >> 6][j] = dot[j];
        __syncthreads();
#pragma unroll
        for (int j = 0; j < G; ++j) dot[j] = (waves[0][j] + waves[1][j]) + (waves[2][j] + waves[3][j]);
      }
      if (lane == 0)
#pragma unroll
        for (int j = 0; j < G; ++j)
          if (j0 + j < p.top_k) p.dw[(size_t)t * p.top_k + j0 + j] = at[j] < 0 ? 0.0f : dot[j];
    }
  }
}

constexpr unsigned kMostGroups = 1u << 20;   // workgroups along the tokens; the kernels loop over the rest

// Lanes a token: of 8 to 256 the ones that leave the fewest idle, more of them
// where that is equal.
int lanes_shift(int pieces) {
  int best = 8;
  int64_t least = INT64_MAX;
  for (int s = 8; s >= 3; --s) {
    const int64_t took = (int64_t)rows::ceil_div(pieces, 1 << s) << s;
    if (took < least) {
      least = took;
      best = s;
    }
  }
  return best;
}

unsigned token_groups(int tokens, int lanes) {
  const unsigned g = (unsigned)rows::ceil_div((int64_t)tokens * lanes, 256);
  return g < kMostGroups ? g : kMostGroups;
}

int pieces_of(const MoveArgs &a) { return rows::ceil_div(a.width, a.in_f32 ? 4 : 8); }

int launch_move(const char *name, void (*kernel)(const MoveArgs, const int, const int), const MoveArgs &a, hipStream_t s) {
  const int pieces = pieces_of(a), shift = lanes_shift(pieces);
  return launch_kernel(name, kernel, dim3(token_groups(a.tokens, 1 << shift), (unsigned)rows::ceil_div(pieces, 1 << shift)),
                       dim3(256), 0, s, a, shift, pieces);
}

// Rows whose every piece is whole and 16-byte aligned.
bool whole(const MoveArgs &a) { return a.width % (a.in_f32 ? 4 : 8) == 0; }

bool far(const MoveArgs &a) {
  return rows::past_caches((int64_t)a.tokens * a.top_k < a.rows ? a.tokens * a.top_k : a.rows, a.width, a.in_f32);
}

template <bool F32>
int spread(const MoveArgs &a, hipStream_t s) {
  return launch_move("rows_spread_kernel",
                     !whole(a) ? rows_spread_kernel<F32, F32 ? 4 : 2, false>
                     : far(a)  ? rows_spread_kernel<F32, 16, true>
                               : rows_spread_kernel<F32, 16, false>,
                     a, s);
}

template <bool ZF32, bool YF32, int G>
int combine(const MoveArgs &a, hipStream_t s) {
  return launch_move("rows_combine_kernel",
                     !whole(a) ? rows_combine_kernel<ZF32, YF32, ZF32 ? 4 : 2, G, false>
                     : far(a)  ? rows_combine_kernel<ZF32, YF32, 16, G, true>
                               : rows_combine_kernel<ZF32, YF32, 16, G, false>,
                     a, s);
}

template <int G>
int combine_of(const MoveArgs &a, hipStream_t s) {
  if (a.in_f32) return a.out_f32 ? combine<true, true, G>(a, s) : combine<true, false, G>(a, s);
  return a.out_f32 ? combine<false, true, G>(a, s) : combine<false, false, G>(a, s);
}

template <bool F32, int LANES, int G>
int grad(const MoveArgs &a, hipStream_t s) {
  return launch_kernel("rows_combine_grad_kernel",
                       !whole(a) ? rows_combine_grad_kernel<F32, F32 ? 4 : 2, LANES, G, false>
                       : far(a)  ? rows_combine_grad_kernel<F32, 16, LANES, G, true>
                                 : rows_combine_grad_kernel<F32, 16, LANES, G, false>,
                       dim3(token_groups(a.tokens, LANES)), dim3(256), 0, s, a, pieces_of(a));
}

template <int G>
int grad_of(const MoveArgs &a, hipStream_t s) {
  const bool wide = pieces_of(a) > 64;
  if (a.in_f32) return wide ? grad<true, 256, G>(a, s) : grad<true, 64, G>(a, s);
  return wide ? grad<false, 256, G>(a, s) : grad<false, 64, G>(a, s);
}

}  // namespace

int launch_rows_spread(const MoveArgs &a, void *stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  return a.in_f32 ? spread<true>(a, s) : spread<false>(a, s);
}

int launch_rows_combine(const MoveArgs &a, void *stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  return a.top_k <= 2 ? combine_of<2>(a, s) : a.top_k <= 4 ? combine_of<4>(a, s) : combine_of<8>(a, s);
}

int launch_rows_combine_grad(const MoveArgs &a, void *stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  return a.top_k <= 2 ? grad_of<2>(a, s) : a.top_k <= 4 ? grad_of<4>(a, s) : grad_of<8>(a, s);
}

}  // namespace qmv
