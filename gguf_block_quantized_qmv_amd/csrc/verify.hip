// Verification of drafted tokens: which drafts stand, and the token that follows
// them, from given random numbers; gfx950.
//
// Of the probabilities only one row of p and of q a request matters beyond the
// drafts' own entries. It is cut into chunks of 1024 tokens for a wave each, which
// leaves two sums by chunk: the weights max(p - q, 0) and p alone. One wave then
// adds up a request's chunks, finds the one in which the running sum passes u times
// the whole, and the token in it. Either a workgroup does all of that for a
// request, or a first launch spreads the chunks over the CUs and a second picks.
//
// Sums are fp64: over a vocabulary of 10^5 an fp32 sum would move the borders
// between tokens by more than a rare token's own weight. A draft's test takes
// the product u * q in fp64, where it is exact.
//
// One request is bound by latency: launches and the chain from a draft's test over
// the sums to the token (vocabulary of 131072, fp32: sums 4.0 us, pick 4.2). A batch
// is bound by memory: 128 requests of 100003 tokens, fp32, with lengths of 0 to 3
// drafts, 74 MB in 14.9 us, 5.0 TB/s of a large copy's 5.2, and 5.0 us to pick.
#include <float.h>

#include "rows_device.h"
#include "rows_internal.h"
#include "rows_layout.h"

namespace qmv {
namespace {

constexpr int kPer = rows::kVerifyChunk / 64;   // tokens a lane

// A chunk of one row from memory. Lane i holds, for each vector h, the values
// (h * 64 + i) * V .. + V - 1 of it; behind the end: zeros.
template <bool F32>
struct Values {
  static constexpr int V = F32 ? 4 : 8, H = kPer / V;
  float v[H][V];

  __device__ __forceinline__ void load(const void *row, int first, int vocab) {
    typedef uint32_t Vec __attribute__((ext_vector_type(4), aligned(2)));   // the start of a row is any element's
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const int at = first + (h * 64 + ((int)threadIdx.x & 63)) * V;
      if (at + V <= vocab) {
        const Vec u = *reinterpret_cast<const Vec *>(static_cast<const char *>(row) + (size_t)at * (F32 ? 4 : 2));
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if constexpr (F32) v[h][i] = __builtin_bit_cast(float, (uint32_t)u[i]);
          else v[h][i] = __builtin_bit_cast(float, i % 2 ? u[i / 2] & 0xFFFF0000u : u[i / 2] << 16);
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          v[h][i] = 0.0f;
          if (at + i < vocab) {
            if constexpr (F32) v[h][i] = static_cast<const float *>(row)[at + i];
            else v[h][i] = bf16_bits_to_f32(static_cast<const uint16_t *>(row)[at + i]);
          }
        }
      }
    }
  }
};

__device__ __forceinline__ float entry(const void *row, int f32, int i) {
  return f32 ? static_cast<const float *>(row)[i] : bf16_bits_to_f32(static_cast<const uint16_t *>(row)[i]);
}

// p - q where that is a weight: what is negative or not finite counts as zero.
// Tested in fp64: with the tests in fp32 the sums' kernel takes 87 registers instead
// of 52, and 128 rows of 131072 bf16 26 us instead of 23.
__device__ __forceinline__ double weight(float p, float q) {
  const double d = (double)p - (double)q;
  return d > 0.0 && d <= DBL_MAX ? d : 0.0;
}

__device__ __forceinline__ const void *row_of(const void *p, int f32, size_t row, int vocab) {
  return static_cast<const char *>(p) + row * vocab * (f32 ? 4 : 2);
}

// The draft that decides: the first `accepted` stand; `refused`: the next one,
// `token`, does not, else there is none.
struct Outcome {
  int accepted, token;
  bool refused;
};

__device__ __forceinline__ int drafts_of(const VerifyArgs &a, int r) {
  if (!a.lengths) return a.drafts;
  const int n = a.lengths[r];
  return n < 0 ? 0 : n > a.drafts ? a.drafts : n;
}

// Lane i of every wave holds draft i against its row.
__device__ __forceinline__ Outcome decide(const VerifyArgs &a, int r) {
  const int lane = (int)threadIdx.x & 63;
  const int length = drafts_of(a, r);
  bool stands = false;
  int token = -1;
  if (lane < length) {
    token = a.tokens[(size_t)r * a.drafts + lane];
    if ((unsigned)token < (unsigned)a.vocab) {
      const float u = a.u[(size_t)r * (a.drafts + 1) + lane];
      const float p = entry(row_of(a.p, a.f32, (size_t)r * (a.drafts + 1) + lane, a.vocab), a.f32, token);
      const float q = a.q ? entry(row_of(a.q, a.f32, (size_t)r * a.drafts + lane, a.vocab), a.f32, token) : 1.0f;
      stands = (double)u * (double)q < (double)p;
    }
  }
  const uint64_t fails = ~__ballot(stands);   // the lanes from `length` on fail, 32 of them at least
  const int n = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)fails) - 1);
  return Outcome{n, __builtin_amdgcn_readlane(token, n), n < length};
}

// Sums over a wave's lanes up to and with each lane, and its last lane's value.
template <int CTRL, int ROWS>
__device__ __forceinline__ double add_from(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, CTRL, ROWS, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(u >> 32), CTRL, ROWS, 0xF, false);
  return v + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_upto(double v) {
  v = add_from<0x111, 0xF>(v);   // as the whole numbers' sum in rows_device.h
  v = add_from<0x112, 0xF>(v);
  v = add_from<0x114, 0xF>(v);
  v = add_from<0x118, 0xF>(v);
  v = add_from<0x142, 0xA>(v);
  return add_from<0x143, 0xC>(v);
}
__device__ __forceinline__ double of_lane(double v, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)u, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// p and q of a chunk: the weights, and p's own, by which a refused draft without
// any weight picks.
template <bool F32>
struct Chunk {
  static constexpr int V = Values<F32>::V, H = Values<F32>::H;
  Values<F32> p, q;
  int first, zero;   // zero: a token without q that was refused

  __device__ __forceinline__ Chunk(const VerifyArgs &a, int r, const Outcome &o, int chunk) {
    first = chunk * rows::kVerifyChunk;
    zero = o.refused && !a.q ? o.token : -1;
    p.load(row_of(a.p, F32, (size_t)r * (a.drafts + 1) + o.accepted, a.vocab), first, a.vocab);
    if (o.refused && a.q) {
      q.load(row_of(a.q, F32, (size_t)r * a.drafts + o.accepted, a.vocab), first, a.vocab);
    } else {
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int i = 0; i < V; ++i) q.v[h][i] = 0.0f;
    }
  }
  __device__ __forceinline__ int token(int h, int i) const { return first + (h * 64 + ((int)threadIdx.x & 63)) * V + i; }
  __device__ __forceinline__ double left(int h, int i) const { return weight(p.v[h][i], 0.0f); }
  __device__ __forceinline__ double rest(int h, int i) const {
    return token(h, i) == zero ? 0.0 : weight(p.v[h][i], q.v[h][i]);
  }
};

// A chunk's two sums, by one wave.
template <bool F32>
__device__ __forceinline__ void sum_chunk(const VerifyArgs &a, int r, const Outcome &o, int chunk, double *sums) {
  const Chunk<F32> c(a, r, o, chunk);
  double s = 0.0, t = 0.0;
#pragma unroll
  for (int h = 0; h < c.H; ++h)
#pragma unroll
    for (int i = 0; i < c.V; ++i) {
      s += c.rest(h, i);
      t += c.left(h, i);
    }
  s = wave_upto(s);
  t = wave_upto(t);
  if ((threadIdx.x & 63) == 63) {
    sums[chunk * 2] = s;
    sums[chunk * 2 + 1] = t;
  }
}

// The lanes that hold something, in the order of what they hold: the first and the last.
__device__ __forceinline__ int first_lane(uint64_t b) { return __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)b) - 1); }
__device__ __forceinline__ int last_lane(uint64_t b) { return __builtin_amdgcn_readfirstlane(63 - __clzll((long long)b)); }

// The token that follows, and the request's row of `out`, by one wave.
template <bool F32>
__device__ __forceinline__ void pick(const VerifyArgs &a, int r, const Outcome &o, const float u, const double *sums,
                                     const int chunks) {
  const int lane = (int)threadIdx.x & 63;
  const int per = rows::ceil_div(chunks, 64), c0 = lane * per;   // neighbouring chunks a lane
  double own[2] = {0.0, 0.0}, upto[2];
  for (int c = c0; c < c0 + per && c < chunks; ++c) {
    own[0] += sums[c * 2];
    own[1] += sums[c * 2 + 1];
  }
  upto[0] = wave_upto(own[0]);
  upto[1] = wave_upto(own[1]);
  const int kind = of_lane(upto[0], 63) > 0.0 ? 0 : 1;   // without a weight: p's own
  const double total = of_lane(kind ? upto[1] : upto[0], 63);
  // From one on (or NaN) no running sum may lie above it: these are of another order than the whole and can
  // round above it before the last weight.
  const double target = u < 1.0f ? (double)u * total : __builtin_inf();
  int token = -1;
  if (total > 0.0) {
    // the first chunk whose running sum lies above the target, else the last with a weight
    int first = -1, last = -1;
    double run = kind ? upto[1] - own[1] : upto[0] - own[0], base = 0.0, base_last = 0.0;
    for (int c = c0; c < c0 + per && c < chunks; ++c) {
      const double s = sums[c * 2 + kind];
      if (s > 0.0) {
        last = c;
        base_last = run;
        if (first < 0 && run + s > target) {
          first = c;
          base = run;
        }
      }
      run += s;
    }
    const uint64_t above = __ballot(first >= 0);
    const int of = above ? first_lane(above) : last_lane(__ballot(last >= 0));
    double at = of_lane(above ? base : base_last, of);
    const Chunk<F32> c(a, r, o, __builtin_amdgcn_readlane(above ? first : last, of));
    // the same for its tokens, vector by vector
    int end = -1;
#pragma unroll
    for (int h = 0; h < c.H; ++h) {
      double v[c.V], s = 0.0;
#pragma unroll
      for (int i = 0; i < c.V; ++i) {
        v[i] = kind ? c.left(h, i) : c.rest(h, i);
        s += v[i];
      }
      const double with = wave_upto(s);
      double here = at + (with - s);
      at += of_lane(with, 63);
      int t = -1, e = -1;
#pragma unroll
      for (int i = 0; i < c.V; ++i) {
        here += v[i];
        if (v[i] > 0.0) {
          e = c.token(h, i);
          if (t < 0 && here > target) t = e;
        }
      }
      const uint64_t up = __ballot(t >= 0), some = __ballot(e >= 0);
      if (up && token < 0) token = __builtin_amdgcn_readlane(t, first_lane(up));
      if (some) end = __builtin_amdgcn_readlane(e, last_lane(some));
    }
    if (token < 0) token = end;
  }
  if (lane <= a.drafts)
    a.out[(size_t)r * (a.drafts + 1) + lane] =
        lane < o.accepted ? a.tokens[(size_t)r * a.drafts + lane] : lane == o.accepted ? token : -1;
}

template <bool F32>
__global__ __launch_bounds__(256) void verify_sums_kernel(const VerifyArgs a, const int chunks) {
  const int r = (int)blockIdx.y, chunk = (int)blockIdx.x * 4 + ((int)threadIdx.x >> 6);
  if (chunk >= chunks) return;
  const Outcome o = decide(a, r);
  if (chunk == 0 && (threadIdx.x & 63) == 0) a.accepted[r] = o.accepted;
  sum_chunk<F32>(a, r, o, chunk, a.sums + (size_t)r * chunks * 2);
}

template <bool F32>
__global__ __launch_bounds__(64) void verify_pick_kernel(const VerifyArgs a, const int chunks) {
  const int r = (int)blockIdx.x;
  Outcome o;
  o.accepted = a.accepted[r];
  o.refused = o.accepted < drafts_of(a, r);
  o.token = o.refused ? a.tokens[(size_t)r * a.drafts + o.accepted] : -1;
  pick<F32>(a, r, o, a.u[(size_t)r * (a.drafts + 1) + a.drafts], a.sums + (size_t)r * chunks * 2, chunks);
}

// Both for one request in a workgroup of 16 waves.
template <bool F32>
__global__ __launch_bounds__(1024) void verify_whole_kernel(const VerifyArgs a, const int chunks) {
  extern __shared__ double sums[];
  const int r = (int)blockIdx.x, wave = (int)threadIdx.x >> 6;
  const float u = a.u[(size_t)r * (a.drafts + 1) + a.drafts];
  const Outcome o = decide(a, r);
  for (int c = wave; c < chunks; c += 16) sum_chunk<F32>(a, r, o, c, sums);
  __syncthreads();
  if (wave) return;
  if (threadIdx.x == 0) a.accepted[r] = o.accepted;
  pick<F32>(a, r, o, u, sums, chunks);
}

template <bool F32>
int launch(const VerifyArgs &a, hipStream_t s) {
  const int chunks = rows::ceil_div(a.vocab, rows::kVerifyChunk);
  if (!a.sums)
    return launch_kernel("verify_whole_kernel", verify_whole_kernel<F32>, dim3((unsigned)a.requests), dim3(1024),
                         (size_t)chunks * 16, s, a, chunks);
  const int rc = launch_kernel("verify_sums_kernel", verify_sums_kernel<F32>,
                               dim3((unsigned)rows::ceil_div(chunks, 4), (unsigned)a.requests), dim3(256), 0, s, a, chunks);
  if (rc) return rc;
  return launch_kernel("verify_pick_kernel", verify_pick_kernel<F32>, dim3((unsigned)a.requests), dim3(64), 0, s, a, chunks);
}

}  // namespace

int launch_verify_drafts(const VerifyArgs &a, void *stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  return a.f32 ? launch<true>(a, s) : launch<false>(a, s);
}

}  // namespace qmv
