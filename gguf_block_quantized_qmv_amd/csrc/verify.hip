// Verification of drafted tokens: which drafts stand, and the token that follows
// them, from given random numbers; gfx950.
//
// Of the probabilities only one row of p and of q a request matters beyond the
// drafts' own entries. The first launch cuts that row into chunks of 4096 for a
// workgroup each and leaves two sums by chunk: the weights max(p - q, 0) and p
// alone. The second adds up a request's chunks, finds the one in which the
// running sum passes u times the whole, and the token in it.
//
// Sums are fp64: over a vocabulary of 10^5 an fp32 sum would move the borders
// between tokens by more than a rare token's own weight. A draft's test takes
// the product u * q in fp64, where it is exact.
#include <limits.h>

#include "qmv_device.h"
#include "rows_internal.h"
#include "rows_layout.h"

namespace qmv {
namespace {

constexpr int kPer = rows::kVerifyChunk / 256;   // tokens a thread

// kPer values of one row from memory. Thread i holds, for each vector h, the
// values (h * 256 + i) * V .. + V - 1 of the chunk; behind the end: zeros.
template <bool F32>
struct Values {
  static constexpr int V = F32 ? 4 : 8, H = kPer / V;
  float v[H][V];

  __device__ __forceinline__ void load(const void *row, int first, int vocab) {
    typedef uint32_t Vec __attribute__((ext_vector_type(4), aligned(2)));   // the start of a row is any element's
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const int at = first + (h * 256 + (int)threadIdx.x) * V;
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

// A weight: what is negative or not finite counts as zero.
__device__ __forceinline__ double weight(double d) { return d > 0.0 && d <= 1.7976931348623157e308 ? d : 0.0; }

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
__device__ __forceinline__ Outcome judge(const VerifyArgs &a, int r) {
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

// The weights of a chunk, and p alone, by which a refused draft without any picks.
template <bool F32>
__device__ __forceinline__ void weights(const VerifyArgs &a, int r, const Outcome &o, int first, double (&rest)[kPer],
                                        double (&left)[kPer]) {
  constexpr int V = Values<F32>::V, H = Values<F32>::H;
  Values<F32> p, q;
  p.load(row_of(a.p, F32, (size_t)r * (a.drafts + 1) + o.accepted, a.vocab), first, a.vocab);
  const bool drafted = o.refused && a.q;
  if (drafted) q.load(row_of(a.q, F32, (size_t)r * a.drafts + o.accepted, a.vocab), first, a.vocab);
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const double v = (double)p.v[h][i];
      left[h * V + i] = weight(v);
      double d = v;
      if (drafted) d = v - (double)q.v[h][i];
      else if (o.refused && first + (h * 256 + (int)threadIdx.x) * V + i == o.token) d = 0.0;
      rest[h * V + i] = weight(d);
    }
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

template <bool F32>
__global__ __launch_bounds__(256) void verify_sums_kernel(const VerifyArgs a, const int chunks) {
  __shared__ double waves[4][2];
  const int r = (int)blockIdx.y, chunk = (int)blockIdx.x;
  const Outcome o = judge(a, r);
  if (chunk == 0 && threadIdx.x == 0) a.accepted[r] = o.accepted;
  double rest[kPer], left[kPer], s = 0.0, t = 0.0;
  weights<F32>(a, r, o, chunk * rows::kVerifyChunk, rest, left);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    s += rest[i];
    t += left[i];
  }
  s = wave_sum(s);
  t = wave_sum(t);
  if ((threadIdx.x & 63) == 0) {
    waves[threadIdx.x >> 6][0] = s;
    waves[threadIdx.x >> 6][1] = t;
  }
  __syncthreads();
  if (threadIdx.x < 2)
    a.sums[((size_t)r * chunks + chunk) * 2 + threadIdx.x] =
        (waves[0][threadIdx.x] + waves[1][threadIdx.x]) + (waves[2][threadIdx.x] + waves[3][threadIdx.x]);
}

// Inclusive sum over the wave.
__device__ __forceinline__ double wave_scan(double v) {
  const int lane = (int)threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// Least of the workgroup's values.
__device__ __forceinline__ int least(int v, int *waves) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_xor(v, d);
    v = o < v ? o : v;
  }
  __syncthreads();   // the last reads of `waves`
  if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = v;
  __syncthreads();
  const int a = waves[0] < waves[1] ? waves[0] : waves[1], b = waves[2] < waves[3] ? waves[2] : waves[3];
  return a < b ? a : b;
}

template <bool F32>
__global__ __launch_bounds__(256) void verify_pick_kernel(const VerifyArgs a, const int chunks) {
  constexpr int V = Values<F32>::V, H = Values<F32>::H;
  __shared__ double sums[2][4], runs[H][4], found_base;
  __shared__ int waves[4];
  const int r = (int)blockIdx.x, tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6;
  Outcome o;
  o.accepted = a.accepted[r];
  o.refused = o.accepted < drafts_of(a, r);
  o.token = o.refused ? a.tokens[(size_t)r * a.drafts + o.accepted] : -1;
  const float u = a.u[(size_t)r * (a.drafts + 1) + a.drafts];

  // every thread's neighbouring chunks, both sums
  const int per = rows::ceil_div(chunks, 256), c0 = tid * per;
  const double *sum = a.sums + (size_t)r * chunks * 2;
  double upto[2] = {0.0, 0.0}, own[2];
  for (int c = c0; c < c0 + per && c < chunks; ++c)
#pragma unroll
    for (int k = 0; k < 2; ++k) upto[k] += sum[c * 2 + k];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    own[k] = upto[k];
    upto[k] = wave_scan(upto[k]);
    if (lane == 63) sums[k][wave] = upto[k];
  }
  __syncthreads();
  double all[2], before[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    double s = 0.0;
    before[k] = 0.0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if (w == wave) before[k] = s;
      s += sums[k][w];
    }
    all[k] = s;
    before[k] += upto[k] - own[k];
  }
  const int kind = all[0] > 0.0 ? 0 : 1;
  const double total = kind ? all[1] : all[0], target = (double)u * total;
  int token = -1;
  if (total > 0.0) {
    // the first chunk whose running sum lies above the target, else the last with a weight
    int first = INT_MAX, last = INT_MAX;   // last: negated, so that the least is the last
    double run = kind ? before[1] : before[0], base = 0.0, base_last = 0.0;
    for (int c = c0; c < c0 + per && c < chunks; ++c) {
      const double s = sum[c * 2 + kind];
      if (s > 0.0) {
        last = -c;
        base_last = run;
        if (first == INT_MAX && run + s > target) {
          first = c;
          base = run;
        }
      }
      run += s;
    }
    int chunk = least(first, waves);
    if (chunk == INT_MAX) {
      const int l = least(last, waves);
      chunk = -l;
      if (last == l) found_base = base_last;
    } else if (first == chunk) {
      found_base = base;
    }
    __syncthreads();
    double rest[kPer], left[kPer], part[H];
    weights<F32>(a, r, o, chunk * rows::kVerifyChunk, rest, left);
#pragma unroll
    for (int h = 0; h < H; ++h) {
      double s = 0.0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (kind) rest[h * V + i] = left[h * V + i];
        s += rest[h * V + i];
      }
      part[h] = wave_scan(s);
      if (lane == 63) runs[h][wave] = part[h];
      part[h] -= s;
    }
    __syncthreads();
    double at = found_base;
    first = last = INT_MAX;
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        if (w == wave) {
          double here = at + part[h];
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const double v = rest[h * V + i];
            here += v;
            const int t = chunk * rows::kVerifyChunk + (h * 256 + tid) * V + i;
            if (v > 0.0) {
              last = -t;
              if (first == INT_MAX && here > target) first = t;
            }
          }
        }
        at += runs[h][w];
      }
    token = least(first, waves);
    if (token == INT_MAX) token = -least(last, waves);
  }
  if (tid <= a.drafts)
    a.out[(size_t)r * (a.drafts + 1) + tid] =
        tid < o.accepted ? a.tokens[(size_t)r * a.drafts + tid] : tid == o.accepted ? token : -1;
}

template <bool F32>
int launch(const VerifyArgs &a, hipStream_t s) {
  const int chunks = rows::ceil_div(a.vocab, rows::kVerifyChunk);
  const int rc = launch_kernel("verify_sums_kernel", verify_sums_kernel<F32>, dim3((unsigned)chunks, (unsigned)a.requests),
                               dim3(256), 0, s, a, chunks);
  if (rc) return rc;
  return launch_kernel("verify_pick_kernel", verify_pick_kernel<F32>, dim3((unsigned)a.requests), dim3(256), 0, s, a, chunks);
}

}  // namespace

int launch_verify_drafts(const VerifyArgs &a, void *stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  return a.f32 ? launch<true>(a, s) : launch<false>(a, s);
}

}  // namespace qmv
