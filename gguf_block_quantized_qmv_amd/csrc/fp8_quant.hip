// Rows of activations to e4m3 with one fp32 scale per 128 values, plain or as
// silu(gate) * up; gfx950.
//
// Sixteen lanes hold one block of 128 values, eight each, in registers: the
// block's largest magnitude is a maximum over the lanes' values and then over
// one DPP row of 16 lanes, so the values are read once and the codes written
// once. Bound by memory: 2 or 4 bytes read and 1 + 4/128 written per value.
// 4096 x 5120 in bf16 takes 12.9 us, 4.9 TB/s of those bytes (a large copy: 5.2);
// 4099 x 776 gated from fp32 8.3 us; one row of 5120 6 us, a launch's own time.
#include "fp8_internal.h"
#include "fp8_layout.h"
#include "qmv_device.h"
#include "../../include/qmm_fp8.h"

namespace qmv {
namespace {

constexpr float kMax = 448.0f;           // largest e4m3 value
constexpr float kTiny = 1.17549435e-38f;  // 2^-126

// Eight consecutive values of a row as fp32 (exact).
template <bool F32>
__device__ __forceinline__ void load8(const void *__restrict__ x, size_t at, float (&v)[8]) {
  if constexpr (F32) {
    const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(x) + at);
    const float4 a = p[0], b = p[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(x) + at);
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_bits_to_f32(u[i] & 0xFFFFu);
      v[2 * i + 1] = __builtin_bit_cast(float, u[i] & 0xFFFF0000u);
    }
  }
}

// Maximum over each group of 16 lanes of non-negative floats' bit patterns,
// where infinity and then NaN order above every finite value.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
  return v > o ? v : o;
}
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
  v = dpp_max<0xB1>(v);
  v = dpp_max<0x4E>(v);
  v = dpp_max<0x141>(v);
  return dpp_max<0x140>(v);
}

// Past 448 only by the rounding of the quotient; a NaN stays.
__device__ __forceinline__ float clamp448(float v) { return v > kMax ? kMax : v < -kMax ? -kMax : v; }

template <bool F32, bool GATED>
__global__ __launch_bounds__(256) void fp8_quant_kernel(const void *__restrict__ x, uint8_t *__restrict__ xq,
                                                        float *__restrict__ xs, const int m, const int k,
                                                        const int nb) {
  const int group = (int)threadIdx.x >> 4, lane = (int)threadIdx.x & 15;
  const int r = (int)blockIdx.x * 16 + group;
  const int b = (int)blockIdx.y;
  if (r >= m) return;
  const int col = b * 128 + lane * 8;
  const size_t ld = GATED ? 2 * (size_t)k : (size_t)k;
  float v[8];
  const bool in = col < k;   // k is a multiple of 8: eight values are all in or all out
  if (in) {
    load8<F32>(x, (size_t)r * ld + col, v);
    if constexpr (GATED) {
      float u[8];
      load8<F32>(x, (size_t)r * ld + k + col, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = v[i] / (1.0f + expf(-v[i])) * u[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  }
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t a = __builtin_bit_cast(uint32_t, v[i]) & 0x7FFFFFFFu;
    top = a > top ? a : top;
  }
  top = row16_max(top);
  float scale = __builtin_bit_cast(float, top) / kMax;
  scale = scale < kTiny ? kTiny : scale;   // a NaN stays
  if (lane == 0) xs[(size_t)b * m + r] = scale;
  if (!in) return;
  uint32_t code[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int c = __builtin_amdgcn_cvt_pk_fp8_f32(clamp448(v[4 * h] / scale), clamp448(v[4 * h + 1] / scale), 0, false);
    c = __builtin_amdgcn_cvt_pk_fp8_f32(clamp448(v[4 * h + 2] / scale), clamp448(v[4 * h + 3] / scale), c, true);
    code[h] = (uint32_t)c;
  }
  *reinterpret_cast<uint2 *>(xq + (size_t)r * k + col) = make_uint2(code[0], code[1]);
}

template <bool F32, bool GATED>
int launch(const void *x, uint8_t *xq, float *xs, int m, int k, hipStream_t s) {
  const int nb = fp8::blocks_of(k);
  return launch_kernel("fp8_quant_kernel", fp8_quant_kernel<F32, GATED>,
                       dim3((unsigned)fp8::ceil_div(m, 16), (unsigned)nb), dim3(256), 0, s, x, xq, xs, m, k, nb);
}

}  // namespace

int launch_fp8_quant(const void *x, bool x_f32, bool gated, uint8_t *xq, float *xs, int m, int k, void *stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (x_f32) return gated ? launch<true, true>(x, xq, xs, m, k, s) : launch<true, false>(x, xq, xs, m, k, s);
  return gated ? launch<false, true>(x, xq, xs, m, k, s) : launch<false, false>(x, xq, xs, m, k, s);
}

}  // namespace qmv
