// epilogue.cuh — bias, activation and residual on the W4A4 GEMM's accumulator.
//
//   y = act(acc / (g_a g_b) + bias[n]) + residual[m][n]
// evaluated in FP32 and rounded once to the output type. The news article
// "Qwen3.8-27B最激进4bit量化开源，权重显存暴降2.9倍！" §02 only names the 4-bit
// product; the epilogue is the model's own and is written from the formulas:
//   relu       max(z, 0)
//   silu       z / (1 + e^-z)
//   gelu       z/2 erfc(-z / sqrt 2)
//   gelu_tanh  z/2 (1 + tanh u) = z / (1 + e^-2u), u = sqrt(2/pi) (z + 0.044715 z^3)
// Without the fusion the bf16 product makes one more round trip through
// memory per step (2 m n bytes written, read and written again) and is
// rounded once more on the way.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

namespace nvfp4 {
namespace epi {

enum : int { kNone = 0, kRelu = 1, kSilu = 2, kGelu = 3, kGeluTanh = 4 };

struct Args {
  const __nv_bfloat16* bias;      // [N] or null
  const __nv_bfloat16* residual;  // [M][ldr] or null; may be Y itself
  int64_t ldr;
  int act;
};

// z / (1 + e^t). The fast exponential and division (a few FP32 ulp) serve
// every finite z: where e^t leaves the fast division's range (above 2^126) or
// overflows, the quotient is given as 0 and the true value is below 1e-35.
__device__ __forceinline__ float over_one_plus_exp(float z, float t) {
  return __fdividef(z, 1.0f + __expf(t));
}

template <int ACT>
__device__ __forceinline__ float activate(float z) {
  if (ACT == kRelu) return fmaxf(z, 0.0f);
  if (ACT == kSilu) return over_one_plus_exp(z, -z);
  if (ACT == kGelu) return 0.5f * z * erfcf(-0.70710678f * z);
  if (ACT == kGeluTanh) return over_one_plus_exp(z, -1.59576912f * (z + 0.044715f * z * z * z));
  return z;
}

template <int ACT, int N>
__device__ __forceinline__ void activate_all(float (&z)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) z[i] = activate<ACT>(z[i]);
}

// `act` is uniform over the grid: one branch per N values.
template <int N>
__device__ __forceinline__ void activate_n(int act, float (&z)[N]) {
  switch (act) {
    case kRelu: activate_all<kRelu>(z); break;
    case kSilu: activate_all<kSilu>(z); break;
    case kGelu: activate_all<kGelu>(z); break;
    case kGeluTanh: activate_all<kGeluTanh>(z); break;
    default: break;
  }
}

// Eight bf16 of a 16-byte vector added to z[0..8).
__device__ __forceinline__ void add_bf16x8(float* z, const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    z[2 * e] += __uint_as_float(w[e] << 16);
    z[2 * e + 1] += __uint_as_float(w[e] & 0xFFFF0000u);
  }
}

// 8 bf16 at p, of which the first `left` lie inside the row (the others read
// as 0): a vector load where all do.
__device__ __forceinline__ uint4 load_bf16x8(const __nv_bfloat16* p, int left) {
  if (left >= 8) return *reinterpret_cast<const uint4*>(p);
  const uint16_t* u = reinterpret_cast<const uint16_t*>(p);
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t lo = 2 * e < left ? u[2 * e] : 0u;
    const uint32_t hi = 2 * e + 1 < left ? u[2 * e + 1] : 0u;
    w[e] = lo | (hi << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 32 consecutive columns of one output row: acc (FP32 bits) -> y (FP32 bits).
// bias32: shared-memory copy of the columns' bias (null without a bias), the
// same addresses for the whole warp; res: this row's residual at the first
// column, or null; left: columns of the row from the first on. All residual
// loads come first; the arithmetic goes 8 columns at a time, so that a thread
// which holds 128 accumulator columns stays inside its 168 registers.
__device__ __forceinline__ void apply32(uint32_t (&acc)[32], float alpha, int act,
                                        const uint16_t* bias32, const __nv_bfloat16* res,
                                        int left) {
  uint4 rv[4];
#pragma unroll
  for (int u = 0; u < 4; ++u)
    rv[u] = res != nullptr && left > 8 * u ? load_bf16x8(res + 8 * u, left - 8 * u)
                                           : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    float z[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = __uint_as_float(acc[8 * u + i]) * alpha;
    if (bias32 != nullptr) add_bf16x8(z, *reinterpret_cast<const uint4*>(bias32 + 8 * u));
    activate_n(act, z);
    add_bf16x8(z, rv[u]);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[8 * u + i] = __float_as_uint(z[i]);
  }
}

}  // namespace epi
}  // namespace nvfp4
