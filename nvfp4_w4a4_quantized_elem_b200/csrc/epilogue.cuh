// epilogue.cuh — bias, activation and residual on the W4A4 GEMM's accumulator.
//
//   y = act(acc / (g_a g_b) + bias[n]) + residual[m][n]
// evaluated in FP32 and rounded once to the output type. The news article
// "Qwen3.8-27B最激进4bit量化开源，权重显存暴降2.9倍！" §02 only names the 4-bit
// product; the epilogue is the model's own and is written from the formulas:
//   relu       max(z, 0)
//   silu       z / (1 + e^-z)
//   gelu       z/2 (1 + erf(z / sqrt 2)) = z Phi(z)
//   gelu_tanh  z/2 (1 + tanh u) = z / (1 + e^-2u), u = sqrt(2/pi) (z + 0.044715 z^3)
// Without the fusion the bf16 product makes one more round trip through
// memory per step (2 m n bytes written, read and written again) and is
// rounded once more on the way.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "ptx.cuh"

namespace nvfp4 {
namespace epi {

enum : int { kNone = 0, kRelu = 1, kSilu = 2, kGelu = 3, kGeluTanh = 4 };

struct Args {
  const __nv_bfloat16* bias;      // [N] or null
  const __nv_bfloat16* residual;  // [M][ldr] or null; may be Y itself
  int64_t ldr;
  int act;
};

// z / (1 + 2^t), two instructions of the special-function unit. Where 2^t
// overflows or its reciprocal is subnormal (t > 126) the quotient is given as
// 0; the true value is below 1e-35.
__device__ __forceinline__ float over_one_plus_ex2(float z, float t) {
  return z * ptx::rcp(1.0f + ptx::ex2(t));
}

// z Phi(z) = max(z, 0) - |z| Q(|z|), Q(a) = erfc(a / sqrt 2) / 2, without the
// cancellation of z/2 + z/2 erf, which leaves no digit below z = -5.5. Q(a) =
// e^{-a^2/2} F(a) with F smooth: t P(t) with t = 1 / (1 + 0.3 a), P of degree 7
// fitted to the least largest relative error on [0, 14.5] (1.7e-7, a linear
// program). What is left is the exponential's, |z|^2/2 steps in the far tail.
// Beyond |z| = 20, where Q is below 1e-88, |z| stands at 20 (so that -inf gives 0).
__device__ __forceinline__ float gelu(float z) {
  const float a = fminf(fabsf(z), 20.0f);
  const float t = ptx::rcp(fmaf(0.3f, a, 1.0f));
  float p = fmaf(0.0354235582f, t, -0.156157714f);
  p = fmaf(p, t, 0.204555524f);
  p = fmaf(p, t, -0.0520328607f);
  p = fmaf(p, t, 0.127691165f);
  p = fmaf(p, t, 0.100176129f);
  p = fmaf(p, t, 0.120712108f);
  p = fmaf(p, t, 0.119632009f);
  const float q = (p * t) * ptx::ex2((a * a) * -0.72134752f);  // 2^(-a^2/2 log2(e))
  return fmaf(-a, q, z < 0.0f ? 0.0f : z);  // (a NaN stays one)
}

template <int ACT>
__device__ __forceinline__ float activate(float z) {
  if (ACT == kRelu) return z < 0.0f ? 0.0f : z;  // (a NaN stays one)
  if (ACT == kSilu) return over_one_plus_ex2(z, -1.44269504f * z);
  if (ACT == kGelu) return gelu(z);
  if (ACT == kGeluTanh)  // -2u log2(e) = z (-2.30220819 - 0.102943240 z^2)
    return over_one_plus_ex2(z, z * fmaf(z * z, -0.102943240f, -2.30220819f));
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

// The residual of a chunk of 32 rows x 32 columns, held by a warp as it is
// loaded: four lanes per row, 16 bytes each, so that every sector that comes
// from L2 is used whole (a lane per row, 16 bytes at a time, fetched them
// twice: the L1 that the GEMM's shared memory leaves does not hold 16 warps'
// lines). exchange() hands each lane its own row by way of the warp's 2 KiB
// staging chunk, in the layout that the output goes through it.
struct ResChunk {
  uint4 v[4];
  __device__ __forceinline__ void load(const __nv_bfloat16* res, int64_t ld, int rows, int cols,
                                       int lane) {
    const int u = lane & 3, left = cols - 8 * u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * i + (lane >> 2);
      v[i] = r < rows && left > 0 ? load_bf16x8(res + r * ld + 8 * u, left)
                                  : make_uint4(0u, 0u, 0u, 0u);
    }
  }
  __device__ __forceinline__ void exchange(uint8_t* chunk, int lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * i + (lane >> 2), u = lane & 3;
      *reinterpret_cast<uint4*>(chunk + r * 64 + ((u ^ ((r >> 1) & 3)) << 4)) = v[i];
    }
    __syncwarp();
#pragma unroll
    for (int u = 0; u < 4; ++u)
      v[u] = *reinterpret_cast<const uint4*>(chunk + lane * 64 + ((u ^ ((lane >> 1) & 3)) << 4));
  }
};

// 32 consecutive columns of one output row, acc (FP32 bits) in place:
// act(acc alpha + bias). bias32: shared-memory copy of the columns' bias (null
// without one), the same addresses for the whole warp.
template <int ACT>
__device__ __forceinline__ void apply32_as(uint32_t (&acc)[32], float alpha,
                                           const uint16_t* bias32) {
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    float z[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = __uint_as_float(acc[8 * u + i]) * alpha;
    if (bias32 != nullptr) add_bf16x8(z, *reinterpret_cast<const uint4*>(bias32 + 8 * u));
    activate_all<ACT>(z);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[8 * u + i] = __float_as_uint(z[i]);
  }
}

__device__ __forceinline__ void apply32(uint32_t (&acc)[32], float alpha, int act,
                                        const uint16_t* bias32) {
  switch (act) {
    case kRelu: apply32_as<kRelu>(acc, alpha, bias32); break;
    case kSilu: apply32_as<kSilu>(acc, alpha, bias32); break;
    case kGelu: apply32_as<kGelu>(acc, alpha, bias32); break;
    case kGeluTanh: apply32_as<kGeluTanh>(acc, alpha, bias32); break;
    default: apply32_as<kNone>(acc, alpha, bias32); break;
  }
}

// The exchanged residual added to them.
__device__ __forceinline__ void add_residual(uint32_t (&acc)[32], const ResChunk& r) {
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    float z[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = __uint_as_float(acc[8 * u + i]);
    add_bf16x8(z, r.v[u]);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[8 * u + i] = __float_as_uint(z[i]);
  }
}

}  // namespace epi
}  // namespace nvfp4
