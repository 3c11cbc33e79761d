// linear_attention_step.cuh — one token of the gated (delta-rule) linear
// attention recurrence per sequence, states updated in place.
//
//   S <- e^g S;  u = beta (v - S^T k)  (u = v without beta);  S <- S + k u^T
//   o = scale * S^T q
// per value head, S [d_k][d_v] FP32 in a pool of slots. (News article
// "Qwen3.8-27B最激进4bit量化开源，权重显存暴降2.9倍！" §01: the gated delta rule
// of the recurrent layers; its printed formula did not survive extraction,
// this is the Gated DeltaNet form its text describes.)
//
// What it cannot do without: S read and written once, 8 d_k d_v bytes per head
// against 6-8 FLOP per element, so DRAM bounds it. Both products with S need
// it whole before u is known; written out,
//   S^T k and S^T q of the OLD state:  p = S^T k,  r = S^T q
//   u = beta (v - e^g p),  o = scale (e^g r + (q.k) u),  S <- e^g S + k u^T
// one pass over the registers gives both sums, with one reduction between the
// threads, and S goes from memory to registers and back without shared memory.
// A CTA of 128 threads owns COLS of the d_v columns of one (token, head): row
// groups of COLS / 4 lanes with a float4 of columns each, whole 128-byte lines
// per row, 8 rows a thread. COLS = 32 for d_k = 128 (one token of 32 heads
// already gives 128 CTAs), 64 for d_k = 64 where d_v allows: with 4 rows a thread
// there were too few bytes in flight (256 rows of 24 heads 76 -> 66 us). 64
// registers, so that 8 CTAs share an SM (96 left to the compiler, 5 CTAs: 256
// rows of 32 heads x 128 x 128 took 199 us instead of 162, 5.8 TB/s).
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "ptx.cuh"

namespace nvfp4 {
namespace la {

constexpr int kStepThreads = 128;

// d_v columns per CTA
__host__ __device__ constexpr int step_cols(int d_k, int d_v) {
  return d_k == 64 && d_v % 64 == 0 ? 64 : 32;
}

struct StepArgs {
  const __nv_bfloat16* q;   // [batch][ldq], head h at h * d_k
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;   // [batch][ldv], head h at h * d_v
  int64_t ldq, ldk, ldv, ldo;
  const float* decay;       // [batch][h_v], log decay g
  const float* beta;        // [batch][h_v] or null
  float scale;
  int batch, h_k, h_v, d_v;
  float* state;             // [n_slots][h_v][d_k][d_v]
  int n_slots;
  const int32_t* slots;     // [batch] or null (token b uses slot b)
  __nv_bfloat16* o;         // [batch][ldo]
};

// Tokens that name the same slot are taken in order by the CTAs of the first
// of them, with the state kept in registers between them; a token whose slot
// lies outside the pool is padding, its row of o stays as it was.
template <int DK, int COLS>
__global__ void __launch_bounds__(kStepThreads, 8)
    step_kernel(const StepArgs a) {
  constexpr int LANES = COLS / 4;                // lanes of a row
  constexpr int GROUPS = kStepThreads / LANES;   // rows at a time
  constexpr int R = DK / GROUPS;                 // rows per thread
  __shared__ float s_q[DK], s_k[DK];
  __shared__ float4 s_red[2][4][LANES];
  __shared__ float s_qk[4];
  __shared__ int s_next;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int col = (t % LANES) * 4, row0 = t / LANES;   // this thread's columns, first row
  const int blocks = a.d_v / COLS;
  const int h = (blockIdx.x / blocks) % a.h_v;
  int b = blockIdx.x / blocks / a.h_v;
  const int c0 = (blockIdx.x % blocks) * COLS;
  const int hk = h / (a.h_v / a.h_k);
  ptx::grid_dep_launch();
  ptx::grid_dep_wait();
  const int slot = a.slots != nullptr ? a.slots[b] : b;
  if (slot < 0 || slot >= a.n_slots) return;
  float* const S = a.state + (static_cast<int64_t>(slot) * a.h_v + h) * DK * a.d_v + c0 + col;
  float4 s[R];
#pragma unroll
  for (int i = 0; i < R; ++i)
    s[i] = __ldcs(reinterpret_cast<const float4*>(S + static_cast<int64_t>(row0 + GROUPS * i) * a.d_v));
  while (true) {
    // the next token of this slot; an earlier one means other CTAs own it
    int next = a.batch;
    if (a.slots != nullptr) {
      if (t == 0) s_next = a.batch;
      __syncthreads();
      int earlier = 0;
      for (int i = t; i < a.batch; i += kStepThreads)
        if (a.slots[i] == slot) {
          if (i < b) earlier = 1;
          else if (i > b) { atomicMin(&s_next, i); break; }
        }
      if (__syncthreads_or(earlier) && b == static_cast<int>(blockIdx.x / blocks / a.h_v)) return;
      next = s_next;
    }
    const float g = a.decay[static_cast<int64_t>(b) * a.h_v + h];
    const float beta = a.beta != nullptr ? a.beta[static_cast<int64_t>(b) * a.h_v + h] : 0.0f;
    float qk = 0.0f;
    for (int i = t; i < DK; i += kStepThreads) {
      const float qi = __bfloat162float(a.q[b * a.ldq + static_cast<int64_t>(hk) * DK + i]);
      const float ki = __bfloat162float(a.k[b * a.ldk + static_cast<int64_t>(hk) * DK + i]);
      s_q[i] = qi;
      s_k[i] = ki;
      qk += qi * ki;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) qk += __shfl_xor_sync(0xFFFFFFFFu, qk, d);
    if (lane == 0) s_qk[warp] = qk;
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = __bfloat162float(a.v[b * a.ldv + static_cast<int64_t>(h) * a.d_v + c0 + col + j]);
    __syncthreads();
    float4 p = make_float4(0, 0, 0, 0), r = p;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float ki = s_k[row0 + GROUPS * i], qi = s_q[row0 + GROUPS * i];
      p.x += ki * s[i].x; p.y += ki * s[i].y; p.z += ki * s[i].z; p.w += ki * s[i].w;
      r.x += qi * s[i].x; r.y += qi * s[i].y; r.z += qi * s[i].z; r.w += qi * s[i].w;
    }
#pragma unroll
    for (int d = LANES; d <= 16; d <<= 1) {
      p.x += __shfl_xor_sync(0xFFFFFFFFu, p.x, d); p.y += __shfl_xor_sync(0xFFFFFFFFu, p.y, d);
      p.z += __shfl_xor_sync(0xFFFFFFFFu, p.z, d); p.w += __shfl_xor_sync(0xFFFFFFFFu, p.w, d);
      r.x += __shfl_xor_sync(0xFFFFFFFFu, r.x, d); r.y += __shfl_xor_sync(0xFFFFFFFFu, r.y, d);
      r.z += __shfl_xor_sync(0xFFFFFFFFu, r.z, d); r.w += __shfl_xor_sync(0xFFFFFFFFu, r.w, d);
    }
    if (lane < LANES) {
      s_red[0][warp][lane] = p;
      s_red[1][warp][lane] = r;
    }
    __syncthreads();
    float pj[4] = {0, 0, 0, 0}, rj[4] = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float4 x = s_red[0][w][t % LANES], y = s_red[1][w][t % LANES];
      pj[0] += x.x; pj[1] += x.y; pj[2] += x.z; pj[3] += x.w;
      rj[0] += y.x; rj[1] += y.y; rj[2] += y.z; rj[3] += y.w;
    }
    qk = s_qk[0] + s_qk[1] + s_qk[2] + s_qk[3];
    const float e = expf(g);
    float u[4], out[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u[j] = a.beta != nullptr ? beta * (v[j] - e * pj[j]) : v[j];
      out[j] = a.scale * (e * rj[j] + qk * u[j]);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float ki = s_k[row0 + GROUPS * i];
      s[i].x = e * s[i].x + ki * u[0]; s[i].y = e * s[i].y + ki * u[1];
      s[i].z = e * s[i].z + ki * u[2]; s[i].w = e * s[i].w + ki * u[3];
    }
    if (row0 == 0) {
      __nv_bfloat16* o = a.o + b * a.ldo + static_cast<int64_t>(h) * a.d_v + c0 + col;
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = __float2bfloat16_rn(out[j]);
    }
    if (next >= a.batch) break;
    b = next;
    __syncthreads();  // s_q, s_k and the sums are read above
  }
#pragma unroll
  for (int i = 0; i < R; ++i)
    __stcs(reinterpret_cast<float4*>(S + static_cast<int64_t>(row0 + GROUPS * i) * a.d_v), s[i]);
}

}  // namespace la
}  // namespace nvfp4
