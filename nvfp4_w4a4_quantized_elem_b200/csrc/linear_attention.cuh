// linear_attention.cuh — gated (delta-rule) linear attention over packed
// prompts, in chunks of 64 tokens.
//
// Per value head, with S [d_k][d_v] FP32 and g_t the log decay:
//   S_t = e^{g_t} S_{t-1} + k_t u_t^T,  o_t = scale S_t^T q_t,
//   u_t = beta_t (v_t - e^{g_t} S_{t-1}^T k_t)   (delta rule), or u_t = v_t.
// (News article "Qwen3.8-27B最激进4bit量化开源，权重显存暴降2.9倍！" §01 names the
// gated delta rule; its formula did not survive extraction, this is the Gated
// DeltaNet form its text describes.)
// Over a chunk with start state S, G_t = g_1 + .. + g_t, and rows of K, Q, V, U
// per token, unrolling gives
//   (I + L) U = diag(beta) (V - diag(e^G) K S),  L_tj = beta_t e^{G_t-G_j} k_t.k_j, j < t
//   O = diag(e^G) Q S + A U,                      A_tj = e^{G_t-G_j} q_t.k_j, j <= t
//   S' = e^{G_64} S + K^T diag(e^{G_64-G}) U
// so with T = (I + L)^-1 diag(beta) and X = V - diag(e^G) K S
//   [U; O - diag(e^G) Q S] = [T; A T] X:
// three products per chunk depend on one another, [K; Q] S, [T; AT] X and
// K^T U~, all with 128 rows on the MMA's M side (tokens of K and Q together,
// then of U and O together, then d_k) and a block of d_v columns as its N.
//
// Two kernels. prepare_kernel, parallel over chunks and heads, computes what
// does not depend on S: the swizzled bf16 image of [K; Q] (rows past a
// sequence's end zero), [T; AT] and the decay factors. chain_kernel walks a
// sequence's chunks in order, one CTA per (sequence, head, d_v block), with S
// in FP32 registers.
//
// Precision: q, k, v are bf16 and enter the products exactly. S, X, U, T, A
// are FP32 values; as MMA operands each is split into bf16 hi + lo (16 bits,
// residual 2^-17 of the value), products hi hi + hi lo + lo hi, accumulated
// in FP32: one bf16 operand alone would leave 2^-9 in the FP32 states. G is
// summed in FP64: the difference of two FP32 sums of strong decays would lose
// the weak decays between them.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "fault.cuh"
#include "gemm_skinny.cuh"
#include "ptx.cuh"

namespace nvfp4 {
namespace la {

constexpr int C = 64;                       // tokens per chunk
constexpr int kHalfBytes = 128 * 128;       // [K; Q] image: 128 rows x 64 of d_k
constexpr int kTTBytes = 128 * 128;         // [T; AT] image: 128 rows x 64, one piece
constexpr int kGateFloats = 2 * C + 4;      // e^G, e^{G_64 - G}, e^{G_64}
constexpr int kGateBytes = (kGateFloats * 4 + 127) / 128 * 128;
constexpr uint64_t kWaitLimitNs = 2000000000ull;

enum : uint32_t { kFaultPrepare = 512u, kFaultChainMma = 1024u, kFaultChain = 2048u };

__host__ __device__ constexpr int kq_bytes(int dk) { return dk / 64 * kHalfBytes; }
constexpr int kHeadBytes = 2 * kTTBytes + kGateBytes;  // per (chunk, value head)

struct Args {
  const __nv_bfloat16* q;   // [total][ldq], head h at h * d_k
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;   // [total][ldv], head h at h * d_v
  int64_t ldq, ldk, ldv, ldo;
  const float* decay;       // [total][h_v], log decay
  const float* beta;        // [total][h_v] or null (no delta rule)
  float scale;
  int total, h_k, h_v, d_v, n_seq;
  const int32_t* cu;        // [n_seq + 1] or null (one sequence of total tokens)
  float* state;             // [n_slots][h_v][d_k][d_v] or null
  int n_slots;
  const int32_t* slots;     // [n_seq] or null (sequence b uses slot b)
  const int32_t* resume;    // [n_seq] or null (every sequence starts from zero)
  __nv_bfloat16* o;         // [total][ldo]
  uint8_t* kq;              // [chunk slots][h_k] images
  uint8_t* tt;              // [chunk slots][h_v] images and gates
};

// Sequence b's tokens [start, end): offsets outside [0, total] or decreasing
// ones are cut to it, so no access leaves the buffers.
__device__ __forceinline__ void seq_range(const Args& a, int b, int& start, int& end) {
  if (a.cu == nullptr) {
    start = 0;
    end = a.total;
    return;
  }
  start = min(max(a.cu[b], 0), a.total);
  end = min(max(a.cu[b + 1], start), a.total);
}

// Chunk i of sequence b has slot start/64 + b + i: ceil(len/64) <= (end/64 -
// start/64) + 1, so the slots of different sequences do not meet, and all lie
// below total/64 + n_seq.
__device__ __forceinline__ int first_slot(int start, int b) { return start / C + b; }

// Two FP32 values -> packed bf16 hi parts, and the packed bf16 of the rests.
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  const __nv_bfloat162 l = __floats2bfloat162_rn(x - __low2float(h), y - __high2float(h));
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

// Row `k` of an MN-major operand without swizzle (8 x 16-byte core matrices,
// 128 bytes apart along k, `n_stride` bytes apart along n): 8 consecutive n.
__device__ __forceinline__ uint32_t mn_off(int k, int n8, int n_stride) {
  return static_cast<uint32_t>((k >> 3) * 128 + (k & 7) * 16 + n8 * n_stride);
}

// N FP32 values of operand row k -> hi and lo pieces in shared memory.
template <int N>
__device__ __forceinline__ void store_row_split(uint32_t hi_base, uint32_t lo_base, int k,
                                                int n_stride, const float (&x)[N]) {
#pragma unroll
  for (int n8 = 0; n8 < N / 8; ++n8) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) split2(x[8 * n8 + 2 * e], x[8 * n8 + 2 * e + 1], h[e], l[e]);
    const uint32_t off = mn_off(k, n8, n_stride);
    ptx::st_shared_v4(hi_base + off, h[0], h[1], h[2], h[3]);
    ptx::st_shared_v4(lo_base + off, l[0], l[1], l[2], l[3]);
  }
}

// 16-byte unit `u` of row r in a 128-byte-row, 128-byte-swizzled image.
__device__ __forceinline__ uint32_t sw128(int r, int u) {
  return static_cast<uint32_t>(r * 128 + ((u ^ (r & 7)) << 4));
}

template <int N>
__device__ __forceinline__ void tc_ld(uint32_t taddr, float (&x)[N]) {
  static_assert(N % 32 == 0, "32 columns per load");
#pragma unroll
  for (int i = 0; i < N; i += 32) {
    uint32_t r[32];
    ptx::tc_ld_32x32b_x32(taddr + i, r);
#pragma unroll
    for (int j = 0; j < 32; ++j) x[i + j] = __uint_as_float(r[j]);
  }
  ptx::tc_wait_ld();
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity,
                                          volatile uint32_t* abort_flag, uint32_t who) {
  return __all_sync(0xFFFFFFFFu,
                    skinny::wait_bounded(bar, parity, abort_flag, who, kWaitLimitNs));
}

// ------------------------------------------------------------------ prepare --

constexpr int kPrepThreads = 128;
constexpr int kLd = 65;                       // row pitch of the FP32 64x64 tiles
constexpr int kTileBytes = (C * kLd * 4 + 127) / 128 * 128;

template <int DK>
struct PrepCfg {
  static constexpr int KQ = kq_bytes(DK);
  static constexpr int A_OFF = KQ;                       // A pieces, then the image (2 x 16 KiB)
  static constexpr int L_OFF = A_OFF + 2 * kTTBytes;     // L (FP32), then T's pieces
  static constexpr int T_OFF = L_OFF + kTileBytes;       // (I + L)^-1 (FP32)
  static constexpr int M_OFF = T_OFF + kTileBytes;       // 32x33 scratch of the inverse
  static constexpr int G_OFF = M_OFF + 32 * 33 * 4 + 128;
  static constexpr int SMEM = 1024 + G_OFF + C * 8 + C * 4 + 64;
};

// (I + L)^-1 of the strictly lower triangular L (FP32, unit diagonal implied):
// the four 16x16 diagonal blocks by forward substitution, one thread per
// column; then twice [P 0; L21 Q]^-1 = [P^-1 0; -Q^-1 L21 P^-1 Q^-1].
__device__ __forceinline__ void invert_unit_lower(const float* L, float* T, float* M, int t) {
  if (t < C) {
    const int b0 = t & ~15, j = t & 15;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = i == j ? 1.0f : 0.0f;
#pragma unroll
      for (int m = 0; m < i; ++m) s -= L[(b0 + i) * kLd + b0 + m] * x[m];
      x[i] = i < j ? 0.0f : s;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) T[(b0 + i) * kLd + b0 + j] = x[i];
  }
  __syncthreads();
#pragma unroll 1
  for (int w = 16; w < C; w *= 2) {
    const int per = w * w, n = per * (C / (2 * w));
    for (int i = t; i < n; i += kPrepThreads) {   // M = L21 P^-1
      const int b = i / per, r = (i % per) / w, c = i % w, o = 2 * w * b;
      float s = 0.0f;
      for (int m = c; m < w; ++m) s += L[(o + w + r) * kLd + o + m] * T[(o + m) * kLd + o + c];
      M[b * w * 17 * (w / 16) + r * (w + 1) + c] = s;
    }
    __syncthreads();
    for (int i = t; i < n; i += kPrepThreads) {   // T21 = -Q^-1 M
      const int b = i / per, r = (i % per) / w, c = i % w, o = 2 * w * b;
      float s = 0.0f;
      for (int m = 0; m <= r; ++m)
        s += T[(o + w + r) * kLd + o + w + m] * M[b * w * 17 * (w / 16) + m * (w + 1) + c];
      T[(o + w + r) * kLd + o + c] = -s;
    }
    __syncthreads();
  }
}

template <int DK>
__global__ void __launch_bounds__(kPrepThreads)
    prepare_kernel(const Args a) {
  using P = PrepCfg<DK>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  float* const L = reinterpret_cast<float*>(smem + P::L_OFF);
  float* const T = reinterpret_cast<float*>(smem + P::T_OFF);
  float* const M = reinterpret_cast<float*>(smem + P::M_OFF);
  double* const G = reinterpret_cast<double*>(smem + P::G_OFF);
  float* const Beta = reinterpret_cast<float*>(G + C);
  uint64_t* const bar = reinterpret_cast<uint64_t*>(Beta + C);
  uint32_t* const tmem_holder = reinterpret_cast<uint32_t*>(bar + 1);
  volatile uint32_t* const abort_flag = tmem_holder + 1;

  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int h = blockIdx.x % a.h_v, hk = h / (a.h_v / a.h_k);
  const int slot = blockIdx.x / a.h_v;
  ptx::grid_dep_launch();
  ptx::grid_dep_wait();
  // the last sequence whose first slot is at or below this one
  int lo = 0, hi = a.n_seq - 1, start, end;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    seq_range(a, mid, start, end);
    if (first_slot(start, mid) <= slot) lo = mid; else hi = mid - 1;
  }
  seq_range(a, lo, start, end);
  const int64_t tok0 = start + static_cast<int64_t>(slot - first_slot(start, lo)) * C;
  if (slot < first_slot(start, lo) || tok0 >= end) return;
  const int len = static_cast<int>(min(static_cast<int64_t>(C), end - tok0));

  if (t == 0) {
    ptx::mbar_init(bar, 1);
    *abort_flag = 0u;
    ptx::fence_mbarrier_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(tmem_holder, 128);
    ptx::tmem_relinquish();
  }
  // [K; Q] -> the swizzled image, rows past the sequence zero
  constexpr int kUnits = DK / 8;
  for (int i = t; i < 128 * kUnits; i += kPrepThreads) {
    const int r = i / kUnits, u = i % kUnits, tok = r & (C - 1);
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (tok < len) {
      const __nv_bfloat16* row = r < C ? a.k + (tok0 + tok) * a.ldk : a.q + (tok0 + tok) * a.ldq;
      x = *reinterpret_cast<const uint4*>(row + static_cast<int64_t>(hk) * DK + 8 * u);
    }
    *reinterpret_cast<uint4*>(smem + (u / 8) * kHalfBytes + sw128(r, u % 8)) = x;
  }
  // G_t in FP64 (a decay of e^-1000 is zero in FP32 and FP64 sums keep the
  // weak ones beside it, so -inf counts as that), beta
  if (warp == 0) {
    const int i0 = 2 * lane;
    const float* g = a.decay + tok0 * a.h_v + h;
    const double x0 = i0 < len ? fmax(static_cast<double>(g[static_cast<int64_t>(i0) * a.h_v]), -1000.0) : 0.0;
    const double x1 = i0 + 1 < len ? fmax(static_cast<double>(g[static_cast<int64_t>(i0 + 1) * a.h_v]), -1000.0) : 0.0;
    double s = x0 + x1;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const double y = __shfl_up_sync(0xFFFFFFFFu, s, d);
      if (lane >= d) s += y;
    }
    G[i0] = s - x1;
    G[i0 + 1] = s;
  } else if (warp >= 2) {
    const int i = t - 64;
    Beta[i] = i < len ? (a.beta != nullptr ? a.beta[(tok0 + i) * a.h_v + h] : 1.0f) : 0.0f;
  }
  ptx::fence_proxy_async_smem();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const uint32_t sb = ptx::smem_u32(smem);
  if (t == 0) {
    // [K; Q] K^T: 128 x 64
    constexpr uint32_t kScores = ptx::idesc_bf16(128, C, false, false);
#pragma unroll
    for (int s = 0; s < DK / 16; ++s) {
      const uint64_t d = ptx::smem_desc(sb + (s / 4) * kHalfBytes + (s % 4) * 32, 16, 1024, 2);
      ptx::tc_mma_bf16(tmem, d, d, kScores, s != 0);
    }
    ptx::tc_commit(bar);
    if (h % (a.h_v / a.h_k) == 0) {  // the group's first head writes the image
      ptx::bulk_store(a.kq + (static_cast<int64_t>(slot) * a.h_k + hk) * P::KQ, smem, P::KQ);
      ptx::bulk_commit_group();
    }
  }
  bool ok = warp_wait(bar, 0, abort_flag, kFaultPrepare);
  ptx::tc_fence_after();
  const int row = t & (C - 1);
  uint8_t* const out = a.tt + (static_cast<int64_t>(slot) * a.h_v + h) * kHeadBytes;
  {
    float x[C];
    tc_ld(tmem + (static_cast<uint32_t>(warp * 32) << 16), x);
    const double gt = G[row];
    if (t < C) {
      const float bt = Beta[row];
#pragma unroll
      for (int j = 0; j < C; ++j)
        L[row * kLd + j] = j < row ? bt * expf(static_cast<float>(gt - G[j])) * x[j] : 0.0f;
      float* gate = reinterpret_cast<float*>(out + 2 * kTTBytes);
      gate[row] = expf(static_cast<float>(gt));
      gate[C + row] = expf(static_cast<float>(G[C - 1] - gt));
      if (row == 0) gate[2 * C] = expf(static_cast<float>(G[C - 1]));
    } else {
      // A, zero above the diagonal, as the rows 64..127 of a K-major operand
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        uint32_t hh[4], ll[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = 8 * u + 2 * e;
          const float a0 = j <= row ? expf(static_cast<float>(gt - G[j])) * x[j] : 0.0f;
          const float a1 = j + 1 <= row ? expf(static_cast<float>(gt - G[j + 1])) * x[j + 1] : 0.0f;
          split2(a0, a1, hh[e], ll[e]);
        }
        ptx::st_shared_v4(sb + P::A_OFF + sw128(C + row, u), hh[0], hh[1], hh[2], hh[3]);
        ptx::st_shared_v4(sb + P::A_OFF + kTTBytes + sw128(C + row, u), ll[0], ll[1], ll[2], ll[3]);
      }
    }
  }
  if (a.beta != nullptr) {
    for (int i = t; i < C * kLd; i += kPrepThreads) T[i] = 0.0f;
    __syncthreads();
    invert_unit_lower(L, T, M, t);
    float x[C];
    if (t < C) {
#pragma unroll
      for (int j = 0; j < C; ++j) x[j] = T[row * kLd + j] * Beta[j];
      // over L, which the inverse no longer needs
      store_row_split(sb + P::L_OFF, sb + P::L_OFF + 8192, row, 1024, x);
    }
    ptx::fence_proxy_async_smem();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (t == 0 && ok) {
      constexpr uint32_t kAT = ptx::idesc_bf16(128, C, false, true);
      const uint32_t ap[3] = {0, 0, kTTBytes}, tp[3] = {0, 8192, 0};
#pragma unroll
      for (int c = 0; c < 3; ++c)
#pragma unroll
        for (int s = 0; s < C / 16; ++s)
          ptx::tc_mma_bf16(tmem + C, ptx::smem_desc(sb + P::A_OFF + ap[c] + s * 32, 16, 1024, 2),
                           ptx::smem_desc(sb + P::L_OFF + tp[c] + s * 256, 128, 1024, 0), kAT,
                           (c | s) != 0);
      ptx::tc_commit(bar);
    }
    ok = ok && warp_wait(bar, 1, abort_flag, kFaultPrepare);
    ptx::tc_fence_after();
    if (t >= C) tc_ld(tmem + (static_cast<uint32_t>(warp * 32) << 16) + C, x);
    __syncthreads();  // every warp saw the product done: its operands may be overwritten
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      uint32_t hh[4], ll[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) split2(x[8 * u + 2 * e], x[8 * u + 2 * e + 1], hh[e], ll[e]);
      ptx::st_shared_v4(sb + P::A_OFF + sw128(t, u), hh[0], hh[1], hh[2], hh[3]);
      ptx::st_shared_v4(sb + P::A_OFF + kTTBytes + sw128(t, u), ll[0], ll[1], ll[2], ll[3]);
    }
  } else if (t < C) {
    // without the delta rule T = I (exact in its hi piece) and AT = A stands
    // in its rows already
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint32_t one = (row >> 3) == u ? 0x3F80u << (16 * (row & 1)) : 0u;
      const int e = (row & 7) >> 1;
      ptx::st_shared_v4(sb + P::A_OFF + sw128(row, u), e == 0 ? one : 0u, e == 1 ? one : 0u,
                        e == 2 ? one : 0u, e == 3 ? one : 0u);
      ptx::st_shared_v4(sb + P::A_OFF + kTTBytes + sw128(row, u), 0u, 0u, 0u, 0u);
    }
  }
  ptx::fence_proxy_async_smem();
  ptx::tc_fence_before();
  __syncthreads();
  if (t == 0) {
    ptx::bulk_store(out, smem + P::A_OFF, 2 * kTTBytes);
    ptx::bulk_commit_group();
    ptx::bulk_wait_group_all();
  }
  ptx::tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    ptx::tmem_dealloc(tmem, 128);
  }
}

// -------------------------------------------------------------------- chain --

constexpr int kChainThreads = 160;   // 4 compute warps, 1 warp that loads and issues MMAs

template <int DK, int DVB>
struct ChainCfg {
  static constexpr int STAGE = kq_bytes(DK) + 2 * kTTBytes;
  static constexpr int S_PIECE = DK * DVB * 2;
  static constexpr int X_PIECE = C * DVB * 2;
  static constexpr int S_OFF = 2 * STAGE;
  static constexpr int X_OFF = S_OFF + 2 * S_PIECE;
  static constexpr int U_OFF = X_OFF + 2 * X_PIECE;
  static constexpr int BAR_OFF = U_OFF + 2 * X_PIECE;
  static constexpr int SMEM = 1024 + BAR_OFF + 128;
  static constexpr uint32_t TMEM = 3 * DVB <= 128 ? 128 : 256;
  static_assert(SMEM <= 227 * 1024, "shared memory per CTA");
};

template <int DK, int DVB>
__global__ void __launch_bounds__(kChainThreads)
    chain_kernel(const Args a) {
  using P = ChainCfg<DK, DVB>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* const full = reinterpret_cast<uint64_t*>(smem + P::BAR_OFF);  // [2] stage loaded
  uint64_t* const s_ready = full + 2;   // operand pieces written by the compute warps
  uint64_t* const x_ready = full + 3;
  uint64_t* const u_ready = full + 4;
  uint64_t* const d1 = full + 5;        // products complete
  uint64_t* const d2 = full + 6;
  uint64_t* const d3 = full + 7;
  uint64_t* const drain = full + 8;
  uint32_t* const tmem_holder = reinterpret_cast<uint32_t*>(full + 9);
  volatile uint32_t* const abort_flag = tmem_holder + 1;

  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int blocks = a.d_v / DVB;
  const int c0 = (blockIdx.x % blocks) * DVB;
  const int h = (blockIdx.x / blocks) % a.h_v;
  const int b = blockIdx.x / blocks / a.h_v;
  const int hk = h / (a.h_v / a.h_k);
  if (t == 0) {
    ptx::mbar_init(&full[0], 1);
    ptx::mbar_init(&full[1], 1);
    ptx::mbar_init(s_ready, 4);
    ptx::mbar_init(x_ready, 2);
    ptx::mbar_init(u_ready, 2);
    ptx::mbar_init(d1, 1);
    ptx::mbar_init(d2, 1);
    ptx::mbar_init(d3, 1);
    ptx::mbar_init(drain, 1);
    *abort_flag = 0u;
    ptx::fence_mbarrier_init();
  }
  if (warp == 4) {
    ptx::tmem_alloc(tmem_holder, P::TMEM);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  ptx::grid_dep_launch();
  ptx::grid_dep_wait();
  const uint32_t tmem = *tmem_holder;
  const uint32_t sb = ptx::smem_u32(smem);
  int start, end;
  seq_range(a, b, start, end);
  const int n = (end - start + C - 1) / C;
  const int slot0 = first_slot(start, b);

  if (warp == 4) {
    if (lane == 0) {
      auto load = [&](int c) {
        uint8_t* st = smem + (c & 1) * P::STAGE;
        const int64_t cs = slot0 + c;
        ptx::mbar_arrive_expect_tx(&full[c & 1], P::STAGE);
        ptx::bulk_load(st, a.kq + (cs * a.h_k + hk) * kq_bytes(DK), kq_bytes(DK), &full[c & 1]);
        ptx::bulk_load(st + kq_bytes(DK), a.tt + (cs * a.h_v + h) * kHeadBytes, 2 * kTTBytes,
                       &full[c & 1]);
      };
      constexpr uint32_t kI1 = ptx::idesc_bf16(128, DVB, false, true);
      constexpr uint32_t kI3 = ptx::idesc_bf16(128, DVB, true, true);
      constexpr uint32_t kSN = DK * 16, kXN = C * 16;  // bytes between groups of 8 columns
      int loaded = 0, seen = 0;  // chunks requested; chunks whose load was waited for
      bool ok = true;
      if (n > 0) load(loaded++);
      for (int c = 0; c < n && ok; ++c) {
        const uint32_t par = c & 1;
        const uint32_t kq = sb + par * P::STAGE, tt = kq + kq_bytes(DK);
        // S in place: the previous chunk's products, the last readers of the
        // other stage, are complete
        ok = skinny::wait_bounded(s_ready, par, abort_flag, kFaultChainMma);
        if (!ok) break;
        if (c + 1 < n) load(loaded++);
        ok = skinny::wait_bounded(&full[par], (c >> 1) & 1, abort_flag, kFaultChainMma);
        if (!ok) break;
        ++seen;
        ptx::tc_fence_after();
#pragma unroll
        for (int p = 0; p < 2; ++p)   // [K; Q] S
#pragma unroll
          for (int s = 0; s < DK / 16; ++s)
            ptx::tc_mma_bf16(tmem, ptx::smem_desc(kq + (s / 4) * kHalfBytes + (s % 4) * 32, 16, 1024, 2),
                             ptx::smem_desc(sb + P::S_OFF + p * P::S_PIECE + s * 256, 128, kSN, 0),
                             kI1, (p | s) != 0);
        ptx::tc_commit(d1);
        ok = skinny::wait_bounded(x_ready, par, abort_flag, kFaultChainMma);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t tp[3] = {0, 0, kTTBytes}, xp[3] = {0, P::X_PIECE, 0};
#pragma unroll
        for (int p = 0; p < 3; ++p)   // [T; AT] X
#pragma unroll
          for (int s = 0; s < C / 16; ++s)
            ptx::tc_mma_bf16(tmem + DVB, ptx::smem_desc(tt + tp[p] + s * 32, 16, 1024, 2),
                             ptx::smem_desc(sb + P::X_OFF + xp[p] + s * 256, 128, kXN, 0), kI1,
                             (p | s) != 0);
        ptx::tc_commit(d2);
        ok = skinny::wait_bounded(u_ready, par, abort_flag, kFaultChainMma);
        if (!ok) break;
        ptx::tc_fence_after();
#pragma unroll
        for (int p = 0; p < 2; ++p)   // K^T U~ (64 of d_k: the upper rows repeat the lower)
#pragma unroll
          for (int s = 0; s < C / 16; ++s)
            ptx::tc_mma_bf16(tmem + 2 * DVB,
                             ptx::smem_desc(kq + s * 2048, DK == 128 ? kHalfBytes : 0, 1024, 2),
                             ptx::smem_desc(sb + P::U_OFF + p * P::X_PIECE + s * 256, 128, kXN, 0),
                             kI3, (p | s) != 0);
        ptx::tc_commit(d3);
      }
      if (!ok) {  // let what is in flight end before the CTA does
        ptx::tc_commit(drain);
        skinny::drain_wait(drain, 0);
        for (int c = seen; c < loaded; ++c) skinny::drain_wait(&full[c & 1], (c >> 1) & 1);
      } else if (n > 0) {
        skinny::drain_wait(d3, (n - 1) & 1);  // the last product, should the others give up on it
      }
    }
  } else {
    const int row = t & (C - 1);     // token of the chunk
    const bool is_k = t < C;         // rows of K and U; else rows of Q and O
    const uint32_t lanes = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    // the state: this thread holds row t of d_k
    int slot = -1;
    if (a.state != nullptr) {
      slot = a.slots != nullptr ? a.slots[b] : b;
      if (slot < 0 || slot >= a.n_slots) slot = -1;
      if (slot >= 0 && a.slots != nullptr) {  // only the first sequence that names a slot has it
        int earlier = 0;
        for (int i = lane; i < b; i += 32) earlier |= a.slots[i] == slot;
        if (__any_sync(0xFFFFFFFFu, earlier)) slot = -1;
      }
    }
    float* const state = a.state + ((static_cast<int64_t>(slot) * a.h_v + h) * DK + t) * a.d_v + c0;
    float S[DVB];
#pragma unroll
    for (int j = 0; j < DVB; ++j) S[j] = 0.0f;
    if (slot >= 0 && t < DK && a.resume != nullptr && a.resume[b] != 0) {
#pragma unroll
      for (int j = 0; j < DVB / 4; ++j) {
        const float4 x = reinterpret_cast<const float4*>(state)[j];
        S[4 * j] = x.x; S[4 * j + 1] = x.y; S[4 * j + 2] = x.z; S[4 * j + 3] = x.w;
      }
    }
    const bool delta = a.beta != nullptr;
    bool ok = true;
    for (int c = 0; c < n; ++c) {
      const uint32_t par = c & 1;
      if (DK == 128 || t < DK)
        store_row_split(sb + P::S_OFF, sb + P::S_OFF + P::S_PIECE, t, DK * 16, S);
      ptx::fence_proxy_async_smem();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(s_ready);
      const int64_t tok = start + static_cast<int64_t>(c) * C + row;
      const bool live = tok < end;
      const float* gate = reinterpret_cast<const float*>(
          a.tt + (static_cast<int64_t>(slot0 + c) * a.h_v + h) * kHeadBytes + 2 * kTTBytes);
      const float eg = gate[row], erest = gate[C + row], eall = gate[2 * C];
      uint4 v[DVB / 8];
#pragma unroll
      for (int u = 0; u < DVB / 8; ++u) {
        v[u] = make_uint4(0u, 0u, 0u, 0u);
        if (is_k && live)
          v[u] = *reinterpret_cast<const uint4*>(a.v + tok * a.ldv + static_cast<int64_t>(h) * a.d_v +
                                                 c0 + 8 * u);
      }
      float D[DVB], inter[DVB];
      if (!(ok = warp_wait(d1, par, abort_flag, kFaultChain))) break;
      ptx::tc_fence_after();
      tc_ld(lanes, D);
      if (is_k) {
#pragma unroll
        for (int u = 0; u < DVB / 8; ++u) {
          const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = 8 * u + 2 * e;
            const float v0 = __uint_as_float(w[e] << 16), v1 = __uint_as_float(w[e] & 0xFFFF0000u);
            D[j] = delta ? v0 - eg * D[j] : v0;
            D[j + 1] = delta ? v1 - eg * D[j + 1] : v1;
          }
        }
        store_row_split(sb + P::X_OFF, sb + P::X_OFF + P::X_PIECE, row, C * 16, D);
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(x_ready);
      } else {
#pragma unroll
        for (int j = 0; j < DVB; ++j) inter[j] = eg * D[j];
      }
      if (!(ok = warp_wait(d2, par, abort_flag, kFaultChain))) break;
      ptx::tc_fence_after();
      tc_ld(lanes + DVB, D);
      if (is_k) {
#pragma unroll
        for (int j = 0; j < DVB; ++j) D[j] *= erest;
        store_row_split(sb + P::U_OFF, sb + P::U_OFF + P::X_PIECE, row, C * 16, D);
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(u_ready);
      } else if (live) {
        __nv_bfloat16* o = a.o + tok * a.ldo + static_cast<int64_t>(h) * a.d_v + c0;
#pragma unroll
        for (int u = 0; u < DVB / 8; ++u) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = 8 * u + 2 * e;
            const __nv_bfloat162 p = __floats2bfloat162_rn(a.scale * (inter[j] + D[j]),
                                                           a.scale * (inter[j + 1] + D[j + 1]));
            w[e] = *reinterpret_cast<const uint32_t*>(&p);
          }
          *reinterpret_cast<uint4*>(o + 8 * u) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      if (!(ok = warp_wait(d3, par, abort_flag, kFaultChain))) break;
      ptx::tc_fence_after();
      tc_ld(lanes + 2 * DVB, D);
#pragma unroll
      for (int j = 0; j < DVB; ++j) S[j] = eall * S[j] + D[j];
    }
    if (ok && slot >= 0 && t < DK) {
#pragma unroll
      for (int j = 0; j < DVB / 4; ++j)
        reinterpret_cast<float4*>(state)[j] =
            make_float4(S[4 * j], S[4 * j + 1], S[4 * j + 2], S[4 * j + 3]);
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 4) {
    __syncwarp();
    ptx::tmem_dealloc(tmem, P::TMEM);
  }
}

}  // namespace la
}  // namespace nvfp4
