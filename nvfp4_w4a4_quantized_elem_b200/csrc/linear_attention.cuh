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
//   (I + L) U = X,  X = diag(beta) (V - diag(e^G) K S)
//     L_tj = beta_t e^{G_t-G_j} k_t.k_j for j < t
//   O = diag(e^G) Q S + A U,  A_tj = e^{G_t-G_j} q_t.k_j for j <= t
//   S' = e^{G_64} S + K^T U~,  U~ = diag(e^{G_64-G}) U
// so with T = (I + L)^-1:  [U; O - diag(e^G) Q S] = [T; A T] X. Three products
// per chunk depend on one another, [K; Q] S, [T; AT] X and K^T U~, all with
// 128 rows on the MMA's M side (tokens of K and Q together, then of U and O
// together, then d_k) and a block of d_v columns as its N. Without the delta
// rule T = I and X = V.
//
// Two kernels. prepare_kernel, parallel over chunks and heads, computes what
// does not depend on S: the swizzled bf16 image of [K; Q] (rows past a
// sequence's end zero), [T; AT] and the decay factors. chain_kernel walks a
// sequence's chunks in order, one CTA per (sequence, head, d_v block), with S
// in FP32 registers; plain_kernel takes its place without the delta rule.
// Measured: 8192 tokens, 16 key and 32 value heads of 128: prepare 98 us, chain
// 338 us (128 steps of 2.6 us); 7777 tokens in 23 prompts, 48 value heads: 150
// and 368 us, 500 together; 4096 tokens in 3 prompts, 24 heads of 64 x 128 without
// the delta rule: 21 and 75 to 102 us, by the longest prompt. All of them are bound
// by latency, the chains by that of their dependent products.
//
// Precision: q, k, v are bf16 and enter the products exactly. FP32 operands are
// cut into bf16 pieces, products accumulated in FP32. X and U~, on which the
// FP32 states rest directly, take three pieces (24 bits, nothing is lost); S,
// which returns into the state only through beta K S, and T and A T, whose unit
// diagonal is exact, take two (2^-18 of the value is lost). One bf16 operand
// alone would leave 2^-9 in the states. Measured, relative error of the states
// after 2048 tokens: 7e-7 with a layer's gates, 1.7e-6 with a hundredth of the
// decay, 3.1e-6 with beta up to 2 as well (the same chunks in FP32: 1.4e-7 to
// 3.4e-7; token by token in FP32: 2.6e-7 to 2.9e-6). With a third piece of S and
// T 2.5e-7 to 5.2e-7, the same outputs after their rounding to bf16, and 9 to 17%
// more time (8192 tokens of 32 heads 424 -> 493 us, 23 ragged prompts 501 -> 544):
// not taken. G is summed in FP64 and kept as two FP32 parts: the difference of two
// FP32 sums of strong decays would lose the weak decays between them.
//
// What is not finite. A chunk's products reach every row of it, with zeros where
// the recurrence has nothing, and zero times a NaN is one: an infinity or a NaN in a
// token also reaches the tokens before it in its chunk. The chains look at the
// outputs as they store them and, where one is not finite, go over the
// sequence again when they are through, token by token, with its outputs from that
// chunk on and its state from there.
#pragma once

#include <cuda_bf16.h>
#include <climits>
#include <cstdint>

#include "fault.cuh"
#include "ptx.cuh"

namespace nvfp4 {
namespace la {

constexpr int C = 64;                       // tokens per chunk
constexpr int kHalfBytes = 128 * 128;       // [K; Q] image: 128 rows x 64 of d_k
constexpr int kTTBytes = 128 * 128;         // [T; AT] image: 128 rows x 64, one piece
constexpr int kGateFloats = 3 * C + 4;      // e^G, e^{G_64 - G}, beta; e^{G_64}, valid word
constexpr int kGateBytes = (kGateFloats * 4 + 127) / 128 * 128;
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // per wait, unless a self-test sets less
constexpr uint64_t kDrainLimitNs = 100000000ull;

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
  uint64_t wait_limit_ns;
  // self-test: the CTA of the first or the second kernel whose first product or
  // first load is never issued (-1: none)
  int stall_prepare, stall_chain;
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

// An FP32 value is the sum of three bf16 values, its 24 bits cut 8 by 8: the
// upper half-word of x, of the (exact) rest, and of the rest of that. Takes the
// next piece of x and y, packed, and leaves the rests in them.
__device__ __forceinline__ uint32_t take_piece(float& x, float& y) {
  const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
  x -= __uint_as_float(a & 0xFFFF0000u);
  y -= __uint_as_float(b & 0xFFFF0000u);
  return __byte_perm(a, b, 0x7632);
}

// Two pieces are rounded instead: 2^-18 of the value is left.
__device__ __forceinline__ uint32_t round_piece(float x, float y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t take_rounded(float& x, float& y) {
  const uint32_t w = round_piece(x, y);
  x -= __uint_as_float(w << 16);
  y -= __uint_as_float(w & 0xFFFF0000u);
  return w;
}

// Row `k` of an MN-major operand without swizzle (8 x 16-byte core matrices,
// 128 bytes apart along k, `n_stride` bytes apart along n): 8 consecutive n.
__device__ __forceinline__ uint32_t mn_off(int k, int n8, int n_stride) {
  return static_cast<uint32_t>((k >> 3) * 128 + (k & 7) * 16 + n8 * n_stride);
}

// N FP32 values of operand row k -> PIECES bf16 pieces, `piece` bytes apart.
template <int PIECES, int N>
__device__ __forceinline__ void store_row_split(uint32_t base, int piece, int k, int n_stride,
                                                const float (&x)[N]) {
#pragma unroll
  for (int n8 = 0; n8 < N / 8; ++n8) {
    float r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = x[8 * n8 + e];
    const uint32_t at = base + mn_off(k, n8, n_stride);
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = PIECES == 2 ? take_rounded(r[2 * e], r[2 * e + 1])
                           : take_piece(r[2 * e], r[2 * e + 1]);
      ptx::st_shared_v4(at + p * piece, w[0], w[1], w[2], w[3]);
    }
  }
}

// 16-byte unit `u` of row r in a 128-byte-row, 128-byte-swizzled image.
__device__ __forceinline__ uint32_t sw128(int r, int u) {
  return static_cast<uint32_t>(r * 128 + ((u ^ (r & 7)) << 4));
}

// 32 FP32 values -> two rounded pieces each, packed in their place: of every 8
// values 4 words of first pieces, then 4 of second ones.
__device__ __forceinline__ void pack_row(float (&x)[32]) {
#pragma unroll
  for (int u = 0; u < 32; u += 8) {
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      w[e] = take_rounded(x[u + 2 * e], x[u + 2 * e + 1]);
      w[4 + e] = round_piece(x[u + 2 * e], x[u + 2 * e + 1]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) x[u + e] = __uint_as_float(w[e]);
  }
}

__device__ __forceinline__ void st_packed(uint32_t at, int piece, const float* x) {
#pragma unroll
  for (int p = 0; p < 2; ++p)
    ptx::st_shared_v4(at + p * piece, __float_as_uint(x[4 * p]), __float_as_uint(x[4 * p + 1]),
                      __float_as_uint(x[4 * p + 2]), __float_as_uint(x[4 * p + 3]));
}

// A packed row r, from its 16-byte unit u0 on -> hi and lo images of the rows
// (`piece` apart).
__device__ __forceinline__ void store_image_row(uint32_t base, int piece, int r, int u0,
                                                const float (&x)[32]) {
#pragma unroll
  for (int u = 0; u < 4; ++u) st_packed(base + sw128(r, u0 + u), piece, &x[8 * u]);
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

// The slow part of a wait, out of line: many tries between two looks at the
// clock, up to the limit.
__device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t parity,
                                       volatile uint32_t* abort_flag, uint32_t who,
                                       uint64_t limit_ns) {
  const uint64_t t0 = ptx::globaltimer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (ptx::mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (ptx::globaltimer_ns() - t0 > limit_ns) {
      *abort_flag = 1u;
      atomicOr(&g_fault_word, who);
      return false;
    }
  }
}

// Bounded wait: one try in line, the rest out of line (the waits of the chain
// are short and stand one behind the other).
__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity,
                                             volatile uint32_t* abort_flag, uint32_t who,
                                             uint64_t limit_ns) {
  return ptx::mbar_try_wait(bar, parity) || wait_long(bar, parity, abort_flag, who, limit_ns);
}

// Used only while aborting: wait for in-flight asynchronous work, bounded.
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = ptx::globaltimer_ns();
  while (!ptx::mbar_try_wait(bar, parity)) {
    if (ptx::globaltimer_ns() - t0 > kDrainLimitNs) return;
  }
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity,
                                          volatile uint32_t* abort_flag, uint32_t who,
                                          uint64_t limit_ns) {
  return __all_sync(0xFFFFFFFFu, wait_bounded(bar, parity, abort_flag, who, limit_ns));
}

// ------------------------------------------------------------------ prepare --

constexpr int kPrepThreads = 256;
constexpr int kLd = 68;                       // row pitch (floats) of the 64x64 tiles
constexpr int kTileBytes = C * kLd * 4;
constexpr int kMLd = 36;                      // row pitch of the inverse's 32x32 scratch
constexpr int kMBytes = 32 * kMLd * 4;

// Shared memory: the [K; Q] image, over which L and T = (I + L)^-1 are written
// once the scores are taken; T's pieces go over L, the two pieces of the
// [T; AT] image over T and, the product A T done, over T's pieces. A's pieces
// are the rows 64..127 of 128-row operands whose rows 0..63 lie in whatever
// stands before them: those rows of the product are not read. Four CTAs of 256
// threads per SM: the kernel is a chain of short dependent phases (20 K cycles
// a CTA among four: 5 K for K and Q to arrive, 6 K for L and its inverse), and
// what fills their gaps is other CTAs.
template <int DK>
struct PrepCfg {
  static constexpr int KQ = kq_bytes(DK);
  static constexpr int L_OFF = 0;
  static constexpr int T_OFF = kTileBytes;
  static constexpr int A_OFF = 2 * kTileBytes;             // hi rows, then lo rows
  static constexpr int A_PIECE = kTTBytes / 2;
  static constexpr int G_OFF = A_OFF + 2 * A_PIECE;        // G, beta
  static constexpr int M_OFF = G_OFF + C * 8 + C * 4;      // scratch of the inverse
  static constexpr int BAR_OFF = M_OFF + kMBytes;
  static constexpr int SMEM = BAR_OFF + 64;                // the base is 1024-byte aligned
  static_assert(KQ <= A_OFF && kTTBytes <= kTileBytes && kTileBytes % 1024 == 0 &&
                4 * (SMEM + 1024) <= 228 * 1024, "regions, four CTAs per SM");
};

// acc (16x8, FP32) += A (16 x 8 KS, row-major) B (8 KS x 8, row-major) by
// mma.sync.m16n8k8 on tf32: FP32 values as two tf32 pieces each, products
// hi hi + hi lo + lo hi (2^-21 of the operands' product is lost). The fragment
// loads are single words, 32 banks (A) or 16 (B) at a time.
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4],
                                         const uint32_t (&b)[2]) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
      " {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  hi = __float_as_uint(x) & 0xFFFFE000u;
  lo = __float_as_uint(x - __uint_as_float(hi));
}

__device__ __forceinline__ void tile_mac(float (&acc)[4], const float* A, int lda, const float* B,
                                         int ldb, int steps, int lane) {
  const int g = lane >> 2, q = lane & 3;
  for (int k = 0; k < 8 * steps; k += 8) {
    uint32_t ah[4], al[4], bh[2], bl[2];
    split_tf32(A[g * lda + k + q], ah[0], al[0]);
    split_tf32(A[(g + 8) * lda + k + q], ah[1], al[1]);
    split_tf32(A[g * lda + k + q + 4], ah[2], al[2]);
    split_tf32(A[(g + 8) * lda + k + q + 4], ah[3], al[3]);
    split_tf32(B[(k + q) * ldb + g], bh[0], bl[0]);
    split_tf32(B[(k + q + 4) * ldb + g], bh[1], bl[1]);
    mma_tf32(acc, al, bh);
    mma_tf32(acc, ah, bl);
    mma_tf32(acc, ah, bh);
  }
}

__device__ __forceinline__ void tile_store(float* D, int ld, const float (&acc)[4], float sign,
                                           int lane) {
  const int g = lane >> 2, c = 2 * (lane & 3);
  *reinterpret_cast<float2*>(D + g * ld + c) = make_float2(sign * acc[0], sign * acc[1]);
  *reinterpret_cast<float2*>(D + (g + 8) * ld + c) = make_float2(sign * acc[2], sign * acc[3]);
}

// T = (I + L)^-1 for the strictly lower triangular L: the 16x16 diagonal blocks
// by FP32 forward substitution, one thread per column, then twice
// [P 0; B Q]^-1 = [P^-1 0; -Q^-1 B P^-1 Q^-1], with 16- and 32-wide blocks on split
// tf32 tiles, 16x8 each, zero k-steps of the triangles left out. (On the FP32
// units these products read shared memory 16 bytes a lane for every few
// multiply-adds and were what bounded the whole kernel: 73% of the shared
// memory's bandwidth.) T's 16x16 blocks above the diagonal are not written.
//
// The 32x32 block at (o, o), by the warp that wrote L there: no other warp is
// waited for, and those of A work meanwhile.
__device__ __forceinline__ void invert_block(const float* L, float* T, float* M, int o, int lane) {
  L += o * kLd + o;
  T += o * kLd + o;
  {
    const int b0 = lane & 16, j = lane & 15;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s[4] = {i == j ? 1.0f : 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int m = 0; m < i; m += 4) {
        const float4 l = *reinterpret_cast<const float4*>(L + (b0 + i) * kLd + b0 + m);
        s[0] -= l.x * x[m];
        if (m + 1 < i) s[1] -= l.y * x[m + 1];
        if (m + 2 < i) s[2] -= l.z * x[m + 2];
        if (m + 3 < i) s[3] -= l.w * x[m + 3];
      }
      x[i] = i < j ? 0.0f : (s[0] + s[1]) + (s[2] + s[3]);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) T[(b0 + i) * kLd + b0 + j] = x[i];
  }
  __syncwarp();
  float acc[2][4] = {};
#pragma unroll
  for (int c = 0; c < 2; ++c) tile_mac(acc[c], L + 16 * kLd, kLd, T + 8 * c, kLd, 2, lane);
#pragma unroll
  for (int c = 0; c < 2; ++c) tile_store(M + 8 * c, kMLd, acc[c], 1.0f, lane);
  __syncwarp();
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    acc[c][0] = acc[c][1] = acc[c][2] = acc[c][3] = 0.0f;
    tile_mac(acc[c], T + 16 * kLd + 16, kLd, M + 8 * c, kMLd, 2, lane);
  }
#pragma unroll
  for (int c = 0; c < 2; ++c) tile_store(T + 16 * kLd + 8 * c, kLd, acc[c], -1.0f, lane);
}

// The 32x32 block below the diagonal, by all eight warps: row tile i, column
// tile j; the second product needs both row tiles of the first.
__device__ __forceinline__ void invert_below(const float* L, float* T, float* M, int warp,
                                             int lane) {
  const int i = warp >> 2, j = warp & 3;
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  tile_mac(acc, L + (32 + 16 * i) * kLd + 8 * j, kLd, T + 8 * j * kLd + 8 * j, kLd, 4 - j, lane);
  tile_store(M + 16 * i * kMLd + 8 * j, kMLd, acc, 1.0f, lane);
  switch (j) {  // the two warps of column tile j
    case 0: asm volatile("bar.sync 1, 64;" ::: "memory"); break;
    case 1: asm volatile("bar.sync 2, 64;" ::: "memory"); break;
    case 2: asm volatile("bar.sync 3, 64;" ::: "memory"); break;
    default: asm volatile("bar.sync 4, 64;" ::: "memory"); break;
  }
  acc[0] = acc[1] = acc[2] = acc[3] = 0.0f;
  tile_mac(acc, T + (32 + 16 * i) * kLd + 32, kLd, M + 8 * j, kMLd, 2 + 2 * i, lane);
  tile_store(T + (32 + 16 * i) * kLd + 8 * j, kLd, acc, -1.0f, lane);
}

// x[j] (column j0 + j) *= f e^{G_t - G_j} up to column `last`, zero beyond (a
// score that is not finite, too). Without branches: a branch per block of
// columns puts x into local memory.
__device__ __forceinline__ void decay_row(float (&x)[32], const float2* G, int row, int j0,
                                          int last, float f) {
  const float2 gt = G[row];
#pragma unroll
  for (int j = 0; j < 32; j += 2) {
    const float4 g = *reinterpret_cast<const float4*>(G + j0 + j);
    const float e0 = f * ptx::ex2((gt.x - g.x) + (gt.y - g.y));
    const float e1 = f * ptx::ex2((gt.x - g.z) + (gt.y - g.w));
    x[j] = j0 + j <= last ? e0 * x[j] : 0.0f;
    x[j + 1] = j0 + j + 1 <= last ? e1 * x[j + 1] : 0.0f;
  }
}

template <int DK>
__global__ void __launch_bounds__(kPrepThreads, 4)
    prepare_kernel(const Args a) {
  using P = PrepCfg<DK>;
  extern __shared__ __align__(1024) uint8_t smem_la[];
  uint8_t* const smem = smem_la;
  float* const L = reinterpret_cast<float*>(smem + P::L_OFF);
  float* const T = reinterpret_cast<float*>(smem + P::T_OFF);
  float* const M = reinterpret_cast<float*>(smem + P::M_OFF);
  float2* const G = reinterpret_cast<float2*>(smem + P::G_OFF);  // G log2(e), two parts
  float* const Beta = reinterpret_cast<float*>(G + C);
  uint64_t* const bar = reinterpret_cast<uint64_t*>(smem + P::BAR_OFF);
  uint32_t* const tmem_holder = reinterpret_cast<uint32_t*>(bar + 1);
  volatile uint32_t* const abort_flag = tmem_holder + 1;
  int2* const found = reinterpret_cast<int2*>(bar + 2);  // the chunk's first token, its tokens
  uint64_t* const drain = bar + 3;

  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int h = blockIdx.x % a.h_v, group = a.h_v / a.h_k, hk = h / group;
  const int slot = blockIdx.x / a.h_v;
  if (t == 0) {
    ptx::mbar_init(bar, 1);
    ptx::mbar_init(drain, 1);
    *found = make_int2(0, 0);
    // the swizzled images need the alignment that the declaration asks for
    *abort_flag = (ptx::smem_u32(smem) & 1023u) != 0u ? 1u : 0u;
    if (*abort_flag) atomicOr(&g_fault_word, kFaultPrepare);
    ptx::fence_mbarrier_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(tmem_holder, 128);
    ptx::tmem_relinquish();
  }
  // The chain's CTAs may start only when every CTA here has its tensor memory:
  // they take theirs and wait for this grid.
  __syncthreads();
  ptx::grid_dep_launch();
  ptx::grid_dep_wait();
  // the sequence that has this slot, if one does
  for (int i = t; i < a.n_seq; i += kPrepThreads) {
    int start, end;
    seq_range(a, i, start, end);
    const int64_t c = slot - first_slot(start, i), left = end - start - c * C;
    if (c >= 0 && left > 0)
      *found = make_int2(start + static_cast<int>(c) * C, static_cast<int>(min(left, int64_t{C})));
  }
  __syncthreads();
  const int64_t tok0 = found->x;
  const int len = found->y;
  if (len == 0) {  // a slot between two sequences' chunks
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 1) ptx::tmem_dealloc(*tmem_holder, 128);
    return;
  }

  // decays and beta, requested before the keys, whose loads cover them (as
  // FP32: a conversion here would wait for them)
  float g0 = 0.0f, g1 = 0.0f;
  float bt = 0.0f;
  if (warp == 0) {
    const float* g = a.decay + tok0 * a.h_v + h;
    if (2 * lane < len) g0 = g[static_cast<int64_t>(2 * lane) * a.h_v];
    if (2 * lane + 1 < len) g1 = g[static_cast<int64_t>(2 * lane + 1) * a.h_v];
  } else if (t >= 64 && t < 128 && t - 64 < len) {
    bt = a.beta != nullptr ? a.beta[(tok0 + t - 64) * a.h_v + h] : 1.0f;
  }
  // [K; Q] -> the swizzled image, rows past the sequence zero; the group's
  // first head also writes it out
  {
    constexpr int kUnits = DK / 8;            // 16-byte units per row
    constexpr int kStep = kPrepThreads / kUnits;  // rows per pass
    uint8_t* const image = a.kq + (static_cast<int64_t>(slot) * a.h_k + hk) * P::KQ;
    const int u = t % kUnits;
    uint4 x[128 / kStep];
#pragma unroll
    for (int i = 0; i < 128 / kStep; ++i) {
      const int r = t / kUnits + i * kStep, tok = r & (C - 1);
      x[i] = make_uint4(0u, 0u, 0u, 0u);
      if (tok < len) {
        const __nv_bfloat16* row = r < C ? a.k + (tok0 + tok) * a.ldk : a.q + (tok0 + tok) * a.ldq;
        x[i] = *reinterpret_cast<const uint4*>(row + static_cast<int64_t>(hk) * DK + 8 * u);
      }
    }
#pragma unroll
    for (int i = 0; i < 128 / kStep; ++i) {
      const int r = t / kUnits + i * kStep;
      const uint32_t off = (u / 8) * kHalfBytes + sw128(r, u % 8);
      *reinterpret_cast<uint4*>(smem + off) = x[i];
      if (h % group == 0) *reinterpret_cast<uint4*>(image + off) = x[i];
    }
  }
  if (warp == 0) {
    // G in FP64 (a decay of e^-1000 is zero, so -inf counts as that)
    constexpr double kLog2e = 1.4426950408889634;
    const double x0 = (g0 < -1000.0f ? -1000.0 : static_cast<double>(g0)) * kLog2e;
    const double x1 = (g1 < -1000.0f ? -1000.0 : static_cast<double>(g1)) * kLog2e;
    double s = x0 + x1;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const double y = __shfl_up_sync(0xFFFFFFFFu, s, d);
      if (lane >= d) s += y;
    }
    // (a token's decay does not reach the one before it)
    const double before = __shfl_up_sync(0xFFFFFFFFu, s, 1);
    const double s0 = fabs(x1) < INFINITY ? s - x1 : (lane > 0 ? before : 0.0) + x0;
    const float h0 = static_cast<float>(s0), h1 = static_cast<float>(s);
    G[2 * lane] = make_float2(h0, static_cast<float>(s0 - h0));
    G[2 * lane + 1] = make_float2(h1, static_cast<float>(s - h1));
  } else if (t >= 64 && t < 128) {
    Beta[t - 64] = bt;
  }
  ptx::fence_proxy_async_smem();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const uint32_t sb = ptx::smem_u32(smem);
  bool ok = *abort_flag == 0u;
  if (t == 0 && ok && a.stall_prepare != static_cast<int>(blockIdx.x)) {
    // [K; Q] K^T: 128 x 64
    constexpr uint32_t kScores = ptx::idesc_bf16(128, C, false, false);
#pragma unroll
    for (int s = 0; s < DK / 16; ++s) {
      const uint64_t d = ptx::smem_desc(sb + (s / 4) * kHalfBytes + (s % 4) * 32, 16, 1024, 2);
      ptx::tc_mma_bf16(tmem, d, d, kScores, s != 0);
    }
    ptx::tc_commit(bar);
  }
  ok = ok && warp_wait(bar, 0, abort_flag, kFaultPrepare, a.wait_limit_ns);
  ptx::tc_fence_after();
  __syncthreads();  // every warp saw the scores: L may go over their operands
  // this thread: row r of the 128 (a token's row of L and T, then of A and AT),
  // columns [j0, j0 + 32)
  const int r = (warp & 3) * 32 + lane, row = r & (C - 1), j0 = 32 * (warp >> 2);
  const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + j0;
  const bool delta = a.beta != nullptr;
  uint8_t* const out = a.tt + (static_cast<int64_t>(slot) * a.h_v + h) * kHeadBytes;
  // all of this warp's 32 x 32 block lies above the diagonal, of every matrix here
  const bool above = j0 > (row | 31);
  float x[32];  // from pack_row() on, packed pieces
  if (above) {
#pragma unroll
    for (int j = 0; j < 32; ++j) x[j] = 0.0f;
  } else {
    tc_ld(lanes, x);
  }
  if (r < C) {
    const float f = Beta[row];
    if (j0 == 0) {
      const float2 gt = G[row], ge = G[C - 1];
      float* gate = reinterpret_cast<float*>(out + 2 * kTTBytes);
      gate[row] = ptx::ex2(gt.x + gt.y);
      gate[C + row] = ptx::ex2((ge.x - gt.x) + (ge.y - gt.y));
      gate[2 * C + row] = f;
      if (row == 0) gate[3 * C] = ptx::ex2(ge.x + ge.y);
    }
    if (delta) {
      if (!above) {
        decay_row(x, G, row, j0, row - 1, f);
#pragma unroll
        for (int j = 0; j < 32; j += 4)
          *reinterpret_cast<float4*>(L + row * kLd + j0 + j) =
              make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
        if (j0 == (row & 32)) {  // warps 0 and 5: the blocks on the diagonal
          __syncwarp();
          invert_block(L, T, M + 16 * kMLd * (j0 >> 5), j0, lane);
        }
      }
    }
  } else {
    if (!above) {
      decay_row(x, G, row, j0, row, 1.0f);
      pack_row(x);
    }
    if (delta) store_image_row(sb + P::A_OFF, P::A_PIECE, row, j0 / 8, x);  // rows from a multiple of 8
  }
  if (delta) {
    __syncthreads();
    invert_below(L, T, M, warp, lane);
    __syncthreads();
    if (r < C) {
      if (!above) {
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (j0 + j <= (row | 15)) v = *reinterpret_cast<const float4*>(T + row * kLd + j0 + j);
          x[j] = v.x; x[j + 1] = v.y; x[j + 2] = v.z; x[j + 3] = v.w;
        }
        pack_row(x);
      }
      // over L, which the inverse no longer needs
#pragma unroll
      for (int n8 = 0; n8 < 4; ++n8)
        st_packed(sb + P::L_OFF + mn_off(row, j0 / 8 + n8, 1024), 8192, &x[8 * n8]);
    }
    ptx::fence_proxy_async_smem();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (t == 0 && ok) {
      // A T as A_hi [T_hi | T_lo] + A_lo T_hi over the scores, the two column
      // blocks added by the reader
      constexpr uint32_t kBoth = ptx::idesc_bf16(128, 2 * C, false, true);
      constexpr uint32_t kOne = ptx::idesc_bf16(128, C, false, true);
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int s = 0; s < C / 16; ++s)
          ptx::tc_mma_bf16(tmem,
                           ptx::smem_desc(sb + P::A_OFF + (p - 1) * P::A_PIECE + s * 32, 16, 1024, 2),
                           ptx::smem_desc(sb + P::L_OFF + s * 256, 128, 1024, 0),
                           p == 0 ? kBoth : kOne, (p | s) != 0);
      ptx::tc_commit(bar);
    }
    ok = ok && warp_wait(bar, 1, abort_flag, kFaultPrepare, a.wait_limit_ns);
    ptx::tc_fence_after();
    if (r >= C && !above) {
      float y[32];
      tc_ld(lanes, x);
      tc_ld(lanes + C, y);
#pragma unroll
      for (int j = 0; j < 32; ++j) x[j] += y[j];
      pack_row(x);
    }
    __syncthreads();  // every warp saw the product done: the image may go over T's pieces
  }
  // hi image at T_OFF, lo image at L_OFF; without the delta rule A itself stands
  // in the place of AT, and T = I is left out
  if (delta || r >= C) store_image_row(sb + P::T_OFF, P::L_OFF - P::T_OFF, r, j0 / 8, x);
  ptx::fence_proxy_async_smem();
  ptx::tc_fence_before();
  __syncthreads();
  // A CTA that gave up says so to the chains, which then leave their states
  // alone, and lets its products end before their tensor memory goes.
  const bool failed = *abort_flag != 0u;  // (not written behind the barrier above)
  if (t == 0) {
    reinterpret_cast<uint32_t*>(out + 2 * kTTBytes)[3 * C + 1] = failed ? 0u : 1u;
    if (failed) {
      ptx::tc_commit(drain);
      drain_wait(drain, 0);
    } else {
      const int skip = delta ? 0 : kTTBytes / 2;
      ptx::bulk_store(out + skip, smem + P::T_OFF + skip, kTTBytes - skip);
      ptx::bulk_store(out + kTTBytes + skip, smem + P::L_OFF + skip, kTTBytes - skip);
      ptx::bulk_commit_group();
      // (the grid's end waits for the writes; the CTA only for its shared memory)
      ptx::bulk_wait_group_read<0>();
    }
  }
  if (failed) __syncthreads();
  ptx::tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    ptx::tmem_dealloc(tmem, 128);
  }
}

// -------------------------------------------------------------------- chain --

constexpr int kSPieces = 2, kPieces = 3;   // of S; of X and U~
constexpr int kCols = 16;                  // columns of d_v per compute thread

// The pieces of an operand lie side by side on the N side, [hi | mid | lo], and
// the reader adds the column blocks of the result: an MMA with 128 rows and K
// = 16 takes 30 cycles for 32 columns and 50 for 96 (measured), behind ~300
// cycles from its issue to the arrival of its commit, so pieces in N cost less
// than pieces one after the other. Compute threads hold one row, 16 columns
// wide (the splitting stands on the critical path: 32 columns a thread took 400
// cycles more per operand, 8 no fewer); one more warp loads and issues the MMAs.
// (The kernel of the delta rule; the plain one is below.)
// A step of one chunk is a chain of latencies (4.4 K cycles, 1.2 K of them in
// MMAs), so two CTAs share an SM and fill each other's gaps; for that the
// shared memory is cut to half an SM's: S, X and U~ take turns in one region,
// [T; AT] has one buffer (reloaded behind its product, two products ahead of
// its next use), only [K; Q] two. D1 and D3 share tensor-memory columns. 64
// columns per CTA and one CTA per SM took 6.8 K cycles per step.
// DVB columns of d_v per CTA: 32, or 16 where those CTAs are no more than the
// SMs. The MMAs read their 128 rows from shared memory whatever their columns,
// so 16 do not halve a step, but shorten it: 8192 tokens of 8 and 16 heads of 128
// take 306 and 330 us, 356 and 381 with 32 columns; of 32 heads 461 against 426.
template <int DK, int DVB>
struct ChainCfg {
  static constexpr int WARPS = 4 * (DVB / kCols);
  static constexpr int THREADS = 32 * WARPS + 32;
  static constexpr int S_PIECE = DK * DVB * 2;
  static constexpr int X_PIECE = C * DVB * 2;
  static constexpr int TT_OFF = 2 * kq_bytes(DK);
  static constexpr int R_OFF = TT_OFF + 2 * kTTBytes;
  static constexpr int R_BYTES = kSPieces * S_PIECE > kPieces * X_PIECE ? kSPieces * S_PIECE
                                                                        : kPieces * X_PIECE;
  static constexpr int BAR_OFF = R_OFF + R_BYTES;
  static constexpr int SMEM = BAR_OFF + 128;   // the base is 1024-byte aligned
  static constexpr uint32_t D2_COL = kPieces * DVB;
  static constexpr uint32_t TMEM = DVB == 32 ? 256 : 128;
  static_assert(2 * (SMEM + 1024) <= 228 * 1024 && 2 * D2_COL <= TMEM, "two CTAs per SM");
};

// The pool slot of sequence b, or -1: only the first sequence that names a slot
// has it. Called by whole warps.
__device__ __forceinline__ int state_slot(const Args& a, int b, int lane) {
  if (a.state == nullptr) return -1;
  const int slot = a.slots != nullptr ? a.slots[b] : b;
  if (slot < 0 || slot >= a.n_slots) return -1;
  int earlier = 0;
  if (a.slots != nullptr)
    for (int i = lane; i < b; i += 32) earlier |= a.slots[i] == slot;
  return __any_sync(0xFFFFFFFFu, earlier) ? -1 : slot;
}

// 16 columns of a state row, zero unless the sequence resumes.
__device__ __forceinline__ void load_state(const Args& a, bool has, int b, const float* row,
                                           float (&S)[kCols]) {
#pragma unroll
  for (int j = 0; j < kCols; ++j) S[j] = 0.0f;
  if (has && a.resume != nullptr && a.resume[b] != 0) {
#pragma unroll
    for (int j = 0; j < kCols / 4; ++j) {
      const float4 x = reinterpret_cast<const float4*>(row)[j];
      S[4 * j] = x.x; S[4 * j + 1] = x.y; S[4 * j + 2] = x.z; S[4 * j + 3] = x.w;
    }
  }
}

__device__ __forceinline__ void store_state(float* row, const float (&S)[kCols]) {
#pragma unroll
  for (int j = 0; j < kCols / 4; ++j)
    reinterpret_cast<float4*>(row)[j] = make_float4(S[4 * j], S[4 * j + 1], S[4 * j + 2], S[4 * j + 3]);
}

// Whether prepare_kernel finished the chunk with this word (the same for the
// whole CTA); if not, the CTA's other warps are told to stop.
__device__ __forceinline__ bool prepared(float word, volatile uint32_t* abort_flag) {
  if (__float_as_uint(word) == 1u) return true;
  *abort_flag = 1u;
  return false;
}

struct StateRow {
  float x[kCols];
};

// The tokens [tok, end) one by one, by the four warps that hold the rows of 16
// columns of S: as step_kernel does, with the sums over d_k by shuffles and, between
// the warps, through `scratch`, two tokens' worth in turns (one barrier a token).
// Outputs from token `from` on.
static_assert(2 * kCols == 32, "a sum per lane");
constexpr int kTokenFloats = 2 * kCols + 1;            // S^T k, S^T q, q.k of a warp's rows
constexpr int kScratchBytes = 2 * 4 * kTokenFloats * 4;   // per 16 columns

template <int DK>
__device__ __noinline__ StateRow token_by_token(const Args& a, float* scratch, int64_t tok, int64_t end,
                                                int64_t from, int h, int64_t col, int warp, int lane,
                                                StateRow S) {
  const int k_row = (warp & 3) * 32 + lane, hk = h / (a.h_v / a.h_k);
  const bool live = k_row < DK;
  const int64_t at = static_cast<int64_t>(hk) * DK + k_row;
  // a token's inputs, asked for a token ahead
  __nv_bfloat16 k = {}, q = {};
  float g = 0.0f, beta = 0.0f;
  uint4 v[kCols / 8];
  const auto fetch = [&](int64_t t) {
    if (live) {
      k = a.k[t * a.ldk + at];
      q = a.q[t * a.ldq + at];
    }
    g = a.decay[t * a.h_v + h];
    if (a.beta != nullptr) beta = a.beta[t * a.h_v + h];
#pragma unroll
    for (int u = 0; u < kCols / 8; ++u)
      v[u] = *reinterpret_cast<const uint4*>(a.v + t * a.ldv + col + 8 * u);
  };
  if (tok < end) fetch(tok);
#pragma unroll 1
  for (int turn = 0; tok < end; ++tok, turn ^= 1) {
    const float kk = __bfloat162float(k), qq = __bfloat162float(q), e = expf(g), b = beta;
    uint4 vv[kCols / 8];
#pragma unroll
    for (int u = 0; u < kCols / 8; ++u) vv[u] = v[u];
    if (tok + 1 < end) fetch(tok + 1);
    // 32 sums over the lanes, halved as they go: lane i is left with sum i
    float x[2 * kCols], qk = live ? kk * qq : 0.0f;
#pragma unroll
    for (int j = 0; j < kCols; ++j) {
      x[j] = live ? kk * S.x[j] : 0.0f;
      x[kCols + j] = live ? qq * S.x[j] : 0.0f;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
#pragma unroll
      for (int j = 0; j < d; ++j) {
        const bool up = (lane & d) != 0;
        const float give = up ? x[j] : x[j + d], keep = up ? x[j + d] : x[j];
        x[j] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, d);
      }
      qk += __shfl_xor_sync(0xFFFFFFFFu, qk, d);
    }
    float* const all = scratch + turn * 4 * kTokenFloats;
    float* const mine = all + (warp & 3) * kTokenFloats;
    mine[lane] = x[0];
    if (lane == 0) mine[2 * kCols] = qk;
    if (warp < 4)  // the warps of these columns
      asm volatile("bar.sync 1, 128;" ::: "memory");
    else
      asm volatile("bar.sync 2, 128;" ::: "memory");
    const auto sum = [&](int j) {
      return (all[j] + all[kTokenFloats + j]) + (all[2 * kTokenFloats + j] + all[3 * kTokenFloats + j]);
    };
    qk = sum(2 * kCols);
#pragma unroll
    for (int j = 0; j < kCols; ++j) {
      const uint4& w = vv[j / 8];
      const uint32_t pair = j % 8 < 2 ? w.x : j % 8 < 4 ? w.y : j % 8 < 6 ? w.z : w.w;
      const float vj = __uint_as_float((j & 1) != 0 ? pair & 0xFFFF0000u : pair << 16);
      const float u = a.beta != nullptr ? b * (vj - e * sum(j)) : vj;
      if (k_row == 0 && tok >= from)
        a.o[tok * a.ldo + col + j] = __float2bfloat16_rn(a.scale * (e * sum(kCols + j) + qk * u));
      S.x[j] = live ? e * S.x[j] + kk * u : 0.0f;
    }
  }
  return S;
}

// o = scale (e^G (Q S) + A U), 16 columns of one token. Whether one of them is not
// finite: 0 x is 0 or NaN.
__device__ __forceinline__ bool store_out(__nv_bfloat16* o, float scale, float eg,
                                          const float (&qs)[kCols], const float (&au)[kCols]) {
  const __nv_bfloat162 zero = __floats2bfloat162_rn(0.0f, 0.0f);
  __nv_bfloat162 z = zero;
#pragma unroll
  for (int u = 0; u < kCols / 8; ++u) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = 8 * u + 2 * e;
      w[e] = round_piece(scale * (eg * qs[j] + au[j]), scale * (eg * qs[j + 1] + au[j + 1]));
      z = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w[e]), zero, z);
    }
    *reinterpret_cast<uint4*>(o + 8 * u) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return (*reinterpret_cast<const uint32_t*>(&z) & 0x7FFF7FFFu) != 0u;
}

// This thread's 16 columns of the BLOCKS column blocks of a result, added.
template <int BLOCKS, int DVB>
__device__ __forceinline__ void ld_sum(uint32_t taddr, float (&x)[kCols]) {
  float y[BLOCKS - 1][kCols];
  ptx::tc_ld_32x32b_x16(taddr, x);
#pragma unroll
  for (int i = 0; i < BLOCKS - 1; ++i) ptx::tc_ld_32x32b_x16(taddr + (i + 1) * DVB, y[i]);
  ptx::tc_wait_ld();
#pragma unroll
  for (int j = 0; j < kCols; ++j)
#pragma unroll
    for (int i = 0; i < BLOCKS - 1; ++i) x[j] += y[i][j];
}

template <int DK, int DVB>
__global__ void __launch_bounds__(ChainCfg<DK, DVB>::THREADS, 2)
    chain_kernel(const __grid_constant__ Args a) {
  using P = ChainCfg<DK, DVB>;
  extern __shared__ __align__(1024) uint8_t smem_la[];
  uint8_t* const smem = smem_la;
  uint64_t* const full = reinterpret_cast<uint64_t*>(smem + P::BAR_OFF);  // [2] K; Q loaded
  uint64_t* const s_ready = full + 2;   // operand pieces written by the compute warps
  uint64_t* const x_ready = full + 3;
  uint64_t* const u_ready = full + 4;
  uint64_t* const d1 = full + 5;        // products complete
  uint64_t* const d2 = full + 6;
  uint64_t* const d3 = full + 7;
  uint64_t* const full_tt = full + 8;   // T; AT loaded
  uint64_t* const drain = full + 9;
  uint32_t* const tmem_holder = reinterpret_cast<uint32_t*>(full + 10);
  volatile uint32_t* const abort_flag = tmem_holder + 1;
  int* const not_finite = reinterpret_cast<int*>(tmem_holder + 2);  // first such chunk

  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int blocks = a.d_v / DVB;
  const int c0 = (blockIdx.x % blocks) * DVB;
  const int h = (blockIdx.x / blocks) % a.h_v;
  const int b = blockIdx.x / blocks / a.h_v;
  const int hk = h / (a.h_v / a.h_k);
  constexpr int kMmaWarp = P::WARPS;
  if (t == 0) {
    ptx::mbar_init(&full[0], 1);
    ptx::mbar_init(&full[1], 1);
    ptx::mbar_init(s_ready, P::WARPS);
    ptx::mbar_init(x_ready, P::WARPS);
    ptx::mbar_init(u_ready, P::WARPS / 2);
    ptx::mbar_init(d1, 1);
    ptx::mbar_init(d2, 1);
    ptx::mbar_init(d3, 1);
    ptx::mbar_init(full_tt, 1);
    ptx::mbar_init(drain, 1);
    *not_finite = INT_MAX;
    // the swizzled images need the alignment that the declaration asks for
    *abort_flag = (ptx::smem_u32(smem) & 1023u) != 0u ? 1u : 0u;
    if (*abort_flag) atomicOr(&g_fault_word, kFaultChain);
    ptx::fence_mbarrier_init();
  }
  if (warp == kMmaWarp) {
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

  if (warp == kMmaWarp) {
    if (lane == 0) {
      auto load_kq = [&](int c) {
        ptx::mbar_arrive_expect_tx(&full[c & 1], kq_bytes(DK));
        ptx::bulk_load(smem + (c & 1) * kq_bytes(DK),
                       a.kq + ((static_cast<int64_t>(slot0) + c) * a.h_k + hk) * kq_bytes(DK),
                       kq_bytes(DK), &full[c & 1]);
      };
      auto load_tt = [&](int c) {
        ptx::mbar_arrive_expect_tx(full_tt, 2 * kTTBytes);
        ptx::bulk_load(smem + P::TT_OFF,
                       a.tt + ((static_cast<int64_t>(slot0) + c) * a.h_v + h) * kHeadBytes,
                       2 * kTTBytes, full_tt);
      };
      constexpr uint32_t kI1 = ptx::idesc_bf16(128, kSPieces * DVB, false, true);
      constexpr uint32_t kI2 = ptx::idesc_bf16(128, kPieces * DVB, false, true);
      constexpr uint32_t kI2lo = ptx::idesc_bf16(128, 2 * DVB, false, true);
      constexpr uint32_t kI3 = ptx::idesc_bf16(128, kPieces * DVB, true, true);
      constexpr uint32_t kSN = DK * 16, kXN = C * 16;  // bytes between groups of 8 columns
      const uint32_t r = sb + P::R_OFF, tt = sb + P::TT_OFF;
      int kq_asked = 0, kq_seen = 0, tt_asked = 0, tt_seen = 0;  // chunks
      bool ok = *abort_flag == 0u;
      if (n > 0 && ok) {
        if (a.stall_chain != static_cast<int>(blockIdx.x)) load_kq(kq_asked++);
        load_tt(tt_asked++);
      }
      for (int c = 0; c < n && ok; ++c) {
        const uint32_t par = c & 1;
        const uint32_t kq = sb + par * kq_bytes(DK);
        ok = wait_bounded(&full[par], (c >> 1) & 1, abort_flag, kFaultChainMma, a.wait_limit_ns);
        if (!ok) break;
        ++kq_seen;
        ok = wait_bounded(s_ready, par, abort_flag, kFaultChainMma, a.wait_limit_ns);
        if (!ok) break;
        ptx::tc_fence_after();
#pragma unroll
        for (int s = 0; s < DK / 16; ++s)   // [K; Q] S
          ptx::tc_mma_bf16(tmem, ptx::smem_desc(kq + (s / 4) * kHalfBytes + (s % 4) * 32, 16, 1024, 2),
                           ptx::smem_desc(r + s * 256, 128, kSN, 0), kI1, s != 0);
        ptx::tc_commit(d1);
        // S in place means that the previous chunk's products, the last
        // readers of the other buffer, are complete
        if (c + 1 < n) load_kq(kq_asked++);
        ok = wait_bounded(full_tt, par, abort_flag, kFaultChainMma, a.wait_limit_ns);
        if (!ok) break;
        ++tt_seen;
        ok = wait_bounded(x_ready, par, abort_flag, kFaultChainMma, a.wait_limit_ns);
        if (!ok) break;
        ptx::tc_fence_after();
#pragma unroll
        for (int p = 0; p < 2; ++p)   // [T; AT] X: hi with all of X, lo with its hi and mid
#pragma unroll
          for (int s = 0; s < C / 16; ++s)
            ptx::tc_mma_bf16(tmem + P::D2_COL, ptx::smem_desc(tt + p * kTTBytes + s * 32, 16, 1024, 2),
                             ptx::smem_desc(r + s * 256, 128, kXN, 0), p == 0 ? kI2 : kI2lo,
                             (p | s) != 0);
        ptx::tc_commit(d2);
        ok = wait_bounded(u_ready, par, abort_flag, kFaultChainMma, a.wait_limit_ns);
        if (!ok) break;
        ptx::tc_fence_after();
#pragma unroll
        for (int s = 0; s < C / 16; ++s)   // K^T U~ (64 of d_k: the upper rows repeat the lower)
          ptx::tc_mma_bf16(tmem, ptx::smem_desc(kq + s * 2048, DK == 128 ? kHalfBytes : 0, 1024, 2),
                           ptx::smem_desc(r + s * 256, 128, kXN, 0), kI3, s != 0);
        ptx::tc_commit(d3);
        if (c + 1 < n) load_tt(tt_asked++);  // U~ in place means [T; AT] X complete
      }
      if (!ok) {  // let what is in flight end before the CTA does
        ptx::tc_commit(drain);
        drain_wait(drain, 0);
        for (int c = kq_seen; c < kq_asked; ++c) drain_wait(&full[c & 1], (c >> 1) & 1);
        if (tt_seen < tt_asked) drain_wait(full_tt, tt_seen & 1);
      } else if (n > 0) {
        drain_wait(d3, (n - 1) & 1);  // the last product, should the others give up on it
      }
    }
  } else {
    const int k_row = (warp & 3) * 32 + lane;   // row of d_k
    const int row = k_row & (C - 1);            // token of the chunk
    const bool is_k = (warp & 3) < 2;           // rows of K and U; else rows of Q and O
    const int cols = (warp >> 2) * kCols;       // this thread's columns of the block
    const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + cols;
    const int slot = state_slot(a, b, lane);
    const int64_t col = static_cast<int64_t>(h) * a.d_v + c0 + cols;  // column of V and O
    float* const state = a.state + ((static_cast<int64_t>(slot) * a.h_v + h) * DK + k_row) * a.d_v +
                         c0 + cols;
    float S[kCols];
    load_state(a, slot >= 0 && k_row < DK, b, state, S);
    // what the next chunk needs from memory, requested a chunk ahead
    float eg = 0.0f, erest = 0.0f, bt = 0.0f;
    float2 all = make_float2(0.0f, 0.0f);   // e^{G_64}; the word that says the chunk was prepared
    uint4 v[kCols / 8];
    auto fetch = [&](int c) {
      const int64_t tok = start + static_cast<int64_t>(c) * C + row;
      const float* gate = reinterpret_cast<const float*>(
          a.tt + (static_cast<int64_t>(slot0 + c) * a.h_v + h) * kHeadBytes + 2 * kTTBytes);
      eg = gate[row];
      erest = gate[C + row];
      bt = gate[2 * C + row];
      all = *reinterpret_cast<const float2*>(gate + 3 * C);
#pragma unroll
      for (int u = 0; u < kCols / 8; ++u) {
        v[u] = make_uint4(0u, 0u, 0u, 0u);
        if (is_k && tok < end) v[u] = *reinterpret_cast<const uint4*>(a.v + tok * a.ldv + col + 8 * u);
      }
    };
    auto arrive = [&](uint64_t* bar) {
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar);
    };
    auto publish = [&](uint64_t* bar) {  // operand rows written
      ptx::fence_proxy_async_smem();
      arrive(bar);
    };
    const uint32_t r_s = sb + P::R_OFF + (cols / 8) * (DK * 16);  // this thread's columns
    const uint32_t r_x = sb + P::R_OFF + (cols / 8) * (C * 16);
    bool ok = true;
    if (n > 0) fetch(0);
    for (int c = 0; c < n; ++c) {
      const uint32_t par = c & 1;
      if (!(ok = prepared(all.y, abort_flag))) break;
      if (DK == 128 || k_row < DK) store_row_split<kSPieces>(r_s, P::S_PIECE, k_row, DK * 16, S);
      publish(s_ready);
      const int64_t tok = start + static_cast<int64_t>(c) * C + row;
      const float eg_c = eg, erest_c = erest, eall_c = all.x;
      float D[kCols], Q[kCols];
      if (!(ok = warp_wait(d1, par, abort_flag, kFaultChain, a.wait_limit_ns))) break;
      ptx::tc_fence_after();
      ld_sum<kSPieces, DVB>(lanes, Q);
      if (is_k) {
#pragma unroll
        for (int u = 0; u < kCols / 8; ++u) {
          const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = 8 * u + 2 * e;
            const float v0 = __uint_as_float(w[e] << 16), v1 = __uint_as_float(w[e] & 0xFFFF0000u);
            D[j] = bt * (v0 - eg_c * Q[j]);
            D[j + 1] = bt * (v1 - eg_c * Q[j + 1]);
          }
        }
        store_row_split<kPieces>(r_x, P::X_PIECE, row, C * 16, D);
        publish(x_ready);
      } else {
        arrive(x_ready);  // Q S is taken: the product after next may go over it
      }
      if (c + 1 < n) fetch(c + 1);
      if (!(ok = warp_wait(d2, par, abort_flag, kFaultChain, a.wait_limit_ns))) break;
      ptx::tc_fence_after();
      ld_sum<kPieces, DVB>(lanes + P::D2_COL, D);
      if (is_k) {
#pragma unroll
        for (int j = 0; j < kCols; ++j) D[j] *= erest_c;
        store_row_split<kPieces>(r_x, P::X_PIECE, row, C * 16, D);
        publish(u_ready);
      } else if (tok < end) {
        if (store_out(a.o + tok * a.ldo + col, a.scale, eg_c, Q, D)) atomicMin(not_finite, c);
      }
      if (!(ok = warp_wait(d3, par, abort_flag, kFaultChain, a.wait_limit_ns))) break;
      ptx::tc_fence_after();
      ld_sum<kPieces, DVB>(lanes, D);
#pragma unroll
      for (int j = 0; j < kCols; ++j) S[j] = eall_c * S[j] + D[j];
    }
    // every compute warp is through its chunks, and all products are complete
    asm volatile("bar.sync 3, %0;" ::"n"(32 * P::WARPS) : "memory");
    const int bad = *static_cast<volatile int*>(not_finite);
    if (ok && *abort_flag == 0u && bad < n) {
      StateRow row_of_s;
      load_state(a, slot >= 0 && k_row < DK, b, state, row_of_s.x);
      row_of_s = token_by_token<DK>(a, reinterpret_cast<float*>(smem + P::R_OFF + (warp >> 2) * kScratchBytes),
                                    start, end, start + static_cast<int64_t>(bad) * C, h, col, warp, lane,
                                    row_of_s);
#pragma unroll
      for (int j = 0; j < kCols; ++j) S[j] = row_of_s.x[j];
    }
    if (ok && slot >= 0 && k_row < DK) store_state(state, S);
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == kMmaWarp) {
    __syncwarp();
    ptx::tmem_dealloc(tmem, P::TMEM);
  }
}

// ------------------------------------------------- chain without the delta rule --

// Without the delta rule U = V, and of a chunk's products only Q S waits for the
// state: A V and K^T U~, U~ = diag(e^{G_64-G}) V, need V alone, and the state's
// own chain is S' = e^{G_64} S + K^T U~ in registers. So A V and K^T U~ of a chunk
// run while its state is cut into pieces and the chunk before is written out,
// and a step takes one product's latency instead of three. V enters in one
// piece (exact). Of the image only the rows of A are there: the product's
// rows 0..63, which would be V itself, come from whatever stands before them in
// shared memory and are not read. The rest is chain_kernel's.
// With 128 of d_k two CTAs fit an SM only if A has one buffer (A_BUFS), asked for
// when the product before is complete: 8192 tokens of 64 heads take 360 us so,
// 523 with two buffers and one CTA per SM; where the CTAs are no more than the
// SMs, two buffers take 277 us for 32 heads, one 289. DVB as chain_kernel's: 8192
// tokens of 8 heads take 193 us with 16 columns, 207 with 32.
template <int DK, int DVB, int A_BUFS>
struct PlainCfg {
  static constexpr int WARPS = 4 * (DVB / kCols);
  static constexpr int THREADS = 32 * WARPS + 32;
  static constexpr int S_PIECE = DK * DVB * 2;
  static constexpr int X_PIECE = C * DVB * 2;
  static constexpr int A_BYTES = kTTBytes / 2;       // one piece of A
  static constexpr int A_OFF = 2 * kq_bytes(DK);     // [A_BUFS][2] pieces
  static constexpr int S_OFF = A_OFF + A_BUFS * 2 * A_BYTES;
  static constexpr int V_OFF = S_OFF + kSPieces * S_PIECE;
  static constexpr int U_OFF = V_OFF + X_PIECE;
  static constexpr int BAR_OFF = U_OFF + kPieces * X_PIECE;
  static constexpr int SMEM = BAR_OFF + 128;   // the base is 1024-byte aligned
  // tensor memory: Q S (with K S), A V (with I V), K^T U~
  static constexpr uint32_t D1 = 0, D2 = kSPieces * DVB, D3 = D2 + DVB;
  static constexpr uint32_t TMEM = DVB == 32 ? 256 : 128;
  static constexpr int PER_SM = DK == 64 || A_BUFS == 1 ? 2 : 1;
  static_assert(PER_SM * (SMEM + 1024) <= 228 * 1024 && D3 + kPieces * DVB <= TMEM, "CTAs per SM");
};

template <int DK, int DVB, int A_BUFS>
__global__ void __launch_bounds__(PlainCfg<DK, DVB, A_BUFS>::THREADS,
                                  PlainCfg<DK, DVB, A_BUFS>::PER_SM)
    plain_kernel(const __grid_constant__ Args a) {
  using P = PlainCfg<DK, DVB, A_BUFS>;
  extern __shared__ __align__(1024) uint8_t smem_la[];
  uint8_t* const smem = smem_la;
  uint64_t* const full = reinterpret_cast<uint64_t*>(smem + P::BAR_OFF);  // [2] K; Q loaded
  uint64_t* const full_a = full + 2;    // [A_BUFS] A loaded
  uint64_t* const v_ready = full + 4;   // V and U~ written, A V and K^T U~ before them taken
  uint64_t* const s_ready = full + 5;   // S written, Q S before it taken
  uint64_t* const d1 = full + 6;        // Q S, A V, K^T U~ complete
  uint64_t* const d2 = full + 7;
  uint64_t* const d3 = full + 8;
  uint64_t* const drain = full + 9;
  uint32_t* const tmem_holder = reinterpret_cast<uint32_t*>(full + 10);
  volatile uint32_t* const abort_flag = tmem_holder + 1;
  int* const not_finite = reinterpret_cast<int*>(tmem_holder + 2);  // first such chunk

  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int blocks = a.d_v / DVB;
  const int c0 = (blockIdx.x % blocks) * DVB;
  const int h = (blockIdx.x / blocks) % a.h_v;
  const int b = blockIdx.x / blocks / a.h_v;
  const int hk = h / (a.h_v / a.h_k);
  constexpr int kMmaWarp = P::WARPS;
  if (t == 0) {
    ptx::mbar_init(&full[0], 1);
    ptx::mbar_init(&full[1], 1);
    for (int i = 0; i < A_BUFS; ++i) ptx::mbar_init(&full_a[i], 1);
    ptx::mbar_init(v_ready, P::WARPS);
    ptx::mbar_init(s_ready, P::WARPS);
    ptx::mbar_init(d1, 1);
    ptx::mbar_init(d2, 1);
    ptx::mbar_init(d3, 1);
    ptx::mbar_init(drain, 1);
    *not_finite = INT_MAX;
    // the swizzled images need the alignment that the declaration asks for
    *abort_flag = (ptx::smem_u32(smem) & 1023u) != 0u ? 1u : 0u;
    if (*abort_flag) atomicOr(&g_fault_word, kFaultChain);
    ptx::fence_mbarrier_init();
  }
  if (warp == kMmaWarp) {
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

  // every barrier's phase c is chunk c's
  if (warp == kMmaWarp) {
    if (lane == 0) {
      auto load_kq = [&](int c) {
        ptx::mbar_arrive_expect_tx(&full[c & 1], kq_bytes(DK));
        ptx::bulk_load(smem + (c & 1) * kq_bytes(DK),
                       a.kq + ((static_cast<int64_t>(slot0) + c) * a.h_k + hk) * kq_bytes(DK),
                       kq_bytes(DK), &full[c & 1]);
      };
      auto load_a = [&](int c) {
        const uint8_t* const image =
            a.tt + ((static_cast<int64_t>(slot0) + c) * a.h_v + h) * kHeadBytes + P::A_BYTES;
        uint8_t* const pieces = smem + P::A_OFF + c % A_BUFS * 2 * P::A_BYTES;
        uint64_t* const bar = &full_a[c % A_BUFS];
        ptx::mbar_arrive_expect_tx(bar, 2 * P::A_BYTES);
        ptx::bulk_load(pieces, image, P::A_BYTES, bar);
        ptx::bulk_load(pieces + P::A_BYTES, image + kTTBytes, P::A_BYTES, bar);
      };
      constexpr uint32_t kI1 = ptx::idesc_bf16(128, kSPieces * DVB, false, true);
      constexpr uint32_t kI2 = ptx::idesc_bf16(128, DVB, false, true);
      constexpr uint32_t kI3 = ptx::idesc_bf16(128, kPieces * DVB, true, true);
      constexpr uint32_t kSN = DK * 16, kXN = C * 16;  // bytes between groups of 8 columns
      int kq_asked = 0, kq_seen = 0, a_asked = 0, a_seen = 0;  // chunks
      bool ok = *abort_flag == 0u;
      if (n > 0 && ok) {
        if (a.stall_chain != static_cast<int>(blockIdx.x)) load_kq(kq_asked++);
        load_a(a_asked++);
      }
      for (int c = 0; c < n && ok; ++c) {
        const uint32_t par = c & 1;
        const uint32_t kq = sb + par * kq_bytes(DK);
        ok = wait_bounded(&full[par], (c >> 1) & 1, abort_flag, kFaultChainMma, a.wait_limit_ns);
        if (!ok) break;
        ++kq_seen;
        ok = wait_bounded(v_ready, par, abort_flag, kFaultChainMma, a.wait_limit_ns);
        if (!ok) break;
        ptx::tc_fence_after();
#pragma unroll
        for (int s = 0; s < C / 16; ++s)   // K^T U~ (64 of d_k: the upper rows repeat the lower)
          ptx::tc_mma_bf16(tmem + P::D3,
                           ptx::smem_desc(kq + s * 2048, DK == 128 ? kHalfBytes : 0, 1024, 2),
                           ptx::smem_desc(sb + P::U_OFF + s * 256, 128, kXN, 0), kI3, s != 0);
        ptx::tc_commit(d3);
        const uint32_t pieces = sb + P::A_OFF + c % A_BUFS * 2 * P::A_BYTES;
        ok = wait_bounded(&full_a[c % A_BUFS], (c / A_BUFS) & 1, abort_flag, kFaultChainMma, a.wait_limit_ns);
        if (!ok) break;
        ++a_seen;
#pragma unroll
        for (int p = 0; p < 2; ++p)        // [*; A] V, A in two pieces
#pragma unroll
          for (int s = 0; s < C / 16; ++s)
            ptx::tc_mma_bf16(tmem + P::D2,
                             ptx::smem_desc(pieces + (p - 1) * P::A_BYTES + s * 32, 16, 1024, 2),
                             ptx::smem_desc(sb + P::V_OFF + s * 256, 128, kXN, 0), kI2, (p | s) != 0);
        ptx::tc_commit(d2);
        ok = wait_bounded(s_ready, par, abort_flag, kFaultChainMma, a.wait_limit_ns);
        if (!ok) break;
        // S in place: Q S of the chunk before is taken, and with it the last
        // reader of the other buffers complete
        if (c + 1 < n) load_kq(kq_asked++);
        if (A_BUFS > 1 && c + 1 < n) load_a(a_asked++);
        ptx::tc_fence_after();
#pragma unroll
        for (int s = 0; s < DK / 16; ++s)   // [K; Q] S
          ptx::tc_mma_bf16(tmem + P::D1, ptx::smem_desc(kq + (s / 4) * kHalfBytes + (s % 4) * 32, 16, 1024, 2),
                           ptx::smem_desc(sb + P::S_OFF + s * 256, 128, kSN, 0), kI1, s != 0);
        ptx::tc_commit(d1);
        if (A_BUFS == 1 && c + 1 < n) {
          ok = wait_bounded(d2, par, abort_flag, kFaultChainMma, a.wait_limit_ns);
          if (!ok) break;
          load_a(a_asked++);
        }
      }
      if (!ok) {  // let what is in flight end before the CTA does
        ptx::tc_commit(drain);
        drain_wait(drain, 0);
        for (int c = kq_seen; c < kq_asked; ++c) drain_wait(&full[c & 1], (c >> 1) & 1);
        for (int c = a_seen; c < a_asked; ++c) drain_wait(&full_a[c % A_BUFS], (c / A_BUFS) & 1);
      } else if (n > 0) {
        drain_wait(d1, (n - 1) & 1);  // the last product, should the others give up on it
      }
    }
  } else {
    const int k_row = (warp & 3) * 32 + lane;   // row of d_k
    const int row = k_row & (C - 1);            // token of the chunk
    const bool is_v = (warp & 3) < 2;           // rows of V and U~; else rows of Q and O
    const int cols = (warp >> 2) * kCols;       // this thread's columns of the block
    const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + cols;
    const int slot = state_slot(a, b, lane);
    const int64_t col = static_cast<int64_t>(h) * a.d_v + c0 + cols;  // column of V and O
    float* const state = a.state + ((static_cast<int64_t>(slot) * a.h_v + h) * DK + k_row) * a.d_v +
                         c0 + cols;
    float S[kCols];
    load_state(a, slot >= 0 && k_row < DK, b, state, S);
    // what the next chunk needs from memory, requested a chunk ahead
    float gate = 0.0f;   // e^{G_64 - G} of rows of V, e^G of rows of Q
    float2 all = make_float2(0.0f, 0.0f);   // as chain_kernel's
    uint4 v[kCols / 8];
    auto fetch = [&](int c) {
      const int64_t tok = start + static_cast<int64_t>(c) * C + row;
      const float* g = reinterpret_cast<const float*>(
          a.tt + ((static_cast<int64_t>(slot0) + c) * a.h_v + h) * kHeadBytes + 2 * kTTBytes);
      gate = g[(is_v ? C : 0) + row];
      all = *reinterpret_cast<const float2*>(g + 3 * C);
#pragma unroll
      for (int u = 0; u < kCols / 8; ++u) {
        v[u] = make_uint4(0u, 0u, 0u, 0u);
        if (is_v && tok < end) v[u] = *reinterpret_cast<const uint4*>(a.v + tok * a.ldv + col + 8 * u);
      }
    };
    auto arrive = [&](uint64_t* bar) {
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar);
    };
    auto publish = [&](uint64_t* bar) {  // operand rows written
      ptx::fence_proxy_async_smem();
      arrive(bar);
    };
    const uint32_t r_s = sb + P::S_OFF + (cols / 8) * (DK * 16);  // this thread's columns
    const uint32_t r_v = sb + P::V_OFF + (cols / 8) * (C * 16);
    const uint32_t r_u = sb + P::U_OFF + (cols / 8) * (C * 16);
    bool ok = true;
    float eg_before = 0.0f, eall_before = 0.0f;
    if (n > 0) fetch(0);
    // Chunk c begins where chunk c - 1 ends: its rows of the state and its
    // outputs are taken from tensor memory here.
    for (int c = 0; c <= n; ++c) {
      const uint32_t par = c & 1, before = par ^ 1;
      float D[kCols], AV[kCols];
      if (c > 0) {
        if (!(ok = warp_wait(d3, before, abort_flag, kFaultChain, a.wait_limit_ns))) break;
        ptx::tc_fence_after();
        ld_sum<kPieces, DVB>(lanes + P::D3, D);
        if (!(ok = warp_wait(d2, before, abort_flag, kFaultChain, a.wait_limit_ns))) break;
        ptx::tc_fence_after();
        if (!is_v) {
          ptx::tc_ld_32x32b_x16(lanes + P::D2, AV);
          ptx::tc_wait_ld();
        }
      }
      const float eg = gate, e_all = all.x;
      if (c < n) {
        if (!(ok = prepared(all.y, abort_flag))) break;
        if (is_v) {
          float u[kCols];
#pragma unroll
          for (int i = 0; i < kCols / 8; ++i) {
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            ptx::st_shared_v4(r_v + mn_off(row, i, C * 16), w[0], w[1], w[2], w[3]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              u[8 * i + 2 * e] = eg * __uint_as_float(w[e] << 16);
              u[8 * i + 2 * e + 1] = eg * __uint_as_float(w[e] & 0xFFFF0000u);
            }
          }
          store_row_split<kPieces>(r_u, P::X_PIECE, row, C * 16, u);
          publish(v_ready);
        } else {
          arrive(v_ready);
        }
        if (c + 1 < n) fetch(c + 1);
      }
      if (c > 0) {
#pragma unroll
        for (int j = 0; j < kCols; ++j) S[j] = eall_before * S[j] + D[j];
        if (!(ok = warp_wait(d1, before, abort_flag, kFaultChain, a.wait_limit_ns))) break;
        ptx::tc_fence_after();
      }
      if (c > 0 && !is_v) ld_sum<kSPieces, DVB>(lanes + P::D1, D);  // Q S
      if (c < n) {
        if (DK == 128 || k_row < DK) store_row_split<kSPieces>(r_s, P::S_PIECE, k_row, DK * 16, S);
        publish(s_ready);
      }
      if (c > 0 && !is_v) {
        const int64_t tok = start + static_cast<int64_t>(c - 1) * C + row;
        if (tok < end && store_out(a.o + tok * a.ldo + col, a.scale, eg_before, D, AV))
          atomicMin(not_finite, c - 1);
      }
      eg_before = eg;
      eall_before = e_all;
    }
    // every compute warp is through its chunks, and all products are complete
    asm volatile("bar.sync 3, %0;" ::"n"(32 * P::WARPS) : "memory");
    const int bad = *static_cast<volatile int*>(not_finite);
    if (ok && *abort_flag == 0u && bad < n) {
      StateRow row_of_s;
      load_state(a, slot >= 0 && k_row < DK, b, state, row_of_s.x);
      row_of_s = token_by_token<DK>(a, reinterpret_cast<float*>(smem + P::V_OFF + (warp >> 2) * kScratchBytes),
                                    start, end, start + static_cast<int64_t>(bad) * C, h, col, warp, lane,
                                    row_of_s);
#pragma unroll
      for (int j = 0; j < kCols; ++j) S[j] = row_of_s.x[j];
    }
    if (ok && slot >= 0 && k_row < DK) store_state(state, S);
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == kMmaWarp) {
    __syncwarp();
    ptx::tmem_dealloc(tmem, P::TMEM);
  }
}

}  // namespace la
}  // namespace nvfp4
