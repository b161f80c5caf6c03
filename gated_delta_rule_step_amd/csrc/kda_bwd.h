// Parameter block, workspace layout and device helpers of the prefill gradient's
// kernels (gfx950). The method is described in kda_backward.hip.
#pragma once

#include <float.h>
#include <stdint.h>

#include <atomic>

#include "../../include/kda_backward.h"
#include "kda_common.h"

namespace kda {
namespace bwd {

constexpr int C = 64;        // tokens per chunk
constexpr int NB = C / 16;   // 16-token blocks per chunk
constexpr int NP = NB * (NB - 1) / 2;
constexpr int kThreads = 512;
constexpr int kMaxOrderedDocs = 256;
constexpr int kCus = 256;
constexpr float kL2Eps = 1e-6f;

struct BwdParams {
  int32_t n_docs, H;
  int64_t slots;  // chunk slots: n_docs + total_tokens / C
  const int32_t* cu_seqlens;
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  const uint16_t* g;
  const uint16_t* beta;
  int64_t q_stride, k_stride, v_stride, g_stride, beta_stride;
  const float* A_log;
  const float* dt_bias;
  float lower_bound, scale;
  int32_t gate_mode, state_dtype, use_initial;
  const void* pool;
  int64_t num_slots, slot_stride;
  const int32_t* state_indices;
  const uint16_t* dout;
  int64_t dout_stride;
  const float* d_final;
  uint16_t* dq;
  uint16_t* dk;
  uint16_t* dv;
  uint16_t* dg;
  uint16_t* dbeta;
  int64_t dq_stride, dk_stride, dv_stride, dg_stride, dbeta_stride;
  float* dA_log;
  float* ddt_bias;
  float* d_initial;
  uint8_t* ops;    // [slot][h][kOps]
  float* partial;  // [slot][h][2][D]: of ddt_bias and dA_log, per channel
};

struct DocOrder {
  int32_t n;  // 0: natural order
  int32_t deep;  // the first of them, whose chains take the form of least latency
  int32_t doc[kMaxOrderedDocs];
};

// A (chunk, head)'s part of the workspace, in bytes. The chains' left operands are
// fp16 high and low parts in fragment order, 16 bytes (8 contraction indices) a lane:
//   W, Z        [rt 4][kt 4][hi, lo][lane]  token 16 rt + lane % 16, key channels
//               32 kt + 4 (lane / 16) + 0..3 and 16 further
//   KE, KG, QG  [m 8][t 2][hi, lo][lane]    key channel 16 m + lane % 16, tokens
//               32 t + 4 (lane / 16) + 0..3 and 16 further
//   O           [vt 8][t 2][lane]           value channel 16 vt + lane % 16, tokens as in KE,
//               scaled per value channel
// X0 and DV0 are accumulator tiles [vt 8][rt 4][lane][4 tokens], X and DV rows
// [token][value], S and dS rows [key][value], all fp32.
constexpr int kOpTail = 0;               // e^Gl [128], beta [64], scales (below)
constexpr int kOpW = 1024;               // T e^G k
constexpr int kOpKE = kOpW + 32768;      // e^(Gl-G) k
constexpr int kOpZ = kOpKE + 32768;      // T^T (beta e^(Gl-G) k)
constexpr int kOpKG = kOpZ + 32768;      // e^G k
constexpr int kOpQG = kOpKG + 32768;     // e^G q_hat
constexpr int kOpX0 = kOpQG + 32768;     // T V
constexpr int kOpDV0 = kOpX0 + 32768;    // T^T P^T dO
constexpr int kOpO = kOpDV0 + 32768;     // dO, as QG's right side (fp16)
constexpr int kOpUnO = kOpO + 16384;     // what undoes O's scales [128]
constexpr int kOpX = kOpUnO + 512;       // x
constexpr int kOpDV = kOpX + 32768;      // dV
constexpr int kOpS = kOpDV + 32768;      // S entering the chunk
constexpr int kOpDS = kOpS + 65536;      // dS leaving it
constexpr int kOps = kOpDS + 65536;
// In floats. A token block of each operand has a scale of its own, a power of two: decays
// over a chunk span far more than fp16. What undoes it: of W and Z on the product's rows, of
// KG (and QG) and KE on the right side's.
constexpr int kTailBeta = D, kTailUnW = D + C, kTailUnZ = kTailUnW + NB,
              kTailDnKG = kTailUnZ + NB, kTailDnKE = kTailDnKG + NB;

__device__ __forceinline__ f32x4 mfma4(f32x4 a, f32x4 b, f32x4 c) {
#pragma unroll
  for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
  return c;
}
__device__ __forceinline__ f32x4 zero4() { return f32x4{0.f, 0.f, 0.f, 0.f}; }
__device__ __forceinline__ f32x4 lds4(const float* p) { return *reinterpret_cast<const f32x4*>(p); }
// 4 elements down a column
__device__ __forceinline__ f32x4 col4(const float* p, int stride) {
  return f32x4{p[0], p[stride], p[2 * stride], p[3 * stride]};
}

typedef u32x4 u32x4_u __attribute__((aligned(2)));  // any bf16 address
typedef __fp16 f16x8 __attribute__((__vector_size__(8 * sizeof(__fp16))));  // MFMA operand

// fp32 as fp16 high + low parts: 22 bits and a sign. Three products (high high,
// high low, low high) then leave out 2^-22 of a term, what four fp32 additions may round.
__device__ __forceinline__ void split4h(f32x4 x, u32x2& hi, u32x2& lo) {
  hi = u32x2{pack_f16x2(x[0], x[1]), pack_f16x2(x[2], x[3])};
  lo = u32x2{pack_f16x2(x[0] - f16_lo(hi[0]), x[1] - f16_hi(hi[0])),
             pack_f16x2(x[2] - f16_lo(hi[1]), x[3] - f16_hi(hi[1]))};
}
__device__ __forceinline__ f16x8 join8(u32x2 a, u32x2 b) {
  return __builtin_bit_cast(f16x8, u32x4{a[0], a[1], b[0], b[1]});
}
__device__ __forceinline__ f32x4 mfma32(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// fp16 holds 2^-24 to 2^16, so operands of any size are scaled by a power of two that
// brings their largest magnitude to 2^14 .. 2^15; `un` undoes it.
struct Scale {
  float up, un;
};
__device__ __forceinline__ Scale scale_for(float top) {
  int e = int(__float_as_uint(top) >> 23);
  e = e < 40 ? 40 : (e > 250 ? 250 : e);
  return {__uint_as_float(uint32_t(268 - e) << 23), __uint_as_float(uint32_t(e - 14) << 23)};
}
// The power of two that brings x into [1, 2), and its inverse.
__device__ __forceinline__ Scale unit_scale(float x) {
  int e = int(__float_as_uint(x) >> 23);
  e = e < 40 ? 40 : (e > 214 ? 214 : e);
  return {__uint_as_float(uint32_t(254 - e) << 23), __uint_as_float(uint32_t(e) << 23)};
}
constexpr float kFixedUp = 4096.0f, kFixedUn = 1.0f / 4096.0f;  // operands within +-1

typedef __fp16 f16x4 __attribute__((__vector_size__(4 * sizeof(__fp16))));
// The same over one block of 16: half `u` of the fragments.
__device__ __forceinline__ f16x4 half8(f16x8 x, int u) {
  const u32x4 w = __builtin_bit_cast(u32x4, x);
  return __builtin_bit_cast(f16x4, u32x2{w[2 * u], w[2 * u + 1]});
}
__device__ __forceinline__ f32x4 mfma_split16(f16x8 ah, f16x8 al, f16x8 bh, f16x8 bl, int u) {
  f32x4 c = zero4();
  c = __builtin_amdgcn_mfma_f32_16x16x16f16(half8(al, u), half8(bh, u), c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_16x16x16f16(half8(ah, u), half8(bl, u), c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_16x16x16f16(half8(ah, u), half8(bh, u), c, 0, 0, 0);
}
// With a right side that its high part holds exactly.
__device__ __forceinline__ f32x4 mfma_high16(f16x8 ah, f16x8 al, f16x8 b, int u) {
  f32x4 c = zero4();
  c = __builtin_amdgcn_mfma_f32_16x16x16f16(half8(al, u), half8(b, u), c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_16x16x16f16(half8(ah, u), half8(b, u), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma_split(f16x8 ah, f16x8 al, f16x8 bh, f16x8 bl, f32x4 c) {
  c = mfma32(al, bh, c);
  c = mfma32(ah, bl, c);
  return mfma32(ah, bh, c);
}

// The largest magnitude over the four lanes that share a column of an accumulator tile.
__device__ __forceinline__ float column_max(float x) {
  x = fmaxf(x, __shfl_xor(x, 16));
  return fmaxf(x, __shfl_xor(x, 32));
}

__device__ __forceinline__ float row16_max(float x) {
  x = fmaxf(x, dpp<0xB1>(x));
  x = fmaxf(x, dpp<0x4E>(x));
  x = fmaxf(x, dpp<0x141>(x));
  return fmaxf(x, dpp<0x140>(x));
}

// The largest of a wave, in every lane.
__device__ __forceinline__ float wave_max(float x) { return column_max(row16_max(x)); }
// A value that is the same in every lane, in a scalar register.
__device__ __forceinline__ float uniform(float x) {
  return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(x)));
}
__device__ __forceinline__ float uniform_bits(uint32_t x) {
  return __uint_as_float(__builtin_amdgcn_readfirstlane(x));
}

// Sum over the four 16-lane rows of a wave (lanes of equal lane % 16).
__device__ __forceinline__ float rows_sum(float x) {
  x += __shfl_xor(x, 16);
  return x + __shfl_xor(x, 32);
}

// First chunk slot of document i; slots of a document follow each other.
__device__ __forceinline__ int64_t doc_slot0(const int32_t* cu, int i) {
  return int64_t(i) + int64_t(cu[i]) / C;
}
// The document of chunk slot sigma: the largest i <= n_docs with doc_slot0(i) <=
// sigma (doc_slot0 rises strictly from 0). A wave asks for 64 documents at a time.
__device__ __forceinline__ int find_doc(const int32_t* cu, int n_docs, int64_t sigma) {
  int lo = 0, len = n_docs + 1;
  while (len > 1) {
    const int stride = (len + 63) / 64;
    const int off = int(threadIdx.x & 63) * stride;
    const bool le = off < len && doc_slot0(cu, lo + off) <= sigma;
    lo += (__builtin_popcountll(__ballot(le)) - 1) * stride;
    len = min(stride, n_docs + 1 - lo);
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

struct Chunk {
  int doc;
  int64_t t0;  // first token
  int c;       // tokens; 0: a slot between documents
  bool active;
};
__device__ __forceinline__ Chunk chunk_of(const BwdParams& p, int64_t sigma) {
  Chunk ch = {0, 0, 0, false};
  ch.doc = find_doc(p.cu_seqlens, p.n_docs, sigma);
  if (ch.doc >= p.n_docs) return ch;
  // the same in every lane: kept in scalar registers, addresses with them
  const int32_t start = __builtin_amdgcn_readfirstlane(p.cu_seqlens[ch.doc]);
  const int32_t end = __builtin_amdgcn_readfirstlane(p.cu_seqlens[ch.doc + 1]);
  const int32_t slot = __builtin_amdgcn_readfirstlane(p.state_indices[ch.doc]);
  const int64_t off = (sigma - (int64_t(ch.doc) + start / C)) * C;
  if (off >= end - start) return ch;
  ch.t0 = start + off;
  ch.c = int(min<int64_t>(C, end - start - off));
  ch.active = slot >= 0 && int64_t(slot) < p.num_slots;
  return ch;
}

// A chunk's rows of a bf16 tensor from channel `col` on: one scalar base and 32-bit lane
// offsets (the host keeps strides within 2^25 elements, so 64 rows span less than 2^32
// bytes).
struct Rows {
  uint16_t* base;
  uint32_t stride;
  __device__ __forceinline__ uint32_t offset(int t, int col) const {
    return uint32_t(t) * stride + uint32_t(col) * 2u;
  }
  // `t` more rows (the same for all lanes) after a lane's offset
  __device__ __forceinline__ uint16_t* from(uint32_t off, int t) const {
    return reinterpret_cast<uint16_t*>(reinterpret_cast<uint8_t*>(base) +
                                       (off + uint32_t(t) * stride));
  }
  // the same, but no further than offset `last`
  __device__ __forceinline__ uint16_t* upto(uint32_t off, int t, uint32_t last) const {
    return from(min(off + uint32_t(t) * stride, last), 0);
  }
  __device__ __forceinline__ uint16_t* at(int t, int col) const { return from(offset(t, col), 0); }
};
__device__ __forceinline__ Rows rows_of(const uint16_t* x, const Chunk& ch, int64_t stride,
                                        int64_t col) {
  return {const_cast<uint16_t*>(x) + ch.t0 * stride + col, uint32_t(stride * 2)};
}

// Here and below a chunk's missing tokens read its last one and drop the value: a
// load behind a branch would be waited for one at a time.

// 1 / |q|, 1 / |k| (with the epsilon) and beta of the chunk's tokens, to LDS: 16
// lanes per token. Padding rows get zeros. With SLOPE, beta's derivative by its input too: of a
// logit, beta (1 - beta) with 1 - beta as e^-x beta, which does not cancel near 1 (e^-x kept
// finite: where it would overflow, beta is 0).
template <bool SLOPE>
__device__ __forceinline__ void token_scalars(const BwdParams& p, const Chunk& ch, int h,
                                              float* rq, float* rk, float* beta, float* slope) {
  constexpr int N = C / (kThreads / 16);
  const int c0 = (threadIdx.x & 15) * 8;
  const Rows qr = rows_of(p.q, ch, p.q_stride, int64_t(h) * D);
  const Rows kr = rows_of(p.k, ch, p.k_stride, int64_t(h) * D);
  const Rows br = rows_of(p.beta, ch, p.beta_stride, h);
  u32x4 qw[N], kw[N];
  uint16_t bw[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int t = min(int(threadIdx.x >> 4) + j * (kThreads / 16), ch.c - 1);
    qw[j] = *reinterpret_cast<const u32x4_u*>(qr.at(t, c0));
    kw[j] = *reinterpret_cast<const u32x4_u*>(kr.at(t, c0));
    bw[j] = *br.at(t, 0);
  }
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int t = (threadIdx.x >> 4) + j * (kThreads / 16);
    float x[8], sq = 0.f, sk = 0.f;
    unpack8_bf16(qw[j], x);
#pragma unroll
    for (int i = 0; i < 8; ++i) sq = fmaf(x[i], x[i], sq);
    unpack8_bf16(kw[j], x);
#pragma unroll
    for (int i = 0; i < 8; ++i) sk = fmaf(x[i], x[i], sk);
    sq = row16_sum(sq);
    sk = row16_sum(sk);
    if ((threadIdx.x & 15) == 0) {
      float b = bf1(bw[j]), by = 1.0f;
      if (!(p.gate_mode & KDA_BETA_PRESIGMOID)) {
        const float e = expf(-b);
        b = 1.0f / (1.0f + e);
        by = fminf(e, FLT_MAX) * b * b;
      }
      if constexpr (SLOPE) slope[t] = by;
      rq[t] = t < ch.c ? 1.0f / sqrtf(sq + kL2Eps) : 0.f;
      rk[t] = t < ch.c ? 1.0f / sqrtf(sk + kL2Eps) : 0.f;
      beta[t] = t < ch.c ? b : 0.f;
    }
  }
}

// A lane's share of the chunk: key channel `kc`, tokens 16 b + 4 g4 + i.
struct RawLane {
  uint16_t k[NB][4], q[NB][4], g[NB][4];
};
__device__ __forceinline__ int64_t gate_channel(const BwdParams& p, int h, int kc) {
  return (p.gate_mode & KDA_GATE_PER_HEAD) ? h : int64_t(h) * D + kc;
}
__device__ __forceinline__ void load_lane(const BwdParams& p, const Chunk& ch, int h, int kc,
                                          int g4, RawLane& raw) {
  const bool head = p.gate_mode & KDA_GATE_PER_HEAD;
  const Rows qr = rows_of(p.q, ch, p.q_stride, int64_t(h) * D);
  const Rows kr = rows_of(p.k, ch, p.k_stride, int64_t(h) * D);
  const Rows gr = rows_of(p.g, ch, p.g_stride, head ? h : int64_t(h) * D);
  const int gc = head ? 0 : kc;
  const uint32_t k0 = kr.offset(4 * g4, kc), q0 = qr.offset(4 * g4, kc), g0 = gr.offset(4 * g4, gc);
  const uint32_t kl = kr.offset(ch.c - 1, kc), ql = qr.offset(ch.c - 1, kc),
                 gl = gr.offset(ch.c - 1, gc);
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      raw.k[b][i] = *kr.upto(k0, 16 * b + i, kl);
      raw.q[b][i] = *qr.upto(q0, 16 * b + i, ql);
      raw.g[b][i] = *gr.upto(g0, 16 * b + i, gl);
    }
}

// Decays are products of a_t = e^g_t, never exponentials of sums: 16 factors keep a
// relative error of a few 2^-24 where a sum of 16 gates of size 5 would lose ten times
// that. `up` reaches from the middle of the token's block (after its 8th token)
// to the token, its inverse back; both lie within e^(+-44). head and tail are the
// block's two halves.
__device__ __forceinline__ float inverse(float x) { return __builtin_amdgcn_rcpf(x); }

// log(1 + e) for e >= 0. The sum 1 + e is rounded by up to 2^-24, which is half of e itself
// where the gates of a slowly decaying head lie (e of 1e-7), so small e take four terms of the
// series: below 1/32 they leave out 2e-7 of the result, and above it the rounding is at most
// 2e-6 of it. dA_log, a sum of gates, needs that, and so do decays over many like tokens.
__device__ __forceinline__ float log1p_of(float e) {
  const float series = e * fmaf(-e, fmaf(-e, fmaf(-e, 0.25f, 1.f / 3.f), 0.5f), 1.f);
  return e < 1.f / 32.f ? series : LN2 * __builtin_amdgcn_logf(1.0f + e);
}

struct Lane {
  float k[NB][4], q[NB][4];  // k_hat, q_hat
  float up[NB][4];
  float head[NB], tail[NB];
};
// PRE: the gate input is the log-decay itself (KDA_GATE_PRECOMPUTED). With SLOPE, `keep`
// takes each token's log-decay and its derivative by the gate input: 2 x 16 floats per
// thread, kThreads apart.
template <bool PRE, bool SLOPE>
__device__ __forceinline__ void make_lane(const BwdParams& p, const Chunk& ch, int h, int kc,
                                          int g4, const RawLane& raw, const float* rq,
                                          const float* rk, Lane& ln, float* keep) {
  const float ea = PRE ? 0.f : expf(p.A_log[h]);
  const float dtb = PRE ? 0.f : p.dt_bias[gate_channel(p, h, kc)];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    __builtin_amdgcn_sched_barrier(0);  // a block at a time: the raw values make room
    const f32x4 rq4 = lds4(rq + 16 * b + 4 * g4), rk4 = lds4(rk + 16 * b + 4 * g4);
    float a[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool valid = 16 * b + 4 * g4 + i < ch.c;
      ln.k[b][i] = bf1(raw.k[b][i]) * rk4[i];  // missing tokens: rk, rq are zeros
      ln.q[b][i] = bf1(raw.q[b][i]) * rq4[i];
      const float x = bf1(raw.g[b][i]);
      float g, s = 0.f;
      if constexpr (PRE) {
        g = gate_given(x, p.lower_bound);
        s = x >= p.lower_bound && x <= 0.f ? 1.f : 0.f;
      } else {
        // softplus and sigmoid from one exponential (hardware exp2, log2, rcp), which is
        // kept finite: log(1 + e^y) is y long before
        const float y = x + dtb;
        const float e = fexp(fminf(y, 80.f));
        const float gu = -ea * fmaxf(y, log1p_of(e));
        g = fmaxf(gu, p.lower_bound);
        if (SLOPE) s = gu >= p.lower_bound ? -ea * (e * __builtin_amdgcn_rcpf(1.0f + e)) : 0.f;
      }
      a[i] = fexp(valid ? g : 0.f);
      if constexpr (SLOPE) {
        keep[(4 * b + i) * kThreads] = g;
        keep[(16 + 4 * b + i) * kThreads] = valid ? s : 0.f;
      }
    }
    // From the lane's first token on; then the lanes between it and the block's middle, and
    // the block's other half.
    const float a1 = a[0] * a[1], a2 = a1 * a[2], all = a2 * a[3];
    const float near = __shfl_xor(all, 16);
    const float half = all * near;
    const float other = __shfl_xor(half, 32);
    ln.head[b] = g4 < 2 ? half : other;
    ln.tail[b] = g4 < 2 ? other : half;
    // from the middle to the lane's first token: back over its own and the next lane's
    // tokens (lanes 0; 1 only its own), or over the lane before (3; none for 2)
    const float base = g4 == 0 || g4 == 3 ? near : 1.f;
    const float from = g4 < 2 ? inverse(all * base) : base;
    ln.up[b][0] = from * a[0];
    ln.up[b][1] = from * a1;
    ln.up[b][2] = from * a2;
    ln.up[b][3] = from * all;
  }
}

// Dynamic LDS beyond 64 KiB is allowed once per kernel and device, before its first launch
// there. The device's entry in `done` is only ever set, so calls from several threads at
// worst allow it twice.
constexpr int kMaxDevices = 64;
inline hipError_t allow_lds(const void* kernel, size_t bytes,
                            std::atomic<bool> (&done)[kMaxDevices]) {
  int dev = -1;
  if (const hipError_t e = hipGetDevice(&dev)) return e;
  if (dev < 0 || dev >= kMaxDevices) return hipErrorInvalidDevice;
  if (done[dev].load(std::memory_order_relaxed)) return hipSuccess;
  const hipError_t e =
      hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
  if (e == hipSuccess) done[dev].store(true, std::memory_order_relaxed);
  return e;
}

hipError_t launch_prep(const BwdParams& p, hipStream_t stream);
hipError_t launch_chains(const BwdParams& p, const DocOrder& ord, hipStream_t stream);
// Whether the chains of the document that is `rank`th in length take the form of least latency.
bool deep_chains(int64_t total_tokens, int H, int rank, int len);
hipError_t launch_grads(const BwdParams& p, hipStream_t stream);
hipError_t launch_params(const BwdParams& p, hipStream_t stream);  // dA_log, ddt_bias

}  // namespace bwd
}  // namespace kda
