// Gradients of the chunked varlen prefill (gfx950).
//
// The recurrence and its adjoint, per (document, head), are given token by
// token in kda_backward.h. Here they run in chunks of 64 tokens (WY
// representation of the delta rule, Yang et al., "Parallelizing Linear
// Transformers with the Delta Rule over Sequence Length", 2024, the decay per
// key channel). With G_r the log-decay summed from the chunk's first token to
// r, q' = scale q_hat, S[k][v] the state entering and dS the state gradient
// leaving the chunk:
//   A[r,j] = beta_j sum_k k_r k_j e^(G_r - G_j)  (j < r)
//   P[r,j] = beta_j sum_k q'_r k_j e^(G_r - G_j) (j <= r)
//   T  = (1 + A)^-1
//   x  = T V - (T e^G k) S                  (x_r = v_r - S' k_r)
//   S1 = e^Gl S + (beta e^(Gl-G) k)^T x     (Gl: the chunk's sum)
//   dV = T^T P^T dO + (T^T beta e^(Gl-G) k) dS
//   dS0 = e^Gl dS + (e^G q')^T dO - (e^G k)^T dV
// beta stays with the writing token j throughout, so nothing is ever divided by
// it. The two recursions, S up and dS down the document, need each other's
// results nowhere, and neither needs more of a chunk than prep_kernel leaves:
// chain_kernel runs both at once. Then every chunk is on its own again
// (grad_kernel):
//   DP = tril(dO x^T, -1), dp = its diagonal, DA = -tril(dV x^T, -1)
//   dq'  = e^G (dO S^T)  + sum_j DP[r,j] beta_j k_j e^(G_r-G_j)
//   drow = -e^G (dV S^T) + sum_j DA[r,j] beta_j k_j e^(G_r-G_j)
//   col  = e^(Gl-G) (x dS^T) + sum_r (DA[r,j] k_r + DP[r,j] q'_r) e^(G_r-G_j)
// and, with dp_r beta_r k_r added to dq'_r and dp_r q'_r to col_r,
//   dk_hat = drow + beta col,  dbeta = k_hat . col,  dq_hat = scale dq'
// Each weight e^(G_r-G_j) rises by dg_t for all j < t <= r, so dg is a suffix sum
// of q' dq' + k drow - beta k col before those two (what token t uses as reader less
// as writer),
// to which the chunk's end adds what leaves it: e^Gl sum_v S dS + sum_t beta k
// e^(Gl-G) (x dS^T).
//
// Decays. A chunk is four 16-token blocks. With lam the log-decay summed inside a
// block and tau the block's total, readers hold e^(lam - tau/2) and writers
// e^(tau/2 - lam), both within e^(+-44) (|lower_bound| <= 5.5); a pair of blocks
// I >= J then lacks e^(sum of tau from the middle of J to the middle of I), one
// factor per pair and channel. No sum runs over more than 16 tokens before it is
// exponentiated, which keeps the weights' relative error near 16 * 2^-24 of the
// gates.
//
// Every product runs on fp32 MFMA (16x16x4). An operand tile is read as 4
// consecutive elements along the contraction by each lane, and the four
// instructions they feed take contraction indices 4 (lane / 16) + j, so that an
// accumulator tile (rows 4 (lane / 16) + i) serves as the next product's right
// operand as it is.

#include <math.h>
#include <stdint.h>

#include "../../include/kda_backward.h"
#include "kda_common.h"

namespace kda {
namespace {

constexpr int C = 64;        // tokens per chunk
constexpr int NB = C / 16;   // 16-token blocks per chunk
constexpr int RS = D + 4;    // padded row (fp32) of [token][channel] LDS arrays
constexpr int AS = C + 4;    // padded row of [token][token] LDS arrays
constexpr int NP = NB * (NB - 1) / 2;  // pairs of different blocks
constexpr int kThreads = 512;
constexpr int kMaxOrderedDocs = 256;
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
  float* ops;      // [slot][h][kOps]
  float* partial;  // [slot][h][2][D]: of ddt_bias and dA_log, per channel
};

struct DocOrder {
  int32_t n;  // 0: natural order
  int32_t doc[kMaxOrderedDocs];
};

// A (chunk, head)'s part of the workspace, fp32 elements. Operands that an MFMA
// reads as its left side are in fragment order [tile][tile][lane][4].
constexpr int kTile = C * D;
constexpr int kOpW = 0;              // -T e^G k       [rt 4][m 8][lane][4 channels]
constexpr int kOpKE = kTile;         // beta e^(Gl-G) k [m 8][rt 4][lane][4 tokens]
constexpr int kOpZ = 2 * kTile;      // T^T (beta e^(Gl-G) k), as W
constexpr int kOpKG = 3 * kTile;     // -e^G k, as KE
constexpr int kOpQG = 4 * kTile;     // e^G q', as KE
constexpr int kOpX = 5 * kTile;      // T V, then x [token][value]
constexpr int kOpDV = 6 * kTile;     // T^T P^T dO, then dV [token][value]
constexpr int kOpS = 7 * kTile;      // S [key][value] entering the chunk
constexpr int kOpDS = kOpS + D * D;  // dS [key][value] leaving it
constexpr int kOpEG = kOpDS + D * D; // e^Gl [key]
constexpr int kOps = kOpEG + D;

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
// sigma (doc_slot0 rises strictly from 0).
__device__ int find_doc(const int32_t* cu, int n_docs, int64_t sigma) {
  int lo = 0, hi = n_docs + 1;
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (doc_slot0(cu, mid) <= sigma) lo = mid;
    else hi = mid;
  }
  return lo;
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
  const int64_t start = p.cu_seqlens[ch.doc];
  const int64_t len = int64_t(p.cu_seqlens[ch.doc + 1]) - start;
  const int64_t off = (sigma - doc_slot0(p.cu_seqlens, ch.doc)) * C;
  if (off >= len) return ch;
  ch.t0 = start + off;
  ch.c = int(min<int64_t>(C, len - off));
  const int32_t slot = p.state_indices[ch.doc];
  ch.active = slot >= 0 && int64_t(slot) < p.num_slots;
  return ch;
}

// 1 / |q|, 1 / |k| (with the epsilon) and beta of the chunk's tokens, to LDS: 16
// lanes per token. Padding rows get zeros.
__device__ void token_scalars(const BwdParams& p, const Chunk& ch, int h, float* rq, float* rk,
                              float* beta) {
  const int c0 = (threadIdx.x & 15) * 8;
  for (int t = threadIdx.x >> 4; t < C; t += kThreads / 16) {
    float sq = 0.f, sk = 0.f;
    if (t < ch.c) {
      float x[8];
      unpack8_bf16(*reinterpret_cast<const u32x4_u*>(p.q + (ch.t0 + t) * p.q_stride + h * D + c0),
                   x);
#pragma unroll
      for (int i = 0; i < 8; ++i) sq = fmaf(x[i], x[i], sq);
      unpack8_bf16(*reinterpret_cast<const u32x4_u*>(p.k + (ch.t0 + t) * p.k_stride + h * D + c0),
                   x);
#pragma unroll
      for (int i = 0; i < 8; ++i) sk = fmaf(x[i], x[i], sk);
    }
    sq = row16_sum(sq);
    sk = row16_sum(sk);
    if ((threadIdx.x & 15) == 0) {
      rq[t] = t < ch.c ? 1.0f / sqrtf(sq + kL2Eps) : 0.f;
      rk[t] = t < ch.c ? 1.0f / sqrtf(sk + kL2Eps) : 0.f;
      float b = 0.f;
      if (t < ch.c) {
        b = bf1(p.beta[(ch.t0 + t) * p.beta_stride + h]);
        if (!(p.gate_mode & KDA_BETA_PRESIGMOID)) b = sigmoidf(b);
      }
      beta[t] = b;
    }
  }
}

// A lane's share of the chunk: key channel `kc`, tokens 16 b + 4 g4 + i.
struct Lane {
  float k[NB][4], q[NB][4];      // k_hat, q'
  float g[NB][4], slope[NB][4];  // log-decay and its derivative by the gate input
  float lam[NB][4];              // log-decay summed from the block's first token
  float tau[NB];                 // the block's total
};

template <bool SLOPE>
__device__ __forceinline__ void load_lane(const BwdParams& p, const Chunk& ch, int h, int kc,
                                          int g4, const float* rq, const float* rk, Lane& ln) {
  const bool pre = p.gate_mode & KDA_GATE_PRECOMPUTED;
  const bool head = p.gate_mode & KDA_GATE_PER_HEAD;
  const int64_t gch = head ? h : int64_t(h) * D + kc;
  const float ea = pre ? 0.f : expf(p.A_log[h]);
  const float dtb = pre ? 0.f : p.dt_bias[gch];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 16 * b + 4 * g4 + i;
      float k = 0.f, q = 0.f, g = 0.f, s = 0.f;
      if (t < ch.c) {
        k = bf1(p.k[(ch.t0 + t) * p.k_stride + h * D + kc]) * rk[t];
        q = bf1(p.q[(ch.t0 + t) * p.q_stride + h * D + kc]) * rq[t] * p.scale;
        const float x = bf1(p.g[(ch.t0 + t) * p.g_stride + gch]);
        if (pre) {
          g = gate_given(x, p.lower_bound);
          s = x >= p.lower_bound && x <= 0.f ? 1.f : 0.f;
        } else {
          const float y = x + dtb;
          const float gu = -ea * (y > 20.f ? y : log1pf(expf(y)));
          g = fmaxf(gu, p.lower_bound);
          if (SLOPE) s = gu >= p.lower_bound ? -ea * sigmoidf(y) : 0.f;
        }
      }
      ln.k[b][i] = k;
      ln.q[b][i] = q;
      if constexpr (SLOPE) {
        ln.g[b][i] = g;
        ln.slope[b][i] = s;
      }
      sum += g;
      ln.lam[b][i] = sum;
    }
    // the sums of the lanes with earlier tokens, then the block's total
    const float s1 = __shfl_xor(sum, 16);
    const float pair = sum + s1;
    const float other = __shfl_xor(pair, 32);
    const float before = ((g4 & 1) ? s1 : 0.f) + ((g4 & 2) ? other : 0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) ln.lam[b][i] += before;
    ln.tau[b] = pair + other;
  }
}

__host__ __device__ constexpr int pair_index(int I, int J) { return I * (I - 1) / 2 + J; }

// ---------------------------------------------------------------------------
// Preparation: one workgroup per (chunk, head); a wave owns 16 channels.
struct PrepSmem {
  float km[C * RS];    // e^(lam - tau/2) k
  float kb[C * RS];    // beta e^(tau/2 - lam) k
  float qm[C * RS];    // e^(lam - tau/2) q', then V and dO (bf16)
  float am[C * AS];    // A
  float pm[C * AS];    // P
  float tm[C * AS];    // T
  float pair[NP * D];  // factor of a block pair
  float rq[C], rk[C], beta[C];
};
constexpr int VS = 2 * RS;  // row of V and dO in uint16: V first, dO from RS on

__global__ __launch_bounds__(kThreads) void prep_kernel(BwdParams p) {
  extern __shared__ __align__(16) float smem_raw[];
  PrepSmem& s = *reinterpret_cast<PrepSmem*>(smem_raw);
  const int64_t sigma = blockIdx.x;
  const int h = blockIdx.y;
  const Chunk ch = chunk_of(p, sigma);
  if (ch.c == 0 || !ch.active) return;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int g4 = lane >> 4, n16 = lane & 15;
  const int kc = 16 * w + n16;
  float* ops = p.ops + (sigma * p.H + h) * int64_t(kOps);

  token_scalars(p, ch, h, s.rq, s.rk, s.beta);
  __syncthreads();

  // ---- the decayed rows, and what depends on them channel by channel alone
  f32x4 kg[NB], ke[NB];  // e^G k, beta e^(Gl-G) k: 4 tokens of channel kc
  {
    Lane ln;
    load_lane<false>(p, ch, h, kc, g4, s.rq, s.rk, ln);
    float from[NB], to[NB];  // middle of the block from the chunk's start, to its end
    float o = 0.f;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      from[b] = o + 0.5f * ln.tau[b];
      o += ln.tau[b];
    }
    float e = 0.f;
#pragma unroll
    for (int b = NB - 1; b >= 0; --b) {
      to[b] = e + 0.5f * ln.tau[b];
      e += ln.tau[b];
    }
    if (g4 == 0) {
      ops[kOpEG + kc] = expf(o);
#pragma unroll
      for (int I = 1; I < NB; ++I) {
        float mid = 0.f;
#pragma unroll
        for (int J = I - 1; J >= 0; --J) {
          s.pair[pair_index(I, J) * D + kc] = expf(0.5f * (ln.tau[I] + ln.tau[J]) + mid);
          mid += ln.tau[J];
        }
      }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const float ef = expf(from[b]), et = expf(to[b]);
      f32x4 qg;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 16 * b + 4 * g4 + i;
        const float x = ln.lam[b][i] - 0.5f * ln.tau[b];
        const float up = expf(x), down = expf(-x);
        const float km = ln.k[b][i] * up, qm = ln.q[b][i] * up;
        const float kb = ln.k[b][i] * down * s.beta[t];
        s.km[t * RS + kc] = km;
        s.qm[t * RS + kc] = qm;
        s.kb[t * RS + kc] = kb;
        kg[b][i] = km * ef;
        qg[i] = qm * ef;
        ke[b][i] = kb * et;
      }
      const int at = ((w * NB + b) * 64 + lane) * 4;
      *reinterpret_cast<f32x4*>(ops + kOpKE + at) = ke[b];
      *reinterpret_cast<f32x4*>(ops + kOpKG + at) = -kg[b];
      *reinterpret_cast<f32x4*>(ops + kOpQG + at) = qg;
    }
  }
  __syncthreads();

  // ---- A and P, block by block (10 each on and below the diagonal)
  for (int task = w; task < NB * (NB + 1); task += kThreads / 64) {
    const bool is_p = task >= NB * (NB + 1) / 2;
    int I = 0, J = is_p ? task - NB * (NB + 1) / 2 : task;
    while (J > I) J -= ++I;
    const float* left = (is_p ? s.qm : s.km) + (16 * I + n16) * RS + 4 * g4;
    const float* right = s.kb + (16 * J + n16) * RS + 4 * g4;
    f32x4 acc = zero4();
#pragma unroll
    for (int m = 0; m < D / 16; ++m) {
      f32x4 a = lds4(left + 16 * m);
      if (I != J) a *= lds4(s.pair + pair_index(I, J) * D + 16 * m + 4 * g4);
      acc = mfma4(a, lds4(right + 16 * m), acc);
    }
    float* dst = (is_p ? s.pm : s.am) + (16 * I + 4 * g4) * AS + 16 * J + n16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int over = I == J ? n16 - (4 * g4 + i) : -1;  // column beyond the row
      dst[i * AS] = over < 0 || (is_p && over == 0) ? acc[i] : 0.f;
    }
  }
  __syncthreads();

  // ---- T = (1 + A)^-1. Diagonal blocks: N = -A is strictly lower, N^16 = 0, so
  // the inverse is (1 + N)(1 + N^2)(1 + N^4)(1 + N^8). A product X Y takes X^T as
  // its left fragment, so every power is kept with its transpose.
  if (w < NB) {
    const float* a = s.am + 16 * w * AS + 16 * w;
    f32x4 n = -col4(a + 4 * g4 * AS + n16, AS), nt = -lds4(a + n16 * AS + 4 * g4);
    f32x4 r = n, rt = nt;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float one = 4 * g4 + i == n16 ? 1.f : 0.f;
      r[i] += one;
      rt[i] += one;
    }
#pragma unroll
    for (int step = 0; step < 3; ++step) {
      const f32x4 n2 = mfma4(nt, n, zero4()), n2t = mfma4(n, nt, zero4());
      const f32x4 r2 = mfma4(rt, n2, r), r2t = mfma4(n2, rt, rt);
      n = n2, nt = n2t, r = r2, rt = r2t;
    }
    float* dst = s.tm + (16 * w + 4 * g4) * AS + 16 * w + n16;
#pragma unroll
    for (int i = 0; i < 4; ++i) dst[i * AS] = r[i];
  }
  // V and dO (bf16) take the place of e^(lam - tau/2) q'
  {
    uint16_t* vo = reinterpret_cast<uint16_t*>(s.qm);
    const int c0 = (threadIdx.x & 15) * 8;
    for (int t = threadIdx.x >> 4; t < C; t += kThreads / 16) {
      u32x4 a = {0u, 0u, 0u, 0u}, b = a;
      if (t < ch.c) {
        a = *reinterpret_cast<const u32x4_u*>(p.v + (ch.t0 + t) * p.v_stride + h * D + c0);
        b = *reinterpret_cast<const u32x4_u*>(p.dout + (ch.t0 + t) * p.dout_stride + h * D + c0);
      }
      typedef u32x4 u32x4_8 __attribute__((aligned(8)));
      *reinterpret_cast<u32x4_8*>(vo + t * VS + c0) = a;
      *reinterpret_cast<u32x4_8*>(vo + t * VS + RS + c0) = b;
    }
  }
  __syncthreads();
  // T_IJ = -T_II sum_K A_IK T_KJ, one wave per block column
  if (w < NB - 1) {
    f32x4 t[NB];
    t[0] = col4(s.tm + (16 * w + 4 * g4) * AS + 16 * w + n16, AS);
    for (int I = w + 1; I < NB; ++I) {
      f32x4 acc = zero4();
#pragma unroll
      for (int d = 0; d < NB - 1; ++d)
        if (w + d < I) acc = mfma4(lds4(s.am + (16 * I + n16) * AS + 16 * (w + d) + 4 * g4), t[d], acc);
      acc = mfma4(lds4(s.tm + (16 * I + n16) * AS + 16 * I + 4 * g4), -acc, zero4());
#pragma unroll
      for (int d = 1; d < NB; ++d)
        if (w + d == I) t[d] = acc;
      float* dst = s.tm + (16 * I + 4 * g4) * AS + 16 * w + n16;
#pragma unroll
      for (int i = 0; i < 4; ++i) dst[i * AS] = acc[i];
    }
  }
  __syncthreads();

  // ---- products with T for the wave's 16 channels
  const uint16_t* vo = reinterpret_cast<const uint16_t*>(s.qm);
  f32x4 vv[NB], oo[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 16 * b + 4 * g4 + i;
      vv[b][i] = bf1(vo[t * VS + kc]);
      oo[b][i] = bf1(vo[t * VS + RS + kc]);
    }
  f32x4 y[NB];  // P^T dO
#pragma unroll
  for (int r = 0; r < NB; ++r) {
    f32x4 wt = zero4(), xx = zero4(), z = zero4();
    y[r] = zero4();
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if (b <= r) {
        const f32x4 t = lds4(s.tm + (16 * r + n16) * AS + 16 * b + 4 * g4);
        wt = mfma4(kg[b], t, wt);  // transposed: rows are channels
        xx = mfma4(t, vv[b], xx);
      }
      if (b >= r) {
        const int at = (16 * b + 4 * g4) * AS + 16 * r + n16;
        z = mfma4(ke[b], col4(s.tm + at, AS), z);  // transposed
        y[r] = mfma4(col4(s.pm + at, AS), oo[b], y[r]);
      }
    }
    const int at = ((r * 8 + w) * 64 + lane) * 4;
    *reinterpret_cast<f32x4*>(ops + kOpW + at) = -wt;
    *reinterpret_cast<f32x4*>(ops + kOpZ + at) = z;
#pragma unroll
    for (int i = 0; i < 4; ++i) ops[kOpX + (16 * r + 4 * g4 + i) * D + kc] = xx[i];
  }
#pragma unroll
  for (int r = 0; r < NB; ++r) {
    f32x4 d = zero4();
#pragma unroll
    for (int b = r; b < NB; ++b)
      d = mfma4(col4(s.tm + (16 * b + 4 * g4) * AS + 16 * r + n16, AS), y[b], d);
#pragma unroll
    for (int i = 0; i < 4; ++i) ops[kOpDV + (16 * r + 4 * g4 + i) * D + kc] = d[i];
  }
}

// ---------------------------------------------------------------------------
// Chains: the states up each (document, head), and the state gradients down.
// Value channels do not mix in either, so a wave owns 16 of them, with all 128 key
// channels in eight accumulator tiles.
constexpr int kChainWaves = 2;
constexpr int kParts = D / 16 / kChainWaves;

__device__ __forceinline__ float pool_at(const BwdParams& p, int64_t e) {
  if (p.state_dtype == KDA_STATE_FP8)
    return f8x2_lo(static_cast<const uint8_t*>(p.pool)[e])[0];
  const uint16_t b = static_cast<const uint16_t*>(p.pool)[e];
  return p.state_dtype == KDA_STATE_FP16 ? f16_lo(b) : bf1(b);
}

__global__ __launch_bounds__(64 * kChainWaves) void chain_kernel(BwdParams p, DocOrder ord) {
  const int64_t chains = int64_t(p.n_docs) * p.H;
  const int64_t id = int64_t(blockIdx.x) / kParts;
  const bool down = id & 1;
  const int64_t chain = id >> 1;
  if (chain >= chains) return;
  const int lane = threadIdx.x & 63;
  const int g4 = lane >> 4, n16 = lane & 15;
  const int v = 16 * (int(blockIdx.x % kParts) * kChainWaves + int(threadIdx.x >> 6)) + n16;
  const int h = int(chain % p.H);
  const int rank = int(chain / p.H);
  const int doc = ord.n > 0 ? ord.doc[rank] : rank;
  const int64_t t0 = p.cu_seqlens[doc];
  const int64_t len = int64_t(p.cu_seqlens[doc + 1]) - t0;
  const int32_t slot = p.state_indices[doc];
  const bool active = slot >= 0 && int64_t(slot) < p.num_slots;
  const int64_t chunks = (len + C - 1) / C;
  const int64_t state = (int64_t(doc) * p.H + h) * HEAD_ELEMS + v * D + 4 * g4;
  float* ops0 = p.ops + (doc_slot0(p.cu_seqlens, doc) * p.H + h) * int64_t(kOps);
  const int64_t step = int64_t(p.H) * kOps;

  f32x4 s[8];  // [key 16 m + 4 g4 + i][value v]
#pragma unroll
  for (int m = 0; m < 8; ++m) s[m] = zero4();

  if (!down) {
    if (!active || len == 0) return;
    if (p.use_initial) {
      const int64_t e = int64_t(slot) * p.slot_stride + int64_t(h) * HEAD_ELEMS + v * D + 4 * g4;
#pragma unroll
      for (int m = 0; m < 8; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[m][i] = pool_at(p, e + 16 * m + i);
    }
    for (int64_t n = 0; n < chunks; ++n) {
      float* ops = ops0 + n * step;
#pragma unroll
      for (int m = 0; m < 8; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) ops[kOpS + (16 * m + 4 * g4 + i) * D + v] = s[m][i];
      f32x4 x[NB];
#pragma unroll
      for (int r = 0; r < NB; ++r) {
        x[r] = col4(ops + kOpX + (16 * r + 4 * g4) * D + v, D);
#pragma unroll
        for (int m = 0; m < 8; ++m)
          x[r] = mfma4(lds4(ops + kOpW + ((r * 8 + m) * 64 + lane) * 4), s[m], x[r]);
#pragma unroll
        for (int i = 0; i < 4; ++i) ops[kOpX + (16 * r + 4 * g4 + i) * D + v] = x[r][i];
      }
      if (n + 1 == chunks) return;  // the state after the last chunk is not needed
#pragma unroll
      for (int m = 0; m < 8; ++m) {
        s[m] *= lds4(ops + kOpEG + 16 * m + 4 * g4);
#pragma unroll
        for (int r = 0; r < NB; ++r)
          s[m] = mfma4(lds4(ops + kOpKE + ((m * NB + r) * 64 + lane) * 4), x[r], s[m]);
      }
    }
    return;
  }

  if (p.d_final && active) {
#pragma unroll
    for (int m = 0; m < 8; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[m][i] = p.d_final[state + 16 * m + i];
  }
  if (active) {
    for (int64_t n = chunks - 1; n >= 0; --n) {
      float* ops = ops0 + n * step;
      const int64_t tc = t0 + n * C;
      const int c = int(min<int64_t>(C, len - n * C));
#pragma unroll
      for (int m = 0; m < 8; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) ops[kOpDS + (16 * m + 4 * g4 + i) * D + v] = s[m][i];
      f32x4 x[NB], o[NB];
#pragma unroll
      for (int r = 0; r < NB; ++r) {
        x[r] = col4(ops + kOpDV + (16 * r + 4 * g4) * D + v, D);
#pragma unroll
        for (int m = 0; m < 8; ++m)
          x[r] = mfma4(lds4(ops + kOpZ + ((r * 8 + m) * 64 + lane) * 4), s[m], x[r]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ops[kOpDV + (16 * r + 4 * g4 + i) * D + v] = x[r][i];
          const int t = 16 * r + 4 * g4 + i;
          o[r][i] = t < c ? bf1(p.dout[(tc + t) * p.dout_stride + h * D + v]) : 0.f;
        }
      }
#pragma unroll
      for (int m = 0; m < 8; ++m) {
        s[m] *= lds4(ops + kOpEG + 16 * m + 4 * g4);
#pragma unroll
        for (int r = 0; r < NB; ++r) {
          s[m] = mfma4(lds4(ops + kOpKG + ((m * NB + r) * 64 + lane) * 4), x[r], s[m]);
          s[m] = mfma4(lds4(ops + kOpQG + ((m * NB + r) * 64 + lane) * 4), o[r], s[m]);
        }
      }
    }
  }
  if (p.d_initial) {
#pragma unroll
    for (int m = 0; m < 8; ++m) *reinterpret_cast<f32x4*>(p.d_initial + state + 16 * m) = s[m];
  }
}

// ---------------------------------------------------------------------------
// Gradients: one workgroup per (chunk, head); a wave owns 16 key channels of all
// tokens, so that the decays and the sums over tokens stay in its registers.
struct GradSmem {
  float dO[C * RS], dV[C * RS], x[C * RS];
  float dp[C * AS], da[C * AS];
  float red[4][8][C];  // sums over a wave's 16 channels, per token
  float diag[C];       // DP's diagonal
  float rq[C], rk[C], beta[C];
};

__device__ __forceinline__ void zero_row(uint16_t* p, int64_t t, int64_t stride, int64_t at, int n) {
  for (int e = threadIdx.x; e < n; e += kThreads) p[t * stride + at + e] = 0;
}

__global__ __launch_bounds__(kThreads) void grad_kernel(BwdParams p) {
  extern __shared__ __align__(16) float smem_raw[];
  GradSmem& s = *reinterpret_cast<GradSmem*>(smem_raw);
  const int64_t sigma = blockIdx.x;
  const int h = blockIdx.y;
  const Chunk ch = chunk_of(p, sigma);
  float* partial = p.partial + (sigma * p.H + h) * int64_t(2 * D);
  const bool per_head = p.gate_mode & KDA_GATE_PER_HEAD;
  if (ch.c == 0 || !ch.active) {
    if (threadIdx.x < 2 * D) partial[threadIdx.x] = 0.f;
    for (int t = 0; t < ch.c; ++t) {
      zero_row(p.dq, ch.t0 + t, p.dq_stride, int64_t(h) * D, D);
      zero_row(p.dk, ch.t0 + t, p.dk_stride, int64_t(h) * D, D);
      zero_row(p.dv, ch.t0 + t, p.dv_stride, int64_t(h) * D, D);
      zero_row(p.dg, ch.t0 + t, p.dg_stride, per_head ? h : int64_t(h) * D, per_head ? 1 : D);
      zero_row(p.dbeta, ch.t0 + t, p.dbeta_stride, h, 1);
    }
    return;
  }
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int g4 = lane >> 4, n16 = lane & 15;
  const int kc = 16 * w + n16;
  const float* ops = p.ops + (sigma * p.H + h) * int64_t(kOps);

  token_scalars(p, ch, h, s.rq, s.rk, s.beta);
  {
    const int c0 = (threadIdx.x & 31) * 4;
    for (int t = threadIdx.x >> 5; t < C; t += kThreads / 32) {
      const f32x4 dv = lds4(ops + kOpDV + t * D + c0);
      *reinterpret_cast<f32x4*>(s.dV + t * RS + c0) = dv;
      *reinterpret_cast<f32x4*>(s.x + t * RS + c0) = lds4(ops + kOpX + t * D + c0);
      f32x4 o = zero4();
      if (t < ch.c) {
        const uint16_t* src = p.dout + (ch.t0 + t) * p.dout_stride + h * D + c0;
        uint16_t* dst = p.dv + (ch.t0 + t) * p.dv_stride + h * D + c0;
        typedef u32x2 u32x2_u __attribute__((aligned(2)));
        const u32x2 b = *reinterpret_cast<const u32x2_u*>(src);
        o = f32x4{bf_lo(b[0]), bf_hi(b[0]), bf_lo(b[1]), bf_hi(b[1])};
        *reinterpret_cast<u32x2_u*>(dst) = u32x2{pack_bf16x2(dv[0], dv[1]), pack_bf16x2(dv[2], dv[3])};
      }
      *reinterpret_cast<f32x4*>(s.dO + t * RS + c0) = o;
    }
  }
  __syncthreads();

  // ---- DP = tril(dO x^T), DA = -tril(dV x^T, -1). A token's use of its own key has no
  // decay: DP's diagonal is kept apart, out of the sums that give dg.
  for (int task = w; task < NB * (NB + 1); task += kThreads / 64) {
    const bool is_p = task >= NB * (NB + 1) / 2;
    int I = 0, J = is_p ? task - NB * (NB + 1) / 2 : task;
    while (J > I) J -= ++I;
    const float* left = (is_p ? s.dO : s.dV) + (16 * I + n16) * RS + 4 * g4;
    const float* right = s.x + (16 * J + n16) * RS + 4 * g4;
    f32x4 acc = zero4();
#pragma unroll
    for (int m = 0; m < D / 16; ++m) acc = mfma4(lds4(left + 16 * m), lds4(right + 16 * m), acc);
    if (!is_p) acc = -acc;
    float* dst = (is_p ? s.dp : s.da) + (16 * I + 4 * g4) * AS + 16 * J + n16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int over = I == J ? n16 - (4 * g4 + i) : -1;
      dst[i * AS] = over < 0 ? acc[i] : 0.f;
      if (is_p && over == 0) s.diag[16 * I + n16] = acc[i];
    }
  }

  // ---- dO S^T, dV S^T, x dS^T for the wave's channels
  f32x4 sq[NB], sk[NB], se[NB];
  float last = 0.f;  // e^Gl sum_v S dS, later with the writers' part
  {
#pragma unroll
    for (int r = 0; r < NB; ++r) sq[r] = sk[r] = se[r] = zero4();
    const float* S = ops + kOpS + kc * D + 4 * g4;
    const float* dS = ops + kOpDS + kc * D + 4 * g4;
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      const f32x4 a = lds4(S + 16 * m), b = lds4(dS + 16 * m);
#pragma unroll
      for (int i = 0; i < 4; ++i) last = fmaf(a[i], b[i], last);
#pragma unroll
      for (int r = 0; r < NB; ++r) {
        const int at = (16 * r + n16) * RS + 16 * m + 4 * g4;
        sq[r] = mfma4(lds4(s.dO + at), a, sq[r]);
        sk[r] = mfma4(lds4(s.dV + at), a, sk[r]);
        se[r] = mfma4(lds4(s.x + at), b, se[r]);
      }
    }
    last = rows_sum(last) * ops[kOpEG + kc];
  }
  Lane ln;
  load_lane<true>(p, ch, h, kc, g4, s.rq, s.rk, ln);
  __syncthreads();

  // ---- inside the chunk: readers' rows and writers' columns
  f32x4 up[NB], km[NB], qm[NB], kb[NB];
  float bt[NB][4];
  float fI[NB], tJ[NB];  // e^(from the chunk's start to the block's middle), (to the end)
  {
    float o = 0.f;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      fI[b] = expf(o + 0.5f * ln.tau[b]);
      o += ln.tau[b];
    }
    o = 0.f;
#pragma unroll
    for (int b = NB - 1; b >= 0; --b) {
      tJ[b] = expf(o + 0.5f * ln.tau[b]);
      o += ln.tau[b];
    }
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = ln.lam[b][i] - 0.5f * ln.tau[b];
        bt[b][i] = s.beta[16 * b + 4 * g4 + i];
        up[b][i] = expf(x);
        km[b][i] = ln.k[b][i] * up[b][i];
        qm[b][i] = ln.q[b][i] * up[b][i];
        kb[b][i] = ln.k[b][i] * expf(-x) * bt[b][i];
      }
  }
  f32x4 cq[NB], ck[NB], cc[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) cq[b] = ck[b] = cc[b] = zero4();
#pragma unroll
  for (int I = 0; I < NB; ++I) {
    float mid = 0.f;
#pragma unroll
    for (int J = I; J >= 0; --J) {
      f32x4 kj = kb[J], ki = km[I], qi = qm[I];
      if (J < I) {
        const float f = expf(0.5f * (ln.tau[I] + ln.tau[J]) + mid);
        mid += ln.tau[J];
        kj *= f;
        ki *= f;
        qi *= f;
      }
      const int row = (16 * I + n16) * AS + 16 * J + 4 * g4;
      const int col = (16 * I + 4 * g4) * AS + 16 * J + n16;
      cq[I] = mfma4(lds4(s.dp + row), kj, cq[I]);
      ck[I] = mfma4(lds4(s.da + row), kj, ck[I]);
      cc[J] = mfma4(col4(s.dp + col, AS), qi, cc[J]);
      cc[J] = mfma4(col4(s.da + col, AS), ki, cc[J]);
    }
  }

  // ---- put together; sums over the channels per token through LDS
  float dG[NB][4];
  float ends = 0.f;
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float e = up[b][i];
      const float down = expf(0.5f * ln.tau[b] - ln.lam[b][i]);
      const float end = down * tJ[b] * se[b][i];
      const float self = s.diag[16 * b + 4 * g4 + i];
      float dq = e * fmaf(fI[b], sq[b][i], cq[b][i]);         // dq'
      const float dr = e * fmaf(-fI[b], sk[b][i], ck[b][i]);  // drow
      float col = fmaf(down, cc[b][i], end);
      const float kbeta = ln.k[b][i] * bt[b][i];
      ends = fmaf(kbeta, end, ends);
      dG[b][i] = ln.q[b][i] * dq + ln.k[b][i] * dr - kbeta * col;
      dq = fmaf(self, kbeta, dq);
      col = fmaf(self, ln.q[b][i], col);
      cq[b][i] = dq * p.scale;
      ck[b][i] = fmaf(bt[b][i], col, dr);
      const float a0 = row16_sum(ln.q[b][i] * dq);  // q_hat . dq_hat
      const float a1 = row16_sum(ln.k[b][i] * ck[b][i]);
      const float a2 = row16_sum(ln.k[b][i] * col);
      if (n16 == 0) {
        const int t = 16 * b + 4 * g4 + i;
        s.red[0][w][t] = a0;
        s.red[1][w][t] = a1;
        s.red[2][w][t] = a2;
      }
    }
  // dg: the suffix sums over the chunk's tokens
  float sum_b = 0.f, sum_a = 0.f;  // of ddt_bias, dA_log
  {
    float after = last + rows_sum(ends);
#pragma unroll
    for (int b = NB - 1; b >= 0; --b) {
      float sum = 0.f;
#pragma unroll
      for (int i = 3; i >= 0; --i) {
        sum += dG[b][i];
        dG[b][i] = sum;
      }
      const float s1 = __shfl_xor(sum, 16);
      const float pair = sum + s1;
      const float other = __shfl_xor(pair, 32);
      const float later = after + ((g4 & 1) ? 0.f : s1) + ((g4 & 2) ? 0.f : other);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float dg = dG[b][i] + later;
        dG[b][i] = dg;
        const float inside = ln.slope[b][i] != 0.f ? ln.g[b][i] : 0.f;
        sum_b = fmaf(dg, ln.slope[b][i], sum_b);
        sum_a = fmaf(dg, inside, sum_a);
        if (per_head) {
          const float a3 = row16_sum(dg);
          if (n16 == 0) s.red[3][w][16 * b + 4 * g4 + i] = a3;
        }
      }
      after += pair + other;
    }
  }
  sum_b = rows_sum(sum_b);
  sum_a = rows_sum(sum_a);
  if (g4 == 0) {
    partial[kc] = sum_b;
    partial[D + kc] = sum_a;
  }
  __syncthreads();
  if (threadIdx.x < C * 4) {  // add the eight waves' sums
    const int which = threadIdx.x / C, t = threadIdx.x % C;
    if (which < 3 || per_head) {
      float x = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) x += s.red[which][i][t];
      s.red[which][0][t] = x;
      if (which == 2 && t < ch.c) {
        if (!(p.gate_mode & KDA_BETA_PRESIGMOID)) x *= s.beta[t] * (1.f - s.beta[t]);
        p.dbeta[(ch.t0 + t) * p.dbeta_stride + h] = to_bf16(x);
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 16 * b + 4 * g4 + i;
      if (t < ch.c) {
        // q' = scale q_hat: q_hat (q_hat . dq_hat) from q' and its dot product
        const float rq = s.rq[t], rk = s.rk[t];
        const float qhat = bf1(p.q[(ch.t0 + t) * p.q_stride + h * D + kc]) * rq;
        const float dq = rq * fmaf(-qhat, s.red[0][0][t], cq[b][i]);
        const float dk = rk * fmaf(-ln.k[b][i], s.red[1][0][t], ck[b][i]);
        p.dq[(ch.t0 + t) * p.dq_stride + h * D + kc] = to_bf16(dq);
        p.dk[(ch.t0 + t) * p.dk_stride + h * D + kc] = to_bf16(dk);
        if (!per_head)
          p.dg[(ch.t0 + t) * p.dg_stride + h * D + kc] = to_bf16(dG[b][i] * ln.slope[b][i]);
        else if (w == 0 && n16 == 0)
          p.dg[(ch.t0 + t) * p.dg_stride + h] = to_bf16(s.red[3][0][t] * ln.slope[b][i]);
      }
    }
}

// dA_log and ddt_bias: the partial sums of a head, added in the order of the chunk
// slots by 8 groups of 128 lanes (a channel each), then group by group.
__global__ __launch_bounds__(1024) void param_kernel(BwdParams p) {
  __shared__ float sum[2][8][D];
  __shared__ float half[4];
  const int h = blockIdx.x;
  const int c = threadIdx.x & (D - 1), grp = threadIdx.x / D;
  float b = 0.f, a = 0.f;
  for (int64_t n = grp; n < p.slots; n += 8) {
    const float* x = p.partial + (n * p.H + h) * int64_t(2 * D);
    b += x[c];
    a += x[D + c];
  }
  sum[0][grp][c] = b;
  sum[1][grp][c] = a;
  __syncthreads();
  const bool per_head = p.gate_mode & KDA_GATE_PER_HEAD;
  float t = 0.f;
  if (grp < 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) t += sum[grp][i][c];
    if (grp == 0 && !per_head && p.ddt_bias) p.ddt_bias[h * D + c] = t;
    // a head's one value: the sum over its channels
    t = rows_sum(row16_sum(t));
    if ((threadIdx.x & 63) == 0) half[threadIdx.x >> 6] = t;
  }
  __syncthreads();
  if (grp < 2 && c == 0) {
    t = half[2 * grp] + half[2 * grp + 1];
    if (grp == 1 && p.dA_log) p.dA_log[h] = t;
    if (grp == 0 && per_head && p.ddt_bias) p.ddt_bias[h] = t;
  }
}

// ---------------------------------------------------------------------------
// host

int64_t slots_of(int32_t n_docs, int64_t total_tokens) { return n_docs + total_tokens / C; }

// Dynamic LDS beyond 64 KiB is allowed once per kernel.
hipError_t allow_lds() {
  static const hipError_t e = [] {
    const hipError_t a = hipFuncSetAttribute(reinterpret_cast<const void*>(prep_kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize,
                                             int(sizeof(PrepSmem)));
    if (a != hipSuccess) return a;
    return hipFuncSetAttribute(reinterpret_cast<const void*>(grad_kernel),
                               hipFuncAttributeMaxDynamicSharedMemorySize, int(sizeof(GradSmem)));
  }();
  return e;
}

hipError_t launch_backward(const BwdParams& p, int64_t total_tokens, const int32_t* cu_host,
                           hipStream_t stream) {
  if (const hipError_t e = allow_lds()) return e;
  const int64_t chains = int64_t(p.n_docs) * p.H;
  if (p.slots > 0x7fffffff || chains * 2 * kParts > 0x7fffffff) return hipErrorInvalidValue;
  DocOrder ord;
  ord.n = 0;
  if (p.n_docs <= kMaxOrderedDocs) {  // the longest documents first
    for (int d = 0; d < p.n_docs; ++d) {
      const int len = cu_host[d + 1] - cu_host[d];
      int at = d;
      for (; at > 0 && cu_host[ord.doc[at - 1] + 1] - cu_host[ord.doc[at - 1]] < len; --at)
        ord.doc[at] = ord.doc[at - 1];
      ord.doc[at] = d;
    }
    ord.n = p.n_docs;
  }
  if (total_tokens > 0) {
    hipLaunchKernelGGL(prep_kernel, dim3(unsigned(p.slots), unsigned(p.H)), dim3(kThreads),
                       sizeof(PrepSmem), stream, p);
    if (const hipError_t e = hipGetLastError()) return e;
  }
  if (total_tokens > 0 || p.d_initial) {
    hipLaunchKernelGGL(chain_kernel, dim3(unsigned(chains * 2 * kParts)), dim3(64 * kChainWaves),
                       0, stream, p, ord);
    if (const hipError_t e = hipGetLastError()) return e;
  }
  if (total_tokens > 0) {
    hipLaunchKernelGGL(grad_kernel, dim3(unsigned(p.slots), unsigned(p.H)), dim3(kThreads),
                       sizeof(GradSmem), stream, p);
    if (const hipError_t e = hipGetLastError()) return e;
  }
  if (p.dA_log || p.ddt_bias) {
    BwdParams all = p;
    if (total_tokens == 0) all.slots = 0;  // nothing was written: the sums are zero
    hipLaunchKernelGGL(param_kernel, dim3(unsigned(p.H)), dim3(1024), 0, stream, all);
  }
  return hipGetLastError();
}

}  // namespace
}  // namespace kda

extern "C" size_t kda_prefill_backward_workspace_size(int32_t n_docs, int64_t total_tokens,
                                                      int32_t H, int32_t K, int32_t V) {
  if (n_docs < 0 || total_tokens < 0 || total_tokens > INT32_MAX || H < 1 || H > 65535 ||
      K != kda::D || V != kda::D)
    return 0;
  return size_t(kda::slots_of(n_docs, total_tokens)) * size_t(H) * (kda::kOps + 2 * kda::D) * 4;
}

extern "C" kda_status kda_prefill_varlen_backward(
    int32_t n_docs, int64_t total_tokens, int32_t H, int32_t K, int32_t V,
    const int32_t* cu_seqlens_host, const int32_t* cu_seqlens, const void* q,
    int64_t q_tok_stride, const void* k, int64_t k_tok_stride, const void* v,
    int64_t v_tok_stride, const void* g_raw, int64_t g_tok_stride, const void* beta_raw,
    int64_t beta_tok_stride, const float* A_log, const float* dt_bias, float lower_bound,
    float scale, int32_t gate_mode, int32_t state_dtype, const void* state_pool,
    int64_t num_slots, int64_t slot_stride, const int32_t* state_indices,
    int32_t use_initial_state, const void* d_out, int64_t d_out_tok_stride,
    const float* d_final_state, void* dq, int64_t dq_tok_stride, void* dk, int64_t dk_tok_stride,
    void* dv, int64_t dv_tok_stride, void* dg, int64_t dg_tok_stride, void* dbeta,
    int64_t dbeta_tok_stride, float* dA_log, float* ddt_bias, float* d_initial_state,
    void* workspace, size_t workspace_bytes, hipStream_t stream) {
  using kda::D;
  if (n_docs < 0 || total_tokens < 0 || H < 1 || num_slots < 0) return KDA_ERR_BAD_SHAPE;
  if (K != D || V != D || H > 65535) return KDA_ERR_UNSUPPORTED;
  if (!(lower_bound >= -5.5f && lower_bound <= 5.5f)) return KDA_ERR_UNSUPPORTED;
  if (gate_mode & ~(KDA_GATE_PRECOMPUTED | KDA_BETA_PRESIGMOID | KDA_GATE_PER_HEAD))
    return KDA_ERR_UNSUPPORTED;
  const bool pre = gate_mode & KDA_GATE_PRECOMPUTED;
  if (pre && (lower_bound > 0.0f || dA_log || ddt_bias)) return KDA_ERR_UNSUPPORTED;
  if (state_dtype < KDA_STATE_BF16 || state_dtype > KDA_STATE_FP8) return KDA_ERR_UNSUPPORTED;
  if (!cu_seqlens_host) return KDA_ERR_NULL_POINTER;
  if (cu_seqlens_host[0] != 0) return KDA_ERR_BAD_SEQLENS;
  for (int32_t d = 0; d < n_docs; ++d)
    if (cu_seqlens_host[d + 1] < cu_seqlens_host[d]) return KDA_ERR_BAD_SEQLENS;
  if (int64_t(cu_seqlens_host[n_docs]) != total_tokens) return KDA_ERR_BAD_SEQLENS;
  if (n_docs > 0) {
    if (!pre && (!A_log || !dt_bias)) return KDA_ERR_NULL_POINTER;
    if (!cu_seqlens || !state_indices) return KDA_ERR_NULL_POINTER;
    if (total_tokens > 0 && (!q || !k || !v || !g_raw || !beta_raw || !d_out || !dq || !dk ||
                             !dv || !dg || !dbeta))
      return KDA_ERR_NULL_POINTER;
    if (use_initial_state && num_slots > 0 && !state_pool) return KDA_ERR_NULL_POINTER;
    const int64_t W = int64_t(H) * D;
    const int64_t gw = (gate_mode & KDA_GATE_PER_HEAD) ? H : W;
    const int64_t in[] = {q_tok_stride, k_tok_stride, v_tok_stride, g_tok_stride,
                          beta_tok_stride, d_out_tok_stride, slot_stride};
    for (const int64_t s : in)
      if (s < 0) return KDA_ERR_BAD_STRIDE;
    const int64_t out[][2] = {{dq_tok_stride, W}, {dk_tok_stride, W}, {dv_tok_stride, W},
                              {dg_tok_stride, gw}, {dbeta_tok_stride, H}};
    for (const auto& s : out)
      if (s[0] < 0 || (total_tokens > 1 && s[0] < s[1])) return KDA_ERR_BAD_STRIDE;
    if (use_initial_state && num_slots > 1 && slot_stride < W * D) return KDA_ERR_BAD_STRIDE;
    if (reinterpret_cast<uintptr_t>(d_initial_state) & 15u) return KDA_ERR_UNSUPPORTED;
    if (total_tokens > 0) {
      if (workspace_bytes < kda_prefill_backward_workspace_size(n_docs, total_tokens, H, K, V))
        return KDA_ERR_WORKSPACE_TOO_SMALL;
      if (!workspace) return KDA_ERR_NULL_POINTER;
      if (reinterpret_cast<uintptr_t>(workspace) & 255u) return KDA_ERR_UNSUPPORTED;
    }
  }

  kda::BwdParams p;
  p.n_docs = n_docs;
  p.H = H;
  p.slots = kda::slots_of(n_docs, total_tokens);
  p.cu_seqlens = cu_seqlens;
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.g = static_cast<const uint16_t*>(g_raw);
  p.beta = static_cast<const uint16_t*>(beta_raw);
  p.q_stride = q_tok_stride;
  p.k_stride = k_tok_stride;
  p.v_stride = v_tok_stride;
  p.g_stride = g_tok_stride;
  p.beta_stride = beta_tok_stride;
  p.A_log = A_log;
  p.dt_bias = dt_bias;
  p.lower_bound = lower_bound;
  p.scale = scale;
  p.gate_mode = gate_mode;
  p.state_dtype = state_dtype;
  p.use_initial = use_initial_state ? 1 : 0;
  p.pool = state_pool;
  p.num_slots = num_slots;
  p.slot_stride = slot_stride;
  p.state_indices = state_indices;
  p.dout = static_cast<const uint16_t*>(d_out);
  p.dout_stride = d_out_tok_stride;
  p.d_final = d_final_state;
  p.dq = static_cast<uint16_t*>(dq);
  p.dk = static_cast<uint16_t*>(dk);
  p.dv = static_cast<uint16_t*>(dv);
  p.dg = static_cast<uint16_t*>(dg);
  p.dbeta = static_cast<uint16_t*>(dbeta);
  p.dq_stride = dq_tok_stride;
  p.dk_stride = dk_tok_stride;
  p.dv_stride = dv_tok_stride;
  p.dg_stride = dg_tok_stride;
  p.dbeta_stride = dbeta_tok_stride;
  p.dA_log = dA_log;
  p.ddt_bias = ddt_bias;
  p.d_initial = d_initial_state;
  p.ops = static_cast<float*>(workspace);
  p.partial = p.ops + (total_tokens > 0 ? p.slots * int64_t(H) * kda::kOps : 0);
  if (n_docs == 0 && !dA_log && !ddt_bias) return KDA_OK;
  return kda::launch_backward(p, total_tokens, cu_seqlens_host, stream) == hipSuccess
             ? KDA_OK : KDA_ERR_LAUNCH;
}
