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
// Each weight e^(G_r-G_j) grows with dg_t for all j < t <= r, so dg_t is the sum over
// those pairs of their part in the loss, with S as a token before all others and dS as one
// behind them (grad_kernel says how it adds them up).
//
// Decays. A chunk is four 16-token blocks. Inside a block the weight of a pair is a
// reader's factor from the block's middle times a writer's factor to it, both
// within e^(+-44) (|lower_bound| <= 5.5); pairs of different blocks take what lies between
// the two middles, or, factored at the blocks' borders, weights of at most 1. All of them
// are products of the a_t = e^g_t.
//
// Precision. States, sums and decays are fp32. Products run either on fp32 MFMA or on
// fp16 MFMA with both sides split into high and low parts (22 bits and a sign each, three
// terms), which leaves out 2^-22 of a term, two bits more than fp32 rounds, in 3/16 of its
// time; fp16's range is met by power-of-two scales. Operand tiles are read as consecutive
// contraction indices per lane, in an order that lets an accumulator tile (rows
// 4 (lane / 16) + i) serve as the next product's right operand as it is.

#include <math.h>
#include <stdint.h>

#include "kda_bwd.h"

namespace kda {
namespace bwd {
namespace {

int64_t slots_of(int32_t n_docs, int64_t total_tokens) { return n_docs + total_tokens / C; }

hipError_t launch_backward(const BwdParams& p, int64_t total_tokens, const int32_t* cu_host,
                           hipStream_t stream) {
  const int64_t chains = int64_t(p.n_docs) * p.H;
  if (p.slots > 0x7fffffff || chains > 0x7fffffff / 16) return hipErrorInvalidValue;
  DocOrder ord;
  ord.n = ord.deep = 0;
  if (p.n_docs <= kMaxOrderedDocs) {  // the longest documents first
    for (int d = 0; d < p.n_docs; ++d) {
      const int len = cu_host[d + 1] - cu_host[d];
      int at = d;
      for (; at > 0 && cu_host[ord.doc[at - 1] + 1] - cu_host[ord.doc[at - 1]] < len; --at)
        ord.doc[at] = ord.doc[at - 1];
      ord.doc[at] = d;
    }
    ord.n = p.n_docs;
    while (ord.deep < ord.n &&
           deep_chains(total_tokens, p.H, ord.deep,
                       cu_host[ord.doc[ord.deep] + 1] - cu_host[ord.doc[ord.deep]]))
      ++ord.deep;
  }
  if (total_tokens > 0)
    if (const hipError_t e = launch_prep(p, stream)) return e;
  if (p.n_docs > 0 && (total_tokens > 0 || p.d_initial))
    if (const hipError_t e = launch_chains(p, ord, stream)) return e;
  if (total_tokens > 0)
    if (const hipError_t e = launch_grads(p, stream)) return e;
  if (p.dA_log || p.ddt_bias) {
    BwdParams all = p;
    if (total_tokens == 0) all.slots = 0;  // nothing was written: the sums are zero
    return launch_params(all, stream);
  }
  return hipSuccess;
}

}  // namespace
}  // namespace bwd
}  // namespace kda

extern "C" size_t kda_prefill_backward_workspace_size(int32_t n_docs, int64_t total_tokens,
                                                      int32_t H, int32_t K, int32_t V) {
  if (n_docs < 0 || total_tokens < 0 || total_tokens > INT32_MAX || H < 1 || H > 65535 ||
      K != kda::D || V != kda::D)
    return 0;
  return size_t(kda::bwd::slots_of(n_docs, total_tokens)) * size_t(H) *
         (kda::bwd::kOps + 2 * kda::D * 4);
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
  if (!(lower_bound >= -5.5f && lower_bound <= 0.0f)) return KDA_ERR_UNSUPPORTED;
  if (gate_mode & ~(KDA_GATE_PRECOMPUTED | KDA_BETA_PRESIGMOID | KDA_GATE_PER_HEAD))
    return KDA_ERR_UNSUPPORTED;
  const bool pre = gate_mode & KDA_GATE_PRECOMPUTED;
  if (pre && (dA_log || ddt_bias)) return KDA_ERR_UNSUPPORTED;
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
    // a chunk's rows are addressed by 32-bit offsets
    constexpr int64_t kMaxStride = int64_t(1) << 25;
    for (int i = 0; i < 6; ++i)
      if (in[i] > kMaxStride) return KDA_ERR_UNSUPPORTED;
    const int64_t out[][2] = {{dq_tok_stride, W}, {dk_tok_stride, W}, {dv_tok_stride, W},
                              {dg_tok_stride, gw}, {dbeta_tok_stride, H}};
    for (const auto& s : out)
      if (s[0] < 0 || (total_tokens > 1 && s[0] < s[1])) return KDA_ERR_BAD_STRIDE;
    for (const auto& s : out)
      if (s[0] > kMaxStride) return KDA_ERR_UNSUPPORTED;
    if (use_initial_state && num_slots > 1 && slot_stride < W * D) return KDA_ERR_BAD_STRIDE;
    if (reinterpret_cast<uintptr_t>(d_initial_state) & 15u) return KDA_ERR_UNSUPPORTED;
    if (total_tokens > 0) {
      if (workspace_bytes < kda_prefill_backward_workspace_size(n_docs, total_tokens, H, K, V))
        return KDA_ERR_WORKSPACE_TOO_SMALL;
      if (!workspace) return KDA_ERR_NULL_POINTER;
      if (reinterpret_cast<uintptr_t>(workspace) & 255u) return KDA_ERR_UNSUPPORTED;
    }
  }

  kda::bwd::BwdParams p;
  p.n_docs = n_docs;
  p.H = H;
  p.slots = kda::bwd::slots_of(n_docs, total_tokens);
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
  p.ops = static_cast<uint8_t*>(workspace);
  p.partial = reinterpret_cast<float*>(
      p.ops + (total_tokens > 0 ? p.slots * int64_t(H) * kda::bwd::kOps : 0));
  if (n_docs == 0 && !dA_log && !ddt_bias) return KDA_OK;
  return kda::bwd::launch_backward(p, total_tokens, cu_seqlens_host, stream) == hipSuccess
             ? KDA_OK : KDA_ERR_LAUNCH;
}
