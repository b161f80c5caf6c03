/*
 * kda_backward.h -- gradients of the varlen prefill (kda.h), for training.
 *
 * kda_prefill_varlen runs the gated delta-rule recurrence over packed documents;
 * the call here takes the same inputs and the gradient of a loss by its outputs,
 * and returns the gradients by every input. Nothing is kept between the two
 * calls: the states the gradient needs are computed again.
 *
 * With a_t = exp(g_t), everything per (document, head), S[v][c]:
 *   forward  S' = S_{t-1} diag(a_t), x_t = v_t - S' k_hat, u_t = beta_t x_t,
 *            S_t = S' + u_t k_hat^T, o_t = scale S_t q_hat
 *   adjoint  dS += scale do_t q_hat^T,  dq_hat = scale S_t^T do_t,
 *            dv_t = beta_t dS k_hat,  dbeta_t = (dS k_hat) . x_t,
 *            dk_hat = dS^T u_t - S'^T dv_t,  dS -= dv_t k_hat^T,
 *            dg_t[c] = sum_v dS[v][c] S'[v][c],  dS = dS diag(a_t)
 * and through the prologue of kda.h: the L2 norms of q and k, the gate and its
 * clamp, the sigmoid of beta.
 *
 * Conventions, layouts, gate modes and errors are those of kda.h.
 */
#ifndef KDA_BACKWARD_H_
#define KDA_BACKWARD_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * kda_prefill_backward_workspace_size -- bytes of device workspace
 * kda_prefill_varlen_backward needs for these sizes (0 when K or V is not 128 or
 * a size is invalid). Pure host arithmetic: about 7.0 KB per token and head (per
 * 64-token chunk and head: the state that enters it, the state gradient that
 * leaves it, and the chunk's operands, fp32).
 */
size_t kda_prefill_backward_workspace_size(int32_t n_docs, int64_t total_tokens, int32_t H,
                                           int32_t K, int32_t V);

/*
 * kda_prefill_varlen_backward -- gradients of one kda_prefill_varlen call.
 *
 *  n_docs .. state_dtype  as for kda_prefill_varlen
 *  state_pool, num_slots, slot_stride, state_indices
 *                     the pool as it was BEFORE the forward call (which writes
 *                     final states into it); only read, and only with
 *                     use_initial_state (may be NULL without; num_slots still
 *                     bounds the indices). A document whose slot lies outside
 *                     [0, num_slots) was inactive: its gradients are +0.0 and it
 *                     adds nothing to dA_log and ddt_bias. Two documents may
 *                     share a slot here (it is only read).
 *  use_initial_state  1: chains started from their slots; 0: from zeros
 *  d_out              bf16, the gradient at `out`, element (t, h*128 + v) at
 *                     t*d_out_tok_stride + h*128 + v
 *  d_final_state      fp32 [n_docs, H, 128, 128], element (v, c) at v*128 + c: the
 *                     gradient at the final states (taken before they are rounded
 *                     to the pool's type); NULL: zeros
 *  dq, dk, dv         bf16 out, laid out like q, k, v with strides of their own
 *  dg                 bf16 out, like g_raw: the gradient at the gate logits (or at
 *                     the log-decay); zero where the clamp held: below
 *                     lower_bound, or with KDA_GATE_PRECOMPUTED outside
 *                     [lower_bound, 0]. With KDA_GATE_PER_HEAD one value a head.
 *  dbeta              bf16 out, like beta_raw
 *  dA_log             fp32 [H] out, ddt_bias fp32 [H*128] (or [H]) out: summed over
 *                     all tokens in an order that depends on the sizes only; each
 *                     may be NULL, and must be with KDA_GATE_PRECOMPUTED
 *  d_initial_state    fp32 [n_docs, H, 128, 128] out, 16-byte aligned: the gradient
 *                     at the state each document started from (with
 *                     use_initial_state = 0: at the zeros); NULL: not stored. May
 *                     be d_final_state itself.
 *  workspace          >= kda_prefill_backward_workspace_size(...) bytes, 256-byte
 *                     aligned; meaningless afterwards
 * Apart from that no output may overlap an input or another output. The state's
 * rounding at the end of a forward call, and those of its checkpoints, have no
 * gradient (they pass it on unchanged). States, their gradients, sums and decays
 * are fp32. Statuses as for kda_prefill_varlen; KDA_ERR_UNSUPPORTED for a
 * lower_bound outside [-5.5, 0], for dA_log or ddt_bias with KDA_GATE_PRECOMPUTED, for
 * more than 65535 heads and for a token stride beyond 2^25 elements. Any
 * 2-byte-aligned bf16 pointer (fp32: 4-byte; fp8 states: any) and any stride is
 * accepted. total_tokens = 0 writes zeros to dA_log and ddt_bias and passes
 * d_final_state on to d_initial_state.
 */
kda_status kda_prefill_varlen_backward(
    int32_t n_docs, int64_t total_tokens, int32_t H, int32_t K, int32_t V,
    const int32_t* cu_seqlens_host, const int32_t* cu_seqlens,
    const void* q, int64_t q_tok_stride, const void* k, int64_t k_tok_stride,
    const void* v, int64_t v_tok_stride, const void* g_raw, int64_t g_tok_stride,
    const void* beta_raw, int64_t beta_tok_stride,
    const float* A_log, const float* dt_bias, float lower_bound, float scale,
    int32_t gate_mode, int32_t state_dtype,
    const void* state_pool, int64_t num_slots, int64_t slot_stride,
    const int32_t* state_indices, int32_t use_initial_state,
    const void* d_out, int64_t d_out_tok_stride, const float* d_final_state,
    void* dq, int64_t dq_tok_stride, void* dk, int64_t dk_tok_stride,
    void* dv, int64_t dv_tok_stride, void* dg, int64_t dg_tok_stride,
    void* dbeta, int64_t dbeta_tok_stride,
    float* dA_log, float* ddt_bias, float* d_initial_state,
    void* workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_BACKWARD_H_ */
