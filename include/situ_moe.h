/* situ_moe.h — the operators around the expert activation in one MoE layer, in the same C ABI as
 * situ_glu.h (libsitu_glu.so): top-k routing, tokens sorted by expert and back, and the per-expert
 * (or dense) matrix product with bias, activation and residual, each with its gradient.
 *
 *   route:    p, ids   = softmax over the K largest router scores of a token
 *   plan:     the token-expert pairs in expert order ("rows"): expert e owns rows
 *             expert_offsets[e] .. expert_offsets[e+1]-1, by ascending token, then choice, within e
 *   dispatch: h[row]   = (weight ·) x[token]
 *   linear:   out[row] = act(a[row]·W_eᵀ + b_e) + residual[row]
 *   combine:  y[token] = residual[token] + Σ_k weight[token,k]·o[row(token,k)]
 *
 * ("Kimi K3 模型结构（9）：显存", the expert equation y = Σ_{e in top-k} p_e·o_e and its gradients;
 * "Inside Kimi K3", section "Idea One", the top-k routing sketch.) The rows are the ones that
 * situ_glu_fwd_gateup and situ_glu_bwd_router_dgrad take.
 *
 * Conventions are those of situ_glu.h: device pointers, contiguous row-major tensors, the caller
 * owns every buffer (workspaces included; the library allocates nothing), work is enqueued on
 * `stream` without a host wait, every argument is checked on the host before any launch, and the
 * result is a status code (SITU_GLU_OK, _INVALID_ARG, _OVERLAP, _CUDA_ERROR). Element types are
 * SITU_BF16 or SITU_FP32 where a function takes one. expert_offsets are non-decreasing, from 0 to at
 * most R (what situ_dispatch_plan gives). Others are clamped into [0, R], and in the products an expert
 * that begins before an earlier one ends has no rows: nothing is accessed outside the buffers and the
 * work stays bounded. A call without rows (T, R or the like = 0)
 * succeeds; outputs that do not depend on rows (gradients of weights and biases, offsets) are
 * written all the same.
 */
#ifndef SITU_MOE_H
#define SITU_MOE_H

#include "situ_glu.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { SITU_BF16 = 0, SITU_FP32 = 1 };
enum { SITU_ACT_NONE = 0, SITU_ACT_RELU = 1, SITU_ACT_SILU = 2, SITU_ACT_GELU = 3 }; /* gelu: z·Φ(z), by erf */

#define SITU_MAX_EXPERTS 1024
#define SITU_MAX_TOPK 32

/* ---- routing ------------------------------------------------------------------------------
 * logits [T, E] of `type`; for every token the K largest scores in descending order, of equal ones
 * the lower index first (-0 equals +0): ids int32 [T, K] and p fp32 [T, K] = softmax over them in
 * fp32. A score of -inf is never chosen: where fewer than K are left, the remaining places hold
 * id -1 and p 0 (a token whose scores are all -inf has no expert). Other masked values, such as
 * the type's lowest finite one, are scores like any other. NaN ranks above everything; a token
 * with a chosen NaN or +inf has p = NaN at its live places. 1 <= E <= 1024, 1 <= K <= min(E, 32). */
int situ_route_topk(const void* logits, int type, float* p, int32_t* ids, int64_t T, int64_t E, int64_t K,
                    cudaStream_t stream);

/* dlogits [T, E] of `type`: p_k·(dp_k − Σ_j p_j·dp_j) at ids[t, k], 0 elsewhere; places whose id is
 * outside [0, E) take no part (dp is not used there). dp fp32 [T, K], or, with row_of int32 [T, K]
 * given, dp fp32 [R] in row order (the dp of situ_glu_bwd_router_dgrad): place (t, k) takes
 * dp[row_of[t, k]], and takes no part where that is outside [0, R). A token's ids are distinct. */
int situ_route_topk_bwd(const int32_t* ids, const float* p, const float* dp, const int32_t* row_of, int64_t R,
                        void* dlogits, int type, int64_t T, int64_t E, int64_t K, cudaStream_t stream);

/* ---- tokens sorted by expert and back -----------------------------------------------------
 * The row plan of ids int32 [T, K] (an id outside [0, E) has no row): expert_offsets int64 [E+1],
 * row_of int32 [T, K] (-1 without a row), src int32 [T·K] (t·K + k of each row; -1 past the last
 * row) and, if p fp32 [T, K] and p_rows are given, p_rows fp32 [T·K] (p of each row; 0 past the
 * last row). A stable sort: no result depends on timing. T·K <= 2^31 - 1, 1 <= E <= 1024.
 * workspace: situ_dispatch_plan_workspace(T, K, E) bytes, 4-byte aligned (0: may be NULL). */
int64_t situ_dispatch_plan_workspace(int64_t T, int64_t K, int64_t E);
int situ_dispatch_plan(const int32_t* ids, const float* p, int64_t* expert_offsets, int32_t* row_of, int32_t* src,
                       float* p_rows, void* workspace, int64_t workspace_bytes, int64_t T, int64_t K, int64_t E,
                       cudaStream_t stream);

/* h [R, D] of `type`: h[row_of[t, k]] = x[t] (weights NULL) or weights[t, k]·x[t] (weights fp32
 * [T, K]; the product in fp32, rounded once); rows from expert_offsets[E] on are zeroed. x [T, D]
 * of `type`; row_of entries outside [0, R) are skipped. row_of and expert_offsets are those of one
 * plan: a row before expert_offsets[E] that row_of does not name is not written (to drop a pair, give
 * it no expert before the plan). Its gradient is situ_combine. Any D >= 1 (16-byte vectors where D and
 * the pointers allow). */
int situ_dispatch(const void* x, int type, const int32_t* row_of, const int64_t* expert_offsets, int64_t E,
                  const float* weights, void* h, int64_t T, int64_t K, int64_t R, int64_t D, cudaStream_t stream);

/* y [T, D] = residual + Σ_k weights[t, k]·o[row_of[t, k]] (k ascending, fp32, rounded once); without
 * weights they are 1, without residual it is 0. o [R, D], residual [T, D] (may be y itself) and y of
 * `type`. Entries of row_of outside [0, R) are skipped. */
int situ_combine(const void* o, int type, const int32_t* row_of, const float* weights, const void* residual, void* y,
                 int64_t T, int64_t K, int64_t R, int64_t D, cudaStream_t stream);

/* Its gradient: dout_rows [R, D] of `type`, row_of[t, k] = weights[t, k]·dy[t] (rounded once; rows
 * from expert_offsets[E] on are zeroed, others that row_of does not name are not written), and
 * dweights fp32 [T, K] = <dy[t], o[row_of[t, k]]> (0 without a row). The residual's gradient is dy itself. */
int situ_combine_bwd(const void* dy, const void* o, int type, const int32_t* row_of, const float* weights,
                     const int64_t* expert_offsets, int64_t E, void* dout_rows, float* dweights, int64_t T, int64_t K,
                     int64_t R, int64_t D, cudaStream_t stream);

/* ---- matrix product with bias, activation and residual ------------------------------------
 * For every row r of expert e: z = a[r]·W_eᵀ + b_e, out[r] = act(z) + residual[r], evaluated in
 * fp32 from the fp32 accumulator and rounded once. a bf16 [R, K], w bf16 [E, N, K] (the nn.Linear
 * layout), bias fp32 [E, N] or NULL, residual bf16 [R, N] or NULL, out [R, N] of out_type, pre bf16
 * [R, N] or NULL (receives z rounded to bf16, what the backward reads). expert_offsets int64 [E+1],
 * or NULL with E = 1: one weight for all rows. Rows outside every expert's range are not written.
 * N % 8 == 0, K % 8 == 0; 1 <= E <= 1024; R <= 2^31 - 1025; a, w, residual, out and pre 16-byte
 * aligned. status (device int, zeroed by the caller, may be NULL) turns 1 if a pipeline wait timed out.
 * The tensor cores cut each 16-deep step's fp32 sum towards zero: an fp32 out is off by 1e-6 of its
 * norm at K = 1024 and by 1.9e-5 at 16384 (situ_linear_wgrad, whose contraction is the rows, adds
 * 512-row chunks rounded to nearest instead: 5e-7 at any R). */
int situ_linear_fwd(const void* a, const void* w, const int64_t* expert_offsets, int64_t E, const float* bias,
                    const void* residual, int act, void* out, int out_type, void* pre, int* status, int64_t R,
                    int64_t N, int64_t K, cudaStream_t stream);

/* dz = dout·act'(pre), rounded to bf16 (the operand of the two products below, as a bf16 layer's
 * gradients are: relative 1.7e-3 of the norm, in an fp32 dw too), and dbias fp32
 * [E, N] = the sum of the unrounded dz over each expert's rows. dout, pre and dz bf16 [R, N]; with
 * SITU_ACT_NONE pre and dz are not used (dz = dout) and may be NULL. dbias may be NULL; with it,
 * workspace holds situ_linear_act_bwd_workspace(R, N, E) bytes, 4-byte aligned. dz of rows outside
 * every expert's range is not written. N % 8 == 0; dout, pre and dz 16-byte aligned. */
int64_t situ_linear_act_bwd_workspace(int64_t R, int64_t N, int64_t E);
int situ_linear_act_bwd(const void* dout, const void* pre, int act, const int64_t* expert_offsets, int64_t E, void* dz,
                        float* dbias, void* workspace, int64_t workspace_bytes, int64_t R, int64_t N,
                        cudaStream_t stream);

/* da bf16 [R, K] = dz·W_e (fp32 accumulation, rounded once); arguments as situ_linear_fwd. */
int situ_linear_dgrad(const void* dz, const void* w, const int64_t* expert_offsets, int64_t E, void* da, int* status,
                      int64_t R, int64_t N, int64_t K, cudaStream_t stream);

/* dw [E, N, K] of dw_type: dW_e = Σ over the expert's rows of dz[r]ᵀ·a[r] (fp32 accumulation; zeros
 * for an expert without rows). dz bf16 [R, N], a bf16 [R, K]. workspace:
 * situ_linear_wgrad_workspace(R, N, K, E) bytes, 16-byte aligned (0: may be NULL). */
int64_t situ_linear_wgrad_workspace(int64_t R, int64_t N, int64_t K, int64_t E);
int situ_linear_wgrad(const void* dz, const void* a, const int64_t* expert_offsets, int64_t E, void* dw, int dw_type,
                      void* workspace, int64_t workspace_bytes, int* status, int64_t R, int64_t N, int64_t K,
                      cudaStream_t stream);

/* Self-test of the failure path of the linear operator's waits (faults nothing), as
 * situ_glu_selftest_wait_timeout: two CTAs of a cluster wait on barriers nothing completes, give up
 * after about 2 s, write 1 to *status (device int, zeroed by the caller) and return normally. */
int situ_linear_selftest_wait_timeout(int* status, unsigned long long* elapsed_ns, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SITU_MOE_H */
