/*
 * mgg/layer_ops.h - C ABI of the operators that stand around the grouped products of
 * moe_grouped_gemm_nt.h in an MoE layer (same library, same status codes and error text):
 *
 *   route_topk                    top-k routing with per-expert counts and a balance loss
 *   route_topk_backward           gradient of the logits
 *   block_norm                    the norm before a block
 *   block_norm_backward           its gradients
 *   block_residual_norm           the norm after a block fused with its gate, residual scale
 *                                 and residual sum, and with the next block's norm
 *   block_residual_norm_backward  its gradients
 *   grouped_newton_schulz         every expert's weight update orthogonalised by
 *                                 Newton-Schulz products
 *
 * Common rules, as in moe_grouped_gemm_nt.h: every pointer is caller-owned device memory
 * unless stated otherwise; host arguments are validated first and nothing is enqueued on an
 * error; a call enqueues kernels on `stream` and returns, never allocates, synchronizes or
 * reads device memory on the host, and may be captured into a hipGraph; results are bitwise
 * identical from call to call on the same inputs (float sums have a fixed order; the only
 * atomics are integer counters, whose sums do not depend on order). Where a call needs
 * scratch memory the caller passes a workspace of at least the size that the entry point's
 * `_workspace` function returns, 256-byte aligned; its contents need no preparation and mean
 * nothing after the call. Inputs must not overlap outputs or the workspace.
 * Row strides (ld*) count elements and are at least the row's length. Rows need no alignment
 * beyond their element's. Activations are bfloat16 or float32 (mgg_act); all arithmetic is
 * float32 or wider, rounded once when an output is stored.
 */
#ifndef MGG_LAYER_OPS_H
#define MGG_LAYER_OPS_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#include "moe_grouped_gemm_nt.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { MGG_ACT_BF16 = 0, MGG_ACT_F32 = 1 } mgg_act;
typedef enum { MGG_SCORE_SOFTMAX = 0, MGG_SCORE_SIGMOID = 1 } mgg_score;
typedef enum { MGG_GATE_NONE = 0, MGG_GATE_TOKEN = 1, MGG_GATE_ELEMENT = 2 } mgg_gate;

/*
 * Top-k routing. Row t holds the logits l[t, e] of G experts.
 *   softmax: q = p = softmax(l[t]), experts ordered by l;
 *   sigmoid: q = sigmoid(l[t]), p = q / sum_e q, experts ordered by l, or by q + bias
 *            (float64) when a bias is given.
 * ids[t] = the first k experts in descending order, the lower index first among equals. An
 * expert whose logit is -inf or NaN (or whose biased score is NaN or -inf) is never taken;
 * places left over hold id -1 and weight 0. weights[t, j] = scale * q[ids[t, j]], divided by
 * the sum of the row's chosen q when `renormalize` is set. The bias enters the selection only.
 * A row of -inf has p = 0 everywhere. A NaN logit, and with softmax +inf, makes its row's p
 * and its sequence's loss NaN.
 *
 * Rows form S sequences: sequence s holds rows [start_s, end_s) with
 *   end_s = seq_ends[s] clamped to [0, T] and raised to the largest earlier end,
 *   start_s = end_{s-1} (0 for s = 0);
 * rows past the last end are padding (ids -1, weights 0, counted nowhere). seq_ends NULL
 * (S = 1): one sequence of all T rows. With n_s = end_s - start_s and c_s[e] the number of
 * times that sequence s chose expert e,
 *   balance[s] = sum_e (G c_s[e] / (k n_s)) * (sum_{t in s} p[t, e] / n_s),  0 if n_s = 0:
 * 1 when both are even over the experts.
 *
 *   T, G, k     0 <= T <= 2^30; 1 <= G <= 4096; 1 <= k <= min(G, 32). Up to 320 experts a choice
 *               of more than about 10 takes several times as long as one of 8, with a bias
 *               several tens of times from 16 on.
 *   logits      [T] rows of G (ld >= G).      bias  float32 [G] or NULL (sigmoid only).
 *   seq_ends    device int32 [S] or NULL, read by the kernels on every launch; S <= 65535.
 *   scale       finite.
 *   ids, weights   int32 / float32 [T][k].
 *   counts      int32 [S][G]; tokens int32 [S] (n_s); balance float32 [S]. All three, or all
 *               three NULL (then no workspace is needed and one kernel is launched).
 */
size_t route_topk_workspace(int T, int G, int S);
mgg_status route_topk(mgg_act dt, int T, int G, int k, const void* logits, int64_t ld,
                      const float* bias, mgg_score score, int renormalize, float scale, int S,
                      const int32_t* seq_ends, int32_t* ids, float* weights, int32_t* counts,
                      int32_t* tokens, float* balance, void* workspace,
                      size_t workspace_bytes, hipStream_t stream);

/*
 * Gradient of the logits, from the gradients of the weights and of the balance losses; counts
 * and ids carry none. Padding rows get 0. A NULL d_weights or d_balance counts as 0 (not
 * both, unless T = 0). ids, counts and tokens are route_topk's (ids outside [0, G) are
 * skipped); counts and tokens may be NULL when d_balance is.
 *   d_weights   float32 [T][k]; d_balance float32 [S].
 *   d_logits    [T][G] in the logits' type.
 */
mgg_status route_topk_backward(mgg_act dt, int T, int G, int k, const void* logits, int64_t ld,
                               mgg_score score, int renormalize, float scale, int S,
                               const int32_t* seq_ends, const int32_t* ids,
                               const int32_t* counts, const int32_t* tokens,
                               const float* d_weights, const float* d_balance,
                               void* d_logits, hipStream_t stream);

/*
 * The end of a block and the start of the next. With rms(v; w) = v / sqrt(mean(v^2) + eps) * w
 * over a row of H,
 *   z     = rms(y; w_after), or y when w_after is NULL        (y: the block's output)
 *   g     = sigmoid(gate) per token or per element, or 1
 *   x_out = alpha * x + beta * scale[c] * g * z               (scale NULL: 1)
 *   u     = rms(x_out; w_before)                              (x_out before its rounding)
 *
 *   0 <= T <= 2^30; 1 <= H <= 32768; eps > 0, not subnormal; alpha, beta finite.
 *   The squares of a row sum to less than float32's largest, 3.4e38. Rows wider than 16384 in
 *   bfloat16 or 8192 in float32 take up to four times as long for their bytes as others.
 *   x, y        [T] rows of H; gate: [T] values (MGG_GATE_TOKEN, ld_gate the step from one to
 *               the next, >= 1) or [T] rows of H (MGG_GATE_ELEMENT), in the activations' type.
 *   scale, w_after, w_before   [H] of `param`, or NULL.
 *   x_out, u    [T][H]; u NULL exactly when w_before is.
 * Workspace: none.
 */
typedef struct {
  mgg_act dtype;  /* of x, y, gate, outputs and activation gradients */
  mgg_act param;  /* of scale, w_after and w_before */
  int T, H;
  const void* x;
  int64_t ldx;
  const void* y;
  int64_t ldy;
  mgg_gate gate_kind;
  const void* gate;
  int64_t ld_gate;
  const void* scale;
  const void* w_after;
  const void* w_before;
  float alpha, beta, eps;
} mgg_block;

mgg_status block_residual_norm(const mgg_block* block, void* x_out, void* u,
                               hipStream_t stream);

/*
 * Its gradients. Here block->x is the stream AFTER the block (x_out as stored); alpha, beta
 * and eps as in the forward call. d_x is the gradient of x_out as the rest of the model sees
 * it, d_u that of u (NULL exactly when w_before is); d_x may be NULL (0) when d_u is given.
 *   D        = d_x + the gradient that u sends to x_out
 *   d_x_in   = alpha * D;   d_y, d_gate: gradients of y and of the gate's input
 *   d_scale, d_w_after, d_w_before   float32 [H], summed over the rows.
 * d_gate, d_scale, d_w_after and d_w_before are given exactly when the input they belong to is.
 * d_gate is contiguous ([T] or [T][H]), d_x_in and d_y are [T][H].
 */
size_t block_residual_norm_backward_workspace(int T, int H);
mgg_status block_residual_norm_backward(const mgg_block* block, const void* d_x, int64_t ld_dx,
                                        const void* d_u, int64_t ld_du, void* d_x_in,
                                        void* d_y, void* d_gate, float* d_scale,
                                        float* d_w_after, float* d_w_before, void* workspace,
                                        size_t workspace_bytes, hipStream_t stream);

/*
 * The norm before a block alone: u = rms(x; w), and its gradients d_x_in = d_x + (what d_u
 * sends to x) and d_w (float32 [H]); d_x NULL counts as 0. The workspace is
 * block_residual_norm_backward's.
 */
mgg_status block_norm(mgg_act dt, mgg_act param, int T, int H, const void* x, int64_t ldx,
                      const void* w, float eps, void* u, hipStream_t stream);
mgg_status block_norm_backward(mgg_act dt, mgg_act param, int T, int H, const void* x,
                               int64_t ldx, const void* w, float eps, const void* d_x,
                               int64_t ld_dx, const void* d_u, int64_t ld_du, void* d_x_in,
                               float* d_w, void* workspace, size_t workspace_bytes,
                               hipStream_t stream);

/*
 * Orthogonalised update of G matrices [M][N] at once (the weight gradients, or momenta of
 * them, that grouped_gemm_kgrouped writes). For each matrix
 *   X = X / (|X|_F + eps);   for each step s:  A = X X^T,
 *   X = a_s X + (b_s A + c_s A A) X        (for M > N the same on the transposed matrix)
 *   out = scale * X.
 * Products are of float32 grade, also where |X|_F is far below eps: each operand is held as the
 * sum of two fp16 numbers, times a power of two of its matrix's and step's own, and multiplied as
 * three fp16 matrix products with float32 accumulation. A matrix of zeros gives zeros; a matrix
 * with a NaN or infinity gives NaN and leaves the others alone.
 *
 *   G, M, N     1 <= G <= 4096; 1 <= M, N <= 32768.
 *   X           [G][M][N] of `dt`; out [G][M][N] of `out_dt`. Either may be bf16 or float32.
 *   steps       1 .. 32; coeffs: HOST float [steps][3], (a, b, c) of each step. Refused
 *               (MGG_EUNSUPPORTED) when they send a singular value in [0, 1] above 3.9, where
 *               the fp16 halves would overflow.
 *   eps         > 0; scale finite.
 */
size_t grouped_newton_schulz_workspace(int G, int M, int N);
mgg_status grouped_newton_schulz(mgg_act dt, mgg_act out_dt, int G, int M, int N,
                                 const void* X, void* out, int steps, const float* coeffs,
                                 float eps, float scale, void* workspace,
                                 size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MGG_LAYER_OPS_H */
