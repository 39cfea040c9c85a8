/*
 * mgg/linear.h - C ABI of the dense products of an MoE model (router, gate, shared expert,
 * projections) with bias, activation and residual in their epilogue, and their gradients. Same
 * library, status codes, error text and common rules as mgg/layer_ops.h; as there, rows may be
 * strided and need no alignment beyond their element's.
 */
#ifndef MGG_LINEAR_H
#define MGG_LINEAR_H

#include "mgg/layer_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MGG_FUNC_NONE = 0,
  MGG_FUNC_RELU = 1,   /* max(z, 0); its gradient at 0 is 0 */
  MGG_FUNC_GELU = 2,   /* z Phi(z), Phi the normal distribution function (erf, no fit by tanh) */
  MGG_FUNC_SILU = 3,   /* z sigmoid(z) */
  MGG_FUNC_SWIGLU = 4  /* silu(z[:, :N/2]) * z[:, N/2:]: gate columns, then up columns */
} mgg_func;

/*
 *   z   = x w^T + bias
 *   out = f(z) + residual
 * with C = N columns of `out` (N/2 for MGG_FUNC_SWIGLU, N even).
 *
 *   0 <= M <= 2^30; 1 <= N, K <= 2^20. Operands that do not have 16-byte aligned rows of whole
 *   16 bytes (or whose rows lie more than 2^20 elements apart) are copied to the workspace first,
 *   unless the call has few rows.
 *   dtype       of x, w and z: bfloat16, or float32 (multiplied in float32).
 *   out_dt      of out and residual.    bias_dt   of bias.
 *   x           [M] rows of K (ldx >= K);  w  [N] rows of K (ldw >= K).
 *   bias        [N], or NULL.   residual  [M] rows of C (ld_res >= C), or NULL.
 */
typedef struct {
  mgg_act dtype, out_dt, bias_dt;
  int M, N, K;
  mgg_func func;
  const void* x;
  int64_t ldx;
  const void* w;
  int64_t ldw;
  const void* bias;
  const void* residual;
  int64_t ld_res;
} mgg_linear;

/*
 *   out   [M][C] of out_dt.
 *   z     [M][N] of dtype, or NULL: z before f, rounded; what the backward call reads.
 * The workspace may be NULL where its size is 0.
 */
size_t linear_act_workspace(const mgg_linear* linear);
mgg_status linear_act(const mgg_linear* linear, void* out, void* z, void* workspace,
                      size_t workspace_bytes, hipStream_t stream);

/*
 * Its gradients, from the gradient d_out of out and z as stored (z NULL exactly for
 * MGG_FUNC_NONE). With dz = d_out * f'(z), held in dtype:
 *   d_x = dz w     [M][K] of dtype, or NULL
 *   d_w = dz^T x   [N][K] of dw_dt, or NULL
 *   d_bias = the sums of dz (before its rounding) over the rows, float32 [N], or NULL
 * At least one is given. The residual's gradient is d_out. linear->bias and residual are not
 * read; out_dt is d_out's type.
 *   z, d_out    [M] rows of N (ldz >= N) and of C (ld_dout >= C).
 */
size_t linear_act_backward_workspace(const mgg_linear* linear, const void* z, int64_t ldz,
                                     const void* d_out, int64_t ld_dout, const void* d_x,
                                     const void* d_w, const float* d_bias);
mgg_status linear_act_backward(const mgg_linear* linear, const void* z, int64_t ldz,
                               const void* d_out, int64_t ld_dout, void* d_x, void* d_w,
                               mgg_act dw_dt, float* d_bias, void* workspace,
                               size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MGG_LINEAR_H */
