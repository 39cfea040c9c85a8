/*
 * mgg/few_tokens.h - C ABI of a whole MoE layer for the few tokens of a decoding step: both
 * products of every chosen expert, the gated unit between them, the weighted sum over a token's
 * experts and the residual, in two kernels. It takes route_topk's choices as they are and the
 * grouped products' weights in their layouts (moe_grouped_gemm_nt.h); nothing is sorted, padded
 * or quantized. Same library, status codes, error text and common rules as mgg/layer_ops.h.
 */
#ifndef MGG_FEW_TOKENS_H
#define MGG_FEW_TOKENS_H

#include "mgg/layer_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Expert weights: bfloat16, FP8 E4M3 or FP4 E2M1 (two per byte, the even K element low). */
typedef enum { MGG_WEIGHT_BF16 = 0, MGG_WEIGHT_FP8 = 1, MGG_WEIGHT_FP4 = 2 } mgg_weight;

/*
 * For every token t, over its places j with e = ids[t, j] in [0, G):
 *   [g; u]  = W13[e] x[t]                    (g: rows 0 .. I-1, u: rows I .. 2I-1)
 *   out[t]  = residual[t] + sum_j weights[t, j] * W2[e] (silu(g) * u)
 * Other ids are skipped (route_topk's -1: whatever weight stands there has no effect); a token
 * that names no expert gets its residual, or 0. An expert named twice by a token counts with the
 * sum of its weights. Weights are dequantized, activations are not quantized; sums are float32.
 * Between the products silu(g) * u is held as bfloat16 where the output is bfloat16, as between
 * the grouped products, and as the sum of three (float32's 24 bits) where it is float32.
 *
 *   T, k, G     0 <= T <= 128; 1 <= k <= 32; 1 <= G <= 4096. The time goes with the experts
 *               that are named.
 *   H, I        1 <= H, I <= 2^16, multiples of 8 (bfloat16 weights) or of 128 (FP8, FP4).
 *   x           bfloat16, [T] rows of H (ldx >= H).
 *   ids         int32 [T][k]; weights float32 [T][k].
 *   W13, W2     [G][2I][H] and [G][H][I] (FP4: half as many bytes a row), 16-byte aligned.
 *   S13, S2     their scales (NULL for bfloat16), of format `sf` and granularity `gran`:
 *               BLOCK128 [G][ceil(N/128)][K/128], CHANNEL [G][K/128][N] (FP8), or BLOCK32
 *               [G][K/128][N][4] in UE8M0 (FP4), with N, K = 2I, H and H, I.
 *   residual    [T] rows of H (ld_res >= H) in the output's type, or NULL.
 *   out         [T][H] of `out_dt`.
 */
size_t moe_few_tokens_workspace(int T, int k, int G, int I);
mgg_status moe_few_tokens(mgg_weight wt, int T, int k, int G, int H, int I, const void* x,
                          int64_t ldx, const int32_t* ids, const float* weights,
                          const void* W13, const void* S13, const void* W2, const void* S2,
                          mgg_sf_fmt sf, mgg_sfb_gran gran, mgg_act out_dt,
                          const void* residual, int64_t ld_res, void* out, void* workspace,
                          size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MGG_FEW_TOKENS_H */
