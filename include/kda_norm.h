/*
 * kda_norm.h -- C ABI of the norms around a block, with its gate, residual and residual scale, for
 * AMD Instinct MI355X (gfx950). Same library and conventions as kda.h.
 *
 * Per row of D channels, with the block's output f and the residual stream x:
 *
 *     p     = f * norm_weight / sqrt(mean(f^2) + eps)            (post-norm; p = f without it)
 *     u     = sigmoid(gate) * p                                  (u = p without a gate)
 *     x_out = x + scale * scale_weight * u                       (x = 0 without a residual)
 *     n     = x_out * pre_weight / sqrt(mean(x_out^2) + pre_eps) (the next block's pre-norm)
 *
 * With no residual and no pre-norm, rows of a head's dv channels and scale 1 it is the output gate
 * of the KDA core (kda_gating's epilogue), and kda_block_norm_bwd is its backward.
 *
 *  - Weights are fp32 and NULL means ones. Everything in between is fp32: n is computed from
 *    x_out before x_out is rounded; every output is rounded once.
 *  - 1 <= D <= KDA_NORM_MAX_D. The sums of a row's squares, of f and of x_out, must be finite in
 *    fp32, not their means alone: past that (values of 2^57 in all of 16384 channels) the norm is
 *    0. A row that holds a non-finite value gives non-finite outputs in its own row (and weight
 *    gradients), no others.
 *  - Every tensor is dense, its base aligned to its element (16-byte bases take wide accesses);
 *    workspaces are aligned to 16 bytes. Sums over rows run in a fixed order:
 *    the same inputs give the same bits on every call.
 */
#ifndef KDA_NORM_H
#define KDA_NORM_H

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

#define KDA_NORM_MAX_D 16384

typedef struct kda_norm_desc {
    int64_t rows;       /* >= 0                                                                */
    int64_t D;          /* channels per row, 1 .. KDA_NORM_MAX_D                               */
    int32_t in_dtype;   /* kda_dtype of f, gate, df, dgate                                     */
    int32_t res_dtype;  /* kda_dtype of x, x_out, dx, dx_out                                   */
    int32_t out_dtype;  /* kda_dtype of n, dn                                                  */
    int32_t post_norm;  /* 1: normalise f; 0: p = f (norm_weight must be NULL)                 */
    int32_t pre_norm;   /* 1: n is wanted; 0: not (n, dn and pre_weight must be NULL)          */
    float scale;        /* residual scale, finite                                              */
    float eps;          /* > 0 (read with post_norm)                                           */
    float pre_eps;      /* > 0 (read with pre_norm)                                            */
} kda_norm_desc;

/*
 *   f, gate       : [rows, D] in_dtype; gate may be NULL
 *   x             : [rows, D] res_dtype, or NULL (no residual)
 *   norm_weight, scale_weight, pre_weight : [D] fp32, or NULL (ones)
 *   x_out         : [rows, D] res_dtype (written), or NULL to skip; may be x
 *   n             : [rows, D] out_dtype (written), with pre_norm
 * One of x_out and n is required. No output may overlap an input (x_out = x aside) or another.
 */
kda_status kda_block_norm_fwd(const kda_norm_desc* desc, const void* f, const void* gate, const void* x,
                              const float* norm_weight, const float* scale_weight,
                              const float* pre_weight, void* x_out, void* n, void* stream);

/* Bytes of device workspace kda_block_norm_bwd needs (0 for an invalid desc or no rows). */
size_t kda_block_norm_bwd_workspace_bytes(const kda_norm_desc* desc);

/*
 * Backward: for L with dL/dx_out = dx_out and dL/dn = dn, writes the gradients of every input.
 * The forward's inputs are read again (x as it was before an in-place forward).
 *   dx_out        : [rows, D] res_dtype, or NULL (zero)
 *   dn            : [rows, D] out_dtype, with pre_norm, or NULL (zero); one of the two is required
 *   df            : [rows, D] in_dtype (written)
 *   dgate         : [rows, D] in_dtype (written) with gate, else NULL
 *   dx            : [rows, D] res_dtype (written) with x, or NULL to skip; may be dx_out
 *   dnorm_weight, dscale_weight, dpre_weight : [D] fp32 (written: sums over the rows; zeros
 *                   without rows), or NULL to skip. dnorm_weight needs post_norm, dpre_weight
 *                   pre_norm; each may be asked for where the weight itself is NULL (ones)
 *   workspace     : kda_block_norm_bwd_workspace_bytes(desc) bytes, 16-byte aligned; needed only
 *                   where a weight gradient is asked for
 * No output may overlap an input (dx = dx_out aside), the workspace or another output.
 */
kda_status kda_block_norm_bwd(const kda_norm_desc* desc, const void* f, const void* gate, const void* x,
                              const float* norm_weight, const float* scale_weight,
                              const float* pre_weight, const void* dx_out, const void* dn, void* df,
                              void* dgate, void* dx, float* dnorm_weight, float* dscale_weight,
                              float* dpre_weight, void* workspace, size_t workspace_bytes,
                              void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_NORM_H */
