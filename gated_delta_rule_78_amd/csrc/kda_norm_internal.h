// Internal launcher interface of the block norms (include/kda_norm.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

struct NormArgs {
    int64_t rows, D;
    bool in_bf16, res_bf16, out_bf16;
    bool post, pre;
    float scale, eps, pre_eps;
    const void *f, *gate, *x;
    const float *w_post, *lam, *w_pre;
    void *x_out, *n;
    // backward
    const void *dx_out, *dn;
    void *df, *dgate, *dx;
    float *dw_post, *dlam, *dw_pre;
    float* ws;
};

namespace norm {

// Workgroups at most: what 256 CUs hold at a time (16 waves a CU in the backward, whose column sums
// cost traffic per workgroup; 24 in the forward).
inline int fwd_groups(int threads) { return 256 * 24 * 64 / threads; }
inline int bwd_groups(int threads) { return 256 * 16 * 64 / threads; }

// Instantiated per type of f (kda_norm_*.hip).
template <typename TI>
hipError_t launch_i(const NormArgs& a, bool bwd, hipStream_t st);
// dnorm_weight, dscale_weight and dpre_weight from the sums of `groups` workgroups.
hipError_t launch_colsum(const NormArgs& a, int groups, hipStream_t st);

}  // namespace norm

size_t norm_bwd_ws_bytes(int64_t rows, int64_t D);
hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t st);
hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t st);

}  // namespace kda
