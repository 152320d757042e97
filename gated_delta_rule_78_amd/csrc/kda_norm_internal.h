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

size_t norm_bwd_ws_bytes(int64_t rows, int64_t D);
hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t st);
hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t st);

}  // namespace kda
