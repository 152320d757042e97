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

// Workgroups at most: 24 waves a CU in the forward. In the backward 8 for rows on 8 elements that
// read 4 or 5 tensors, whose streams then stay nearer to each other in HBM (5 of 32M bf16 elements:
// 104-111 us, against 111-120 with 16); 16 for fewer tensors, which need more rows in flight (2 of
// them: 51-65 us against 60-84), and where rows start off 8 elements (reads = 0), whose masks cost
// issue slots (rows of 1001: 132 us against 204). One workgroup of 512 or 1024 threads a CU.
inline int fwd_groups(int threads) { return 256 * 24 * 64 / threads; }
inline int bwd_groups(int threads, int reads) {
    const int waves = threads / 64, most = reads >= 4 || (reads && waves == 8) ? 8 : 16;
    return 256 * (waves > most ? 1 : most / waves);
}

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
