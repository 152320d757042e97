// C ABI of the block norms: argument validation and dispatch (include/kda_norm.h).
#include "kda_norm.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda_check.h"
#include "kda_norm_internal.h"

namespace {

using kda::NormArgs;
using kda::Operand;
using kda::elem_bytes;

bool finite(float v) { return v >= -3.4028234e38f && v <= 3.4028234e38f; }   // NaN fails

kda_status check_desc(const kda_norm_desc* d) {
    if (!d) return KDA_ERR_INVALID_ARG;
    if (d->rows < 0 || d->D < 1) return KDA_ERR_INVALID_ARG;
    if (!kda::valid_dtype(d->in_dtype) || !kda::valid_dtype(d->res_dtype) || !kda::valid_dtype(d->out_dtype))
        return KDA_ERR_INVALID_ARG;
    if ((d->post_norm != 0 && d->post_norm != 1) || (d->pre_norm != 0 && d->pre_norm != 1)) return KDA_ERR_INVALID_ARG;
    if (!finite(d->scale)) return KDA_ERR_INVALID_ARG;
    if (d->post_norm && (!(d->eps > 0.f) || !finite(d->eps))) return KDA_ERR_INVALID_ARG;
    if (d->pre_norm && (!(d->pre_eps > 0.f) || !finite(d->pre_eps))) return KDA_ERR_INVALID_ARG;
    if (d->D > KDA_NORM_MAX_D || d->rows >= (int64_t)1 << 31) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

NormArgs to_args(const kda_norm_desc* d, const void* f, const void* gate, const void* x, const float* w_post,
                 const float* lam, const float* w_pre) {
    NormArgs a{};
    a.rows = d->rows; a.D = d->D;
    a.in_bf16 = d->in_dtype == KDA_BF16; a.res_bf16 = d->res_dtype == KDA_BF16; a.out_bf16 = d->out_dtype == KDA_BF16;
    a.post = d->post_norm != 0; a.pre = d->pre_norm != 0;
    a.scale = d->scale; a.eps = d->eps; a.pre_eps = d->pre_eps;
    a.f = f; a.gate = gate; a.x = x;
    a.w_post = w_post; a.lam = lam; a.w_pre = w_pre;
    return a;
}

}  // namespace

extern "C" {

kda_status kda_block_norm_fwd(const kda_norm_desc* d, const void* f, const void* gate, const void* x,
                              const float* norm_weight, const float* scale_weight, const float* pre_weight,
                              void* x_out, void* n, void* stream) {
    const kda_status ds = check_desc(d);
    if (ds != KDA_OK) return ds;
    if ((norm_weight && !d->post_norm) || (pre_weight && !d->pre_norm)) return KDA_ERR_INVALID_ARG;
    if (d->rows == 0) return KDA_OK;
    if (!f || (!x_out && !n) || (d->pre_norm != 0) != (n != nullptr)) return KDA_ERR_INVALID_ARG;
    const int64_t m = d->rows * d->D, w = d->D * 4;
    const int64_t ein = elem_bytes(d->in_dtype), eres = elem_bytes(d->res_dtype), eout = elem_bytes(d->out_dtype);
    const Operand in[] = {{x, m * eres, eres}, {f, m * ein, ein}, {gate, m * ein, ein}, {norm_weight, w, 4}, {scale_weight, w, 4},
                          {pre_weight, w, 4}};
    const Operand out[] = {{x_out, m * eres, eres}, {n, m * eout, eout}};
    if (!kda::operands_ok(in, out, 0, 0)) return KDA_ERR_INVALID_ARG;
    NormArgs a = to_args(d, f, gate, x, norm_weight, scale_weight, pre_weight);
    a.x_out = x_out; a.n = n;
    return kda::launch_norm_fwd(a, reinterpret_cast<hipStream_t>(stream)) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

size_t kda_block_norm_bwd_workspace_bytes(const kda_norm_desc* d) {
    if (check_desc(d) != KDA_OK || d->rows == 0) return 0;
    return kda::norm_bwd_ws_bytes(d->rows, d->D);
}

kda_status kda_block_norm_bwd(const kda_norm_desc* d, const void* f, const void* gate, const void* x,
                              const float* norm_weight, const float* scale_weight, const float* pre_weight,
                              const void* dx_out, const void* dn, void* df, void* dgate, void* dx,
                              float* dnorm_weight, float* dscale_weight, float* dpre_weight, void* workspace,
                              size_t workspace_bytes, void* stream) {
    const kda_status ds = check_desc(d);
    if (ds != KDA_OK) return ds;
    if (((norm_weight || dnorm_weight) && !d->post_norm) || ((pre_weight || dpre_weight || dn) && !d->pre_norm))
        return KDA_ERR_INVALID_ARG;
    const bool rows = d->rows > 0;
    if (rows) {
        if (!f || !df || (!dx_out && !dn)) return KDA_ERR_INVALID_ARG;
        if ((gate != nullptr) != (dgate != nullptr) || (dx && !x)) return KDA_ERR_INVALID_ARG;
    }
    const bool sums = dnorm_weight || dscale_weight || dpre_weight;
    const size_t need = rows && sums ? kda::norm_bwd_ws_bytes(d->rows, d->D) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    const int64_t m = d->rows * d->D, w = d->D * 4;
    const int64_t ein = elem_bytes(d->in_dtype), eres = elem_bytes(d->res_dtype), eout = elem_bytes(d->out_dtype);
    const Operand in[] = {{dx_out, m * eres, eres}, {x, m * eres, eres}, {f, m * ein, ein}, {gate, m * ein, ein}, {norm_weight, w, 4},
                          {scale_weight, w, 4}, {pre_weight, w, 4}, {dn, m * eout, eout}};
    const Operand out[] = {{dx, m * eres, eres}, {df, m * ein, ein}, {dgate, m * ein, ein}, {dnorm_weight, w, 4}, {dscale_weight, w, 4},
                           {dpre_weight, w, 4}, {need > 0 ? workspace : nullptr, (int64_t)need, 16}};
    if (!kda::operands_ok(in, out, 0, 0)) return KDA_ERR_INVALID_ARG;
    NormArgs a = to_args(d, f, gate, x, norm_weight, scale_weight, pre_weight);
    a.dx_out = dx_out; a.dn = dn;
    a.df = df; a.dgate = dgate; a.dx = dx;
    a.dw_post = dnorm_weight; a.dlam = dscale_weight; a.dw_pre = dpre_weight;
    a.ws = need > 0 ? static_cast<float*>(workspace) : nullptr;
    if (!rows && !sums) return KDA_OK;
    return kda::launch_norm_bwd(a, reinterpret_cast<hipStream_t>(stream)) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

}  // extern "C"
