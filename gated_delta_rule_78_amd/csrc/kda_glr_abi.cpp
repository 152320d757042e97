// C ABI of the gated linear recurrence: argument validation and dispatch (include/kda_glr.h).
#include "kda_glr.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda_check.h"
#include "kda_glr_internal.h"
#include "kda_glr_plan.h"

namespace {

using kda::GlrArgs;
using kda::Operand;
using kda::elem_bytes;

kda_status check_desc(const kda_glr_desc* d, bool step) {
    if (!d) return KDA_ERR_INVALID_ARG;
    if (d->N < 1 || d->H < 1 || d->d < 1) return KDA_ERR_INVALID_ARG;
    if (!step && (d->T < 0 || (d->packed != 0 && d->packed != 1))) return KDA_ERR_INVALID_ARG;
    if (!kda::valid_dtype(d->in_dtype) || !kda::valid_dtype(d->out_dtype)) return KDA_ERR_INVALID_ARG;
    if (d->scale < KDA_GLR_ONE || d->scale > KDA_GLR_NORM) return KDA_ERR_INVALID_ARG;
    if (!step && d->T >= ((int64_t)1 << 31) - KDA_GLR_CHUNK) return KDA_ERR_UNSUPPORTED;
    // a tile's elements are addressed with 32 bits
    if (d->d > KDA_GLR_MAX_D) return KDA_ERR_UNSUPPORTED;
    // element counts must fit comfortably in 64-bit byte offsets
    const double T = step ? 1.0 : (double)(d->T > 0 ? d->T : 1);
    if ((double)d->N * (double)d->H * T * (double)d->d > 1e17) return KDA_ERR_INVALID_ARG;
    // sequences, blocks of rows and tiles of one launch are numbered with 32 bits
    const double blocks = !step && d->packed ? (double)d->H : (double)d->N * (double)d->H;
    const double tiles = blocks * (T / 64.0 + 1.0) * ((double)d->d / 16.0 + 1.0);
    if ((double)d->N * (double)d->H >= 2147483648.0 || tiles >= 2147483648.0) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

kda_status check_gates(const kda_glr_desc* d, const kda_glr_gates* g) {
    if (!g) return KDA_ERR_INVALID_ARG;
    if ((g->log_alpha != nullptr) == (g->z != nullptr)) return KDA_ERR_INVALID_ARG;
    if ((g->z != nullptr) != (g->A_log != nullptr)) return KDA_ERR_INVALID_ARG;
    if (g->z && (!(d->g_min < 0.f) || d->g_min < -3.0e38f)) return KDA_ERR_INVALID_ARG;   // NaN fails too
    return KDA_OK;
}

GlrArgs to_args(const kda_glr_desc* d, const kda_glr_gates* g) {
    GlrArgs a{};
    a.N = d->N; a.H = d->H; a.T = d->T; a.d = d->d;
    a.packed = d->packed != 0;
    a.blocks = a.packed ? d->H : d->N * d->H;
    a.nch = kda::ceil_to(d->T, KDA_GLR_CHUNK);
    a.in_bf16 = d->in_dtype == KDA_BF16; a.out_bf16 = d->out_dtype == KDA_BF16;
    a.scale = d->scale; a.g_min = d->g_min;
    if (g) { a.la = g->log_alpha; a.z = g->z; a.A_log = g->A_log; a.u = g->in_gate; }
    return a;
}

}  // namespace

extern "C" {

size_t kda_glr_fwd_workspace_bytes(const kda_glr_desc* d) {
    if (check_desc(d, false) != KDA_OK || d->T == 0) return 0;
    const GlrArgs a = to_args(d, nullptr);
    return kda::glr::fwd_launchable(a) ? kda::glr_fwd_ws_bytes(a) : 0;
}

kda_status kda_glr_fwd(const kda_glr_desc* d, const void* x, const kda_glr_gates* gates, const int32_t* cu_seqlens,
                       const float* S0, void* y, float* S_T, float* entry_states, void* workspace,
                       size_t workspace_bytes, void* stream) {
    const kda_status ds = check_desc(d, false);
    if (ds != KDA_OK) return ds;
    const bool packed = d->packed != 0;
    if (packed != (cu_seqlens != nullptr)) return KDA_ERR_INVALID_ARG;
    const bool rows = d->T > 0;
    if (rows) {
        if (!x || !y) return KDA_ERR_INVALID_ARG;
        const kda_status gs = check_gates(d, gates);
        if (gs != KDA_OK) return gs;
    }
    GlrArgs a = to_args(d, rows ? gates : nullptr);
    if (!kda::glr::fwd_launchable(a)) return KDA_ERR_UNSUPPORTED;
    const int64_t n = a.blocks * d->T * d->d, ein = elem_bytes(d->in_dtype), eout = elem_bytes(d->out_dtype);
    const int64_t states = d->N * d->H * d->d * 4;
    const size_t need = rows ? kda::glr_fwd_ws_bytes(a) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    if (cu_seqlens && !kda::aligned(cu_seqlens, 4)) return KDA_ERR_INVALID_ARG;
    const Operand in[] = {{S0, states, 4}, {rows ? x : nullptr, n * ein, ein}, {a.la, n * ein, ein},
                          {a.z, n * ein, ein}, {a.u, n * ein, ein}, {a.A_log, d->H * d->d * 4, 4}};
    const Operand out[] = {{S_T, states, 4}, {rows ? y : nullptr, n * eout, eout},
                           {rows ? entry_states : nullptr, a.blocks * a.nch * d->d * 4, 4},
                           {need > 0 ? workspace : nullptr, (int64_t)need, 16}};
    if (!kda::operands_ok(in, out, 0, 0)) return KDA_ERR_INVALID_ARG;
    const kda::Range rcu = kda::range_of(cu_seqlens, packed ? (d->N + 1) * 4 : 0);
    for (const Operand& o : out)
        if (kda::overlaps(o.range(), rcu)) return KDA_ERR_INVALID_ARG;
    a.x = x; a.cu = cu_seqlens; a.S0 = S0; a.y = y; a.S_T = S_T;
    a.entry = rows ? entry_states : nullptr;
    a.ws = static_cast<unsigned char*>(workspace);
    return kda::launch_glr_fwd(a, reinterpret_cast<hipStream_t>(stream)) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

size_t kda_glr_bwd_workspace_bytes(const kda_glr_desc* d, int32_t has_entry_states, int32_t has_z) {
    if (check_desc(d, false) != KDA_OK || d->T == 0) return 0;
    GlrArgs a = to_args(d, nullptr);
    static float some;
    a.entry = has_entry_states ? &some : nullptr;   // only whether they are there is looked at
    a.z = has_z ? &some : nullptr;
    return kda::glr::bwd_launchable(a) ? kda::glr_bwd_ws_bytes(a) : 0;
}

kda_status kda_glr_bwd(const kda_glr_desc* d, const void* x, const kda_glr_gates* gates, const int32_t* cu_seqlens,
                       const float* S0, const float* entry_states, const void* dy, const float* dS_T, void* dx,
                       void* ddecay, void* din_gate, float* dA_log, float* dS0, void* workspace,
                       size_t workspace_bytes, void* stream) {
    const kda_status ds = check_desc(d, false);
    if (ds != KDA_OK) return ds;
    const bool packed = d->packed != 0;
    if (packed != (cu_seqlens != nullptr)) return KDA_ERR_INVALID_ARG;
    const bool rows = d->T > 0;
    if (rows) {
        if (!x || !dy || !dx || !ddecay) return KDA_ERR_INVALID_ARG;
        const kda_status gs = check_gates(d, gates);
        if (gs != KDA_OK) return gs;
        if ((gates->z != nullptr) != (dA_log != nullptr) || (gates->in_gate != nullptr) != (din_gate != nullptr))
            return KDA_ERR_INVALID_ARG;
    }
    GlrArgs a = to_args(d, rows ? gates : nullptr);
    const int64_t n = rows ? a.blocks * d->T * d->d : 0;
    const int64_t ein = elem_bytes(d->in_dtype), eout = elem_bytes(d->out_dtype);
    const int64_t states = d->N * d->H * d->d * 4;
    a.entry = rows ? const_cast<float*>(entry_states) : nullptr;
    if (!kda::glr::bwd_launchable(a)) return KDA_ERR_UNSUPPORTED;
    const size_t need = rows ? kda::glr_bwd_ws_bytes(a) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    if (cu_seqlens && !kda::aligned(cu_seqlens, 4)) return KDA_ERR_INVALID_ARG;
    const Operand in[] = {{S0, states, 4}, {dS_T, states, 4}, {x, n * ein, ein}, {a.la, n * ein, ein},
                          {a.z, n * ein, ein}, {a.u, n * ein, ein}, {a.A_log, d->H * d->d * 4, 4}, {dy, n * eout, eout}, {a.entry, a.blocks * a.nch * d->d * 4, 4}};
    const Operand out[] = {{dS0, states, 4}, {dx, n * ein, ein}, {ddecay, n * ein, ein}, {din_gate, n * ein, ein},
                           {dA_log, d->H * d->d * 4, 4}, {need > 0 ? workspace : nullptr, (int64_t)need, 16}};
    if (!kda::operands_ok(in, out)) return KDA_ERR_INVALID_ARG;
    const kda::Range rcu = kda::range_of(cu_seqlens, packed ? (d->N + 1) * 4 : 0);
    for (const Operand& o : out)
        if (kda::overlaps(o.range(), rcu)) return KDA_ERR_INVALID_ARG;
    a.x = x; a.cu = cu_seqlens; a.S0 = S0; a.dy = dy; a.dST = dS_T;
    a.dx = dx; a.dd = ddecay; a.du = din_gate; a.dA = dA_log; a.dS0 = dS0;
    a.ws = static_cast<unsigned char*>(workspace);
    return kda::launch_glr_bwd(a, reinterpret_cast<hipStream_t>(stream)) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

kda_status kda_glr_step(const kda_glr_desc* d, const void* x, const kda_glr_gates* gates, float* S, void* y,
                        void* stream) {
    const kda_status ds = check_desc(d, true);
    if (ds != KDA_OK) return ds;
    const kda_status gs = check_gates(d, gates);
    if (gs != KDA_OK) return gs;
    if (!x || !S || !y) return KDA_ERR_INVALID_ARG;
    kda_glr_desc one = *d;
    one.T = 1; one.packed = 0;
    GlrArgs a = to_args(&one, gates);
    if (!kda::glr::step_launchable(a)) return KDA_ERR_UNSUPPORTED;
    const int64_t n = d->N * d->H * d->d, ein = elem_bytes(d->in_dtype), eout = elem_bytes(d->out_dtype);
    const Operand in[] = {{x, n * ein, ein}, {a.la, n * ein, ein}, {a.z, n * ein, ein}, {a.u, n * ein, ein},
                          {a.A_log, d->H * d->d * 4, 4}};
    const Operand out[] = {{S, n * 4, 4}, {y, n * eout, eout}};
    if (!kda::operands_ok(in, out)) return KDA_ERR_INVALID_ARG;
    a.x = x; a.S = S; a.y = y;
    return kda::launch_glr_step(a, reinterpret_cast<hipStream_t>(stream)) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

}  // extern "C"
