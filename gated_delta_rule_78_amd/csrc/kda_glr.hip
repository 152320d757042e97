// Gated linear recurrence for gfx950: workspaces, plans and the single-token step.
#include "kda_glr_device.h"
#include "kda_internal.h"

namespace kda {
namespace glr {

// One token of every sequence: S = alpha S + w i x in place, y = S. Bound by the state's read and
// write, and by the launch for a few sequences.
template <int SCALE, typename TIn, typename TOut>
__global__ __launch_bounds__(256) void glr_step_kernel(GlrArgs a) {
    const int64_t n = a.N * a.H * a.d;
    for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < n; at += (int64_t)gridDim.x * 256) {
        float la;
        if (a.z) la = a.g_min * sigmoid_f(exp_f(a.A_log[at % (a.H * a.d)]) * ld_f((const TIn*)a.z + at));
        else la = ld_f((const TIn*)a.la + at);
        const float alpha = exp_f(la);
        float b = ld_f((const TIn*)a.x + at) * scale_w<SCALE>(la, alpha);
        if (a.u) b *= sigmoid_f(ld_f((const TIn*)a.u + at));
        const float st = fmaf(alpha, a.S[at], b);
        a.S[at] = st;
        st_f((TOut*)a.y + at, st);
    }
}

template <int SCALE, typename TIn, typename TOut>
static hipError_t launch_step_t(const GlrArgs& a, hipStream_t st) {
    const int64_t n = a.N * a.H * a.d;
    const int64_t grid = (n + 255) / 256 < (1 << 20) ? (n + 255) / 256 : (1 << 20);
    hipLaunchKernelGGL((glr_step_kernel<SCALE, TIn, TOut>), dim3((unsigned)grid), dim3(256), 0, st, a);
    return hipGetLastError();
}

template <int SCALE>
static hipError_t launch_step_s(const GlrArgs& a, hipStream_t st) {
    if (a.in_bf16 && a.out_bf16) return launch_step_t<SCALE, bf16_t, bf16_t>(a, st);
    if (a.in_bf16) return launch_step_t<SCALE, bf16_t, float>(a, st);
    if (a.out_bf16) return launch_step_t<SCALE, float, bf16_t>(a, st);
    return launch_step_t<SCALE, float, float>(a, st);
}

// Workspace in order: counters, first sequences, chain words, dA_log parts, entry states.
struct Plan {
    GlrWs ws;
    float* entry;
    size_t bytes;
};

static Plan make_plan(const GlrArgs& a, unsigned char* base, bool with_dA, bool with_entry) {
    Plan p{};
    p.ws.rows = KDA_GLR_CHUNK;
    p.ws.nt = (a.T + KDA_GLR_CHUNK - 1) / KDA_GLR_CHUNK;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        unsigned char* r = base ? base + at : nullptr;
        at += (bytes + 255) & ~(size_t)255;
        return r;
    };
    const size_t words = (size_t)(a.blocks * p.ws.nt * a.d);
    const int64_t chains = a.blocks * ((a.d + kCW - 1) / kCW);
    p.ws.counters = chains < (int64_t)kCounters ? chains : (int64_t)kCounters;
    if (p.ws.nt > 1) p.ws.ticket = reinterpret_cast<uint32_t*>(take((size_t)p.ws.counters * kCounterStride * 4));
    if (a.packed) p.ws.seq = reinterpret_cast<int32_t*>(take((size_t)(p.ws.nt + 1) * 4));
    if (p.ws.nt > 1) {
        p.ws.span = reinterpret_cast<u64*>(take(words * 8));
        p.ws.state = reinterpret_cast<u64*>(take(words * 8));
    }
    if (with_dA) p.ws.dA = reinterpret_cast<float*>(take(words * 4));
    if (with_entry) p.entry = reinterpret_cast<float*>(take((size_t)(a.blocks * a.nch * a.d) * 4));
    p.bytes = at;
    return p;
}

// Whether every row of these tensors starts on 4 elements of its type.
static bool rows_of_4(const GlrArgs& a) {
    if (a.d % 4 != 0) return false;
    uintptr_t in = 0, out = 0;
    for (const void* p : {a.x, a.la, a.z, a.u, (const void*)a.dx, (const void*)a.dd, (const void*)a.du, (const void*)a.S})
        in |= reinterpret_cast<uintptr_t>(p);
    for (const void* p : {(const void*)a.y, a.dy}) out |= reinterpret_cast<uintptr_t>(p);
    return (in & (a.in_bf16 ? 7 : 15)) == 0 && (out & (a.out_bf16 ? 7 : 15)) == 0;
}

}  // namespace glr

size_t glr_fwd_ws_bytes(const GlrArgs& a) { return glr::make_plan(a, nullptr, false, false).bytes; }
size_t glr_bwd_ws_bytes(const GlrArgs& a) { return glr::make_plan(a, nullptr, a.z != nullptr, a.entry == nullptr).bytes; }

hipError_t launch_glr_fwd(const GlrArgs& a, hipStream_t st) {
    if (a.T == 0) {   // no tokens: S_T = S0
        if (!a.S_T || a.S_T == a.S0) return hipSuccess;
        return launch_copy_or_zero(a.S_T, a.S0, a.N * a.H * a.d, st);
    }
    glr::Plan p = glr::make_plan(a, a.ws, false, false);
    p.ws.vec = glr::rows_of_4(a) ? 4 : 1;
    return glr::launch_fwd_tiles(a, p.ws, st);
}

hipError_t launch_glr_bwd(const GlrArgs& a, hipStream_t st) {
    if (a.T == 0) {   // no tokens: dS0 = dS_T, dA_log = 0
        if (a.dA) {
            const hipError_t e = launch_copy_or_zero(a.dA, nullptr, a.H * a.d, st);
            if (e != hipSuccess) return e;
        }
        return a.dS0 ? launch_copy_or_zero(a.dS0, a.dST, a.N * a.H * a.d, st) : hipSuccess;
    }
    glr::Plan p = glr::make_plan(a, a.ws, a.z != nullptr, a.entry == nullptr);
    p.ws.vec = glr::rows_of_4(a) ? 4 : 1;
    GlrArgs b = a;
    if (!b.entry) {   // the forward again, for its entry states alone
        b.entry = p.entry;
        b.y = nullptr; b.S_T = nullptr;
        const hipError_t e = glr::launch_fwd_tiles(b, p.ws, st);
        if (e != hipSuccess) return e;
    }
    return glr::launch_bwd_tiles(b, p.ws, st);
}

hipError_t launch_glr_step(const GlrArgs& a, hipStream_t st) {
    if (a.scale == KDA_GLR_ONE) return glr::launch_step_s<KDA_GLR_ONE>(a, st);
    if (a.scale == KDA_GLR_LEAKY) return glr::launch_step_s<KDA_GLR_LEAKY>(a, st);
    return glr::launch_step_s<KDA_GLR_NORM>(a, st);
}

}  // namespace kda
