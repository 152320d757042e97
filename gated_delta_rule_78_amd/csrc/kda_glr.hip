// Gated linear recurrence for gfx950 (include/kda_glr.h): per (sequence, head, channel)
//     h_t = alpha_t h_{t-1} + w(alpha_t) i_t x_t,   y_t = h_t,
// and its reverse, with g_t = dL/dh_t:
//     g_t = dy_t + alpha_{t+1} g_{t+1}  (dS_T added at a sequence's last row),
//     dx_t = g_t w_t i_t,  din_gate_t = g_t w_t x_t i_t (1 - i_t),
//     dlog_alpha_t = g_t (alpha_t h_{t-1} + w'_t i_t x_t),
//     dz_t = dlog_alpha_t g_min e^A s_t (1 - s_t),  dA_log = sum_t dlog_alpha_t log_alpha_t (1 - s_t) e^A z_t,
//     dS0 = alpha_1 g_1.
//
// One thread per (head, channel) walks every sequence in order.
#include "kda_glr_device.h"
#include "kda_glr_internal.h"
#include "kda_internal.h"

namespace kda {
namespace glr {

constexpr int kCh = KDA_GLR_CHUNK;

struct Row {
    float alpha, om, w, i, la, s, x;
};

template <int SCALE, typename TIn>
__device__ __forceinline__ Row load_row(const GlrArgs& a, int64_t at, float eA) {
    Row r;
    r.x = ld_f((const TIn*)a.x + at);
    if (a.z) {
        r.s = sigmoid_f(eA * ld_f((const TIn*)a.z + at));
        r.la = a.g_min * r.s;
    } else {
        r.s = 0.f;
        r.la = ld_f((const TIn*)a.la + at);
    }
    r.om = 0.f;
    decay_f<SCALE != KDA_GLR_ONE>(r.la, r.alpha, r.om);
    r.w = scale_w<SCALE>(r.alpha, r.om);
    r.i = a.u ? sigmoid_f(ld_f((const TIn*)a.u + at)) : 1.f;
    return r;
}

// Rows of sequence n inside its block.
__device__ __forceinline__ void rows_of(const GlrArgs& a, int64_t n, int64_t& r0, int64_t& r1) {
    r0 = 0; r1 = a.T;
    if (a.packed) {
        r0 = a.cu[n]; r1 = a.cu[n + 1];
        r0 = r0 < 0 ? 0 : r0;
        r1 = r1 > a.T ? a.T : r1;
    }
}

template <int SCALE, typename TIn, typename TOut>
__global__ __launch_bounds__(64) void glr_fwd_kernel(GlrArgs a) {
    const int64_t hc = (int64_t)blockIdx.x * 64 + threadIdx.x;
    if (hc >= a.H * a.d) return;
    const int64_t h = hc / a.d, c = hc % a.d;
    const float eA = a.z ? exp_f(a.A_log[hc]) : 0.f;
    for (int64_t n = 0; n < a.N; ++n) {
        int64_t r0, r1;
        rows_of(a, n, r0, r1);
        const int64_t b = a.packed ? h : n * a.H + h, sidx = (n * a.H + h) * a.d + c;
        float st = a.S0 ? a.S0[sidx] : 0.f;
        for (int64_t t = r0; t < r1; ++t) {
            if (a.entry && t % kCh == 0) a.entry[(b * a.nch + t / kCh) * a.d + c] = st;
            const int64_t at = (b * a.T + t) * a.d + c;
            const Row r = load_row<SCALE, TIn>(a, at, eA);
            st = fmaf(r.alpha, st, r.w * r.i * r.x);
            if (a.y) st_f((TOut*)a.y + at, st);
        }
        if (a.S_T) a.S_T[sidx] = st;
    }
}

template <int SCALE, typename TIn, typename TOut>
__global__ __launch_bounds__(64) void glr_bwd_kernel(GlrArgs a) {
    const int64_t hc = (int64_t)blockIdx.x * 64 + threadIdx.x;
    if (hc >= a.H * a.d) return;
    const int64_t h = hc / a.d, c = hc % a.d;
    const float eA = a.z ? exp_f(a.A_log[hc]) : 0.f;
    float dA = 0.f;
    float prev[kCh];
    for (int64_t n = 0; n < a.N; ++n) {
        int64_t r0, r1;
        rows_of(a, n, r0, r1);
        const int64_t b = a.packed ? h : n * a.H + h, sidx = (n * a.H + h) * a.d + c;
        float g = a.dST ? a.dST[sidx] : 0.f;
        for (int64_t k = r1 > r0 ? (r1 - 1) / kCh : -1; k >= r0 / kCh && k >= 0; --k) {
            const int64_t lo = r0 > k * kCh ? r0 : k * kCh, hi = r1 < (k + 1) * kCh ? r1 : (k + 1) * kCh;
            float st = lo == r0 ? (a.S0 ? a.S0[sidx] : 0.f) : a.entry[(b * a.nch + k) * a.d + c];
            for (int64_t t = lo; t < hi; ++t) {
                prev[t - k * kCh] = st;
                const Row r = load_row<SCALE, TIn>(a, (b * a.T + t) * a.d + c, eA);
                st = fmaf(r.alpha, st, r.w * r.i * r.x);
            }
            for (int64_t t = hi - 1; t >= lo; --t) {
                const int64_t at = (b * a.T + t) * a.d + c;
                const Row r = load_row<SCALE, TIn>(a, at, eA);
                g += ld_f((const TOut*)a.dy + at);
                const float gw = g * r.w;
                st_f((TIn*)a.dx + at, gw * r.i);
                if (a.du) st_f((TIn*)a.du + at, gw * r.i * (1.f - r.i) * r.x);
                float dla = r.alpha * prev[t - k * kCh];
                if constexpr (SCALE != KDA_GLR_ONE) dla = fmaf(scale_dw<SCALE>(r.alpha, r.om), r.i * r.x, dla);
                dla *= g;
                if (a.z) {
                    const float e = dla * r.la * (1.f - r.s) * eA;
                    st_f((TIn*)a.dd + at, e);
                    dA = fmaf(e, ld_f((const TIn*)a.z + at), dA);
                } else {
                    st_f((TIn*)a.dd + at, dla);
                }
                g *= r.alpha;
            }
        }
        if (a.dS0) a.dS0[sidx] = g;
    }
    if (a.dA) a.dA[hc] = dA;
}

template <int SCALE, typename TIn, typename TOut>
__global__ __launch_bounds__(256) void glr_step_kernel(GlrArgs a) {
    const int64_t n = a.N * a.H * a.d;
    for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < n; at += (int64_t)gridDim.x * 256) {
        const float eA = a.z ? exp_f(a.A_log[at % (a.H * a.d)]) : 0.f;
        const Row r = load_row<SCALE, TIn>(a, at, eA);
        const float st = fmaf(r.alpha, a.S[at], r.w * r.i * r.x);
        a.S[at] = st;
        st_f((TOut*)a.y + at, st);
    }
}

enum { kFwd, kBwd, kStep };

template <int SCALE, typename TIn, typename TOut>
static hipError_t launch_t(const GlrArgs& a, int what, hipStream_t st) {
    const int64_t hd = a.H * a.d;
    if (what == kStep) {
        const int64_t n = a.N * hd;
        const int64_t grid = (n + 255) / 256 < (1 << 20) ? (n + 255) / 256 : (1 << 20);
        hipLaunchKernelGGL((glr_step_kernel<SCALE, TIn, TOut>), dim3((unsigned)grid), dim3(256), 0, st, a);
    } else if (what == kBwd) {
        hipLaunchKernelGGL((glr_bwd_kernel<SCALE, TIn, TOut>), dim3((unsigned)((hd + 63) / 64)), dim3(64), 0, st, a);
    } else {
        hipLaunchKernelGGL((glr_fwd_kernel<SCALE, TIn, TOut>), dim3((unsigned)((hd + 63) / 64)), dim3(64), 0, st, a);
    }
    return hipGetLastError();
}

template <int SCALE>
static hipError_t launch_s(const GlrArgs& a, int what, hipStream_t st) {
    if (a.in_bf16 && a.out_bf16) return launch_t<SCALE, bf16_t, bf16_t>(a, what, st);
    if (a.in_bf16) return launch_t<SCALE, bf16_t, float>(a, what, st);
    if (a.out_bf16) return launch_t<SCALE, float, bf16_t>(a, what, st);
    return launch_t<SCALE, float, float>(a, what, st);
}

static hipError_t launch(const GlrArgs& a, int what, hipStream_t st) {
    if (a.scale == KDA_GLR_ONE) return launch_s<KDA_GLR_ONE>(a, what, st);
    if (a.scale == KDA_GLR_LEAKY) return launch_s<KDA_GLR_LEAKY>(a, what, st);
    return launch_s<KDA_GLR_NORM>(a, what, st);
}

}  // namespace glr

size_t glr_fwd_ws_bytes(const GlrArgs&) { return 0; }
size_t glr_bwd_ws_bytes(const GlrArgs& a) { return a.entry ? 0 : (size_t)(a.blocks * a.nch * a.d) * 4; }

hipError_t launch_glr_fwd(const GlrArgs& a, hipStream_t st) {
    if (a.T == 0) {   // no tokens: S_T = S0
        if (!a.S_T || a.S_T == a.S0) return hipSuccess;
        return launch_copy_or_zero(a.S_T, a.S0, a.N * a.H * a.d, st);
    }
    return glr::launch(a, glr::kFwd, st);
}

hipError_t launch_glr_bwd(const GlrArgs& a, hipStream_t st) {
    if (a.T == 0) {   // no tokens: dS0 = dS_T, dA_log = 0
        if (a.dA) {
            const hipError_t e = launch_copy_or_zero(a.dA, nullptr, a.H * a.d, st);
            if (e != hipSuccess) return e;
        }
        return a.dS0 ? launch_copy_or_zero(a.dS0, a.dST, a.N * a.H * a.d, st) : hipSuccess;
    }
    GlrArgs b = a;
    if (!b.entry) {   // the forward's chunk entry states into the workspace
        b.entry = reinterpret_cast<float*>(a.ws);
        b.y = nullptr; b.S_T = nullptr;
        const hipError_t e = glr::launch(b, glr::kFwd, st);
        if (e != hipSuccess) return e;
    }
    return glr::launch(b, glr::kBwd, st);
}

hipError_t launch_glr_step(const GlrArgs& a, hipStream_t st) { return glr::launch(a, glr::kStep, st); }

}  // namespace kda
