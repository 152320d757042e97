// Gated linear recurrence for gfx950, short sequences and the single-token step: a thread owns VEC
// channels of a block of rows and walks its rows in order, the next ones' loads in flight. Bound by
// HBM where the channels fill the GPU, by the launch for a few sequences (a step of 32 heads of 128
// channels with both gates, fp32 states: 2.7 us for one sequence, 5.3 for 256). VEC is 4 where that
// divides the channels (no two threads may share one: states are updated in place), else 1. At most
// one chunk of rows, so the only entry state is S0.
#include "kda_glr_device.h"
#include "kda_glr_plan.h"

namespace kda {
namespace glr {

// Z, U: whether the decay comes from z and whether there is an input gate.
template <int SCALE, int Z, int U, typename TIn, int VEC>
__global__ __launch_bounds__(kRowsThreads) void glr_rows_kernel(GlrArgs a) {
    constexpr int AHEAD = 4;        // rows in flight
    const uint32_t per = (uint32_t)(a.d / VEC);
    const int64_t i = (int64_t)blockIdx.x * kRowsThreads + threadIdx.x, all = a.blocks * per;
    if (i >= all) return;
    const int64_t block = all >> 32 ? i / per : (uint32_t)i / per;
    const int64_t ch0 = (i - block * per) * VEC;
    const int64_t state = block * a.d + ch0;
    const int64_t head = a.blocks >> 32 ? block % a.H : (uint32_t)block % (uint32_t)a.H;
    const TIn* dec = (const TIn*)(Z ? a.z : a.la) + block * a.T * a.d + ch0;
    const TIn* xp = (const TIn*)a.x + block * a.T * a.d + ch0;
    const TIn* up = (const TIn*)a.u + block * a.T * a.d + ch0;
    RawRow<TIn, VEC> xr[AHEAD], dr[AHEAD], ur[AHEAD];
    auto fetch = [&](int k, int64_t t) {
        const int64_t off = (t < a.T ? t : a.T - 1) * a.d;
        dr[k] = load_row<TIn, VEC>(dec + off);
        xr[k] = load_row<TIn, VEC>(xp + off);
        if (U) ur[k] = load_row<TIn, VEC>(up + off);
    };
    // a single row (a step) is fetched alone
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
        if (k < a.T) fetch(k, k);
    float h[VEC], cz[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) h[v] = 0.f;
    if (a.S0) load_f32<VEC>(a.S0 + state, h);
    if (Z) {
        load_f32<VEC>(a.A_log + head * a.d + ch0, cz);
#pragma unroll
        for (int v = 0; v < VEC; ++v) cz[v] = -kLog2e * exp_f(cz[v]);
    }
    if (a.entry) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) a.entry[state + v] = h[v];
    }
    const float gy = a.g_min * kLog2e;
    for (int64_t t0 = 0; t0 < a.T; t0 += AHEAD) {
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int64_t t = t0 + k;
            if (t >= a.T) break;
            float x[VEC], q[VEC], g[VEC];
            unpack(xr[k], x);
            unpack(dr[k], q);
            if (U) unpack(ur[k], g);
            if (t + AHEAD < a.T) fetch(k, t + AHEAD);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float y = Z ? gy * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(cz[v] * q[v])) : q[v] * kLog2e;
                const float alpha = __builtin_amdgcn_exp2f(y);
                float b = U ? x[v] * sigmoid_f(g[v]) : x[v];
                if (SCALE != KDA_GLR_ONE) b *= scale_w<SCALE>(y, alpha);
                h[v] = fmaf(alpha, h[v], b);
            }
            if (a.y) {
                const int64_t at = (block * a.T + t) * a.d + ch0;
                if (a.out_bf16) store_row<VEC>((bf16_t*)a.y + at, h);
                else store_row<VEC>((float*)a.y + at, h);
            }
        }
    }
    if (a.S_T) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) a.S_T[state + v] = h[v];
    }
}

template <int SCALE, typename TIn, int VEC>
static hipError_t launch_rows_v(const GlrArgs& a, hipStream_t st) {
    const dim3 grid((unsigned)rows_groups(a)), threads(kRowsThreads);
    if (a.z && a.u) hipLaunchKernelGGL((glr_rows_kernel<SCALE, 1, 1, TIn, VEC>), grid, threads, 0, st, a);
    else if (a.z) hipLaunchKernelGGL((glr_rows_kernel<SCALE, 1, 0, TIn, VEC>), grid, threads, 0, st, a);
    else if (a.u) hipLaunchKernelGGL((glr_rows_kernel<SCALE, 0, 1, TIn, VEC>), grid, threads, 0, st, a);
    else hipLaunchKernelGGL((glr_rows_kernel<SCALE, 0, 0, TIn, VEC>), grid, threads, 0, st, a);
    return hipGetLastError();
}

template <int SCALE, typename TIn>
static hipError_t launch_rows_t(const GlrArgs& a, hipStream_t st) {
    return a.d % 4 == 0 ? launch_rows_v<SCALE, TIn, 4>(a, st) : launch_rows_v<SCALE, TIn, 1>(a, st);
}

hipError_t launch_rows(const GlrArgs& a, hipStream_t st) {
    if (a.scale == KDA_GLR_ONE) return a.in_bf16 ? launch_rows_t<KDA_GLR_ONE, bf16_t>(a, st) : launch_rows_t<KDA_GLR_ONE, float>(a, st);
    if (a.scale == KDA_GLR_LEAKY)
        return a.in_bf16 ? launch_rows_t<KDA_GLR_LEAKY, bf16_t>(a, st) : launch_rows_t<KDA_GLR_LEAKY, float>(a, st);
    return a.in_bf16 ? launch_rows_t<KDA_GLR_NORM, bf16_t>(a, st) : launch_rows_t<KDA_GLR_NORM, float>(a, st);
}

// The backward of blocks of at most kRowsBwd rows (formulas: kda_glr_bwd.h): the states before each
// row in registers, then the rows from the last to the first, read again from the caches.
template <int SCALE, typename TIn, typename TOut, int VEC>
__global__ __launch_bounds__(kRowsThreads) void glr_rows_bwd_kernel(GlrArgs a, float* parts) {
    const uint32_t per = (uint32_t)(a.d / VEC);
    const int64_t i = (int64_t)blockIdx.x * kRowsThreads + threadIdx.x, all = a.blocks * per;
    if (i >= all) return;
    const int64_t block = all >> 32 ? i / per : (uint32_t)i / per;
    const int64_t ch0 = (i - block * per) * VEC;
    const int64_t state = block * a.d + ch0;
    const int64_t head = a.blocks >> 32 ? block % a.H : (uint32_t)block % (uint32_t)a.H;
    const int64_t base = block * a.T * a.d + ch0;
    const TIn* dec = (const TIn*)(a.z ? a.z : a.la) + base;
    const TIn* xp = (const TIn*)a.x + base;
    const TIn* up = (const TIn*)a.u + base;
    const TOut* yp = (const TOut*)a.dy + base;
    float h[VEC], g[VEC], eA[VEC], dA[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) h[v] = g[v] = dA[v] = eA[v] = 0.f;
    if (a.S0) load_f32<VEC>(a.S0 + state, h);
    if (a.dST) load_f32<VEC>(a.dST + state, g);
    if (a.z) {
        load_f32<VEC>(a.A_log + head * a.d + ch0, eA);
#pragma unroll
        for (int v = 0; v < VEC; ++v) eA[v] = exp_f(eA[v]);
    }
    const float gy = a.g_min * kLog2e;
    struct Row {
        float x[VEC], q[VEC], al[VEC], w[VEC], gi[VEC], s[VEC];
    };
    auto row = [&](int t, Row& r) {
        const int64_t off = t * a.d;
        float u[VEC];
        unpack(load_row<TIn, VEC>(xp + off), r.x);
        unpack(load_row<TIn, VEC>(dec + off), r.q);
        if (a.u) unpack(load_row<TIn, VEC>(up + off), u);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            float y = r.q[v] * kLog2e;
            r.s[v] = 0.f;
            if (a.z) {
                r.s[v] = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * eA[v] * r.q[v]));
                y = gy * r.s[v];
            }
            r.al[v] = __builtin_amdgcn_exp2f(y);
            r.gi[v] = a.u ? sigmoid_f(u[v]) : 1.f;
            r.w[v] = scale_w<SCALE>(y, r.al[v]);
        }
    };
    float prev[kRowsBwd][VEC];
#pragma unroll
    for (int t = 0; t < kRowsBwd; ++t) {
        if (t >= a.T) continue;
        Row r;
        row(t, r);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            prev[t][v] = h[v];
            h[v] = fmaf(r.al[v], h[v], r.x[v] * r.gi[v] * r.w[v]);
        }
    }
#pragma unroll
    for (int t = kRowsBwd - 1; t >= 0; --t) {
        if (t >= a.T) continue;
        Row r;
        row(t, r);
        float dy[VEC], ox[VEC], od[VEC], ou[VEC];
        unpack(load_row<TOut, VEC>(yp + t * a.d), dy);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const float gr = g[v] + dy[v], alpha = r.al[v];
            ox[v] = gr * r.w[v] * r.gi[v];
            ou[v] = ox[v] * r.x[v] * (1.f - r.gi[v]);
            float e = alpha * prev[t][v];
            if (SCALE == KDA_GLR_LEAKY) e = fmaf(-alpha, r.x[v] * r.gi[v], e);
            if (SCALE == KDA_GLR_NORM) {
                // dw / dlog_alpha = -alpha^2 / w, taken as 0 where w = 0
                const float aw = r.w[v] > 0.f ? alpha * __builtin_amdgcn_rcpf(r.w[v]) : 0.f;
                e = fmaf(-alpha * aw, r.x[v] * r.gi[v], e);
            }
            e *= gr;
            if (a.z) {
                e *= r.s[v] * (1.f - r.s[v]) * (a.g_min * eA[v]);
                dA[v] = fmaf(e, r.q[v], dA[v]);
            }
            od[v] = e;
            g[v] = alpha * gr;
        }
        const int64_t at = base + t * a.d;
        store_row<VEC>((TIn*)a.dx + at, ox);
        store_row<VEC>((TIn*)a.dd + at, od);
        if (a.u) store_row<VEC>((TIn*)a.du + at, ou);
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        if (a.dS0) a.dS0[state + v] = g[v];
        if (a.z) parts[state + v] = dA[v];
    }
}

template <int SCALE, typename TIn, typename TOut>
static hipError_t launch_rows_bwd_t(const GlrArgs& a, float* parts, hipStream_t st) {
    const dim3 grid((unsigned)rows_groups(a)), threads(kRowsThreads);
    if (a.d % 4 == 0) hipLaunchKernelGGL((glr_rows_bwd_kernel<SCALE, TIn, TOut, 4>), grid, threads, 0, st, a, parts);
    else hipLaunchKernelGGL((glr_rows_bwd_kernel<SCALE, TIn, TOut, 1>), grid, threads, 0, st, a, parts);
    return hipGetLastError();
}

template <int SCALE>
static hipError_t launch_rows_bwd_s(const GlrArgs& a, float* parts, hipStream_t st) {
    if (a.in_bf16 && a.out_bf16) return launch_rows_bwd_t<SCALE, bf16_t, bf16_t>(a, parts, st);
    if (a.in_bf16) return launch_rows_bwd_t<SCALE, bf16_t, float>(a, parts, st);
    if (a.out_bf16) return launch_rows_bwd_t<SCALE, float, bf16_t>(a, parts, st);
    return launch_rows_bwd_t<SCALE, float, float>(a, parts, st);
}

hipError_t launch_rows_bwd(const GlrArgs& a, float* parts, hipStream_t st) {
    if (a.scale == KDA_GLR_ONE) return launch_rows_bwd_s<KDA_GLR_ONE>(a, parts, st);
    if (a.scale == KDA_GLR_LEAKY) return launch_rows_bwd_s<KDA_GLR_LEAKY>(a, parts, st);
    return launch_rows_bwd_s<KDA_GLR_NORM>(a, parts, st);
}

}  // namespace glr
}  // namespace kda
