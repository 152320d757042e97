// Backward of the head norms with rotation, instantiated per type in kda_rope_{bf16,f32}.hip.
//
//   dy = R^T dz,  xh = x / sqrt(mean x^2 + eps),  dweight = sum dy xh,
//   dx = (t - xh mean(t xh)) / sqrt(mean x^2 + eps),  t = dy weight        (dx = dy without norm)
//
// Workgroups walk blocks of tokens with the weights' sums in registers; each writes its sums once,
// and a second launch adds them in order (rope_colsum_kernel).
#pragma once

#include "kda_rope_fwd.h"

namespace kda {
namespace rope {

template <typename T, int LAY, bool KEYS>
__device__ __forceinline__ void grad_rows(const RopeArgs& a, const Lane& l, const Token* tok, const float2* cs, int ntok,
                                          uint32_t magic, float* dw) {
    constexpr int U = sizeof(T) == 2 ? 2 : 1;
    const int H = KEYS ? a.Hk : a.Hq, rg = 64 / l.lpr, rows = ntok * H, P = a.d / 2;
    const T* src = static_cast<const T*>(KEYS ? a.k : a.q);
    const T* grd = static_cast<const T*>(KEYS ? a.dko : a.dqo);
    T* dst = static_cast<T*>(KEYS ? a.dk : a.dq);
    const int64_t sh = KEYS ? a.sk.h : a.sq.h, gh = KEYS ? a.sko.h : a.sqo.h, dh = KEYS ? a.sdk.h : a.sdq.h;
    const float inv_d = 1.f / (float)a.d;
    float w[16];
    if (a.norm) load_weight<LAY>(l, KEYS ? a.wk : a.wq, w);
    for (int base = (threadIdx.x >> 6) * rg * U; base < rows; base += kWaves * rg * U) {
        float z[U][16], x[U][16];
        int tk[U];
        int64_t out[U];
        bool on[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = base + u * rg + l.g;
            on[u] = r < rows;
            const int rr = on[u] ? r : 0;
            const int t = div_heads(rr, magic), h = rr - t * H;
            tk[u] = t;
            out[u] = (KEYS ? tok[t].sdk : tok[t].sdq) + h * dh;
            load_row<T, LAY>(l, grd + ((KEYS ? tok[t].ko : tok[t].qo) + h * gh), on[u], z[u]);
            if (a.norm) load_row<T, LAY>(l, src + ((KEYS ? tok[t].k : tok[t].q) + h * sh), on[u], x[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            to_pairs<LAY>(z[u]);
            if (a.rot) {
                float co[8], si[8];
                load_angles<LAY>(l, cs + tk[u] * P, co, si);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float va = z[u][j], vb = z[u][8 + j];
                    z[u][j] = fmaf(va, co[j], vb * si[j]);
                    z[u][8 + j] = fmaf(vb, co[j], -va * si[j]);
                }
            }
            if (a.norm) {
                to_pairs<LAY>(x[u]);
                float s = 0.f;
#pragma unroll
                for (int j = 0; j < 16; ++j) s = fmaf(x[u][j], x[u][j], s);
                s = row_sum(s, l.lpr);
                const float r = 1.f / sqrtf(fmaf(s, inv_d, a.eps));
                float m = 0.f;
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    x[u][j] *= r;
                    dw[j] = fmaf(z[u][j], x[u][j], dw[j]);
                    z[u][j] *= w[j];
                    m = fmaf(z[u][j], x[u][j], m);
                }
                m = row_sum(m, l.lpr) * inv_d;
#pragma unroll
                for (int j = 0; j < 16; ++j) z[u][j] = r * fmaf(-m, x[u][j], z[u][j]);
            }
            from_pairs<LAY>(z[u]);
            if (on[u]) store_row<T, LAY>(l, dst + out[u], z[u]);
        }
    }
}

// Sums of the workgroup's waves and row groups into ws[group][KEYS][d].
template <int LAY>
__device__ __forceinline__ void put_sums(const RopeArgs& a, const Lane& l, float* dw, float* part, int kind) {
    const int wave = threadIdx.x >> 6;
#pragma unroll
    for (int j = 0; j < 16; ++j)
        for (int m = l.lpr; m < 64; m <<= 1) dw[j] += __shfl_xor(dw[j], m);
    from_pairs<LAY>(dw);
    if (l.g == 0) store_row<float, LAY>(l, part + (size_t)wave * a.d, dw);
    lds_barrier();
    for (int c = threadIdx.x; c < a.d; c += kThreads) {
        float s = part[c];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) s += part[w * a.d + c];
        a.ws[((int64_t)blockIdx.x * 2 + kind) * a.d + c] = s;
    }
    lds_barrier();
}

template <typename T, int LAY>
__global__ __launch_bounds__(kThreads) void rope_bwd_kernel(RopeArgs a, Shape s, int sums) {
    extern __shared__ __align__(16) float2 cs[];     // the tokens' angles, or the waves' weight sums
    __shared__ Token tok[kMaxTokens];
    const int64_t all = a.B * a.T;
    const Lane l = make_lane<LAY>(a, s.lpr);
    float dwq[16], dwk[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) dwq[j] = dwk[j] = 0.f;
    for (int64_t u0 = (int64_t)blockIdx.x * s.tokens; u0 < all; u0 += (int64_t)gridDim.x * s.tokens) {
        const int ntok = (int)(all - u0 < s.tokens ? all - u0 : s.tokens);
        lds_barrier();                               // the block before is through with LDS
        fill_tokens<false>(a, tok, u0, ntok);
        lds_barrier();
        if (a.rot) {
            fill_angles(a, tok, ntok, cs);
            lds_barrier();
        }
        if (a.Hq) grad_rows<T, LAY, false>(a, l, tok, cs, ntok, s.mq, dwq);
        if (a.Hk) grad_rows<T, LAY, true>(a, l, tok, cs, ntok, s.mk, dwk);
    }
    if (sums) {
        float* part = reinterpret_cast<float*>(cs);
        lds_barrier();
        put_sums<LAY>(a, l, dwq, part, 0);
        put_sums<LAY>(a, l, dwk, part, 1);
    }
}

template <typename T>
hipError_t launch_grads(const RopeArgs& a, const Shape& s, int lay, int groups, bool sums, hipStream_t st) {
    const dim3 grid((unsigned)groups), block(kThreads);
    size_t lds = a.rot ? (size_t)s.tokens * (a.d / 2) * sizeof(float2) : 0;
    const size_t part = (size_t)kWaves * a.d * sizeof(float);
    if (sums && part > lds) lds = part;
    const int sm = sums;
    switch (lay) {
        case kHalfWide: hipLaunchKernelGGL((rope_bwd_kernel<T, kHalfWide>), grid, block, lds, st, a, s, sm); break;
        case kInterWide: hipLaunchKernelGGL((rope_bwd_kernel<T, kInterWide>), grid, block, lds, st, a, s, sm); break;
        case kHalfElem: hipLaunchKernelGGL((rope_bwd_kernel<T, kHalfElem>), grid, block, lds, st, a, s, sm); break;
        default: hipLaunchKernelGGL((rope_bwd_kernel<T, kInterElem>), grid, block, lds, st, a, s, sm); break;
    }
    return hipGetLastError();
}

}  // namespace rope
}  // namespace kda
