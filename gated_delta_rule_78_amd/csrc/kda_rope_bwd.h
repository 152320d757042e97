// Backward of the head norms with rotation, instantiated per type in kda_rope_{bf16,f32}.hip.
//
//   dy = R^T dz,  xh = x / sqrt(mean x^2 + eps),  dweight = sum dy xh,
//   dx = (t - xh mean(t xh)) / sqrt(mean x^2 + eps),  t = dy weight        (dx = dy without norm)
//
// Workgroups walk blocks of tokens of one tensor with the weight's sums in registers; each writes its
// sums once, and a second launch adds them in order (rope_colsum_kernel).
#pragma once

#include "kda_rope_fwd.h"

namespace kda {
namespace rope {

template <typename T, int LAY>
__global__ __launch_bounds__(kThreads, kLaysWide<LAY> ? 3 : 2) void rope_bwd_kernel(RopeArgs a, Shape s, int sums) {
    extern __shared__ __align__(16) float2 cs[];     // the tokens' angles, or the waves' weight sums
    __shared__ Token tok[kMaxTokens];
    const int64_t wg = blockIdx.x;
    const bool keys = wg >= s.group0[1];
    const int kind = keys ? kKeys : kQueries;
    const int64_t all = a.B * a.T, groups = s.group0[kind + 1] - s.group0[kind];
    const Lane l = make_lane<LAY>(a, s.lpr);
    const int rg = 64 / l.lpr, P = a.d / 2;
    const T *src = static_cast<const T*>(keys ? a.k : a.q), *grd = static_cast<const T*>(keys ? a.dko : a.dqo);
    T* dst = static_cast<T*>(keys ? a.dk : a.dq);
    const kda_row_strides &si = keys ? a.sk : a.sq, &sg = keys ? a.sko : a.sqo, &so = keys ? a.sdk : a.sdq;
    const float inv_d = 1.f / (float)a.d;
    float w[16], dw[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) dw[j] = 0.f;
    if (a.norm) load_weight<LAY>(l, keys ? a.wk : a.wq, w);
    for (int64_t g = wg - s.group0[kind]; g * s.tokens[kind] < all; g += groups) {
        int ntok;
        const Rows3 rows = rows_of(a, s, kind, g, ntok);
        int r = (threadIdx.x >> 6) * rg + l.g;
        Row row = rows.row(r < rows.count ? r : 0);
        Raw<T, LAY> rz, rx;
        auto load = [&]() {
            rz.load(l, grd + row.at(sg));
            if (a.norm) rx.load(l, src + row.at(si));
        };
        load();
        lds_barrier();                               // the block before is through with LDS
        fill_tokens<false>(a, tok, rows.u0, ntok, kind);
        lds_barrier();
        if (a.rot) {
            fill_angles(a, tok, ntok, cs);
            lds_barrier();
        }
#pragma unroll 1
        for (int first = (threadIdx.x >> 6) * rg; first < rows.count; first += kWaves * rg) {
            const bool on = r < rows.count;
            const Row now = row;
            float z[16], x[16];
            rz.get(l, z);
            if (a.norm) rx.get(l, x);
            r += kWaves * rg;
            if (first + kWaves * rg < rows.count) {
                row = rows.row(r < rows.count ? r : 0);
                load();
            }
            if (a.rot) {
                float co[8], sn[8];
                load_angles<LAY>(l, cs + now.t * P, co, sn);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float va = z[j], vb = z[8 + j];
                    z[j] = fmaf(va, co[j], vb * sn[j]);
                    z[8 + j] = fmaf(vb, co[j], -va * sn[j]);
                }
            }
            if (a.norm) {
                float q = 0.f, m = 0.f;
#pragma unroll
                for (int j = 0; j < 16; ++j) q = fmaf(x[j], x[j], q);
                const float n = inv_root(fmaf(row_sum(q, l.lpr), inv_d, a.eps));
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    x[j] *= n;
                    if (on) dw[j] = fmaf(z[j], x[j], dw[j]);
                    z[j] *= w[j];
                    m = fmaf(z[j], x[j], m);
                }
                m = row_sum(m, l.lpr) * inv_d;
#pragma unroll
                for (int j = 0; j < 16; ++j) z[j] = n * fmaf(-m, x[j], z[j]);
            }
            from_pairs<LAY>(z);
            if (on) store_row<T, LAY>(l, dst + now.at(so), z);
        }
    }
    if (sums) {
        // the sums of the wave's row groups, then of the waves, into ws[workgroup][d]
        float* part = reinterpret_cast<float*>(cs);
        lds_barrier();
#pragma unroll 1
        for (int m = l.lpr; m < 64; m <<= 1) {
#pragma unroll
            for (int j = 0; j < 16; ++j) dw[j] += __shfl_xor(dw[j], m);
        }
        from_pairs<LAY>(dw);
        if (l.g == 0) store_row<float, LAY>(l, part + (size_t)(threadIdx.x >> 6) * a.d, dw);
        lds_barrier();
        for (int c = threadIdx.x; c < a.d; c += kThreads) {
            float v = part[c];
#pragma unroll
            for (int i = 1; i < kWaves; ++i) v += part[i * a.d + c];
            a.ws[wg * a.d + c] = v;
        }
    }
}

template <typename T>
hipError_t launch_grads(const RopeArgs& a, const Shape& s, int lay, bool sums, hipStream_t st) {
    const dim3 grid((unsigned)s.group0[2]), block(kThreads);
    const int most = s.tokens[0] > s.tokens[1] ? s.tokens[0] : s.tokens[1];
    size_t lds = a.rot ? (size_t)most * (a.d / 2) * sizeof(float2) : 0;
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
