// Elementwise arithmetic of the gated linear recurrence: the gates and their derivatives.
#pragma once

#include "kda_glr.h"
#include "kda_math.h"

namespace kda {
namespace glr {

// alpha = e^la and, with W, 1 - alpha without the cancellation near alpha = 1: for la > -0.35 from
// e^la - 1 = la (1 + la/2 (1 + la/3 (...))), cut after la^8 / 8! (relative error 0.35^8 / 9! < 1e-9).
template <bool W>
__device__ __forceinline__ void decay_f(float la, float& alpha, float& one_minus) {
    alpha = exp_f(la);
    if constexpr (W) {
        float p = fmaf(la, 1.f / 8.f, 1.f);
        p = fmaf(p * la, 1.f / 7.f, 1.f);
        p = fmaf(p * la, 1.f / 6.f, 1.f);
        p = fmaf(p * la, 1.f / 5.f, 1.f);
        p = fmaf(p * la, 1.f / 4.f, 1.f);
        p = fmaf(p * la, 1.f / 3.f, 1.f);
        p = fmaf(p * la, 1.f / 2.f, 1.f);
        one_minus = la > -0.35f ? -la * p : 1.f - alpha;
    }
}

// The input scale w(alpha) from alpha and 1 - alpha.
template <int SCALE>
__device__ __forceinline__ float scale_w(float alpha, float one_minus) {
    if constexpr (SCALE == KDA_GLR_ONE) return 1.f;
    if constexpr (SCALE == KDA_GLR_LEAKY) return one_minus;
    return __builtin_amdgcn_sqrtf(one_minus * (1.f + alpha));
}

// dw / dlog_alpha: 0, -alpha, -alpha^2 / w (taken as 0 where w = 0).
template <int SCALE>
__device__ __forceinline__ float scale_dw(float alpha, float one_minus) {
    if constexpr (SCALE == KDA_GLR_ONE) return 0.f;
    if constexpr (SCALE == KDA_GLR_LEAKY) return -alpha;
    const float w2 = one_minus * (1.f + alpha);
    return w2 > 0.f ? -alpha * alpha * __builtin_amdgcn_rsqf(w2) : 0.f;
}

}  // namespace glr
}  // namespace kda
