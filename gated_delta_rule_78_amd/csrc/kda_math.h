// fp32 exponential and logistic function of the elementwise kernels.
#pragma once

#include "kda_device.h"

namespace kda {

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2eLo = 1.9259629911266175e-8f;   // log2(e) - (float)log2(e)

// e^x to about 1 ulp: x log2(e) as a rounded product plus its error, the error applied to first
// order. Infinities and NaN skip the correction (it would be inf - inf).
__device__ __forceinline__ float exp_f(float x) {
    const float h = x * kLog2e;
    const float l = fmaf(x, kLog2eLo, fmaf(x, kLog2e, -h));
    const float e = __builtin_amdgcn_exp2f(h);
    return fabsf(x) < 256.f ? fmaf(e * l, kLn2, e) : e;
}

__device__ __forceinline__ float sigmoid_f(float x) { return __builtin_amdgcn_rcpf(1.f + exp_f(-x)); }

}  // namespace kda
