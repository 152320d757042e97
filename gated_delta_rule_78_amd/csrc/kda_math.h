// fp32 exponential and logistic function of the elementwise kernels.
#pragma once

#include "kda_device.h"

namespace kda {

// e^x on the hardware's exponential: off by its rounding (1 ulp) and by |x| 2^-24 from the
// rounding of x log2(e).
__device__ __forceinline__ float exp_f(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

__device__ __forceinline__ float sigmoid_f(float x) { return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(x * -kLog2e)); }

}  // namespace kda
