// The main launch of the attention over a paged cache, instantiated per head sizes in kda_attn_d*.hip.
#pragma once

#include "kda_attn_kernels.h"

namespace kda {
namespace attn {

template <int DK, int DV>
hipError_t launch_main(const AttnArgs& a, bool narrow, int64_t groups, hipStream_t st) {
    const dim3 grid((unsigned)groups), block(narrow ? kThreads : kWideThreads);
    if (narrow)
        hipLaunchKernelGGL((attn_narrow_kernel<DK, DV>), grid, block, 0, st, a);
    else
        hipLaunchKernelGGL((attn_wide_kernel<DK, DV>), grid, block, 0, st, a);
    return hipGetLastError();
}

}  // namespace attn
}  // namespace kda
