// Attention over a paged cache: the launches of a call (kda_attn_plan.h).
#include "kda_attn_kernels.h"

namespace kda {
namespace attn {

namespace {

template <int DK, int DV>
hipError_t launch(const AttnArgs& a, hipStream_t st) {
    hipError_t e = hipSuccess;
    for (int k = 0; k < 2 && e == hipSuccess; ++k) {
        const bool narrow = k == 0;
        if (!(narrow ? has_narrow(a) : has_wide(a))) continue;
        e = launch_main<DK, DV>(a, narrow, groups_most(a, narrow), st);
        if (e != hipSuccess || !may_cut(a)) continue;
        const dim3 grid((unsigned)join_groups(a, narrow));
        if (narrow)
            hipLaunchKernelGGL((attn_join_kernel<DV, true>), grid, dim3(kJoinThreads), 0, st, a);
        else
            hipLaunchKernelGGL((attn_join_kernel<DV, false>), grid, dim3(kJoinThreads), 0, st, a);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace
}  // namespace attn

size_t attn_ws_bytes(const AttnArgs& a) {
    using namespace attn;
    int64_t b = kHeadBytes;
    if (has_narrow(a)) b += slots_most(true) * partial_bytes(kNarrowRows, a.dv);
    if (has_wide(a)) b += slots_most(false) * partial_bytes(kWideRows, a.dv);
    return (size_t)b;
}

hipError_t launch_paged_attn(const AttnArgs& args, hipStream_t st) {
    using namespace attn;
    AttnArgs a = args;
    set_divisors(a);
    if (a.dk == 128) return a.dv == 128 ? launch<128, 128>(a, st) : launch<128, 64>(a, st);
    return a.dv == 128 ? launch<64, 128>(a, st) : launch<64, 64>(a, st);
}

}  // namespace kda
