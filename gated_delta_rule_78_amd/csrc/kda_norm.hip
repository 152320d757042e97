// Block norms for gfx950: dispatch by type, and the weight gradients' last step.
#include "kda_device.h"
#include "kda_norm_internal.h"

namespace kda {
namespace norm {

// Weight gradients from the workgroups' sums [groups][2][D]: 16 runs of workgroups a column, each
// summed in order by a thread, joined in LDS in order. Latency bound: 4.7 us for 256 workgroups' sums
// of 4096 channels (8.4 MB).
__global__ __launch_bounds__(1024) void norm_colsum_kernel(NormArgs a, int groups) {
    __shared__ float part[16][64];
    const int lane = threadIdx.x & 63, run = threadIdx.x >> 6, k = blockIdx.y;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    if (k == 0 ? !a.dw_post && !a.dlam : !a.dw_pre) return;
    const int each = (groups + 15) / 16, g1 = (run + 1) * each < groups ? (run + 1) * each : groups;
    float s = 0.f;
    if (c < a.D) {
#pragma unroll 8
        for (int g = run * each; g < g1; ++g) s += a.ws[((int64_t)g * 2 + k) * a.D + c];
    }
    part[run][lane] = s;
    lds_barrier();
    if (run != 0 || c >= a.D) return;
#pragma unroll
    for (int i = 1; i < 16; ++i) s += part[i][lane];
    if (k == 1) {
        a.dw_pre[c] = s;
        return;
    }
    if (a.dw_post) a.dw_post[c] = s * a.scale * (a.lam ? a.lam[c] : 1.f);
    if (a.dlam) a.dlam[c] = s * a.scale * (a.w_post ? a.w_post[c] : 1.f);
}

hipError_t launch_colsum(const NormArgs& a, int groups, hipStream_t st) {
    hipLaunchKernelGGL(norm_colsum_kernel, dim3((unsigned)((a.D + 63) / 64), 2), dim3(1024), 0, st, a, groups);
    return hipGetLastError();
}

}  // namespace norm

size_t norm_bwd_ws_bytes(int64_t rows, int64_t D) {
    const int most = norm::bwd_groups(256, 0);   // no launch has more workgroups, nor more than rows
    return (size_t)((rows < most ? rows : most) * 2 * D) * 4;
}

hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t st) {
    return a.in_bf16 ? norm::launch_i<bf16_t>(a, false, st) : norm::launch_i<float>(a, false, st);
}

hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t st) {
    return a.in_bf16 ? norm::launch_i<bf16_t>(a, true, st) : norm::launch_i<float>(a, true, st);
}

}  // namespace kda
