// Attention over a paged cache: the plan of a call and its launches (kda_attn_plan.h).
#include "kda_attn_kernels.h"

namespace kda {
namespace attn {

// One workgroup: each kind's units of keys, its chunk length, and running sums over the sequences of
// workgroups, partial results and cut (tile, head)s.
__global__ __launch_bounds__(1024) void attn_plan_kernel(AttnArgs a) {
    __shared__ unsigned long long units[2];
    __shared__ int carry[2][3], wave_sum[16][6];
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    if (tid < 2) units[tid] = 0;
    if (tid < 6) carry[tid / 3][tid % 3] = 0;
    __syncthreads();
    unsigned long long mine[2] = {0, 0};
    for (int64_t s = tid; s < a.N; s += 1024) {
        int64_t first;
        int n, kv;
        if (!sequence(a, s, first, n, kv)) continue;
#pragma unroll
        for (int k = 0; k < 2; ++k)
            mine[k] += tiles_of(a, n, k == 0) * tile_units(a, kv, k == 0 ? kNarrowRows : kWideRows) * a.Hk;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (mine[k]) atomicAdd(&units[k], mine[k]);       // whole numbers: any order
    __syncthreads();
    int64_t len[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        len[k] = (int64_t)((units[k] + target(k == 0) - 1) / target(k == 0));
        if (len[k] < kMinUnits) len[k] = kMinUnits;
    }
    PlanEntry* plan = static_cast<PlanEntry*>(a.ws);
    for (int64_t s0 = 0; s0 < a.N; s0 += 1024) {
        const int64_t s = s0 + tid;
        int v[6] = {0, 0, 0, 0, 0, 0}, chunks[2] = {1, 1};
        int64_t first;
        int n, kv;
        if (s < a.N && sequence(a, s, first, n, kv)) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int64_t tiles = tiles_of(a, n, k == 0) * a.Hk;
                chunks[k] = (int)((tile_units(a, kv, k == 0 ? kNarrowRows : kWideRows) + len[k] - 1) / len[k]);
                v[3 * k] = (int)(tiles * chunks[k]);
                v[3 * k + 1] = chunks[k] > 1 ? v[3 * k] : 0;
                v[3 * k + 2] = chunks[k] > 1 ? (int)tiles : 0;
            }
        }
        int in[6];
#pragma unroll
        for (int i = 0; i < 6; ++i) {
            int x = v[i];
            for (int m = 1; m < 64; m <<= 1) {
                const int y = __shfl_up(x, m);
                if (lane >= m) x += y;
            }
            if (lane == 63) wave_sum[wv][i] = x;
            in[i] = x - v[i];
        }
        __syncthreads();
        int total[6];
#pragma unroll
        for (int i = 0; i < 6; ++i) {
            in[i] += carry[i / 3][i % 3];
            total[i] = carry[i / 3][i % 3];
            for (int w = 0; w < 16; ++w) {
                if (w < wv) in[i] += wave_sum[w][i];
                total[i] += wave_sum[w][i];
            }
        }
        if (s < a.N)
#pragma unroll
            for (int k = 0; k < 2; ++k) plan[k * (a.N + 1) + s] = PlanEntry{in[3 * k], in[3 * k + 1], in[3 * k + 2], chunks[k]};
        __syncthreads();
        if (tid == 0)
            for (int i = 0; i < 6; ++i) carry[i / 3][i % 3] = total[i];
        __syncthreads();
    }
    if (tid < 2) plan[tid * (a.N + 1) + a.N] = PlanEntry{carry[tid][0], carry[tid][1], carry[tid][2], 1};
}

namespace {

// Workgroups at most: every tile once, and the chunks beyond the first of each.
int64_t groups_most(const AttnArgs& a, bool narrow) {
    const int64_t tiles = tiles_most(a, narrow ? kNarrowRows : kWideRows, narrow) * a.Hk;
    return tiles + (may_cut(a) ? target(narrow) : 0);
}

template <int DK, int DV>
hipError_t launch(const AttnArgs& a, hipStream_t st) {
    hipLaunchKernelGGL(attn_plan_kernel, dim3(1), dim3(1024), 0, st, a);
    hipError_t e = hipGetLastError();
    for (int k = 0; k < 2 && e == hipSuccess; ++k) {
        const bool narrow = k == 0;
        if (!(narrow ? has_narrow(a) : has_wide(a))) continue;
        e = launch_main<DK, DV>(a, narrow, groups_most(a, narrow), st);
        if (e != hipSuccess || !may_cut(a)) continue;
        const int rows = narrow ? kNarrowRows : kWideRows, each = 4;
        const dim3 grid((unsigned)target(narrow), (unsigned)(rows / each));
        if (narrow)
            hipLaunchKernelGGL((attn_join_kernel<DV, true>), grid, dim3(kThreads), 0, st, a, each);
        else
            hipLaunchKernelGGL((attn_join_kernel<DV, false>), grid, dim3(kThreads), 0, st, a, each);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace
}  // namespace attn

size_t attn_ws_bytes(const AttnArgs& a) {
    using namespace attn;
    int64_t b = plan_bytes(a.N);
    if (has_narrow(a)) b += slots_most(true) * partial_bytes(kNarrowRows, a.dv);
    if (has_wide(a)) b += slots_most(false) * partial_bytes(kWideRows, a.dv);
    return (size_t)b;
}

hipError_t launch_paged_attn(const AttnArgs& a, hipStream_t st) {
    using namespace attn;
    for (int k = 0; k < 2; ++k)     // a launch has fewer than 2^32 threads
        if (groups_most(a, k == 0) >= (int64_t)1 << 23) return hipErrorInvalidConfiguration;
    if (a.dk == 128) return a.dv == 128 ? launch<128, 128>(a, st) : launch<128, 64>(a, st);
    return a.dv == 128 ? launch<64, 128>(a, st) : launch<64, 64>(a, st);
}

}  // namespace kda
