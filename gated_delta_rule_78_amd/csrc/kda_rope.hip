// Head norms with rotation and the cache append: which layout and how many tokens a workgroup takes,
// and the weight gradients' last step (include/kda_attn.h).
#include "kda_rope.h"

namespace kda {
namespace rope {

template <typename TI, typename TO, bool APPEND>
hipError_t launch_rows(const RopeArgs& a, const Shape& s, int lay, hipStream_t st);
template <typename T>
hipError_t launch_grads(const RopeArgs& a, const Shape& s, int lay, bool sums, hipStream_t st);

// dq_weight and dk_weight from the workgroups' sums [workgroup][d]: 16 runs of workgroups a channel,
// each summed in order by a thread, joined in LDS in order.
__global__ __launch_bounds__(1024) void rope_colsum_kernel(RopeArgs a, Shape s) {
    __shared__ float part[16][64];
    const int lane = threadIdx.x & 63, run = threadIdx.x >> 6, k = blockIdx.y;
    const int c = blockIdx.x * 64 + lane;
    float* out = k == 0 ? a.dwq : a.dwk;
    if (!out) return;
    const int64_t g0 = s.group0[k], groups = s.group0[k + 1] - g0, each = (groups + 15) / 16;
    const int64_t g1 = (run + 1) * each < groups ? (run + 1) * each : groups;
    float v = 0.f;
    if (c < a.d) {
#pragma unroll 8
        for (int64_t g = run * each; g < g1; ++g) v += a.ws[(g0 + g) * a.d + c];
    }
    part[run][lane] = v;
    lds_barrier();
    if (run != 0 || c >= a.d) return;
#pragma unroll
    for (int i = 1; i < 16; ++i) v += part[i][lane];
    out[c] = v;
}

namespace {

// Workgroups of a tensor that keep weight sums, two a CU: 8192 tokens of 32 + 8 bf16 heads of 128, both directions,
// 77.4 us; 1024 of them 82.1, 256 90.7.
constexpr int64_t kMaxGroups = 512;

bool on8(int64_t v) { return (v & 7) == 0; }
bool on16b(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool rows_on8(const void* p, const kda_row_strides& s, int64_t B, int64_t H, int64_t T) {
    return on16b(p) && (B == 1 || on8(s.b)) && (H == 1 || on8(s.h)) && (T == 1 || on8(s.t));
}
bool pages_on8(const void* p, const kda_page_strides& s) { return on16b(p) && on8(s.p) && on8(s.h) && on8(s.t); }

// 16-byte accesses where rows start on them and runs of 8 channels stay whole, else element by element: 8192
// tokens of 32 + 8 heads of 128 34 and 62 us in bf16, 68 and 86 in fp32 (appended with 8 value heads 40 and 72, 56
// and 81).
int layout(const RopeArgs& a, bool wide) {
    // runs of 8 pairs inside the rotated half and inside the rest; interleaved whole pairs of runs
    wide = wide && (a.interleaved ? a.d % 16 == 0 : a.rot % 16 == 0 && (a.d - a.rot) % 16 == 0);
    return (a.interleaved ? kInterWide : kHalfWide) + (wide ? 0 : 2);
}

uint32_t magic(int h) { return h > 1 ? (uint32_t)((((uint64_t)1 << 32) + h - 1) / h) : 0; }

// Tokens of a workgroup: `unroll` passes of its waves (4: rows to ask for ahead), fewer to make 256 workgroups of
// a tensor, or 128 where one pass takes their rows. 1554 tokens of 5 + 1 fp32 heads of 90, both directions: 18.5 us,
// 23 with 256 workgroups throughout, 20.3 with 128, 31 with 512; 32 + 8 bf16 heads of 128: 26.6, 26.7, 27.2, 28.9.
Shape shape(const RopeArgs& a, int unroll, bool append, int64_t most_groups) {
    Shape s{};
    s.lpr = 1;
    while (s.lpr * 16 < a.d) s.lpr *= 2;
    const int64_t all = a.B * a.T, pass = (int64_t)kWaves * (64 / s.lpr) * unroll;
    const int heads[3] = {a.Hq, a.Hk, append ? a.Hk : 0};
    for (int k = 0; k < 3; ++k) {
        int64_t n = 0, groups = 0;
        if (heads[k] && all) {
            n = pass / heads[k];
            const int64_t one = pass / unroll / heads[k], half = all / 128, full = one < half ? one : half;
            const int64_t spread = all / 256 > full ? all / 256 : full, fit = 8192 / a.d;     // 32 KB of angles
            n = n < spread ? n : spread;
            n = n < fit ? n : fit;
            n = n < 1 ? 1 : n > kMaxTokens ? kMaxTokens : n;
            groups = (all + n - 1) / n;
            groups = groups < most_groups ? groups : most_groups;
        }
        s.tokens[k] = (int)n;
        s.group0[k + 1] = s.group0[k] + groups;
        s.magic[k] = magic(heads[k]);
    }
    return s;
}

constexpr int64_t kNoLimit = (int64_t)1 << 40;
// A launch has fewer than 2^32 threads.
bool too_many(const Shape& s) { return s.group0[3] >= (int64_t)1 << 24; }

}  // namespace
}  // namespace rope

size_t rope_bwd_ws_bytes(int64_t tokens, int64_t d) {
    const int64_t g = tokens < rope::kMaxGroups ? tokens : rope::kMaxGroups;
    return (size_t)(g * 2 * d) * 4;
}

hipError_t launch_rope_fwd(const RopeArgs& a, hipStream_t st) {
    using namespace rope;
    const bool wide = (!a.Hq || (rows_on8(a.q, a.sq, a.B, a.Hq, a.T) && rows_on8(a.q_out, a.sqo, a.B, a.Hq, a.T))) &&
                      (!a.Hk || (rows_on8(a.k, a.sk, a.B, a.Hk, a.T) && rows_on8(a.k_out, a.sko, a.B, a.Hk, a.T)));
    const Shape s = shape(a, 4, false, kNoLimit);
    if (too_many(s)) return hipErrorNotSupported;
    const int lay = layout(a, wide);
    return a.in_bf16 ? launch_rows<bf16_t, bf16_t, false>(a, s, lay, st) : launch_rows<float, float, false>(a, s, lay, st);
}

hipError_t launch_rope_append(const RopeArgs& a, hipStream_t st) {
    using namespace rope;
    const bool wide = (!a.Hq || (rows_on8(a.q, a.sq, a.B, a.Hq, a.T) && rows_on8(a.q_out, a.sqo, a.B, a.Hq, a.T))) &&
                      rows_on8(a.k, a.sk, a.B, a.Hk, a.T) && pages_on8(a.k_out, a.skc);
    Shape s = shape(a, 4, true, kNoLimit);
    s.v_wide = a.dv % 8 == 0 && rows_on8(a.v, a.sv, a.B, a.Hk, a.T) && pages_on8(a.v_out, a.svc);
    s.v_lanes = 1;
    while (s.v_lanes < kThreads && s.v_lanes * (s.v_wide ? 8 : 1) < a.dv) s.v_lanes *= 2;
    if (too_many(s)) return hipErrorNotSupported;
    const int lay = layout(a, wide);
    return a.in_bf16 ? launch_rows<bf16_t, bf16_t, true>(a, s, lay, st) : launch_rows<float, bf16_t, true>(a, s, lay, st);
}

hipError_t launch_rope_bwd(const RopeArgs& a, hipStream_t st) {
    using namespace rope;
    const bool sums = a.dwq || a.dwk;
    const bool wide = (!a.Hq || (rows_on8(a.dqo, a.sqo, a.B, a.Hq, a.T) && rows_on8(a.dq, a.sdq, a.B, a.Hq, a.T) &&
                                 (!a.norm || rows_on8(a.q, a.sq, a.B, a.Hq, a.T)))) &&
                      (!a.Hk || (rows_on8(a.dko, a.sko, a.B, a.Hk, a.T) && rows_on8(a.dk, a.sdk, a.B, a.Hk, a.T) &&
                                 (!a.norm || rows_on8(a.k, a.sk, a.B, a.Hk, a.T))));
    const Shape s = shape(a, 4, false, sums ? kMaxGroups : kNoLimit);
    if (too_many(s)) return hipErrorNotSupported;
    if (a.B * a.T > 0) {
        const int lay = layout(a, wide);
        const hipError_t e = a.in_bf16 ? launch_grads<bf16_t>(a, s, lay, sums, st) : launch_grads<float>(a, s, lay, sums, st);
        if (e != hipSuccess) return e;
    }
    if (sums) hipLaunchKernelGGL(rope_colsum_kernel, dim3((unsigned)((a.d + 63) / 64), 2), dim3(1024), 0, st, a, s);
    return hipGetLastError();
}

}  // namespace kda
