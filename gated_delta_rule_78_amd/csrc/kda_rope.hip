// Head norms with rotation and the cache append: which layout and how many tokens a workgroup takes,
// and the weight gradients' last step (include/kda_attn.h).
#include "kda_rope.h"

namespace kda {
namespace rope {

template <typename TI, typename TO, bool APPEND>
hipError_t launch_rows(const RopeArgs& a, const Shape& s, int lay, bool v_wide, hipStream_t st);
template <typename T>
hipError_t launch_grads(const RopeArgs& a, const Shape& s, int lay, int groups, bool sums, hipStream_t st);

// dq_weight and dk_weight from the workgroups' sums [groups][2][d]: 16 runs of workgroups a channel,
// each summed in order by a thread, joined in LDS in order.
__global__ __launch_bounds__(1024) void rope_colsum_kernel(RopeArgs a, int groups) {
    __shared__ float part[16][64];
    const int lane = threadIdx.x & 63, run = threadIdx.x >> 6, k = blockIdx.y;
    const int c = blockIdx.x * 64 + lane;
    float* out = k == 0 ? a.dwq : a.dwk;
    if (!out) return;
    const int each = (groups + 15) / 16, g1 = (run + 1) * each < groups ? (run + 1) * each : groups;
    float s = 0.f;
    if (c < a.d) {
#pragma unroll 8
        for (int g = run * each; g < g1; ++g) s += a.ws[((int64_t)g * 2 + k) * a.d + c];
    }
    part[run][lane] = s;
    lds_barrier();
    if (run != 0 || c >= a.d) return;
#pragma unroll
    for (int i = 1; i < 16; ++i) s += part[i][lane];
    out[c] = s;
}

namespace {

// Workgroups that keep weight sums: 4 a CU.
constexpr int kMaxGroups = 1024;

bool on8(int64_t v) { return (v & 7) == 0; }
bool on16b(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool rows_on8(const kda_row_strides& s, int64_t B) { return (B == 1 || on8(s.b)) && on8(s.h) && on8(s.t); }

int layout(const RopeArgs& a, bool wide) {
    // runs of 8 pairs inside the rotated half and inside the rest; interleaved only whole pairs of runs
    wide = wide && (a.interleaved ? a.d % 16 == 0 : a.rot % 16 == 0 && (a.d - a.rot) % 16 == 0);
    return (a.interleaved ? kInterWide : kHalfWide) + (wide ? 0 : 2);
}

// A launch has fewer than 2^32 threads.
bool too_many(const RopeArgs& a, const Shape& s) { return (a.B * a.T + s.tokens - 1) / s.tokens >= (int64_t)1 << 24; }

uint32_t magic(int h) { return h > 1 ? (uint32_t)((((uint64_t)1 << 32) + h - 1) / h) : 0; }

Shape shape(const RopeArgs& a, int64_t elements) {
    Shape s;
    s.lpr = 1;
    while (s.lpr * 16 < a.d) s.lpr *= 2;
    // tokens a workgroup: about `elements` of work each, fewer where that leaves CUs without a workgroup
    const int64_t row = (int64_t)(a.Hq + a.Hk) * a.d, all = a.B * a.T;
    int64_t n = elements / row, most = all / 512;
    if (n > most) n = most;
    if (n > 8192 / a.d) n = 8192 / a.d;            // 32 KB of angles
    s.tokens = (int)(n < 1 ? 1 : n > kMaxTokens ? kMaxTokens : n);
    s.mq = magic(a.Hq);
    s.mk = magic(a.Hk);
    return s;
}

}  // namespace
}  // namespace rope

size_t rope_bwd_ws_bytes(int64_t tokens, int64_t d) {
    const int64_t g = tokens < rope::kMaxGroups ? tokens : rope::kMaxGroups;
    return (size_t)(g * 2 * d) * 4;
}

hipError_t launch_rope_fwd(const RopeArgs& a, hipStream_t st) {
    using namespace rope;
    const bool wide = (!a.Hq || (on16b(a.q) && on16b(a.q_out) && rows_on8(a.sq, a.B) && rows_on8(a.sqo, a.B))) &&
                      (!a.Hk || (on16b(a.k) && on16b(a.k_out) && rows_on8(a.sk, a.B) && rows_on8(a.sko, a.B)));
    const Shape s = shape(a, 20480);
    if (too_many(a, s)) return hipErrorInvalidConfiguration;
    const int lay = layout(a, wide);
    return a.in_bf16 ? launch_rows<bf16_t, bf16_t, false>(a, s, lay, false, st)
                     : launch_rows<float, float, false>(a, s, lay, false, st);
}

hipError_t launch_rope_append(const RopeArgs& a, hipStream_t st) {
    using namespace rope;
    const bool wide = (!a.Hq || (on16b(a.q) && on16b(a.q_out) && rows_on8(a.sq, a.B) && rows_on8(a.sqo, a.B))) &&
                      on16b(a.k) && on16b(a.k_out) && rows_on8(a.sk, a.B) && on8(a.skc.p) && on8(a.skc.h) && on8(a.skc.t);
    const bool v_wide = a.dv % 8 == 0 && on16b(a.v) && on16b(a.v_out) && rows_on8(a.sv, a.B) && on8(a.svc.p) &&
                        on8(a.svc.h) && on8(a.svc.t);
    const Shape s = shape(a, 20480);
    if (too_many(a, s)) return hipErrorInvalidConfiguration;
    const int lay = layout(a, wide);
    return a.in_bf16 ? launch_rows<bf16_t, bf16_t, true>(a, s, lay, v_wide, st)
                     : launch_rows<float, bf16_t, true>(a, s, lay, v_wide, st);
}

hipError_t launch_rope_bwd(const RopeArgs& a, hipStream_t st) {
    using namespace rope;
    const bool sums = a.dwq || a.dwk;
    const bool wide = (!a.Hq || (on16b(a.dqo) && on16b(a.dq) && rows_on8(a.sqo, a.B) && rows_on8(a.sdq, a.B) &&
                                 (!a.norm || (on16b(a.q) && rows_on8(a.sq, a.B))))) &&
                      (!a.Hk || (on16b(a.dko) && on16b(a.dk) && rows_on8(a.sko, a.B) && rows_on8(a.sdk, a.B) &&
                                 (!a.norm || (on16b(a.k) && rows_on8(a.sk, a.B)))));
    int groups = 0;
    if (a.B * a.T > 0) {
        const Shape s = shape(a, 20480);
        if (too_many(a, s)) return hipErrorInvalidConfiguration;
        const int64_t blocks = (a.B * a.T + s.tokens - 1) / s.tokens;
        groups = (int)(sums && blocks > kMaxGroups ? kMaxGroups : blocks);
        const int lay = layout(a, wide);
        const hipError_t e = a.in_bf16 ? launch_grads<bf16_t>(a, s, lay, groups, sums, st)
                                       : launch_grads<float>(a, s, lay, groups, sums, st);
        if (e != hipSuccess) return e;
    }
    if (sums) hipLaunchKernelGGL(rope_colsum_kernel, dim3((unsigned)((a.d + 63) / 64), 2), dim3(1024), 0, st, a, groups);
    return hipGetLastError();
}

}  // namespace kda
