// Gated linear recurrence for gfx950: workspaces, plans and dispatch.
#include "kda_glr_device.h"
#include "kda_glr_plan.h"
#include "kda_internal.h"

namespace kda {
namespace glr {

// The first sequence that ends behind row (N if none does).
__device__ __forceinline__ int64_t sequence_behind(const GlrArgs& a, int64_t row) {
    int64_t lo = 0, hi = a.N;
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if ((int64_t)a.cu[mid + 1] > row) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// Before a chained or packed launch: the chain's words and counters, the rows where sequences start
// and end, and the states of empty sequences (dst = src or zero).
__global__ __launch_bounds__(256) void glr_prepare_kernel(GlrArgs a, GlrWs ws, const float* src, float* dst) {
    const int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
    if (a.packed) {
        // 32 rows a thread, from sequence to sequence; an empty one (they may be many) is left by search
        for (int64_t i = i0; i < ws.nt * ws.rows / 32; i += step) {
            const int64_t r0 = i * 32, r1 = r0 + 32 < a.T ? r0 + 32 : a.T;
            uint32_t sb = 0, eb = 0;
            int64_t s = r0 < a.T ? sequence_behind(a, r0) : a.N;
            while (s < a.N) {
                const int64_t c0 = a.cu[s], c1 = a.cu[s + 1];
                if (c0 >= r1) break;
                if (c1 <= c0) {
                    const int64_t next = sequence_behind(a, c0);
                    if (next <= s) break;   // lengths out of order
                    s = next;
                    continue;
                }
                if (c0 >= r0) { sb |= 1u << (c0 - r0); ws.start[c0] = (int32_t)s; }
                if (c1 - 1 >= r0 && c1 - 1 < r1) { eb |= 1u << (c1 - 1 - r0); ws.end[c1 - 1] = (int32_t)s; }
                ++s;
            }
            ws.sbits[i] = sb;
            ws.ebits[i] = eb;
        }
        const int64_t per = a.H * a.d;
        for (int64_t i = dst ? i0 : a.N * per; i < a.N * per; i += step) {
            const int64_t s = i / per;
            if (a.cu[s + 1] <= a.cu[s] && src != dst) dst[i] = src ? src[i] : 0.f;
        }
    }
    if (ws.nt <= 1) return;
    for (int64_t i = i0; i < ws.counters; i += step) ws.ticket[i * kCounterStride] = 0;
    const int64_t words = a.blocks * ws.nt * a.d;
    for (int64_t i = i0; i < words; i += step) {
        ws.span[i] = kNone;
        ws.state[i] = kNone;
    }
}

static hipError_t launch_prepare(const GlrArgs& a, const GlrWs& ws, const float* src, float* dst, hipStream_t st) {
    if (ws.nt <= 1 && !a.packed) return hipSuccess;
    int64_t n = ws.nt > 1 ? a.blocks * ws.nt * a.d : 1;
    if (a.packed && ws.nt * ws.rows / 32 > n) n = ws.nt * ws.rows / 32;
    if (a.packed && dst && a.N * a.H * a.d > n) n = a.N * a.H * a.d;
    int64_t grid = (n + 255) / 256;
    if (grid > 2048) grid = 2048;
    hipLaunchKernelGGL(glr_prepare_kernel, dim3((unsigned)grid), dim3(256), 0, st, a, ws, src, dst);
    return hipGetLastError();
}

// dA_log [H,d] from the n parts of a head (one per tile of each of its blocks of rows, [blocks][nt][d]),
// in order: 16 runs of parts a channel, each summed by a thread, joined in LDS. Many parts (N large
// and H small leaves few workgroups) take two launches: workgroup y sums parts [y chunk, (y + 1) chunk)
// into the first of them, then one sums every chunk'th (`last`).
__global__ __launch_bounds__(1024) void glr_dA_kernel(GlrArgs a, GlrWs ws, int64_t n, int64_t chunk, bool last) {
    __shared__ float part[16][64];
    const int lane = threadIdx.x & 63, run = threadIdx.x >> 6;
    const int64_t ntc = (a.d + 63) / 64, head = blockIdx.x / ntc, ch = (int64_t)(blockIdx.x % ntc) * 64 + lane;
    const int64_t k0 = last ? 0 : blockIdx.y * chunk, step = last ? chunk : 1;
    const int64_t left = last ? (n + chunk - 1) / chunk : n - k0, count = last || left < chunk ? left : chunk;
    const int64_t each = (count + 15) / 16;
    auto at = [&](int64_t k) { return ws.dA + ((k / ws.nt * a.H + head) * ws.nt + k % ws.nt) * a.d + ch; };
    float s = 0.f;
    if (ch < a.d) {
        const int64_t i1 = (run + 1) * each < count ? (run + 1) * each : count;
#pragma unroll 8
        for (int64_t i = run * each; i < i1; ++i) s += *at(k0 + i * step);
    }
    part[run][lane] = s;
    __syncthreads();
    if (run == 0 && ch < a.d) {
#pragma unroll
        for (int i = 1; i < 16; ++i) s += part[i][lane];
        if (last) a.dA[head * a.d + ch] = s;
        else *at(k0) = s;
    }
}

static hipError_t launch_dA(const GlrArgs& a, const GlrWs& ws, hipStream_t st) {
    const int64_t n = (a.packed ? 1 : a.N) * ws.nt;
    const unsigned gx = (unsigned)dA_groups(a);
    int64_t chunk = 1;
    if (n > 512) {
        chunk = 256;
        while (chunk * chunk < n) chunk *= 2;
        hipLaunchKernelGGL(glr_dA_kernel, dim3(gx, (unsigned)((n + chunk - 1) / chunk)), dim3(kDAThreads), 0, st, a, ws, n, chunk, false);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(glr_dA_kernel, dim3(gx), dim3(kDAThreads), 0, st, a, ws, n, chunk, true);
    return hipGetLastError();
}

// Workspace in order: counters, marked rows, chain words, dA_log parts.
struct Plan {
    GlrWs ws;
    size_t bytes;
};

static Plan make_plan(const GlrArgs& a, unsigned char* base, bool backward) {
    Plan p{};
    const Tiling t = tiling(a, backward);
    const int64_t rows = t.rows;
    const bool with_dA = backward && a.z;
    p.ws.vec = t.vec;
    p.ws.rows = rows;
    p.ws.nt = t.nt;
    p.ws.narrow = t.narrow;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        unsigned char* r = base ? base + at : nullptr;
        at += (bytes + 255) & ~(size_t)255;
        return r;
    };
    const size_t words = (size_t)(a.blocks * p.ws.nt * a.d);
    const int64_t chains = chain_count(a.blocks, a.d, p.ws.narrow);
    p.ws.counters = chains < (int64_t)kCounters ? chains : (int64_t)kCounters;
    if (p.ws.nt > 1) p.ws.ticket = reinterpret_cast<uint32_t*>(take((size_t)p.ws.counters * kCounterStride * 4));
    if (a.packed) {
        p.ws.sbits = reinterpret_cast<uint32_t*>(take((size_t)(p.ws.nt * rows / 8)));
        p.ws.ebits = reinterpret_cast<uint32_t*>(take((size_t)(p.ws.nt * rows / 8)));
        p.ws.start = reinterpret_cast<int32_t*>(take((size_t)a.T * 4));
        p.ws.end = reinterpret_cast<int32_t*>(take((size_t)a.T * 4));
    }
    if (p.ws.nt > 1) {
        p.ws.span = reinterpret_cast<u64*>(take(words * 8));
        p.ws.state = reinterpret_cast<u64*>(take(words * 8));
    }
    if (with_dA) p.ws.dA = reinterpret_cast<float*>(take(words * 4));
    p.bytes = at;
    return p;
}

template <bool PACKED, typename TIn>
static hipError_t launch_fwd_s(const GlrArgs& a, const GlrWs& ws, hipStream_t st) {
    if (a.scale == KDA_GLR_ONE) return launch_fwd_t<KDA_GLR_ONE, PACKED, TIn>(a, ws, st);
    if (a.scale == KDA_GLR_LEAKY) return launch_fwd_t<KDA_GLR_LEAKY, PACKED, TIn>(a, ws, st);
    return launch_fwd_t<KDA_GLR_NORM, PACKED, TIn>(a, ws, st);
}

static hipError_t launch_fwd_tiles(const GlrArgs& a, const GlrWs& ws, hipStream_t st) {
    const hipError_t e = launch_prepare(a, ws, a.S0, a.S_T, st);
    if (e != hipSuccess) return e;
    if (a.in_bf16) return a.packed ? launch_fwd_s<true, bf16_t>(a, ws, st) : launch_fwd_s<false, bf16_t>(a, ws, st);
    return a.packed ? launch_fwd_s<true, float>(a, ws, st) : launch_fwd_s<false, float>(a, ws, st);
}

template <bool PACKED, typename TIn>
static hipError_t launch_bwd_s(const GlrArgs& a, const GlrWs& ws, hipStream_t st) {
    if (a.scale == KDA_GLR_ONE) return launch_bwd_t<KDA_GLR_ONE, PACKED, TIn>(a, ws, st);
    if (a.scale == KDA_GLR_LEAKY) return launch_bwd_t<KDA_GLR_LEAKY, PACKED, TIn>(a, ws, st);
    return launch_bwd_t<KDA_GLR_NORM, PACKED, TIn>(a, ws, st);
}

static hipError_t launch_bwd_tiles(const GlrArgs& a, const GlrWs& ws, hipStream_t st) {
    const hipError_t e = launch_prepare(a, ws, a.dST, a.dS0, st);
    if (e != hipSuccess) return e;
    if (a.in_bf16) return a.packed ? launch_bwd_s<true, bf16_t>(a, ws, st) : launch_bwd_s<false, bf16_t>(a, ws, st);
    return a.packed ? launch_bwd_s<true, float>(a, ws, st) : launch_bwd_s<false, float>(a, ws, st);
}

}  // namespace glr

size_t glr_fwd_ws_bytes(const GlrArgs& a) { return glr::make_plan(a, nullptr, false).bytes; }

// The backward's own workspace, or, where it runs the forward first, one that holds either's (one
// after the other) with the entry states behind.
size_t glr_bwd_ws_bytes(const GlrArgs& a) {
    const size_t own = glr::make_plan(a, nullptr, true).bytes;
    if (a.entry) return own;
    const size_t fwd = glr::make_plan(a, nullptr, false).bytes;
    return (own > fwd ? own : fwd) + (size_t)(a.blocks * a.nch * a.d) * 4;
}

hipError_t launch_glr_fwd(const GlrArgs& a, hipStream_t st) {
    if (a.T == 0) {   // no tokens: S_T = S0
        if (!a.S_T || a.S_T == a.S0) return hipSuccess;
        return launch_copy_or_zero(a.S_T, a.S0, a.N * a.H * a.d, st);
    }
    if (glr::by_rows(a)) return glr::launch_rows(a, st);
    return glr::launch_fwd_tiles(a, glr::make_plan(a, a.ws, false).ws, st);
}

hipError_t launch_glr_bwd(const GlrArgs& a, hipStream_t st) {
    if (a.T == 0) {   // no tokens: dS0 = dS_T, dA_log = 0
        if (a.dA) {
            const hipError_t e = launch_copy_or_zero(a.dA, nullptr, a.H * a.d, st);
            if (e != hipSuccess) return e;
        }
        return a.dS0 ? launch_copy_or_zero(a.dS0, a.dST, a.N * a.H * a.d, st) : hipSuccess;
    }
    const glr::Plan p = glr::make_plan(a, a.ws, true);
    GlrArgs b = a;
    hipError_t e = hipSuccess;
    if (glr::bwd_by_rows(a)) {
        e = glr::launch_rows_bwd(a, p.ws.dA, st);
    } else {
        if (!b.entry) {   // the forward again, for its entry states alone
            const glr::Plan f = glr::make_plan(a, a.ws, false);
            b.entry = reinterpret_cast<float*>(a.ws + (p.bytes > f.bytes ? p.bytes : f.bytes));
            e = glr::by_rows(b) ? glr::launch_rows(b, st) : glr::launch_fwd_tiles(b, f.ws, st);
            if (e != hipSuccess) return e;
        }
        e = glr::launch_bwd_tiles(b, p.ws, st);
    }
    if (e != hipSuccess || !a.z) return e;
    return glr::launch_dA(a, p.ws, st);
}

// A step is a prefill of one token whose states are read and written in place.
hipError_t launch_glr_step(const GlrArgs& a, hipStream_t st) {
    GlrArgs b = a;
    b.S0 = a.S; b.S_T = a.S;
    return glr::launch_rows(b, st);
}

}  // namespace kda
