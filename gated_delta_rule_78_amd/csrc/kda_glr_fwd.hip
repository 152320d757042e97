// Gated linear recurrence for gfx950, forward (include/kda_glr.h):
//     h_t = alpha_t h_{t-1} + w(alpha_t) i_t x_t,   y_t = h_t.
//
// The operator moves one word in per tensor and one out per element and computes a few dozen
// instructions, so HBM bounds it and every input should be read once. The rows of a block are split
// into tiles: a workgroup holds its tile's decays and inputs in registers, reduces them to the
// tile's span h -> A h + b (a scan over threads, waves and LDS), gets the state before the tile
// from the chain of the tiles before it (kda_glr_device.h), and runs the recurrence again from
// there with the rows still in registers. The chain is waited for once per tile, when the spans of
// the tiles before it, which depend on nothing, are usually there.
#include "kda_glr_device.h"

namespace kda {
namespace glr {

constexpr int kCh = KDA_GLR_CHUNK;

template <int SCALE, bool PACKED, typename TIn, typename TOut, int VEC, int L>
__global__ __launch_bounds__(kThreads) void glr_fwd_kernel(GlrArgs a, GlrWs ws) {
    using G = Tile<VEC>;
    constexpr int CT = G::CT, SPW = G::SPW, W = G::W;
    constexpr int ROWS = kThreads / CT * L;
    static_assert(kCh % L == 0, "a chunk starts at a thread's first row");
    __shared__ float wtA[W][kCW], wth[W][kCW], hin[kCW];
    __shared__ int32_t start[PACKED ? ROWS : 1], end[PACKED ? ROWS : 1];
    __shared__ uint32_t ticket;

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int ct = tid % CT, sub = tid / CT;
    const uint32_t ntc = (uint32_t)((a.d + kCW - 1) / kCW), chains = (uint32_t)a.blocks * ntc;
    const bool chained = ws.nt > 1;
    uint32_t c = blockIdx.x / chains, chain = blockIdx.x % chains;
    if (chained) {
        if (tid == 0) ticket = atomicAdd(ws.ticket + chain % kCounters * kCounterStride, 1u);
        __syncthreads();
        next_tile(__builtin_amdgcn_readfirstlane(ticket), chains, c, chain);
    }
    const int64_t block = chain / ntc;
    const int ch_tile = (int)(chain % ntc) * kCW;
    const int ch0 = ch_tile + ct * VEC;
    const bool on = ch0 < a.d;
    const int64_t row0 = (int64_t)c * ROWS;
    const int rows_here = (int)(a.T - row0 < ROWS ? a.T - row0 : ROWS);
    const uint32_t d = (uint32_t)a.d;
    const int64_t base = (block * a.T + row0) * a.d + ch0;
    const int head = (int)(PACKED ? block : block % a.H);

    RawRow<TIn, VEC> xr[L], dr[L], ur[L];
    const TIn* dec = (const TIn*)(a.z ? a.z : a.la);
    if (on) {
        const uint32_t last = (uint32_t)(rows_here - 1) * d;
#pragma unroll
        for (int r = 0; r < L; ++r) {
            uint32_t off = (uint32_t)(sub * L + r) * d;
            off = off < last ? off : last;
            dr[r] = *reinterpret_cast<const RawRow<TIn, VEC>*>(dec + base + off);
            xr[r] = *reinterpret_cast<const RawRow<TIn, VEC>*>((const TIn*)a.x + base + off);
            if (a.u) ur[r] = *reinterpret_cast<const RawRow<TIn, VEC>*>((const TIn*)a.u + base + off);
        }
    }
    float cz[VEC];
    if (a.z && on) {
        load_f32<VEC>(a.A_log + (int64_t)head * a.d + ch0, cz);
#pragma unroll
        for (int v = 0; v < VEC; ++v) cz[v] = -kLog2e * exp_f(cz[v]);
    }
    int lo = 0, hi = rows_here;     // rows of the tile that are in a sequence
    if constexpr (PACKED) {
        mark_rows<ROWS>(a, row0, ws.seq[c], ws.seq[c + 1], start, end);
        const int64_t c0 = a.cu[0] - row0, c1 = a.cu[a.N] - row0;
        lo = c0 > 0 ? (int)(c0 < ROWS ? c0 : ROWS) : 0;
        hi = c1 < hi ? (int)(c1 > 0 ? c1 : 0) : hi;
    }
    const bool ragged = lo > 0 || hi < ROWS;

    // decays and scaled inputs; the thread's span
    float al[L][VEC], b[L][VEC];
    Span sp[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) sp[v] = Span{1.f, 0.f};
#pragma unroll
    for (int r = 0; r < L; ++r) {
        float x[VEC], q[VEC], g[VEC];
        unpack(xr[r], x);
        unpack(dr[r], q);
        if (a.u) unpack(ur[r], g);
        const int row = sub * L + r;
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            float la = q[v];
            if (a.z) la = a.g_min * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(cz[v] * q[v]));
            al[r][v] = exp_f(la);
            float i = x[v];
            if (a.u) i *= sigmoid_f(g[v]);
            b[r][v] = SCALE == KDA_GLR_ONE ? i : i * scale_w<SCALE>(la, al[r][v]);
        }
        if (ragged && (row < lo || row >= hi)) {   // passes the state on
#pragma unroll
            for (int v = 0; v < VEC; ++v) { al[r][v] = 1.f; b[r][v] = 0.f; }
        }
        if constexpr (PACKED) {
            const int s = start[row];
            if (s >= 0 && on) {   // a sequence starts: its S0 becomes part of b, the state before is cut off
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    if (a.S0) b[r][v] = fmaf(al[r][v], a.S0[((int64_t)s * a.H + head) * a.d + ch0 + v], b[r][v]);
                    al[r][v] = -1.f;
                }
            }
        }
#pragma unroll
        for (int v = 0; v < VEC; ++v) sp[v] = compose<PACKED>(sp[v], Span{al[r][v], b[r][v]});
    }

    // spans over the sub-chunks of the wave (inclusive), then over the waves
#pragma unroll
    for (int m = 1; m < SPW; m <<= 1) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const Span l{__shfl_up(sp[v].A, m * CT), __shfl_up(sp[v].h, m * CT)};
            const Span o = compose<PACKED>(l, sp[v]);
            if (lane >= m * CT) sp[v] = o;
        }
    }
    if (lane >= 64 - CT) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) { wtA[wave][ct * VEC + v] = sp[v].A; wth[wave][ct * VEC + v] = sp[v].h; }
    }
    __syncthreads();
    if (wave == 0) {   // lane = channel: the tile's span, the chain
        const int ch = ch_tile + lane;
        Span tot{wtA[0][lane], wth[0][lane]};
#pragma unroll
        for (int w = 1; w < W; ++w) tot = compose<PACKED>(tot, Span{wtA[w][lane], wth[w][lane]});
        float h = 0.f;
        if (ch < a.d) {
            if (!PACKED && c == 0 && a.S0) h = a.S0[block * a.d + ch];
            if (chained) {
                const int64_t word = (block * ws.nt + c) * a.d + ch;
                const bool more = (int64_t)c + 1 < ws.nt;
                const bool cut = PACKED && __float_as_int(tot.A) < 0;
                if (cut && more) publish(ws.state + word, 0, tot.h);
                if (c > 0) {
                    if (!cut && more) publish_span(ws.span + word, tot);
                    h = look_back<PACKED>(ws.span + word, ws.state + word, a.d, c);
                }
                if (!cut && more) publish(ws.state + word, 0, apply<PACKED>(tot, h));
            }
        }
        hin[lane] = h;
    }
    __syncthreads();
    if (!on) return;

    // the state before the thread's first row
    float h[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) h[v] = hin[ct * VEC + v];
#pragma unroll
    for (int w = 0; w < W - 1; ++w)
        if (w < wave) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) h[v] = apply<PACKED>(Span{wtA[w][ct * VEC + v], wth[w][ct * VEC + v]}, h[v]);
        }
    if constexpr (SPW > 1) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const Span l{__shfl_up(sp[v].A, CT), __shfl_up(sp[v].h, CT)};
            const float hl = apply<PACKED>(l, h[v]);
            if (lane >= CT) h[v] = hl;
        }
    }
    if (a.entry && (sub * L) % kCh == 0 && sub * L < rows_here) {
        float* e = a.entry + (block * a.nch + (row0 + sub * L) / kCh) * a.d + ch0;
#pragma unroll
        for (int v = 0; v < VEC; ++v) e[v] = h[v];
    }
    TOut* y = (TOut*)a.y + base;
#pragma unroll
    for (int r = 0; r < L; ++r) {
        const int row = sub * L + r;
#pragma unroll
        for (int v = 0; v < VEC; ++v) h[v] = apply<PACKED>(Span{al[r][v], b[r][v]}, h[v]);
        if (row >= lo && row < hi && a.y) store_row<VEC>(y + (uint32_t)row * d, h);
        if constexpr (PACKED) {
            const int s = end[row];
            if (s >= 0 && a.S_T) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) a.S_T[((int64_t)s * a.H + head) * a.d + ch0 + v] = h[v];
            }
        } else {
            if (row0 + row == a.T - 1 && a.S_T) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) a.S_T[block * a.d + ch0 + v] = h[v];
            }
        }
    }
}

// Before a chained or packed launch: the chain's words and counter, the first sequence of every
// tile, and the states of empty sequences (dst = src or zero).
__global__ __launch_bounds__(256) void glr_prepare_kernel(GlrArgs a, GlrWs ws, const float* src, float* dst) {
    const int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
    if (ws.nt > 1) {
        for (int64_t i = i0; i < ws.counters; i += step) ws.ticket[i * kCounterStride] = 0;
        const int64_t words = a.blocks * ws.nt * a.d;
        for (int64_t i = i0; i < words; i += step) {
            ws.span[i] = kNone;
            ws.state[i] = kNone;
        }
    }
    if (!a.packed) return;
    for (int64_t i = i0; i <= ws.nt; i += step) {
        int64_t lo = 0, hi = a.N;   // the first sequence that ends behind the tile's first row
        if (i == ws.nt) lo = a.N;
        while (lo < hi) {
            const int64_t mid = (lo + hi) >> 1;
            if ((int64_t)a.cu[mid + 1] > i * ws.rows) hi = mid;
            else lo = mid + 1;
        }
        ws.seq[i] = (int32_t)lo;
    }
    if (!dst) return;
    const int64_t per = a.H * a.d;
    for (int64_t i = i0; i < a.N * per; i += step) {
        const int64_t s = i / per;
        if (a.cu[s + 1] <= a.cu[s] && (!src || src != dst)) dst[i] = src ? src[i] : 0.f;
    }
}

hipError_t launch_prepare(const GlrArgs& a, const GlrWs& ws, const float* src, float* dst, hipStream_t st) {
    if (ws.nt <= 1 && !a.packed) return hipSuccess;
    int64_t n = ws.nt > 1 ? a.blocks * ws.nt * a.d : 1;
    if (a.packed && ws.nt + 1 > n) n = ws.nt + 1;
    if (a.packed && dst && a.N * a.H * a.d > n) n = a.N * a.H * a.d;
    int64_t grid = (n + 255) / 256;
    if (grid > 2048) grid = 2048;
    hipLaunchKernelGGL(glr_prepare_kernel, dim3((unsigned)grid), dim3(256), 0, st, a, ws, src, dst);
    return hipGetLastError();
}

// 4 channels a thread where every row of every tensor starts on 4 elements, else 1. Rows a thread
// are chosen so that a tile has kCh rows either way.
template <int SCALE, bool PACKED, typename TIn, typename TOut>
static hipError_t launch_fwd_t(const GlrArgs& a, const GlrWs& ws, hipStream_t st) {
    const int64_t ntc = (a.d + kCW - 1) / kCW;
    const dim3 grid((unsigned)(a.blocks * ntc * ws.nt));
    if (ws.vec == 4)
        hipLaunchKernelGGL((glr_fwd_kernel<SCALE, PACKED, TIn, TOut, 4, kCh * 16 / kThreads>), grid, dim3(kThreads), 0, st, a, ws);
    else
        hipLaunchKernelGGL((glr_fwd_kernel<SCALE, PACKED, TIn, TOut, 1, kCh * 64 / kThreads>), grid, dim3(kThreads), 0, st, a, ws);
    return hipGetLastError();
}

template <int SCALE, bool PACKED>
static hipError_t launch_fwd_s(const GlrArgs& a, const GlrWs& ws, hipStream_t st) {
    if (a.in_bf16 && a.out_bf16) return launch_fwd_t<SCALE, PACKED, bf16_t, bf16_t>(a, ws, st);
    if (a.in_bf16) return launch_fwd_t<SCALE, PACKED, bf16_t, float>(a, ws, st);
    if (a.out_bf16) return launch_fwd_t<SCALE, PACKED, float, bf16_t>(a, ws, st);
    return launch_fwd_t<SCALE, PACKED, float, float>(a, ws, st);
}

hipError_t launch_fwd_tiles(const GlrArgs& a, const GlrWs& ws, hipStream_t st) {
    const hipError_t e = launch_prepare(a, ws, a.S0, a.S_T, st);
    if (e != hipSuccess) return e;
    if (a.packed) {
        if (a.scale == KDA_GLR_ONE) return launch_fwd_s<KDA_GLR_ONE, true>(a, ws, st);
        if (a.scale == KDA_GLR_LEAKY) return launch_fwd_s<KDA_GLR_LEAKY, true>(a, ws, st);
        return launch_fwd_s<KDA_GLR_NORM, true>(a, ws, st);
    }
    if (a.scale == KDA_GLR_ONE) return launch_fwd_s<KDA_GLR_ONE, false>(a, ws, st);
    if (a.scale == KDA_GLR_LEAKY) return launch_fwd_s<KDA_GLR_LEAKY, false>(a, ws, st);
    return launch_fwd_s<KDA_GLR_NORM, false>(a, ws, st);
}

}  // namespace glr
}  // namespace kda
