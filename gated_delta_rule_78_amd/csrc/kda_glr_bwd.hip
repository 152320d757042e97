// Gated linear recurrence for gfx950, backward (include/kda_glr.h). With g_t = dL/dh_t:
//     g_t = dy_t + alpha_{t+1} g_{t+1}  (dS_T in place of the carry at a sequence's last row),
//     dx_t = g_t w_t i_t,  din_gate_t = g_t w_t x_t i_t (1 - i_t),
//     dlog_alpha_t = g_t (alpha_t h_{t-1} + w'_t i_t x_t),
//     dz_t = dlog_alpha_t log_alpha_t e^A (1 - s_t),  dA_log = sum_t dz_t z_t,  dS0 = alpha_1 g_1.
//
// The tiles, their chain and their bound are the forward's, the chain run from the last tile to the
// first with spans g -> A g + b; the states h_{t-1} are run again inside the tile from the entry
// state that the forward stored, so that every tensor is read once here too.
#include "kda_glr_device.h"

namespace kda {
namespace glr {

constexpr int kCh = KDA_GLR_CHUNK;

template <int SCALE, bool PACKED, typename TIn, typename TOut, int VEC, int L>
__global__ __launch_bounds__(kThreads) void glr_bwd_kernel(GlrArgs a, GlrWs ws) {
    using G = Tile<VEC>;
    constexpr int CT = G::CT, SPW = G::SPW, W = G::W;
    constexpr int ROWS = kThreads / CT * L;
    static_assert(ROWS == kCh, "a tile starts at an entry state");
    __shared__ float wtA[W][kCW], wth[W][kCW], wtg[W][kCW], wtR[W][kCW], gin[kCW];
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
    c = (uint32_t)ws.nt - 1 - c;   // the last tile first
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
    RawRow<TOut, VEC> yr[L];
    const TIn* dec = (const TIn*)(a.z ? a.z : a.la);
    float hin[VEC];
    if (on) {
        const uint32_t last = (uint32_t)(rows_here - 1) * d;
#pragma unroll
        for (int r = 0; r < L; ++r) {
            uint32_t off = (uint32_t)(sub * L + r) * d;
            off = off < last ? off : last;
            dr[r] = *reinterpret_cast<const RawRow<TIn, VEC>*>(dec + base + off);
            yr[r] = *reinterpret_cast<const RawRow<TOut, VEC>*>((const TOut*)a.dy + base + off);
            xr[r] = *reinterpret_cast<const RawRow<TIn, VEC>*>((const TIn*)a.x + base + off);
            if (a.u) ur[r] = *reinterpret_cast<const RawRow<TIn, VEC>*>((const TIn*)a.u + base + off);
        }
        load_f32<VEC>(a.entry + (block * a.nch + c) * a.d + ch0, hin);
    }
    float eA[VEC];
    if (a.z && on) {
        load_f32<VEC>(a.A_log + (int64_t)head * a.d + ch0, eA);
#pragma unroll
        for (int v = 0; v < VEC; ++v) eA[v] = exp_f(eA[v]);
    }
    int lo = 0, hi = rows_here;
    if constexpr (PACKED) {
        mark_rows<ROWS>(a, row0, ws.seq[c], ws.seq[c + 1], start, end);
        const int64_t c0 = a.cu[0] - row0, c1 = a.cu[a.N] - row0;
        lo = c0 > 0 ? (int)(c0 < ROWS ? c0 : ROWS) : 0;
        hi = c1 < hi ? (int)(c1 > 0 ? c1 : 0) : hi;
    }
    const bool ragged = lo > 0 || hi < ROWS;

    // decays, scaled inputs and output gradients; the thread's spans in both directions
    float al[L][VEC], b[L][VEC], dy[L][VEC];
    Span sf[VEC], sr[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) sf[v] = Span{1.f, 0.f};
#pragma unroll
    for (int r = 0; r < L; ++r) {
        float x[VEC], q[VEC], g[VEC];
        unpack(xr[r], x);
        unpack(dr[r], q);
        unpack(yr[r], dy[r]);
        if (a.u) unpack(ur[r], g);
        const int row = sub * L + r;
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            float la = q[v];
            if (a.z) la = a.g_min * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * eA[v] * q[v]));
            al[r][v] = exp_f(la);
            float i = x[v];
            if (a.u) i *= sigmoid_f(g[v]);
            b[r][v] = SCALE == KDA_GLR_ONE ? i : i * scale_w<SCALE>(la, al[r][v]);
        }
        if (ragged && (row < lo || row >= hi)) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) { al[r][v] = 1.f; b[r][v] = 0.f; dy[r][v] = 0.f; }
        }
        Span f[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) f[v] = Span{al[r][v], b[r][v]};
        if constexpr (PACKED) {
            const int s = start[row], e = end[row];
            if (s >= 0 && on) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    if (a.S0) f[v].h = b[r][v] = fmaf(al[r][v], a.S0[((int64_t)s * a.H + head) * a.d + ch0 + v], b[r][v]);
                    f[v].A = -1.f;
                }
            }
            if (e >= 0 && on && a.dST) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) dy[r][v] += a.dST[((int64_t)e * a.H + head) * a.d + ch0 + v];
            }
        }
#pragma unroll
        for (int v = 0; v < VEC; ++v) sf[v] = compose<PACKED>(sf[v], f[v]);
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) sr[v] = Span{1.f, 0.f};
#pragma unroll
    for (int r = L - 1; r >= 0; --r) {
        const bool cut = PACKED && end[sub * L + r] >= 0;
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            // the row maps the carry g behind it to alpha (dy + g)
            const Span s{cut ? -1.f : al[r][v], al[r][v] * dy[r][v]};
            sr[v] = compose<PACKED>(sr[v], s);
        }
    }

    // forward spans up to the thread, reverse spans behind it: within the wave, then over the waves
#pragma unroll
    for (int m = 1; m < SPW; m <<= 1) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const Span l{__shfl_up(sf[v].A, m * CT), __shfl_up(sf[v].h, m * CT)};
            const Span o = compose<PACKED>(l, sf[v]);
            const Span rl{__shfl_down(sr[v].A, m * CT), __shfl_down(sr[v].h, m * CT)};
            const Span ro = compose<PACKED>(rl, sr[v]);
            if (lane >= m * CT) sf[v] = o;
            if (lane < 64 - m * CT) sr[v] = ro;
        }
    }
    if (lane >= 64 - CT) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) { wtA[wave][ct * VEC + v] = sf[v].A; wth[wave][ct * VEC + v] = sf[v].h; }
    }
    if (lane < CT) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) { wtR[wave][ct * VEC + v] = sr[v].A; wtg[wave][ct * VEC + v] = sr[v].h; }
    }
    __syncthreads();
    if (wave == 0) {   // lane = channel: the tile's reverse span, the chain
        const int ch = ch_tile + lane;
        Span tot{wtR[W - 1][lane], wtg[W - 1][lane]};
#pragma unroll
        for (int w = W - 2; w >= 0; --w) tot = compose<PACKED>(tot, Span{wtR[w][lane], wtg[w][lane]});
        float g = 0.f;
        if (ch < a.d) {
            const bool first = (int64_t)c + 1 == ws.nt;
            if (!PACKED && first && a.dST) g = a.dST[block * a.d + ch];
            const bool cut = PACKED && __float_as_int(tot.A) < 0;
            if (chained) {
                const int64_t word = (block * ws.nt + c) * a.d + ch;
                const bool more = c > 0;
                if (cut && more) publish(ws.state + word, 0, tot.h);
                if (!first) {
                    if (!cut && more) publish_span(ws.span + word, tot);
                    g = look_back<PACKED>(ws.span + word, ws.state + word, -a.d, ws.nt - 1 - c);
                }
                if (!cut && more) publish(ws.state + word, 0, apply<PACKED>(tot, g));
            }
            if (!PACKED && c == 0 && a.dS0) a.dS0[block * a.d + ch] = apply<PACKED>(tot, g);
        }
        gin[lane] = g;
    }
    __syncthreads();

    float dA[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) dA[v] = 0.f;
    if (on) {
        // the state before the thread's rows and the carry behind them
        float h[VEC], g[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) { h[v] = hin[v]; g[v] = gin[ct * VEC + v]; }
#pragma unroll
        for (int w = 0; w < W - 1; ++w)
            if (w < wave) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) h[v] = apply<PACKED>(Span{wtA[w][ct * VEC + v], wth[w][ct * VEC + v]}, h[v]);
            }
#pragma unroll
        for (int w = W - 1; w > 0; --w)
            if (w > wave) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) g[v] = apply<PACKED>(Span{wtR[w][ct * VEC + v], wtg[w][ct * VEC + v]}, g[v]);
            }
        if constexpr (SPW > 1) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const Span l{__shfl_up(sf[v].A, CT), __shfl_up(sf[v].h, CT)};
                const Span rl{__shfl_down(sr[v].A, CT), __shfl_down(sr[v].h, CT)};
                const float hl = apply<PACKED>(l, h[v]), gl = apply<PACKED>(rl, g[v]);
                if (lane >= CT) h[v] = hl;
                if (lane < 64 - CT) g[v] = gl;
            }
        }
        // the states before each row, in place of b
#pragma unroll
        for (int r = 0; r < L; ++r) {
            const bool cut = PACKED && start[sub * L + r] >= 0;
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float hn = cut ? b[r][v] : fmaf(al[r][v], h[v], b[r][v]);
                b[r][v] = h[v];
                h[v] = hn;
            }
            if constexpr (PACKED) {
                if (cut) {
                    const int s = start[sub * L + r];
#pragma unroll
                    for (int v = 0; v < VEC; ++v) b[r][v] = a.S0 ? a.S0[((int64_t)s * a.H + head) * a.d + ch0 + v] : 0.f;
                }
            }
        }
        TIn *dx = (TIn*)a.dx + base, *dd = (TIn*)a.dd + base, *du = (TIn*)a.du + base;
#pragma unroll
        for (int r = L - 1; r >= 0; --r) {
            const int row = sub * L + r;
            const uint32_t off = (uint32_t)row * d;
            float x[VEC], q[VEC], u[VEC], ox[VEC], od[VEC], ou[VEC];
            unpack(xr[r], x);
            unpack(dr[r], q);
            if (a.u) unpack(ur[r], u);
            const bool live = row >= lo && row < hi;
            if constexpr (PACKED)
                if (end[row] >= 0) {
#pragma unroll
                    for (int v = 0; v < VEC; ++v) g[v] = 0.f;
                }
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float al_ = al[r][v];
                float la = q[v], s = 0.f, w, dw;
                if (a.z) {
                    s = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * eA[v] * q[v]));
                    la = a.g_min * s;
                }
                scale_w_dw<SCALE>(la, al_, w, dw);
                const float i = a.u ? sigmoid_f(u[v]) : 1.f;
                const float gr = g[v] + dy[r][v];
                ox[v] = gr * w * i;
                ou[v] = ox[v] * (1.f - i) * x[v];
                float e = al_ * b[r][v];
                if (SCALE != KDA_GLR_ONE) e = fmaf(dw, i * x[v], e);
                e *= gr;
                if (a.z) {
                    e *= la * (1.f - s) * eA[v];
                    if (live) dA[v] = fmaf(e, q[v], dA[v]);
                }
                od[v] = e;
                g[v] = al_ * gr;
            }
            if (live) {
                store_row<VEC>(dx + off, ox);
                store_row<VEC>(dd + off, od);
                if (a.u) store_row<VEC>(du + off, ou);
            }
            if constexpr (PACKED) {
                const int s = start[row];
                if (s >= 0 && a.dS0) {
#pragma unroll
                    for (int v = 0; v < VEC; ++v) a.dS0[((int64_t)s * a.H + head) * a.d + ch0 + v] = g[v];
                }
            }
        }
    }
    if (!a.z) return;
    // the tile's part of dA_log: over the sub-chunks of the wave, then the waves
#pragma unroll
    for (int m = CT; m < 64; m <<= 1)
#pragma unroll
        for (int v = 0; v < VEC; ++v) dA[v] += __shfl_xor(dA[v], m);
    __syncthreads();
    if (lane < CT) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) wth[wave][ct * VEC + v] = dA[v];
    }
    __syncthreads();
    if (wave == 0 && ch_tile + lane < a.d) {
        float s = wth[0][lane];
#pragma unroll
        for (int w = 1; w < W; ++w) s += wth[w][lane];
        ws.dA[(block * ws.nt + c) * a.d + ch_tile + lane] = s;
    }
}

// dA_log [H,d] from the tiles' parts [blocks][nt][d], in order: 16 groups of tiles a channel, each
// summed by a thread, joined in LDS.
__global__ __launch_bounds__(1024) void glr_dA_kernel(GlrArgs a, GlrWs ws) {
    __shared__ float part[16][64];
    const int lane = threadIdx.x & 63, grp = threadIdx.x >> 6;
    const int64_t ch = (int64_t)blockIdx.x * 64 + lane, head = blockIdx.y;
    const int64_t per = a.packed ? 1 : a.N, n = per * ws.nt, each = (n + 15) / 16;
    float s = 0.f;
    if (ch < a.d) {
        const int64_t k1 = (grp + 1) * each < n ? (grp + 1) * each : n;
#pragma unroll 8
        for (int64_t k = grp * each; k < k1; ++k) {
            const int64_t block = (k / ws.nt) * a.H + head, c = k % ws.nt;
            s += ws.dA[(block * ws.nt + c) * a.d + ch];
        }
    }
    part[grp][lane] = s;
    __syncthreads();
    if (grp == 0 && ch < a.d) {
#pragma unroll
        for (int i = 1; i < 16; ++i) s += part[i][lane];
        a.dA[head * a.d + ch] = s;
    }
}

template <int SCALE, bool PACKED, typename TIn, typename TOut>
static hipError_t launch_bwd_t(const GlrArgs& a, const GlrWs& ws, hipStream_t st) {
    const int64_t ntc = (a.d + kCW - 1) / kCW;
    const dim3 grid((unsigned)(a.blocks * ntc * ws.nt));
    if (ws.vec == 4)
        hipLaunchKernelGGL((glr_bwd_kernel<SCALE, PACKED, TIn, TOut, 4, kCh * 16 / kThreads>), grid, dim3(kThreads), 0, st, a, ws);
    else
        hipLaunchKernelGGL((glr_bwd_kernel<SCALE, PACKED, TIn, TOut, 1, kCh * 64 / kThreads>), grid, dim3(kThreads), 0, st, a, ws);
    return hipGetLastError();
}

template <int SCALE, bool PACKED>
static hipError_t launch_bwd_s(const GlrArgs& a, const GlrWs& ws, hipStream_t st) {
    if (a.in_bf16 && a.out_bf16) return launch_bwd_t<SCALE, PACKED, bf16_t, bf16_t>(a, ws, st);
    if (a.in_bf16) return launch_bwd_t<SCALE, PACKED, bf16_t, float>(a, ws, st);
    if (a.out_bf16) return launch_bwd_t<SCALE, PACKED, float, bf16_t>(a, ws, st);
    return launch_bwd_t<SCALE, PACKED, float, float>(a, ws, st);
}

hipError_t launch_bwd_tiles(const GlrArgs& a, const GlrWs& ws, hipStream_t st) {
    hipError_t e = launch_prepare(a, ws, a.dST, a.dS0, st);
    if (e != hipSuccess) return e;
    if (a.packed) {
        if (a.scale == KDA_GLR_ONE) e = launch_bwd_s<KDA_GLR_ONE, true>(a, ws, st);
        else if (a.scale == KDA_GLR_LEAKY) e = launch_bwd_s<KDA_GLR_LEAKY, true>(a, ws, st);
        else e = launch_bwd_s<KDA_GLR_NORM, true>(a, ws, st);
    } else {
        if (a.scale == KDA_GLR_ONE) e = launch_bwd_s<KDA_GLR_ONE, false>(a, ws, st);
        else if (a.scale == KDA_GLR_LEAKY) e = launch_bwd_s<KDA_GLR_LEAKY, false>(a, ws, st);
        else e = launch_bwd_s<KDA_GLR_NORM, false>(a, ws, st);
    }
    if (e != hipSuccess || !a.z) return e;
    hipLaunchKernelGGL(glr_dA_kernel, dim3((unsigned)((a.d + 63) / 64), (unsigned)a.H), dim3(1024), 0, st, a, ws);
    return hipGetLastError();
}

}  // namespace glr
}  // namespace kda
