// Gated linear recurrence for gfx950, backward (include/kda_glr.h). With g_t = dL/dh_t:
//     g_t = dy_t + alpha_{t+1} g_{t+1}  (dS_T in place of the carry at a sequence's last row),
//     dx_t = g_t w_t i_t,  din_gate_t = g_t w_t x_t i_t (1 - i_t),
//     dlog_alpha_t = g_t (alpha_t h_{t-1} + w'_t i_t x_t),
//     dz_t = dlog_alpha_t log_alpha_t e^A (1 - s_t),  dA_log = sum_t dz_t z_t,  dS0 = alpha_1 g_1.
//
// The tiles, their chain and their bound are the forward's (kda_glr_fwd.h), the chain run from the
// last tile to the first with spans g -> A g + b; the states h_{t-1} are run again inside the tile
// from the entry state that the forward stored, so that every tensor is read once here too (fp32
// rows without z: dy twice). Between the passes over the rows the gates stay in registers (computing
// them twice costs more issue slots than the memory leaves free) and x, z and dy wait in LDS as they
// were read: 128 registers a thread hold no more, and 168 would leave one workgroup a CU (no LDS:
// 270 us for both directions of the shape below, against 200; 256 threads of 8 rows: 211 against 202).
//
// Measured, bf16 with both gates and w = sqrt(1 - alpha^2): 2 x 4096 rows of 4096 channels 122 us for
// 470 MB read and written, 3.8 TB/s; its issue slots (85 an element, 60 % of the SIMDs' by counters) and
// the latency of a tile's start, with two workgroups a CU, share the bound. Packed batches spill there
// (24 registers a thread): 12 sequences, 32 x 8192 rows of 128 channels, take 191 us.
#pragma once

#include "kda_glr_device.h"
#include "kda_glr_plan.h"

namespace kda {
namespace glr {

// Workgroups a CU: two with 48 KiB of rows in LDS, which hold all of a bf16 tile and x of an fp32
// one (dy and z are read again); or one, with the registers and the LDS for everything, where fp32
// rows come with z (2 x 4096 rows of 4096 fp32 channels, both gates: 225 us against 257, and 294
// with two and nothing in LDS; without z two win, 145 against 154).
template <int Z, typename TIn, int VEC>
constexpr int groups_a_cu() {
    return sizeof(TIn) == 4 && (Z != 0 || VEC == 1) ? 1 : 2;
}

template <int SCALE, bool PACKED, bool NARROW, int Z, int U, typename TIn, typename TOut, int VEC, int L, int THREADS>
__global__ __launch_bounds__(THREADS, (2 * groups_a_cu<Z, TIn, VEC>())) void glr_bwd_kernel(GlrArgs a, GlrWs ws) {
    using G = Tile<VEC, L, THREADS>;
    constexpr int CT = G::CT, SPW = G::SPW, W = G::W, ROWS = G::ROWS;
    static_assert(ROWS == KDA_GLR_CHUNK, "a tile starts at an entry state");
    __shared__ float wtA[W][kCW], wth[W][kCW], wtg[W][kCW], wtR[W][kCW], gin[kCW];
    __shared__ __align__(16) float turn[W][SPW > 1 ? 2 * SPW * kCW : 1];
    // the rows in LDS: x, then dy, then z, as far as they fit
    constexpr int kStash = (groups_a_cu<Z, TIn, VEC>() == 1 ? 96 : 48) << 10, XB = THREADS * L * VEC * (int)sizeof(TIn), YB = THREADS * L * VEC * (int)sizeof(TOut);
    constexpr bool SX = XB <= kStash, SY = XB + YB <= kStash, SZ = Z != 0 && 2 * XB + (SY ? YB : 0) <= kStash;
    __shared__ RawRow<TIn, VEC> xs[SX ? L : 1][THREADS], zs[SZ ? L : 1][THREADS];
    __shared__ RawRow<TOut, VEC> ys[SY ? L : 1][THREADS];
    __shared__ uint32_t ticket;
    const bool has_z = Z == 2 ? a.z != nullptr : Z == 1, has_u = U == 2 ? a.u != nullptr : U == 1;

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int ct = tid % CT, sub = tid / CT, row_t = sub * L;
    const uint32_t ntc = NARROW ? 1 : (uint32_t)((a.d + kCW - 1) / kCW), per = NARROW ? heads_a_tile(a.d) : 1;
    const uint32_t chains = (uint32_t)chain_count(a.blocks, a.d, NARROW);
    const bool chained = ws.nt > 1;
    uint32_t c = blockIdx.x / chains, chain = chain_of(blockIdx.x % chains, chains);
    if (chained) {
        if (tid == 0) ticket = atomicAdd(ws.ticket + chain % kCounters * kCounterStride, 1u);
        lds_barrier();
        next_tile(__builtin_amdgcn_readfirstlane(ticket), chains, c, chain);
    }
    c = (uint32_t)ws.nt - 1 - c;   // the last tile first
    const int64_t block0 = (int64_t)(chain / ntc) * per;   // the tile's first block of rows
    const uint32_t tile = chain % ntc;                      // across the head's channels
    const uint32_t d = (uint32_t)a.d;
    const Place<NARROW, VEC> at(ct * VEC, tile, d, a.blocks - block0);
    const bool on = at.on;
    const uint32_t ch0 = at.ch;
    const int64_t block = block0 + at.local;
    // as a lane of one channel: the block, the channel, and whether there is one
    const Place<NARROW, VEC> own(lane / VEC * VEC, tile, d, a.blocks - block0);
    const bool has_ch = own.on;
    const int64_t block_l = block0 + own.local;
    const uint32_t ch = own.ch + lane % VEC;
    const int64_t row0 = (int64_t)c * ROWS;
    const int rows_here = (int)(a.T - row0 < ROWS ? a.T - row0 : ROWS);
    const int64_t base = (block0 * a.T + row0) * a.d;
    const int head = (int)(PACKED ? block : block % a.H);

    int lo = 0, hi = rows_here;     // rows of the tile that are in a sequence
    uint32_t sbits = 0, ebits = 0;  // the thread's rows where one starts or ends
    if constexpr (PACKED) {
        sbits = bits_at<L>(ws.sbits, row0 + row_t);
        ebits = bits_at<L>(ws.ebits, row0 + row_t);
        live_rows(a, row0, ROWS, lo, hi);
    }
    // (narrow heads: a tile's blocks lie within 2^31 elements)
    const uint32_t in_tile = (NARROW ? at.local * (uint32_t)(a.T * a.d) : 0) + ch0;
    const uint32_t off0 = (uint32_t)row_t * d + in_tile, last_off = (uint32_t)(rows_here - 1) * d + in_tile;
    const TIn* dec = (const TIn*)(has_z ? a.z : a.la) + base;
    const TIn* xp = (const TIn*)a.x + base;
    const TIn* up = (const TIn*)a.u + base;
    const TOut* yp = (const TOut*)a.dy + base;

    // decays and gates; the thread's spans, forwards (state) and backwards (a row maps the carry g to
    // alpha (dy + g)), rows from the last to the first
    float al[L][VEC], w[L][VEC], gi[L][VEC], s[L][VEC];
    Span sf[VEC], sr[VEC];
    const bool plain = !PACKED || (sbits | ebits) == 0;
    {
        RawRow<TIn, VEC> xr[L], dr[L], ur[L];
        RawRow<TOut, VEC> yr[L];
#pragma unroll
        for (int r = 0; r < L; ++r) {
            const uint32_t off = row_offset(off0, r, d, last_off);
            dr[r] = load_row<TIn, VEC>(dec + off);
            xr[r] = load_row<TIn, VEC>(xp + off);
            if (has_u) ur[r] = load_row<TIn, VEC>(up + off);
            yr[r] = load_row<TOut, VEC>(yp + off);
        }
        const float gy = a.g_min * kLog2e;
        float cz[VEC];
        if (has_z) {
            load_f32<VEC>(a.A_log + (int64_t)head * a.d + ch0, cz);
#pragma unroll
            for (int v = 0; v < VEC; ++v) cz[v] = -kLog2e * exp_f(cz[v]);
        }
#pragma unroll
        for (int v = 0; v < VEC; ++v) sf[v] = sr[v] = Span{1.f, 0.f};
#pragma unroll
        for (int r = L - 1; r >= 0; --r) {
            float x[VEC], q[VEC], u[VEC], dy[VEC], b[VEC];
            unpack(xr[r], x);
            unpack(dr[r], q);
            unpack(yr[r], dy);
            if (has_u) unpack(ur[r], u);
            if constexpr (SX) xs[r][tid] = xr[r];
            if constexpr (SZ) zs[r][tid] = dr[r];
            if constexpr (SY) ys[r][tid] = yr[r];
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                float y;
                if (has_z) {
                    s[r][v] = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(cz[v] * q[v]));
                    y = gy * s[r][v];
                } else {
                    y = q[v] * kLog2e;
                }
                al[r][v] = __builtin_amdgcn_exp2f(y);
                b[v] = x[v];
                if (has_u) {
                    gi[r][v] = sigmoid_f(u[v]);
                    b[v] *= gi[r][v];
                }
                if (SCALE != KDA_GLR_ONE) {
                    w[r][v] = scale_w<SCALE>(y, al[r][v]);
                    b[v] *= w[r][v];
                }
            }
            if (row_t + r < lo || row_t + r >= hi) {   // rows in no sequence pass state and carry on
#pragma unroll
                for (int v = 0; v < VEC; ++v) { al[r][v] = 1.f; b[v] = 0.f; dy[v] = 0.f; }
            }
            if (plain) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    sf[v].h = fmaf(sf[v].A, b[v], sf[v].h);
                    sf[v].A *= al[r][v];
                    sr[v].h = al[r][v] * (dy[v] + sr[v].h);
                }
            } else {
                // S0 becomes part of a first row's input, dS_T takes the carry's place at a last row
                const float* p0 = a.S0 && (sbits >> r & 1) ? a.S0 + ((int64_t)ws.start[row0 + row_t + r] * a.H + head) * a.d + ch0 : nullptr;
                const float* p1 = a.dST && (ebits >> r & 1) ? a.dST + ((int64_t)ws.end[row0 + row_t + r] * a.H + head) * a.d + ch0 : nullptr;
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    if (p0) b[v] = fmaf(al[r][v], p0[v], b[v]);
                    if (p1) dy[v] += p1[v];
                    sf[v] = compose<true>(Span{sbits >> r & 1 ? -1.f : al[r][v], b[v]}, sf[v]);
                    sr[v] = ebits >> r & 1 ? Span{-1.f, al[r][v] * dy[v]}
                                           : Span{sr[v].A * al[r][v], al[r][v] * (dy[v] + sr[v].h)};
                }
            }
        }
    }

    if (plain) {   // no cut: the product is the same in both directions
#pragma unroll
        for (int v = 0; v < VEC; ++v) sr[v].A = sf[v].A;
    }

    // forward spans up to the thread, backward spans behind it: over the sub-chunks of the wave, then
    // over the waves, lane = channel
    WaveSpans<PACKED, false, VEC, SPW> wf;
    WaveSpans<PACKED, true, VEC, SPW> wb;
    wf.scan(sf, turn[wave], lane);
    wtA[wave][lane] = wf.total.A;
    wth[wave][lane] = wf.total.h;
    wb.scan(sr, turn[wave], lane);
    wtR[wave][lane] = wb.total.A;
    wtg[wave][lane] = wb.total.h;
    float hw = a.entry[(block_l * a.nch + c) * a.d + ch];
    lds_barrier();
    if (wave == 0) {   // lane = channel: the tile's backward span, the chain
        Span tot{wtR[W - 1][lane], wtg[W - 1][lane]};
#pragma unroll
        for (int i = W - 2; i >= 0; --i) tot = compose<PACKED>(tot, Span{wtR[i][lane], wtg[i][lane]});
        float g = 0.f;
        if (has_ch) {
            const bool first = (int64_t)c + 1 == ws.nt, more = c > 0;
            if (!PACKED && first && a.dST) g = a.dST[block_l * a.d + ch];
            if (chained) {
                const int64_t word = (block_l * ws.nt + c) * a.d + ch;
                const bool cut = PACKED && __float_as_int(tot.A) < 0;
                if (cut && more) publish(ws.state + word, 0, tot.h);
                if (!first) {
                    if (!cut && more) publish_span(ws.span + word, tot);
                    g = look_back<PACKED>(ws.span + word, ws.state + word, -a.d, ws.nt - 1 - c);
                }
                if (!cut && more) publish(ws.state + word, 0, apply<PACKED>(tot, g));
            }
            if (!PACKED && c == 0 && a.dS0) a.dS0[block_l * a.d + ch] = apply<PACKED>(tot, g);
        }
        gin[lane] = g;
    }
    lds_barrier();

    // the state before the wave's rows and the carry behind them, then the thread's
    float gw = gin[lane], h[VEC], g[VEC];
    for (int i = 0; i < wave; ++i) hw = apply<PACKED>(Span{wtA[i][lane], wth[i][lane]}, hw);
    for (int i = W - 1; i > wave; --i) gw = apply<PACKED>(Span{wtR[i][lane], wtg[i][lane]}, gw);
    wf.spread(hw, turn[wave], lane, h);
    wb.spread(gw, turn[wave], lane, g);
    // the state before each row
    auto row_x = [&](int r, float* o) {
        if constexpr (SX) unpack(xs[r][tid], o);
        else unpack(load_row<TIn, VEC>(xp + row_offset(off0, r, d, last_off)), o);
    };
    float prev[L][VEC];
#pragma unroll
    for (int r = 0; r < L; ++r) {
        float x[VEC];
        row_x(r, x);
        if (PACKED && (sbits >> r & 1)) {
#pragma unroll
            for (int v = 0; v < VEC; ++v)
                h[v] = a.S0 ? a.S0[((int64_t)ws.start[row0 + row_t + r] * a.H + head) * a.d + ch0 + v] : 0.f;
        }
#pragma unroll
        for (int v = 0; v < VEC; ++v) prev[r][v] = h[v];
        if (row_t + r < lo || row_t + r >= hi) continue;
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            float b = x[v];
            if (has_u) b *= gi[r][v];
            if (SCALE != KDA_GLR_ONE) b *= w[r][v];
            h[v] = fmaf(al[r][v], h[v], b);
        }
    }
    float eA[VEC], dA[VEC];
    if (has_z) {
        load_f32<VEC>(a.A_log + (int64_t)head * a.d + ch0, eA);
#pragma unroll
        for (int v = 0; v < VEC; ++v) { eA[v] = a.g_min * exp_f(eA[v]); dA[v] = 0.f; }
    }
    TIn *dx = (TIn*)a.dx + base, *dd = (TIn*)a.dd + base, *du = (TIn*)a.du + base;
#pragma unroll
    for (int r = L - 1; r >= 0; --r) {
        float x[VEC], q[VEC], dy[VEC], ox[VEC], od[VEC], ou[VEC];
        const bool live = row_t + r >= lo && row_t + r < hi;
        row_x(r, x);
        const uint32_t off = row_offset(off0, r, d, last_off);
        if constexpr (SZ) unpack(zs[r][tid], q);
        else if (has_z) unpack(load_row<TIn, VEC>(dec + off), q);
        if constexpr (SY) unpack(ys[r][tid], dy);
        else unpack(load_row<TOut, VEC>(yp + off), dy);
        if (PACKED && (ebits >> r & 1)) {
#pragma unroll
            for (int v = 0; v < VEC; ++v)
                g[v] = a.dST ? a.dST[((int64_t)ws.end[row0 + row_t + r] * a.H + head) * a.d + ch0 + v] : 0.f;
        }
        if (!live) continue;
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const float gr = g[v] + dy[v], alpha = al[r][v];
            float ix = x[v];
            ox[v] = SCALE == KDA_GLR_ONE ? gr : gr * w[r][v];
            if (has_u) {
                ix *= gi[r][v];
                ox[v] *= gi[r][v];
                ou[v] = ox[v] * x[v] * (1.f - gi[r][v]);
            }
            float e = alpha * prev[r][v];
            if (SCALE == KDA_GLR_LEAKY) e = fmaf(-alpha, ix, e);
            if (SCALE == KDA_GLR_NORM) {
                // dw / dlog_alpha = -alpha^2 / w, taken as 0 where w = 0
                const float aw = w[r][v] > 0.f ? alpha * __builtin_amdgcn_rcpf(w[r][v]) : 0.f;
                e = fmaf(-alpha * aw, ix, e);
            }
            e *= gr;
            if (has_z) {
                e *= s[r][v] * (1.f - s[r][v]) * eA[v];
                dA[v] = fmaf(e, q[v], dA[v]);
            }
            od[v] = e;
            g[v] = alpha * gr;
        }
        if (on) {
            store_row<VEC>(dx + (off0 + r * d), ox);
            store_row<VEC>(dd + (off0 + r * d), od);
            if (has_u) store_row<VEC>(du + (off0 + r * d), ou);
            if (PACKED && a.dS0 && (sbits >> r & 1)) {
                float* p = a.dS0 + ((int64_t)ws.start[row0 + row_t + r] * a.H + head) * a.d + ch0;
#pragma unroll
                for (int v = 0; v < VEC; ++v) p[v] = g[v];
            }
        }
    }
    if (!has_z) return;
    // the tile's part of dA_log: over the sub-chunks of the wave, then the waves
#pragma unroll
    for (int m = CT; m < 64; m <<= 1)
#pragma unroll
        for (int v = 0; v < VEC; ++v) dA[v] += __shfl_xor(dA[v], m);
    lds_barrier();
    if (lane < CT) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) wth[wave][ct * VEC + v] = dA[v];
    }
    lds_barrier();
    if (wave == 0 && has_ch) {
        float t = wth[0][lane];
#pragma unroll
        for (int i = 1; i < W; ++i) t += wth[i][lane];
        ws.dA[(block_l * ws.nt + c) * a.d + ch] = t;
    }
}

template <int SCALE, bool PACKED, bool NARROW, int Z, int U, typename TIn, int VEC, int L, int THREADS>
static hipError_t launch_bwd_k(const GlrArgs& a, const GlrWs& ws, hipStream_t st) {
    static_assert(THREADS == kTileThreads && Tile<VEC, L, THREADS>::ROWS == kBwdRows, "the plan's tile");
    const dim3 grid((unsigned)(chain_count(a.blocks, a.d, NARROW) * ws.nt));
    if (a.out_bf16)
        hipLaunchKernelGGL((glr_bwd_kernel<SCALE, PACKED, NARROW, Z, U, TIn, bf16_t, VEC, L, THREADS>), grid, dim3(THREADS), 0, st, a, ws);
    else
        hipLaunchKernelGGL((glr_bwd_kernel<SCALE, PACKED, NARROW, Z, U, TIn, float, VEC, L, THREADS>), grid, dim3(THREADS), 0, st, a, ws);
    return hipGetLastError();
}

// 4 channels a thread (ws.vec), 1 for heads of fewer.
template <int SCALE, bool PACKED, typename TIn>
hipError_t launch_bwd_t(const GlrArgs& a, const GlrWs& ws, hipStream_t st) {
    if (ws.narrow) return launch_bwd_k<SCALE, PACKED, true, 2, 2, TIn, 4, 4, 512>(a, ws, st);
    if (ws.vec == 4) {
        if (a.z && a.u) return launch_bwd_k<SCALE, PACKED, false, 1, 1, TIn, 4, 4, 512>(a, ws, st);
        if (a.z) return launch_bwd_k<SCALE, PACKED, false, 1, 0, TIn, 4, 4, 512>(a, ws, st);
        if (a.u) return launch_bwd_k<SCALE, PACKED, false, 0, 1, TIn, 4, 4, 512>(a, ws, st);
        return launch_bwd_k<SCALE, PACKED, false, 0, 0, TIn, 4, 4, 512>(a, ws, st);
    }
    return launch_bwd_k<SCALE, PACKED, false, 2, 2, TIn, 1, 16, 512>(a, ws, st);
}

}  // namespace glr
}  // namespace kda
