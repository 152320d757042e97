// Gated linear recurrence for gfx950, forward (include/kda_glr.h):
//     h_t = alpha_t h_{t-1} + w(alpha_t) i_t x_t,   y_t = h_t.
//
// The operator moves one word in per tensor and one out per element, so HBM bounds it and every
// input should be read once; the gates' exponentials and roots come close behind (46 issue
// slots an element with every gate, 28 with log decays, by counters). The rows of a block are split into tiles: a workgroup holds
// its tile's decays and inputs in registers, reduces them to the tile's span h -> A h + b (a scan
// over threads, waves and LDS), gets the state before the tile from the chain of the tiles before
// it (kda_glr_device.h), and runs the recurrence again from there with the rows still in registers.
// The chain is waited for once per tile, when the spans of the tiles before it, which depend on
// nothing, are usually there.
//
// Measured, bf16 (kernel alone): 32 x 64K rows of 128 channels with log decays 343 us, 4.7 TB/s; 32 x
// 8K rows 41.8 us; 2 x 4096 rows of 4096 channels with both gates and w = sqrt(1 - alpha^2) 67.6 us,
// 4.0 TB/s.
#pragma once

#include "kda_glr_device.h"
#include "kda_glr_plan.h"

namespace kda {
namespace glr {

constexpr int kCh = KDA_GLR_CHUNK;

// Z, U: whether the decay comes from z and whether there is an input gate (2: looked up).
template <int SCALE, bool PACKED, bool NARROW, int Z, int U, typename TIn, int VEC, int L, int THREADS>
__global__ __launch_bounds__(THREADS, 4) void glr_fwd_kernel(GlrArgs a, GlrWs ws) {
    using G = Tile<VEC, L, THREADS>;
    constexpr int CT = G::CT, SPW = G::SPW, W = G::W, ROWS = G::ROWS;
    static_assert(kCh % L == 0 && ROWS % kCh == 0, "a chunk starts at a thread's first row");
    __shared__ float wtA[W][kCW], wth[W][kCW], hin[kCW];
    __shared__ __align__(16) float turn[W][SPW > 1 ? 2 * SPW * kCW : 1];
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
    RawRow<TIn, VEC> xr[L], dr[L], ur[L];
    const TIn* dec = (const TIn*)(has_z ? a.z : a.la) + base;
    const TIn* xp = (const TIn*)a.x + base;
    const TIn* up = (const TIn*)a.u + base;
#pragma unroll
    for (int r = 0; r < L; ++r) {
        const uint32_t off = row_offset(off0, r, d, last_off);
        dr[r] = load_row<TIn, VEC>(dec + off);
        xr[r] = load_row<TIn, VEC>(xp + off);
        if (has_u) ur[r] = load_row<TIn, VEC>(up + off);
    }
    const float gy = a.g_min * kLog2e;
    float cz[VEC];
    if (has_z) {
        load_f32<VEC>(a.A_log + (int64_t)head * a.d + ch0, cz);
#pragma unroll
        for (int v = 0; v < VEC; ++v) cz[v] = -kLog2e * exp_f(cz[v]);
    }
    // decay and scaled input of a row of the thread
    const bool edge = lo > 0 || hi < ROWS;
    auto row_values = [&](int r, float (&al)[VEC], float (&b)[VEC]) {
        float x[VEC], q[VEC], g[VEC];
        unpack(xr[r], x);
        unpack(dr[r], q);
        if (has_u) unpack(ur[r], g);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const float y = has_z ? gy * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(cz[v] * q[v])) : q[v] * kLog2e;
            al[v] = __builtin_amdgcn_exp2f(y);
            b[v] = has_u ? x[v] * sigmoid_f(g[v]) : x[v];
            if (SCALE != KDA_GLR_ONE) b[v] *= scale_w<SCALE>(y, al[v]);
        }
        if (edge && (row_t + r < lo || row_t + r >= hi)) {   // a row in no sequence passes the state on
#pragma unroll
            for (int v = 0; v < VEC; ++v) { al[v] = 1.f; b[v] = 0.f; }
        }
        if (PACKED && (sbits >> r & 1) && a.S0) {   // a sequence's S0 becomes part of its first row's input
            const float* s0 = a.S0 + ((int64_t)ws.start[row0 + row_t + r] * a.H + head) * a.d + ch0;
#pragma unroll
            for (int v = 0; v < VEC; ++v) b[v] = fmaf(al[v], s0[v], b[v]);
        }
    };
    float al[L][VEC], b[L][VEC];
#pragma unroll
    for (int r = 0; r < L; ++r) row_values(r, al[r], b[r]);
    // the thread's span
    Span sp[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) sp[v] = Span{1.f, 0.f};
#pragma unroll
    for (int r = 0; r < L; ++r) {
        if (PACKED && (sbits >> r & 1)) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) sp[v] = Span{-1.f, b[r][v]};
        } else {
#pragma unroll
            for (int v = 0; v < VEC; ++v) sp[v] = compose<false>(sp[v], Span{al[r][v], b[r][v]});
        }
    }

    // spans over the sub-chunks of the wave, then over the waves: lane = channel
    WaveSpans<PACKED, false, VEC, SPW> wave_spans;
    wave_spans.scan(sp, turn[wave], lane);
    wtA[wave][lane] = wave_spans.total.A;
    wth[wave][lane] = wave_spans.total.h;
    lds_barrier();
    if (wave == 0) {   // lane = channel: the tile's span, the chain
        Span tot{wtA[0][lane], wth[0][lane]};
#pragma unroll
        for (int w = 1; w < W; ++w) tot = compose<PACKED>(tot, Span{wtA[w][lane], wth[w][lane]});
        float h = 0.f;
        if (has_ch) {
            if (!PACKED && c == 0 && a.S0) h = a.S0[block_l * a.d + ch];
            if (chained) {
                const int64_t word = (block_l * ws.nt + c) * a.d + ch;
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
    lds_barrier();
    // the state before the wave's first row, then before the thread's
    float hw = hin[lane], h[VEC];
    for (int w = 0; w < wave; ++w) hw = apply<PACKED>(Span{wtA[w][lane], wth[w][lane]}, hw);
    wave_spans.spread(hw, turn[wave], lane, h);
    if (!on) return;
    if (a.entry && row_t % kCh == 0 && row_t < rows_here) {
        float* e = a.entry + (block * a.nch + (row0 + row_t) / kCh) * a.d + ch0;
#pragma unroll
        for (int v = 0; v < VEC; ++v) e[v] = h[v];
    }
    // the recurrence again, from there
    bf16_t* yh = (bf16_t*)a.y + base;
    float* yf = (float*)a.y + base;
#pragma unroll
    for (int r = 0; r < L; ++r) {
        if (PACKED && (sbits >> r & 1)) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) h[v] = b[r][v];
        } else {
#pragma unroll
            for (int v = 0; v < VEC; ++v) h[v] = fmaf(al[r][v], h[v], b[r][v]);
        }
        if (a.y && row_t + r >= lo && row_t + r < hi) {
            if (a.out_bf16) store_row<VEC>(yh + (off0 + r * d), h);
            else store_row<VEC>(yf + (off0 + r * d), h);
        }
        if (PACKED && (ebits >> r & 1) && a.S_T) {
            float* st = a.S_T + ((int64_t)ws.end[row0 + row_t + r] * a.H + head) * a.d + ch0;
#pragma unroll
            for (int v = 0; v < VEC; ++v) st[v] = h[v];
        }
    }
    if constexpr (!PACKED) {
        // rows behind the last one pass the state on, so the last row's state is the thread's last
        const int64_t last = a.T - 1 - row0;
        if (a.S_T && row_t <= last && last < row_t + L) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) a.S_T[block * a.d + ch0 + v] = h[v];
        }
    }
}

template <int SCALE, bool PACKED, bool NARROW, int Z, int U, typename TIn, int VEC, int L, int THREADS>
static hipError_t launch_fwd_k(const GlrArgs& a, const GlrWs& ws, hipStream_t st) {
    static_assert(THREADS == kTileThreads && Tile<VEC, L, THREADS>::ROWS == (VEC == 4 ? kFwdRows : kFwdRows1), "the plan's tile");
    hipLaunchKernelGGL((glr_fwd_kernel<SCALE, PACKED, NARROW, Z, U, TIn, VEC, L, THREADS>),
                       dim3((unsigned)(chain_count(a.blocks, a.d, NARROW) * ws.nt)), dim3(THREADS), 0, st, a, ws);
    return hipGetLastError();
}

// 4 channels a thread (ws.vec), 1 for heads of fewer; narrow heads (ws.narrow) look the gates up.
// 512 threads of 8 rows: a tile of 256 rows halves the chain's links against 128 (64K rows x 4096
// channels: 366 us against 404 with 256 threads, before the last steps), and 8 rows a thread leave
// room for 4 waves a SIMD. 512 rows on 1024 threads wait longer at their barriers (369 us, packed
// batches 81 us against 71). One channel a thread (16 rows) needs four times the accesses: 64 x 4096
// rows of 77 bf16 channels with gates take 106 us that way and 60 with 4, which any head of 4 has.
template <int SCALE, bool PACKED, typename TIn>
hipError_t launch_fwd_t(const GlrArgs& a, const GlrWs& ws, hipStream_t st) {
    if (ws.narrow) return launch_fwd_k<SCALE, PACKED, true, 2, 2, TIn, 4, 8, 512>(a, ws, st);
    if (ws.vec == 4) {
        if (a.z && a.u) return launch_fwd_k<SCALE, PACKED, false, 1, 1, TIn, 4, 8, 512>(a, ws, st);
        if (a.z) return launch_fwd_k<SCALE, PACKED, false, 1, 0, TIn, 4, 8, 512>(a, ws, st);
        if (a.u) return launch_fwd_k<SCALE, PACKED, false, 0, 1, TIn, 4, 8, 512>(a, ws, st);
        return launch_fwd_k<SCALE, PACKED, false, 0, 0, TIn, 4, 8, 512>(a, ws, st);
    }
    return launch_fwd_k<SCALE, PACKED, false, 2, 2, TIn, 1, 16, 512>(a, ws, st);
}

}  // namespace glr
}  // namespace kda
