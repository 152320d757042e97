// Head norms with rotation, forward, and the cache append: one kernel, instantiated per type and
// layout in kda_rope_{bf16,f32}.hip.
#pragma once

#include "kda_rope.h"

namespace kda {
namespace rope {

template <bool APPEND>
__device__ __forceinline__ void fill_tokens(const RopeArgs& a, Token* tok, int64_t u0, int ntok) {
    const int lane = threadIdx.x & 63;
    for (int i = threadIdx.x >> 6; i < ntok; i += kWaves) {      // a wave per token
        const int64_t u = u0 + i, b = u / a.T, t = u - b * a.T;
        Token x;
        x.live = 1;
        x.stored = 0;
        x.q = b * a.sq.b + t * a.sq.t;
        x.k = b * a.sk.b + t * a.sk.t;
        x.qo = b * a.sqo.b + t * a.sqo.t;
        x.ko = b * a.sko.b + t * a.sko.t;
        x.v = x.vo = 0;
        x.sdq = b * a.sdq.b + t * a.sdq.t;
        x.sdk = b * a.sdk.b + t * a.sdk.t;
        int64_t pos;
        if constexpr (APPEND) {
            x.v = b * a.sv.b + t * a.sv.t;
            int64_t s = b, first = 0, n = a.T;
            if (a.packed) {
                s = find_sequence(a.cu, a.N, t);
                x.live = s >= 0 && s < a.N;
                s = x.live ? s : 0;
                first = a.cu[s];
                n = (int64_t)a.cu[s + 1] - first;
            }
            pos = (int64_t)a.kv_lens[s] - n + (t - first);
            if (x.live && pos >= 0 && pos < (int64_t)a.max_pages * a.page_size) {
                const int32_t pg = (int32_t)pos / a.page_size, row = (int32_t)pos - pg * a.page_size;
                const int32_t page = a.table[s * a.table_stride + pg];
                if (page >= 0 && page < a.pages) {
                    x.stored = 1;
                    x.ko = page * a.skc.p + row * a.skc.t;
                    x.vo = page * a.svc.p + row * a.svc.t;
                }
            }
        } else {
            pos = a.positions ? a.positions[u] : t;
        }
        x.pos = (int32_t)pos;
        if (lane == 0) tok[i] = x;
    }
}

// Rows of one kind (queries or keys) of the workgroup's tokens. KEYS: offsets k, ko and `stored`.
template <typename TI, typename TO, int LAY, bool KEYS, bool APPEND>
__device__ __forceinline__ void norm_rows(const RopeArgs& a, const Lane& l, const Token* tok, const float2* cs, int ntok,
                                          uint32_t magic) {
    constexpr int U = sizeof(TI) == 2 ? 4 : 2;
    const int H = KEYS ? a.Hk : a.Hq, rg = 64 / l.lpr, rows = ntok * H, P = a.d / 2;
    const TI* src = static_cast<const TI*>(KEYS ? a.k : a.q);
    TO* dst = static_cast<TO*>(KEYS ? a.k_out : a.q_out);
    const int64_t sh = KEYS ? a.sk.h : a.sq.h;
    const int64_t dh = KEYS ? (APPEND ? a.skc.h : a.sko.h) : a.sqo.h;
    const float inv_d = 1.f / (float)a.d;
    float w[16];
    if (a.norm) load_weight<LAY>(l, KEYS ? a.wk : a.wq, w);
    for (int base = (threadIdx.x >> 6) * rg * U; base < rows; base += kWaves * rg * U) {
        float x[U][16];
        int tk[U];
        int64_t out[U];
        bool on[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = base + u * rg + l.g;
            on[u] = r < rows;
            const int rr = on[u] ? r : 0;
            const int t = div_heads(rr, magic), h = rr - t * H;
            tk[u] = t;
            on[u] = on[u] && (KEYS && APPEND ? tok[t].stored : tok[t].live);
            out[u] = (KEYS ? tok[t].ko : tok[t].qo) + h * dh;
            load_row<TI, LAY>(l, src + ((KEYS ? tok[t].k : tok[t].q) + h * sh), on[u], x[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            to_pairs<LAY>(x[u]);
            if (a.norm) {
                float s = 0.f;
#pragma unroll
                for (int j = 0; j < 16; ++j) s = fmaf(x[u][j], x[u][j], s);
                s = row_sum(s, l.lpr);
                const float r = 1.f / sqrtf(fmaf(s, inv_d, a.eps));
#pragma unroll
                for (int j = 0; j < 16; ++j) x[u][j] = x[u][j] * r * w[j];
            }
            if (a.rot) {
                float co[8], si[8];
                load_angles<LAY>(l, cs + tk[u] * P, co, si);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float va = x[u][j], vb = x[u][8 + j];
                    x[u][j] = fmaf(va, co[j], -vb * si[j]);
                    x[u][8 + j] = fmaf(vb, co[j], va * si[j]);
                }
            }
            from_pairs<LAY>(x[u]);
            if (on[u]) store_row<TO, LAY>(l, dst + out[u], x[u]);
        }
    }
}

// The new tokens' values into the cache: 8 channels an access where rows lie on 16 bytes.
template <typename TI, bool WIDE>
__device__ __forceinline__ void copy_values(const RopeArgs& a, const Token* tok, int ntok) {
    constexpr int V = WIDE ? 8 : 1;
    const int per = a.dv / V, total = ntok * a.Hk * per;
    for (int e = threadIdx.x; e < total; e += kThreads) {
        const int row = e / per, c = (e - row * per) * V, t = row / a.Hk, h = row - t * a.Hk;
        if (!tok[t].stored) continue;
        const TI* p = static_cast<const TI*>(a.v) + (tok[t].v + h * a.sv.h + c);
        bf16_t* o = static_cast<bf16_t*>(a.v_out) + (tok[t].vo + h * a.svc.h + c);
        if constexpr (WIDE) {
            if constexpr (sizeof(TI) == 2) {
                *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(p);
            } else {
                float x[8];
                unpack8(p, x);
                store8(o, x);
            }
        } else {
            st_f(o, ld_f(p));
        }
    }
}

template <typename TI, typename TO, int LAY, bool APPEND>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeArgs a, Shape s, int v_wide) {
    extern __shared__ __align__(16) float2 cs[];
    __shared__ Token tok[kMaxTokens];
    const int64_t u0 = (int64_t)blockIdx.x * s.tokens, all = a.B * a.T;
    const int ntok = (int)(all - u0 < s.tokens ? all - u0 : s.tokens);
    const Lane l = make_lane<LAY>(a, s.lpr);
    fill_tokens<APPEND>(a, tok, u0, ntok);
    lds_barrier();
    if (a.rot) {
        fill_angles(a, tok, ntok, cs);
        lds_barrier();
    }
    if (a.Hq) norm_rows<TI, TO, LAY, false, APPEND>(a, l, tok, cs, ntok, s.mq);
    if (a.Hk) norm_rows<TI, TO, LAY, true, APPEND>(a, l, tok, cs, ntok, s.mk);
    if constexpr (APPEND) {
        if (v_wide)
            copy_values<TI, true>(a, tok, ntok);
        else
            copy_values<TI, false>(a, tok, ntok);
    }
}

template <typename TI, typename TO, bool APPEND>
hipError_t launch_rows(const RopeArgs& a, const Shape& s, int lay, bool v_wide, hipStream_t st) {
    const dim3 grid((unsigned)((a.B * a.T + s.tokens - 1) / s.tokens)), block(kThreads);
    const size_t lds = a.rot ? (size_t)s.tokens * (a.d / 2) * sizeof(float2) : 0;
    const int vw = v_wide;
    switch (lay) {
        case kHalfWide: hipLaunchKernelGGL((rope_kernel<TI, TO, kHalfWide, APPEND>), grid, block, lds, st, a, s, vw); break;
        case kInterWide: hipLaunchKernelGGL((rope_kernel<TI, TO, kInterWide, APPEND>), grid, block, lds, st, a, s, vw); break;
        case kHalfElem: hipLaunchKernelGGL((rope_kernel<TI, TO, kHalfElem, APPEND>), grid, block, lds, st, a, s, vw); break;
        default: hipLaunchKernelGGL((rope_kernel<TI, TO, kInterElem, APPEND>), grid, block, lds, st, a, s, vw); break;
    }
    return hipGetLastError();
}

}  // namespace rope
}  // namespace kda
