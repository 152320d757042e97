// Head norms with rotation, forward, and the cache append: one kernel, instantiated per type and
// layout in kda_rope_{bf16,f32}.hip.
//
// The append takes 43 us for 8192 packed tokens of 32 + 8 bf16 heads of 128 (201 MB, 4.7 TB/s; 12 % more reaches HBM, the
// sequences' rows of a page sharing no run of memory) and 4.0 us for 256 sequences of one token, which is the time from
// cu_seqlens or kv_lens to the table to the store.
#pragma once

#include "kda_rope.h"

namespace kda {
namespace rope {

// Positions of a workgroup's tokens, and for the append their places in the cache; a lane of the first wave a
// token.
template <bool APPEND>
__device__ __forceinline__ void fill_tokens(const RopeArgs& a, Token* tok, int64_t u0, int ntok, int kind) {
    const int i = threadIdx.x;
    if (i >= 64) return;
    const int64_t u = u0 + (i < ntok ? i : 0), b = a.B == 1 ? 0 : u / a.T, t = u - b * a.T;
    Token x;
    x.on = 1;
    x.dst = 0;
    int64_t pos;
    if constexpr (APPEND) {
        int64_t s = b, first = 0, n = a.T;
        bool live = true;
        if (a.packed) {
            // the first token's sequence is that of all tokens before its end, and so on from there
            for (int from = 0; from < ntok;) {
                const int f = find_sequence(a.cu, a.N, u0 + from);
                const int64_t end = (f >= a.N ? a.T : (int64_t)a.cu[f + 1]) - u0;
                if (i >= from) s = f;
                from = end > from ? (end < ntok ? (int)end : ntok) : from + 1;
            }
            live = s >= 0 && s < a.N;
            s = live ? s : 0;
            first = a.cu[s];
            n = (int64_t)a.cu[s + 1] - first;
        }
        pos = (int64_t)a.kv_lens[s] - n + (t - first);
        x.on = live;
        if (kind != kQueries) {
            x.on = 0;
            if (live && pos >= 0 && pos < (int64_t)a.max_pages * a.page_size) {
                const int32_t pg = (int32_t)pos / a.page_size, row = (int32_t)pos - pg * a.page_size;
                const int32_t page = a.table[s * a.table_stride + pg];
                const kda_page_strides& st = kind == kKeys ? a.skc : a.svc;
                x.on = page >= 0 && page < a.pages;
                x.dst = page * st.p + row * st.t;
            }
        }
    } else {
        pos = a.positions ? a.positions[u] : t;
    }
    x.pos = (int32_t)pos;
    if (i < ntok) tok[i] = x;
}

// The new tokens' values into the cache: 8 channels an access where rows lie on 16 bytes, v_lanes lanes a row
// and four rows a thread under way.
template <typename TI, bool WIDE>
__device__ __forceinline__ void copy_values(const RopeArgs& a, const Rows3& rows, const Token* tok, int lanes) {
    constexpr int V = WIDE ? 8 : 1, AT = 4;
    const int rg = kThreads / lanes, shift = __builtin_ctz(lanes);
    const TI* src = static_cast<const TI*>(a.v);
    bf16_t* dst = static_cast<bf16_t*>(a.v_out);
#pragma unroll 1
    for (int c = (threadIdx.x & (lanes - 1)) * V; c < a.dv; c += lanes * V)
#pragma unroll 1
        for (int r0 = threadIdx.x >> shift; r0 < rows.count; r0 += AT * rg) {
            uint4 u[AT], u1[AT];
            float f[AT];
            Row x[AT];
#pragma unroll
            for (int k = 0; k < AT; ++k) {
                x[k] = rows.row(r0 + k * rg < rows.count ? r0 + k * rg : r0);
                const TI* p = src + (x[k].at(a.sv) + c);
                if constexpr (WIDE) {
                    u[k] = *reinterpret_cast<const uint4*>(p);
                    if constexpr (sizeof(TI) == 4) u1[k] = *reinterpret_cast<const uint4*>(p + 4);
                } else {
                    f[k] = ld_f(p);
                }
            }
#pragma unroll
            for (int k = 0; k < AT; ++k) {
                if (r0 + k * rg >= rows.count || !tok[x[k].t].on) continue;
                bf16_t* o = dst + (tok[x[k].t].dst + x[k].h * a.svc.h + c);
                if constexpr (!WIDE) {
                    st_f(o, f[k]);
                } else if constexpr (sizeof(TI) == 2) {
                    *reinterpret_cast<uint4*>(o) = u[k];
                } else {
                    float g[8];
                    unpack16(u[k], src, g);
                    unpack16(u1[k], src, g + 4);
                    store8(o, g);
                }
            }
        }
}

// The rows of workgroup `group` of a kind.
__device__ __forceinline__ Rows3 rows_of(const RopeArgs& a, const Shape& s, int kind, int64_t group, int& ntok) {
    Rows3 r;
    const int64_t u0 = group * s.tokens[kind], all = a.B * a.T;
    ntok = (int)(all - u0 < s.tokens[kind] ? all - u0 : s.tokens[kind]);
    r.u0 = (uint32_t)u0;
    r.T = (uint32_t)a.T;
    r.H = kind == kQueries ? a.Hq : a.Hk;
    r.count = ntok * r.H;
    r.magic = s.magic[kind];
    r.one = a.B == 1;
    return r;
}

template <typename TI, typename TO, int LAY, bool APPEND>
__global__ __launch_bounds__(kThreads, kLaysWide<LAY> ? 5 : 3) void rope_kernel(RopeArgs a, Shape s) {
    extern __shared__ __align__(16) float2 cs[];
    __shared__ Token tok[kMaxTokens];
    // the append's values and keys first: they wait longest, for their places
    const int64_t wg = APPEND ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
    const int kind = wg < s.group0[1] ? kQueries : wg < s.group0[2] ? kKeys : kValues;
    int ntok;
    const Rows3 rows = rows_of(a, s, kind, wg - s.group0[kind], ntok);
    if constexpr (APPEND) {
        if (kind == kValues) {
            fill_tokens<true>(a, tok, rows.u0, ntok, kind);
            lds_barrier();
            if (s.v_wide)
                copy_values<TI, true>(a, rows, tok, s.v_lanes);
            else
                copy_values<TI, false>(a, rows, tok, s.v_lanes);
            return;
        }
    }
    const bool keys = kind == kKeys, to_cache = APPEND && keys;
    const Lane l = make_lane<LAY>(a, s.lpr);
    const int rg = 64 / l.lpr, P = a.d / 2;
    const TI* src = static_cast<const TI*>(keys ? a.k : a.q);
    TO* dst = static_cast<TO*>(keys ? a.k_out : a.q_out);
    const kda_row_strides &si = keys ? a.sk : a.sq, &so = keys ? a.sko : a.sqo;
    const float inv_d = 1.f / (float)a.d;
    int r = (threadIdx.x >> 6) * rg + l.g;
    Row row = rows.row(r < rows.count ? r : 0);
    Raw<TI, LAY> raw;
    raw.load(l, src + row.at(si));
    float w[16];
    if (a.norm) load_weight<LAY>(l, keys ? a.wk : a.wq, w);
    fill_tokens<APPEND>(a, tok, rows.u0, ntok, kind);
    lds_barrier();
    if (a.rot) {
        fill_angles(a, tok, ntok, cs);
        lds_barrier();
    }
#pragma unroll 1
    for (int first = (threadIdx.x >> 6) * rg; first < rows.count; first += kWaves * rg) {
        const bool on = r < rows.count && tok[row.t].on;
        const Row now = row;
        float x[16];
        raw.get(l, x);
        r += kWaves * rg;
        if (first + kWaves * rg < rows.count) {
            row = rows.row(r < rows.count ? r : 0);
            raw.load(l, src + row.at(si));
        }
        if (a.norm) {
            float q = 0.f;
#pragma unroll
            for (int j = 0; j < 16; ++j) q = fmaf(x[j], x[j], q);
            const float n = inv_root(fmaf(row_sum(q, l.lpr), inv_d, a.eps));
#pragma unroll
            for (int j = 0; j < 16; ++j) x[j] = x[j] * n * w[j];
        }
        if (a.rot) {
            float co[8], sn[8];
            load_angles<LAY>(l, cs + now.t * P, co, sn);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float va = x[j], vb = x[8 + j];
                x[j] = fmaf(va, co[j], -vb * sn[j]);
                x[8 + j] = fmaf(vb, co[j], va * sn[j]);
            }
        }
        from_pairs<LAY>(x);
        if (on) store_row<TO, LAY>(l, dst + (to_cache ? tok[now.t].dst + now.h * a.skc.h : now.at(so)), x);
    }
}

template <typename TI, typename TO, bool APPEND>
hipError_t launch_rows(const RopeArgs& a, const Shape& s, int lay, hipStream_t st) {
    const dim3 grid((unsigned)s.group0[3]), block(kThreads);
    const int most = s.tokens[0] > s.tokens[1] ? s.tokens[0] : s.tokens[1];
    const size_t lds = a.rot ? (size_t)most * (a.d / 2) * sizeof(float2) : 0;
    switch (lay) {
        case kHalfWide: hipLaunchKernelGGL((rope_kernel<TI, TO, kHalfWide, APPEND>), grid, block, lds, st, a, s); break;
        case kInterWide: hipLaunchKernelGGL((rope_kernel<TI, TO, kInterWide, APPEND>), grid, block, lds, st, a, s); break;
        case kHalfElem: hipLaunchKernelGGL((rope_kernel<TI, TO, kHalfElem, APPEND>), grid, block, lds, st, a, s); break;
        default: hipLaunchKernelGGL((rope_kernel<TI, TO, kInterElem, APPEND>), grid, block, lds, st, a, s); break;
    }
    return hipGetLastError();
}

}  // namespace rope
}  // namespace kda
