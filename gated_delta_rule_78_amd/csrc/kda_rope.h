// Device code shared by the head norms with rotation and the cache append (include/kda_attn.h).
//
// A workgroup of 256 threads takes the rows (token, head) of a few tokens of one tensor, q or k. It asks
// for its first rows, then forms the tokens' cosines and sines in LDS, once for all heads. A row is held
// by `lpr` lanes, 8 pairs a lane (both members of a pair in one lane, so a rotation needs no exchange),
// 64 / lpr rows a wave at a time, the next ones on their way meanwhile. The code is kept short and its
// loops rolled, since small calls wait for cold code (four rows a lane at once: 11.5 KB and 9 us for
// one token, here 3.0).
//
// The bytes of the rows bound it: 8192 tokens of 32 + 8 bf16 heads of 128 (168 MB) take 33 us, 5.1 TB/s where a large
// copy reaches 5.2, and their backward (252 MB) 46 us, 5.5 TB/s. Both directions in fp32 (671 MB, x once) 170 us, where
// the backward spills 5 registers; heads of 130 by elements 187 us in bf16 and 213 in fp32.
#pragma once

#include "kda_device.h"
#include "kda_rope_internal.h"

namespace kda {
namespace rope {

constexpr int kThreads = 256, kWaves = 4;
constexpr int kMaxTokens = 16;     // of a workgroup

// How a lane's pairs lie in a row. Wide: 16-byte accesses, both runs of 8 channels on 8 elements;
// element: single channels, pair c + lpr * j of lane c.
enum Layout { kHalfWide = 0, kInterWide = 1, kHalfElem = 2, kInterElem = 3 };

template <int LAY>
constexpr bool kLaysWide = LAY == kHalfWide || LAY == kInterWide;

// What a workgroup is about: one tensor's rows (kValues: the append's copy of v).
enum Kind { kQueries = 0, kKeys = 1, kValues = 2 };

// How the rows are shared out: workgroups group0[kind] .. group0[kind + 1] - 1 take `tokens` tokens each
// of a kind.
struct Shape {
    int lpr;                // lanes a row
    int v_wide, v_lanes;    // append: v in 16-byte accesses, by so many lanes a row (a power of two)
    int tokens[3];
    int64_t group0[4];
    uint32_t magic[3];      // ceil(2^32 / heads), 0 for one head
};

// A token of a workgroup, in LDS.
struct Token {
    int64_t dst;            // append: where its k (or v) goes in the cache
    int32_t pos;
    int32_t on;             // its row is to be written
};

// Quotient of a row index by the heads: exact for n < 2^16 with magic = ceil(2^32 / h) (h > 1).
__device__ __forceinline__ int div_heads(int n, uint32_t magic) {
    return magic ? (int)__umulhi((uint32_t)n, magic) : n;
}

// A row: its block, token of the block and head, and its token in the workgroup.
struct Row {
    uint32_t b, u, h;
    int t;
    // element offset; h and t strides have 32 bits
    __device__ __forceinline__ int64_t at(const kda_row_strides& s) const {
        return (int64_t)((uint64_t)b * (uint64_t)s.b + (uint64_t)u * (uint32_t)s.t + (uint64_t)h * (uint32_t)s.h);
    }
};

// The rows of a workgroup: row r is token u0 + r / H, head r % H.
struct Rows3 {
    uint32_t u0, T;
    int H, count;
    uint32_t magic;
    bool one;               // one block of rows: no division by T
    __device__ __forceinline__ Row row(int r) const {
        Row x;
        x.t = div_heads(r, magic);
        x.h = (uint32_t)(r - x.t * H);
        x.u = u0 + x.t;
        x.b = 0;
        if (!one) {
            x.b = x.u / T;
            x.u -= x.b * T;
        }
        return x;
    }
};

// 1 / sqrt(v) for v > 0, subnormal ones too: off by at most one unit in the last place.
__device__ __forceinline__ float inv_root(float v) {
    const bool small = v < 0x1p-96f;
    const float r = __builtin_amdgcn_rsqf(small ? v * 0x1p96f : v);
    return small ? r * 0x1p48f : r;
}

// cos and sin of 2 pi t: t less its nearest quarter in fp64 (exact), then the series of both on
// [-pi/4, pi/4] up to x^9 and x^10, whose next terms are below 2e-9 and 2e-10 there.
__device__ __forceinline__ void sincos_turns(double t, float& s, float& c) {
    const double fr = t - rint(t);
    const double qd = rint(4.0 * fr);
    const float x = (float)(fma(-0.25, qd, fr) * 6.283185307179586);
    const int q = (int)qd & 3;
    const float x2 = x * x;
    float sp = fmaf(x2, 2.7557319e-6f, -1.9841270e-4f);
    sp = fmaf(x2, sp, 8.3333333e-3f);
    sp = fmaf(x2, sp, -1.6666667e-1f);
    sp = fmaf(x * x2, sp, x);
    float cp = fmaf(x2, -2.7557319e-7f, 2.4801587e-5f);
    cp = fmaf(x2, cp, -1.3888889e-3f);
    cp = fmaf(x2, cp, 4.1666667e-2f);
    cp = fmaf(x2, cp, -0.5f);
    cp = fmaf(x2, cp, 1.0f);
    s = (q & 1) ? cp : sp;
    c = (q & 1) ? sp : cp;
    if (q & 2) s = -s;
    if (q == 1 || q == 2) c = -c;
}

// cs[tok][i] = (cos, sin) * scale of the tokens' pairs; pairs past rot/2 keep (1, 0).
__device__ __forceinline__ void fill_angles(const RopeArgs& a, const Token* tok, int ntok, float2* cs) {
    const int P = a.d / 2, R = a.rot / 2;
    for (int e = threadIdx.x; e < ntok * P; e += kThreads) {
        const int t = ntok == 1 ? 0 : e / P, i = e - t * P;
        float2 v = make_float2(1.f, 0.f);
        if (i < R) {
            // one turn is 2 pi; the product of a 32-bit position and a 24-bit frequency is off by 2^-53
            const double turns = (double)tok[t].pos * (double)a.inv_freq[i] * 0.15915494309189535;
            float s, c;
            sincos_turns(turns, s, c);
            v = make_float2(c * a.scale, s * a.scale);
        }
        cs[e] = v;
    }
}

// The sequence of packed row t: the last s with cu[s] <= t (all 64 lanes take part), or -1 / N outside.
__device__ __forceinline__ int find_sequence(const int32_t* cu, int64_t N, int64_t t) {
    const int lane = threadIdx.x & 63;
    int64_t lo = 0, n = N + 1;             // candidates cu[lo .. lo + n)
    bool any = false;
    while (n > 0) {
        const int64_t step = (n + 63) / 64;
        const int64_t i = lo + lane * step;
        const bool le = lane * step < n && (int64_t)cu[i < N ? i : N] <= t;
        const int cnt = __popcll(__ballot(le));
        if (cnt == 0) return any ? (int)lo : -1;   // not even the first candidate
        any = true;
        const int64_t at = (int64_t)(cnt - 1) * step;
        lo += at;
        n = n - at < step ? n - at : step;
        if (step == 1) return (int)lo;
    }
    return -1;
}

// ---- a lane's 8 pairs of a row ------------------------------------------------------------------

struct Lane {
    int c, g;           // place in the row, row of the wave
    int lpr;            // lanes a row, a power of two
    bool live;          // has channels at all
    int oa, ob;         // wide: first channel of either run
    int P, R, H2;       // pairs, rotated pairs, half the others
    // element layouts: the channels of pair p
    template <int LAY>
    __device__ __forceinline__ int ia(int p) const { return LAY == kInterElem ? 2 * p : p < R ? p : R + p; }
    template <int LAY>
    __device__ __forceinline__ int ib(int p) const {
        return LAY == kInterElem ? 2 * p + 1 : p < R ? R + p : R + H2 + p;
    }
};

template <int LAY>
__device__ __forceinline__ Lane make_lane(const RopeArgs& a, int lpr) {
    Lane l;
    const int lane = threadIdx.x & 63;
    l.lpr = lpr;
    l.c = lane & (lpr - 1);
    l.g = lane / lpr;
    l.P = a.d / 2;
    l.R = a.rot / 2;
    l.H2 = (a.d - a.rot) / 2;
    if (LAY == kInterWide) {
        l.oa = 16 * l.c;
        l.ob = l.oa + 8;
        l.live = l.oa < a.d;
        if (!l.live) l.oa = 0, l.ob = 0;
    } else if (LAY == kHalfWide) {
        const int p = 8 * l.c;
        l.live = p < l.P;
        l.oa = p < l.R ? p : l.R + p;                     // rot + (p - rot/2)
        l.ob = p < l.R ? p + l.R : l.R + l.H2 + p;
        if (!l.live) l.oa = 0, l.ob = 0;
    } else {
        l.live = true;
        l.oa = l.ob = 0;
    }
    return l;
}

// The 16 channels as they come from memory, turned into floats only where a row is worked on: several
// rows are in flight, and packed bf16 is half the registers. Interleaved wide rows hold channels in order.
template <typename T, int LAY>
struct Raw {
    static constexpr bool kWide = LAY == kHalfWide || LAY == kInterWide;
    static constexpr int kWords = kWide ? 4 * sizeof(T) / 4 * 4 : 16;      // 8 for bf16, 16 for fp32; elements one each
    uint32_t w[kWords];

    // The row exists: lanes past it read its first channels, so that no load waits for a branch.
    __device__ __forceinline__ void load(const Lane& l, const T* row) {
        if constexpr (kWide) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int k = 0; k < kWords / 8; ++k) {
                    const uint4 u = *reinterpret_cast<const uint4*>(row + (h ? l.ob : l.oa) + k * (16 / (int)sizeof(T)));
                    uint32_t* d = w + h * (kWords / 2) + 4 * k;
                    d[0] = u.x; d[1] = u.y; d[2] = u.z; d[3] = u.w;
                }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int p = l.c + l.lpr * j, q = p < l.P ? p : 0;
                w[j] = bits(row[l.template ia<LAY>(q)]);
                w[8 + j] = bits(row[l.template ib<LAY>(q)]);
            }
        }
    }
    // x[0..7] the first members of the lane's pairs, x[8..15] the second; zeros past the row's end.
    __device__ __forceinline__ void get(const Lane& l, float* x) const {
        if constexpr (kWide && sizeof(T) == 2) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float lo = __uint_as_float(w[j] << 16), hi = __uint_as_float(w[j] & 0xffff0000u);
                if (LAY == kInterWide) {
                    x[j] = lo;
                    x[8 + j] = hi;
                } else {
                    x[2 * j] = lo;
                    x[2 * j + 1] = hi;
                }
            }
        } else if constexpr (kWide) {
#pragma unroll
            for (int j = 0; j < 16; ++j) x[LAY == kInterWide ? (j & 1) * 8 + (j >> 1) : j] = __uint_as_float(w[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) x[j] = sizeof(T) == 2 ? __uint_as_float(w[j] << 16) : __uint_as_float(w[j]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (kWide ? !l.live : l.c + l.lpr * j >= l.P) x[j] = x[8 + j] = 0.f;
    }
    __device__ static __forceinline__ uint32_t bits(bf16_t v) { return v; }
    __device__ static __forceinline__ uint32_t bits(float v) { return __float_as_uint(v); }
};

template <typename T, int LAY>
__device__ __forceinline__ void store_row(const Lane& l, T* row, const float* x) {
    if constexpr (LAY == kHalfWide || LAY == kInterWide) {
        if (l.live) {
            store8(row + l.oa, x);
            store8(row + l.ob, x + 8);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int p = l.c + l.lpr * j;
            if (p < l.P) {
                st_f(row + l.ia<LAY>(p), x[j]);
                st_f(row + l.ib<LAY>(p), x[8 + j]);
            }
        }
    }
}

// Pairs to channels in order, for interleaved wide stores.
template <int LAY>
__device__ __forceinline__ void from_pairs(float* x) {
    if constexpr (LAY == kInterWide) {
        float y[16];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            y[2 * j] = x[j];
            y[2 * j + 1] = x[8 + j];
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = y[j];
    }
}

template <int LAY>
__device__ __forceinline__ void load_weight(const Lane& l, const float* w, float* x) {
    if (!w) {
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = 1.f;
        return;
    }
    if constexpr (LAY == kHalfWide || LAY == kInterWide) {
        // weights have no alignment beyond their element
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const int c = j < 8 ? l.oa + j : l.ob + j - 8;
            x[LAY == kInterWide ? (j & 1) * 8 + (j >> 1) : j] = w[c];
        }
    } else {
        Raw<float, LAY> r;
        r.load(l, w);
        r.get(l, x);
    }
}

// The lane's 8 (cos, sin) of a token.
template <int LAY>
__device__ __forceinline__ void load_angles(const Lane& l, const float2* cs, float* co, float* si) {
    if constexpr (LAY == kHalfWide || LAY == kInterWide) {
        const float4* p = reinterpret_cast<const float4*>(cs + (l.live ? 8 * l.c : 0));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float4 v = p[j];
            co[2 * j] = v.x; si[2 * j] = v.y;
            co[2 * j + 1] = v.z; si[2 * j + 1] = v.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int p = l.c + l.lpr * j;
            const float2 v = cs[p < l.P ? p : 0];
            co[j] = v.x;
            si[j] = v.y;
        }
    }
}

// Sum over the lpr lanes of a row, in every one of them: the lane one further, two further, then the
// mirror images in 8 and 16 lanes (whose 4 and 8 lanes hold the same by then), then across.
__device__ __forceinline__ float row_sum(float s, int lpr) {
    if (lpr > 1) s += dpp_f32<0xB1, 0xf>(s);
    if (lpr > 2) s += dpp_f32<0x4E, 0xf>(s);
    if (lpr > 4) s += dpp_f32<0x141, 0xf>(s);
    if (lpr > 8) s += dpp_f32<0x140, 0xf>(s);
    if (lpr > 16) s += __shfl_xor(s, 16);
    if (lpr > 32) s += __shfl_xor(s, 32);
    return s;
}

}  // namespace rope
}  // namespace kda
