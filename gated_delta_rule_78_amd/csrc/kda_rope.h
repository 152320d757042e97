// Device code shared by the head norms with rotation and the cache append (include/kda_attn.h).
//
// A workgroup of 256 threads takes the rows (token, head) of a few tokens. The tokens' cosines and
// sines are formed once, in LDS, and serve every head. A row is held by `lpr` lanes, 8 pairs a lane
// (both members of a pair in one lane, so a rotation needs no exchange), 64 / lpr rows a wave at a
// time and kUnroll of those in flight.
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

// Per token of a workgroup: element offsets of its rows in every tensor.
struct Token {
    int64_t q, k, v, qo, ko, vo;
    int64_t sdq, sdk;
    int32_t pos;
    int32_t live;     // in a sequence: q is read and written
    int32_t stored;   // append: k and v have a place in the cache
};

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
        const int t = e / P, i = e - t * P;
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

template <typename T>
struct Raw;
template <>
struct Raw<bf16_t> {
    uint4 a, b;
};
template <>
struct Raw<float> {
    uint4 a0, a1, b0, b1;
};

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
    } else if (LAY == kHalfWide) {
        const int p = 8 * l.c;
        l.live = p < l.P;
        l.oa = p < l.R ? p : l.R + p;                     // rot + (p - rot/2)
        l.ob = p < l.R ? p + l.R : l.R + l.H2 + p;
    } else {
        l.live = true;
        l.oa = l.ob = 0;
    }
    return l;
}

template <typename T, int LAY>
__device__ __forceinline__ void load_row(const Lane& l, const T* row, bool on, float* x);

__device__ __forceinline__ void unpack8(const bf16_t* p, float* x) { unpack16(*reinterpret_cast<const uint4*>(p), p, x); }
__device__ __forceinline__ void unpack8(const float* p, float* x) {
    unpack16(*reinterpret_cast<const uint4*>(p), p, x);
    unpack16(*reinterpret_cast<const uint4*>(p + 4), p, x + 4);
}

// x[0..7] the first members of the lane's pairs, x[8..15] the second.
template <typename T, int LAY>
__device__ __forceinline__ void load_row(const Lane& l, const T* row, bool on, float* x) {
    if constexpr (LAY == kHalfWide || LAY == kInterWide) {
        if (on && l.live) {
            unpack8(row + l.oa, x);
            unpack8(row + l.ob, x + 8);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) x[j] = 0.f;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int p = l.c + l.lpr * j;
            const bool in = on && p < l.P;
            x[j] = in ? ld_f(row + l.ia<LAY>(p)) : 0.f;
            x[8 + j] = in ? ld_f(row + l.ib<LAY>(p)) : 0.f;
        }
    }
}

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

// Interleaved wide loads hold channels in order: into first and second members, and back.
template <int LAY>
__device__ __forceinline__ void to_pairs(float* x) {
    if constexpr (LAY == kInterWide) {
        float y[16];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            y[j] = x[2 * j];
            y[8 + j] = x[2 * j + 1];
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = y[j];
    }
}
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
        for (int j = 0; j < 8; ++j) {
            x[j] = l.live ? w[l.oa + j] : 0.f;
            x[8 + j] = l.live ? w[l.ob + j] : 0.f;
        }
        to_pairs<LAY>(x);
    } else {
        load_row<float, LAY>(l, w, true, x);
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

__device__ __forceinline__ float row_sum(float s, int lpr) {
    for (int m = 1; m < lpr; m <<= 1) s += __shfl_xor(s, m);
    return s;
}

// Quotient of a row index by the heads: exact for n < 2^16 with magic = ceil(2^32 / h) (h > 1).
__device__ __forceinline__ int div_heads(int n, uint32_t magic) {
    return magic ? (int)__umulhi((uint32_t)n, magic) : n;
}

struct Shape {
    int lpr;            // lanes a row
    int tokens;         // a workgroup
    uint32_t mq, mk;    // ceil(2^32 / heads), 0 for one head
};

}  // namespace rope
}  // namespace kda
