// Norms around a block for gfx950 (include/kda_norm.h). Per row of D channels:
//     p = f w_post r1,  r1 = 1 / sqrt(mean(f^2) + eps);   u = sigmoid(gate) p;
//     x' = x + scale lam u;   n = x' w_pre r2,  r2 = 1 / sqrt(mean(x'^2) + pre_eps).
// Backward, from D' = dL/dx' (direct) and dn, with t = dn w_pre and xh = x' r2:
//     dx' = D' + r2 (t - xh mean(t xh)),   dx = dx',   dw_pre = sum_rows dn xh;
//     with fh = f r1 and t1 = dx' s scale lam w_post:  dgate = t1 fh (1 - s),
//     df = r1 (t1 - fh mean(t1 fh));
//     with Q = sum_rows dx' s fh:  dw_post = scale lam Q,   dlam = scale w_post Q.
//
// A row lives in the registers of TPR threads (VEC * NV channels each), so every tensor is read
// once and written once: the kernels are bound by HBM. A workgroup walks rows blockIdx.x * RPB, +
// gridDim.x * RPB, ...; the next rows' loads are in flight while the current ones are worked on, and
// the weights of a thread's channels stay in its registers (reloading them for every row moves more
// through L2 than the row itself). Barriers order LDS alone: one that waited for the row's stores
// too would cost the store's latency in every row.
//
// Rows of any length take 16-byte accesses: vectors lie on 8-element boundaries of the whole tensor,
// so a row's first vector may begin up to 7 elements before the row. Workgroups step by a multiple
// of 8 rows, which keeps that offset, and so every thread's channels, the same for all its rows.
// Only a row's first and last vector are masked.
//
// Measured, bf16 (kernel alone): 8192 rows of 4096 with gate and residual, forward 61 us, 5.5 TB/s,
// backward 104 us, 5.2 TB/s (fp32 122 and 197 us); 262144 rows of 128 with a gate, forward 38.9 us, 5.2
// TB/s, backward 58.2 us, 5.8 TB/s. Without the next rows in flight both directions of the first take
// 205 us instead of 183, one call after the other; with 1024 threads a row, 235. Rows off 8 elements:
// 1001 channels 72 and 132 us for the bytes of the first. 16384 channels reach 71 % (forward) and 55 %
// of the 5.3 TB/s of a copy, 10001 38 % and 17 %.
#pragma once

#include "kda_math.h"
#include "kda_norm.h"
#include "kda_norm_internal.h"

namespace kda {
namespace norm {

// VEC consecutive elements as they lie in memory, in 32-bit words (a lone bf16 in the low half).
template <typename T, int VEC>
struct Raw {
    static constexpr int words = VEC * (int)sizeof(T) < 4 ? 1 : VEC * (int)sizeof(T) / 4;
    uint32_t w[words];
};
template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> load_raw(const T* p) {
    Raw<T, VEC> r;
    if constexpr (sizeof(T) * VEC >= 16) {
#pragma unroll
        for (int i = 0; i < r.words / 4; ++i) reinterpret_cast<uint4*>(r.w)[i] = reinterpret_cast<const uint4*>(p)[i];
    } else {
        static_assert(VEC == 1, "wide rows or single elements");
        if constexpr (sizeof(T) == 2) r.w[0] = *p;
        else r.w[0] = __float_as_uint(*p);
    }
    return r;
}
template <typename T, int VEC>
__device__ __forceinline__ float at(const Raw<T, VEC>& r, int i) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(r.w[i]);
    else return __uint_as_float(i & 1 ? r.w[i / 2] & 0xffff0000u : r.w[i / 2] << 16);
}
// Element i of r, which is zero, becomes that at p.
template <typename T, int VEC>
__device__ __forceinline__ void set(Raw<T, VEC>& r, int i, const T* p) {
    if constexpr (sizeof(T) == 4) r.w[i] = __float_as_uint(*p);
    else r.w[i / 2] |= (uint32_t)*p << (i & 1 ? 16 : 0);
}
template <typename T, int VEC>
__device__ __forceinline__ void clear(Raw<T, VEC>& r, int i) {
    if constexpr (sizeof(T) == 4) r.w[i] = 0;
    else r.w[i / 2] &= i & 1 ? 0xffffu : 0xffff0000u;
}
template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float* x) {
    if constexpr (VEC == 8) {
        store8(p, x);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) st_f(p + i, x[i]);
    }
}

template <int TPR>
struct Geo {
    static constexpr int threads = TPR < 256 ? 256 : TPR;
    static constexpr int rows = threads / TPR;                 // rows at a time
    static constexpr int waves = TPR < 64 ? 1 : TPR / 64;      // waves of a row
};

// Sum over the TPR threads of a row, in a fixed order; every thread gets it. `red`: the row's
// waves x N floats; consecutive sums take different ones.
template <int TPR, int N>
__device__ __forceinline__ void row_sum(float (&s)[N], float* red) {
#pragma unroll
    for (int m = 1; m < (TPR < 64 ? TPR : 64); m <<= 1)
#pragma unroll
        for (int j = 0; j < N; ++j) s[j] += __shfl_xor(s[j], m);
    if constexpr (TPR > 64) {
        constexpr int W = Geo<TPR>::waves;
        const int wv = (threadIdx.x % TPR) >> 6;
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int j = 0; j < N; ++j) red[j * W + wv] = s[j];
        lds_barrier();
#pragma unroll
        for (int j = 0; j < N; ++j) {
            s[j] = 0.f;
#pragma unroll
            for (int i = 0; i < W; ++i) s[j] += red[j * W + i];
        }
    }
}

// 1 / sqrt(v), v > 0. The hardware's root takes subnormal numbers for zero (a row of zeros with an eps
// that small has one); they are scaled by an even power of two.
__device__ __forceinline__ float inv_root(float v) {
    const bool small = v < 0x1p-126f;
    return __builtin_amdgcn_rsqf(small ? v * 0x1p100f : v) * (small ? 0x1p50f : 1.f);
}

// A thread's channels of every row it works on: VEC from col on per vector, those inside [0, D).
// ODD: rows may start off 8 elements. FRESH: which elements of a vector lie in the row is worked out
// anew at every use. Kept over the rows, as the compiler would, the conditions take more scalar
// registers than there are, which 1024 threads feel in the forward (rows of 10001 bf16 channels: 167
// us against 227, 6001: 117 against 127); fewer threads and the backward rather have the issue slots
// (1001, backward: 140 us against 174).
template <int VEC, int NV, int TPR, bool ODD, bool FRESH>
struct Cols {
    int col[NV];
    bool full[NV], any[NV];

    __device__ __forceinline__ void init(const NormArgs& a, int64_t row) {
        const int before = ODD ? (int)((row & 7) * (a.D & 7) & 7) : 0;   // (row * D) mod 8
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            col[j] = (j * TPR + (int)(threadIdx.x % TPR)) * VEC - before;
            any[j] = col[j] < a.D && (!ODD || col[j] + VEC > 0);
            full[j] = ODD ? col[j] >= 0 && col[j] + VEC <= a.D : any[j];
        }
    }
    struct In {   // whether element i of a vector lies in the row
        int col, D;
        bool any;
        __device__ __forceinline__ bool operator()(int i) const {
            return ODD ? col + i >= 0 && col + i < D : any;
        }
    };
    __device__ __forceinline__ In in(const NormArgs& a, int j) const {
        int c = col[j];
        if (FRESH) asm volatile("" : "+v"(c));
        return In{c, (int)a.D, any[j]};
    }
};

// The weights of a thread's channels: lp = scale lam w_post and r = w_pre, which is all either
// direction needs. Kept in registers while there are at most 8 channels, else read at every use.
template <int VEC, int NV, typename C>
struct Weights {
    static constexpr bool KEEP = VEC * NV <= 8;
    float lp[KEEP ? NV : 1][VEC], r[KEEP ? NV : 1][VEC];

    __device__ __forceinline__ void load(const NormArgs& a, const C& c, int j, int slot) {
        float p[VEC], l[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) p[i] = l[i] = r[slot][i] = 1.f;
        if (VEC == 8 && c.full[j]) {   // two 16-byte loads, on 4 bytes where rows start off 8 elements
            auto get = [&](const float* w, float* o) {
                if (w) __builtin_memcpy(o, w + c.col[j], VEC * sizeof(float));
            };
            get(a.w_post, p);
            get(a.lam, l);
            get(a.w_pre, r[slot]);
        } else {
            const auto in = c.in(a, j);
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (in(i)) {
                    if (a.w_post) p[i] = a.w_post[c.col[j] + i];
                    if (a.lam) l[i] = a.lam[c.col[j] + i];
                    if (a.w_pre) r[slot][i] = a.w_pre[c.col[j] + i];
                }
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) lp[slot][i] = a.scale * l[i] * p[i];
    }
    __device__ __forceinline__ void init(const NormArgs& a, const C& c) {
        if constexpr (KEEP)
#pragma unroll
            for (int j = 0; j < NV; ++j) load(a, c, j, j);
    }
    // the slot that holds vector j's weights
    __device__ __forceinline__ int at(const NormArgs& a, const C& c, int j) {
        if constexpr (KEEP) return j;
        load(a, c, j, 0);
        return 0;
    }
};

// The vector of a row at element `at`, or zeros where the thread has none (`on` false). A vector
// that would reach past the tensor's `total` elements is read one by one.
template <bool ODD, typename T, int VEC>
__device__ __forceinline__ void fetch(Raw<T, VEC>& r, const void* p, int64_t at, int64_t total, bool on) {
    if (on && (!ODD || at + VEC <= total)) {
        r = load_raw<T, VEC>((const T*)p + at);
    } else {
#pragma unroll
        for (int i = 0; i < r.words; ++i) r.w[i] = 0;
        if (ODD && on) {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (at + i < total) set(r, i, (const T*)p + at + i);
        }
    }
}
// Zeros for a partial vector's elements outside the row (the neighbouring rows').
template <typename T, int VEC, typename C>
__device__ __forceinline__ void mask(Raw<T, VEC>& r, const NormArgs& a, const C& c, int j) {
    const auto in = c.in(a, j);
#pragma unroll
    for (int i = 0; i < VEC; ++i)
        if (!in(i)) clear(r, i);
}
template <typename T, int VEC, int NV, int TPR, bool ODD, bool FRESH>
__device__ __forceinline__ void put(void* p, int64_t at, const float* x, const NormArgs& a,
                                    const Cols<VEC, NV, TPR, ODD, FRESH>& c, int j) {
    if (c.full[j]) {
        store_vec<T, VEC>((T*)p + at, x);
    } else if (ODD && c.any[j]) {
        const auto in = c.in(a, j);
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (in(i)) st_f((T*)p + at + i, x[i]);
    }
}

template <typename TI, typename TR, typename TO, int VEC, int NV, int TPR, bool ODD>
__global__ __launch_bounds__(Geo<TPR>::threads) void norm_fwd_kernel(NormArgs a) {
    constexpr int RPB = Geo<TPR>::rows, W = Geo<TPR>::waves;
    constexpr bool AHEAD = VEC * NV <= 8;   // more channels leave no registers for a second row
    __shared__ float red[2][2][RPB][W];
    const int grp = threadIdx.x / TPR;
    const float inv = 1.f / (float)a.D;
    const int64_t step = (int64_t)gridDim.x * RPB, total = a.rows * a.D;
    int64_t row = (int64_t)blockIdx.x * RPB + grp;
    using C = Cols<VEC, NV, TPR, ODD, ODD && TPR == 1024>;
    C co;
    co.init(a, row);
    Weights<VEC, NV, C> wt;
    Raw<TI, VEC> f[NV], g[NV], fn[NV], gn[NV];
    Raw<TR, VEC> x[NV], xn[NV];
    auto next = [&](int64_t at_row) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const bool on = at_row < a.rows && co.any[j];
            const int64_t at = at_row * a.D + co.col[j];
            fetch<ODD>(fn[j], a.f, at, total, on);
            if (a.gate) fetch<ODD>(gn[j], a.gate, at, total, on);
            if (a.x) fetch<ODD>(xn[j], a.x, at, total, on);
        }
    };
    if (AHEAD) next(row);
    wt.init(a, co);
    int phase = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < a.rows; row0 += step, row += step, phase ^= 1) {
        const int64_t base = row * a.D;
        const bool live = row < a.rows;
        if (!AHEAD) next(row);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            f[j] = fn[j]; g[j] = gn[j]; x[j] = xn[j];
            if (ODD && co.any[j] && !co.full[j]) { mask(f[j], a, co, j); mask(g[j], a, co, j); mask(x[j], a, co, j); }
        }
        if (AHEAD && row0 + step < a.rows) next(row + step);
        float r1 = 1.f;
        if (a.post) {
            float s[1] = {0.f};
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < VEC; ++i) s[0] = fmaf(at(f[j], i), at(f[j], i), s[0]);
            row_sum<TPR>(s, red[phase][0][grp]);
            r1 = inv_root(fmaf(s[0], inv, a.eps));
        }
        float xo[NV][VEC];
        float s2[1] = {0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int k = wt.at(a, co, j);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                xo[j][i] = at(f[j], i) * r1 * wt.lp[k][i];
                if (a.gate) xo[j][i] *= sigmoid_f(at(g[j], i));
                if (a.x) xo[j][i] += at(x[j], i);
                s2[0] = fmaf(xo[j][i], xo[j][i], s2[0]);
            }
            if (a.x_out && live) put<TR>(a.x_out, base + co.col[j], xo[j], a, co, j);
        }
        if (!a.pre) continue;
        row_sum<TPR>(s2, red[phase][1][grp]);
        const float r2 = inv_root(fmaf(s2[0], inv, a.pre_eps));
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int k = wt.at(a, co, j);
            float n[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) n[i] = xo[j][i] * r2 * wt.r[k][i];
            if (live) put<TO>(a.n, base + co.col[j], n, a, co, j);
        }
    }
}

// Two rows of all five tensors, the weights and the column sums: 128 registers hold them for wide
// bf16 rows (4 waves a SIMD), 256 for the others. Rows of 512 threads on 8 elements spill at 128 and
// run one workgroup a CU anyhow.
template <typename TI, typename TR, typename TO, int VEC, int NV, int TPR, bool ODD>
constexpr int bwd_waves() {
    return TPR == 1024 || (VEC == 8 && (TPR != 512 || ODD) && 2 * sizeof(TI) + 2 * sizeof(TR) + sizeof(TO) <= 10) ? 4 : 2;
}

template <typename TI, typename TR, typename TO, int VEC, int NV, int TPR, bool ODD>
__global__ __launch_bounds__(Geo<TPR>::threads, (bwd_waves<TI, TR, TO, VEC, NV, TPR, ODD>())) void norm_bwd_kernel(NormArgs a) {
    constexpr int RPB = Geo<TPR>::rows, W = Geo<TPR>::waves, C = VEC * NV * TPR;
    // past 8 channels a thread (1024 threads, 128 registers each) the column sums live in LDS, one
    // row is in flight, and the gate and x' are computed again instead of kept
    constexpr bool LEAN = VEC * NV > 8;
    __shared__ float red[2][RPB][4][W];
    __shared__ float colsum[LEAN ? 2 * C : RPB > 1 ? RPB * C : 1];
    const int lane = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    const float inv = 1.f / (float)a.D;
    const int64_t step = (int64_t)gridDim.x * RPB, total = a.rows * a.D;
    int64_t row = (int64_t)blockIdx.x * RPB + grp;
    using Co = Cols<VEC, NV, TPR, ODD, false>;
    Co co;
    co.init(a, row);
    Weights<VEC, NV, Co> wt;
    float acc[2][LEAN ? 1 : NV][VEC];      // this thread's columns of Q and dw_pre
    auto slot = [&](int k, int j, int i) -> float& {
        if constexpr (LEAN) return colsum[k * C + (j * VEC + i) * TPR + lane];
        else return acc[k][j][i];
    };
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) slot(k, j, i) = 0.f;
    Raw<TI, VEC> f[NV], g[NV], fn[NV], gn[NV];
    Raw<TR, VEC> x[NV], dxo[NV], xn[NV], dxon[NV];
    Raw<TO, VEC> dn[NV], dnn[NV];
    auto next = [&](int64_t at_row) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const bool on = at_row < a.rows && co.any[j];
            const int64_t at = at_row * a.D + co.col[j];
            fetch<ODD>(fn[j], a.f, at, total, on);
            if (a.gate) fetch<ODD>(gn[j], a.gate, at, total, on);
            if (a.x && a.dn) fetch<ODD>(xn[j], a.x, at, total, on);
            if (a.dx_out) fetch<ODD>(dxon[j], a.dx_out, at, total, on);
            if (a.dn) fetch<ODD>(dnn[j], a.dn, at, total, on);
        }
    };
    if (!LEAN) next(row);
    wt.init(a, co);
    int phase = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < a.rows; row0 += step, row += step, phase ^= 1) {
        const int64_t base = row * a.D;
        const bool live = row < a.rows;
        if (LEAN) next(row);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            f[j] = fn[j]; g[j] = gn[j]; x[j] = xn[j]; dxo[j] = dxon[j]; dn[j] = dnn[j];
            if (ODD && co.any[j] && !co.full[j]) {
                mask(f[j], a, co, j); mask(g[j], a, co, j); mask(x[j], a, co, j);
                mask(dxo[j], a, co, j); mask(dn[j], a, co, j);
            }
        }
        if (!LEAN && row0 + step < a.rows) next(row + step);
        float r1 = 1.f;
        if (a.post) {
            float s[1] = {0.f};
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < VEC; ++i) s[0] = fmaf(at(f[j], i), at(f[j], i), s[0]);
            row_sum<TPR>(s, red[phase][grp][0]);
            r1 = inv_root(fmaf(s[0], inv, a.eps));
        }
        // the gate; x' again, and the pre-norm's part of its gradient
        float r2 = 0.f, m2 = 0.f;
        float sg[LEAN ? 1 : NV][VEC], xo[LEAN ? 1 : NV][VEC];
        auto again = [&](int j, int k, int q) {   // gate and x' of vector j into slot q, weights in slot k
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                sg[q][i] = a.gate ? sigmoid_f(at(g[j], i)) : 1.f;
                xo[q][i] = at(f[j], i) * r1 * wt.lp[k][i] * sg[q][i];
                if (a.x) xo[q][i] += at(x[j], i);
            }
        };
        if (!LEAN || a.dn) {
            float s[2] = {0.f, 0.f};
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int k = wt.at(a, co, j), q = LEAN ? 0 : j;
                again(j, k, q);
                if (!a.dn) continue;
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    s[0] = fmaf(xo[q][i], xo[q][i], s[0]);
                    s[1] = fmaf(at(dn[j], i) * wt.r[k][i], xo[q][i], s[1]);
                }
            }
            if (a.dn) {
                row_sum<TPR>(s, red[phase][grp][1]);
                r2 = inv_root(fmaf(s[0], inv, a.pre_eps));
                m2 = s[1] * inv * r2;   // mean(t xh)
            }
        }
        float t1[NV][VEC];
        float s3[1] = {0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int k = wt.at(a, co, j), q = LEAN ? 0 : j;
            if (LEAN) again(j, k, q);
            float dxv[VEC], dgv[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                float dx = a.dx_out ? at(dxo[j], i) : 0.f;
                if (a.dn) {
                    const float xh = xo[q][i] * r2, d = at(dn[j], i);
                    slot(1, j, i) = fmaf(d, xh, slot(1, j, i));
                    dx += r2 * (d * wt.r[k][i] - xh * m2);
                }
                dxv[i] = dx;
                const float fh = at(f[j], i) * r1, ds = dx * sg[q][i];
                slot(0, j, i) = fmaf(ds, fh, slot(0, j, i));
                t1[j][i] = ds * wt.lp[k][i];
                const float tf = t1[j][i] * fh;
                dgv[i] = tf * (1.f - sg[q][i]);
                s3[0] += tf;
            }
            if (a.dx && live) put<TR>(a.dx, base + co.col[j], dxv, a, co, j);
            if (a.gate && live) put<TI>(a.dgate, base + co.col[j], dgv, a, co, j);
        }
        float m1 = 0.f;
        if (a.post) {
            row_sum<TPR>(s3, red[phase][grp][3]);
            m1 = s3[0] * inv;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float d[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) d[i] = a.post ? r1 * (t1[j][i] - at(f[j], i) * r1 * m1) : t1[j][i];
            if (live) put<TI>(a.df, base + co.col[j], d, a, co, j);
        }
    }
    if (!a.ws) return;
    // this workgroup's column sums, over its row groups through LDS, to the workspace
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float* ws = a.ws + ((int64_t)blockIdx.x * 2 + k) * a.D;
        if constexpr (RPB > 1) {
            lds_barrier();
            for (int c = threadIdx.x; c < RPB * C; c += Geo<TPR>::threads) colsum[c] = 0.f;
            lds_barrier();
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (co.in(a, j)(i)) colsum[grp * C + co.col[j] + i] = slot(k, j, i);
            lds_barrier();
            for (int c = threadIdx.x; c < a.D; c += Geo<TPR>::threads) {
                float s = 0.f;
                for (int r = 0; r < RPB; ++r) s += colsum[r * C + c];
                ws[c] = s;
            }
        } else {
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (co.in(a, j)(i)) ws[co.col[j] + i] = slot(k, j, i);
        }
    }
}

template <typename TI, typename TR, typename TO, int VEC, int NV, int TPR, bool ODD>
static hipError_t launch_g(const NormArgs& a, bool bwd, hipStream_t st) {
    constexpr int RPB = Geo<TPR>::rows, threads = Geo<TPR>::threads;
    const int64_t blocks = (a.rows + RPB - 1) / RPB;
    const int reads = 1 + !!a.gate + (a.x && a.dn) + !!a.dx_out + !!a.dn;
    const int most = bwd ? bwd_groups(threads, VEC == 8 && !ODD ? reads : 0) : fwd_groups(threads);
    const int groups = blocks < most ? (int)blocks : most;
    if (!bwd) {
        hipLaunchKernelGGL((norm_fwd_kernel<TI, TR, TO, VEC, NV, TPR, ODD>), dim3(groups), dim3(threads), 0, st, a);
        return hipGetLastError();
    }
    if (groups > 0)
        hipLaunchKernelGGL((norm_bwd_kernel<TI, TR, TO, VEC, NV, TPR, ODD>), dim3(groups), dim3(threads), 0, st, a);
    if (a.dw_post || a.dlam || a.dw_pre) return launch_colsum(a, groups, st);
    return hipGetLastError();
}

// Whether every tensor and weight starts on 16 bytes.
static bool wide(const NormArgs& a) {
    uintptr_t bits = 0;
    for (const void* p : {a.f, a.gate, a.x, (const void*)a.x_out, (const void*)a.n, a.dx_out, a.dn, (const void*)a.df,
                          (const void*)a.dgate, (const void*)a.dx, (const void*)a.w_post, (const void*)a.lam,
                          (const void*)a.w_pre})
        bits |= reinterpret_cast<uintptr_t>(p);
    return (bits & 15) == 0;
}

// Threads per row by its length (up to 7 elements more where rows do not start on 8), 8 channels a
// thread up to 8192; one channel at a time where a tensor does not start on 16 bytes.
template <typename TI, typename TR, typename TO, bool ODD>
static hipError_t launch_w(const NormArgs& a, int64_t span, bool bwd, hipStream_t st) {
    if (span <= 64) return launch_g<TI, TR, TO, 8, 1, 8, ODD>(a, bwd, st);
    if (span <= 128) return launch_g<TI, TR, TO, 8, 1, 16, ODD>(a, bwd, st);
    if (span <= 256) return launch_g<TI, TR, TO, 8, 1, 32, ODD>(a, bwd, st);
    if (span <= 512) return launch_g<TI, TR, TO, 8, 1, 64, ODD>(a, bwd, st);
    if (span <= 1024) return launch_g<TI, TR, TO, 8, 1, 128, ODD>(a, bwd, st);
    if (span <= 2048) return launch_g<TI, TR, TO, 8, 1, 256, ODD>(a, bwd, st);
    if (span <= 4096) return launch_g<TI, TR, TO, 8, 1, 512, ODD>(a, bwd, st);
    if (span <= 8192) return launch_g<TI, TR, TO, 8, 1, 1024, ODD>(a, bwd, st);
    return launch_g<TI, TR, TO, 8, 2, 1024, ODD>(a, bwd, st);
}

template <typename TI, typename TR, typename TO>
static hipError_t launch_t(const NormArgs& a, bool bwd, hipStream_t st) {
    if (wide(a) && a.D % 8 == 0) return launch_w<TI, TR, TO, false>(a, a.D, bwd, st);
    // past 8192 channels off 8 elements, fp32 vectors of the backward spill more than single channels
    // cost (10001 channels: 1042 us against 735; bf16 585 against 846)
    const bool spills = bwd && sizeof(TI) == 4 && a.D + 7 > 8192;
    if (wide(a) && a.D + 7 <= KDA_NORM_MAX_D && !spills) return launch_w<TI, TR, TO, true>(a, a.D + 7, bwd, st);
    if (a.D <= 512) return launch_g<TI, TR, TO, 1, 8, 64, false>(a, bwd, st);
    if (a.D <= 4096) return launch_g<TI, TR, TO, 1, 8, 512, false>(a, bwd, st);
    return launch_g<TI, TR, TO, 1, 16, 1024, false>(a, bwd, st);
}

template <typename TI>
hipError_t launch_i(const NormArgs& a, bool bwd, hipStream_t st) {
    if (a.res_bf16 && a.out_bf16) return launch_t<TI, bf16_t, bf16_t>(a, bwd, st);
    if (a.res_bf16) return launch_t<TI, bf16_t, float>(a, bwd, st);
    if (a.out_bf16) return launch_t<TI, float, bf16_t>(a, bwd, st);
    return launch_t<TI, float, float>(a, bwd, st);
}

}  // namespace norm
}  // namespace kda
