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
#include "kda_math.h"
#include "kda_norm_internal.h"

namespace kda {
namespace norm {

// VEC consecutive elements as they lie in memory.
template <typename T, int VEC>
struct Raw {
    T v[VEC];
};
template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> load_raw(const T* p) {
    Raw<T, VEC> r;
    if constexpr (sizeof(T) * VEC >= 16) {
#pragma unroll
        for (int i = 0; i < (int)(sizeof(T) * VEC / 16); ++i)
            reinterpret_cast<uint4*>(r.v)[i] = reinterpret_cast<const uint4*>(p)[i];
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) r.v[i] = p[i];
    }
    return r;
}
template <typename T, int VEC>
__device__ __forceinline__ float at(const Raw<T, VEC>& r, int i) { return ld_f(&r.v[i]); }
template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float* x) {
    if constexpr (VEC == 8) {
        store8(p, x);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) st_f(p + i, x[i]);
    }
}
template <int VEC>
__device__ __forceinline__ void load_w(const float* w, int64_t col, float* out) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) out[i] = w ? w[col + i] : 1.f;
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

// The weights of a thread's channels: lp = scale lam w_post and r = w_pre, which is all either
// direction needs. Kept in registers while there are at most 8 channels, else read at every use.
template <int VEC, int NV, int TPR>
struct Weights {
    static constexpr bool KEEP = VEC * NV <= 8;
    float lp[KEEP ? NV : 1][VEC], r[KEEP ? NV : 1][VEC];

    __device__ __forceinline__ static void fetch(const float* w, int col, float* o) {
        if (!w) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) o[i] = 1.f;
        } else if constexpr (VEC == 8) {
            reinterpret_cast<float4*>(o)[0] = reinterpret_cast<const float4*>(w + col)[0];
            reinterpret_cast<float4*>(o)[1] = reinterpret_cast<const float4*>(w + col)[1];
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) o[i] = w[col + i];
        }
    }
    __device__ __forceinline__ void load(const NormArgs& a, int j, int slot) {
        int col = (j * TPR + (int)(threadIdx.x % TPR)) * VEC;
        if (col >= a.D) col = 0;      // not used
        float p[VEC], l[VEC];
        fetch(a.w_post, col, p);
        fetch(a.lam, col, l);
        fetch(a.w_pre, col, r[slot]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) lp[slot][i] = a.scale * l[i] * p[i];
    }
    __device__ __forceinline__ void init(const NormArgs& a) {
        if constexpr (KEEP)
#pragma unroll
            for (int j = 0; j < NV; ++j) load(a, j, j);
    }
    // the slot that holds vector j's weights
    __device__ __forceinline__ int at(const NormArgs& a, int j) {
        if constexpr (KEEP) return j;
        load(a, j, 0);
        return 0;
    }
};

// Loads vector j of a row, or zeros past the row's channels or past the rows.
template <typename T, int VEC>
__device__ __forceinline__ void fetch(Raw<T, VEC>& r, const void* p, int64_t at, bool on) {
    if (on) r = load_raw<T, VEC>((const T*)p + at);
    else
#pragma unroll
        for (int i = 0; i < VEC; ++i) r.v[i] = 0;
}

template <typename TI, typename TR, typename TO, int VEC, int NV, int TPR>
__global__ __launch_bounds__(Geo<TPR>::threads) void norm_fwd_kernel(NormArgs a) {
    constexpr int RPB = Geo<TPR>::rows, W = Geo<TPR>::waves;
    __shared__ float red[2][2][RPB][W];
    const int lane = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    const float inv = 1.f / (float)a.D;
    Weights<VEC, NV, TPR> wt;
    Raw<TI, VEC> f[NV], g[NV], fn[NV], gn[NV];
    Raw<TR, VEC> x[NV], xn[NV];
    const int64_t step = (int64_t)gridDim.x * RPB;
    int64_t row = (int64_t)blockIdx.x * RPB + grp;
    auto next = [&](int64_t at) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = (j * TPR + lane) * VEC;
            const bool on = at < a.rows && col < a.D;
            fetch(fn[j], a.f, at * a.D + col, on);
            if (a.gate) fetch(gn[j], a.gate, at * a.D + col, on);
            if (a.x) fetch(xn[j], a.x, at * a.D + col, on);
        }
    };
    constexpr bool AHEAD = VEC * NV <= 8;   // more channels leave no registers for a second row
    if (AHEAD) next(row);
    wt.init(a);
    int phase = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < a.rows; row0 += step, row += step, phase ^= 1) {
        const int64_t base = row * a.D;
        if (!AHEAD) next(row);
#pragma unroll
        for (int j = 0; j < NV; ++j) { f[j] = fn[j]; g[j] = gn[j]; x[j] = xn[j]; }
        if (AHEAD && row0 + step < a.rows) next(row + step);
        float r1 = 1.f;
        if (a.post) {
            float s[1] = {0.f};
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < VEC; ++i) s[0] = fmaf(at(f[j], i), at(f[j], i), s[0]);
            row_sum<TPR>(s, red[phase][0][grp]);
            r1 = __builtin_amdgcn_rsqf(fmaf(s[0], inv, a.eps));
        }
        float xo[NV][VEC];
        float s2[1] = {0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = (j * TPR + lane) * VEC, k = wt.at(a, j);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                xo[j][i] = at(f[j], i) * r1 * wt.lp[k][i];
                if (a.gate) xo[j][i] *= sigmoid_f(at(g[j], i));
                if (a.x) xo[j][i] += at(x[j], i);
                s2[0] = fmaf(xo[j][i], xo[j][i], s2[0]);
            }
            if (a.x_out && row < a.rows && col < a.D) store_vec<TR, VEC>((TR*)a.x_out + base + col, xo[j]);
        }
        if (!a.pre) continue;
        row_sum<TPR>(s2, red[phase][1][grp]);
        const float r2 = __builtin_amdgcn_rsqf(fmaf(s2[0], inv, a.pre_eps));
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = (j * TPR + lane) * VEC, k = wt.at(a, j);
            float n[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) n[i] = xo[j][i] * r2 * wt.r[k][i];
            if (row < a.rows && col < a.D) store_vec<TO, VEC>((TO*)a.n + base + col, n);
        }
    }
}

// Two rows of all five tensors, the weights and the column sums: 128 registers hold them for wide
// bf16 rows (4 waves a SIMD), 256 for the others.
template <typename TI, typename TR, typename TO, int VEC, int NV, int TPR>
constexpr int bwd_waves() {
    return TPR == 1024 || (VEC == 8 && 2 * sizeof(TI) + 2 * sizeof(TR) + sizeof(TO) <= 10) ? 4 : 2;
}

template <typename TI, typename TR, typename TO, int VEC, int NV, int TPR>
__global__ __launch_bounds__(Geo<TPR>::threads, (bwd_waves<TI, TR, TO, VEC, NV, TPR>())) void norm_bwd_kernel(NormArgs a) {
    constexpr int RPB = Geo<TPR>::rows, W = Geo<TPR>::waves;
    __shared__ float red[2][RPB][4][W];
    __shared__ float colsum[RPB > 1 ? RPB * VEC * NV * TPR : 1];
    const int lane = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    const float inv = 1.f / (float)a.D;
    Weights<VEC, NV, TPR> wt;
    float acc[2][NV][VEC];      // this thread's columns of Q and dw_pre
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[k][j][i] = 0.f;
    Raw<TI, VEC> f[NV], g[NV], fn[NV], gn[NV];
    Raw<TR, VEC> x[NV], dxo[NV], xn[NV], dxon[NV];
    Raw<TO, VEC> dn[NV], dnn[NV];
    const int64_t step = (int64_t)gridDim.x * RPB;
    int64_t row = (int64_t)blockIdx.x * RPB + grp;
    auto next = [&](int64_t at) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = (j * TPR + lane) * VEC;
            const bool on = at < a.rows && col < a.D;
            fetch(fn[j], a.f, at * a.D + col, on);
            if (a.gate) fetch(gn[j], a.gate, at * a.D + col, on);
            if (a.x && a.dn) fetch(xn[j], a.x, at * a.D + col, on);
            if (a.dx_out) fetch(dxon[j], a.dx_out, at * a.D + col, on);
            if (a.dn) fetch(dnn[j], a.dn, at * a.D + col, on);
        }
    };
    constexpr bool AHEAD = VEC * NV <= 8;
    if (AHEAD) next(row);
    wt.init(a);
    int phase = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < a.rows; row0 += step, row += step, phase ^= 1) {
        const int64_t base = row * a.D;
        if (!AHEAD) next(row);
#pragma unroll
        for (int j = 0; j < NV; ++j) { f[j] = fn[j]; g[j] = gn[j]; x[j] = xn[j]; dxo[j] = dxon[j]; dn[j] = dnn[j]; }
        if (AHEAD && row0 + step < a.rows) next(row + step);
        float r1 = 1.f;
        if (a.post) {
            float s[1] = {0.f};
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < VEC; ++i) s[0] = fmaf(at(f[j], i), at(f[j], i), s[0]);
            row_sum<TPR>(s, red[phase][grp][0]);
            r1 = __builtin_amdgcn_rsqf(fmaf(s[0], inv, a.eps));
        }
        // the gate; x' again, and the pre-norm's part of its gradient
        float r2 = 0.f, m2 = 0.f;
        float sg[NV][VEC], xo[NV][VEC];
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) sg[j][i] = a.gate ? sigmoid_f(at(g[j], i)) : 1.f;
        if (a.dn) {
            float s[2] = {0.f, 0.f};
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int k = wt.at(a, j);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    xo[j][i] = at(f[j], i) * r1 * wt.lp[k][i] * sg[j][i];
                    if (a.x) xo[j][i] += at(x[j], i);
                    s[0] = fmaf(xo[j][i], xo[j][i], s[0]);
                    s[1] = fmaf(at(dn[j], i) * wt.r[k][i], xo[j][i], s[1]);
                }
            }
            row_sum<TPR>(s, red[phase][grp][1]);
            r2 = __builtin_amdgcn_rsqf(fmaf(s[0], inv, a.pre_eps));
            m2 = s[1] * inv * r2;   // mean(t xh)
        }
        float t1[NV][VEC];
        float s3[1] = {0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = (j * TPR + lane) * VEC, k = wt.at(a, j);
            const bool out = row < a.rows && col < a.D;
            float dxv[VEC], dgv[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                float dx = a.dx_out ? at(dxo[j], i) : 0.f;
                if (a.dn) {
                    const float xh = xo[j][i] * r2, d = at(dn[j], i);
                    acc[1][j][i] = fmaf(d, xh, acc[1][j][i]);
                    dx += r2 * (d * wt.r[k][i] - xh * m2);
                }
                dxv[i] = dx;
                const float fh = at(f[j], i) * r1, ds = dx * sg[j][i];
                acc[0][j][i] = fmaf(ds, fh, acc[0][j][i]);
                t1[j][i] = ds * wt.lp[k][i];
                const float tf = t1[j][i] * fh;
                dgv[i] = tf * (1.f - sg[j][i]);
                s3[0] += tf;
            }
            if (a.dx && out) store_vec<TR, VEC>((TR*)a.dx + base + col, dxv);
            if (a.gate && out) store_vec<TI, VEC>((TI*)a.dgate + base + col, dgv);
        }
        float m1 = 0.f;
        if (a.post) {
            row_sum<TPR>(s3, red[phase][grp][3]);
            m1 = s3[0] * inv;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = (j * TPR + lane) * VEC;
            float d[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) d[i] = a.post ? r1 * (t1[j][i] - at(f[j], i) * r1 * m1) : t1[j][i];
            if (row < a.rows && col < a.D) store_vec<TI, VEC>((TI*)a.df + base + col, d);
        }
    }
    if (!a.ws) return;
    // this workgroup's column sums: over its row groups through LDS, then to the workspace
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float* ws = a.ws + ((int64_t)blockIdx.x * 2 + k) * a.D;
        if constexpr (RPB > 1) {
            constexpr int C = VEC * NV * TPR;
            lds_barrier();
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < VEC; ++i) colsum[grp * C + (j * TPR + lane) * VEC + i] = acc[k][j][i];
            lds_barrier();
            for (int c = threadIdx.x; c < a.D; c += Geo<TPR>::threads) {
                float s = 0.f;
                for (int r = 0; r < RPB; ++r) s += colsum[r * C + c];
                ws[c] = s;
            }
        } else {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int col = (j * TPR + lane) * VEC;
                if (col < a.D)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) ws[col + i] = acc[k][j][i];
            }
        }
    }
}

// Weight gradients from the workgroups' sums [groups][2][D]: 16 runs of workgroups a column, each
// summed in order by a thread, joined in LDS in order.
__global__ __launch_bounds__(1024) void norm_colsum_kernel(NormArgs a, int groups) {
    __shared__ float part[16][64];
    const int lane = threadIdx.x & 63, run = threadIdx.x >> 6, k = blockIdx.y;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    if (k == 0 ? !a.dw_post && !a.dlam : !a.dw_pre) return;
    const int each = (groups + 15) / 16, g1 = (run + 1) * each < groups ? (run + 1) * each : groups;
    float s = 0.f;
    if (c < a.D) {
#pragma unroll 8
        for (int g = run * each; g < g1; ++g) s += a.ws[((int64_t)g * 2 + k) * a.D + c];
    }
    part[run][lane] = s;
    lds_barrier();
    if (run != 0 || c >= a.D) return;
#pragma unroll
    for (int i = 1; i < 16; ++i) s += part[i][lane];
    if (k == 1) {
        a.dw_pre[c] = s;
        return;
    }
    if (a.dw_post) a.dw_post[c] = s * a.scale * (a.lam ? a.lam[c] : 1.f);
    if (a.dlam) a.dlam[c] = s * a.scale * (a.w_post ? a.w_post[c] : 1.f);
}

// Workgroups at most: what 256 CUs hold at a time (16 waves a CU in the backward, whose column sums
// cost traffic per workgroup; 24 in the forward).
static int fwd_groups(int threads) { return 256 * 24 * 64 / threads; }
static int bwd_groups(int threads) { return 256 * 16 * 64 / threads; }

template <typename TI, typename TR, typename TO, int VEC, int NV, int TPR>
static hipError_t launch_g(const NormArgs& a, bool bwd, hipStream_t st) {
    constexpr int RPB = Geo<TPR>::rows, threads = Geo<TPR>::threads;
    const int64_t blocks = (a.rows + RPB - 1) / RPB;
    const int most = bwd ? bwd_groups(threads) : fwd_groups(threads);
    const int groups = blocks < most ? (int)blocks : most;
    if (!bwd) {
        hipLaunchKernelGGL((norm_fwd_kernel<TI, TR, TO, VEC, NV, TPR>), dim3(groups), dim3(threads), 0, st, a);
        return hipGetLastError();
    }
    if (groups > 0)
        hipLaunchKernelGGL((norm_bwd_kernel<TI, TR, TO, VEC, NV, TPR>), dim3(groups), dim3(threads), 0, st, a);
    if (a.dw_post || a.dlam || a.dw_pre)
        hipLaunchKernelGGL(norm_colsum_kernel, dim3((unsigned)((a.D + 63) / 64), 2), dim3(1024), 0, st, a, groups);
    return hipGetLastError();
}

// Threads per row and channels per thread by D: 16-byte accesses where every row starts on 16
// bytes (D a multiple of 8 and such bases), else one channel at a time.
static bool wide(const NormArgs& a) {
    uintptr_t bits = 0;
    for (const void* p : {a.f, a.gate, a.x, (const void*)a.x_out, (const void*)a.n, a.dx_out, a.dn, (const void*)a.df,
                          (const void*)a.dgate, (const void*)a.dx, (const void*)a.w_post, (const void*)a.lam,
                          (const void*)a.w_pre})
        bits |= reinterpret_cast<uintptr_t>(p);
    return a.D % 8 == 0 && (bits & 15) == 0;
}

template <typename TI, typename TR, typename TO>
static hipError_t launch_t(const NormArgs& a, bool bwd, hipStream_t st) {
    if (wide(a)) {
        if (a.D <= 128) return launch_g<TI, TR, TO, 8, 1, 16>(a, bwd, st);
        if (a.D <= 512) return launch_g<TI, TR, TO, 8, 1, 64>(a, bwd, st);
        if (a.D <= 1024) return launch_g<TI, TR, TO, 8, 1, 128>(a, bwd, st);
        if (a.D <= 2048) return launch_g<TI, TR, TO, 8, 1, 256>(a, bwd, st);
        if (a.D <= 4096) return launch_g<TI, TR, TO, 8, 1, 512>(a, bwd, st);
        if (a.D <= 8192) return launch_g<TI, TR, TO, 8, 1, 1024>(a, bwd, st);
        return launch_g<TI, TR, TO, 8, 2, 1024>(a, bwd, st);
    }
    if (a.D <= 128) return launch_g<TI, TR, TO, 1, 8, 16>(a, bwd, st);
    if (a.D <= 512) return launch_g<TI, TR, TO, 1, 8, 64>(a, bwd, st);
    if (a.D <= 2048) return launch_g<TI, TR, TO, 1, 8, 256>(a, bwd, st);
    if (a.D <= 8192) return launch_g<TI, TR, TO, 1, 8, 1024>(a, bwd, st);
    return launch_g<TI, TR, TO, 1, 16, 1024>(a, bwd, st);
}

template <typename TI>
static hipError_t launch_i(const NormArgs& a, bool bwd, hipStream_t st) {
    if (a.res_bf16 && a.out_bf16) return launch_t<TI, bf16_t, bf16_t>(a, bwd, st);
    if (a.res_bf16) return launch_t<TI, bf16_t, float>(a, bwd, st);
    if (a.out_bf16) return launch_t<TI, float, bf16_t>(a, bwd, st);
    return launch_t<TI, float, float>(a, bwd, st);
}

}  // namespace norm

size_t norm_bwd_ws_bytes(int64_t rows, int64_t D) {
    const int most = norm::bwd_groups(256);   // no launch has more workgroups, nor more than rows
    return (size_t)((rows < most ? rows : most) * 2 * D) * 4;
}

hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t st) {
    return a.in_bf16 ? norm::launch_i<bf16_t>(a, false, st) : norm::launch_i<float>(a, false, st);
}

hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t st) {
    return a.in_bf16 ? norm::launch_i<bf16_t>(a, true, st) : norm::launch_i<float>(a, true, st);
}

}  // namespace kda
