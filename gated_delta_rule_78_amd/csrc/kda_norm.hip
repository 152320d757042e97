// Norms around a block for gfx950 (include/kda_norm.h). Per row of D channels:
//     p = f w_post r1,  r1 = 1 / sqrt(mean(f^2) + eps);   u = sigmoid(gate) p;
//     x' = x + scale lam u;   n = x' w_pre r2,  r2 = 1 / sqrt(mean(x'^2) + pre_eps).
// Backward, from D' = dL/dx' (direct) and dn, with t = dn w_pre and xh = x' r2:
//     dx' = D' + r2 (t - xh mean(t xh)),   dx = dx',   dw_pre = sum_rows dn xh;
//     dlam = scale sum_rows dx' u;   du = dx' scale lam;   dgate = du p s (1 - s);   dp = du s;
//     with t1 = dp w_post and fh = f r1:  df = r1 (t1 - fh mean(t1 fh)),   dw_post = sum_rows dp fh.
//
// A row lives in the registers of TPR threads (VEC * NV channels each), so every tensor is read
// once and written once: the kernels are bound by HBM. Rows of at most 64 threads share a
// 256-thread workgroup and reduce by lane shuffles; wider ones take a workgroup each and meet in
// LDS.
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

// Sum over the TPR threads of a row, in a fixed order; every thread gets it. `red`: TPR / 64
// floats per value and call (wide rows); consecutive calls take different halves of it.
template <int TPR, int N>
__device__ __forceinline__ void row_sum(float (&s)[N], float* red) {
#pragma unroll
    for (int m = 1; m < (TPR < 64 ? TPR : 64); m <<= 1)
#pragma unroll
        for (int j = 0; j < N; ++j) s[j] += __shfl_xor(s[j], m);
    if constexpr (TPR > 64) {
        constexpr int W = TPR / 64;
        const int wv = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int j = 0; j < N; ++j) red[j * W + wv] = s[j];
        __syncthreads();
#pragma unroll
        for (int j = 0; j < N; ++j) {
            s[j] = 0.f;
#pragma unroll
            for (int i = 0; i < W; ++i) s[j] += red[j * W + i];
        }
    }
}

template <int TPR>
struct Geo {
    static constexpr int threads = TPR < 256 ? 256 : TPR;
    static constexpr int rows = threads / TPR;
};

template <typename TI, typename TR, typename TO, int VEC, int NV, int TPR>
__global__ __launch_bounds__(Geo<TPR>::threads) void norm_fwd_kernel(NormArgs a) {
    __shared__ float red[2][TPR > 64 ? TPR / 64 : 1];
    const int lane = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * Geo<TPR>::rows + threadIdx.x / TPR;
    const bool live = row < a.rows;
    const int64_t base = row * a.D;
    const float inv = 1.f / (float)a.D;
    Raw<TI, VEC> f[NV], g[NV];
    Raw<TR, VEC> x[NV];
    bool on[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int col = (j * TPR + lane) * VEC;
        on[j] = live && col < a.D;
        if (on[j]) {
            f[j] = load_raw<TI, VEC>((const TI*)a.f + base + col);
            if (a.gate) g[j] = load_raw<TI, VEC>((const TI*)a.gate + base + col);
            if (a.x) x[j] = load_raw<TR, VEC>((const TR*)a.x + base + col);
        }
    }
    float r1 = 1.f;
    if (a.post) {
        float s[1] = {0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (on[j])
#pragma unroll
                for (int i = 0; i < VEC; ++i) s[0] = fmaf(at(f[j], i), at(f[j], i), s[0]);
        row_sum<TPR>(s, red[0]);
        r1 = __builtin_amdgcn_rsqf(fmaf(s[0], inv, a.eps));
    }
    float xo[NV][VEC];
    float s2[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if (!on[j]) continue;
        const int col = (j * TPR + lane) * VEC;
        float wp[VEC], lm[VEC];
        load_w<VEC>(a.w_post, col, wp);
        load_w<VEC>(a.lam, col, lm);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            float u = at(f[j], i) * r1 * wp[i];
            if (a.gate) u *= sigmoid_f(at(g[j], i));
            xo[j][i] = a.scale * lm[i] * u;
            if (a.x) xo[j][i] += at(x[j], i);
            s2[0] = fmaf(xo[j][i], xo[j][i], s2[0]);
        }
        if (a.x_out) store_vec<TR, VEC>((TR*)a.x_out + base + col, xo[j]);
    }
    if (!a.pre) return;
    row_sum<TPR>(s2, red[1]);
    const float r2 = __builtin_amdgcn_rsqf(fmaf(s2[0], inv, a.pre_eps));
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if (!on[j]) continue;
        const int col = (j * TPR + lane) * VEC;
        float w[VEC], n[VEC];
        load_w<VEC>(a.w_pre, col, w);
#pragma unroll
        for (int i = 0; i < VEC; ++i) n[i] = xo[j][i] * r2 * w[i];
        store_vec<TO, VEC>((TO*)a.n + base + col, n);
    }
}

// Workgroups of the backward: each walks rows blockIdx.x, + gridDim.x, ... and keeps its column
// sums in registers, so that the sums' traffic is workgroups * 3 * D floats, not rows * 3 * D.
constexpr int kBwdGroups = 512;

template <typename TI, typename TR, typename TO, int VEC, int NV, int TPR>
__global__ __launch_bounds__(Geo<TPR>::threads) void norm_bwd_kernel(NormArgs a) {
    constexpr int RPB = Geo<TPR>::rows;
    __shared__ float red[2][4][TPR > 64 ? TPR / 64 : 1];
    __shared__ float colsum[RPB > 1 ? RPB * VEC * NV * TPR : 1];
    const int lane = threadIdx.x % TPR;
    const float inv = 1.f / (float)a.D;
    float acc[3][NV][VEC];
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[k][j][i] = 0.f;
    int phase = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < a.rows; row0 += (int64_t)gridDim.x * RPB, phase ^= 1) {
        const int64_t row = row0 + threadIdx.x / TPR;
        const bool live = row < a.rows;
        const int64_t base = row * a.D;
        Raw<TI, VEC> f[NV], g[NV];
        Raw<TR, VEC> x[NV], dxo[NV];
        Raw<TO, VEC> dn[NV];
        bool on[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = (j * TPR + lane) * VEC;
            on[j] = live && col < a.D;
            if (on[j]) {
                f[j] = load_raw<TI, VEC>((const TI*)a.f + base + col);
                if (a.gate) g[j] = load_raw<TI, VEC>((const TI*)a.gate + base + col);
                if (a.x && a.dn) x[j] = load_raw<TR, VEC>((const TR*)a.x + base + col);
                if (a.dx_out) dxo[j] = load_raw<TR, VEC>((const TR*)a.dx_out + base + col);
                if (a.dn) dn[j] = load_raw<TO, VEC>((const TO*)a.dn + base + col);
            }
        }
        float r1 = 1.f;
        if (a.post) {
            float s[1] = {0.f};
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (on[j])
#pragma unroll
                    for (int i = 0; i < VEC; ++i) s[0] = fmaf(at(f[j], i), at(f[j], i), s[0]);
            row_sum<TPR>(s, red[phase][0]);
            r1 = __builtin_amdgcn_rsqf(fmaf(s[0], inv, a.eps));
        }
        // x' again, and the pre-norm's part of its gradient
        float r2 = 0.f, m2 = 0.f;
        float xo[NV][VEC];
        if (a.dn) {
            float s[2] = {0.f, 0.f};
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (!on[j]) continue;
                const int col = (j * TPR + lane) * VEC;
                float wp[VEC], lm[VEC], w[VEC];
                load_w<VEC>(a.w_post, col, wp);
                load_w<VEC>(a.lam, col, lm);
                load_w<VEC>(a.w_pre, col, w);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    float u = at(f[j], i) * r1 * wp[i];
                    if (a.gate) u *= sigmoid_f(at(g[j], i));
                    xo[j][i] = a.scale * lm[i] * u;
                    if (a.x) xo[j][i] += at(x[j], i);
                    s[0] = fmaf(xo[j][i], xo[j][i], s[0]);
                    s[1] = fmaf(at(dn[j], i) * w[i], xo[j][i], s[1]);
                }
            }
            row_sum<TPR>(s, red[phase][1]);
            r2 = __builtin_amdgcn_rsqf(fmaf(s[0], inv, a.pre_eps));
            m2 = s[1] * inv * r2;   // mean(t xh)
        }
        float t1[NV][VEC];
        float s3[1] = {0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (!on[j]) continue;
            const int col = (j * TPR + lane) * VEC;
            float wp[VEC], lm[VEC], w[VEC], dxv[VEC], dgv[VEC];
            load_w<VEC>(a.w_post, col, wp);
            load_w<VEC>(a.lam, col, lm);
            load_w<VEC>(a.w_pre, col, w);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                float dx = a.dx_out ? at(dxo[j], i) : 0.f;
                if (a.dn) {
                    const float xh = xo[j][i] * r2, d = at(dn[j], i);
                    acc[2][j][i] = fmaf(d, xh, acc[2][j][i]);
                    dx += r2 * (d * w[i] - xh * m2);
                }
                dxv[i] = dx;
                const float fh = at(f[j], i) * r1, p = fh * wp[i];
                const float s = a.gate ? sigmoid_f(at(g[j], i)) : 1.f;
                acc[1][j][i] = fmaf(dx, s * p, acc[1][j][i]);
                const float du = dx * a.scale * lm[i];
                dgv[i] = du * p * s * (1.f - s);
                const float dp = du * s;
                acc[0][j][i] = fmaf(dp, fh, acc[0][j][i]);
                t1[j][i] = dp * wp[i];
                s3[0] = fmaf(t1[j][i], fh, s3[0]);
            }
            if (a.dx) store_vec<TR, VEC>((TR*)a.dx + base + col, dxv);
            if (a.gate) store_vec<TI, VEC>((TI*)a.dgate + base + col, dgv);
        }
        float m1 = 0.f;
        if (a.post) {
            row_sum<TPR>(s3, red[phase][3]);
            m1 = s3[0] * inv;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (!on[j]) continue;
            const int col = (j * TPR + lane) * VEC;
            float d[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                d[i] = a.post ? r1 * (t1[j][i] - at(f[j], i) * r1 * m1) : t1[j][i];
            store_vec<TI, VEC>((TI*)a.df + base + col, d);
        }
    }
    if (!a.ws) return;
    // this workgroup's column sums: over its row groups through LDS, then to the workspace
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        float* ws = a.ws + ((int64_t)blockIdx.x * 3 + k) * a.D;
        if constexpr (RPB > 1) {
            constexpr int W = VEC * NV * TPR;
            __syncthreads();
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    colsum[(threadIdx.x / TPR) * W + (j * TPR + lane) * VEC + i] = acc[k][j][i];
            __syncthreads();
            for (int c = threadIdx.x; c < a.D; c += Geo<TPR>::threads) {
                float s = 0.f;
                for (int r = 0; r < RPB; ++r) s += colsum[r * W + c];
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

// Column sums of the workgroups' partials [groups][3][D]: 16 runs of workgroups a column, each
// summed in order by a thread, joined in LDS in order.
__global__ __launch_bounds__(1024) void norm_colsum_kernel(NormArgs a, int groups) {
    __shared__ float part[16][64];
    const int lane = threadIdx.x & 63, run = threadIdx.x >> 6, k = blockIdx.y;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    float* out = k == 0 ? a.dw_post : k == 1 ? a.dlam : a.dw_pre;
    if (!out) return;
    const int each = (groups + 15) / 16, g1 = (run + 1) * each < groups ? (run + 1) * each : groups;
    float s = 0.f;
    if (c < a.D) {
#pragma unroll 8
        for (int g = run * each; g < g1; ++g) s += a.ws[((int64_t)g * 3 + k) * a.D + c];
    }
    part[run][lane] = s;
    __syncthreads();
    if (run == 0 && c < a.D) {
#pragma unroll
        for (int i = 1; i < 16; ++i) s += part[i][lane];
        out[c] = k == 1 ? s * a.scale : s;
    }
}

template <typename TI, typename TR, typename TO, int VEC, int NV, int TPR>
static hipError_t launch_g(const NormArgs& a, bool bwd, hipStream_t st) {
    constexpr int RPB = Geo<TPR>::rows;
    const int64_t blocks = (a.rows + RPB - 1) / RPB;
    if (!bwd) {
        hipLaunchKernelGGL((norm_fwd_kernel<TI, TR, TO, VEC, NV, TPR>), dim3((unsigned)blocks),
                           dim3(Geo<TPR>::threads), 0, st, a);
        return hipGetLastError();
    }
    const int groups = blocks < kBwdGroups ? (int)blocks : kBwdGroups;
    if (groups > 0)
        hipLaunchKernelGGL((norm_bwd_kernel<TI, TR, TO, VEC, NV, TPR>), dim3(groups), dim3(Geo<TPR>::threads), 0, st, a);
    if (a.dw_post || a.dlam || a.dw_pre)
        hipLaunchKernelGGL(norm_colsum_kernel, dim3((unsigned)((a.D + 63) / 64), 3), dim3(1024), 0, st, a,
                           groups);
    return hipGetLastError();
}

// Threads per row and channels per thread by D: 16-byte accesses where every row starts on 16
// bytes (D a multiple of 8 and such bases), else one channel at a time.
static bool wide(const NormArgs& a) {
    uintptr_t bits = 0;
    for (const void* p : {a.f, a.gate, a.x, (const void*)a.x_out, (const void*)a.n, a.dx_out, a.dn, (const void*)a.df,
                          (const void*)a.dgate, (const void*)a.dx})
        bits |= reinterpret_cast<uintptr_t>(p);
    return a.D % 8 == 0 && (bits & 15) == 0;
}

template <typename TI, typename TR, typename TO>
static hipError_t launch_t(const NormArgs& a, bool bwd, hipStream_t st) {
    if (wide(a)) {
        if (a.D <= 128) return launch_g<TI, TR, TO, 8, 1, 16>(a, bwd, st);
        if (a.D <= 512) return launch_g<TI, TR, TO, 8, 1, 64>(a, bwd, st);
        if (a.D <= 2048) return launch_g<TI, TR, TO, 8, 1, 256>(a, bwd, st);
        if (a.D <= 4096) return launch_g<TI, TR, TO, 8, 2, 256>(a, bwd, st);
        if (a.D <= 8192) return launch_g<TI, TR, TO, 8, 2, 512>(a, bwd, st);
        return launch_g<TI, TR, TO, 8, 2, 1024>(a, bwd, st);
    }
    if (a.D <= 64) return launch_g<TI, TR, TO, 1, 4, 16>(a, bwd, st);
    if (a.D <= 512) return launch_g<TI, TR, TO, 1, 8, 64>(a, bwd, st);
    if (a.D <= 4096) return launch_g<TI, TR, TO, 1, 16, 256>(a, bwd, st);
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
    const int64_t groups = rows < norm::kBwdGroups ? rows : norm::kBwdGroups;
    return (size_t)(groups * 3 * D) * 4;
}

hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t st) {
    return a.in_bf16 ? norm::launch_i<bf16_t>(a, false, st) : norm::launch_i<float>(a, false, st);
}

hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t st) {
    return a.in_bf16 ? norm::launch_i<bf16_t>(a, true, st) : norm::launch_i<float>(a, true, st);
}

}  // namespace kda
