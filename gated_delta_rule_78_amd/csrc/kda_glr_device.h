// Device code shared by the gated linear recurrence's kernels: the gates and their derivatives, the
// composition of row spans and the chain that carries states between tiles (their geometry:
// kda_glr_tiles.h).
#pragma once

#include "kda_glr.h"
#include "kda_glr_internal.h"
#include "kda_glr_tiles.h"
#include "kda_math.h"

namespace kda {
namespace glr {

// Log decays are carried as y = log2(alpha) = log_alpha log2(e).
// 1 - 2^y without the cancellation near y = 0: for y > -0.5 (log_alpha > -0.35) the series
// -y (ln2 + y ln2^2/2 + ... + y^6 ln2^7/5040), cut at a relative error of 0.35^7 / 8! < 2^-25.
__device__ __forceinline__ float one_minus_exp2(float y, float alpha) {
    float p = fmaf(y, 1.5252733804059840e-5f, 1.5403530393381609e-4f);
    p = fmaf(p, y, 1.3333558146428443e-3f);
    p = fmaf(p, y, 9.6181291076284772e-3f);
    p = fmaf(p, y, 5.5504108664821580e-2f);
    p = fmaf(p, y, 2.4022650695910071e-1f);
    p = fmaf(p, y, 6.9314718055994531e-1f);
    return y > -0.5f ? -y * p : 1.f - alpha;
}

// The input scale w(alpha).
template <int SCALE>
__device__ __forceinline__ float scale_w(float y, float alpha) {
    if constexpr (SCALE == KDA_GLR_ONE) return 1.f;
    const float om = one_minus_exp2(y, alpha);
    if constexpr (SCALE == KDA_GLR_LEAKY) return om;
    return __builtin_amdgcn_sqrtf(fmaf(om, alpha, om));   // (1 - alpha)(1 + alpha)
}

// A span of rows maps the state before it to the state after it: h -> A h + b. The sign bit of A
// says that a sequence starts inside the span, which then does not see the state before it at all
// (A's magnitude is not read); log decays give A >= 0 otherwise.
struct Span {
    float A, h;
};
template <bool CUTS>
__device__ __forceinline__ float apply(Span s, float h) {
    const float r = fmaf(s.A, h, s.h);
    if constexpr (!CUTS) return r;
    return __float_as_int(s.A) < 0 ? s.h : r;
}
// First l, then r: a cut in l keeps the sign of the product negative.
template <bool CUTS>
__device__ __forceinline__ Span compose(Span l, Span r) {
    Span o{l.A * r.A, apply<CUTS>(r, l.h)};
    if constexpr (CUTS)
        if (__float_as_int(r.A) < 0) o.A = r.A;
    return o;
}

// ---- the chain -------------------------------------------------------------------------------
// Tiles of one block of rows and channel tile form a chain. A tile publishes its span as one
// 64-bit word per channel as soon as it has read its rows, and the state behind it as another once
// it knows the state before it. Each word holds all a reader needs (all ones: not there yet), so
// relaxed agent-scope accesses suffice: nothing is ordered against anything else. A workgroup
// takes its tile from its chain's counter, in chain order, so every tile it waits for is held by a
// workgroup that started earlier and itself only waits for earlier ones: every wait ends. One
// counter for all chains holds the launch back: a word takes an atomic every 14 ns (64K rows x 4096
// channels: 445 us with one counter). The method is the published single-pass scan with decoupled
// look-back (Merrill and Garland, 2016).

typedef unsigned long long u64;
constexpr u64 kNone = ~0ull;

__device__ __forceinline__ void publish(u64* p, uint32_t hi, float lo) {
    const u64 v = ((u64)hi << 32) | __float_as_uint(lo);
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ u64 peek(const u64* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void publish_span(u64* p, Span s) {
    uint32_t a = __float_as_uint(s.A);
    if (a == 0xffffffffu) a = 0xffc00000u;          // a NaN: any other one, the word must not be kNone
    publish(p, a, s.h);
}

// The state before the tile whose words are span[i * step], state[i * step] at i = 0, from the
// `avail` tiles before it (i = -1, -2, ...): the nearest published state, carried forward over the
// spans in between one by one. A tile's own published state is the same operations on the same
// numbers, so the result does not depend on which one was found. The words are nearly always there
// at the first look, whose latency is what the chain costs (64K rows x 4096 channels: 352 us with a
// single look and no wait, 357 as it is, 328 without the chain), so a wider window gains nothing (a
// window of 5: 380), and neither does a look taken before the tile's own span is known (361): that
// one is too early.
constexpr int kWindow = 3;
template <bool CUTS>
__device__ __forceinline__ float look_back(const u64* span, const u64* state, int64_t step, int64_t avail) {
    const int n = avail < kWindow ? (int)avail : kWindow;
    for (int spin = 0; spin < (1 << 26); ++spin) {
        u64 sp[kWindow], st[kWindow];
#pragma unroll
        for (int i = 0; i < kWindow; ++i)
            if (i < n) {
                st[i] = peek(state - (int64_t)(i + 1) * step);
                if (i + 1 < kWindow) sp[i] = peek(span - (int64_t)(i + 1) * step);
            }
        int found = -1;
        bool ok = true;
#pragma unroll
        for (int i = 0; i < kWindow; ++i)
            if (i < n && found < 0 && ok) {
                if (st[i] != kNone) found = i;
                else if (i + 1 < kWindow) ok = sp[i] != kNone;
            }
        if (found >= 0) {
            float h = 0.f;
#pragma unroll
            for (int i = kWindow - 1; i >= 0; --i) {
                if (i == found) h = __uint_as_float((uint32_t)st[i]);
                else if (i < found) h = apply<CUTS>(Span{__uint_as_float((uint32_t)(sp[i] >> 32)), __uint_as_float((uint32_t)sp[i])}, h);
            }
            return h;
        }
        __builtin_amdgcn_s_sleep(2);
    }
    return __uint_as_float(0x7fc00000u);   // gave up, which the order of the tiles rules out: NaN from here on
}

// Spans of a wave's threads (SPW sub-chunks of CT threads, VEC channels each), turned through LDS so
// that a lane holds one channel: before[s] spans the sub-chunks before s (behind it, BACK), total
// all of them. `buf`: 2 * SPW * kCW floats of the wave's own; its accesses need no barrier.
// Shuffles instead cost twice the LDS accesses and four times the arithmetic, every lane scanning
// its four channels in log steps.
template <bool CUTS, bool BACK, int VEC, int SPW>
struct WaveSpans {
    Span before[SPW], total;

    __device__ __forceinline__ void scan(const Span (&sp)[VEC], float* buf, int lane) {
        if constexpr (SPW == 1) {   // VEC = 1: the lane has its channel already
            total = sp[0];
        } else {
            static_assert(VEC == 4 && SPW == 4, "16 lanes of 4 channels");
            float* own = buf + (lane >> 4) * 2 * kCW + (lane & 15) * 4;
            *reinterpret_cast<float4*>(own) = make_float4(sp[0].A, sp[1].A, sp[2].A, sp[3].A);
            *reinterpret_cast<float4*>(own + kCW) = make_float4(sp[0].h, sp[1].h, sp[2].h, sp[3].h);
            wave_lds_sync();
#pragma unroll
            for (int i = 0; i < SPW; ++i) {
                const int s = BACK ? SPW - 1 - i : i;
                const Span x{buf[2 * s * kCW + lane], buf[(2 * s + 1) * kCW + lane]};
                before[s] = total;
                total = i == 0 ? x : compose<CUTS>(total, x);
            }
        }
    }
    // h at the wave's first row (last, BACK) to h[VEC] at each thread's
    __device__ __forceinline__ void spread(float at, float* buf, int lane, float (&h)[VEC]) const {
        if constexpr (SPW == 1) {
            h[0] = at;
        } else {
#pragma unroll
            for (int i = 0; i < SPW; ++i) {
                const int s = BACK ? SPW - 1 - i : i;
                buf[s * kCW + lane] = i == 0 ? at : apply<CUTS>(before[s], at);
            }
            wave_lds_sync();
            const float4 v = *reinterpret_cast<const float4*>(buf + (lane >> 4) * kCW + (lane & 15) * 4);
            h[0] = v.x; h[1] = v.y; h[2] = v.z; h[3] = v.w;
        }
    }
};

// VEC consecutive elements of a row as they lie in memory.
template <typename T, int VEC>
struct RawRow;
template <> struct RawRow<bf16_t, 4> { uint2 v; };
template <> struct RawRow<float, 4> { float4 v; };
template <> struct RawRow<bf16_t, 1> { bf16_t v; };
template <> struct RawRow<float, 1> { float v; };

__device__ __forceinline__ void unpack(const RawRow<bf16_t, 4>& r, float* o) {
    o[0] = __uint_as_float(r.v.x << 16); o[1] = __uint_as_float(r.v.x & 0xffff0000u);
    o[2] = __uint_as_float(r.v.y << 16); o[3] = __uint_as_float(r.v.y & 0xffff0000u);
}
__device__ __forceinline__ void unpack(const RawRow<float, 4>& r, float* o) {
    o[0] = r.v.x; o[1] = r.v.y; o[2] = r.v.z; o[3] = r.v.w;
}
__device__ __forceinline__ void unpack(const RawRow<bf16_t, 1>& r, float* o) { o[0] = bf16_bits_to_f32(r.v); }
__device__ __forceinline__ void unpack(const RawRow<float, 1>& r, float* o) { o[0] = r.v; }

// Rows may start on any element: one 8- or 16-byte access serves any alignment.
template <typename T, int VEC>
__device__ __forceinline__ RawRow<T, VEC> load_row(const T* p) {
    RawRow<T, VEC> r;
    __builtin_memcpy(&r, p, VEC * sizeof(T));
    return r;
}
template <int VEC>
__device__ __forceinline__ void store_row(bf16_t* p, const float* x) {
    if constexpr (VEC == 4) {
        const uint2 u{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
        __builtin_memcpy(p, &u, 8);
    } else {
        st_f(p, x[0]);
    }
}
template <int VEC>
__device__ __forceinline__ void store_row(float* p, const float* x) {
    __builtin_memcpy(p, x, VEC * 4);
}
template <int VEC>
__device__ __forceinline__ void load_f32(const float* p, float* o) {
    __builtin_memcpy(o, p, VEC * 4);
}

// Which sequences start and end in the rows of a packed batch (glr_prepare_kernel): a bit per
// row, and the sequence where the bit is set. bits_at: those of the L rows from row on (L divides
// 32, row a multiple of L).
template <int L>
__device__ __forceinline__ uint32_t bits_at(const uint32_t* bits, int64_t row) {
    return (bits[row >> 5] >> (row & 31)) & (L == 32 ? ~0u : (1u << L) - 1u);
}
// The rows of a tile that are in a sequence: [lo, hi) (sequences lie back to back).
__device__ __forceinline__ void live_rows(const GlrArgs& a, int64_t row0, int rows, int& lo, int& hi) {
    const int64_t c0 = a.cu[0] - row0, c1 = a.cu[a.N] - row0;
    lo = c0 > 0 ? (int)(c0 < rows ? c0 : rows) : 0;
    hi = c1 < hi ? (int)(c1 > 0 ? c1 : 0) : hi;
}

// Element offset of row r of a thread whose first lies at off0, kept inside the tile (`last`: the
// thread's channel in the tile's last row).
__device__ __forceinline__ uint32_t row_offset(uint32_t off0, int r, uint32_t d, uint32_t last) {
    const uint32_t off = off0 + (uint32_t)r * d;
    return off < last ? off : last;
}

}  // namespace glr
}  // namespace kda
