// Attention of new tokens over a paged cache for gfx950 (include/kda_attn.h), bf16, head sizes as
// template parameters (instantiated in kda_attn_d*.hip).
//
//     x_j = c q . k_j  (c = scale log2 e),  o = sum_j 2^(x_j - m) v_j / l,  l = sum_j 2^(x_j - m)
//
// in one pass over the keys with a running reference m and sum l, both fp32. Products are transposed:
// S^T = K Q^T puts a query in a lane (column n = lane % 32 of the 32x32 product) and the block's keys
// in its registers, so row sums and the rescaling of O^T = V^T P^T need one exchange (the two halves
// of the wave), and the registers of P^T are the second product's operand as they stand: operand slot
// e of half h at k step kk is key 16 kk + 8 (e / 4) + 4 h + e % 4, and V is read with that order by
// transposed LDS reads.
//
// P is rounded to bf16 (half a step, 2^-8, of each probability) to enter the matrix product, l is the
// sum of the unrounded ones.
#pragma once

#include "kda_attn_plan.h"
#include "kda_mfma.h"

namespace kda {
namespace attn {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x16 mfma32(bf16x8 a, bf16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// Maximum and sum over the two lanes of a query, one in each half of the wave.
__device__ __forceinline__ float both_max(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float both_sum(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// 16 bytes a lane from a raw buffer straight into LDS, to lds + 16 lane. Offsets at or past the
// descriptor's size store zeros. The compiler does not count these loads: whoever reads the LDS waits
// with wait_vm first.
// The uniform offset `more` is added behind the check. The LDS address stands in m0, a wait state ahead; scalar
// operands that a vector instruction wrote (lane reads, among them those of spilled registers) need five, which the
// compiler does not keep before an asm: s_nop 4.
__device__ __forceinline__ void load_to_lds(i32x4 r, uint32_t off, uint32_t lds, uint32_t more = 0) {
    const i32x4 rsrc = {uniform(r[0]), uniform(r[1]), uniform(r[2]), uniform(r[3])};
    asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :: "{m0}"(uniform((int)lds)), "v"(off), "s"(rsrc), "s"(uniform((int)more)) : "memory");
}
template <int N>
__device__ __forceinline__ void wait_vm() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}

// n / d by the magic number of d: exact where n d < 2^32.
__device__ __forceinline__ int div_by(int n, uint32_t magic) { return magic ? (int)__umulhi((uint32_t)n, magic) : n; }

// One tile's place: which sequence, rows and keys.
struct Tile {
    int64_t seq, first;     // sequence, first token of it in the rows' T (packed) or 0
    int n, kv;              // its new tokens, its keys
    int row0, rows;         // first row, rows of the sequence in all
    int tok0, rem0;         // token and head (of the group) of row0
    int head;               // key head
    int lo, hi;             // keys that any row sees: [lo, hi)
    int chunk, chunks;
    int64_t slot;           // partial result, when chunks > 1
};

// First token, new tokens and keys of a sequence from its lengths as they stand (c0, c1 with a.packed only); false
// where it has no rows.
__device__ __forceinline__ bool lengths(const AttnArgs& a, int c0, int c1, int kv_len, int64_t& first, int& n, int& kv) {
    const bool ok = c0 >= 0 && c1 >= c0 && c1 <= a.T;
    first = a.packed && ok ? c0 : 0;
    n = a.packed ? (ok ? c1 - c0 : 0) : (int)a.T;
    const int most = a.max_pages * a.page_size;
    kv = kv_len < 0 ? 0 : kv_len > most ? most : kv_len;
    return n > 0;
}
__device__ __forceinline__ bool sequence(const AttnArgs& a, int64_t s, int64_t& first, int& n, int& kv) {
    int c0 = 0, c1 = 0;
    if (a.packed) {
        c0 = a.cu[s];
        c1 = a.cu[s + 1];
    }
    return lengths(a, c0, c1, a.kv_lens[s], first, n, kv);
}
// f(new tokens, keys) for the sequences s, s + step, .. below `end` that have rows, four of them loaded at a time.
template <typename F>
__device__ __forceinline__ void for_sequences(const AttnArgs& a, int s, int step, int end, const F& f) {
    constexpr int AT = 4;
#pragma unroll 1
    for (; s < end; s += AT * step) {
        int c0[AT], c1[AT], v[AT];
#pragma unroll
        for (int i = 0; i < AT; ++i) c0[i] = c1[i] = 0;
        if (a.packed)
#pragma unroll
            for (int i = 0; i < AT; ++i) {
                const int x = s + i * step < end ? s + i * step : s;
                c0[i] = a.cu[x];
                c1[i] = a.cu[x + 1];
            }
#pragma unroll
        for (int i = 0; i < AT; ++i) v[i] = a.kv_lens[s + i * step < end ? s + i * step : s];
#pragma unroll
        for (int i = 0; i < AT; ++i) {
            int64_t first;
            int n, kv;
            if (lengths(a, c0[i], c1[i], v[i], first, n, kv) && s + i * step < end) f(n, kv);
        }
    }
}

// Row row0 + r of a tile: its token and its head in the group.
__device__ __forceinline__ void row_of(const AttnArgs& a, const Tile& t, int r, int& tok, int& hd) {
    const int x = t.rem0 + r, q = div_by(x, a.mG);
    tok = t.tok0 + q;
    hd = x - q * a.G;
}

// 1 / l for a row's sum l. A sum of 0 is that of a token at a negative position, which sees nothing (o = 0), or of
// one that sees scores of -inf alone (0 / 0); else l is at least the probability of the key that set the reference.
__device__ __forceinline__ float inv_sum(float l, int pos) { return l == 0.f ? (pos < 0 ? 0.f : NAN) : 1.f / l; }

// ---- which sequence, tile and chunk a workgroup has ------------------------------------------------

// Running sums over the sequences.
struct Counts {
    int items, slots, cuts;     // workgroups, partial results, (tile, head)s that are cut
};

__device__ __forceinline__ int lane_read(int x, int lane) { return __builtin_amdgcn_readlane(x, lane); }

template <int CTRL, int ROW_MASK>
__device__ __forceinline__ int dpp_i32(int x) {
    return __builtin_amdgcn_update_dpp(0, x, CTRL, ROW_MASK, 0xf, true);
}
__device__ __forceinline__ int wave_scan(int x) {      // inclusive; the steps of wave_prefix_sum
    x += dpp_i32<0x111, 0xf>(x);
    x += dpp_i32<0x112, 0xf>(x);
    x += dpp_i32<0x114, 0xf>(x);
    x += dpp_i32<0x118, 0xf>(x);
    x += dpp_i32<0x142, 0xa>(x);
    x += dpp_i32<0x143, 0xc>(x);
    return x;
}

struct Place {
    int64_t seq, first;
    int n, kv;
    int index;                  // of the workgroup (or cut) within the sequence
    int chunks, slot;           // C; the sequence's first partial result
};

// Where workgroup idx is (CUT: where the idx-th cut (tile, head) is); false behind the last. Uniform.
// all_cuts: how many (tile, head)s are cut in all.
template <bool NARROW, bool CUT>
__device__ __forceinline__ bool find_place(const AttnArgs& a, int idx, Place& out, int& all_cuts) {
    const int lane = threadIdx.x & 63, N = (int)a.N;
    int64_t first = 0;
    int n = 0, kv = 0, k = (N + 63) / 64;
    float tiles = 0.f, units = 0.f;
    auto add = [&](int n_, int kv_) {
        const float t = (float)(tiles_of(a, n_, NARROW) * a.Hk);
        tiles += t;
        units = fmaf(t, (float)tile_units(a, kv_, NARROW), units);
    };
    if (k > 1)
        for_sequences(a, lane, 64, N, add);
    else if (lane < N && sequence(a, lane, first, n, kv))
        add(n, kv);
    const Cut cut = cut_of(lane_value(wave_prefix_sum(tiles), 63), lane_value(wave_prefix_sum(units), 63), NARROW);
    Counts base = {0, 0, 0};
    int lo = 0, left = N;
    for (bool held = k == 1;; held = false) {
        k = (left + 63) / 64;
        Counts c = {0, 0, 0};
        int chunks = 1;
        const int s0 = lo + lane * k, s1 = s0 + k < lo + left ? s0 + k : lo + left;
        auto tally = [&](int n_, int kv_) {
            const int own = tiles_of(a, n_, NARROW) * a.Hk;
            chunks = chunks_of(cut, tile_units(a, kv_, NARROW));
            c.items += own * chunks;
            if (chunks > 1) {
                c.slots += own * chunks;
                c.cuts += own;
            }
        };
        if (k > 1) {
            for_sequences(a, s0, 1, s1, tally);
        } else if (s0 < s1) {
            if (!held) sequence(a, s0, first, n, kv);
            if (n > 0) tally(n, kv);
        }
        const int items = wave_scan(c.items) + base.items - c.items, slots = wave_scan(c.slots) + base.slots - c.slots,
                  cuts = wave_scan(c.cuts) + base.cuts - c.cuts;
        if (lo == 0 && left == N) all_cuts = lane_read(cuts + c.cuts, 63);
        const int at = CUT ? cuts : items, count = CUT ? c.cuts : c.items;
        // (sums that lengths which break the rules drive past 2^31 find nothing)
        const uint64_t mine = __ballot((uint32_t)at <= (uint32_t)idx && idx - at < count);
        if (mine == 0) return false;
        const int w = __builtin_ctzll(mine);
        base = Counts{lane_read(items, w), lane_read(slots, w), lane_read(cuts, w)};
        lo = lo + w * k;
        if (k == 1) {
            out.seq = uniform(lo);
            out.first = uniform(lane_read((int)first, w));
            out.n = uniform(lane_read(n, w));
            out.kv = uniform(lane_read(kv, w));
            out.chunks = uniform(lane_read(chunks, w));
            out.slot = uniform(base.slots);
            out.index = uniform(idx - (CUT ? base.cuts : base.items));
            return true;
        }
        left = left - w * k < k ? left - w * k : k;
    }
}

// ---- a page table walked by one wave ------------------------------------------------------------

// A place among a sequence's pages, all of it uniform but for what is held: lane i holds the addresses
// of one key head's rows in page base + i of either cache (their upper half -1 for a page number
// outside the cache), so that going to a page costs a wave four lane reads.
struct Pages {
    const int32_t* table;
    uint64_t kc, vc;                // the head's rows in page 0 of either cache
    uint32_t kp, vp;                // bytes from page to page
    int max_pages, page_size, pages;
    int pg, row;                    // page index and row of the current key
    int base;
    uint32_t klo, khi, vlo, vhi;    // held

    __device__ __forceinline__ Pages(const AttnArgs& a, int64_t seq, int head, int key) {
        table = a.table + seq * a.table_stride;
        kc = reinterpret_cast<uint64_t>(a.k_cache) + 2 * (uint64_t)(head * a.skc.h);
        vc = reinterpret_cast<uint64_t>(a.v_cache) + 2 * (uint64_t)(head * a.svc.h);
        kp = (uint32_t)(2 * a.skc.p); vp = (uint32_t)(2 * a.svc.p);
        max_pages = a.max_pages;
        page_size = a.page_size;
        pages = a.pages;
        pg = uniform(a.page_shift >= 0 ? key >> a.page_shift : key / page_size);
        row = uniform(key - pg * page_size);
        fetch();
    }
    __device__ __forceinline__ void advance(int keys) {
        row += keys;
        while (row >= page_size) {
            row -= page_size;
            ++pg;
        }
    }
    __device__ __forceinline__ void fetch() {
        base = pg;
        const int i = pg + fresh_lane(), p = i < max_pages ? table[i] : -1;
        const bool ok = p >= 0 && p < pages;
        const uint64_t k = kc + (uint64_t)(uint32_t)(ok ? p : 0) * kp, v = vc + (uint64_t)(uint32_t)(ok ? p : 0) * vp;
        klo = (uint32_t)k; khi = ok ? (uint32_t)(k >> 32) & 0xffff : 0xffffffffu;
        vlo = (uint32_t)v; vhi = ok ? (uint32_t)(v >> 32) & 0xffff : 0xffffffffu;
    }
    // Descriptors of the page `ahead` (< 48) of the current one, of which `valid` rows exist; the others
    // read as zeros.
    template <typename LK, typename LV>
    __device__ __forceinline__ void descriptors(int ahead, int valid, const LK& lk, const LV& lv, i32x4& k, i32x4& v) {
        if (pg + ahead - base >= 64) fetch();
        held_descriptors(pg + ahead - base, valid, lk, lv, k, v);
    }
    template <typename LK, typename LV>
    __device__ __forceinline__ void held_descriptors(int i, int valid, const LK& lk, const LV& lv, i32x4& k, i32x4& v) const {
        const bool all = valid >= page_size, none = valid <= 0;
        const int khi_ = __builtin_amdgcn_readlane(khi, i), vhi_ = __builtin_amdgcn_readlane(vhi, i);
        const bool bad = khi_ < 0 || none;
        const int ks = bad ? 0 : all ? lk.full : (valid - 1) * (int)lk.row_bytes + LK::kRowBytes;
        const int vs = bad ? 0 : all ? lv.full : (valid - 1) * (int)lv.row_bytes + LV::kRowBytes;
        k = i32x4{(int)__builtin_amdgcn_readlane(klo, i), khi_ & 0xffff, ks, kBufFlags};
        v = i32x4{(int)__builtin_amdgcn_readlane(vlo, i), vhi_ & 0xffff, vs, kBufFlags};
    }
};

// LDS tiles: rows of D channels, 16-byte pieces permuted within a row (piece c of row r at place
// c ^ f(r)) so that a wave's reads meet every bank once.
template <int D>
struct TileK {       // read row-wise: lanes 0..31 one row each
    static constexpr int kD = D, kRowBytes = 2 * D, kPieces = D / 8, kRows = 1024 / kRowBytes;   // kRows: of one load
    __device__ static __forceinline__ int f(int row) { return D == 128 ? row & 15 : (row >> 1) & 7; }
};
template <int D>
struct TileV {       // read transposed: 4 rows x 64 bytes a half wave
    static constexpr int kD = D, kRowBytes = 2 * D, kPieces = D / 8, kRows = 1024 / kRowBytes;
    __device__ static __forceinline__ int f(int row) { return D == 128 ? 4 * (row & 3) : 4 * ((row >> 1) & 1); }
};

// The loads of a tile of ROWS keys of one cache by WAVES waves: load i of wave w takes the kRows rows
// from kRows (WAVES i + w) on, all within 16 keys that one page holds.
template <typename L, int ROWS, int WAVES>
struct Loader {
    static constexpr int kLoads = ROWS / (L::kRows * WAVES), kStep = L::kRows * WAVES, kRowBytes = L::kRowBytes;
    uint32_t row_bytes;
    int full;               // bytes from a page's first row of the head to behind its last
    uint32_t lane_row, lane_piece;      // this lane's row's offset within a load's, its piece's in the first load
    int w;

    __device__ __forceinline__ Loader(const kda_page_strides& st, int page_size, int wave) {
        row_bytes = (uint32_t)(2 * st.t);
        full = (page_size - 1) * (int)row_bytes + kRowBytes;
        w = wave;
        const int lane = threadIdx.x & 63, lr = lane / L::kPieces;
        lane_row = (uint32_t)lr * row_bytes;
        lane_piece = 16 * ((lane % L::kPieces) ^ L::f(w * L::kRows) ^ L::f(lr));
    }
    // Load i from the page of descriptor r whose row `row` is the tile's row 0. The piece permutation
    // differs from the first load's by a constant.
    __device__ __forceinline__ void load(i32x4 r, int i, int row, uint32_t lds) const {
        load_to_lds(r, (lane_piece ^ (uint32_t)(16 * L::f(i * kStep))) + lane_row + (uint32_t)(row + first_row(i)) * row_bytes,
                    lds + (i * WAVES + w) * 1024);
    }
    // The same where the page holds all of this load's rows, `row` its first: nothing to check but the page.
    __device__ __forceinline__ void load_whole(i32x4 r, int i, int row, uint32_t lds) const {
        load_to_lds(r, (lane_piece ^ (uint32_t)(16 * L::f(i * kStep))) + lane_row, lds + (i * WAVES + w) * 1024,
                    (uint32_t)row * row_bytes);
    }
    __device__ __forceinline__ int first_row(int i) const { return i * kStep + w * L::kRows; }
};

// Descriptors of the ROWS keys at a walk's place, 16 at a time (all in the first one where one page holds
// them), and the page row of each 16's first key.
template <int ROWS>
struct Block {
    i32x4 k[ROWS / 16], v[ROWS / 16];
    int row[ROWS / 16];
    bool one;

    // keys from `hi` on read as zeros, kb is the first
    template <typename LK, typename LV>
    __device__ __forceinline__ void find(Pages& pg, const LK& lk, const LV& lv, int kb, int hi) {
        one = pg.row + ROWS <= pg.page_size;
        row[0] = pg.row;
        if (one) {
            pg.descriptors(0, hi - kb + pg.row, lk, lv, k[0], v[0]);
            return;
        }
#pragma unroll
        for (int g = 0; g < ROWS / 16; ++g) {
            int ahead = 0;
            row[g] = pg.row + 16 * g;
            while (row[g] >= pg.page_size) {
                row[g] -= pg.page_size;
                ++ahead;
            }
            pg.descriptors(ahead, hi - kb - 16 * g + row[g], lk, lv, k[g], v[g]);
        }
    }
    template <typename L>
    __device__ __forceinline__ void load(const L& l, const i32x4 (&r)[ROWS / 16], uint32_t lds) const {
        if (one) {
#pragma unroll
            for (int i = 0; i < L::kLoads; ++i) l.load(r[0], i, row[0], lds);
            return;
        }
#pragma unroll
        for (int i = 0; i < L::kLoads; ++i)
#pragma unroll
            for (int g = 0; g < ROWS / 16; ++g)
                if (l.first_row(i) >> 4 == g) l.load(r[g], i, row[g] - 16 * g, lds);
    }
};

// ---- one wave's rows against a block of keys ------------------------------------------------------

template <int DK, int DV, int KB>
struct Wave {
    static constexpr int kKS = DK / 16, kDT = DV / 32, kMT = KB / 32;
    bf16x8 Q[kKS];
    f32x16 O[kDT];
    float m, l;             // reference of this lane's query and this half's sum
    int pos, from;          // this lane's query sees keys from + 1 .. pos
    int first, last;        // least and largest position of the wave's live rows
    bool live;              // any row at all

    __device__ __forceinline__ void start(const AttnArgs& a, const Tile& t, int row_base) {
        const int lane = threadIdx.x & 63, h = lane >> 5;
        const int r = t.row0 + row_base + (lane & 31);
        const bool in = r < t.rows;
        int tok, hd;
        row_of(a, t, row_base + (lane & 31), tok, hd);
        pos = in ? t.kv - t.n + tok : -1;
        pos = pos < -1 ? -1 : pos;
        from = a.window > 0 && pos - a.window > -1 ? (int)(pos - a.window) : -1;
        const int r0 = t.row0 + row_base, r1 = r0 + 31 < t.rows ? r0 + 31 : t.rows - 1;
        live = r0 < t.rows;
        int ta, tb, ignored;
        row_of(a, t, row_base, ta, ignored);
        row_of(a, t, r1 - t.row0, tb, ignored);
        first = uniform(live ? t.kv - t.n + ta : -1);
        last = uniform(live ? t.kv - t.n + tb : -1);
        const bf16_t* p = static_cast<const bf16_t*>(a.q) + (a.packed ? 0 : t.seq * a.sq.b) + (t.first + (in ? tok : 0)) * a.sq.t +
                          ((int64_t)t.head * a.G + (in ? hd : 0)) * a.sq.h + 8 * h;
#pragma unroll
        for (int ks = 0; ks < kKS; ++ks) {
            uint4 u = make_uint4(0, 0, 0, 0);
            if (in) u = *reinterpret_cast<const uint4*>(p + 16 * ks);
            u.x ^= a.flip; u.y ^= a.flip; u.z ^= a.flip; u.w ^= a.flip;
            Q[ks] = __builtin_bit_cast(bf16x8, u);
        }
#pragma unroll
        for (int i = 0; i < kDT; ++i)
#pragma unroll
            for (int r2 = 0; r2 < 16; ++r2) O[i][r2] = 0.f;
        m = -INFINITY;
        l = 0.f;
    }

    // Whether any of the wave's rows sees a key of [kb, kb + KB).
    __device__ __forceinline__ bool sees(const AttnArgs& a, int kb) const {
        if (!live || kb > last) return false;
        return a.window <= 0 || (int64_t)kb + KB - 1 > (int64_t)first - a.window;
    }

    // Whether some row does not see some key of [kb, kb + KB).
    __device__ __forceinline__ bool masks(const AttnArgs& a, int kb) const {
        return kb + KB - 1 > first || (a.window > 0 && (int64_t)kb <= (int64_t)last - a.window);
    }

    // S^T = K Q^T of a block, and the registers of P^T that the second product takes.
    struct Scores {
        f32x16 s[kMT];
    };
    struct Probs {
        bf16x8 p[2 * kMT];
    };

    __device__ __forceinline__ void scores(const char* ks_, Scores& S) const {
        const int lane = fresh_lane(), n = lane & 31;
        const char* kp = ks_ + n * TileK<DK>::kRowBytes;
        const int sw = 16 * ((lane >> 5) ^ TileK<DK>::f(n));
        constexpr f32x16 zero = {};
#pragma unroll
        for (int ks = 0; ks < kKS; ++ks)
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt)
                S.s[mt] = mfma32(read16(kp + (sw ^ (32 * ks)) + mt * 32 * TileK<DK>::kRowBytes), Q[ks], ks ? S.s[mt] : zero);
    }

    // MASKED: 0 no row is masked, 1 some may be, 2 as `masked` says.
    template <int MASKED>
    __device__ __forceinline__ void softmax(const AttnArgs& a, Scores& S, Probs& P, int kb, bool masked = true) {
        if (MASKED == 1 || (MASKED == 2 && masked)) {
            const uint32_t span = (uint32_t)(pos - from);      // keys from + 1 .. pos are seen
            const uint32_t j0 = (uint32_t)(kb + 4 * (fresh_lane() >> 5) - from - 1);
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (j0 + (uint32_t)(32 * mt + (r & 3) + 8 * (r >> 2)) >= span) S.s[mt][r] = -INFINITY;
        }
        // the running reference: raised (and O, l scaled down) only when a score passes it by 2^8, which
        // keeps every 2^(x - m) below 2^8
        float mx = S.s[0][0];
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
            for (int r = 0; r < 16; ++r) mx = fmaxf(mx, S.s[mt][r]);
        mx = both_max(mx) * a.c;
        if (__any(mx > m + 8.f)) {
            const float mn = mx > m + 8.f ? mx : m;
            const float f = mn == m ? 1.f : __builtin_amdgcn_exp2f(m - mn);
            m = mn;
            l *= f;
#pragma unroll
            for (int i = 0; i < kDT; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) O[i][r] *= f;
        }
        const float sub = m == -INFINITY ? 0.f : m;
        float sum = 0.f;
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                float p[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    p[e] = __builtin_amdgcn_exp2f(fmaf(S.s[mt][8 * kk + e], a.c, -sub));
                    sum += p[e];
                }
                uint4 u;
                u.x = pack_bf16x2(p[0], p[1]); u.y = pack_bf16x2(p[2], p[3]);
                u.z = pack_bf16x2(p[4], p[5]); u.w = pack_bf16x2(p[6], p[7]);
                P.p[2 * mt + kk] = __builtin_bit_cast(bf16x8, u);
            }
        l += sum;
    }

    // A key that some rows do not see reaches them as a probability of 0 times its value: whether the block
    // at kb has such keys and V holds an infinity or a NaN. A block holds keys up to the tile's last row's (zeros
    // behind them), which a wave of a wide tile may not see though all its rows are one token's; OWN: this wave's
    // rows are all of the tile's, so that rows of one token see the block whole but for the window.
    template <bool OWN>
    __device__ __forceinline__ bool bad_values(const AttnArgs& a, const char* vs_, int kb) const {
        return (!OWN || last != first || a.window > 0) && masks(a, kb) && any_bad(vs_);
    }

    // O^T += V^T P^T. Bad values are left out of the product; the outputs that they belong to get them after it.
    __device__ __forceinline__ void values(const AttnArgs& a, const char* vs_, const Probs& P, int kb) {
        const int lane = fresh_lane(), l16 = lane & 15;
        const int vrow = 4 * (lane >> 5) + (l16 >> 2);
        const char* vp = vs_ + vrow * TileV<DV>::kRowBytes + 8 * (l16 & 1);
        const int piece = (2 * ((lane >> 4) & 1) + ((l16 & 3) >> 1)) ^ TileV<DV>::f(vrow);
        const bool bad = bad_values<false>(a, vs_, kb);
#pragma unroll
        for (int s = 0; s < 2 * kMT; ++s)
#pragma unroll
            for (int dt = 0; dt < kDT; ++dt) {
                bf16x8 v = read_v(vp, piece, s, dt);
                if (bad) v = without_bad(v);
                O[dt] = mfma32(v, P.p[s], O[dt]);
            }
        if (bad) mark_bad(vs_, kb);
    }

    // scores of one block and values of the one before as one stream of products, each operand read from LDS
    // AHEAD products before its own. The order is pinned: left to itself the compiler waits for every
    // operand right after asking for it. Ahead by 4, 8, 12: 3958, 3930, 3942 us for 4096 tokens over 65536 keys.
    __device__ __forceinline__ void scores_values(const char* ks_, Scores& S, const char* vs_, const Probs& P) {
        constexpr int NQ = kKS * kMT, N = NQ + 2 * kMT * kDT, AHEAD = 8;
        const int lane = fresh_lane(), n = lane & 31, l16 = lane & 15;
        const char* kp = ks_ + n * TileK<DK>::kRowBytes;
        const int sw = 16 * ((lane >> 5) ^ TileK<DK>::f(n));
        const int vrow = 4 * (lane >> 5) + (l16 >> 2);
        const char* vp = vs_ + vrow * TileV<DV>::kRowBytes + 8 * (l16 & 1);
        const int piece = (2 * ((lane >> 4) & 1) + ((l16 & 3) >> 1)) ^ TileV<DV>::f(vrow);
        constexpr f32x16 zero = {};
        bf16x8 F[N];
#pragma unroll
        for (int x = 0; x < N + AHEAD; ++x) {
            if (x < NQ)
                F[x] = read16(kp + (sw ^ (32 * (x / kMT))) + (x % kMT) * 32 * TileK<DK>::kRowBytes);
            else if (x < N)
                F[x] = read_v(vp, piece, (x - NQ) / kDT, (x - NQ) % kDT);
            const int y = x - AHEAD;
            if (y >= 0) {
                if (y < NQ)
                    S.s[y % kMT] = mfma32(F[y], Q[y / kMT], y < kMT ? zero : S.s[y % kMT]);
                else
                    O[(y - NQ) % kDT] = mfma32(F[y], P.p[(y - NQ) / kDT], O[(y - NQ) % kDT]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // The values alone, where nothing has to be left out.
    __device__ __forceinline__ void plain_values(const char* vs_, const Probs& P) {
        const int lane = fresh_lane(), l16 = lane & 15;
        const int vrow = 4 * (lane >> 5) + (l16 >> 2);
        const char* vp = vs_ + vrow * TileV<DV>::kRowBytes + 8 * (l16 & 1);
        const int piece = (2 * ((lane >> 4) & 1) + ((l16 & 3) >> 1)) ^ TileV<DV>::f(vrow);
#pragma unroll
        for (int s = 0; s < 2 * kMT; ++s)
#pragma unroll
            for (int dt = 0; dt < kDT; ++dt) O[dt] = mfma32(read_v(vp, piece, s, dt), P.p[s], O[dt]);
    }

    __device__ static __forceinline__ bf16x8 read_v(const char* vp, int piece, int s, int dt) {
        const bf16_t* p = reinterpret_cast<const bf16_t*>(vp + 16 * (piece ^ (4 * dt)) + 16 * s * TileV<DV>::kRowBytes);
        return cat(tr_read(p), tr_read(p + 8 * DV));
    }

    // Whether the V block holds an infinity or a NaN. Only then can a key that some rows do not see
    // reach them: a probability of 0 times it.
    __device__ __forceinline__ bool any_bad(const char* vs_) const {
        const int lane = fresh_lane();
        uint32_t hit = 0;
#pragma unroll 2
        for (int i = 0; i < KB * DV * 2 / 1024; ++i) {
            const uint4 u = *reinterpret_cast<const uint4*>(vs_ + i * 1024 + lane * 16);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
                hit |= (uint32_t)((w[k] & 0x7f80u) == 0x7f80u) | (uint32_t)((w[k] & 0x7f800000u) == 0x7f800000u);
        }
        return __any(hit);
    }

    // V without its infinities and NaN, zeros there.
    __device__ static __forceinline__ bf16x8 without_bad(bf16x8 x) {
        const uint4 u = __builtin_bit_cast(uint4, x);
        uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const bool lo = (w[k] & 0x7f80u) == 0x7f80u, hi = (w[k] & 0x7f800000u) == 0x7f800000u;
            w[k] &= (lo ? 0u : 0xffffu) | (hi ? 0u : 0xffff0000u);
        }
        return __builtin_bit_cast(bf16x8, make_uint4(w[0], w[1], w[2], w[3]));
    }

    // Ones where V holds the infinity of this sign bit or a NaN, zeros elsewhere.
    __device__ static __forceinline__ bf16x8 only_bad(bf16x8 x, uint32_t sign) {
        const uint4 u = __builtin_bit_cast(uint4, x);
        uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t lo = w[k] & 0xffffu, hi = w[k] >> 16, inf = 0x7f80u | sign;
            w[k] = (lo == inf || (lo & 0x7fffu) > 0x7f80u ? 0x3f80u : 0u) | (hi == inf || (hi & 0x7fffu) > 0x7f80u ? 0x3f800000u : 0u);
        }
        return __builtin_bit_cast(bf16x8, make_uint4(w[0], w[1], w[2], w[3]));
    }

    // Takes them out of a block that no other wave reads.
    __device__ static __forceinline__ void clear_bad(char* vs_) {
        const int lane = fresh_lane();
#pragma unroll 2
        for (int i = 0; i < KB * DV * 2 / 1024; ++i) {
            bf16x8* p = reinterpret_cast<bf16x8*>(vs_ + i * 1024 + lane * 16);
            *p = without_bad(*p);
        }
    }

    // Counts, for every output, the infinities of either sign and NaN among the values that its row sees, and adds
    // such an infinity to it: both where there is a NaN, so that it becomes one.
    __device__ __forceinline__ void mark_bad(const char* vs_, int kb) {
        const int lane = fresh_lane(), l16 = lane & 15, h = lane >> 5;
        const int vrow = 4 * h + (l16 >> 2);
        const char* vp = vs_ + vrow * TileV<DV>::kRowBytes + 8 * (l16 & 1);
        const int piece = (2 * ((lane >> 4) & 1) + ((l16 & 3) >> 1)) ^ TileV<DV>::f(vrow);
        const uint32_t span = (uint32_t)(pos - from), j0 = (uint32_t)(kb + 4 * h - from - 1);
#pragma unroll 1
        for (uint32_t sign = 0; sign <= 0x8000u; sign += 0x8000u) {
            const float inf = __uint_as_float(0x7f800000u | sign << 16);
#pragma unroll
            for (int dt = 0; dt < kDT; ++dt) {
                f32x16 C = {};
#pragma unroll
                for (int s = 0; s < 2 * kMT; ++s) {
                    uint32_t seen[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t j = j0 + (uint32_t)(16 * s + 2 * (k & 1) + 8 * (k >> 1));
                        asm volatile("" : "+v"(j));      // formed anew for each product: a rare path, few registers
                        seen[k] = (j < span ? 0x3f80u : 0u) | (j + 1 < span ? 0x3f800000u : 0u);
                    }
                    C = mfma32(only_bad(read_v(vp, piece, s, dt), sign),
                               __builtin_bit_cast(bf16x8, make_uint4(seen[0], seen[1], seen[2], seen[3])), C);
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
                for (int r = 0; r < 16; ++r) O[dt][r] = C[r] > 0.f ? O[dt][r] + inf : O[dt][r];
            }
        }
    }

    // dv of register quad g of tile dt
    __device__ static __forceinline__ int dv_of(int dt, int g) { return 32 * dt + 8 * g + 4 * ((threadIdx.x >> 5) & 1); }

    // Results of a tile whose keys were all here, or a partial one.
    __device__ __forceinline__ void finish(const AttnArgs& a, const Tile& t, int row_base, float* part, int part_rows) {
        const int n = threadIdx.x & 31, h = (threadIdx.x >> 5) & 1;
        const int r = t.row0 + row_base + n;
        l = both_sum(l);
        if (r >= t.rows) return;
        if (t.chunks > 1) {
            float* p = part + (t.slot * part_rows + row_base + n) * (DV + 2);
#pragma unroll
            for (int dt = 0; dt < kDT; ++dt)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    float2* q = reinterpret_cast<float2*>(p + dv_of(dt, g));
                    q[0] = make_float2(O[dt][4 * g], O[dt][4 * g + 1]);
                    q[1] = make_float2(O[dt][4 * g + 2], O[dt][4 * g + 3]);
                }
            if (h == 0) *reinterpret_cast<float2*>(p + DV) = make_float2(m, l);
            return;
        }
        int tok, hd;
        row_of(a, t, row_base + n, tok, hd);
        const int64_t head = (int64_t)t.head * a.G + hd;
        const float inv = inv_sum(l, pos);
        bf16_t* o = static_cast<bf16_t*>(a.o) + (a.packed ? 0 : t.seq * a.so.b) + (t.first + tok) * a.so.t + head * a.so.h;
#pragma unroll
        for (int dt = 0; dt < kDT; ++dt)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                store4(o + dv_of(dt, g), O[dt][4 * g] * inv, O[dt][4 * g + 1] * inv, O[dt][4 * g + 2] * inv, O[dt][4 * g + 3] * inv);
        if (a.lse && h == 0)
            a.lse[(a.packed ? 0 : t.seq * a.Hq * a.T) + head * a.T + t.first + tok] =
                l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    }
};

// The tile and chunk of this workgroup; false behind the last.
template <bool NARROW>
__device__ __forceinline__ bool find_tile(const AttnArgs& a, Tile& t) {
    Place p;
    int all_cuts = 0;
    const bool found = find_place<NARROW, false>(a, blockIdx.x, p, all_cuts);
    if (blockIdx.x == 0 && threadIdx.x == 0) static_cast<int*>(a.ws)[NARROW ? 0 : 1] = all_cuts;
    if (!found) return false;
    t.seq = uniform((int)p.seq);
    t.first = uniform((int)p.first);
    t.n = uniform(p.n);
    t.kv = uniform(p.kv);
    t.rows = t.n * a.G;
    const int rest = uniform(div_by(p.index, a.mHk));
    t.head = uniform(p.index - rest * a.Hk);
    t.chunks = uniform(p.chunks);
    constexpr int R = NARROW ? kNarrowRows : kWideRows;
    const int q = uniform(rest / t.chunks), tile = tiles_of(a, t.n, NARROW) - 1 - q;     // the tiles with the most keys first
    t.chunk = rest - q * t.chunks;
    t.row0 = tile * R;
    t.tok0 = uniform(t.row0 / a.G);
    t.rem0 = t.row0 - t.tok0 * a.G;
    t.slot = p.slot + ((int64_t)tile * a.Hk + t.head) * t.chunks + t.chunk;
    const int r1 = t.row0 + R < t.rows ? t.row0 + R : t.rows;
    int tok1, hd1;
    row_of(a, t, r1 - 1 - t.row0, tok1, hd1);
    const int p0 = t.kv - t.n + t.tok0, p1 = t.kv - t.n + tok1;
    t.hi = uniform(p1 + 1 > 0 ? p1 + 1 : 0);
    const int64_t w0 = a.window > 0 ? (int64_t)p0 - a.window + 1 : 0;
    t.lo = uniform(w0 > 0 ? (int)w0 : 0);
    return true;
}

// Keys [from, to) of this chunk: whole units from the unit of t.lo on.
__device__ __forceinline__ void chunk_keys(const Tile& t, int& from, int& to) {
    const int u0 = t.lo / kUnit, u1 = (t.hi + kUnit - 1) / kUnit;
    const int per = uniform(u1 > u0 ? (u1 - u0 + t.chunks - 1) / t.chunks : 0);
    from = (u0 + t.chunk * per) * kUnit;
    to = from + per * kUnit;
    to = uniform(to < t.hi ? to : t.hi);
}

__device__ __forceinline__ float* partials(const AttnArgs& a, bool narrow) {
    char* p = static_cast<char*>(a.ws) + kHeadBytes;
    if (!narrow && has_narrow(a)) p += slots_most(true) * partial_bytes(kNarrowRows, a.dv);
    return reinterpret_cast<float*>(p);
}

// ---- wide tiles: eight waves of 32 rows share blocks of 64 keys in LDS -----------------------------
//
// The waves form two groups of four, one of each on every SIMD, half a step apart: while one group
// multiplies (the scores of block i and the values of block i - 1) the other does the softmax of its
// scores, so that the SIMD's matrix and vector units work at once. Phase 2i is the first group's
// products of step i and the second's softmax of step i - 1, phase 2i + 1 the other way round; a barrier
// ends each. LDS holds four blocks of keys and values. In its softmax of block i a wave asks for its
// share of block i + 2 (first group) or i + 3 (second): a block's place is free by then, and what is
// asked for is awaited at the barrier before phase 2j, three or four phases later.
//
// Products and their operands bound it, 4 G dk + 4 G dv flops a token and key: 4096 tokens of 32 + 8 heads of 128 over
// 65536 keys take 3720 to 3970 us (from card to card; 1.07 to 1.15 PFLOP/s where a large matrix product reaches 1.38), an 8K
// prompt 532 to 567. A wave has 32 queries, so that each operand of K or V is read from LDS for one product, 1 KB in 32
// cycles of a SIMD: at full rate the four SIMDs would read the 128 bytes a cycle that LDS gives. The matrix units (and
// so LDS) are busy 54 % of the time, the vector units 54 %, little of it at once (45 and 49 % for the prompt), at a
// clock that this load takes down from 2.4 to 1.86 GHz. 256 rows: every key that is read from L2 serves as many rows as
// the registers of eight waves hold; the causal edge costs half a tile. Tiles of four waves, all in step, took 4208 and
// 590 us; blocks asked for in the product phase instead of the softmax leave the prompt at 815 TFLOP/s.

template <int DK, int DV>
__global__ __launch_bounds__(kWideThreads, 2) void attn_wide_kernel(AttnArgs a) {
    constexpr int KB = 64, KBYTES = KB * DK * 2, VBYTES = KB * DV * 2;
    typedef Wave<DK, DV, KB> W;
    typedef Loader<TileK<DK>, KB, kWideWaves> LK;
    typedef Loader<TileV<DV>, KB, kWideWaves> LV;
    __shared__ __align__(1024) char smem[4][KBYTES + VBYTES];
    Tile t;
    if (!find_tile<false>(a, t)) return;
    const int w = uniform(threadIdx.x >> 6);
    int from, to;
    chunk_keys(t, from, to);
    const int nb = to > from ? (to - from + KB - 1) / KB : 0;
    W wave;
    wave.start(a, t, 32 * w);
    if (nb > 0) {
        Pages pg(a, t.seq, t.head, from);
        const LK lk(a.skc, a.page_size, w);
        const LV lv(a.svc, a.page_size, w);
        const uint32_t lds = lds_address(smem);
        int asked = 0;
        auto ask = [&]() {
            if (asked >= nb) return;
            const uint32_t at = lds + (asked & 3) * (KBYTES + VBYTES);
            Block<KB> b;
            b.find(pg, lk, lv, from + asked * KB, t.hi);
            b.load(lk, b.k, at);
            b.load(lv, b.v, at + KBYTES);
            pg.advance(KB);
            ++asked;
        };
        // The next block where that takes no branch: pages of a power of two rows, whose addresses are held. Each
        // load's rows are in one page.
        auto ask_plain_ok = [&]() {
            const int end = from + (asked + 1) * KB;
            return a.page_shift >= 0 && asked < nb && end <= t.hi && ((end - 1) >> a.page_shift) - pg.base < 64;
        };
        auto ask_plain = [&]() {
            const uint32_t at = lds + (asked & 3) * (KBYTES + VBYTES);
            const int kb = from + asked * KB, mask = pg.page_size - 1;
            i32x4 k, v;
#pragma unroll
            for (int i = 0; i < LK::kLoads; ++i) {
                const int key = kb + lk.first_row(i);
                if (i == 0 || a.page_shift < 6)      // a page of 64 rows holds the block
                    pg.held_descriptors((key >> a.page_shift) - pg.base, pg.page_size, lk, lv, k, v);
                lk.load_whole(k, i, key & mask, at);
                if (LK::kLoads == LV::kLoads) lv.load_whole(v, i, key & mask, at + KBYTES);
            }
            if (LK::kLoads != LV::kLoads)
#pragma unroll
                for (int i = 0; i < LV::kLoads; ++i) {
                    const int key = kb + lv.first_row(i);
                    pg.held_descriptors((key >> a.page_shift) - pg.base, pg.page_size, lk, lv, k, v);
                    lv.load_whole(v, i, key & mask, at + KBYTES);
                }
            pg.pg = (kb + KB) >> a.page_shift;
            pg.row = (kb + KB) & mask;
            ++asked;
        };
        // before phase 2i: this wave's share of block i has landed (block i + 1 may be on its way), then everyone's
        auto even = [&](int i) {
            if (i + 1 < nb)
                wait_vm<LK::kLoads + LV::kLoads>();
            else
                wait_vm<0>();
            __builtin_amdgcn_sched_barrier(0);
            lds_barrier();
        };
        auto odd = [&]() {
            __builtin_amdgcn_sched_barrier(0);
            lds_barrier();
        };
        const bool second = w >= 4;
        ask();
        ask();
        if (second) ask();
        typename W::Scores S;
        typename W::Probs P;
        if (second) even(0);
        bool seen = false;
        // steps whose blocks i and i - 1 every row sees whole, and the others (the first and the last among them),
        // in loops of their own (the waves change over at different steps, but pass the same barriers): O stays
        // in one place through either
        // blocks plain0 .. plain1 - 1 every row sees whole
        const int64_t w0 = a.window > 0 ? (int64_t)wave.last - a.window + 1 - from : 0;
        const int plain0 = uniform(w0 > 0 ? (int)((w0 + KB - 1) / KB) : 0);
        const int plain1 = uniform(wave.first - KB + 1 >= from ? (wave.first - KB + 1 - from) / KB + 1 : 0);
        auto plain = [&](int i) { return i > plain0 && i < plain1 && i < nb; };
        int i = 0;
        while (i <= nb) {
            for (; plain(i) && ask_plain_ok(); ++i) {
                if (second) odd(); else even(i);
                wave.scores_values(smem[i & 3], S, smem[(i - 1) & 3] + KBYTES, P);
                if (second) even(i + 1); else odd();
                ask_plain();
                wave.template softmax<0>(a, S, P, 0);
                seen = true;
            }
            for (; plain(i) && !ask_plain_ok(); ++i) {
                if (second) odd(); else even(i);
                wave.scores_values(smem[i & 3], S, smem[(i - 1) & 3] + KBYTES, P);
                if (second) even(i + 1); else odd();
                ask();
                wave.template softmax<0>(a, S, P, 0);
                seen = true;
            }
            for (; i <= nb && !plain(i); ++i) {
                if (second) odd(); else even(i);
                const int kb = from + i * KB;
                const bool sees = i < nb && wave.sees(a, kb);
                if (sees) wave.scores(smem[i & 3], S);
                if (seen) wave.values(a, smem[(i - 1) & 3] + KBYTES, P, kb - KB);
                if (i < nb) {
                    if (second) even(i + 1); else odd();
                    ask();
                    if (sees) wave.template softmax<1>(a, S, P, kb);
                } else if (!second) {
                    odd();
                }
                seen = sees;
            }
        }
    }
    wave.finish(a, t, 32 * w, partials(a, false), kWideRows);
}

// ---- narrow tiles: four waves with the same 32 rows, each its own blocks of 32 keys ----------------
//
// The bytes of the keys and values bound it, where there is enough of them: 256 sequences of one token over up to 16384
// keys (8.62 GB) take 1490 us, 5.8 TB/s, at 8 key heads of 128; one token over 8192 15.2 us (34 MB; 11.1 of it here, 4.4
// in the join), which is the latency from the lengths to the table to the keys to the join. Rows that G and the new
// tokens do not fill (28 of 32 there) cost products that HBM hides: the matrix units are busy 8 % of the time. Eight waves
// and half as many workgroups: 48 us against 37 for 34 sequences over up to 31333 keys of pages of 16, 26.6 against 28.8
// for 16 sequences over 1900.

template <int DK, int DV>
__global__ __launch_bounds__(kThreads, 2) void attn_narrow_kernel(AttnArgs a) {
    constexpr int KB = 32, KBYTES = KB * DK * 2, VBYTES = KB * DV * 2;
    constexpr int kJoin = 32 * (DV + 2) * 4;            // a wave's result, for the join at the end
    constexpr int kWaveBytes = KBYTES + VBYTES > kJoin ? KBYTES + VBYTES : (kJoin + 1023) / 1024 * 1024;
    __shared__ __align__(1024) char smem[kWaves][kWaveBytes];
    Tile t;
    if (!find_tile<true>(a, t)) return;
    const int w = uniform(threadIdx.x >> 6);
    int from, to;
    chunk_keys(t, from, to);
    Wave<DK, DV, KB> wave;
    wave.start(a, t, 0);
    const int mine = from + KB * w;
    Pages pg(a, t.seq, t.head, mine);
    const Loader<TileK<DK>, KB, 1> lk(a.skc, a.page_size, 0);
    const Loader<TileV<DV>, KB, 1> lv(a.svc, a.page_size, 0);
    const uint32_t lds = lds_address(smem[w]);
    // A wave's keys of the next block are asked for once its scores are through with LDS, its values once the
    // products are: one block of LDS a wave, and loads under way all the time.
    Block<KB> b;
    if (mine < to) {
        b.find(pg, lk, lv, mine, t.hi);
        b.load(lk, b.k, lds);
        b.load(lv, b.v, lds + KBYTES);
    }
#pragma unroll 1
    for (int kb = mine; kb < to; kb += KB * kWaves) {
        const bool more = kb + KB * kWaves < to, sees = wave.sees(a, kb), masked = wave.masks(a, kb);
        typename Wave<DK, DV, KB>::Scores S;
        typename Wave<DK, DV, KB>::Probs P;
        wait_vm<Loader<TileV<DV>, KB, 1>::kLoads>();           // the keys; the values may be on their way
        if (sees) wave.scores(smem[w], S);
        wave_lds_sync();
        if (more) {
            pg.advance(KB * kWaves);
            b.find(pg, lk, lv, kb + KB * kWaves, t.hi);
            b.load(lk, b.k, lds);
        }
        if (sees) wave.template softmax<2>(a, S, P, kb, masked);
        if (more)
            wait_vm<Loader<TileK<DK>, KB, 1>::kLoads>();
        else
            wait_vm<0>();
        if (sees) {
            if (masked && wave.template bad_values<true>(a, smem[w] + KBYTES, kb)) {
                wave.mark_bad(smem[w] + KBYTES, kb);
                wave_lds_sync();
                wave.clear_bad(smem[w] + KBYTES);
                wave_lds_sync();
            }
            wave.plain_values(smem[w] + KBYTES, P);
        }
        wave_lds_sync();
        if (more) b.load(lv, b.v, lds + KBYTES);
    }
    // join the waves: every wave leaves m, l, O in LDS; wave w takes the rows' channels in turn
    lds_barrier();
    constexpr int DT = DV / 32;
    const int n = threadIdx.x & 31, h = (threadIdx.x >> 5) & 1;
    wave.l = both_sum(wave.l);
    float* js = reinterpret_cast<float*>(smem[w]);
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int e = 0; e < 4; ++e) js[n * (DV + 2) + Wave<DK, DV, KB>::dv_of(dt, g) + e] = wave.O[dt][4 * g + e];
    if (h == 0) {
        js[n * (DV + 2) + DV] = wave.m;
        js[n * (DV + 2) + DV + 1] = wave.l;
    }
    lds_barrier();
    float* part = partials(a, true);
    const int rows = t.rows - t.row0 < kNarrowRows ? t.rows - t.row0 : kNarrowRows;
    for (int r = w; r < rows; r += kWaves) {
        const int lane = threadIdx.x & 63;
        float mw[kWaves], mm = -INFINITY;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) {
            mw[i] = reinterpret_cast<const float*>(smem[i])[r * (DV + 2) + DV];
            mm = fmaxf(mm, mw[i]);
        }
        float acc[DV / 64], ll = 0.f;
#pragma unroll
        for (int k = 0; k < DV / 64; ++k) acc[k] = 0.f;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) {
            const float* src = reinterpret_cast<const float*>(smem[i]) + r * (DV + 2);
            // 1 where no wave has a reference: sums are 0 then, or NaN, and O is 0, or NaN from values
            const float lw = src[DV + 1], f = mw[i] == mm ? 1.f : __builtin_amdgcn_exp2f(mw[i] - mm);
            ll = fmaf(f, lw, ll);
#pragma unroll
            for (int k = 0; k < DV / 64; ++k) acc[k] = fmaf(f, src[lane + 64 * k], acc[k]);
        }
        if (t.chunks > 1) {
            float* p = part + (t.slot * kNarrowRows + r) * (DV + 2);
#pragma unroll
            for (int k = 0; k < DV / 64; ++k) p[lane + 64 * k] = acc[k];
            if (lane == 0) {
                p[DV] = mm;
                p[DV + 1] = ll;
            }
            continue;
        }
        int tok, hd;
        row_of(a, t, r, tok, hd);
        const int64_t head = (int64_t)t.head * a.G + hd;
        const float inv = inv_sum(ll, t.kv - t.n + tok);
        bf16_t* o = static_cast<bf16_t*>(a.o) + (a.packed ? 0 : t.seq * a.so.b) + (t.first + tok) * a.so.t + head * a.so.h;
#pragma unroll
        for (int k = 0; k < DV / 64; ++k) st_f(o + lane + 64 * k, acc[k] * inv);
        if (a.lse && lane == 0)
            a.lse[(a.packed ? 0 : t.seq * a.Hq * a.T) + head * a.T + t.first + tok] =
                ll == 0.f ? -INFINITY : (mm + log2f(ll)) * 0.6931471805599453f;
    }
}

// ---- the chunks of cut tiles joined ---------------------------------------------------------------

// The workgroups (join_groups) share out the rows of all cut (tile, head)s: a wave a row or, where a row has more
// chunks than a wave keeps loads under way for, a workgroup a row. A lane holds 4 channels, so that a wave
// reads kJoinAhead * (256 / DV) chunks at a time. Latency bounds it: one token over 48K keys of one key head of 64, 380
// chunks of 16 rows, 7 us (31 with a wave a row); 4.0 us for 8 x 64 chunks of 4 rows, 2.1 with nothing to join.
constexpr int kJoinAhead = 8;

// Chunks [c0, c1) of a row: their reference, sum and this lane's channels, the same in all lanes that hold them.
template <int DV>
__device__ __forceinline__ void join_chunks(const float* base, int64_t step, int c0, int c1, float& mm, float& ll, float4& acc) {
    constexpr int LPR = DV / 4, NG = 64 / LPR, AT = kJoinAhead * NG;
    const int lane = threadIdx.x & 63, g = lane / LPR, ch = lane % LPR;
    mm = -INFINITY;
    ll = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (; c0 < c1; c0 += AT) {
        const int left = uniform(c1 - c0);
        float2 ml = make_float2(-INFINITY, 0.f), u[kJoinAhead], v[kJoinAhead];
        if (lane < AT && lane < left) ml = *reinterpret_cast<const float2*>(base + (c0 + lane) * step + DV);
#pragma unroll
        for (int k = 0; k < kJoinAhead; ++k) {
            const int c = k * NG + g;
            if (k * NG >= left) continue;
            const float2* q = reinterpret_cast<const float2*>(base + (c0 + (c < left ? c : left - 1)) * step + 4 * ch);
            u[k] = q[0];
            v[k] = q[1];
        }
        float top = fmaxf(ml.x, mm);
#pragma unroll
        for (int k = 1; k < 64; k <<= 1) top = fmaxf(top, __shfl_xor(top, k));
        const float old = mm == top ? 1.f : __builtin_amdgcn_exp2f(mm - top);
        mm = top;
        const float f = ml.y == 0.f ? 0.f : __builtin_amdgcn_exp2f(ml.x - top);     // a sum of 0: saw no key
        ll = fmaf(ll, old, f * ml.y);
        acc.x *= old; acc.y *= old; acc.z *= old; acc.w *= old;
#pragma unroll
        for (int k = 0; k < kJoinAhead; ++k) {
            const int c = k * NG + g;
            if (k * NG >= left) continue;
            const float wf = __shfl(f, c);
            if (c < left) {
                acc.x = fmaf(wf, u[k].x, acc.x); acc.y = fmaf(wf, u[k].y, acc.y);
                acc.z = fmaf(wf, v[k].x, acc.z); acc.w = fmaf(wf, v[k].y, acc.w);
            }
        }
    }
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) ll += __shfl_xor(ll, k);
#pragma unroll
    for (int k = LPR; k < 64; k <<= 1) {
        acc.x += __shfl_xor(acc.x, k); acc.y += __shfl_xor(acc.y, k);
        acc.z += __shfl_xor(acc.z, k); acc.w += __shfl_xor(acc.w, k);
    }
}

template <int DV, bool NARROW>
__global__ __launch_bounds__(kJoinThreads) void attn_join_kernel(AttnArgs a) {
    constexpr int R = NARROW ? kNarrowRows : kWideRows, NW = kJoinThreads / 64;
    constexpr int LPR = DV / 4, NG = 64 / LPR;
    __shared__ __align__(16) float all[NW][DV + 4];
    const int cuts = static_cast<const int*>(a.ws)[NARROW ? 0 : 1];
    if (cuts <= 0) return;
    // workgroups of a cut; lengths that break the rules may make more cuts than there are workgroups
    const int each = (int)gridDim.x / cuts, share = uniform(each > 0 ? each : 1), cut = uniform(blockIdx.x / share);
    const int part = blockIdx.x - cut * share;
    Place p;
    int all_cuts;
    if (cut >= cuts || !find_place<NARROW, true>(a, cut, p, all_cuts)) return;
    const int C = p.chunks, tile = div_by(p.index, a.mHk), head_k = p.index - tile * a.Hk;
    const int rows = p.n * a.G - tile * R < R ? p.n * a.G - tile * R : R;
    const int64_t slot = p.slot + ((int64_t)tile * a.Hk + head_k) * C, step = (int64_t)R * (DV + 2);
    const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6);
    const bool shared = C > kJoinAhead * NG;
    const int per = shared ? uniform((C + NW - 1) / NW) : C, c0 = shared ? w * per : 0, c1 = c0 + per < C ? c0 + per : C;
    for (int rr = shared ? part : part * NW + w; rr < rows; rr += shared ? share : share * NW) {
        float mm, ll;
        float4 acc;
        join_chunks<DV>(partials(a, NARROW) + (slot * R + rr) * (DV + 2), step, c0, c1, mm, ll, acc);
        if (shared) {
            __syncthreads();
            if (lane < LPR) *reinterpret_cast<float4*>(&all[w][4 * lane]) = acc;
            if (lane == 0) {
                all[w][DV] = mm;
                all[w][DV + 1] = ll;
            }
            __syncthreads();
            if (w > 0) continue;
            const float mw = all[lane % NW][DV];
            ll = all[lane % NW][DV + 1];
            mm = mw;
#pragma unroll
            for (int k = 1; k < NW; k <<= 1) mm = fmaxf(mm, __shfl_xor(mm, k));
            const float f = ll == 0.f ? 0.f : __builtin_amdgcn_exp2f(mw - mm);
            ll *= f;
#pragma unroll
            for (int k = 1; k < NW; k <<= 1) ll += __shfl_xor(ll, k);
            acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                const float wf = __shfl(f, i);
                const float4 x = *reinterpret_cast<const float4*>(&all[i][4 * (lane % LPR)]);
                acc.x = fmaf(wf, x.x, acc.x); acc.y = fmaf(wf, x.y, acc.y);
                acc.z = fmaf(wf, x.z, acc.z); acc.w = fmaf(wf, x.w, acc.w);
            }
        }
        if (lane < LPR) {
            const int r = tile * R + rr, tok = r / a.G, hd = r - tok * a.G;
            const int64_t head = (int64_t)head_k * a.G + hd;
            const float inv = inv_sum(ll, p.kv - p.n + tok);
            bf16_t* o = static_cast<bf16_t*>(a.o) + (a.packed ? 0 : p.seq * a.so.b) + (p.first + tok) * a.so.t + head * a.so.h;
            store4(o + 4 * lane, acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
            if (a.lse && lane == 0)
                a.lse[(a.packed ? 0 : p.seq * a.Hq * a.T) + head * a.T + p.first + tok] =
                    ll == 0.f ? -INFINITY : (mm + log2f(ll)) * 0.6931471805599453f;
        }
    }
}

}  // namespace attn
}  // namespace kda
