// How the attention over a paged cache is cut into work, shared by its kernels and its host side.
//
// The G query heads of a key head are rows of one matrix: row r of a sequence is token r / G, head
// r % G of the group, so that all of them read each key once. A sequence's rows make tiles, narrow
// ones where it has at most narrow_most() rows (the waves of a workgroup then share out the keys), wide
// ones else (the waves share out the rows). A tile's keys are cut into C chunks, C the same for every
// tile of a sequence: ceil(keys / L), L such that the keys of all tiles make about target() chunks.
// Chunks of a cut tile leave their sums in the workspace and a second launch joins them. Every wave
// works out from the lengths which sequence and chunk its workgroup has: 64 sequences take one round
// of loads and a scan over the lanes, as long as it would take to read a list made by another launch.
#pragma once

#include <math.h>
#include <stdint.h>

#include "kda_attn_internal.h"

namespace kda {
namespace attn {

// Times of both sides of a rule are of calls over one set of inputs, which the caches may hold: one token over 8192 keys
// takes 13.7 to 14.1 us then, 15.2 with inputs in turn.
constexpr int kThreads = 256, kWaves = 4;          // narrow tiles
constexpr int kWideThreads = 512, kWideWaves = 8;  // wide tiles
constexpr int kJoinThreads = 256, kJoinGroups = 1024;   // workgroups at most: at least the (tile, head)s that can be cut
constexpr int kNarrowRows = 32, kWideRows = 256;
constexpr int kUnit = 128;             // keys: what L counts in
// A tile of at most so many units is not cut, of `tiles` (tile, head)s in all: with few of them the keys that
// each chunk saves outweigh the partial results and the join early, with more the chunks of cut tiles no longer
// run at once. Whole against cut, heads of 128, us: 8 tiles of 3 units 11.1 : 13.7; 32 tiles, 5 units 16.1 : 14.8;
// 128 tiles, 5, 9 units 14.6 : 17.7, 19.8 : 22.2; 384 tiles, 15 units 71 : 75; wide ones, 8 and 32 tiles of 3 units
// 25.0 : 23.6, 25.4 : 28.3; 128 tiles, 5, 9 units 31 : 40, 43 : 46. Unequal lengths, 75 tiles of up to 12 units
// beside a longer one: 40 : 31.
constexpr float kWholeLeast = 3.f, kWholeMost = 16.f;
__host__ __device__ constexpr float whole_units(float tiles) { return kWholeLeast + (1.f / 16.f) * tiles; }
// Chunks: as many workgroups of a kind as the GPU's 256 CUs hold. Half and twice as many: one token over 8192 keys 15.2 and
// 15.2 us (14.1), 512 tokens over 8000 130 and 110 (92), 8 x 40 tokens over 4000 71 and 69 (53).
__host__ __device__ constexpr int64_t target(bool narrow) { return narrow ? 512 : 256; }

// What the kernels divide by, and a window's reach.
inline uint32_t magic_of(int32_t d) { return d > 1 ? (uint32_t)((((uint64_t)1 << 32) + d - 1) / d) : 0; }
inline void set_divisors(AttnArgs& a) {
    a.mG = magic_of(a.G);
    a.mHk = magic_of(a.Hk);
    for (int k = 0; k < 2; ++k) {
        const int64_t s = a.window + ((k ? kNarrowRows : kWideRows) + a.G - 1) / a.G + kUnit;
        a.span[k] = a.window > 0 && s < 0x7fffffff ? (int32_t)s : 0x7fffffff;
    }
    a.page_shift = -1;
    for (int i = 0; i <= 20; ++i)
        if (a.page_size == 1 << i) a.page_shift = i;
}

// Rows of a sequence that make narrow tiles. Up to one tile's: with wide tiles one token over 8192 keys takes 19.9 us
// against 14.1, 256 sequences of one over up to 16384 1645 against 1490, 32 x 4 tokens of 8 heads of 64 42 against 22.
// Heads of 64: up to 128, each tile reading the keys again (out of
// L2; 32 sequences of 64, 96, 128 rows over 8000 keys: 56, 70, 84 us against 79, 85, 88 with wide tiles). Larger
// heads: one tile's (64, 128 rows in narrow tiles: 115, 180 us against 111, 123).
__host__ __device__ inline int narrow_most(const AttnArgs& a) { return a.dk + a.dv <= 128 ? 128 : kNarrowRows; }

// Keys that the longest tile of a sequence of kv keys reads, in units, and the tiles of its n new tokens.
__host__ __device__ inline int tile_units(const AttnArgs& a, int kv, bool narrow) {
    const int k = kv < a.span[narrow] ? kv : a.span[narrow];
    return k > 0 ? (int)(((uint32_t)k + kUnit - 1) / kUnit) : 1;
}
__host__ __device__ inline int tiles_of(const AttnArgs& a, int n, bool narrow) {
    const uint32_t rows = (uint32_t)n * (uint32_t)a.G;
    const uint32_t each = narrow ? kNarrowRows : kWideRows;
    return (rows <= (uint32_t)narrow_most(a)) == narrow ? (int)((rows + each - 1) / each) : 0;
}

// The chunk length L from the sums over all (tile, head)s: up to `whole` units stay in one chunk, inv = 1 / L. The
// units' sum is taken a hundredth larger, since its rounding may not make L too small: chunks would pass the
// workspace's slots. A tile cut has k > L units in ceil(k / L - 0.001) < 2 k / L chunks, all of them together
// below 2 target(); so there are below target() of them.
struct Cut {
    float whole, inv;
};
__host__ __device__ inline Cut cut_of(float tiles, float units, bool narrow) {
    const float length = fminf(fmaxf(ceilf(units * 1.01f / (float)target(narrow)), 1.f), 16777216.f);
    return {fminf(whole_units(tiles), kWholeMost), 1.f / length};
}
// The main launch and the join both work it out: one rounding, whatever the compiler makes of either.
__host__ __device__ inline int chunks_of(Cut c, int units) {
    return (float)units <= c.whole ? 1 : (int)fmaxf(ceilf(fmaf((float)units, c.inv, -0.001f)), 1.f);
}

// Workspace: two counts, how many (tile, head)s of either kind are cut (the first workgroup of a kind
// writes its one), then the partial results, per kind slots_most() of rows x (DV + 2) floats.
constexpr int64_t kHeadBytes = 256;
__host__ __device__ inline int64_t tiles_most(const AttnArgs& a, int rows, bool narrow) {
    const int64_t all = (a.packed ? a.T : a.N * a.T) * a.G, seqs = a.packed && a.T < a.N ? a.T : a.N;
    const int64_t most = all / rows + seqs, each = narrow_most(a) / kNarrowRows * seqs;
    return narrow && each < most ? each : most;
}
// cut chunks: ceil(k / L) <= 2 k / L of each tile with k > L
__host__ __device__ inline int64_t slots_most(bool narrow) { return 2 * target(narrow); }
__host__ __device__ inline int64_t partial_bytes(int rows, int dv) { return (int64_t)rows * (dv + 2) * 4; }

// Which kinds a call can hold, from what the host knows.
__host__ __device__ inline bool has_narrow(const AttnArgs& a) { return a.packed || a.T * a.G <= narrow_most(a); }
__host__ __device__ inline bool has_wide(const AttnArgs& a) { return a.T * a.G > narrow_most(a); }
// No tile has more keys than the table holds: none is cut when a chunk takes them all.
__host__ __device__ inline bool may_cut(const AttnArgs& a) { return (int64_t)a.max_pages * a.page_size > (int64_t)(kUnit * kWholeLeast); }


// Workgroups at most: every tile once, and the chunks beyond the first of each.
inline int64_t groups_most(const AttnArgs& a, bool narrow) {
    const int64_t tiles = tiles_most(a, narrow ? kNarrowRows : kWideRows, narrow) * a.Hk;
    return tiles + (may_cut(a) ? target(narrow) : 0);
}
// A launch has fewer than 2^32 threads.
inline bool too_many(const AttnArgs& a) {
    return (has_narrow(a) && groups_most(a, true) >= (int64_t)1 << 23) || (has_wide(a) && groups_most(a, false) >= (int64_t)1 << 23);
}

// Workgroups of the join: one a row of all (tile, head)s that can be cut, up to kJoinGroups.
inline int64_t join_groups(const AttnArgs& a, bool narrow) {
    const int rows = narrow ? kNarrowRows : kWideRows;
    const int64_t tiles = tiles_most(a, rows, narrow) * a.Hk, each = a.T * a.G < rows ? a.T * a.G : rows;
    const int64_t cuts = tiles < target(narrow) ? tiles : target(narrow);
    return cuts * each < kJoinGroups ? cuts * each : kJoinGroups;
}

}  // namespace attn
}  // namespace kda
