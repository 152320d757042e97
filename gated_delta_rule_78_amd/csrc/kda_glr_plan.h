// Which kernels a call of the gated linear recurrence takes, and whether their launches can be made.
// Host arithmetic alone, shared by the dispatch (kda_glr.hip) and the argument checks (kda_glr_abi.cpp).
#pragma once

#include "kda_glr.h"
#include "kda_glr_internal.h"
#include "kda_glr_tiles.h"

namespace kda {
namespace glr {

// Whether threads of up to 4 channels walk the rows one by one (kda_glr_rows.hip) instead of tiles of
// 256 of them: short sequences, which would leave a tile's threads idle, and middling ones where there
// are channels enough to fill the GPU. bf16 with gates, 32 heads of 128 channels, by rows / in tiles:
// 512 x 16 rows 49 us / 560, 64 x 64 rows 31 / 75, 64 x 128 rows 70 / 82; 16 x 64 rows 29 / 23,
// 4 x 64 rows 28 / 13.
inline bool by_rows(const GlrArgs& a) {
    if (a.packed || a.T > KDA_GLR_CHUNK) return false;
    return a.T <= 16 || a.blocks * a.d >= (int64_t)1 << 18;
}
inline bool bwd_by_rows(const GlrArgs& a) { return !a.packed && a.T <= kRowsBwd; }   // too few for a tile's threads

// The tiles of a launch: rows per tile, tiles per block, channels per thread, heads side by side.
struct Tiling {
    int64_t rows, nt;
    int vec;
    bool narrow;
};
inline Tiling tiling(const GlrArgs& a, bool backward) {
    Tiling t;
    t.vec = a.d >= 4 ? 4 : 1;
    t.rows = backward ? kBwdRows : t.vec == 4 ? kFwdRows : kFwdRows1;
    t.nt = (a.T + t.rows - 1) / t.rows;
    // Narrow heads share tiles where one each would fill the GPU (1024 x 4096 rows of 8 channels: 70 us
    // against 180); fewer stay apart, each tile's work being a wave's latency (8 x 4096 rows: 15.8 us
    // against 16.3, 4 x 20000 rows of 16 channels: 26.5 against 30.3). 32-bit offsets inside a tile.
    const int64_t per = heads_a_tile(a.d);
    t.narrow = per > 1 && a.blocks * t.nt >= 1024 && per * a.T * a.d < (int64_t)1 << 31;
    return t;
}

// Workgroups of the launches: of tiles (kTileThreads threads each), by rows (kRowsThreads), of dA_log's sum
// (kDAThreads; the first of its two launches has as many in x).
constexpr int kTileThreads = 512, kRowsThreads = 256, kDAThreads = 1024;
inline int64_t tile_groups(const GlrArgs& a, const Tiling& t) { return chain_count(a.blocks, a.d, t.narrow) * t.nt; }
inline int64_t rows_groups(const GlrArgs& a) {
    return (a.blocks * (a.d % 4 == 0 ? a.d / 4 : a.d) + kRowsThreads - 1) / kRowsThreads;
}
inline int64_t dA_groups(const GlrArgs& a) { return (a.d + 63) / 64 * a.H; }

// A launch numbers its threads with 32 bits.
inline bool launchable(int64_t groups, int threads) { return groups < ((int64_t)1 << 32) / threads; }
inline bool step_launchable(const GlrArgs& a) { return launchable(rows_groups(a), kRowsThreads); }
inline bool fwd_launchable(const GlrArgs& a) {
    if (a.T == 0) return true;
    if (by_rows(a)) return launchable(rows_groups(a), kRowsThreads);
    return launchable(tile_groups(a, tiling(a, false)), kTileThreads);
}
// Without entry states the backward runs the forward too; with z it sums dA_log.
inline bool bwd_launchable(const GlrArgs& a) {
    if (a.T == 0) return true;
    if (a.z && !launchable(dA_groups(a), kDAThreads)) return false;
    if (bwd_by_rows(a)) return launchable(rows_groups(a), kRowsThreads);
    return launchable(tile_groups(a, tiling(a, true)), kTileThreads) && (a.entry || fwd_launchable(a));
}

}  // namespace glr
}  // namespace kda
