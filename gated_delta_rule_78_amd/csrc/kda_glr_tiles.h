// Tile geometry of the gated linear recurrence: which channels and blocks of rows a thread of a tile
// works on, and the order in which tiles are taken. Arithmetic alone, for the kernels and the host.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {
namespace glr {

// A tile is some rows of kCW channels, in the registers of THREADS threads: CT lanes lie across the
// channels with VEC channels each (VEC = 4, or 1 for heads of fewer), and each run of CT lanes owns L
// consecutive rows, a sub-chunk. Where the channels are no multiple of VEC, the last lane's are the
// tile's last VEC: those it shares with its neighbour are computed, and written, twice alike. No two
// tiles share a channel: one may have written its final states before the other reads its initial
// ones, which are the same memory where the states are updated in place.
constexpr int kCW = 64;
template <int VEC, int L, int THREADS>
struct Tile {
    static constexpr int CT = kCW / VEC;            // threads across the channels
    static constexpr int SPW = 64 / CT;             // sub-chunks per wave
    static constexpr int W = THREADS / 64;          // waves
    static constexpr int ROWS = THREADS / CT * L;
};

// Narrow heads (d <= kCW / 2) lie side by side in a tile: 4-channel slots of ceil(d / 4) a head.
__host__ __device__ inline uint32_t heads_a_tile(int64_t d) {
    return d > kCW / 2 || d < 4 ? 1 : kCW / (((uint32_t)d + 3) & ~3u);
}
// Tiles across the channels, all blocks together: the chains.
__host__ __device__ inline int64_t chain_count(int64_t blocks, int64_t d, bool narrow) {
    const int64_t n = narrow ? heads_a_tile(d) : 1;
    return n > 1 ? (blocks + n - 1) / n : blocks * ((d + kCW - 1) / kCW);
}
// The first channel of a head's t'th tile (behind the last: d). A last tile that would have fewer
// channels than a vector takes 4 more from the tile before it.
__host__ __device__ __forceinline__ uint32_t tile_begin(uint32_t t, uint32_t d) {
    const uint32_t ch = t * kCW;
    if (ch >= d) return d;
    return ch > 0 && d - ch < 4 ? ch - 4 : ch;
}
// Where a thread's VEC channels lie that has the slot'th channel of tile t across a head: the block
// counted from the tile's first (`left` of them are there), the first channel, and whether there are any.
template <bool NARROW, int VEC>
struct Place {
    uint32_t local, ch;
    bool on;
    __host__ __device__ __forceinline__ Place(int slot, uint32_t t, uint32_t d, int64_t left) {
        local = 0;
        int end = (int)d;
        if constexpr (NARROW) {
            const uint32_t width = (d + 3) & ~3u;
            local = (uint32_t)slot / width;
            slot -= (int)(local * width);
            on = local < kCW / width && local < left;
            if (!on) local = 0;
        } else {
            end = (int)tile_begin(t + 1, d);
            slot += (int)tile_begin(t, d);
            on = slot < end;
        }
        ch = slot + VEC <= end ? slot : end - VEC;
    }
};

// Tiles of a chain are taken from a counter, one for every kCounters-th chain, a cache line each.
constexpr uint32_t kCounters = 1024, kCounterStride = 32;

// The chain of the p'th workgroup of a round over all of them. Workgroups go to the 8 XCDs in turn, so
// neighbouring chains get places 8 apart: where rows do not start on cache lines, chains of the same
// rows share lines, which one L2 then holds and writes whole (8 x 4096 rows of 1001 bf16 channels: 43 us
// against 63; 64 x 4096 rows of 100: 38 against 54).
__host__ __device__ __forceinline__ uint32_t chain_of(uint32_t p, uint32_t chains) {
    const uint32_t x = p % 8, each = chains / 8, more = chains % 8;
    return x * each + (x < more ? x : more) + p / 8;
}

// The tile of ticket k: a counter serves every kCounters-th chain, first tiles first.
__host__ __device__ __forceinline__ void next_tile(uint32_t k, uint32_t chains, uint32_t& c, uint32_t& chain) {
    const uint32_t g = chain % kCounters, n = (chains - g + kCounters - 1) / kCounters;
    c = k / n;
    chain = g + kCounters * (k % n);
}

}  // namespace glr
}  // namespace kda
