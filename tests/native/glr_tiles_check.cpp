// Host-side walk over the tile geometry of the gated linear recurrence (kda_glr_tiles.h): every
// channel of every head belongs to one tile, every tile to one workgroup. Built and run by
// tests/test_glr_tiles.py.
#include <stdint.h>
#include <stdio.h>

#include <vector>

#include "kda_glr_tiles.h"

using kda::glr::Place;
using kda::glr::kCW;

#define CHECK(cond, ...)                                                          \
    do {                                                                          \
        if (!(cond)) {                                                            \
            fprintf(stderr, "FAIL %s:%d: %s: ", __FILE__, __LINE__, #cond);       \
            fprintf(stderr, __VA_ARGS__);                                         \
            return 1;                                                             \
        }                                                                         \
    } while (0)

// Channels of `blocks` heads of d channels: which tile has them, by a thread's vector (VEC channels a
// thread, as they are loaded and stored) and by a lane of one channel (chain words, states).
template <bool NARROW, int VEC>
static int walk(uint32_t d, int64_t blocks) {
    const int64_t per = NARROW ? kda::glr::heads_a_tile(d) : 1, ntc = NARROW ? 1 : (d + kCW - 1) / kCW;
    const int64_t chains = kda::glr::chain_count(blocks, d, NARROW);
    std::vector<int64_t> vec((size_t)(blocks * d), -1), lane(vec);
    for (int64_t chain = 0; chain < chains; ++chain) {
        const int64_t block0 = chain / ntc * per;
        for (int l = 0; l < kCW; ++l) {
            const Place<NARROW, VEC> own(l / VEC * VEC, (uint32_t)(chain % ntc), d, blocks - block0);
            // loads run for places without channels too: inside the head, of a block that is there
            CHECK(own.ch + VEC <= d && block0 + own.local < blocks, "d = %u, lane %d\n", d, l);
            if (!own.on) continue;
            for (int v = 0; v < VEC; ++v) {
                int64_t& owner = vec[(size_t)((block0 + own.local) * d + own.ch + v)];
                CHECK(owner < 0 || owner == chain, "d = %u: channel %u of tiles %lld and %lld\n", d, own.ch + v,
                      (long long)owner, (long long)chain);
                owner = chain;
            }
            lane[(size_t)((block0 + own.local) * d + own.ch + l % VEC)] = chain;
        }
    }
    for (size_t i = 0; i < vec.size(); ++i)
        CHECK(vec[i] >= 0 && lane[i] == vec[i], "d = %u: channel %llu has no tile\n", d, (unsigned long long)(i % d));
    return 0;
}

int main() {
    for (uint32_t d = 1; d <= 520; ++d)
        if (d < 4 ? walk<false, 1>(d, 3) : walk<false, 4>(d, 3)) return 1;
    for (uint32_t d : {1000u, 1023u, 1024u, 1025u, 1026u, 1027u, 1028u, 66049u, 1u << 20, (1u << 20) - 61, (1u << 20) - 62, (1u << 20) - 63})
        if (walk<false, 4>(d, 1)) return 1;
    for (uint32_t d = 4; d <= 32; ++d)
        for (int64_t blocks : {1, 2, 15, 16, 17, 100})
            if (walk<true, 4>(d, blocks)) return 1;
    // the workgroups of a round take every chain once
    for (uint32_t chains : {1u, 7u, 8u, 9u, 1023u, 1026u, 8008u}) {
        std::vector<int> taken(chains, 0);
        for (uint32_t p = 0; p < chains; ++p) {
            const uint32_t c = kda::glr::chain_of(p, chains);
            CHECK(c < chains && ++taken[c] == 1, "%u chains, place %u\n", chains, p);
        }
    }
    printf("glr tiles check: ok\n");
    return 0;
}
