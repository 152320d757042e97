// Host-side check of what the attention's workspace and launches rest on (kda_attn_plan.h): over drawn and adversarial
// lengths the kernels' arithmetic, sums over 64 lanes in their order among it, cuts no more chunks than the workspace
// has slots for, no more tiles than the join has workgroups for, and a call within the rules no more workgroups than
// are launched. Built and run by tests/test_attn_plan.py.
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <random>
#include <vector>

#include "kda_attn_plan.h"

#define CHECK(cond)                                                               \
    do {                                                                          \
        if (!(cond)) {                                                            \
            fprintf(stderr, "FAIL %s:%d: %s\n", __FILE__, __LINE__, #cond);       \
            return 1;                                                             \
        }                                                                         \
    } while (0)

using namespace kda;
using namespace kda::attn;

typedef std::vector<int> Ints;

// wave_prefix_sum's last lane: within rows of 16 by shifts of 1, 2, 4, 8, then row 0 into 1 and 2 into 3, then lane 31
// into rows 2 and 3.
static float wave_sum(const float* lanes) {
    float x[64], y[64];
    memcpy(x, lanes, sizeof(x));
    for (int d = 1; d < 16; d *= 2) {
        for (int i = 0; i < 64; ++i) y[i] = x[i] + (i % 16 >= d ? x[i - d] : 0.f);
        memcpy(x, y, sizeof(x));
    }
    for (int i = 0; i < 64; ++i) y[i] = x[i] + (i / 16 % 2 ? x[i / 16 * 16 - 1] : 0.f);
    memcpy(x, y, sizeof(x));
    return x[63] + x[31];
}

struct Totals {
    int64_t items, slots, cuts;
    int most;       // chunks of a sequence
};

static Totals totals(const AttnArgs& a, const Ints& n, const Ints& kv, bool narrow) {
    float tiles[64] = {}, units[64] = {};
    for (int lane = 0; lane < 64; ++lane)
        for (size_t s = lane; s < n.size(); s += 64) {
            if (n[s] <= 0) continue;
            const float t = (float)(tiles_of(a, n[s], narrow) * a.Hk);
            tiles[lane] += t;
            units[lane] = fmaf(t, (float)tile_units(a, kv[s], narrow), units[lane]);
        }
    const Cut cut = cut_of(wave_sum(tiles), wave_sum(units), narrow);
    Totals r = {0, 0, 0, 0};
    for (size_t s = 0; s < n.size(); ++s) {
        if (n[s] <= 0) continue;
        const int64_t own = (int64_t)tiles_of(a, n[s], narrow) * a.Hk;
        if (own == 0) continue;
        const int c = chunks_of(cut, tile_units(a, kv[s], narrow));
        r.items += own * c;
        if (c > 1) {
            r.slots += own * c;
            r.cuts += own;
            r.most = c > r.most ? c : r.most;
        }
    }
    return r;
}

// valid: within the rules, so that the host's counts of rows hold.
static int check(const AttnArgs& a, const Ints& n, const Ints& kv, bool valid) {
    for (int k = 0; k < 2; ++k) {
        const bool narrow = k == 0;
        if (!(narrow ? has_narrow(a) : has_wide(a))) continue;
        const Totals t = totals(a, n, kv, narrow);
        CHECK(t.slots <= slots_most(narrow));
        CHECK(t.cuts <= target(narrow) && (t.cuts == 0 || may_cut(a)));
        if (!valid || too_many(a)) continue;
        CHECK(t.items <= groups_most(a, narrow));
        CHECK(t.cuts <= join_groups(a, narrow));
    }
    return 0;
}

static AttnArgs args(int64_t N, int64_t T, int Hq, int Hk, int d, bool packed, int max_pages, int page, int64_t window) {
    AttnArgs a{};
    a.N = N; a.T = T; a.Hq = Hq; a.Hk = Hk; a.G = Hq / Hk; a.dk = a.dv = d;
    a.packed = packed; a.max_pages = max_pages; a.page_size = page; a.window = window;
    set_divisors(a);
    return a;
}

int main() {
    std::mt19937_64 rng(5);
    const auto upto = [&](double most) {        // 1 .. most, even over the logarithm
        const double u = std::uniform_real_distribution<double>(0, 1)(rng);
        const double x = pow(most, u);
        return (int64_t)(x < 1 ? 1 : x > most ? most : x);
    };
    int cut = 0, calls = 0;
    for (int round = 0; round < 40000; ++round) {
        const int64_t N = upto(round % 50 == 0 ? 65536 : 600);
        const int Hk = (int)upto(32), G = (int)upto(round % 3 == 0 ? 512 / Hk : 16 < 512 / Hk ? 16 : 512 / Hk);
        const int page = 16 * (int)upto(64);
        const int64_t keys = upto(round % 7 == 0 ? 1 << 30 : 1 << 17);
        const int64_t pages = (keys + page - 1) / page;
        const int max_pages = (int)(pages * page > ((int64_t)1 << 30) ? ((int64_t)1 << 30) / page : pages);
        const int64_t most_kv = (int64_t)max_pages * page;
        const bool packed = round & 1;
        const int kind = round % 11;
        Ints n(N), kv(N);
        int64_t sum = 0;
        const int64_t same_n = upto(kind < 4 ? 4 : 3000), same_kv = upto((double)most_kv);
        for (int64_t s = 0; s < N; ++s) {
            n[s] = (int)(!packed ? same_n : kind % 3 == 0 ? same_n : kind % 5 == 0 && upto(9) > 6 ? 0 : upto(kind < 6 ? 40 : 3000));
            // all alike, one long among short ones, at the borders of units, or spread
            kv[s] = (int)(kind % 4 == 0 ? same_kv : kind % 4 == 1 ? (s == N / 2 ? most_kv : upto(300)) :
                          kind % 4 == 2 ? (int64_t)kUnit * upto((double)(most_kv / kUnit + 1)) + (int64_t)(rng() % 3) - 1 : upto((double)most_kv));
            kv[s] = kv[s] < 0 ? 0 : kv[s] > most_kv ? (int)most_kv : kv[s];
            sum += n[s];
        }
        const int64_t T = packed ? sum : same_n;
        if (T < 1 || (packed ? T : N * T) * G >= ((int64_t)1 << 31)) continue;
        const int64_t window = kind % 5 == 4 ? upto(5000) : 0;
        const AttnArgs a = args(N, T, Hk * G, Hk, round & 4 ? 64 : 128, packed, max_pages, page, window);
        if (check(a, n, kv, true)) {
            fprintf(stderr, "round %d: N %lld T %lld heads %d x %d keys %lld kind %d\n", round, (long long)N, (long long)T, Hk, G,
                    (long long)most_kv, kind);
            return 1;
        }
        ++calls;
        if (has_narrow(a)) cut += totals(a, n, kv, true).cuts > 0;
        if (has_wide(a)) cut += totals(a, n, kv, false).cuts > 0;
        // cu_seqlens that go back and forth: any length up to T for every sequence
        if (packed) {
            for (int64_t s = 0; s < N; ++s) n[s] = (int)(s % 2 ? T : upto((double)T));
            if (check(a, n, kv, false)) return 1;
        }
    }
    CHECK(calls > 30000 && cut > 10000);
    // keys just past what makes one chunk more, for every number of tiles near the chunks aimed for
    for (int k = 0; k < 2; ++k)
        for (int64_t tiles = 1; tiles <= 600; tiles += tiles < 20 ? 1 : 29)
            for (int u = 1; u <= 4000; u += u < 64 ? 1 : 61) {
                const int64_t each = k ? 200 : 1;      // 200 tokens of 2 heads: two wide tiles
                const AttnArgs a = args(tiles, each, 2, 1, 128, false, 8 * u + 8, 16, 0);
                if (check(a, Ints(tiles, (int)each), Ints(tiles, u * kUnit), true)) return 1;
                if (check(a, Ints(tiles, (int)each), Ints(tiles, u * kUnit + 1), true)) return 1;
            }
    printf("attention plan check: ok\n");
    return 0;
}
