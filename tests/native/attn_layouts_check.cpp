// Host-side check of interleaved() (kda_rows.h) for two tensors of unequal widths and inner strides, as the keys and
// values of a cache in one buffer. Built and run by tests/test_attn_layouts.py.
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "kda_rows.h"

#define CHECK(cond)                                                               \
    do {                                                                          \
        if (!(cond)) {                                                            \
            fprintf(stderr, "FAIL %s:%d: %s\n", __FILE__, __LINE__, #cond);       \
            return 1;                                                             \
        }                                                                         \
    } while (0)

using kda::Rows;

static void* P(int64_t elements) { return reinterpret_cast<void*>((uintptr_t)0x7F0000000000ull + 2 * (uintptr_t)elements); }

// Whether a and b share an element, by counting.
static bool share(const Rows& a, const Rows& b, int64_t base) {
    static unsigned char seen[4096];
    memset(seen, 0, sizeof(seen));
    for (int pass = 0; pass < 2; ++pass) {
        const Rows& x = pass ? b : a;
        const int64_t at = (int64_t)((reinterpret_cast<uintptr_t>(x.p) - 0x7F0000000000ull) / 2) - base;
        for (int64_t i = 0; i < x.n[0]; ++i)
            for (int64_t j = 0; j < x.n[1]; ++j)
                for (int64_t k = 0; k < x.n[2]; ++k)
                    for (int64_t e = 0; e < x.d; ++e) {
                        unsigned char& c = seen[at + i * x.s[0] + j * x.s[1] + k * x.s[2] + e];
                        if (pass && c) return true;
                        if (!pass) c = 1;
                    }
    }
    return false;
}

static int check_small() {
    int apart = 0, unequal = 0;
    const int64_t inner[][3] = {{0, 2, 4}, {0, 4, 2}, {0, 6, 3}, {0, 3, 6}, {0, 1, 2}, {0, 2, 1}, {0, 8, 2}, {0, 2, 8}, {0, 5, 12}};
    for (int64_t pages = 1; pages <= 3; ++pages)
        for (int64_t s0 = 4; s0 <= 30; ++s0)
            for (const auto& x : inner)
                for (const auto& y : inner)
                    for (int64_t da = 1; da <= 3; ++da)
                        for (int64_t db = 1; db <= 3; ++db)
                            for (int64_t gap = -30; gap <= 30; ++gap) {
                                const Rows a{P(100), {pages, 2, 2}, {s0, x[1], x[2]}, da, 2};
                                const Rows b{P(100 + gap), {pages, 2, 2}, {s0, y[1], y[2]}, db, 2};
                                if (!a.distinct() || !b.distinct() || !kda::interleaved(a, b)) continue;
                                CHECK(kda::interleaved(b, a));
                                CHECK(!share(a, b, 0));
                                ++apart;
                                unequal += da != db;
                            }
    CHECK(apart > 1000 && unequal > 500);
    return 0;
}

// The buffers that a cache is made of.
static int check_caches() {
    const int64_t pages = 5, Hk = 2, page = 16, dk = 128, dv = 64, both = Hk * page * (dk + dv);
    const auto rows = [&](int64_t at, int64_t p, int64_t h, int64_t t, int64_t d) { return Rows{P(at), {pages, Hk, page}, {p, h, t}, d, 2}; };
    // [pages, (Hk, page, dk) then (Hk, page, dv)], either first
    CHECK(kda::interleaved(rows(0, both, page * dk, dk, dk), rows(Hk * page * dk, both, page * dv, dv, dv)));
    CHECK(kda::interleaved(rows(Hk * page * dv, both, page * dk, dk, dk), rows(0, both, page * dv, dv, dv)));
    // [pages, page, (Hk, dk) then (Hk, dv)]
    CHECK(kda::interleaved(rows(0, both, dk, Hk * (dk + dv), dk), rows(Hk * dk, both, dv, Hk * (dk + dv), dv)));
    // [pages, Hk, page, dk + dv]
    CHECK(kda::interleaved(rows(0, both, page * (dk + dv), dk + dv, dk), rows(dk, both, page * (dk + dv), dk + dv, dv)));
    // the values' last rows in the next page's keys; one row too far to the front
    CHECK(!kda::interleaved(rows(0, both, page * dk, dk, dk), rows(Hk * page * dk + 8, both, page * dv, dv, dv)));
    CHECK(!kda::interleaved(rows(0, both, page * dk, dk, dk), rows(Hk * page * dk - 8, both, page * dv, dv, dv)));
    // no common stride between pages
    CHECK(!kda::interleaved(rows(0, both, page * dk, dk, dk), rows(Hk * page * dk, both + 8, page * dv, dv, dv)));
    return 0;
}

int main() {
    if (check_small() || check_caches()) return 1;
    printf("attention layouts check: ok\n");
    return 0;
}
