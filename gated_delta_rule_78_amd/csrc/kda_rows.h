// Argument checks of strided rows [n0, n1, n2, d] (last dimension contiguous): their extent, whether
// rows share elements, and whether two of them interleave without sharing any.
#pragma once

#include "kda_check.h"

namespace kda {

struct Rows {
    const void* p;          // NULL: absent
    int64_t n[3], s[3];     // sizes and strides (elements) of the three outer dimensions
    int64_t d;              // contiguous elements
    int64_t e;              // bytes of an element

    bool empty() const { return !p || n[0] == 0 || n[1] == 0 || n[2] == 0; }

    // Elements from the first to behind the last; false where that passes 2^61 or a stride is negative.
    bool extent(int64_t* out) const {
        int64_t m = d;
        for (int i = 0; i < 3; ++i) {
            if (n[i] <= 1) continue;
            int64_t t;
            if (s[i] < 0 || __builtin_mul_overflow(n[i] - 1, s[i], &t) || __builtin_add_overflow(m, t, &m)) return false;
        }
        *out = m;
        return m <= (int64_t)1 << 61;
    }
    Range range() const {
        int64_t m = 0;
        if (empty() || !extent(&m)) return Range{0, 0};
        return range_of(p, m * e);
    }
    // Dimensions of more than one row, by falling stride.
    int order(int* o) const {
        int k = 0;
        for (int i = 0; i < 3; ++i)
            if (n[i] > 1) o[k++] = i;
        for (int i = 0; i < k; ++i)
            for (int j = i + 1; j < k; ++j)
                if (s[o[j]] > s[o[i]]) {
                    const int t = o[i];
                    o[i] = o[j];
                    o[j] = t;
                }
        return k;
    }
    // No two rows share elements: every stride steps over all that the smaller ones reach.
    bool distinct() const {
        if (empty()) return true;
        int o[3];
        int64_t reach = d;
        for (int i = order(o) - 1; i >= 0; --i) {
            if (s[o[i]] < reach) return false;
            int64_t t;
            if (__builtin_mul_overflow(n[o[i]] - 1, s[o[i]], &t) || __builtin_add_overflow(reach, t, &reach)) return false;
        }
        return true;
    }
};

inline bool rows_ok(const Rows& r) {
    int64_t m;
    return r.empty() || (aligned(r.p, (uintptr_t)r.e) && r.extent(&m));
}

// a and b, both distinct, of one element type and the same sizes, share no element though their ranges may
// overlap: some outer stride that both have sets b's rows into the gaps that a's leave (or the other way round),
// as the two halves of one buffer. The strides below it may differ, as those of unequal widths do.
inline bool interleaved(const Rows& a, const Rows& b) {
    for (int i = 0; i < 3; ++i)
        if (a.n[i] != b.n[i]) return false;
    int oa[3], ob[3];
    const int k = a.order(oa);
    b.order(ob);
    const intptr_t pa = reinterpret_cast<intptr_t>(a.p), pb = reinterpret_cast<intptr_t>(b.p);
    const bool a_first = pa <= pb;
    const int64_t bytes = a_first ? pb - pa : pa - pb;
    if (bytes % a.e) return false;
    int64_t gap = bytes / a.e;
    for (int i = 0; i < k; ++i) {
        const int64_t step = a.s[oa[i]];
        if (ob[i] != oa[i] || b.s[ob[i]] != step || step < 1) return false;
        if (i > 0 && a.s[oa[i - 1]] % step) return false;    // rows of different outer indices at different places
        // what the dimensions of smaller strides reach
        int64_t ra = a.d, rb = b.d;
        for (int j = i + 1; j < k; ++j) {
            ra += (a.n[oa[j]] - 1) * a.s[oa[j]];
            rb += (b.n[ob[j]] - 1) * b.s[ob[j]];
        }
        gap %= step;
        if (gap >= (a_first ? ra : rb) && gap + (a_first ? rb : ra) <= step) return true;
    }
    return false;
}

// A block table's rows: apart, or one row for every sequence.
inline bool table_ok(int64_t stride, int64_t max_pages) { return stride == 0 || stride >= max_pages; }

template <int NI, int NO>
bool rows_apart(const Range (&in)[NI], const Range (&out)[NO]) {
    for (int i = 0; i < NO; ++i) {
        for (int j = 0; j < NI; ++j)
            if (overlaps(out[i], in[j])) return false;
        for (int j = i + 1; j < NO; ++j)
            if (overlaps(out[i], out[j])) return false;
    }
    return true;
}

}  // namespace kda
