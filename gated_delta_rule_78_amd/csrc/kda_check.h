// Argument checks shared by the C entry points: alignment, element types, overlapping ranges.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "kda.h"

namespace kda {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct Range {
    uintptr_t lo, hi;  // [lo, hi)
};
inline Range range_of(const void* p, int64_t bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Range{lo, lo + (uintptr_t)bytes};
}
inline bool overlaps(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.hi > a.lo && b.hi > b.lo; }

// One operand of a call: its pointer (NULL: not passed), its bytes, the alignment it must have.
struct Operand {
    const void* p;
    int64_t bytes;
    int64_t align;
    Range range() const { return range_of(p, p ? bytes : 0); }
};

// Every operand on its alignment, and no output overlapping an input or another output.
// Output place_out may be the very pointer of input place_in (an in-place call).
template <int NI, int NO>
bool operands_ok(const Operand (&in)[NI], const Operand (&out)[NO], int place_out = -1, int place_in = -1) {
    for (const Operand& a : in)
        if (a.p && !aligned(a.p, (uintptr_t)a.align)) return false;
    for (int i = 0; i < NO; ++i) {
        if (out[i].p && !aligned(out[i].p, (uintptr_t)out[i].align)) return false;
        for (int j = 0; j < NI; ++j) {
            if (i == place_out && j == place_in && out[i].p == in[j].p) continue;
            if (overlaps(out[i].range(), in[j].range())) return false;
        }
        for (int j = i + 1; j < NO; ++j)
            if (overlaps(out[i].range(), out[j].range())) return false;
    }
    return true;
}

inline bool valid_dtype(int32_t d) { return d == KDA_F32 || d == KDA_BF16; }
inline int64_t elem_bytes(int32_t d) { return d == KDA_BF16 ? 2 : 4; }
inline int64_t ceil_to(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace kda
