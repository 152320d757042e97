// Host-side check of the validation layers of the attention layers' operators (kda_rope_abi.cpp,
// kda_attn_abi.cpp) under AddressSanitizer and UndefinedBehaviorSanitizer. Both are built for the host
// only, over stub launchers that record what would have been enqueued. Built and run by
// tests/test_attn_sanitizers.py; every data pointer is a fake address that nothing dereferences.
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "kda_attn.h"
#include "kda_attn_internal.h"
#include "kda_rope_internal.h"
#include "kda_rows.h"

namespace {
int g_rfwd, g_rbwd, g_app, g_attn;
kda::RopeArgs g_rope;
kda::AttnArgs g_a;
}  // namespace

namespace kda {
size_t rope_bwd_ws_bytes(int64_t tokens, int64_t d) { return (size_t)(tokens * d) * 8; }
hipError_t launch_rope_fwd(const RopeArgs& a, hipStream_t) { ++g_rfwd; g_rope = a; return hipSuccess; }
hipError_t launch_rope_bwd(const RopeArgs& a, hipStream_t) { ++g_rbwd; g_rope = a; return hipSuccess; }
hipError_t launch_rope_append(const RopeArgs& a, hipStream_t) { ++g_app; g_rope = a; return hipErrorInvalidValue; }
size_t attn_ws_bytes(const AttnArgs& a) { return (size_t)(a.N * 64); }
hipError_t launch_paged_attn(const AttnArgs& a, hipStream_t) { ++g_attn; g_a = a; return hipSuccess; }
}  // namespace kda

#define CHECK(cond)                                                               \
    do {                                                                          \
        if (!(cond)) {                                                            \
            fprintf(stderr, "FAIL %s:%d: %s\n", __FILE__, __LINE__, #cond);       \
            return 1;                                                             \
        }                                                                         \
    } while (0)

static void* P(uintptr_t i, uintptr_t off = 0) { return reinterpret_cast<void*>(0x7F0000000000ull + (i << 36) + off); }
static float* F(uintptr_t i) { return static_cast<float*>(P(i)); }
static const int32_t* I(uintptr_t i) { return static_cast<const int32_t*>(P(i)); }

static kda_head_rope_desc rdesc() {
    kda_head_rope_desc d;
    memset(&d, 0, sizeof(d));
    d.B = 2; d.Hq = 4; d.Hk = 1; d.T = 7; d.d = 64; d.rot = 32;
    d.q = d.q_out = d.dq = kda_row_strides{4 * 7 * 64, 64, 256};
    d.k = d.k_out = d.dk = kda_row_strides{7 * 64, 64, 64};
    d.dtype = KDA_BF16; d.norm = 1; d.eps = 1e-6f; d.rope_scale = 1.f;
    return d;
}

static int check_rope() {
    kda_head_rope_desc d = rdesc();
    CHECK(kda_head_rope_fwd(nullptr, P(0), P(1), nullptr, nullptr, F(2), nullptr, P(3), P(4), nullptr) == KDA_ERR_INVALID_ARG);
    CHECK(kda_head_rope_fwd(&d, P(0), P(1), nullptr, nullptr, F(2), nullptr, P(3), P(3), nullptr) == KDA_ERR_INVALID_ARG);
    CHECK(g_rfwd == 0);
    CHECK(kda_head_rope_fwd(&d, P(0), P(1), F(5), F(6), F(2), I(7), P(3), P(4), nullptr) == KDA_OK && g_rfwd == 1);
    CHECK(g_rope.Hq == 4 && g_rope.rot == 32 && g_rope.in_bf16 && g_rope.norm && !g_rope.interleaved && g_rope.positions == I(7));
    d.Hq = 0;       // one tensor alone
    CHECK(kda_head_rope_fwd(&d, nullptr, P(1), nullptr, F(6), F(2), nullptr, nullptr, P(4), nullptr) == KDA_OK && g_rfwd == 2);
    d = rdesc();
    d.q.b = INT64_MAX; d.B = 3;
    CHECK(kda_head_rope_fwd(&d, P(0), P(1), nullptr, nullptr, F(2), nullptr, P(3), P(4), nullptr) == KDA_ERR_INVALID_ARG);
    d = rdesc();
    d.B = INT64_MAX; d.T = INT64_MAX;
    CHECK(kda_head_rope_fwd(&d, P(0), P(1), nullptr, nullptr, F(2), nullptr, P(3), P(4), nullptr) == KDA_ERR_UNSUPPORTED);
    d = rdesc();
    const size_t need = kda_head_rope_bwd_workspace_bytes(&d);
    CHECK(need == 14 * 64 * 8);
    CHECK(kda_head_rope_bwd(&d, P(0), P(1), F(5), F(6), F(2), nullptr, P(3), P(4), P(8), P(9), F(10), F(11), P(12), need - 1,
                            nullptr) == KDA_ERR_WORKSPACE);
    CHECK(kda_head_rope_bwd(&d, P(0), P(1), F(5), F(6), F(2), nullptr, P(3), P(4), P(8), P(9), F(10), F(11), P(12), need,
                            nullptr) == KDA_OK && g_rbwd == 1 && g_rope.ws == P(12));
    CHECK(kda_head_rope_bwd(&d, P(0), P(1), F(5), F(6), F(2), nullptr, P(3), P(4), P(8), P(9), nullptr, nullptr, nullptr, 0,
                            nullptr) == KDA_OK && g_rbwd == 2);          // no sums: no workspace
    d.T = 0;
    CHECK(kda_head_rope_bwd(&d, nullptr, nullptr, nullptr, nullptr, F(2), nullptr, nullptr, nullptr, nullptr, nullptr, F(10),
                            nullptr, nullptr, 0, nullptr) == KDA_OK && g_rbwd == 3);   // zeros for the weight
    return 0;
}

static int check_append() {
    kda_kv_append_desc d;
    memset(&d, 0, sizeof(d));
    d.N = 3; d.Hq = 4; d.Hk = 2; d.T = 11; d.dk = 64; d.dv = 48; d.rot = 64; d.pages = 9; d.page_size = 16; d.max_pages = 5;
    d.table_stride = 8;
    d.q = d.q_out = kda_row_strides{0, 64, 256};
    d.k = kda_row_strides{0, 64, 128};
    d.v = kda_row_strides{0, 48, 96};
    d.k_cache = kda_page_strides{2 * 16 * 64, 16 * 64, 64};
    d.v_cache = kda_page_strides{2 * 16 * 48, 16 * 48, 48};
    d.in_dtype = KDA_F32; d.packed = 1; d.norm = 0; d.rope_scale = 1.f;
    CHECK(kda_kv_append(&d, P(0), P(1), P(2), nullptr, nullptr, F(3), nullptr, I(4), I(5), P(6), P(7), P(8), nullptr) == KDA_ERR_INVALID_ARG);
    CHECK(g_app == 0);
    CHECK(kda_kv_append(&d, P(0), P(1), P(2), nullptr, nullptr, F(3), I(9), I(4), I(5), P(6), P(7), P(8), nullptr) == KDA_ERR_HIP && g_app == 1);
    CHECK(g_rope.B == 1 && g_rope.T == 11 && g_rope.N == 3 && g_rope.packed && !g_rope.in_bf16 && g_rope.k_out == P(7) && g_rope.v_out == P(8));
    d.pages = INT64_MAX;
    CHECK(kda_kv_append(&d, P(0), P(1), P(2), nullptr, nullptr, F(3), I(9), I(4), I(5), P(6), P(7), P(8), nullptr) == KDA_ERR_UNSUPPORTED);
    return 0;
}

static int check_attn() {
    kda_paged_attn_desc d;
    memset(&d, 0, sizeof(d));
    d.N = 2; d.Hq = 8; d.Hk = 2; d.T = 3; d.dk = 128; d.dv = 64; d.pages = 9; d.page_size = 32; d.max_pages = 5; d.table_stride = 5;
    d.q = kda_row_strides{8 * 3 * 128, 3 * 128, 128};
    d.o = kda_row_strides{8 * 3 * 64, 64, 8 * 64};
    d.k_cache = kda_page_strides{2 * 32 * 128, 32 * 128, 128};
    d.v_cache = kda_page_strides{2 * 32 * 64, 32 * 64, 64};
    d.scale = -0.5f;
    CHECK(kda_paged_attn_workspace_bytes(&d) == 128);
    CHECK(kda_paged_attn(&d, P(0), P(1), P(2), nullptr, I(3), I(4), P(5), nullptr, P(6), 127, nullptr) == KDA_ERR_WORKSPACE && g_attn == 0);
    CHECK(kda_paged_attn(&d, P(0), P(1), P(2), nullptr, I(3), I(4), P(5), F(7), P(6), 128, nullptr) == KDA_OK && g_attn == 1);
    CHECK(g_a.G == 4 && g_a.flip == 0x80008000u && fabsf(g_a.c - 0.5f * 1.442695f) < 1e-6f && g_a.lse == F(7) && !g_a.packed);
    d.scale = 0.f;
    CHECK(kda_paged_attn(&d, P(0), P(1), P(2), nullptr, I(3), I(4), P(5), nullptr, P(6), 128, nullptr) == KDA_OK && g_a.c > 0.f && g_a.flip == 0);
    d.max_pages = INT64_MAX; d.table_stride = INT64_MAX;
    CHECK(kda_paged_attn(&d, P(0), P(1), P(2), nullptr, I(3), I(4), P(5), nullptr, P(6), 128, nullptr) == KDA_ERR_UNSUPPORTED);
    d.max_pages = 5; d.table_stride = 5; d.T = INT64_MAX;
    CHECK(kda_paged_attn(&d, P(0), P(1), P(2), nullptr, I(3), I(4), P(5), nullptr, P(6), 128, nullptr) == KDA_ERR_UNSUPPORTED);
    return 0;
}

// distinct() and interleaved() against counting every element of small layouts.
static int check_layouts() {
    static unsigned char seen[4096];
    int n = 0;
    for (int64_t s0 = 0; s0 <= 24; s0 += 4)
        for (int64_t s1 = 0; s1 <= 24; s1 += 2)
            for (int64_t s2 = 0; s2 <= 6; ++s2)
                for (int64_t gap = 0; gap <= 30; ++gap) {
                    const kda::Rows a{P(0), {2, 3, 2}, {s0, s1, s2}, 2, 2}, b{P(0, (uintptr_t)(2 * gap)), {2, 3, 2}, {s0, s1, s2}, 2, 2};
                    memset(seen, 0, sizeof(seen));
                    bool self = false, cross = false;
                    for (int pass = 0; pass < 2; ++pass)
                        for (int64_t i = 0; i < 2; ++i)
                            for (int64_t j = 0; j < 3; ++j)
                                for (int64_t k = 0; k < 2; ++k)
                                    for (int64_t e = 0; e < 2; ++e) {
                                        unsigned char& c = seen[i * s0 + j * s1 + k * s2 + e + (pass ? gap : 0)];
                                        if (pass == 0 && c) self = true;
                                        if (pass == 1 && c == 1) cross = true;
                                        c = pass == 0 ? 1 : (unsigned char)(c | 2);
                                    }
                    CHECK(!(a.distinct() && self));                          // never called distinct where rows share
                    if (a.distinct() && kda::interleaved(a, b)) {
                        CHECK(!cross);                                       // nor apart where two tensors share
                        ++n;
                    }
                }
    CHECK(n > 100);
    return 0;
}

int main() {
    if (check_rope() || check_append() || check_attn() || check_layouts()) return 1;
    printf("attention host check: ok\n");
    return 0;
}
