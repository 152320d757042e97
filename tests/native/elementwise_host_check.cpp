// Host-side check of the validation layers of the gated linear recurrence and of the block norms
// (kda_glr_abi.cpp, kda_norm_abi.cpp) under AddressSanitizer and UndefinedBehaviorSanitizer. Both
// are built for the host only, over stub launchers that record what would have been enqueued. Built
// and run by tests/test_elementwise_sanitizers.py; every data pointer is a fake address that nothing
// dereferences.
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "kda_glr.h"
#include "kda_glr_internal.h"
#include "kda_norm.h"
#include "kda_norm_internal.h"

namespace {
int g_fwd, g_bwd, g_step, g_nfwd, g_nbwd;
kda::GlrArgs g_glr;
kda::NormArgs g_norm;
}  // namespace

namespace kda {
size_t glr_fwd_ws_bytes(const GlrArgs& a) { return a.T > 128 ? (size_t)(a.blocks * a.nch * a.d) * 16 : 0; }
size_t glr_bwd_ws_bytes(const GlrArgs& a) { return 256 + (a.entry ? 0 : 64) + (a.z ? 32 : 0); }
hipError_t launch_glr_fwd(const GlrArgs& a, hipStream_t) { ++g_fwd; g_glr = a; return hipSuccess; }
hipError_t launch_glr_bwd(const GlrArgs& a, hipStream_t) { ++g_bwd; g_glr = a; return hipSuccess; }
hipError_t launch_glr_step(const GlrArgs& a, hipStream_t) { ++g_step; g_glr = a; return hipErrorInvalidValue; }
size_t norm_bwd_ws_bytes(int64_t rows, int64_t D) { return (size_t)(rows * D) * 8; }
hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t) { ++g_nfwd; g_norm = a; return hipSuccess; }
hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t) { ++g_nbwd; g_norm = a; return hipSuccess; }
}  // namespace kda

#define CHECK(cond)                                                               \
    do {                                                                          \
        if (!(cond)) {                                                            \
            fprintf(stderr, "FAIL %s:%d: %s\n", __FILE__, __LINE__, #cond);       \
            return 1;                                                             \
        }                                                                         \
    } while (0)

static void* P(uintptr_t gb, uintptr_t off = 0) { return reinterpret_cast<void*>(0x7F0000000000ull + (gb << 30) + off); }
static float* F(uintptr_t gb, uintptr_t off = 0) { return static_cast<float*>(P(gb, off)); }

static kda_glr_desc gdesc(int64_t N, int64_t H, int64_t T, int64_t d, int32_t packed = 0) {
    kda_glr_desc x;
    memset(&x, 0, sizeof(x));
    x.N = N; x.H = H; x.T = T; x.d = d; x.in_dtype = KDA_BF16; x.out_dtype = KDA_F32; x.packed = packed;
    x.scale = KDA_GLR_NORM; x.g_min = -5.f;
    return x;
}

static int check_glr() {
    kda_glr_desc d = gdesc(2, 3, 500, 40);
    kda_glr_gates la{P(1), nullptr, nullptr, nullptr}, z{nullptr, P(1), F(2), P(3)}, none{nullptr, nullptr, nullptr, nullptr};
    const size_t need = kda_glr_fwd_workspace_bytes(&d);
    CHECK(need == 2 * 3 * 4 * 40 * 16 && kda_glr_fwd_workspace_bytes(nullptr) == 0);
    CHECK(kda_glr_fwd(nullptr, P(0), &la, nullptr, nullptr, P(4), nullptr, nullptr, P(5), need, nullptr) == KDA_ERR_INVALID_ARG);
    CHECK(kda_glr_fwd(&d, P(0), nullptr, nullptr, nullptr, P(4), nullptr, nullptr, P(5), need, nullptr) == KDA_ERR_INVALID_ARG);
    CHECK(kda_glr_fwd(&d, P(0), &none, nullptr, nullptr, P(4), nullptr, nullptr, P(5), need, nullptr) == KDA_ERR_INVALID_ARG);
    CHECK(kda_glr_fwd(&d, P(0), &la, nullptr, nullptr, P(4), nullptr, nullptr, P(5), need - 1, nullptr) == KDA_ERR_WORKSPACE);
    CHECK(kda_glr_fwd(&d, P(0), &la, nullptr, nullptr, P(0, 64), nullptr, nullptr, P(5), need, nullptr) == KDA_ERR_INVALID_ARG);
    CHECK(g_fwd == 0);   // nothing enqueued on an error
    CHECK(kda_glr_fwd(&d, P(0), &z, nullptr, F(6), P(4), F(6), F(7), P(5), need, nullptr) == KDA_OK && g_fwd == 1);
    CHECK(g_glr.blocks == 6 && g_glr.nch == 4 && g_glr.z && g_glr.u && !g_glr.la && g_glr.S0 == g_glr.S_T);
    kda_glr_desc huge = gdesc((int64_t)1 << 40, (int64_t)1 << 40, (int64_t)1 << 30, 1 << 19);
    CHECK(kda_glr_fwd(&huge, P(0), &la, nullptr, nullptr, P(4), nullptr, nullptr, P(5), need, nullptr) == KDA_ERR_INVALID_ARG);
    kda_glr_desc pk = gdesc(5, 3, 500, 40, 1);
    CHECK(kda_glr_fwd(&pk, P(0), &la, nullptr, nullptr, P(4), nullptr, nullptr, P(5), need, nullptr) == KDA_ERR_INVALID_ARG);
    CHECK(kda_glr_fwd(&pk, P(0), &la, (const int32_t*)P(8), nullptr, P(4), nullptr, nullptr, P(5), need, nullptr) == KDA_OK);
    CHECK(g_glr.blocks == 3 && g_glr.packed);
    kda_glr_desc empty = gdesc(2, 3, 0, 40);   // no rows: gates and rows are not looked at
    CHECK(kda_glr_fwd(&empty, nullptr, nullptr, nullptr, F(6), nullptr, F(7), nullptr, nullptr, 0, nullptr) == KDA_OK);
    CHECK(g_glr.T == 0 && !g_glr.la && g_glr.S_T == F(7));

    CHECK(kda_glr_bwd(&d, P(0), &z, nullptr, nullptr, nullptr, P(4), nullptr, P(9), P(10), P(11), nullptr, nullptr, P(5),
                      4096, nullptr) == KDA_ERR_INVALID_ARG);   // z without dA_log
    CHECK(kda_glr_bwd(&d, P(0), &z, nullptr, nullptr, nullptr, P(4), nullptr, P(9), P(10), P(11), F(12), nullptr, P(5), 351,
                      nullptr) == KDA_ERR_WORKSPACE);
    CHECK(g_bwd == 0);
    CHECK(kda_glr_bwd(&d, P(0), &z, nullptr, nullptr, nullptr, P(4), nullptr, P(9), P(10), P(11), F(12), nullptr, P(5), 352,
                      nullptr) == KDA_OK && g_bwd == 1);
    CHECK(kda_glr_bwd_workspace_bytes(&d, 0, 1) == 352 && kda_glr_bwd_workspace_bytes(&d, 1, 0) == 256);
    CHECK(kda_glr_bwd(&d, P(0), &la, nullptr, nullptr, F(13), P(4), F(14), P(9), P(10), nullptr, nullptr, F(14), P(5), 256,
                      nullptr) == KDA_ERR_INVALID_ARG);          // dS0 in place of dS_T
    CHECK(kda_glr_step(&d, P(0), &la, F(6), P(4), nullptr) == KDA_ERR_HIP && g_step == 1 && g_glr.T == 1);
    CHECK(kda_glr_step(&d, P(0), &la, F(6), P(6, 32), nullptr) == KDA_ERR_INVALID_ARG && g_step == 1);
    return 0;
}

static int check_norm() {
    kda_norm_desc d;
    memset(&d, 0, sizeof(d));
    d.rows = 10; d.D = 100; d.in_dtype = KDA_BF16; d.res_dtype = KDA_F32; d.out_dtype = KDA_BF16;
    d.post_norm = 1; d.pre_norm = 1; d.scale = 0.5f; d.eps = 1e-6f; d.pre_eps = 1e-6f;
    CHECK(kda_block_norm_fwd(nullptr, P(0), nullptr, nullptr, nullptr, nullptr, nullptr, P(1), P(2), nullptr) == KDA_ERR_INVALID_ARG);
    CHECK(kda_block_norm_fwd(&d, P(0), nullptr, P(3), nullptr, nullptr, nullptr, P(3, 4), P(2), nullptr) == KDA_ERR_INVALID_ARG);
    CHECK(g_nfwd == 0);
    CHECK(kda_block_norm_fwd(&d, P(0), P(4), P(3), F(5), F(6), F(7), P(3), P(2), nullptr) == KDA_OK && g_nfwd == 1);
    CHECK(g_norm.x == g_norm.x_out && g_norm.post && g_norm.pre);
    const size_t need = kda_block_norm_bwd_workspace_bytes(&d);
    CHECK(need == 8000);
    CHECK(kda_block_norm_bwd(&d, P(0), nullptr, P(3), nullptr, nullptr, nullptr, P(8), P(9), P(10), nullptr, P(8), F(11),
                             nullptr, nullptr, P(12), need - 1, nullptr) == KDA_ERR_WORKSPACE);
    CHECK(kda_block_norm_bwd(&d, P(0), nullptr, P(3), nullptr, nullptr, nullptr, P(8), P(9), P(10), nullptr, P(8), F(11),
                             nullptr, nullptr, P(12), need, nullptr) == KDA_OK && g_nbwd == 1 && g_norm.ws);
    CHECK(kda_block_norm_bwd(&d, P(0), nullptr, P(3), nullptr, nullptr, nullptr, P(8), P(9), P(10), nullptr, P(8), nullptr,
                             nullptr, nullptr, nullptr, 0, nullptr) == KDA_OK && !g_norm.ws);   // no sums: no workspace
    d.rows = 0;
    CHECK(kda_block_norm_bwd(&d, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                             nullptr, F(11), nullptr, nullptr, nullptr, 0, nullptr) == KDA_OK && g_nbwd == 3);
    CHECK(kda_block_norm_bwd(&d, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                             nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr) == KDA_OK && g_nbwd == 3);
    return 0;
}

int main() {
    if (check_glr() || check_norm()) return 1;
    printf("elementwise host check: ok\n");
    return 0;
}
