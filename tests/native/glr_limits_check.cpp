// Host-side check of the largest launches of the gated linear recurrence (kda_glr_abi.cpp over stub
// launchers): calls whose launches would number 2^32 threads or more are refused before any of them,
// the ones just below are not. Built and run by tests/test_glr_limits.py; every data pointer is a fake
// address that nothing dereferences.
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "kda_glr.h"
#include "kda_glr_internal.h"

namespace {
int g_launches;
}

namespace kda {
size_t glr_fwd_ws_bytes(const GlrArgs&) { return 256; }
size_t glr_bwd_ws_bytes(const GlrArgs&) { return 256; }
hipError_t launch_glr_fwd(const GlrArgs&, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_glr_bwd(const GlrArgs&, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_glr_step(const GlrArgs&, hipStream_t) { ++g_launches; return hipSuccess; }
}  // namespace kda

#define CHECK(cond)                                                               \
    do {                                                                          \
        if (!(cond)) {                                                            \
            fprintf(stderr, "FAIL %s:%d: %s\n", __FILE__, __LINE__, #cond);       \
            return 1;                                                             \
        }                                                                         \
    } while (0)

// 16 TiB apart
static void* P(uintptr_t i) { return reinterpret_cast<void*>((i + 1) << 44); }
static float* F(uintptr_t i) { return static_cast<float*>(P(i)); }

static kda_glr_desc desc(int64_t N, int64_t H, int64_t T, int64_t d, int32_t packed = 0) {
    kda_glr_desc x;
    memset(&x, 0, sizeof(x));
    x.N = N; x.H = H; x.T = T; x.d = d; x.in_dtype = KDA_BF16; x.out_dtype = KDA_BF16; x.packed = packed;
    x.g_min = -5.f;
    return x;
}

// The status of a call, which has to have launched something exactly if it was accepted, and whose
// workspace query has to agree.
enum { kStep, kFwd, kBwd, kBwdEntry, kBwdZ };
static int status(int op, kda_glr_desc d) {
    const kda_glr_gates la{P(1), nullptr, nullptr, nullptr}, z{nullptr, P(1), F(2), nullptr};
    const int32_t* cu = d.packed ? static_cast<const int32_t*>(P(3)) : nullptr;
    const int before = g_launches;
    const float* entry = op == kBwdEntry ? F(4) : nullptr;
    kda_status st;
    size_t need = 256;
    if (op == kStep) {
        st = kda_glr_step(&d, P(0), &la, F(5), P(6), nullptr);
    } else if (op == kFwd) {
        st = kda_glr_fwd(&d, P(0), &la, cu, nullptr, P(6), nullptr, nullptr, P(7), 256, nullptr);
        need = kda_glr_fwd_workspace_bytes(&d);
    } else {
        st = kda_glr_bwd(&d, P(0), op == kBwdZ ? &z : &la, cu, nullptr, entry, P(6), nullptr, P(8), P(9), nullptr,
                         op == kBwdZ ? F(10) : nullptr, nullptr, P(7), 256, nullptr);
        need = kda_glr_bwd_workspace_bytes(&d, entry != nullptr, op == kBwdZ);
    }
    if ((g_launches == before + 1) != (st == KDA_OK) || (op != kStep && (need == 256) != (st == KDA_OK))) return 1000;
    return st;
}

int main() {
    const int64_t M = (int64_t)1 << 20;
    const int OK = KDA_OK, NO = KDA_ERR_UNSUPPORTED;
    // tiles of 128 rows in the backward: 2^23 of 512 threads are 2^32
    CHECK(status(kBwdEntry, desc(8 * M, 1, 17, 1)) == NO && status(kBwdEntry, desc(8 * M - 1, 1, 17, 1)) == OK);
    CHECK(status(kBwdEntry, desc(4 * M, 1, 129, 3)) == NO && status(kBwdEntry, desc(4 * M - 1, 1, 129, 3)) == OK);
    CHECK(status(kBwdEntry, desc(4 * M, 2, 128, 64)) == NO && status(kBwdEntry, desc(2 * M, 3, 128, 64)) == OK);
    CHECK(status(kBwdEntry, desc(5, 8 * M, 40, 2, 1)) == NO && status(kBwdEntry, desc(5, 8 * M - 1, 40, 2, 1)) == OK);
    // in the forward 256 rows, 128 for fewer than 4 channels; 65 channels are two tiles
    CHECK(status(kFwd, desc(4 * M, 1, 129, 1)) == NO && status(kFwd, desc(4 * M - 1, 1, 129, 1)) == OK);
    CHECK(status(kFwd, desc(8 * M, 1, 129, 40)) == NO && status(kFwd, desc(8 * M - 1, 1, 129, 40)) == OK);
    CHECK(status(kFwd, desc(4 * M, 1, 256, 65)) == NO && status(kFwd, desc(4 * M - 1, 1, 256, 65)) == OK);
    CHECK(status(kFwd, desc(5, 8 * M, 40, 64, 1)) == NO && status(kFwd, desc(5, 8 * M - 1, 40, 64, 1)) == OK);
    // narrow heads share tiles: eight of 8 channels
    CHECK(status(kFwd, desc(16 * M, 1, 129, 8)) == OK && status(kFwd, desc(64 * M, 1, 129, 8)) == NO);
    // short sequences by rows: a thread per 4 channels, or per channel
    CHECK(status(kFwd, desc(1024 * M, 1, 16, 1)) == OK && status(kFwd, desc(1024 * M, 1, 16, 5)) == NO);
    CHECK(status(kFwd, desc(256 * M, 1, 16, 64)) == NO && status(kFwd, desc(256 * M - 16, 1, 16, 64)) == OK);
    CHECK(status(kStep, desc(256 * M, 1, 0, 64)) == NO && status(kStep, desc(256 * M - 16, 1, 0, 64)) == OK);
    CHECK(status(kBwd, desc(256 * M, 1, 16, 64)) == NO && status(kBwd, desc(256 * M - 16, 1, 16, 64)) == OK);
    // the backward runs the forward where it has no entry states
    CHECK(status(kBwd, desc(4 * M - 1, 1, 129, 1)) == OK && status(kBwd, desc(4 * M, 1, 129, 1)) == NO);
    // dA_log: 1024 threads for 64 channels of a head
    CHECK(status(kBwdZ, desc(1, 4 * M, 3, 1)) == NO && status(kBwdZ, desc(1, 4 * M - 1, 3, 1)) == OK);
    CHECK(status(kBwdZ, desc(2, 2 * M, 40, 65)) == NO && status(kBwd, desc(1, 4 * M - 1, 40, 65)) == OK);
    CHECK(status(kBwd, desc(1, 4 * M, 3, 1)) == OK);
    // without tokens there is no such launch
    CHECK(kda_glr_fwd_workspace_bytes(nullptr) == 0);
    kda_glr_desc none = desc(1024 * M, 1, 0, 1);
    CHECK(kda_glr_fwd(&none, nullptr, nullptr, nullptr, nullptr, nullptr, F(5), nullptr, nullptr, 0, nullptr) == KDA_OK);
    printf("glr limits check: ok\n");
    return 0;
}
