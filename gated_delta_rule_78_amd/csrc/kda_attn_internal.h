// Internal launcher interface of the attention over a paged cache (include/kda_attn.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda_attn.h"

namespace kda {

struct AttnArgs {
    int64_t N, T;
    int32_t Hq, Hk, G;          // query heads, key heads, query heads a key head
    int32_t dk, dv;
    int32_t pages, page_size, max_pages;
    int64_t table_stride, window;
    kda_row_strides sq, so;
    kda_page_strides skc, svc;
    bool packed;
    uint32_t mG, mHk;           // ceil(2^32 / G), ceil(2^32 / Hk); 0 for 1
    int32_t span[2];            // keys that a wide, a narrow tile reads at most (the window and its tokens)
    int32_t page_shift;         // log2(page_size), or -1
    float c;                    // |scale| * log2(e), at least the smallest normal number
    uint32_t flip;              // sign bits of two bf16 where scale < 0: q enters negated
    const void *q, *k_cache, *v_cache;
    const int32_t *cu, *kv_lens, *table;
    void* o;
    float* lse;
    void* ws;
};

size_t attn_ws_bytes(const AttnArgs& a);
hipError_t launch_paged_attn(const AttnArgs& a, hipStream_t st);

namespace attn {
// Instantiated per head sizes (kda_attn_d*.hip).
template <int DK, int DV>
hipError_t launch_main(const AttnArgs& a, bool narrow, int64_t groups, hipStream_t st);
}  // namespace attn

}  // namespace kda
