// Internal launcher interface of the head norms with rotation and of the cache append
// (include/kda_attn.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda_attn.h"

namespace kda {

struct RopeArgs {
    int64_t B, T;               // blocks of rows (append: sequences, or 1 packed) and tokens of each
    int32_t Hq, Hk;
    int32_t d, rot, dv;         // dv: append only
    bool in_bf16, interleaved, norm;
    float eps, scale;
    const void *q, *k, *v;
    const float *wq, *wk, *inv_freq;
    const int32_t* positions;
    void *q_out, *k_out;        // append: q_out; k_out is the key cache
    void* v_out;                // append: the value cache
    kda_row_strides sq, sk, sv, sqo, sko;
    // append
    int64_t N;
    bool packed;
    const int32_t *cu, *kv_lens, *table;
    int64_t table_stride;
    int32_t pages, page_size, max_pages;
    kda_page_strides skc, svc;
    // backward: sqo, sko are the strides of the output gradients
    const void *dqo, *dko;
    void *dq, *dk;
    kda_row_strides sdq, sdk;
    float *dwq, *dwk, *ws;
};

size_t rope_bwd_ws_bytes(int64_t tokens, int64_t d);
hipError_t launch_rope_fwd(const RopeArgs& a, hipStream_t st);
hipError_t launch_rope_append(const RopeArgs& a, hipStream_t st);
hipError_t launch_rope_bwd(const RopeArgs& a, hipStream_t st);

}  // namespace kda
