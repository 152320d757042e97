// C ABI of the attention over a paged cache: argument validation and dispatch (include/kda_attn.h).
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kda_attn_internal.h"
#include "kda_attn_plan.h"
#include "kda_rows.h"

namespace {

using kda::AttnArgs;
using kda::Range;
using kda::Rows;
using kda::aligned;
using kda::range_of;

constexpr int64_t kMaxRows = (int64_t)1 << 31, kMaxKeys = (int64_t)1 << 30;
constexpr int64_t kMaxSequences = 1 << 16;     // every workgroup reads all their lengths

kda_status check_desc(const kda_paged_attn_desc* d) {
    if (!d || d->N < 1 || d->Hq < 1 || d->Hk < 1 || d->Hq % d->Hk || d->T < 0 || d->window < 0 ||
        (d->packed != 0 && d->packed != 1))
        return KDA_ERR_INVALID_ARG;
    if (d->pages < 1 || d->page_size < 1 || d->max_pages < 1 || !kda::table_ok(d->table_stride, d->max_pages)) return KDA_ERR_INVALID_ARG;
    if (!(d->scale >= -3.4028234e38f && d->scale <= 3.4028234e38f)) return KDA_ERR_INVALID_ARG;
    if ((d->dk != 64 && d->dk != 128) || (d->dv != 64 && d->dv != 128) || d->page_size % 16 || d->page_size > 1 << 20)
        return KDA_ERR_UNSUPPORTED;
    if (d->Hq > 512 || d->N > kMaxSequences || d->T >= kMaxRows || d->T * d->Hq >= kMaxRows * 64 || d->window >= kMaxRows)
        return KDA_ERR_UNSUPPORTED;
    if (d->T * (d->Hq / d->Hk) >= kMaxRows || (!d->packed && d->N * d->T * (d->Hq / d->Hk) >= kMaxRows)) return KDA_ERR_UNSUPPORTED;
    if (d->pages >= kMaxRows || d->max_pages >= kMaxRows || d->max_pages * d->page_size > kMaxKeys ||
        d->table_stride >= (int64_t)1 << 40)
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

AttnArgs to_args(const kda_paged_attn_desc* d) {
    AttnArgs a{};
    a.N = d->N; a.T = d->T;
    a.Hq = (int32_t)d->Hq; a.Hk = (int32_t)d->Hk; a.G = a.Hq / a.Hk;
    a.dk = (int32_t)d->dk; a.dv = (int32_t)d->dv;
    a.pages = (int32_t)d->pages; a.page_size = (int32_t)d->page_size; a.max_pages = (int32_t)d->max_pages;
    a.table_stride = d->table_stride; a.window = d->window;
    a.sq = d->q; a.so = d->o; a.skc = d->k_cache; a.svc = d->v_cache;
    a.packed = d->packed != 0;
    const float c = fabsf(d->scale) * 1.4426950408889634f;
    a.c = c < 1.17549435e-38f ? 1.17549435e-38f : c > 3.4028234e38f ? 3.4028234e38f : c;
    a.flip = d->scale < 0.f ? 0x80008000u : 0u;
    return a;
}

bool on8(int64_t n, int64_t s) { return n <= 1 || (s & 7) == 0; }

}  // namespace

extern "C" {

size_t kda_paged_attn_workspace_bytes(const kda_paged_attn_desc* d) {
    if (check_desc(d) != KDA_OK || d->T == 0) return 0;
    const AttnArgs a = to_args(d);
    return kda::attn::too_many(a) ? 0 : kda::attn_ws_bytes(a);
}

kda_status kda_paged_attn(const kda_paged_attn_desc* d, const void* q, const void* k_cache, const void* v_cache,
                          const int32_t* cu_seqlens, const int32_t* kv_lens, const int32_t* block_table, void* o, float* lse,
                          void* workspace, size_t workspace_bytes, void* stream) {
    const kda_status ds = check_desc(d);
    if (ds != KDA_OK) return ds;
    if ((cu_seqlens != nullptr) != (d->packed != 0)) return KDA_ERR_INVALID_ARG;
    if (d->T == 0) return KDA_OK;
    if (!q || !k_cache || !v_cache || !kv_lens || !block_table || !o) return KDA_ERR_INVALID_ARG;
    if (!aligned(kv_lens, 4) || !aligned(block_table, 4) || (cu_seqlens && !aligned(cu_seqlens, 4)) || (lse && !aligned(lse, 4)))
        return KDA_ERR_INVALID_ARG;
    for (const void* p : {q, k_cache, v_cache, (const void*)o})
        if (!aligned(p, 16)) return KDA_ERR_INVALID_ARG;
    const int64_t B = d->packed ? 1 : d->N;
    const Rows rq{q, {B, d->Hq, d->T}, {d->q.b, d->q.h, d->q.t}, d->dk, 2};
    const Rows ro{o, {B, d->Hq, d->T}, {d->o.b, d->o.h, d->o.t}, d->dv, 2};
    const Rows kc{k_cache, {d->pages, d->Hk, d->page_size}, {d->k_cache.p, d->k_cache.h, d->k_cache.t}, d->dk, 2};
    const Rows vc{v_cache, {d->pages, d->Hk, d->page_size}, {d->v_cache.p, d->v_cache.h, d->v_cache.t}, d->dv, 2};
    for (const Rows* r : {&rq, &ro, &kc, &vc}) {
        if (!rows_ok(*r)) return KDA_ERR_INVALID_ARG;
        for (int i = 0; i < 3; ++i)
            if (!on8(r->n[i], r->s[i])) return KDA_ERR_UNSUPPORTED;
    }
    if (!ro.distinct()) return KDA_ERR_INVALID_ARG;
    // a page's rows are reached by 32-bit offsets
    for (const Rows* r : {&kc, &vc})
        if ((r->n[0] > 1 && r->s[0] >= (int64_t)1 << 31) || r->s[2] >= (int64_t)1 << 30 || ((d->page_size - 1) * r->s[2] + r->d) * 2 >= (int64_t)1 << 31)
            return KDA_ERR_UNSUPPORTED;
    const AttnArgs plan = to_args(d);
    if (kda::attn::too_many(plan)) return KDA_ERR_UNSUPPORTED;
    const size_t need = kda::attn_ws_bytes(plan);
    if (!workspace || workspace_bytes < need) return KDA_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return KDA_ERR_INVALID_ARG;
    const Range in[] = {rq.range(), kc.range(), vc.range(), range_of(cu_seqlens, cu_seqlens ? (d->N + 1) * 4 : 0),
                        range_of(kv_lens, d->N * 4), range_of(block_table, ((d->N - 1) * d->table_stride + d->max_pages) * 4)};
    const Range out[] = {ro.range(), range_of(lse, lse ? B * d->Hq * d->T * 4 : 0), range_of(workspace, (int64_t)need)};
    if (!kda::rows_apart(in, out)) return KDA_ERR_INVALID_ARG;
    AttnArgs a = plan;
    a.q = q; a.k_cache = k_cache; a.v_cache = v_cache;
    a.cu = cu_seqlens; a.kv_lens = kv_lens; a.table = block_table;
    a.o = o; a.lse = lse; a.ws = workspace;
    return kda::launch_paged_attn(a, reinterpret_cast<hipStream_t>(stream)) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

}  // extern "C"
