// C ABI of the head norms with rotation and of the cache append: argument validation and dispatch
// (include/kda_attn.h).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda_rope_internal.h"
#include "kda_rows.h"

namespace {

using kda::Range;
using kda::RopeArgs;
using kda::Rows;
using kda::aligned;
using kda::elem_bytes;
using kda::range_of;

constexpr int64_t kMaxHeads = 4096, kMaxRows = (int64_t)1 << 31;

bool finite(float v) { return v >= -3.4028234e38f && v <= 3.4028234e38f; }   // NaN fails
bool flag(int32_t v) { return v == 0 || v == 1; }

Rows rows(const void* p, int64_t B, int64_t H, int64_t T, int64_t d, const kda_row_strides& s, int64_t e) {
    return Rows{H > 0 ? p : nullptr, {B, H, T}, {s.b, s.h, s.t}, d, e};
}

// Kernels take strides of heads and tokens in 32 bits.
bool strides_fit(const Rows& r) {
    return r.empty() || ((r.n[1] <= 1 || r.s[1] < (int64_t)1 << 32) && (r.n[2] <= 1 || r.s[2] < (int64_t)1 << 32));
}

// What norm and rotation need, whoever applies them.
kda_status check_rotation(int64_t d, int64_t rot, int32_t interleaved, int32_t norm, float eps, float scale) {
    if (d < 2 || (d & 1) || rot < 0 || (rot & 1) || rot > d || !flag(interleaved) || !flag(norm)) return KDA_ERR_INVALID_ARG;
    if (norm && (!(eps > 0.f) || !finite(eps))) return KDA_ERR_INVALID_ARG;
    if (rot && !finite(scale)) return KDA_ERR_INVALID_ARG;
    return d > KDA_ROPE_MAX_D ? KDA_ERR_UNSUPPORTED : KDA_OK;
}

bool weights_ok(const float* wq, const float* wk, const float* inv_freq, int64_t rot, int32_t norm) {
    if (!norm && (wq || wk)) return false;
    if ((rot > 0) != (inv_freq != nullptr)) return false;
    return (!wq || aligned(wq, 4)) && (!wk || aligned(wk, 4)) && (!inv_freq || aligned(inv_freq, 4));
}

kda_status check_desc(const kda_head_rope_desc* d) {
    if (!d || d->B < 1 || d->Hq < 0 || d->Hk < 0 || d->Hq + d->Hk < 1 || d->T < 0 || !kda::valid_dtype(d->dtype))
        return KDA_ERR_INVALID_ARG;
    const kda_status s = check_rotation(d->d, d->rot, d->interleaved, d->norm, d->eps, d->rope_scale);
    if (s != KDA_OK) return s;
    if (d->Hq > kMaxHeads || d->Hk > kMaxHeads || d->B >= kMaxRows || d->T >= kMaxRows || d->B * d->T >= kMaxRows)
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

RopeArgs to_args(const kda_head_rope_desc* d, const void* q, const void* k, const float* wq, const float* wk,
                 const float* inv_freq, const int32_t* positions) {
    RopeArgs a{};
    a.B = d->B; a.T = d->T;
    a.Hq = (int32_t)d->Hq; a.Hk = (int32_t)d->Hk;
    a.d = (int32_t)d->d; a.rot = (int32_t)d->rot;
    a.in_bf16 = d->dtype == KDA_BF16;
    a.interleaved = d->interleaved != 0; a.norm = d->norm != 0;
    a.eps = d->eps; a.scale = d->rope_scale;
    a.q = q; a.k = k; a.wq = wq; a.wk = wk; a.inv_freq = inv_freq; a.positions = positions;
    a.sq = d->q; a.sk = d->k; a.sqo = d->q_out; a.sko = d->k_out; a.sdq = d->dq; a.sdk = d->dk;
    return a;
}

// hipErrorNotSupported: more workgroups than a launch can have.
kda_status status(hipError_t e) { return e == hipSuccess ? KDA_OK : e == hipErrorNotSupported ? KDA_ERR_UNSUPPORTED : KDA_ERR_HIP; }

}  // namespace

extern "C" {

kda_status kda_head_rope_fwd(const kda_head_rope_desc* d, const void* q, const void* k, const float* q_weight,
                             const float* k_weight, const float* inv_freq, const int32_t* positions, void* q_out,
                             void* k_out, void* stream) {
    const kda_status ds = check_desc(d);
    if (ds != KDA_OK) return ds;
    if (!weights_ok(q_weight, k_weight, inv_freq, d->rot, d->norm)) return KDA_ERR_INVALID_ARG;
    if (d->T == 0) return KDA_OK;
    if ((d->Hq && (!q || !q_out)) || (d->Hk && (!k || !k_out)) || (positions && !aligned(positions, 4)))
        return KDA_ERR_INVALID_ARG;
    const int64_t e = elem_bytes(d->dtype), w = d->d * 4;
    const Rows rq = rows(q, d->B, d->Hq, d->T, d->d, d->q, e), rk = rows(k, d->B, d->Hk, d->T, d->d, d->k, e);
    const Rows oq = rows(q_out, d->B, d->Hq, d->T, d->d, d->q_out, e), ok = rows(k_out, d->B, d->Hk, d->T, d->d, d->k_out, e);
    if (!rows_ok(rq) || !rows_ok(rk) || !rows_ok(oq) || !rows_ok(ok) || !oq.distinct() || !ok.distinct())
        return KDA_ERR_INVALID_ARG;
    for (const Rows* r : {&rq, &rk, &oq, &ok})
        if (!strides_fit(*r)) return KDA_ERR_UNSUPPORTED;
    const Range in[] = {rq.range(), rk.range(), range_of(q_weight, q_weight ? w : 0), range_of(k_weight, k_weight ? w : 0),
                        range_of(inv_freq, d->rot * 2), range_of(positions, positions ? d->B * d->T * 4 : 0)};
    const Range out[] = {oq.range(), ok.range()};
    if (!kda::rows_apart(in, out)) return KDA_ERR_INVALID_ARG;
    RopeArgs a = to_args(d, q, k, q_weight, k_weight, inv_freq, positions);
    a.q_out = q_out; a.k_out = k_out;
    return status(kda::launch_rope_fwd(a, reinterpret_cast<hipStream_t>(stream)));
}

size_t kda_head_rope_bwd_workspace_bytes(const kda_head_rope_desc* d) {
    if (check_desc(d) != KDA_OK || d->T == 0 || !d->norm) return 0;
    return kda::rope_bwd_ws_bytes(d->B * d->T, d->d);
}

kda_status kda_head_rope_bwd(const kda_head_rope_desc* d, const void* q, const void* k, const float* q_weight,
                             const float* k_weight, const float* inv_freq, const int32_t* positions, const void* dq_out,
                             const void* dk_out, void* dq, void* dk, float* dq_weight, float* dk_weight, void* workspace,
                             size_t workspace_bytes, void* stream) {
    const kda_status ds = check_desc(d);
    if (ds != KDA_OK) return ds;
    if (!weights_ok(q_weight, k_weight, inv_freq, d->rot, d->norm)) return KDA_ERR_INVALID_ARG;
    if (!d->norm && (dq_weight || dk_weight)) return KDA_ERR_INVALID_ARG;
    if ((dq_weight && (!d->Hq || !aligned(dq_weight, 4))) || (dk_weight && (!d->Hk || !aligned(dk_weight, 4))))
        return KDA_ERR_INVALID_ARG;
    const bool any = d->T > 0, sums = dq_weight || dk_weight;
    if (any) {
        if ((d->Hq && (!dq_out || !dq || (d->norm && !q))) || (d->Hk && (!dk_out || !dk || (d->norm && !k))))
            return KDA_ERR_INVALID_ARG;
        if (positions && !aligned(positions, 4)) return KDA_ERR_INVALID_ARG;
    }
    const size_t need = any && sums ? kda::rope_bwd_ws_bytes(d->B * d->T, d->d) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    if (need > 0 && !aligned(workspace, 16)) return KDA_ERR_INVALID_ARG;
    const int64_t e = elem_bytes(d->dtype), w = d->d * 4, B = d->B, T = d->T;
    const Rows rq = rows(d->norm ? q : nullptr, B, d->Hq, T, d->d, d->q, e), rk = rows(d->norm ? k : nullptr, B, d->Hk, T, d->d, d->k, e);
    const Rows zq = rows(dq_out, B, d->Hq, T, d->d, d->q_out, e), zk = rows(dk_out, B, d->Hk, T, d->d, d->k_out, e);
    const Rows oq = rows(dq, B, d->Hq, T, d->d, d->dq, e), ok = rows(dk, B, d->Hk, T, d->d, d->dk, e);
    if (!rows_ok(rq) || !rows_ok(rk) || !rows_ok(zq) || !rows_ok(zk) || !rows_ok(oq) || !rows_ok(ok) || (any && (!oq.distinct() || !ok.distinct())))
        return KDA_ERR_INVALID_ARG;
    for (const Rows* r : {&rq, &rk, &zq, &zk, &oq, &ok})
        if (!strides_fit(*r)) return KDA_ERR_UNSUPPORTED;
    const Range in[] = {rq.range(), rk.range(), zq.range(), zk.range(), range_of(q_weight, q_weight ? w : 0),
                        range_of(k_weight, k_weight ? w : 0), range_of(inv_freq, d->rot * 2),
                        range_of(positions, positions ? B * T * 4 : 0)};
    const Range out[] = {oq.range(), ok.range(), range_of(dq_weight, dq_weight ? w : 0),
                         range_of(dk_weight, dk_weight ? w : 0), range_of(workspace, (int64_t)need)};
    if (!kda::rows_apart(in, out)) return KDA_ERR_INVALID_ARG;
    if (!any && !sums) return KDA_OK;
    RopeArgs a = to_args(d, q, k, q_weight, k_weight, inv_freq, positions);
    a.dqo = dq_out; a.dko = dk_out; a.dq = dq; a.dk = dk;
    a.dwq = dq_weight; a.dwk = dk_weight; a.ws = static_cast<float*>(workspace);
    return status(kda::launch_rope_bwd(a, reinterpret_cast<hipStream_t>(stream)));
}

kda_status kda_kv_append(const kda_kv_append_desc* d, const void* q, const void* k, const void* v, const float* q_weight,
                         const float* k_weight, const float* inv_freq, const int32_t* cu_seqlens, const int32_t* kv_lens,
                         const int32_t* block_table, void* q_out, void* k_cache, void* v_cache, void* stream) {
    if (!d || d->N < 1 || d->Hq < 0 || d->Hk < 1 || d->T < 0 || d->dv < 1 || !kda::valid_dtype(d->in_dtype) || !flag(d->packed))
        return KDA_ERR_INVALID_ARG;
    if (d->pages < 1 || d->page_size < 1 || d->max_pages < 1 || !kda::table_ok(d->table_stride, d->max_pages)) return KDA_ERR_INVALID_ARG;
    const kda_status rs = check_rotation(d->dk, d->rot, d->interleaved, d->norm, d->eps, d->rope_scale);
    if (rs != KDA_OK) return rs;
    if (d->Hq > kMaxHeads || d->Hk > kMaxHeads || d->dv > KDA_ROPE_MAX_D || d->N >= kMaxRows || d->T >= kMaxRows ||
        (!d->packed && d->N * d->T >= kMaxRows))
        return KDA_ERR_UNSUPPORTED;
    if (d->pages >= kMaxRows || d->page_size > 1 << 20 || d->max_pages >= kMaxRows || d->max_pages * d->page_size >= kMaxRows ||
        d->table_stride >= (int64_t)1 << 40)
        return KDA_ERR_UNSUPPORTED;
    if (!weights_ok(q_weight, k_weight, inv_freq, d->rot, d->norm)) return KDA_ERR_INVALID_ARG;
    if ((cu_seqlens != nullptr) != (d->packed != 0)) return KDA_ERR_INVALID_ARG;
    if (d->T == 0) return KDA_OK;
    if (!k || !v || !kv_lens || !block_table || !k_cache || !v_cache || (d->Hq && (!q || !q_out))) return KDA_ERR_INVALID_ARG;
    if (!aligned(kv_lens, 4) || !aligned(block_table, 4) || (cu_seqlens && !aligned(cu_seqlens, 4))) return KDA_ERR_INVALID_ARG;
    const int64_t e = elem_bytes(d->in_dtype), B = d->packed ? 1 : d->N, w = d->dk * 4;
    const Rows rq = rows(q, B, d->Hq, d->T, d->dk, d->q, e), rk = rows(k, B, d->Hk, d->T, d->dk, d->k, e);
    const Rows rv = rows(v, B, d->Hk, d->T, d->dv, d->v, e), oq = rows(q_out, B, d->Hq, d->T, d->dk, d->q_out, 2);
    const Rows kc{k_cache, {d->pages, d->Hk, d->page_size}, {d->k_cache.p, d->k_cache.h, d->k_cache.t}, d->dk, 2};
    const Rows vc{v_cache, {d->pages, d->Hk, d->page_size}, {d->v_cache.p, d->v_cache.h, d->v_cache.t}, d->dv, 2};
    for (const Rows* r : {&rq, &rk, &rv, &oq, &kc, &vc})
        if (!rows_ok(*r)) return KDA_ERR_INVALID_ARG;
    if (!oq.distinct() || !kc.distinct() || !vc.distinct()) return KDA_ERR_INVALID_ARG;
    for (const Rows* r : {&rq, &rk, &rv, &oq})
        if (!strides_fit(*r)) return KDA_ERR_UNSUPPORTED;
    const Range in[] = {rq.range(), rk.range(), rv.range(), range_of(q_weight, q_weight ? w : 0),
                        range_of(k_weight, k_weight ? w : 0), range_of(inv_freq, d->rot * 2),
                        range_of(cu_seqlens, cu_seqlens ? (d->N + 1) * 4 : 0), range_of(kv_lens, d->N * 4),
                        range_of(block_table, ((d->N - 1) * d->table_stride + d->max_pages) * 4)};
    // the caches may interleave: each is checked against the rest, then they against each other
    const Range out_k[] = {oq.range(), kc.range()}, out_v[] = {oq.range(), vc.range()};
    if (!kda::rows_apart(in, out_k) || !kda::rows_apart(in, out_v)) return KDA_ERR_INVALID_ARG;
    if (kda::overlaps(kc.range(), vc.range()) && !kda::interleaved(kc, vc)) return KDA_ERR_INVALID_ARG;
    RopeArgs a{};
    a.B = B; a.T = d->T; a.N = d->N;
    a.Hq = (int32_t)d->Hq; a.Hk = (int32_t)d->Hk;
    a.d = (int32_t)d->dk; a.rot = (int32_t)d->rot; a.dv = (int32_t)d->dv;
    a.in_bf16 = d->in_dtype == KDA_BF16;
    a.interleaved = d->interleaved != 0; a.norm = d->norm != 0; a.packed = d->packed != 0;
    a.eps = d->eps; a.scale = d->rope_scale;
    a.q = q; a.k = k; a.v = v; a.wq = q_weight; a.wk = k_weight; a.inv_freq = inv_freq;
    a.q_out = q_out; a.k_out = k_cache; a.v_out = v_cache;
    a.sq = d->q; a.sk = d->k; a.sv = d->v; a.sqo = d->q_out; a.skc = d->k_cache; a.svc = d->v_cache;
    a.cu = cu_seqlens; a.kv_lens = kv_lens; a.table = block_table; a.table_stride = d->table_stride;
    a.pages = (int32_t)d->pages; a.page_size = (int32_t)d->page_size; a.max_pages = (int32_t)d->max_pages;
    return status(kda::launch_rope_append(a, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
