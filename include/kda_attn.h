/*
 * kda_attn.h -- C ABI of the softmax-attention layers that stand between KDA layers in a hybrid
 * stack, for AMD Instinct MI355X (gfx950): the per-head norm of queries and keys with the position
 * rotation, the append of new tokens to a paged cache, and the attention of new tokens over that
 * cache. Same library, same conventions as kda.h (device pointers owned by the caller, asynchronous
 * on `stream`, arguments validated before any device work, kda_status, no allocation, no
 * synchronisation, no state kept between calls).
 *
 *  - Heads' rows have the core's shapes, [B,H,T,d] or packed [H,T,d], with the strides the caller
 *    gives: slices of one projection's output [T, (Hq + 2 Hk) d] are read where they are. The last
 *    dimension is contiguous. Strides are in elements and not negative, those of heads and tokens
 *    below 2^32; an input's may be 0 (a tensor expanded along that dimension), an output's rows
 *    must not share elements.
 *  - Bases are aligned to their element unless a call says more; rows on 16 bytes take wide accesses.
 *  - No output may overlap an input or another output, taken as the ranges from a tensor's first
 *    element to its last (k_cache and v_cache may interleave in one buffer: a page's keys and values, or a
 *    row's, side by side, of whatever widths).
 *  - Everything between inputs and outputs is fp32 or wider; every output is rounded once.
 *  - A launch has fewer than 2^32 threads. A call that would need more is refused with
 *    KDA_ERR_UNSUPPORTED, and its workspace query answers 0 in the attention: from 2^24 workgroups of
 *    a few tokens of one tensor in the norm and the append, from 2^23 tiles of a key head (256 rows of
 *    one sequence, or 32 where it has few) in the attention.
 */
#ifndef KDA_ATTN_H
#define KDA_ATTN_H

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Channels of a head at most, where rows are normed, rotated or appended. */
#define KDA_ROPE_MAX_D 1024

/* Strides of [B,H,T,d] rows, in elements; b is not read for packed rows and for B = 1. */
typedef struct kda_row_strides {
    int64_t b, h, t;
} kda_row_strides;

/* Strides of a paged cache [pages, Hk, page_size, d], in elements. */
typedef struct kda_page_strides {
    int64_t p, h, t;
} kda_page_strides;

/*
 * Norm and rotation of a head's row x of d channels at position pos:
 *
 *     y   = weight * x / sqrt(mean(x^2) + eps)                    (y = x without norm)
 *     z_a = rope_scale * (y_a cos th - y_b sin th)
 *     z_b = rope_scale * (y_b cos th + y_a sin th),   th = pos * inv_freq[i],  i < rot / 2,
 *
 * over the pairs (a, b) of the first rot channels: (i, i + rot/2), or (2i, 2i + 1) interleaved.
 * Channels from rot on are y. Frequencies that a longer context scales come in inv_freq, the factor
 * that goes with them in rope_scale. Angles are formed and reduced in fp64 from the fp32 frequency
 * and are off by at most 2^-51 of their size: 2^-31 at a million radians, 2^-20 at 2^31. The sum of a
 * row's squares must be finite in fp32.
 */
typedef struct kda_head_rope_desc {
    int64_t B;            /* blocks of rows, >= 1                                               */
    int64_t Hq, Hk;       /* heads of q and of k, 0 .. 4096 (0: that tensor is absent)          */
    int64_t T;            /* tokens per block, >= 0; B * T < 2^31                               */
    int64_t d;            /* channels per head, even, 2 .. KDA_ROPE_MAX_D                       */
    int64_t rot;          /* channels rotated, even, 0 .. d                                     */
    kda_row_strides q, k;         /* of q, k (and, in the backward, read again)                 */
    kda_row_strides q_out, k_out; /* of q_out, k_out; in the backward of dq_out, dk_out         */
    kda_row_strides dq, dk;       /* of dq, dk (backward only)                                  */
    int32_t dtype;        /* kda_dtype of every row                                             */
    int32_t interleaved;  /* 1: pairs (2i, 2i + 1); 0: pairs (i, i + rot/2)                     */
    int32_t norm;         /* 1: RMS norm; 0: none (weights must be NULL)                        */
    float eps;            /* > 0 (read with norm)                                               */
    float rope_scale;     /* finite (read with rot > 0)                                         */
} kda_head_rope_desc;

/*
 *   q, k               : [B,Hq,T,d], [B,Hk,T,d] dtype
 *   q_weight, k_weight : [d] fp32, or NULL (ones)
 *   inv_freq           : [rot / 2] fp32, finite; NULL exactly when rot = 0
 *   positions          : [B,T] int32, any value, or NULL (0 .. T-1 in each block)
 *   q_out, k_out       : like q, k (written)
 */
kda_status kda_head_rope_fwd(const kda_head_rope_desc* desc, const void* q, const void* k, const float* q_weight,
                             const float* k_weight, const float* inv_freq, const int32_t* positions,
                             void* q_out, void* k_out, void* stream);

/* Bytes of device workspace kda_head_rope_bwd needs (0 for an invalid desc, no rows or no norm). */
size_t kda_head_rope_bwd_workspace_bytes(const kda_head_rope_desc* desc);

/*
 * Backward: for L with dL/dq_out = dq_out and dL/dk_out = dk_out writes the gradients of q, k and the
 * weights. q and k are read with norm only (they may be NULL without it).
 *   dq, dk               : like q, k (written)
 *   dq_weight, dk_weight : [d] fp32 (written: sums over all rows, in a fixed order; zeros without
 *                          rows), or NULL to skip; need norm. Each may be asked for where the
 *                          weight itself is NULL (ones)
 *   workspace            : kda_head_rope_bwd_workspace_bytes(desc) bytes, 16-byte aligned; needed
 *                          only where a weight gradient is asked for
 */
kda_status kda_head_rope_bwd(const kda_head_rope_desc* desc, const void* q, const void* k, const float* q_weight,
                             const float* k_weight, const float* inv_freq, const int32_t* positions,
                             const void* dq_out, const void* dk_out, void* dq, void* dk, float* dq_weight,
                             float* dk_weight, void* workspace, size_t workspace_bytes, void* stream);

/*
 * The paged cache. Keys and values are bf16, k_cache [pages, Hk, page_size, dk] and v_cache
 * [pages, Hk, page_size, dv]. Position j of sequence s is row j % page_size of page
 * block_table[s][j / page_size]; sequences may share pages. kv_lens[s] counts the positions that hold
 * a token, the new ones of this step included: the n_s new tokens of sequence s are its last,
 * token i at position kv_lens[s] - n_s + i.
 *
 * New tokens come packed, sequence s the rows cu_seqlens[s] .. cu_seqlens[s+1]-1 of every head, or
 * as T rows of every sequence. cu_seqlens, kv_lens and block_table are read on the device only.
 * cu_seqlens must not decrease nor leave [0, T]. Rows before cu_seqlens[0] and from cu_seqlens[N] on
 * are in no sequence: they may be read but are not used, and their outputs are left as they were.
 * Values that break these rules, lengths past max_pages * page_size and page numbers outside
 * [0, pages) give undefined numbers but no access outside the tensors.
 */
typedef struct kda_kv_append_desc {
    int64_t N;            /* sequences, >= 1                                                    */
    int64_t Hq, Hk;       /* heads of q (0: no q) and of k and v (>= 1), up to 4096             */
    int64_t T;            /* packed: rows per head; else new tokens per sequence; >= 0, all
                             rows together < 2^31                                               */
    int64_t dk, dv;       /* channels of k (and q): even, 2 .. KDA_ROPE_MAX_D; of v: from 1     */
    int64_t rot;          /* channels rotated, even, 0 .. dk                                    */
    int64_t pages;        /* pages of the cache, 1 .. 2^31 - 1                                  */
    int64_t page_size;    /* rows of a page, 1 .. 2^20                                          */
    int64_t max_pages;    /* entries of a sequence in block_table; max_pages * page_size < 2^31 */
    int64_t table_stride; /* from a sequence's entries to the next one's, >= max_pages, or 0:
                             the same pages for every sequence                                  */
    kda_row_strides q, k, v, q_out;
    kda_page_strides k_cache, v_cache;
    int32_t in_dtype;     /* kda_dtype of q, k, v; q_out and the cache are bf16                 */
    int32_t packed;       /* 1: cu_seqlens says which rows are whose; 0: T rows a sequence      */
    int32_t interleaved, norm;
    float eps, rope_scale;
} kda_kv_append_desc;

/*
 * Norm and rotation of the new tokens' k at their positions into the cache, v copied beside it, norm
 * and rotation of q into q_out, in one launch. A token at a negative position (kv_lens[s] < n_s), past
 * max_pages * page_size or on a page outside [0, pages) is not stored; its q is rotated all the same.
 *   q             : [N,Hq,T,dk] (packed [Hq,T,dk]) in_dtype, or NULL with Hq = 0
 *   k, v          : [N,Hk,T,dk], [N,Hk,T,dv] (packed [Hk,T,..]) in_dtype
 *   q_weight, k_weight, inv_freq : as kda_head_rope_fwd
 *   cu_seqlens    : int32 [N+1] with packed, else NULL
 *   kv_lens       : int32 [N]; block_table: int32 [N, max_pages]
 *   q_out         : like q, bf16 (written); k_cache, v_cache: the new positions' rows written, no others
 * Two tokens must not fall on the same row of the same page.
 */
kda_status kda_kv_append(const kda_kv_append_desc* desc, const void* q, const void* k, const void* v,
                         const float* q_weight, const float* k_weight, const float* inv_freq,
                         const int32_t* cu_seqlens, const int32_t* kv_lens, const int32_t* block_table,
                         void* q_out, void* k_cache, void* v_cache, void* stream);

typedef struct kda_paged_attn_desc {
    int64_t N;            /* sequences, 1 .. 65536                                              */
    int64_t Hq, Hk;       /* query heads, up to 512, and key heads; Hq a multiple of Hk: query head
                             h reads key head h / (Hq / Hk)                                     */
    int64_t T;            /* packed: rows per head; else new tokens per sequence; the rows of
                             a key head's queries, all sequences together, < 2^31              */
    int64_t dk, dv;       /* 64 or 128 each: other widths, which the append takes, are refused
                             with KDA_ERR_UNSUPPORTED                                          */
    int64_t pages;        /* pages of the cache, 1 .. 2^31 - 1                                  */
    int64_t page_size;    /* rows of a page, a multiple of 16, up to 2^20                       */
    int64_t max_pages;    /* as kda_kv_append_desc, but max_pages * page_size <= 2^30           */
    int64_t table_stride;
    int64_t window;       /* keys that a query sees, its own among them, below 2^31; 0: all
                             before it                                                         */
    kda_row_strides q, o;
    kda_page_strides k_cache, v_cache;
    int32_t packed;
    float scale;          /* of the scores, finite                                              */
} kda_paged_attn_desc;

/* Bytes of device workspace kda_paged_attn needs (0 for an invalid desc or no rows). */
size_t kda_paged_attn_workspace_bytes(const kda_paged_attn_desc* desc);

/*
 * Attention of the new tokens over their sequences' positions in the cache, the new ones among them
 * (kda_kv_append stores those first): a token at position p sees positions j <= p, with a window
 * those with j > p - window,
 *
 *     o = sum_j softmax_j(scale * q . k_j) v_j,     lse = log sum_j exp(scale * q . k_j).
 *
 * A token that sees no position (one at a negative position) has o = 0 and lse = -inf. One that sees
 * scores of -inf alone (keys with an infinity) has lse = -inf and o = 0 / 0, NaN. What stands in rows
 * that a token does not see, NaN among it, does not reach its output.
 *   q           : [N,Hq,T,dk] (packed [Hq,T,dk]) bf16; k_cache, v_cache as above. Bases on 16 bytes,
 *                 strides multiples of 8 elements; from page to page less than 2^31
 *                 elements, the rows of one page and head within 2^31 bytes
 *   o           : [N,Hq,T,dv] (packed [Hq,T,dv]) bf16 (written), base on 16 bytes, strides as q's
 *   lse         : fp32 [N,Hq,T] (packed [Hq,T]), dense (written), or NULL to skip
 *   workspace   : kda_paged_attn_workspace_bytes(desc) bytes, 16-byte aligned; calls that overlap in
 *                 time need one each; nothing in it has to be cleared or kept
 * Sums run in an order that the lengths alone fix: the same call gives the same bits.
 */
kda_status kda_paged_attn(const kda_paged_attn_desc* desc, const void* q, const void* k_cache, const void* v_cache,
                          const int32_t* cu_seqlens, const int32_t* kv_lens, const int32_t* block_table, void* o,
                          float* lse, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_ATTN_H */
