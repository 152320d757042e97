/*
 * kda_glr.h -- C ABI of the gated linear recurrence, the elementwise sibling of the KDA core
 * (kda.h), for AMD Instinct MI355X (gfx950). Same library, same conventions (device pointers owned
 * by the caller, asynchronous on `stream`, arguments validated before any device work, kda_status,
 * no allocation, no synchronisation, no state kept between calls).
 *
 * Per (sequence, head, channel) a scalar fp32 state h evolves token by token as
 *
 *     h_t = alpha_t h_{t-1} + w(alpha_t) i_t x_t,        y_t = h_t,
 *
 *   alpha_t = exp(log_alpha_t), the log decay given or computed from its pre-activation z as
 *             log_alpha_t = g_min * sigmoid(exp(A_log[h, c]) * z_t)     (kda_gating's decay
 *             equation, with one log scale per channel instead of one per head);
 *   i_t     = sigmoid(in_gate_t), or 1 without an input gate;
 *   w       = 1, 1 - alpha, or sqrt(1 - alpha^2) (kda_glr_scale).
 *
 *  - Rows are tokens, the last dimension is the d >= 1 channels of a head: [B,H,T,d], or a packed
 *    batch [H,T,d]. Rows of D channels per token with no head split are H = 1, d = D.
 *  - Everything between the inputs and the outputs is computed in fp32; y and the gradients of
 *    tensors are rounded once.
 *  - Log decays must be <= 0; -inf is allowed (alpha = 0: the state restarts). Positive or NaN log
 *    decays give undefined numbers. A non-finite x, decay or state makes the later outputs of its
 *    own channel and sequence non-finite (also past alpha = 0), and no others.
 *  - Every tensor is dense, its base aligned to its element; workspaces are aligned to 16 bytes.
 *  - Long sequences pass their states between workgroups of one launch, which wait for each other.
 *    The order in which they start lets every wait end. Each is bounded all the same (2^26 looks,
 *    over half a minute): one that gave up would hand on NaN, which makes the outputs behind it NaN
 *    while the call has long returned KDA_OK.
 *  - Every sum runs in a fixed order: the same inputs give the same bits on every call.
 *  - A launch has fewer than 2^32 threads. A call that would need more is refused with
 *    KDA_ERR_UNSUPPORTED, and its workspace query answers 0: from 2^23 tiles on (at most 64 channels
 *    by 256 rows of a block, 128 rows in the backward and for d < 4), 2^22 heads with z in the
 *    backward (d <= 64), or 2^34 channels of all sequences in a step or in 16 rows and fewer.
 */
#ifndef KDA_GLR_H
#define KDA_GLR_H

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Channels per head at most. */
#define KDA_GLR_MAX_D (1 << 20)

/* Rows per chunk of the sequence split: entry states are stored every KDA_GLR_CHUNK rows. */
#define KDA_GLR_CHUNK 128

typedef enum kda_glr_scale {
    KDA_GLR_ONE = 0,    /* w = 1                                                                */
    KDA_GLR_LEAKY = 1,  /* w = 1 - alpha                                                        */
    KDA_GLR_NORM = 2    /* w = sqrt(1 - alpha^2); the backward takes dw/dlog_alpha = 0 at
                           alpha = 1, where w = 0 and the derivative has no value. Log decays
                           within 2^-126 of 0 (subnormal ones) may count as 0                  */
} kda_glr_scale;

/* Shape and types of one call over a batch of sequences. */
typedef struct kda_glr_desc {
    int64_t N;          /* sequences, >= 1                                                     */
    int64_t H;          /* heads, >= 1                                                         */
    int64_t T;          /* packed: rows per head; else tokens per sequence. 0 <= T < 2^31 - 128 */
    int64_t d;          /* channels per head, 1 .. KDA_GLR_MAX_D                               */
    int32_t in_dtype;   /* kda_dtype of x, log_alpha / z, in_gate and of their gradients       */
    int32_t out_dtype;  /* kda_dtype of y and dy                                               */
    int32_t packed;     /* 1: sequence s is rows cu_seqlens[s] .. cu_seqlens[s+1]-1 of every
                           head; 0: N sequences of T tokens                                    */
    int32_t scale;      /* kda_glr_scale                                                       */
    float g_min;        /* decay lower bound, < 0 (read with z only)                           */
} kda_glr_desc;

/* The gates of a call: exactly one of log_alpha and z, A_log with z. */
typedef struct kda_glr_gates {
    const void* log_alpha;   /* log decay, shape of x, in_dtype                                */
    const void* z;           /* decay pre-activation, shape of x, in_dtype                     */
    const float* A_log;      /* [H,d] fp32 log scale of z; g_min * exp(A_log) and g_min *      */
                             /* log2(e) must be finite in fp32                                 */
    const void* in_gate;     /* input gate pre-activation, shape of x, in_dtype, or NULL       */
} kda_glr_gates;

/* Bytes of device workspace kda_glr_fwd needs (0 when it needs none, and for an invalid desc). */
size_t kda_glr_fwd_workspace_bytes(const kda_glr_desc* desc);

/*
 * Prefill: (x, gates, S0) -> (y, S_T).
 *   x, gates     : [N,H,T,d] in_dtype, packed [H,T,d]
 *   cu_seqlens   : packed: DEVICE int32 [N+1], non-decreasing, within [0, T]; read on the device
 *                  only. Rows before cu_seqlens[0] and from cu_seqlens[N] on are in no sequence:
 *                  they are not read into any state and y (and every gradient) is left as it was
 *                  there. Lengths that break these rules give undefined numbers but no access
 *                  outside the tensors. NULL when packed = 0.
 *   S0           : [N,H,d] fp32 entry states, or NULL (zero)
 *   y            : x's shape, out_dtype (written)
 *   S_T          : [N,H,d] fp32 states after each sequence's last token (written; an empty
 *                  sequence's is its S0), or NULL to skip; may be S0, must not overlap it partially
 *   entry_states : fp32 [N*H, ceil(T/KDA_GLR_CHUNK), d], packed [H, ceil(T/KDA_GLR_CHUNK), d]:
 *                  the state before row c*KDA_GLR_CHUNK of each block of rows (written; what
 *                  kda_glr_bwd restarts from), or NULL to skip
 *   workspace    : kda_glr_fwd_workspace_bytes(desc) bytes, 16-byte aligned. Calls that overlap in
 *                  time need a workspace each; nothing in it has to be cleared or kept.
 * No output may overlap an input, the workspace or another output (S_T = S0 aside).
 */
kda_status kda_glr_fwd(const kda_glr_desc* desc, const void* x, const kda_glr_gates* gates,
                       const int32_t* cu_seqlens, const float* S0, void* y, float* S_T,
                       float* entry_states, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of device workspace kda_glr_bwd needs; has_entry_states: the call passes entry_states. */
size_t kda_glr_bwd_workspace_bytes(const kda_glr_desc* desc, int32_t has_entry_states, int32_t has_z);

/*
 * Backward: for L with dL/dy = dy and dL/dS_T = dS_T, writes the gradients of every input.
 *   inputs as kda_glr_fwd; entry_states: what kda_glr_fwd wrote for these inputs, or NULL (the
 *   call recomputes them into its workspace)
 *   dy           : y's shape, out_dtype       dS_T : [N,H,d] fp32, or NULL (zero)
 *   dx           : x's shape, in_dtype (written)
 *   ddecay       : gradient of log_alpha (or, with z, of z): its shape, in_dtype (written)
 *   din_gate     : with in_gate: gradient, in_dtype (written); else NULL
 *   dA_log       : with z: [H,d] fp32 (written, summed over sequences and tokens); else NULL
 *   dS0          : [N,H,d] fp32 (written; an empty sequence's is its dS_T), or NULL to skip
 * No output may overlap an input, the workspace or another output.
 */
kda_status kda_glr_bwd(const kda_glr_desc* desc, const void* x, const kda_glr_gates* gates,
                       const int32_t* cu_seqlens, const float* S0, const float* entry_states,
                       const void* dy, const float* dS_T, void* dx, void* ddecay, void* din_gate,
                       float* dA_log, float* dS0, void* workspace, size_t workspace_bytes, void* stream);

/*
 * One token of N sequences: x, gates [N,H,d]; S [N,H,d] fp32 read and overwritten in place;
 * y [N,H,d] out_dtype (written). desc->T and desc->packed are not read. No output may overlap an
 * input or the other.
 */
kda_status kda_glr_step(const kda_glr_desc* desc, const void* x, const kda_glr_gates* gates,
                        float* S, void* y, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_GLR_H */
