// Internal launcher interface of the gated linear recurrence (include/kda_glr.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

// Rows come in blocks: N*H blocks of T rows (block n*H + h), or, packed, H blocks of T rows that
// hold every sequence. A block's rows split into nch chunks.
struct GlrArgs {
    int64_t N, H, T, d;
    int64_t blocks, nch;
    bool in_bf16, out_bf16, packed;
    int scale;               // kda_glr_scale
    float g_min;
    const void *x, *la, *z;  // one of la and z
    const float* A_log;
    const void* u;           // input gate pre-activation or NULL
    const int32_t* cu;       // packed: [N+1]
    const float* S0;         // [N,H,d] or NULL
    void* y;
    float* S_T;
    float* entry;            // [blocks][nch][d]: forward writes (may be NULL), backward reads
    // backward
    const void* dy;
    const float* dST;
    void *dx, *dd, *du;
    float *dA, *dS0;
    unsigned char* ws;
    // step: x, gates and y as [N,H,d], S updated in place
    float* S;
};

namespace glr {

// Workspace of a tiled launch, carved by kda_glr.hip: the tile counters, the rows where sequences
// start and end (packed), the chain's two words per tile and channel, the tiles' parts of dA_log.
struct GlrWs {
    uint32_t* ticket;                    // counters, a cache line each
    int64_t counters;
    uint32_t *sbits, *ebits;             // packed: a bit per row, [nt * rows / 32]
    int32_t *start, *end;                // packed: the sequence of a marked row, [T]
    unsigned long long *span, *state;    // [blocks][nt][d]
    float* dA;                           // [blocks][nt][d]
    int64_t nt, rows;                    // tiles per block, rows per tile
    int vec;                             // channels per thread: 4 or 1
    bool narrow;                         // several heads side by side in a tile
};

// Rows of a tile: forward with 4 channels and with 1 channel a thread, backward.
constexpr int kFwdRows = 256, kFwdRows1 = 128, kBwdRows = 128;

// Instantiated per input type (kda_glr_fwd_*.hip, kda_glr_bwd_*.hip).
template <int SCALE, bool PACKED, typename TIn>
hipError_t launch_fwd_t(const GlrArgs& a, const GlrWs& ws, hipStream_t st);
template <int SCALE, bool PACKED, typename TIn>
hipError_t launch_bwd_t(const GlrArgs& a, const GlrWs& ws, hipStream_t st);

// The forward of blocks of at most KDA_GLR_CHUNK rows, a thread per 4 channels, or per channel where 4
// do not divide them (kda_glr_rows.hip).
hipError_t launch_rows(const GlrArgs& a, hipStream_t st);
// The backward of blocks of at most kRowsBwd rows; `parts`: [blocks][d] parts of dA_log (with z).
constexpr int kRowsBwd = 16;
hipError_t launch_rows_bwd(const GlrArgs& a, float* parts, hipStream_t st);

}  // namespace glr

size_t glr_fwd_ws_bytes(const GlrArgs& a);
size_t glr_bwd_ws_bytes(const GlrArgs& a);
hipError_t launch_glr_fwd(const GlrArgs& a, hipStream_t st);
hipError_t launch_glr_bwd(const GlrArgs& a, hipStream_t st);
hipError_t launch_glr_step(const GlrArgs& a, hipStream_t st);

}  // namespace kda
