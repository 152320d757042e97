// Compiled to assembly by tests/test_attn_lds_loads.py, never run: a load into LDS by the attention's inline assembly
// between two of the compiler's own, which take their LDS address from m0 as well.
#include "kda_attn_kernels.h"

__global__ void lds_loads(const float* in, kda::attn::i32x4 r, unsigned off, unsigned at, float* out) {
    __shared__ __align__(1024) float lds[1024];
    const auto rs = kda::make_rsrc(in, 4096);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (kda::lds_void*)lds, 4, (int)off, 0, 0, 0);
    kda::attn::load_to_lds(r, off, kda::attn::lds_address(lds) + at);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (kda::lds_void*)lds, 4, (int)off + 256, 0, 256, 0);
    kda::attn::wait_vm<0>();
    kda::lds_barrier();
    out[threadIdx.x] = lds[threadIdx.x];
}

// Loads whose descriptors are read from lanes right before them.
__global__ void lane_descriptors(const int* in, unsigned off, unsigned at, float* out) {
    __shared__ __align__(1024) float lds[4096];
    int w[4], n = (int)at;
    for (int k = 0; k < 4; ++k) w[k] = in[threadIdx.x + 64 * k];
    for (int i = 0; i < n; ++i) {
        kda::attn::i32x4 r;
        for (int k = 0; k < 4; ++k) r[k] = __builtin_amdgcn_readlane(w[k], i);
        kda::attn::load_to_lds(r, off, kda::attn::lds_address(lds) + 1024 * (i & 3), (unsigned)__builtin_amdgcn_readlane(w[0], i + 1));
    }
    kda::attn::wait_vm<0>();
    kda::lds_barrier();
    out[threadIdx.x] = lds[threadIdx.x];
}
