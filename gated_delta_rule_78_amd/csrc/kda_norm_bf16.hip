// The block norms for bf16 block outputs (kda_norm_kernels.h).
#include "kda_norm_kernels.h"

template hipError_t kda::norm::launch_i<kda::bf16_t>(const kda::NormArgs&, bool, hipStream_t);
