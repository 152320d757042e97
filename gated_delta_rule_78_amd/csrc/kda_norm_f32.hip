// The block norms for fp32 block outputs (kda_norm_kernels.h).
#include "kda_norm_kernels.h"

template hipError_t kda::norm::launch_i<float>(const kda::NormArgs&, bool, hipStream_t);
