// Attention over a paged cache with heads of 128 and 128 channels (kda_attn_main.h).
#include "kda_attn_main.h"

template hipError_t kda::attn::launch_main<128, 128>(const kda::AttnArgs&, bool, int64_t, hipStream_t);
