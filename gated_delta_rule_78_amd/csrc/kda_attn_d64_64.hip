// Attention over a paged cache with heads of 64 and 64 channels (kda_attn_main.h).
#include "kda_attn_main.h"

template hipError_t kda::attn::launch_main<64, 64>(const kda::AttnArgs&, bool, int64_t, hipStream_t);
