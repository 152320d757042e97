// Head norms with rotation and the cache append for fp32 rows (kda_rope_fwd.h, kda_rope_bwd.h).
#include "kda_rope_bwd.h"

namespace kda {
namespace rope {
template hipError_t launch_rows<float, float, false>(const RopeArgs&, const Shape&, int, hipStream_t);
template hipError_t launch_rows<float, bf16_t, true>(const RopeArgs&, const Shape&, int, hipStream_t);
template hipError_t launch_grads<float>(const RopeArgs&, const Shape&, int, bool, hipStream_t);
}  // namespace rope
}  // namespace kda
