// The backward of the gated linear recurrence for fp32 inputs (kda_glr_bwd.h).
#include "kda_glr_bwd.h"

namespace kda {
namespace glr {

template hipError_t launch_bwd_t<KDA_GLR_ONE, false, float>(const GlrArgs&, const GlrWs&, hipStream_t);
template hipError_t launch_bwd_t<KDA_GLR_LEAKY, false, float>(const GlrArgs&, const GlrWs&, hipStream_t);
template hipError_t launch_bwd_t<KDA_GLR_NORM, false, float>(const GlrArgs&, const GlrWs&, hipStream_t);
template hipError_t launch_bwd_t<KDA_GLR_ONE, true, float>(const GlrArgs&, const GlrWs&, hipStream_t);
template hipError_t launch_bwd_t<KDA_GLR_LEAKY, true, float>(const GlrArgs&, const GlrWs&, hipStream_t);
template hipError_t launch_bwd_t<KDA_GLR_NORM, true, float>(const GlrArgs&, const GlrWs&, hipStream_t);

}  // namespace glr
}  // namespace kda
