// The forward of the gated linear recurrence for bf16 inputs (kda_glr_fwd.h).
#include "kda_glr_fwd.h"

namespace kda {
namespace glr {

template hipError_t launch_fwd_t<KDA_GLR_ONE, false, bf16_t>(const GlrArgs&, const GlrWs&, hipStream_t);
template hipError_t launch_fwd_t<KDA_GLR_LEAKY, false, bf16_t>(const GlrArgs&, const GlrWs&, hipStream_t);
template hipError_t launch_fwd_t<KDA_GLR_NORM, false, bf16_t>(const GlrArgs&, const GlrWs&, hipStream_t);
template hipError_t launch_fwd_t<KDA_GLR_ONE, true, bf16_t>(const GlrArgs&, const GlrWs&, hipStream_t);
template hipError_t launch_fwd_t<KDA_GLR_LEAKY, true, bf16_t>(const GlrArgs&, const GlrWs&, hipStream_t);
template hipError_t launch_fwd_t<KDA_GLR_NORM, true, bf16_t>(const GlrArgs&, const GlrWs&, hipStream_t);

}  // namespace glr
}  // namespace kda
