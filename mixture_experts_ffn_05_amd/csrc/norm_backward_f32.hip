// Norms around a block, backward, for f32 activations.
#include "norm_backward.h"

namespace moe {

hipError_t launch_norm_in_backward_f32(const NormArgs& a, hipStream_t s) { return launch_type<float, false>(a, s); }
hipError_t launch_norm_out_backward_f32(const NormArgs& a, hipStream_t s) { return launch_type<float, true>(a, s); }

}  // namespace moe
