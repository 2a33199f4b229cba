// Norms around a block, backward, for bf16 activations.
#include "norm_backward.h"

namespace moe {

hipError_t launch_norm_in_backward_bf16(const NormArgs& a, hipStream_t s) { return launch_type<bf16_t, false>(a, s); }
hipError_t launch_norm_out_backward_bf16(const NormArgs& a, hipStream_t s) { return launch_type<bf16_t, true>(a, s); }

}  // namespace moe
