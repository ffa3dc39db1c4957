// The block norms of fp16 activations.
#include "block_norm_kernels.hpp"

namespace iris {

template hipError_t launch_norm<f16>(const NormArgs&, bool, bool, hipStream_t);
template hipError_t launch_norm_bwd<f16>(const NormBwdArgs&, bool, bool, hipStream_t);

}  // namespace iris
