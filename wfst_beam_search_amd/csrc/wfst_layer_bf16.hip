// The output layer for hidden states in bfloat16.
#include "wfst_layer_kernels.h"

namespace wfst {

hipError_t launch_layer_bf16(const Layer &l, const LayerCall &c, hipStream_t s) { return layer_xt<__bf16>(l, c, s); }

}  // namespace wfst
