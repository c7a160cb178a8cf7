// The output layer for hidden states in binary32.
#include "wfst_layer_kernels.h"

namespace wfst {

hipError_t launch_layer_f32(const Layer &l, const LayerCall &c, hipStream_t s) { return layer_xt<float>(l, c, s); }

}  // namespace wfst
