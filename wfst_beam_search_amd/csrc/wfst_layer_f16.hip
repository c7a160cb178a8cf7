// The output layer for hidden states in binary16.
#include "wfst_layer_kernels.h"

namespace wfst {

hipError_t launch_layer_f16(const Layer &l, const LayerCall &c, hipStream_t s) { return layer_xt<_Float16>(l, c, s); }

}  // namespace wfst
