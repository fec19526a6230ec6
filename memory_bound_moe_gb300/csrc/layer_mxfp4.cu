// The MoE layer for a few tokens with MXFP4 weights (layer_kernels.cuh).
#include "layer_kernels.cuh"

namespace moe {

cudaError_t launch_layer_mxfp4(const LayerArgs& a, int num_sms, cudaStream_t stream) {
    return launch_layer_f<kWMxfp4>(a, num_sms, stream);
}

}  // namespace moe
