// The MoE layer for a few tokens with MXFP4 weights (layer_fp4.cuh).
#include "layer_fp4.cuh"

namespace moe {

cudaError_t launch_layer_mxfp4(const LayerArgs& a, int num_sms, cudaStream_t stream) {
    return launch_layer_fp4<kWMxfp4>(a, num_sms, stream);
}

}  // namespace moe
