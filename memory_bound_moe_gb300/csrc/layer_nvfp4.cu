// The MoE layer for a few tokens with NVFP4 weights (layer_fp4.cuh).
#include "layer_fp4.cuh"

namespace moe {

cudaError_t launch_layer_nvfp4(const LayerArgs& a, int num_sms, cudaStream_t stream) {
    return launch_layer_fp4<kWNvfp4>(a, num_sms, stream);
}

}  // namespace moe
