// The MoE layer for a few tokens with bfloat16 weights (layer_kernels.cuh).
#include "layer_kernels.cuh"

namespace moe {

cudaError_t launch_layer_bf16(const LayerArgs& a, int num_sms, cudaStream_t stream) {
    return launch_layer_f<kWBf16>(a, num_sms, stream);
}

}  // namespace moe
