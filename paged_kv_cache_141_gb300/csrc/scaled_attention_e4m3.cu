// scaled_attention_e4m3.cu -- attention over block-scaled E4M3 codes (see
// scaled_attention.cuh).
#include "scaled_attention.cuh"

namespace pagedkv {

cudaError_t launch_scaled_attention_e4m3(const ScaledAttnParams& p, int head_size, cudaStream_t stream) {
    return launch_scaled<e4m3_t>(p, head_size, stream);
}

}  // namespace pagedkv
