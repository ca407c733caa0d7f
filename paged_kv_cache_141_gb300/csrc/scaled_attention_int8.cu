// scaled_attention_int8.cu -- attention over block-scaled 8-bit integer codes (see
// scaled_attention.cuh).
#include "scaled_attention.cuh"

namespace pagedkv {

cudaError_t launch_scaled_attention_int8(const ScaledAttnParams& p, int head_size, cudaStream_t stream) {
    return launch_scaled<int8_code_t>(p, head_size, stream);
}

}  // namespace pagedkv
