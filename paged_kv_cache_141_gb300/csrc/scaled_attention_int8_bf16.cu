// scaled_attention_int8_bf16.cu -- attention over block-scaled 8-bit integer codes, bfloat16
// queries and outputs (see scaled_attention.cuh).
#include "scaled_attention.cuh"

namespace pagedkv {

cudaError_t launch_scaled_attention_int8_bf16(const ScaledAttnParams& p, int head_size, cudaStream_t stream) {
    return launch_scaled_warps<int8_code_t, false>(p, head_size, stream);
}

}  // namespace pagedkv
