// scaled_attention_int8_f16.cu -- attention over block-scaled 8-bit integer codes, binary16
// queries and outputs (see scaled_attention.cuh).
#include "scaled_attention.cuh"

namespace pagedkv {

cudaError_t launch_scaled_attention_int8_f16(const ScaledAttnParams& p, int head_size, cudaStream_t stream) {
    return launch_scaled_warps<int8_code_t, true>(p, head_size, stream);
}

}  // namespace pagedkv
