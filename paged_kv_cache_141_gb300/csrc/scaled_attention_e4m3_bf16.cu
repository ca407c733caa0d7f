// scaled_attention_e4m3_bf16.cu -- attention over block-scaled E4M3 codes, bfloat16
// queries and outputs (see scaled_attention.cuh).
#include "scaled_attention.cuh"

namespace pagedkv {

cudaError_t launch_scaled_attention_e4m3_bf16(const ScaledAttnParams& p, int head_size, cudaStream_t stream) {
    return launch_scaled_warps<e4m3_t, false>(p, head_size, stream);
}

}  // namespace pagedkv
