// scaled_prefill_e4m3_bf16.cu -- attention of many query rows over block-scaled
// E4M3 codes, bfloat16 queries and outputs (see scaled_prefill.cuh).
#include "scaled_prefill.cuh"

namespace pagedkv {

cudaError_t launch_scaled_prefill_e4m3_bf16(const ScaledAttnParams& p, int head_size, cudaStream_t stream) {
    return launch_scaled_prefill<e4m3_t, false>(p, head_size, stream);
}

}  // namespace pagedkv
