// scaled_prefill_int8_f16.cu -- attention of many query rows over block-scaled
// 8-bit integer codes, binary16 queries and outputs (see scaled_prefill.cuh).
#include "scaled_prefill.cuh"

namespace pagedkv {

cudaError_t launch_scaled_prefill_int8_f16(const ScaledAttnParams& p, int head_size, cudaStream_t stream) {
    return launch_scaled_prefill<int8_code_t, true>(p, head_size, stream);
}

}  // namespace pagedkv
