// scaled_prefill_int8.cu -- attention of many query rows over block-scaled 8-bit integer
// codes (see scaled_prefill.cuh).
#include "scaled_prefill.cuh"

namespace pagedkv {

template cudaError_t launch_scaled_prefill<int8_code_t, 64>(const ScaledAttnParams& p, cudaStream_t stream);
template cudaError_t launch_scaled_prefill<int8_code_t, 128>(const ScaledAttnParams& p, cudaStream_t stream);

}  // namespace pagedkv
