// scaled_prefill_e4m3.cu -- attention of many query rows over block-scaled E4M3
// codes (see scaled_prefill.cuh).
#include "scaled_prefill.cuh"

namespace pagedkv {

template cudaError_t launch_scaled_prefill<e4m3_t, 64>(const ScaledAttnParams& p, cudaStream_t stream);
template cudaError_t launch_scaled_prefill<e4m3_t, 128>(const ScaledAttnParams& p, cudaStream_t stream);

}  // namespace pagedkv
