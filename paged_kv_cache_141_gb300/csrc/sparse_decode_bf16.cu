// sparse_decode_bf16.cu -- the fused block-sparse decode for bfloat16 caches.
#include "sparse_decode.cuh"

namespace pagedkv {

cudaError_t launch_sparse_decode_bf16(const SparseParams& p, int head_size, cudaStream_t stream) {
    return launch_sparse_types<__nv_bfloat16, __nv_bfloat16>(p, head_size, stream);
}

}  // namespace pagedkv
