// sparse_decode_f16.cu -- the fused block-sparse decode for binary16 caches.
#include "sparse_decode.cuh"

namespace pagedkv {

cudaError_t launch_sparse_decode_f16(const SparseParams& p, int head_size, cudaStream_t stream) {
    return launch_sparse_types<__half, __half>(p, head_size, stream);
}

}  // namespace pagedkv
