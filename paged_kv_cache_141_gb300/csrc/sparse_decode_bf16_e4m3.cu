// sparse_decode_bf16_e4m3.cu -- the fused block-sparse decode for E4M3 caches with a bfloat16 query.
#include "sparse_decode.cuh"

namespace pagedkv {

cudaError_t launch_sparse_decode_bf16_e4m3(const SparseParams& p, int head_size, cudaStream_t stream) {
    return launch_sparse_types<__nv_bfloat16, e4m3_t>(p, head_size, stream);
}

}  // namespace pagedkv
