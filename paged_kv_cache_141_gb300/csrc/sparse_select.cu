// sparse_select.cu -- the selection of a block-sparse decode as a table of
// slabs (block * Hkv + head) in ascending block order, so that only its last
// block, the newest, can be partial: the paged decode reads it as a block
// table of S * Hkv one-head sequences. For the shapes that the fused kernel
// (sparse_decode.cuh) does not take.
#include "sparse_select.cuh"

namespace pagedkv {

namespace {

constexpr int NT = 256;

template <typename T, int D, bool kOneTile>
__global__ void __launch_bounds__(NT, 2)
select_blocks_kernel(const __grid_constant__ SelectParams p) {
    begin_overlapped();
    extern __shared__ __align__(16) uint8_t dyn[];
    __shared__ SelShared<NT> sh;
    cg::cluster_group cluster = cg::this_cluster();
    const SelRow rw(p, cluster, dyn);
    if (!std::is_same<T, float>::value && rw.scored) stage_sides<T, D, NT>(p, rw);
    score_and_take<T, D, kOneTile, NT>(p, sh, cluster, rw);
    if (rw.rank != 0) return;
    int32_t* slabs = p.slab_tables + (size_t)rw.row * p.table_width;
    int32_t* out = p.selected ? p.selected + (size_t)rw.row * p.num_select : nullptr;
    const int total = rw.n < p.num_select ? rw.n : p.num_select;
    for_taken(sh, rw, [&](int at, int b) {
        slabs[at] = slab_of(p, rw, b);
        if (out) out[at] = b;
    });
    if (threadIdx.x == 0)
        p.slab_lens[rw.row] = total * p.block_size - (rw.n * p.block_size - rw.L);
    if (out)
        for (int i = total + threadIdx.x; i < p.num_select; i += NT) out[i] = -1;
}

template <typename T, int D>
cudaError_t launch_select(SelectParams p, cudaStream_t stream) {
    const int rows = p.num_seqs * p.num_kv_heads;
    const int C = select_cluster(rows, p.max_ctx_blocks);
    const int smem = select_smem<T, D>(p);
    // one MMA tile of heads, or (binary32 has no tiles) any number
    auto kernel = std::is_same<T, float>::value || p.group <= 8 ? select_blocks_kernel<T, D, true>
                                                                : select_blocks_kernel<T, D, false>;
    return launch_cluster(kernel, p, rows * C, C, NT, smem, stream);
}

template <typename T>
cudaError_t launch_select_d(const SelectParams& p, int head_size, cudaStream_t stream) {
    switch (head_size) {
    case 64: return launch_select<T, 64>(p, stream);
    case 128: return launch_select<T, 128>(p, stream);
    default: return launch_select<T, 256>(p, stream);
    }
}

}  // namespace

cudaError_t launch_select_blocks(const SelectParams& p, int head_size, pa_dtype q_dtype,
                                 cudaStream_t stream) {
    switch (q_dtype) {
    case PA_F32: return launch_select_d<float>(p, head_size, stream);
    case PA_F16: return launch_select_d<__half>(p, head_size, stream);
    default: return launch_select_d<__nv_bfloat16>(p, head_size, stream);
    }
}

}  // namespace pagedkv
