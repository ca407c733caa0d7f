// sparse_select.cu -- which blocks a block-sparse decode reads. For a sequence
// of n blocks and each KV head h,
//     score(b) = max over the group's query heads g of
//                sum_d max(q_gd lo_bd, q_gd hi_bd),
// the largest value q_g . k can take for keys within block b's bounds. The
// first `first_blocks` and the newest `recent_blocks` blocks are always taken;
// of the others the num_select - first - recent of largest score (ties: the
// lowest index; a NaN score counts as +infinity, so that a NaN key is read and
// shows, as it would in the dense decode). n <= num_select: every block.
// The order is that of the exact scores, held here in binary64.
//
// The selection goes out as a table of slabs (block * Hkv + head) in ascending
// block order, so that only its last block, the newest, can be partial: the
// paged decode reads it as a block table of S * Hkv one-head sequences.
#include "device_common.cuh"
#include "launch.h"

namespace pagedkv {

namespace {

constexpr int kScoreThreads = 256;
constexpr int kSelectThreads = 512;

// The sequence's length as the decode takes it (clamped to what the table and
// the bound allow).
__device__ __forceinline__ int clamped_len(const SelectParams& p, int s, bool& bad) {
    int L = p.context_lens[s];
    const int64_t tab = (int64_t)p.max_blocks * p.block_size;
    const int cap = tab < p.max_context_len ? (int)tab : p.max_context_len;
    bad = L < 0 || L > cap;
    return L < 0 ? 0 : (L > cap ? cap : L);
}

// One warp per (row, block).
template <typename T, int D>
__global__ void __launch_bounds__(kScoreThreads)
block_scores_kernel(const __grid_constant__ SelectParams p) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int b = blockIdx.x * (kScoreThreads / 32) + (threadIdx.x >> 5);
    for (int row = blockIdx.y; row < p.num_seqs * p.num_kv_heads; row += gridDim.y) {
        const int s = row / p.num_kv_heads;
        const int h = row - s * p.num_kv_heads;
        bool bad;
        const int L = clamped_len(p, s, bad);
        const int n = (L + p.block_size - 1) / p.block_size;
        if (b >= n || n <= p.num_select) continue;
        const int64_t blk = p.block_tables[(size_t)s * p.max_blocks + b];
        double best = -INFINITY;
        if (blk >= 0 && blk < p.num_blocks) {
            const T* bounds = static_cast<const T*>(p.k_bounds) + ((size_t)blk * p.num_kv_heads + h) * 2 * D + lane * E;
            float lo[E], hi[E], q[E];
            RowLoader<T, E>::load(bounds, lo);
            RowLoader<T, E>::load(bounds + D, hi);
            for (int g = 0; g < p.group; ++g) {
                RowLoader<T, E>::load(static_cast<const T*>(p.query) +
                                      ((size_t)s * p.num_q_heads + h * p.group + g) * D + lane * E, q);
                double sum = 0.0;
#pragma unroll
                for (int i = 0; i < E; ++i)
                    sum += (double)q[i] * (double)(q[i] < 0.f ? lo[i] : hi[i]);
#pragma unroll
                for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
                if (isnan(sum)) sum = INFINITY;
                best = sum > best ? sum : best;
            }
        }
        if (lane == 0) p.scores[(size_t)row * p.max_ctx_blocks + b] = best;
    }
}

// One CTA per row: a block is taken if fewer than the wanted number of
// candidates come before it; the taken ones go out in block order.
__global__ void __launch_bounds__(kSelectThreads)
select_blocks_kernel(const __grid_constant__ SelectParams p) {
    __shared__ int warp_count[kSelectThreads / 32];
    __shared__ int base;
    const int row = blockIdx.x;
    const int s = row / p.num_kv_heads;
    const int h = row - s * p.num_kv_heads;
    bool bad;
    const int L = clamped_len(p, s, bad);
    if (bad && h == 0 && threadIdx.x == 0 && p.status) atomicOr(p.status, PA_DEV_BAD_LEN);
    const int B = p.block_size;
    const int n = (L + B - 1) / B;
    const int want = p.num_select - p.first_blocks - p.recent_blocks;
    const int lo = p.first_blocks, hi = n - p.recent_blocks;   // the candidates
    const double* score = p.scores + (size_t)row * p.max_ctx_blocks;
    const int32_t* table = p.block_tables + (size_t)s * p.max_blocks;
    int32_t* slabs = p.slab_tables + (size_t)row * p.table_width;
    int32_t* out = p.selected ? p.selected + (size_t)row * p.num_select : nullptr;
    if (threadIdx.x == 0) base = 0;
    __syncthreads();
    for (int b0 = 0; b0 < n; b0 += kSelectThreads) {
        const int b = b0 + threadIdx.x;
        bool take = b < n && (n <= p.num_select || b < lo || b >= hi);
        if (b < n && !take) {
            const double mine = score[b];
            int before = 0;
            for (int o = lo; o < hi && before < want; ++o) {
                const double x = score[o];
                before += x > mine || (x == mine && o < b);
            }
            take = before < want;
        }
        const uint32_t votes = __ballot_sync(0xffffffffu, take);
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        if (lane == 0) warp_count[warp] = __popc(votes);
        __syncthreads();
        int at = base + __popc(votes & ((1u << lane) - 1));
        for (int w = 0; w < warp; ++w) at += warp_count[w];
        if (take) {
            const int64_t blk = table[b];
            slabs[at] = blk >= 0 && blk < p.num_blocks ? (int32_t)(blk * p.num_kv_heads + h) : -1;
            if (out) out[at] = b;
        }
        __syncthreads();
        if (threadIdx.x == 0)
            for (int w = 0; w < kSelectThreads / 32; ++w) base += warp_count[w];
        __syncthreads();
    }
    const int taken = base;                                   // min(n, num_select)
    if (threadIdx.x == 0) p.slab_lens[row] = taken * B - (n * B - L);
    if (out)
        for (int i = taken + threadIdx.x; i < p.num_select; i += kSelectThreads) out[i] = -1;
}

template <typename T>
void launch_scores(const SelectParams& p, int head_size, cudaStream_t stream) {
    const int rows = p.num_seqs * p.num_kv_heads;
    const dim3 grid((p.max_ctx_blocks + kScoreThreads / 32 - 1) / (kScoreThreads / 32),
                    rows < 65535 ? rows : 65535);
    switch (head_size) {
    case 64: block_scores_kernel<T, 64><<<grid, kScoreThreads, 0, stream>>>(p); break;
    case 128: block_scores_kernel<T, 128><<<grid, kScoreThreads, 0, stream>>>(p); break;
    default: block_scores_kernel<T, 256><<<grid, kScoreThreads, 0, stream>>>(p); break;
    }
}

}  // namespace

cudaError_t launch_select_blocks(const SelectParams& p, int head_size, pa_dtype q_dtype,
                                 cudaStream_t stream) {
    if (p.max_ctx_blocks > p.num_select) {                    // else every block is taken
        switch (q_dtype) {
        case PA_F32: launch_scores<float>(p, head_size, stream); break;
        case PA_F16: launch_scores<__half>(p, head_size, stream); break;
        default: launch_scores<__nv_bfloat16>(p, head_size, stream); break;
        }
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    select_blocks_kernel<<<p.num_seqs * p.num_kv_heads, kSelectThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace pagedkv
