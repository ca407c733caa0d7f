// key_bounds.cu -- the summaries that the block-sparse decode scores: for a
// cache block and KV head the elementwise minimum and maximum of its keys,
//     lo_d = min_t k[t][d],   hi_d = max_t k[t][d]
// over the block's tokens below the sequence's length. A step changes only
// the blocks that hold its new tokens, so those are recomputed from the cache
// (whole blocks: no state carries over from earlier calls, and a repeated or
// replayed call gives the same bounds).
//
// One warp per (sequence, touched block, KV head): D / 8 lanes hold a token's
// row, eight elements each, and the warp's 256 / D lane groups take
// alternate tokens. Comparisons are exact, so the order of tokens does not
// matter; a NaN key makes both of its component's bounds NaN. E4M3 codes
// widen exactly to binary16 and from there to bfloat16. Bound by reading the
// keys once (bandwidth), or by launch and load latency for a decode step.
#include "device_common.cuh"
#include "launch.h"

namespace pagedkv {

namespace {

constexpr int kBoundsThreads = 128;

__device__ __forceinline__ float nan_min(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float nan_max(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

template <typename CT, typename BT, int D>
__global__ void __launch_bounds__(kBoundsThreads)
key_bounds_kernel(const __grid_constant__ BoundsParams p) {
    constexpr int LANES = D / 8;               // lanes per token row
    constexpr int ROWS = 32 / LANES;           // token rows per step of the warp
    const int lane = threadIdx.x & 31;
    const int64_t unit = ((int64_t)blockIdx.x * kBoundsThreads + threadIdx.x) >> 5;
    const int64_t sj = unit / p.num_kv_heads;
    const int h = (int)(unit - sj * p.num_kv_heads);
    const int s = (int)(sj / p.touched);
    if (s >= p.num_seqs) return;
    const int B = p.block_size;
    const int L = p.context_lens[s];
    const int n = p.new_tokens ? p.new_tokens[s] : (L > 0 ? 1 : 0);
    const int64_t tab = (int64_t)p.max_blocks * B;
    if (L < 0 || L > p.max_context_len || L > tab || n < 0 || n > L || n > p.max_new_tokens) {
        if (lane == 0 && p.status) atomicOr(p.status, PA_DEV_BAD_LEN);
        return;
    }
    if (n == 0) return;
    const int j = (L - n) / B + (int)(sj - (int64_t)s * p.touched);
    if ((int64_t)j * B >= L) return;
    const int64_t blk = p.block_tables[(size_t)s * p.max_blocks + j];
    if (blk < 0 || blk >= p.num_blocks) {
        if (lane == 0 && p.status) atomicOr(p.status, PA_DEV_BAD_BLOCK_ID);
        return;
    }
    const int tokens = min(B, L - j * B);
    const int c = (lane & (LANES - 1)) * 8;
    const size_t slab = (size_t)blk * p.num_kv_heads + h;
    const CT* keys = static_cast<const CT*>(p.k_cache) + slab * B * D + c;
    float lo[8], hi[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo[i] = __int_as_float(0x7f800000);
        hi[i] = __int_as_float(0xff800000);
    }
#pragma unroll 4
    for (int r = lane / LANES; r < tokens; r += ROWS) {
        float x[8];
        RowLoader<CT, 8>::load(keys + (size_t)r * D, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo[i] = nan_min(lo[i], x[i]);
            hi[i] = nan_max(hi[i], x[i]);
        }
    }
#pragma unroll
    for (int m = LANES; m < 32; m <<= 1) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo[i] = nan_min(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], m));
            hi[i] = nan_max(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], m));
        }
    }
    // the values are the cache's own, so the conversions below are exact
    if (lane < 2 * LANES || ROWS == 1) {
        BT* out = static_cast<BT*>(p.k_bounds) + slab * 2 * D + c;
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            if (ROWS > 1 && side != lane / LANES) continue;
#pragma unroll
            for (int i = 0; i < 8; ++i) out[side * D + i] = from_float<BT>(side ? hi[i] : lo[i]);
        }
    }
}

template <typename CT, typename BT>
cudaError_t launch_bounds(const BoundsParams& p, int head_size, cudaStream_t stream) {
    const int64_t units = (int64_t)p.num_seqs * p.touched * p.num_kv_heads;
    const int64_t grid = (units * 32 + kBoundsThreads - 1) / kBoundsThreads;
    if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    switch (head_size) {
    case 64: key_bounds_kernel<CT, BT, 64><<<(unsigned)grid, kBoundsThreads, 0, stream>>>(p); break;
    case 128: key_bounds_kernel<CT, BT, 128><<<(unsigned)grid, kBoundsThreads, 0, stream>>>(p); break;
    default: key_bounds_kernel<CT, BT, 256><<<(unsigned)grid, kBoundsThreads, 0, stream>>>(p); break;
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_key_bounds(const BoundsParams& p, int head_size, pa_dtype cache_dtype,
                              pa_dtype bounds_dtype, cudaStream_t stream) {
    if (cache_dtype == PA_FP8_E4M3)
        return bounds_dtype == PA_F16 ? launch_bounds<e4m3_t, __half>(p, head_size, stream)
                                      : launch_bounds<e4m3_t, __nv_bfloat16>(p, head_size, stream);
    switch (cache_dtype) {
    case PA_F32: return launch_bounds<float, float>(p, head_size, stream);
    case PA_F16: return launch_bounds<__half, __half>(p, head_size, stream);
    default: return launch_bounds<__nv_bfloat16, __nv_bfloat16>(p, head_size, stream);
    }
}

}  // namespace pagedkv
