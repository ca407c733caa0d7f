// key_bounds.cu -- the summaries that the block-sparse decode scores: for a
// cache block and KV head the elementwise minimum and maximum of its keys,
//     lo_d = min_t k[t][d],   hi_d = max_t k[t][d]
// over the block's tokens below the sequence's length. A step changes only
// the blocks that hold its new tokens, so those are recomputed from the cache
// (whole blocks: no state carries over from earlier calls, and a repeated or
// replayed call gives the same bounds).
//
// One warp per (sequence, touched block, KV head). A row's lanes hold 16 bytes
// each (32 for binary32) and the warp's lane groups take alternate tokens, four
// loads of each in flight; the comparisons run on packed 16-bit pairs, E4M3
// codes widened to binary16 (exactly). Across the groups, one half of the warp
// reduces the minima and the other the maxima. Comparisons are exact, so the
// order of tokens does not matter; a NaN key makes both of its component's
// bounds NaN. Measured (8 heads of 128): 32 chunks of 1000 E4M3 tokens 12 us, 3.4 TB/s:
// each pair of codes is converted before it is compared, and four loads a lane do
// not cover the latency beside that (issue slots 59 % used). The same in bf16 17 us,
// 4.4 TB/s, in binary32 26 us, 5.8 TB/s. The newest block of 64 sequences 3.2 us, launch
// and load latency.
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

// This warp's block of sequence s (grid x: touched blocks and heads, y:
// sequences): the slab (block * Hkv + head) and the tokens it holds, 0 where
// there is nothing to do.
__device__ __forceinline__ int bounds_unit(const BoundsParams& p, int s, int lane, size_t& slab) {
    const uint32_t unit = (blockIdx.x * kBoundsThreads + threadIdx.x) >> 5;
    const uint32_t nth = unit / (uint32_t)p.num_kv_heads;     // of the touched blocks
    const int h = (int)(unit - nth * p.num_kv_heads);
    if (nth >= (uint32_t)p.touched) return 0;
    const int B = p.block_size;
    const int L = p.context_lens[s];
    const int n = p.new_tokens ? p.new_tokens[s] : (L > 0 ? 1 : 0);
    const int64_t tab = (int64_t)p.max_blocks * B;
    if (L < 0 || L > p.max_context_len || L > tab || n < 0 || n > L || n > p.max_new_tokens) {
        if (lane == 0 && p.status) atomicOr(p.status, PA_DEV_BAD_LEN);
        return 0;
    }
    if (n == 0) return 0;
    const int j = (L - n) / B + (int)nth;                     // below 2^31: touched blocks end by L + B
    if ((int64_t)j * B >= L) return 0;
    const int64_t blk = p.block_tables[(size_t)s * p.max_blocks + j];
    if (blk < 0 || blk >= p.num_blocks) {
        if (lane == 0 && p.status) atomicOr(p.status, PA_DEV_BAD_BLOCK_ID);
        return 0;
    }
    slab = (size_t)blk * p.num_kv_heads + h;
    return min(B, L - j * B);
}

// Packed pairs of a 16-bit type: the cache's own, or binary16 for E4M3 codes.
template <typename CT> struct Pairs { using T2 = __half2; };
template <> struct Pairs<__nv_bfloat16> { using T2 = __nv_bfloat162; };

template <typename CT, typename BT, int D>
__global__ void __launch_bounds__(kBoundsThreads)
key_bounds_kernel(const __grid_constant__ BoundsParams p) {
    begin_overlapped();
    constexpr bool kFp8 = std::is_same<CT, e4m3_t>::value;
    using T2 = typename Pairs<CT>::T2;
    constexpr int E = 16 / (int)sizeof(CT);    // elements per lane
    constexpr int W = E / 2;                   // pairs per lane
    constexpr int LANES = D / E;               // lanes per token row
    constexpr int ROWS = 32 / LANES;           // token rows per step of the warp
    constexpr int kBatch = 4;
    const int lane = threadIdx.x & 31;
    for (int s = blockIdx.y; s < p.num_seqs; s += gridDim.y) {
        size_t slab = 0;
        const int tokens = bounds_unit(p, s, lane, slab);
        if (tokens == 0) continue;
        const int c = (lane & (LANES - 1)) * E;
        const CT* keys = static_cast<const CT*>(p.k_cache) + slab * p.block_size * D + c;
        auto as2 = [](uint32_t w) { return *reinterpret_cast<T2*>(&w); };
        auto bits = [](T2 x) { return *reinterpret_cast<uint32_t*>(&x); };
        T2 lo[W], hi[W];
        const int r0 = lane / LANES;
        // a lane group without a token of its own starts from the first token too
        for (int r = 0; r < tokens; r += kBatch * ROWS) {
            uint4 x[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int t = r + k * ROWS + r0;
                x[k] = *reinterpret_cast<const uint4*>(keys + (t < tokens ? t : 0) * D);
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const uint32_t ws[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    T2 v;
                    if constexpr (kFp8) {
                        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
                            static_cast<__nv_fp8x2_storage_t>(ws[i / 2] >> (16 * (i & 1)) & 0xffffu), __NV_E4M3);
                        v = *reinterpret_cast<const T2*>(&h);
                    } else {
                        v = as2(ws[i]);
                    }
                    lo[i] = r == 0 && k == 0 ? v : __hmin2_nan(lo[i], v);
                    hi[i] = r == 0 && k == 0 ? v : __hmax2_nan(hi[i], v);
                }
            }
        }
        auto store = [&](BT* out, const T2 (&v)[W]) {
            uint32_t w[W];
#pragma unroll
            for (int i = 0; i < W; ++i) {
                if constexpr (kFp8 && std::is_same<BT, __nv_bfloat16>::value) {
                    const __nv_bfloat162 b = __float22bfloat162_rn(__half22float2(v[i]));      // exact
                    w[i] = *reinterpret_cast<const uint32_t*>(&b);
                } else {
                    w[i] = bits(v[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < W; i += 4)
                *reinterpret_cast<uint4*>(out + 2 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
        };
        BT* out = static_cast<BT*>(p.k_bounds) + slab * 2 * D + c;
        if constexpr (ROWS == 1) {
            store(out, lo);
            store(out + D, hi);
        } else {
            // lanes 0-15 go on with the minima, 16-31 with the maxima
            const bool upper = lane >= 16;
            T2 v[W];
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const T2 o = as2(__shfl_xor_sync(0xffffffffu, bits(upper ? lo[i] : hi[i]), 16));
                v[i] = upper ? __hmax2_nan(hi[i], o) : __hmin2_nan(lo[i], o);
#pragma unroll
                for (int m = 8; m >= LANES; m >>= 1) {
                    const T2 y = as2(__shfl_xor_sync(0xffffffffu, bits(v[i]), m));
                    v[i] = upper ? __hmax2_nan(v[i], y) : __hmin2_nan(v[i], y);
                }
            }
            if ((lane & 15) < LANES) store(out + (upper ? D : 0), v);
        }
    }
}

// Binary32 caches: eight elements per lane.
template <int D>
__global__ void __launch_bounds__(kBoundsThreads)
key_bounds_f32_kernel(const __grid_constant__ BoundsParams p) {
    begin_overlapped();
    constexpr int LANES = D / 8;               // lanes per token row
    constexpr int ROWS = 32 / LANES;           // token rows per step of the warp
    const int lane = threadIdx.x & 31;
    for (int s = blockIdx.y; s < p.num_seqs; s += gridDim.y) {
        size_t slab = 0;
        const int tokens = bounds_unit(p, s, lane, slab);
        if (tokens == 0) continue;
        const int c = (lane & (LANES - 1)) * 8;
        const float* keys = static_cast<const float*>(p.k_cache) + slab * p.block_size * D + c;
        float lo[8], hi[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo[i] = __int_as_float(0x7f800000);
            hi[i] = __int_as_float(0xff800000);
        }
#pragma unroll 4
        for (int r = lane / LANES; r < tokens; r += ROWS) {
            float x[8];
            RowLoader<float, 8>::load(keys + (size_t)r * D, x);
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
        if (lane < LANES) {
            float* out = static_cast<float*>(p.k_bounds) + slab * 2 * D + c;
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
                *reinterpret_cast<float4*>(out + i) = make_float4(lo[i], lo[i + 1], lo[i + 2], lo[i + 3]);
                *reinterpret_cast<float4*>(out + D + i) = make_float4(hi[i], hi[i + 1], hi[i + 2], hi[i + 3]);
            }
        }
    }
}

template <typename CT, typename BT>
cudaError_t launch_bounds(const BoundsParams& p, int head_size, cudaStream_t stream) {
    const int64_t units = (int64_t)p.touched * p.num_kv_heads;         // kMaxBoundsUnits at most
    const int64_t gx = (units * 32 + kBoundsThreads - 1) / kBoundsThreads;
    const dim3 grid((unsigned)gx, p.num_seqs < 65535 ? p.num_seqs : 65535);
    auto launch = [&](void (*kernel)(BoundsParams)) {
        return launch_overlapped(kernel, p, grid, kBoundsThreads, 0, stream);
    };
    if constexpr (std::is_same<CT, float>::value) {
        switch (head_size) {
        case 64: return launch(key_bounds_f32_kernel<64>);
        case 128: return launch(key_bounds_f32_kernel<128>);
        default: return launch(key_bounds_f32_kernel<256>);
        }
    } else {
        switch (head_size) {
        case 64: return launch(key_bounds_kernel<CT, BT, 64>);
        case 128: return launch(key_bounds_kernel<CT, BT, 128>);
        default: return launch(key_bounds_kernel<CT, BT, 256>);
        }
    }
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
