// rope_and_cache.cu -- the KV append with the position rotation applied on the
// way: one pass takes a step's new queries, keys and values from the
// projection to where the attention reads them. Per token t and head row x
// (head_size D, rotated width R <= D):
//   y = x * rsqrt(mean(x^2) + eps) * weight        (only where a weight is given)
//   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin) for the R/2 pairs,
//       pair i = (i, i + R/2) or (2i, 2i + 1), with cos and sin read from the
//       table row of the position that frequency i follows: positions[axis(i)][t];
//   components past R pass through. Queries go to query_out, keys and values
//   to their slot in the cache (same type, or E4M3 codes of x / scale).
// Everything between the load and the one rounding at the store is binary32
// (a 16-bit intermediate between the norm, the rotation and the E4M3
// conversion would round up to three times).
//
// The work is a few flops per byte moved: HBM traffic bounds it for prompts,
// launch and load latency for decode steps. A head row belongs to D / 16
// neighbouring lanes; each holds both partners of eight pairs, as two 16-byte
// vectors (16-bit types), so the rotation needs no exchange between lanes and
// the norm log2(D / 16) shuffles. The lanes read their eight (cos, sin) once
// and use them for every head they take.
#include "device_common.cuh"
#include "kv_store.cuh"
#include "launch.h"

namespace pagedkv {

namespace {

constexpr int kRopeThreads = 256;

// Eight consecutive elements of type T as 16-byte words.
template <typename T>
struct Chunk {
    static constexpr int kWords = 8 * (int)sizeof(T) / 16;   // 1 (16-bit), 2 (binary32)
    uint4 w[kWords];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
    }
    __device__ __forceinline__ void store(T* p) const {
#pragma unroll
        for (int i = 0; i < kWords; ++i) reinterpret_cast<uint4*>(p)[i] = w[i];
    }
    __device__ __forceinline__ void widen(float (&x)[8]) const {
        constexpr int N = Vec16<T>::n;
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            float y[N];
            widen16<T>(w[i], y);
#pragma unroll
            for (int j = 0; j < N; ++j) x[i * N + j] = y[j];
        }
    }
    __device__ __forceinline__ void round_from(const float (&x)[8]) {
        if constexpr (std::is_same<T, float>::value) {
#pragma unroll
            for (int i = 0; i < kWords; ++i)
                w[i] = make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]),
                                  __float_as_uint(x[4 * i + 2]), __float_as_uint(x[4 * i + 3]));
        } else {
            uint32_t u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (std::is_same<T, __half>::value) {
                    const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
                    u[i] = *reinterpret_cast<const uint32_t*>(&h);
                } else {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                    u[i] = *reinterpret_cast<const uint32_t*>(&h);
                }
            }
            w[0] = make_uint4(u[0], u[1], u[2], u[3]);
        }
    }
};

// Eight binary32 values as E4M3 codes of x / scale (the KV write's conversion).
__device__ __forceinline__ void store8_e4m3(uint8_t* dst, const float (&x)[8], float scale) {
    uint32_t packed[2];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float2 q = make_float2(__fdiv_rn(x[i], scale), __fdiv_rn(x[i + 1], scale));
        const uint32_t two = __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
        if ((i & 2) == 0) packed[i / 4] = two;
        else packed[i / 4] |= two << 16;
    }
    *reinterpret_cast<uint2*>(dst) = make_uint2(packed[0], packed[1]);
}

// One head row per D / 16 lanes; a row group takes every `groups`-th of its
// token's Hq + 2 Hkv rows (queries, keys, values), up to kRows of them, with
// all their loads issued before the first is used.
template <typename T, bool kE4M3, int D, int kRows>
__global__ void __launch_bounds__(kRopeThreads)
rope_and_cache_kernel(const __grid_constant__ RopeParams p) {
    constexpr int LANES = D / 16;
    const int lane = threadIdx.x & 31;
    const uint32_t g = (blockIdx.x * (uint32_t)kRopeThreads + threadIdx.x) / LANES;
    const int c = lane & (LANES - 1);
    const uint32_t tl = g / (uint32_t)p.groups;
    if (tl >= (uint32_t)p.num_tokens) return;
    const int64_t t = p.first_token + tl;
    const int h0 = (int)(g - tl * (uint32_t)p.groups);
    const int Hq = p.num_q_heads, Hkv = p.num_kv_heads, H = Hq + 2 * Hkv;
    const int half = p.rotary_dim >> 1;
    const bool rotates = 16 * c < p.rotary_dim;
    // element offsets of the lane's two chunks in a head row
    int a_off = 16 * c, b_off = 16 * c + 8;
    if (!p.adjacent_pairs && rotates) {
        a_off = 8 * c;
        b_off = half + 8 * c;
    }

    Chunk<T> xa[kRows], xb[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int h = h0 + i * p.groups;
        if (h < H) {
            const T* src;
            if (h < Hq) src = static_cast<const T*>(p.query) + t * p.query_stride + (int64_t)h * D;
            else if (h < Hq + Hkv) src = static_cast<const T*>(p.key) + t * p.key_stride + (int64_t)(h - Hq) * D;
            else src = static_cast<const T*>(p.value) + t * p.value_stride + (int64_t)(h - Hq - Hkv) * D;
            xa[i].load(src + a_off);
            xb[i].load(src + b_off);
        }
    }

    const int64_t slot = p.slots[t];
    int64_t pos[4];
    bool ok = true;
#pragma unroll
    for (int a = 0; a < 4; ++a) {
        pos[a] = p.positions[(a < p.num_axes ? a : 0) * p.total_tokens + t];
        ok = ok && pos[a] >= 0 && pos[a] < p.max_position;
    }
    const bool stores = slot >= 0 && slot < p.num_blocks * p.block_size;
    if (h0 == 0 && c == 0 && p.status) {
        if (!ok) atomicOr(p.status, PA_DEV_BAD_POSITION);
        if (slot >= 0 && !stores) atomicOr(p.status, PA_DEV_BAD_SLOT);
    }
    if (!ok) return;                                          // the whole token is skipped

    float cs[8], sn[8];
    if (rotates) {
        const uint32_t axes = p.num_axes == 1 ? 0 : (p.freq_axes[c >> 1] >> (16 * (c & 1))) & 0xffffu;
        const uint32_t a0 = axes & 3;
        if (axes == a0 * 0x5555u) {                           // the eight frequencies follow one axis
            const int64_t q = a0 == 0 ? pos[0] : a0 == 1 ? pos[1] : a0 == 2 ? pos[2] : pos[3];
            const float* row = p.cos_sin + q * p.rotary_dim + 8 * c;
            RowLoader<float, 8>::load(row, cs);
            RowLoader<float, 8>::load(row + half, sn);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t a = (axes >> (2 * j)) & 3;
                const int64_t q = a == 0 ? pos[0] : a == 1 ? pos[1] : a == 2 ? pos[2] : pos[3];
                const float* row = p.cos_sin + q * p.rotary_dim + 8 * c + j;
                cs[j] = row[0];
                sn[j] = row[half];
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) { cs[j] = 1.f; sn[j] = 0.f; }
    }
    size_t cache_row = 0;                                     // row of the token's slot under KV head 0
    if (stores) {
        const int64_t blk = slot / p.block_size;
        cache_row = (size_t)blk * Hkv * p.block_size + (size_t)(slot - blk * p.block_size);
    }
    const uint32_t mask = (uint32_t)((1ull << LANES) - 1) << (lane & ~(LANES - 1));

#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int h = h0 + i * p.groups;
        if (h >= H) break;
        const bool is_q = h < Hq, is_v = h >= Hq + Hkv;
        if (!is_q && !stores) continue;
        const size_t dst = is_q ? (size_t)(t * Hq + h) * D
                                : (cache_row + (size_t)(h - Hq - (is_v ? Hkv : 0)) * p.block_size) * D;
        if (is_v) {
            if constexpr (kE4M3) {
                float x[8];
                uint8_t* v = static_cast<uint8_t*>(p.v_cache) + dst;
                xa[i].widen(x);
                store8_e4m3(v + a_off, x, p.v_scale);
                xb[i].widen(x);
                store8_e4m3(v + b_off, x, p.v_scale);
            } else {
                T* v = static_cast<T*>(p.v_cache) + dst;
                xa[i].store(v + a_off);
                xb[i].store(v + b_off);
            }
            continue;
        }
        float a[8], b[8];
        xa[i].widen(a);
        xb[i].widen(b);
        const float* w = is_q ? p.q_weight : p.k_weight;
        if (w) {
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(a[j], a[j], fmaf(b[j], b[j], ss));
#pragma unroll
            for (int m = LANES / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(mask, ss, m);
            const float r = rsqrtf(ss * (1.f / D) + p.eps);
            float wa[8], wb[8];
            RowLoader<float, 8>::load(w + a_off, wa);
            RowLoader<float, 8>::load(w + b_off, wb);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                a[j] *= r * wa[j];
                b[j] *= r * wb[j];
            }
        }
        if (rotates) {
            if (p.adjacent_pairs) {
                // a and b are 16 neighbouring components: pairs (2j, 2j + 1)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float u = a[2 * j], v = a[2 * j + 1], y = b[2 * j], z = b[2 * j + 1];
                    a[2 * j] = u * cs[j] - v * sn[j];
                    a[2 * j + 1] = v * cs[j] + u * sn[j];
                    b[2 * j] = y * cs[j + 4] - z * sn[j + 4];
                    b[2 * j + 1] = z * cs[j + 4] + y * sn[j + 4];
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float u = a[j], v = b[j];
                    a[j] = u * cs[j] - v * sn[j];
                    b[j] = v * cs[j] + u * sn[j];
                }
            }
        }
        if (!is_q && kE4M3) {
            uint8_t* k = static_cast<uint8_t*>(p.k_cache) + dst;
            store8_e4m3(k + a_off, a, p.k_scale);
            store8_e4m3(k + b_off, b, p.k_scale);
        } else {
            T* y = (is_q ? static_cast<T*>(p.query_out) : static_cast<T*>(p.k_cache)) + dst;
            xa[i].round_from(a);
            xb[i].round_from(b);
            xa[i].store(y + a_off);
            xb[i].store(y + b_off);
        }
    }
}

template <typename T, bool kE4M3, int D, int kRows>
cudaError_t launch_rows(RopeParams p, cudaStream_t stream) {
    constexpr int kPerCta = kRopeThreads / (D / 16);
    p.groups = (p.num_q_heads + 2 * p.num_kv_heads + kRows - 1) / kRows;
    // token ranges whose thread indices stay below 2^31
    int64_t step = (1ll << 30) / ((int64_t)p.groups * (D / 16));
    if (step < 1) step = 1;
    for (int64_t t0 = 0; t0 < p.total_tokens; t0 += step) {
        const int64_t n = p.total_tokens - t0 < step ? p.total_tokens - t0 : step;
        p.first_token = t0;
        p.num_tokens = (int)n;
        const int64_t grid = (n * p.groups + kPerCta - 1) / kPerCta;
        rope_and_cache_kernel<T, kE4M3, D, kRows><<<(unsigned)grid, kRopeThreads, 0, stream>>>(p);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <typename T, bool kE4M3>
cudaError_t launch_rope(const RopeParams& p, int head_size, cudaStream_t stream) {
    switch (head_size) {
    case 64: return launch_rows<T, kE4M3, 64, 1>(p, stream);
    case 128: return launch_rows<T, kE4M3, 128, 1>(p, stream);
    default: return launch_rows<T, kE4M3, 256, 1>(p, stream);
    }
}

}  // namespace

cudaError_t launch_rope_and_cache(const RopeParams& p, int head_size, pa_dtype in_dtype,
                                  pa_dtype cache_dtype, cudaStream_t stream) {
    const bool fp8 = cache_dtype == PA_FP8_E4M3;
    switch (in_dtype) {
    case PA_F32: return fp8 ? launch_rope<float, true>(p, head_size, stream)
                            : launch_rope<float, false>(p, head_size, stream);
    case PA_F16: return fp8 ? launch_rope<__half, true>(p, head_size, stream)
                            : launch_rope<__half, false>(p, head_size, stream);
    default: return fp8 ? launch_rope<__nv_bfloat16, true>(p, head_size, stream)
                        : launch_rope<__nv_bfloat16, false>(p, head_size, stream);
    }
}

}  // namespace pagedkv
