// scaled_append.cu -- the KV write into a cache of 8-bit codes with a scale for
// each (block, KV head). For a block that receives new rows x of a head:
//     fresh = max |x| / 127                            (8-bit integers)
//           = the least power of two with max |x| <= 448 fresh      (E4M3)
//     scale' = max(scale, fresh) where the block holds older tokens, else fresh,
// never below 2^-96; codes of new rows are x / scale' rounded to nearest even, and
// where the scale has grown the older tokens' codes c become c scale / scale',
// rounded alike. (A code's error stays within half a step of the final scale for each
// growth. E4M3's steps are relative: powers of two cost no precision, and a growth
// moves exponents, exact but for codes that become subnormal.) A NaN or an
// infinity among the new rows makes the block's scale NaN, and everything that
// is read through it.
//
// One warp per (sequence, touched block, KV head, K or V). A row's lanes hold 16
// bytes each (32 for binary32 at head size 256) and the warp's lane groups take alternate rows;
// the block's new rows stay in registers between the maximum and the codes (up to
// kPasses rows of each group; further ones are read again, from L1). The new rows
// are read once and the codes written once: HBM-bound for prompts (32 chunks of 1,001 tokens,
// 8 heads of 128, bfloat16 to E4M3: 32.7 us, 6.0 TB/s, 43.6 with rows widened in registers and
// the block's id loaded before its rows), launch and two dependent loads for decode steps (128
// tokens 3.5 us).
#include "device_common.cuh"
#include "kv_store.cuh"
#include "launch.h"

namespace pagedkv {

namespace {

constexpr int kAppendThreads = 128;
constexpr float kLeastScale = 0x1p-96f;

struct Int8Codes {
    static constexpr bool kInt = true;
};
struct E4m3Codes {
    static constexpr bool kInt = false;
};

template <typename QT, int D>
struct AppendShape {
    static constexpr int V = 16 / (int)sizeof(QT);                 // elements of a 16-byte vector
    static constexpr int E = D / V > 32 ? 2 * V : V;               // elements of a lane
    static constexpr int LANES = D / E;                            // lanes of a row
    static constexpr int ROWS = 32 / LANES;                        // rows at a time
    static constexpr int kPasses = E * (int)sizeof(QT) > 16 ? 8 : (ROWS == 1 ? 16 : 8);   // of them in registers
};

// A lane's E elements of a row as they lie, and widened.
template <typename QT, int E>
struct RowBits {
    uint4 w[E * sizeof(QT) / 16];
    __device__ __forceinline__ void load(const QT* p) {
#pragma unroll
        for (int i = 0; i < (int)(E * sizeof(QT) / 16); ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < (int)(E * sizeof(QT) / 16); ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void widen(float (&x)[E]) const {
        constexpr int V = 16 / (int)sizeof(QT);
#pragma unroll
        for (int i = 0; i < E / V; ++i) {
            float y[V];
            widen16<QT>(w[i], y);
#pragma unroll
            for (int k = 0; k < V; ++k) x[i * V + k] = y[k];
        }
    }
    // The largest magnitude's bits, of `m` too: magnitudes order as integers, infinities
    // and NaN above all others (16-bit types: two at a time).
    __device__ __forceinline__ uint32_t largest(uint32_t m) const {
#pragma unroll
        for (int i = 0; i < (int)(E * sizeof(QT) / 16); ++i) {
            const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
                m = sizeof(QT) == 2 ? __vmaxu2(m, v[k] & 0x7fff7fffu) : max(m, v[k] & 0x7fffffffu);
        }
        return m;
    }
    // That magnitude in binary32, of the whole warp.
    __device__ __forceinline__ static float magnitude(uint32_t m) {
        if constexpr (sizeof(QT) == 2) m = max(m & 0xffffu, m >> 16);
        m = __reduce_max_sync(0xffffffffu, m);
        if constexpr (std::is_same<QT, float>::value) return __uint_as_float(m);
        else if constexpr (std::is_same<QT, __half>::value) return __half2float(__ushort_as_half((unsigned short)m));
        else return __uint_as_float(m << 16);
    }
};

template <bool kInt>
__device__ __forceinline__ float fresh_scale(float most) {
    if (!(most < INFINITY)) return NAN;
    if (kInt) return fmaxf(__fdiv_rn(most, 127.f), kLeastScale);
    // 448 = 1.75 * 2^8: the exponent of `most`, one more where its significand is above 1.75
    const uint32_t bits = __float_as_uint(most);
    const int e = (int)(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u);
    return most > 0.f && e > 127 - 96 ? __uint_as_float((uint32_t)e << 23) : kLeastScale;
}

// x / scale to the nearest integer: by the reciprocal, whose product is within 2^-15 of
// the quotient (|quotient| <= 127.5), and by a division where that leaves a doubt.
__device__ __forceinline__ int quotient(float x, float scale, float inv) {
    float y = x * inv;
    if (!(fabsf(fabsf(y - rintf(y)) - 0.5f) > 0x1p-14f)) y = __fdiv_rn(x, scale);
    return min(127, max(-127, __float2int_rn(y)));
}

// E codes of x / scale, packed in bytes. `inv`: 1 / scale, exact for powers of two.
template <bool kInt, int E>
__device__ __forceinline__ void encode(const float (&x)[E], float scale, float inv, uint32_t (&w)[E / 4]) {
#pragma unroll
    for (int i = 0; i < E; i += 4) {
        if constexpr (kInt) {
            uint32_t r = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                r |= (uint32_t)(quotient(x[i + j], scale, inv) & 0xff) << (8 * j);
            }
            w[i / 4] = r;
        } else {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[i] * inv, x[i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[i + 2] * inv, x[i + 3] * inv), __NV_SATFINITE, __NV_E4M3);
            w[i / 4] = lo | hi << 16;
        }
    }
}

// The same codes under another scale.
template <bool kInt>
__device__ __forceinline__ uint32_t recode(uint32_t w, float ratio) {
    uint32_t r = 0;
    if constexpr (kInt) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float c = (float)(int8_t)(w >> (8 * j));
            r |= (uint32_t)(__float2int_rn(c * ratio) & 0xff) << (8 * j);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
            float2 f = e4m3x2_to_float2((uint16_t)(w >> (8 * j)));
            f.x *= ratio;
            f.y *= ratio;
            r |= (uint32_t)__nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3) << (8 * j);
        }
    }
    return r;
}

template <int N>
__device__ __forceinline__ void store_words(uint8_t* p, const uint32_t (&w)[N]) {
    if constexpr (N == 1) *reinterpret_cast<uint32_t*>(p) = w[0];
    else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

template <typename QT, bool kInt, int D>
__global__ void __launch_bounds__(kAppendThreads)
scaled_append_kernel(const __grid_constant__ ScaledAppendParams p) {
    begin_overlapped();
    using A = AppendShape<QT, D>;
    constexpr int E = A::E, ROWS = A::ROWS, P = A::kPasses;
    const int lane = threadIdx.x & 31;
    const uint32_t unit = (blockIdx.x * kAppendThreads + threadIdx.x) >> 5;
    const uint32_t heads = 2u * p.num_kv_heads;
    const uint32_t nth = unit / heads;                             // of the touched blocks
    if (nth >= (uint32_t)p.touched) return;
    const int hk = (int)(unit - nth * heads);
    const bool is_v = hk >= p.num_kv_heads;
    const int h = is_v ? hk - p.num_kv_heads : hk;
    const int s = blockIdx.y;
    const int B = p.block_size;
    const int L = p.context_lens[s];
    int64_t row0 = s, n = L > 0 ? 1 : 0;
    if (p.query_start) {
        row0 = p.query_start[s];
        n = p.query_start[s + 1] - row0;
    }
    if (L < 0 || L > (int64_t)p.max_blocks * B || n < 0 || n > L || n > p.max_new_tokens || row0 < 0 ||
        row0 + n > p.num_tokens) {
        if (lane == 0 && p.status) atomicOr(p.status, PA_DEV_BAD_LEN);
        return;
    }
    if (n == 0) return;
    const int start = L - (int)n;                                  // the first new position
    const int64_t j = start / B + (int64_t)nth;
    if (j * B >= L) return;
    // the block's id and its new rows load together
    const int64_t blk = p.block_tables[(size_t)s * p.max_blocks + j];
    const int base = (int)(j * B);
    const int lo = max(start - base, 0), hi = min(L - base, B);    // the new rows of the block
    const int64_t stride = is_v ? p.value_stride : p.key_stride;
    const QT* src = static_cast<const QT*>(is_v ? p.value : p.key) + (row0 + base - start) * stride + (size_t)h * D;
    const int r0 = lane / A::LANES, e0 = (lane % A::LANES) * E;
    RowBits<QT, E> x[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int r = lo + i * ROWS + r0;
        if (r < hi) x[i].load(src + r * stride + e0);
        else x[i].clear();
    }
    if (blk < 0 || blk >= p.num_blocks) {
        if (lane == 0 && p.status) atomicOr(p.status, PA_DEV_BAD_BLOCK_ID);
        return;
    }
    const size_t slab = (size_t)blk * p.num_kv_heads + h;
    float* scales = (is_v ? p.v_scales : p.k_scales) + slab;
    const float before = lo > 0 ? *scales : 0.f;
    uint8_t* dst = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + slab * B * D;
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) bits = x[i].largest(bits);
    for (int r = lo + P * ROWS + r0; r < hi; r += ROWS) {
        RowBits<QT, E> y;
        y.load(src + r * stride + e0);
        bits = y.largest(bits);
    }
    const float most = RowBits<QT, E>::magnitude(bits);
    float scale = fresh_scale<kInt>(most);
    if (lo > 0) {
        float t;
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(t) : "f"(before), "f"(scale));
        scale = t;
        if (scale != before) {
            const float ratio = __fdiv_rn(before, scale);
            for (int r = r0; r < lo; r += ROWS) {
                uint32_t* w = reinterpret_cast<uint32_t*>(dst + (size_t)r * D + e0);
#pragma unroll
                for (int k = 0; k < E / 4; ++k) w[k] = recode<kInt>(w[k], ratio);
            }
        }
    }
    const float inv = __fdiv_rn(1.f, scale);
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int r = lo + i * ROWS + r0;
        if (r < hi) {
            float v[E];
            x[i].widen(v);
            uint32_t w[E / 4];
            encode<kInt, E>(v, scale, inv, w);
            store_words(dst + (size_t)r * D + e0, w);
        }
    }
    for (int r = lo + P * ROWS + r0; r < hi; r += ROWS) {
        RowBits<QT, E> y;
        y.load(src + r * stride + e0);
        float v[E];
        y.widen(v);
        uint32_t w[E / 4];
        encode<kInt, E>(v, scale, inv, w);
        store_words(dst + (size_t)r * D + e0, w);
    }
    if (lane == 0) *scales = scale;
}

template <typename QT, bool kInt>
cudaError_t launch_typed(const ScaledAppendParams& p, int head_size, cudaStream_t stream) {
    const uint64_t warps = (uint64_t)p.touched * 2 * p.num_kv_heads;
    const dim3 grid((unsigned)((warps * 32 + kAppendThreads - 1) / kAppendThreads), p.num_seqs);
    switch (head_size) {
    case 64: return launch_overlapped(scaled_append_kernel<QT, kInt, 64>, p, grid, kAppendThreads, 0, stream);
    case 128: return launch_overlapped(scaled_append_kernel<QT, kInt, 128>, p, grid, kAppendThreads, 0, stream);
    case 256: return launch_overlapped(scaled_append_kernel<QT, kInt, 256>, p, grid, kAppendThreads, 0, stream);
    }
    return cudaErrorInvalidValue;
}

template <typename QT>
cudaError_t launch_type(const ScaledAppendParams& p, int head_size, pa_dtype cache_dtype, cudaStream_t stream) {
    return cache_dtype == PA_INT8 ? launch_typed<QT, true>(p, head_size, stream)
                                  : launch_typed<QT, false>(p, head_size, stream);
}

}  // namespace

cudaError_t launch_scaled_append(const ScaledAppendParams& p, int head_size, pa_dtype in_dtype,
                                 pa_dtype cache_dtype, cudaStream_t stream) {
    switch (in_dtype) {
    case PA_F32: return launch_type<float>(p, head_size, cache_dtype, stream);
    case PA_F16: return launch_type<__half>(p, head_size, cache_dtype, stream);
    default: return launch_type<__nv_bfloat16>(p, head_size, cache_dtype, stream);
    }
}

}  // namespace pagedkv
