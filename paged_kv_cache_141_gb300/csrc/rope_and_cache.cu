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
constexpr int kSms = 152;
// Warps that an SM holds of each kernel: of the one with a row per lane group,
// and of the one that walks a token's rows, which keeps more in registers.
constexpr int64_t kRowWarps = 24, kTokenWarps = 16;

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

// Eight binary32 values as E4M3 codes of x / scale, the KV write's conversion: an
// IEEE division, then round to nearest even with saturation. The division is
// most of a row's arithmetic, and the code rarely needs it: x * inv (inv =
// 1 / scale, rounded; both roundings move the quotient by less than 2 units in
// its last place) gives the same code unless the quotient lies that close to a
// midpoint of two codes, whose low 20 mantissa bits are 0x80000. Those, and
// quotients below E4M3's normal range (other midpoints), are divided; inv = 0
// (a scale whose reciprocal is out of range) divides all.
__device__ __forceinline__ void store8_e4m3(uint8_t* dst, const float (&x)[8], float scale, float inv) {
    float q[8];
    bool divide = inv == 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        q[i] = __fmul_rn(x[i], inv);
        const uint32_t u = __float_as_uint(q[i]) & 0x7fffffffu;
        divide |= (u & 0xfffffu) - 0x7fffcu <= 8u || (u < 0x3c800000u && u != 0u);         // 2^-6
    }
    if (divide) {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = __fdiv_rn(x[i], scale);
    }
    uint32_t packed[2];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const uint32_t two = __nv_cvt_float2_to_fp8x2(make_float2(q[i], q[i + 1]), __NV_SATFINITE, __NV_E4M3);
        if ((i & 2) == 0) packed[i / 4] = two;
        else packed[i / 4] |= two << 16;
    }
    *reinterpret_cast<uint2*>(dst) = make_uint2(packed[0], packed[1]);
}

// A lane's place in its head row: chunks a and b (eight elements each), and the
// cosines and sines of its eight pairs.
template <typename T, int D>
struct Turn {
    static constexpr int LANES = D / 16;
    int a_off, b_off;
    bool rotates, adjacent;
    uint32_t mask;                                             // the row's lanes
    float cs[8], sn[8];

    __device__ __forceinline__ Turn(const RopeParams& p, int lane) {
        const int c = lane & (LANES - 1);
        rotates = 16 * c < p.rotary_dim;
        adjacent = p.adjacent_pairs;
        a_off = 16 * c;
        b_off = 16 * c + 8;
        if (!adjacent && rotates) {
            a_off = 8 * c;
            b_off = (p.rotary_dim >> 1) + 8 * c;
        }
        mask = (uint32_t)((1ull << LANES) - 1) << (lane & ~(LANES - 1));
    }

    // The token's positions into angles; false: one lies outside the table.
    __device__ __forceinline__ bool load(const RopeParams& p, int64_t t, int lane) {
        const int c = lane & (LANES - 1);
        const int half = p.rotary_dim >> 1;
        int64_t pos[4];
        bool ok = true;
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            pos[a] = p.positions[(a < p.num_axes ? a : 0) * p.total_tokens + t];
            ok = ok && pos[a] >= 0 && pos[a] < p.max_position;
        }
        if (!ok) return false;
        if (!rotates) return true;
        const uint32_t axes = p.num_axes == 1 ? 0 : (p.freq_axes[c >> 1] >> (16 * (c & 1))) & 0xffffu;
        auto row_of = [&](uint32_t a) {                        // table row of axis a, at this lane's frequencies
            return p.cos_sin + (a == 0 ? pos[0] : a == 1 ? pos[1] : a == 2 ? pos[2] : pos[3]) * p.rotary_dim + 8 * c;
        };
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
            const uint32_t four = (axes >> (2 * j)) & 0xffu;
            if (four == (four & 3) * 0x55u) {                  // the four frequencies follow one axis
                const float* row = row_of(four & 3) + j;
                const float4 x = *reinterpret_cast<const float4*>(row);
                const float4 y = *reinterpret_cast<const float4*>(row + half);
                cs[j] = x.x; cs[j + 1] = x.y; cs[j + 2] = x.z; cs[j + 3] = x.w;
                sn[j] = y.x; sn[j + 1] = y.y; sn[j + 2] = y.z; sn[j + 3] = y.w;
            } else {
#pragma unroll
                for (int k = j; k < j + 4; ++k) {
                    const float* row = row_of((axes >> (2 * k)) & 3) + k;
                    cs[k] = row[0];
                    sn[k] = row[half];
                }
            }
        }
        return true;
    }

    __device__ __forceinline__ void norm(float (&a)[8], float (&b)[8], const float (&wa)[8],
                                         const float (&wb)[8], float eps) const {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(a[j], a[j], fmaf(b[j], b[j], ss));
#pragma unroll
        for (int m = LANES / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(mask, ss, m);
        const float r = rsqrtf(ss * (1.f / D) + eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            a[j] *= r * wa[j];
            b[j] *= r * wb[j];
        }
    }

    __device__ __forceinline__ void rotate(float (&a)[8], float (&b)[8]) const {
        if (!rotates) return;
        if (adjacent) {
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
};

// The slot's row under KV head 0 (rows are D elements), or -1: nothing stored.
__device__ __forceinline__ int64_t cache_row(const RopeParams& p, int64_t slot) {
    if (slot < 0 || slot >= p.num_blocks * p.block_size) return -1;
    const int64_t blk = slot / p.block_size;
    return blk * p.num_kv_heads * p.block_size + (slot - blk * p.block_size);
}

__device__ __forceinline__ void flag_token(const RopeParams& p, bool ok, int64_t slot, int64_t row) {
    if (!p.status) return;
    if (!ok) atomicOr(p.status, PA_DEV_BAD_POSITION);
    if (slot >= 0 && row < 0) atomicOr(p.status, PA_DEV_BAD_SLOT);
}

// Decode steps: one head row per D / 16 lanes and nothing more, so that all of
// a step's latencies overlap. Measured: 1 token 2.6 us, 256 tokens of 32/8 heads
// of 128 3.2 us (in a graph): launch and four loads that depend on each other.
template <typename T, bool kE4M3, int D>
__global__ void __launch_bounds__(kRopeThreads)
rope_and_cache_kernel(const __grid_constant__ RopeParams p) {
    begin_overlapped();
    constexpr int LANES = D / 16;
    const int lane = threadIdx.x & 31;
    const uint32_t g = (blockIdx.x * (uint32_t)kRopeThreads + threadIdx.x) / LANES;
    const int Hq = p.num_q_heads, Hkv = p.num_kv_heads;
    const uint32_t H = Hq + 2 * Hkv;
    const uint32_t tl = g / H;
    if (tl >= (uint32_t)p.total_tokens) return;
    const int64_t t = tl;
    const int h = (int)(g - tl * H);
    const bool is_q = h < Hq, is_v = h >= Hq + Hkv;
    Turn<T, D> turn(p, lane);
    const T* src;
    if (is_q) src = static_cast<const T*>(p.query) + t * p.query_stride + (int64_t)h * D;
    else if (!is_v) src = static_cast<const T*>(p.key) + t * p.key_stride + (int64_t)(h - Hq) * D;
    else src = static_cast<const T*>(p.value) + t * p.value_stride + (int64_t)(h - Hq - Hkv) * D;
    Chunk<T> xa, xb;
    xa.load(src + turn.a_off);
    xb.load(src + turn.b_off);
    const float* w = is_v ? nullptr : (is_q ? p.q_weight : p.k_weight);
    float wa[8], wb[8];
    if (w) {
        RowLoader<float, 8>::load(w + turn.a_off, wa);
        RowLoader<float, 8>::load(w + turn.b_off, wb);
    }
    const int64_t slot = p.slots[t];
    const bool ok = turn.load(p, t, lane);
    const int64_t row0 = cache_row(p, slot);
    if (h == 0 && (lane & (LANES - 1)) == 0) flag_token(p, ok, slot, row0);
    if (!ok || (!is_q && row0 < 0)) return;                    // the token, or its store, is skipped
    const size_t dst = is_q ? (size_t)(t * Hq + h) * D
                            : (size_t)(row0 + (int64_t)(h - Hq - (is_v ? Hkv : 0)) * p.block_size) * D;
    if (is_v && !kE4M3) {
        xa.store(static_cast<T*>(p.v_cache) + dst + turn.a_off);
        xb.store(static_cast<T*>(p.v_cache) + dst + turn.b_off);
        return;
    }
    float a[8], b[8];
    xa.widen(a);
    xb.widen(b);
    if (w) turn.norm(a, b, wa, wb, p.eps);
    if (!is_v) turn.rotate(a, b);
    if (!is_q && kE4M3) {
        uint8_t* y = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + dst;
        const float scale = is_v ? p.v_scale : p.k_scale, inv = is_v ? p.v_inv : p.k_inv;
        store8_e4m3(y + turn.a_off, a, scale, inv);
        store8_e4m3(y + turn.b_off, b, scale, inv);
    } else {
        T* y = static_cast<T*>(is_q ? p.query_out : p.k_cache) + dst;
        xa.round_from(a);
        xb.round_from(b);
        xa.store(y + turn.a_off);
        xb.store(y + turn.b_off);
    }
}

// Prompts: a token has 2^group_shift row groups of D / 16 lanes. They take its
// heads in turn, kRows of them with all loads issued before the first is used
// (keys and values together); the first ones of the queries are on their way
// while the token's position becomes angles, which with the weights are loaded
// once for all the rows that a group takes. Measured: 16 x 512 tokens of 32/32
// heads of 128, fp16, 63 us, 6.4 TB/s: bound by memory. 32 x 1001 tokens of 32/8
// heads with norms, bf16, 129 us, 6.2 TB/s: 16 warps per SM (two CTAs of up to 128
// registers a thread) just do not cover the latency.
template <typename T, bool kE4M3, int D, int kRows>
__global__ void __launch_bounds__(kRopeThreads, 2)
rope_and_cache_prompt_kernel(const __grid_constant__ RopeParams p) {
    begin_overlapped();
    constexpr int LANES = D / 16;
    const int lane = threadIdx.x & 31;
    const int groups = 1 << p.group_shift;
    const int64_t g = ((int64_t)blockIdx.x * kRopeThreads + threadIdx.x) / LANES;
    const int64_t t = g >> p.group_shift;
    const int grp = (int)g & (groups - 1);
    if (t >= p.total_tokens) return;
    const int Hq = p.num_q_heads, Hkv = p.num_kv_heads, B = p.block_size;
    Turn<T, D> turn(p, lane);
    Chunk<T> xa[kRows], xb[kRows];
    // rows h0, h0 + groups, ... of the token: of its queries, or of its keys (the
    // first Hkv) and values
    const T* query = static_cast<const T*>(p.query) + t * p.query_stride;
    const T* key = static_cast<const T*>(p.key) + t * p.key_stride;
    const T* value = static_cast<const T*>(p.value) + t * p.value_stride;
    auto load_queries = [&](int h0) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int h = h0 + i * groups;
            if (h < Hq) {
                xa[i].load(query + h * D + turn.a_off);
                xb[i].load(query + h * D + turn.b_off);
            }
        }
    };
    auto load_keys_values = [&](int h0) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int h = h0 + i * groups;
            if (h < 2 * Hkv) {
                const T* src = h < Hkv ? key + h * D : value + (h - Hkv) * D;
                xa[i].load(src + turn.a_off);
                xb[i].load(src + turn.b_off);
            }
        }
    };
    load_queries(grp);
    const int64_t slot = p.slots[t];
    const bool ok = turn.load(p, t, lane);
    const int64_t row0 = cache_row(p, slot);
    if (grp == 0 && (lane & (LANES - 1)) == 0) flag_token(p, ok, slot, row0);
    if (!ok) return;

    float wa[8], wb[8];
    auto load_weights = [&](const float* w) {
        if (w) {
            RowLoader<float, 8>::load(w + turn.a_off, wa);
            RowLoader<float, 8>::load(w + turn.b_off, wb);
        }
    };
    load_weights(p.q_weight);
    T* q_out = static_cast<T*>(p.query_out) + (size_t)t * Hq * D;
    for (int h0 = grp; h0 < Hq; h0 += kRows * groups) {
        if (h0 != grp) load_queries(h0);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int h = h0 + i * groups;
            if (h >= Hq) break;
            float a[8], b[8];
            xa[i].widen(a);
            xb[i].widen(b);
            if (p.q_weight) turn.norm(a, b, wa, wb, p.eps);
            turn.rotate(a, b);
            xa[i].round_from(a);
            xb[i].round_from(b);
            xa[i].store(q_out + h * D + turn.a_off);
            xb[i].store(q_out + h * D + turn.b_off);
        }
    }
    if (row0 < 0) return;
    load_weights(p.k_weight);
    const size_t cell0 = (size_t)row0 * D, step = (size_t)B * D;           // elements of the caches
    for (int h0 = grp; h0 < 2 * Hkv; h0 += kRows * groups) {
        load_keys_values(h0);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int h = h0 + i * groups;
            if (h >= 2 * Hkv) break;
            const bool is_v = h >= Hkv;
            const size_t dst = cell0 + (is_v ? h - Hkv : h) * step;
            void* cache = is_v ? p.v_cache : p.k_cache;
            float a[8], b[8];
            if (kE4M3 || !is_v) {
                xa[i].widen(a);
                xb[i].widen(b);
            }
            if (!is_v) {
                if (p.k_weight) turn.norm(a, b, wa, wb, p.eps);
                turn.rotate(a, b);
            }
            if constexpr (kE4M3) {
                uint8_t* y = static_cast<uint8_t*>(cache) + dst;
                const float scale = is_v ? p.v_scale : p.k_scale, inv = is_v ? p.v_inv : p.k_inv;
                store8_e4m3(y + turn.a_off, a, scale, inv);
                store8_e4m3(y + turn.b_off, b, scale, inv);
            } else {
                if (!is_v) {
                    xa[i].round_from(a);
                    xb[i].round_from(b);
                }
                T* y = static_cast<T*>(cache) + dst;
                xa[i].store(y + turn.a_off);
                xb[i].store(y + turn.b_off);
            }
        }
    }
}

// The row groups of a token that make the call shortest: its time goes as the
// waves of warps on the device times the batches of kRows rows that each warp
// walks through, so few tokens want many groups and many tokens the count that
// divides both evenly; of equals the fewest, which load the angles least often.
// Measured with 1, 2, 4 and 8 groups (bf16, 32/8 heads of 128 with norms): 700
// tokens 19.5, 11.0, 6.9, 4.6 us, 3000 tokens 26.6, 18.5, 19.0 us, 32032 tokens
// 134, 129, 133 us; with 8/1 heads 32032 tokens take 31, 36 and 50 us.
inline int row_group_shift(const RopeParams& p, int lanes, int rows) {
    int best_shift = 0;
    int64_t best = INT64_MAX;
    for (int shift = 0; shift <= 5; ++shift) {
        const int64_t warps = ((p.total_tokens << shift) * lanes + 31) / 32;
        const int64_t waves = (warps + kSms * kTokenWarps - 1) / (kSms * kTokenWarps);
        const int64_t taken = (int64_t)rows << shift;
        const int64_t batches = (p.num_q_heads + taken - 1) / taken + (2 * (int64_t)p.num_kv_heads + taken - 1) / taken;
        if (waves * batches < best) {
            best = waves * batches;
            best_shift = shift;
        }
    }
    return best_shift;
}

template <typename T, bool kE4M3, int D>
cudaError_t launch_head_size(const RopeParams& p, cudaStream_t stream) {
    const int64_t H = p.num_q_heads + 2 * (int64_t)p.num_kv_heads;
    constexpr int LANES = D / 16;
    // A row per lane group while all of them are resident at once: 300 tokens of
    // 48 rows of 128 with norms take 3.6 us so and 3.9 in row groups, 600 tokens
    // 5.9 and 4.5 (MHA without norms: 128 tokens of 96 rows 3.2 and 3.2, 300 5.0
    // and 3.9).
    if (p.total_tokens * H * LANES <= kSms * kRowWarps * 32) {
        const int64_t grid = (p.total_tokens * H * LANES + kRopeThreads - 1) / kRopeThreads;
        return launch_overlapped(rope_and_cache_kernel<T, kE4M3, D>, p, dim3((unsigned)grid), kRopeThreads, 0,
                                 stream);
    }
    constexpr int kRows = sizeof(T) == 4 ? 2 : 4;
    RopeParams q = p;
    q.group_shift = row_group_shift(p, LANES, kRows);
    const int64_t grid = ((p.total_tokens << q.group_shift) * LANES + kRopeThreads - 1) / kRopeThreads;
    if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    return launch_overlapped(rope_and_cache_prompt_kernel<T, kE4M3, D, kRows>, q, dim3((unsigned)grid),
                             kRopeThreads, 0, stream);
}

template <typename T, bool kE4M3>
cudaError_t launch_rope(const RopeParams& p, int head_size, cudaStream_t stream) {
    switch (head_size) {
    case 64: return launch_head_size<T, kE4M3, 64>(p, stream);
    case 128: return launch_head_size<T, kE4M3, 128>(p, stream);
    default: return launch_head_size<T, kE4M3, 256>(p, stream);
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
