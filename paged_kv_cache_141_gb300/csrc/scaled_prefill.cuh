// scaled_prefill.cuh -- attention over block-scaled 8-bit codes for many query rows
// (prompt chunks, large groups' drafts) on the 5th-generation tensor cores.
//
// Work unit: (sequence, KV head, two tiles of 128 query rows, partition of the
// context), one CTA on an SM. Rows are (query token, head of the group) pairs,
// token-major, as in scaled_attention.cuh, whose definitions hold here. Key tiles of
// 128. Roles:
//   warps 0-3, 4-7   softmax of query tile 0, 1: a thread a row;
//   warp 9           issues tcgen05.mma (one lane), tiles interleaved: S0, S1, then
//                    PV0, S0', PV1, S1', ...
//   warps 8, 10, 12  load K: codes from the cache's blocks into registers, a slice of
//   and 11, 13, 15   32 keys ahead (V: the other three), widened to binary16 -- exactly,
//                    as in scaled_attention.cuh -- into the swizzled tiles that the MMAs read.
// The codes go through registers and not through shared memory: binary16 tiles and queries
// take all of it, and the widening needs the registers anyway.
//
// The scales stay out of the tiles. Blocks are multiples of 16 tokens here, so a
// group of 16 columns of S has one key scale a and one value scale b: with raw
// scores s and the row's unit u (scale, log2 e and the query's power of two),
//     weight = 2^(s (u a) + (log2 b - e + 6) - m),
// one fused multiply-add and one exponential a score; the maximum is taken over raw
// scores within a group (a >= 0) and the row's sum gets each group's weights divided by
// 2^(log2 b - e + 6) again. e follows the largest value scale, with two octaves to spare:
// weights reach the MMA below 2^15, rounded to binary16 (2^-11 of themselves; with a
// binary16 output, whose own step is no larger, in two terms, 2^-22). A value scale more than 2^60 below the largest counts
// as that: its weights vanish in binary16 either way.
//
// Every wait is bounded, as in prefill_tc.cuh.
#pragma once

#include "prefill_tc.cuh"
#include "scaled_attention.cuh"

namespace pagedkv {

constexpr int kSpLoaders = 3;                      // warps an operand
constexpr int kSpSlice = 32;                       // keys a warp widens at a time
constexpr int kSpRing = 4;                         // tiles whose scales are kept: K stages + 1 at least
constexpr float kSpMoveLog2 = 8.f;                 // the running maximum moves when a score passes it by this

template <int D>
struct SpShape {
    static constexpr int N = 128;
    static constexpr int kQBytes = kTcRows * D * 2;                    // a query tile
    static constexpr int kTile = N * D * 2;                            // a K (V) stage
    static constexpr int NSK = 2, NSV = 3;
    static constexpr int kKOff = 2 * kQBytes;
    static constexpr int kVOff = kKOff + NSK * kTile;
    static constexpr int kBarOff = kVOff + NSV * kTile;
    // k_full[NSK] k_empty[NSK] v_full[NSV] v_empty[NSV] scales[kSpRing] s_full[2] p_full[2] drain q_ready
    static constexpr int kNumBars = 2 * NSK + 2 * NSV + kSpRing + 6;
    static constexpr int kMiscOff = kBarOff + kNumBars * 8;            // tmem base, abort flag
    static constexpr int kScaleOff = (kMiscOff + 16 + 15) / 16 * 16;   // [kSpRing][8] pairs (a, log2 b)
    static constexpr int kMulOff = kScaleOff + kSpRing * 8 * 8;        // [256] the rows' units
    static constexpr int kBytes = kMulOff + 256 * 4;
    static constexpr int kAlloc = kBytes + 1024;
    static constexpr int kTmemCols = 512;
    static constexpr int kTileCols = N + D;                            // S (then P), O
    static_assert(2 * kTileCols <= kTmemCols, "TMEM columns");
    static_assert(kAlloc <= kTcSmemLimit, "shared memory");
    static_assert(kSpRing >= NSK + 1 && kSpRing >= NSV + 1, "scales live until both softmaxes have read them");
};

// One loader warp's slices of an operand: slice n = 4 j + q is keys 32 q .. of tile j.
template <typename CT, int D, int NS, bool kKeys>
__device__ __forceinline__ void sp_load(const ScaledAttnParams& p, uint8_t* ring, float2* scales, uint64_t* full,
                                        uint64_t* empty, uint64_t* scale_bar, int s, int kvh, int T0, int kend, int ntiles,
                                        int which, int lane, volatile int* abort_flag) {
    using Sh = SpShape<D>;
    constexpr int CPR = D / 16;                    // 16-code chunks of a row
    constexpr int PER = kSpSlice * CPR / 32;       // of a lane's
    const int32_t* table = p.block_tables + (size_t)s * p.max_blocks;
    const uint8_t* cache = kKeys ? p.k_cache : p.v_cache;
    const float* block_scales = kKeys ? p.k_scales : p.v_scales;
    const int B = p.block_size;
    const int last = 4 * ntiles;
    // eight lanes that store together hold two rows of one 64-column span, in all banks
    const int chunk = D == 128 ? (lane & 3) + ((lane >> 1) & 4) : lane & 3;
    const int row0 = D == 128 ? ((lane >> 2) & 1) + ((lane >> 4) << 1) : lane >> 2;
    constexpr int STEP = 32 / CPR;                 // rows of a pass
    auto block_of = [&](int n) {
        const int key = T0 + n * kSpSlice + lane;
        return n < last && key < kend ? table[key / B] : -1;
    };
    uint4 buf[PER];
    float scale = 0.f;
    auto fetch = [&](int n, int blk, uint4 (&w)[PER], float& sc) {
        const int key = T0 + n * kSpSlice + lane;
        bool there = n < last && key < kend;
        if (there && (blk < 0 || blk >= p.num_blocks)) {
            if (p.status) atomicOr(p.status, PA_DEV_BAD_BLOCK_ID);
            there = false;
        }
        const int64_t slab = there ? (int64_t)blk * p.num_kv_heads + kvh : 0;
        const int64_t row = there ? slab * B + (key - key / B * B) : -1;
        sc = there && (lane & 15) == 0 ? block_scales[slab] : 0.f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int64_t r = __shfl_sync(0xffffffffu, row, i * STEP + row0);
            w[i] = r >= 0 ? *reinterpret_cast<const uint4*>(cache + (size_t)r * D + chunk * 16) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    int blk = block_of(which);
    if (which < last) fetch(which, blk, buf, scale);
    blk = block_of(which + kSpLoaders);
    for (int n = which; n < last; n += kSpLoaders) {
        uint4 ahead[PER];
        float scale_ahead = 0.f;
        const int j = n >> 2, q = n & 3;
        if ((lane & 15) == 0) {
            float* sp = reinterpret_cast<float*>(scales + (j % kSpRing) * 8 + q * 2 + (lane >> 4));
            if (kKeys) sp[0] = scale;
            else sp[1] = log2f(scale);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&scale_bar[j % kSpRing]);
        fetch(n + kSpLoaders, blk, ahead, scale_ahead);
        blk = block_of(n + 2 * kSpLoaders);
        const int st = j % NS;
        if (j >= NS) {
            const bool ok = tc_wait(&empty[st], (uint32_t)((j / NS - 1) & 1), p.status, abort_flag);
            if (!__all_sync(0xffffffffu, ok)) return;
        }
        uint8_t* tile = ring + st * Sh::kTile;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int r = q * kSpSlice + i * STEP + row0;
            const uint32_t in[4] = {buf[i].x, buf[i].y, buf[i].z, buf[i].w};
            uint32_t o[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t w = biased<CT>(in[k]);
                o[2 * k] = widen2<CT>(w, 0x4140);
                o[2 * k + 1] = widen2<CT>(w, 0x4342);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
                *reinterpret_cast<uint4*>(tile + sw128_chunk<Sh::N>(r, 2 * chunk + h)) = make_uint4(o[4 * h], o[4 * h + 1], o[4 * h + 2], o[4 * h + 3]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[st]);     // the MMA issuer, which waits for it, has the fence between the proxies
#pragma unroll
        for (int i = 0; i < PER; ++i) buf[i] = ahead[i];
        scale = scale_ahead;
    }
}

template <typename CT, int D, bool kTwoTerms>
__global__ void __launch_bounds__(kTcThreadsFp8, 1)
scaled_prefill_kernel(const __grid_constant__ ScaledAttnParams p) {
    begin_overlapped();
    using Sh = SpShape<D>;
    constexpr bool kFp8 = std::is_same<CT, e4m3_t>::value;
    constexpr int N = Sh::N, NSK = Sh::NSK, NSV = Sh::NSV;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* k_full = reinterpret_cast<uint64_t*>(sm + Sh::kBarOff);
    uint64_t* k_empty = k_full + NSK;
    uint64_t* v_full = k_empty + NSK;
    uint64_t* v_empty = v_full + NSV;
    uint64_t* scale_bar = v_empty + NSV;           // [kSpRing]
    uint64_t* s_full = scale_bar + kSpRing;        // [2], by query tile
    uint64_t* p_full = s_full + 2;                 // [2]
    uint64_t* drain = p_full + 2;
    uint64_t* q_ready = drain + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + Sh::kMiscOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + Sh::kMiscOff + 4);
    float2* scales = reinterpret_cast<float2*>(sm + Sh::kScaleOff);
    float* mul = reinterpret_cast<float*>(sm + Sh::kMulOff);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int s = blockIdx.z;
    const int pair = blockIdx.y / p.num_kv_heads, kvh = blockIdx.y - pair * p.num_kv_heads;
    int L, q0, Q;
    if (!scaled_sequence(p, s, tid == 0 && blockIdx.x == 0 && blockIdx.y == 0, L, q0, Q)) return;
    const int G = p.group;
    const int row0 = pair * 2 * kTcRows, rows = min(2 * kTcRows, Q * G - row0);
    if (rows <= 0) return;
    const bool two = rows > kTcRows;
    const int first_pos = L - Q;
    const int seen = first_pos + (row0 + rows - 1) / G + 1;
    const int T0 = blockIdx.x * p.partition_size;
    if (T0 >= seen) return;                        // (an empty context has no query here)
    const int kend = min(T0 + p.partition_size, seen);
    const int ntiles = (kend - T0 + N - 1) / N;

    if (tid == kTcKWarp * 32) {
        for (int i = 0; i < NSK; ++i) {
            mbar_init(&k_full[i], N / kSpSlice);
            mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < NSV; ++i) {
            mbar_init(&v_full[i], N / kSpSlice);
            mbar_init(&v_empty[i], 1);
        }
        for (int i = 0; i < kSpRing; ++i) mbar_init(&scale_bar[i], 2 * N / kSpSlice);
        for (int t = 0; t < 2; ++t) {
            mbar_init(&s_full[t], 1);
            mbar_init(&p_full[t], kTcRows);
        }
        mbar_init(drain, 1);
        mbar_init(q_ready, kTcSoftmaxThreads / 32);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == kTcMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(tmem_slot)), "r"(Sh::kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp >= kTcSoftmaxThreads / 32) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTcProducerRegs));
        if (warp == 8 || warp == 10 || warp == 12) {
            sp_load<CT, D, NSK, true>(p, sm + Sh::kKOff, scales, k_full, k_empty, scale_bar, s, kvh, T0, kend, ntiles,
                                      (warp - 8) >> 1, lane, abort_flag);
        } else if (warp == 11 || warp == 13 || warp == 15) {
            sp_load<CT, D, NSV, false>(p, sm + Sh::kVOff, scales, v_full, v_empty, scale_bar, s, kvh, T0, kend, ntiles,
                                       (warp - 11) >> 1, lane, abort_flag);
        } else if (warp == kTcMmaWarp && lane == 0) {
            constexpr uint32_t idS = tc_idesc<__half>(kTcRows, N, 0);
            constexpr uint32_t idO = tc_idesc<__half>(kTcRows, D, 1);
            const int last_t = two ? 1 : 0;
            auto qk = [&](int t, int j) -> bool {
                const int st = j % NSK;
                if (t == 0) {
                    if (!tc_wait(&k_full[st], (uint32_t)((j / NSK) & 1), p.status, abort_flag)) return false;
                    fence_async_smem();
                    tc_fence_after();
                }
                const uint32_t qa = smem_u32(sm + t * Sh::kQBytes);
                const uint32_t ka = smem_u32(sm + Sh::kKOff + st * Sh::kTile);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = (uint32_t)(kk & 3) * 32u;
                    tc_mma(tmem + t * Sh::kTileCols, tc_desc(qa + (kk >> 2) * (kTcRows * 128) + off, 16, 1024),
                           tc_desc(ka + (kk >> 2) * (N * 128) + off, 16, 1024), idS, kk > 0);
                }
                if (t == last_t) tc_commit(&k_empty[st]);
                tc_commit(&s_full[t]);
                return true;
            };
            auto pv = [&](int t, int j) -> bool {
                const int st = j % NSV;
                if (!tc_wait(&p_full[t], (uint32_t)(j & 1), p.status, abort_flag)) return false;
                if (t == 0) {
                    if (!tc_wait(&v_full[st], (uint32_t)((j / NSV) & 1), p.status, abort_flag)) return false;
                    fence_async_smem();
                }
                tc_fence_after();
                const uint32_t va = smem_u32(sm + Sh::kVOff + st * Sh::kTile);
                const uint32_t pt = tmem + t * Sh::kTileCols;
#pragma unroll
                for (int u = 0; u < (kTwoTerms ? 2 : 1); ++u)
#pragma unroll
                    for (int kk = 0; kk < N / 16; ++kk)
                        tc_mma_ts(pt + N, pt + u * (N / 2) + kk * 8, tc_desc(va + kk * 2048, N * 128, 1024), idO,
                                  j > 0 || u > 0 || kk > 0);
                if (t == last_t) tc_commit(&v_empty[st]);
                return true;
            };
            bool ok = tc_wait(q_ready, 0u, p.status, abort_flag);
            tc_fence_after();
            if (ok) ok = qk(0, 0);
            if (ok && two) ok = qk(1, 0);
            for (int j = 0; j < ntiles && ok; ++j) {
                ok = pv(0, j);
                if (ok && j + 1 < ntiles) ok = qk(0, j + 1);
                if (ok && two) {
                    ok = pv(1, j);
                    if (ok && j + 1 < ntiles) ok = qk(1, j + 1);
                }
            }
            // everything issued ends before the epilogue reads O and before TMEM is freed
            tc_commit(drain);
            mbar_wait_bounded(drain, 0, p.status);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTcSoftmaxRegs));
        const int qt = warp >> 2;
        const int r = tid & (kTcRows - 1);
        // ---- the query, under a power of two for each row: a group of lanes a row
        {
            constexpr int CPR = D / 8;                                 // 16-byte chunks of a row
            constexpr int RPW = 32 / CPR;                              // rows at a time
            const int c = lane % CPR;
            uint4 v[32 / RPW];
#pragma unroll
            for (int i = 0; i < 32 / RPW; ++i) {
                const int rr = warp * 32 + i * RPW + lane / CPR, row = row0 + rr;
                v[i] = make_uint4(0u, 0u, 0u, 0u);
                if (rr < rows)
                    v[i] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.query) +
                                                           ((size_t)(q0 + row / G) * p.num_q_heads + kvh * G + row % G) * D + c * 8);
            }
#pragma unroll
            for (int i = 0; i < 32 / RPW; ++i) {
                const int rr = warp * 32 + i * RPW + lane / CPR;
                uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                uint32_t m2 = 0u;                                      // magnitudes order as integers
#pragma unroll
                for (int k = 0; k < 4; ++k) m2 = __vmaxu2(m2, w[k] & 0x7FFF7FFFu);
                m2 = max(m2 & 0xFFFFu, m2 >> 16);
#pragma unroll
                for (int m = CPR / 2; m; m >>= 1) m2 = max(m2, __shfl_xor_sync(0xffffffffu, m2, m));
                const float mx = p.bf16 ? unpack2<__nv_bfloat16>(m2).x : unpack2<__half>(m2).x;
                const uint32_t ex = min(max(__float_as_uint(mx) >> 23, 1u), 252u);
                const float unit = mx > 0.f && mx < INFINITY ? __uint_as_float(ex << 23) : 1.f;
                const float inv = 1.f / unit;                          // exact
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 f = p.bf16 ? unpack2<__nv_bfloat16>(w[k]) : unpack2<__half>(w[k]);
                    w[k] = pack2<__half>(f.x * inv, f.y * inv);
                }
                const int tr = rr & (kTcRows - 1);
                *reinterpret_cast<uint4*>(sm + (rr >> 7) * Sh::kQBytes + sw128_chunk<kTcRows>(tr, c)) = make_uint4(w[0], w[1], w[2], w[3]);
                if (c == 0) mul[rr] = p.q_mul * unit * (kFp8 ? 256.f : 1.f);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_ready);
        }
        if (qt == 0 || two) {
            const uint32_t sbuf = tmem + ((uint32_t)((warp & 3) * 32) << 16) + qt * Sh::kTileCols;
            const uint32_t obuf = sbuf + N;
            const int rr = qt * kTcRows + r;
            const bool valid = rr < rows;
            const int row = row0 + min(rr, rows - 1);
            const int token = row / G;
            const int pos = first_pos + token;                         // the last key that the row sees
            const float hm = mul[rr];
            float m = -INFINITY, l = 0.f;
            float e_ref = -1e4f;                                       // value scales up to 2^e_ref fit the weights
            bool ok = true;
            for (int j = 0; j < ntiles; ++j) {
                ok = tc_wait(&scale_bar[j % kSpRing], (uint32_t)((j / kSpRing) & 1), p.status, abort_flag) &&
                     tc_wait(&s_full[qt], (uint32_t)(j & 1), p.status, abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                uint32_t xr[N];
#pragma unroll
                for (int c = 0; c < N; c += 32) tc_ld32(sbuf + c, *reinterpret_cast<uint32_t(*)[32]>(xr + c));
                const float2* sp = scales + (j % kSpRing) * 8;         // broadcast reads
                // the group's scale on the row's scores; zero must not meet a masked one
                auto on_row = [&](float a) {
                    const float k = a * hm;
                    return k == 0.f ? 1.17549435e-38f : k;
                };
                tc_wait_ld();
                float x[N];
#pragma unroll
                for (int c = 0; c < N; ++c) x[c] = __uint_as_float(xr[c]);
                const int key0 = T0 + j * N;
                if (key0 + N - 1 > pos) {
#pragma unroll
                    for (int c = 0; c < N; ++c)
                        if (key0 + c > pos) x[c] = -INFINITY;
                }
                float m_cand = m, b_most = sp[0].y;
#pragma unroll
                for (int g = 0; g < 8; ++g) {
                    float y = fmax3(x[16 * g], x[16 * g + 1], x[16 * g + 2]);
                    float z = fmax3(x[16 * g + 3], x[16 * g + 4], x[16 * g + 5]);
                    y = fmax3(y, x[16 * g + 6], x[16 * g + 7]);
                    z = fmax3(z, x[16 * g + 8], x[16 * g + 9]);
                    y = fmax3(y, x[16 * g + 10], x[16 * g + 11]);
                    z = fmax3(z, x[16 * g + 12], x[16 * g + 13]);
                    y = fmax3(y, x[16 * g + 14], x[16 * g + 15]);
                    const float2 ab = sp[g];
                    m_cand = fmaxf(m_cand, fmaxf(y, z) * on_row(ab.x));
                    b_most = fmaxf(b_most, ab.y);
                }
                const bool wider = b_most > e_ref;                     // the same for every row
                const bool moved = m_cand > m + kSpMoveLog2;
                const float m_use = moved ? m_cand : m;
                const float al = m == -INFINITY ? 1.f : fast_exp2(m - m_use);
                float drop = 1.f;
                if (wider) {
                    const float e_new = ceilf(b_most) + 2.f;
                    drop = fast_exp2(e_ref - e_new);
                    e_ref = e_new;
                }
                l *= al;
                const float m_sub = m_use == -INFINITY ? 0.f : m_use;
                m = m_use;
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int g = 2 * h; g < 2 * h + 2; ++g) {
                        const float2 ab = sp[g];
                        const float lift = (ab.y < e_ref - 60.f ? -60.f : ab.y - e_ref) + 6.f;
                        const float k1 = on_row(ab.x);
                        const float2 k2 = make_float2(k1, k1);
                        const float2 c2 = make_float2(lift - m_sub, lift - m_sub);
                        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                        for (int c = 0; c < 16; c += 2) {
                            const float2 t = __ffma2_rn(make_float2(x[16 * g + c], x[16 * g + c + 1]), k2, c2);
                            const float2 e = make_float2(fast_exp2(t.x), fast_exp2(t.y));
                            sum[(c >> 1) & 1] = __fadd2_rn(sum[(c >> 1) & 1], e);
                            const uint32_t w = pack2<__half>(e.x, e.y);
                            hi[(16 * g + c - 32 * h) / 2] = w;
                            if constexpr (kTwoTerms) {
                                const float2 rest = __ffma2_rn(unpack2<__half>(w), make_float2(-1.f, -1.f), e);
                                lo[(16 * g + c - 32 * h) / 2] = pack2<__half>(rest.x, rest.y);
                            }
                        }
                        sum[0] = __fadd2_rn(sum[0], sum[1]);
                        l = fmaf(sum[0].x + sum[0].y, fast_exp2(-lift), l);
                    }
                    tc_st_n<16>(sbuf + h * 16, hi);
                    if constexpr (kTwoTerms) tc_st_n<16>(sbuf + N / 2 + h * 16, lo);
                }
                if (j > 0 && __any_sync(0xffffffffu, moved || wider)) {
                    // O holds the tiles before this one: S of this tile came after their P.V
                    const float alpha = al * drop;
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t o[32];
                        tc_ld32(obuf + c, o);
                        tc_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        tc_st32(obuf + c, o);
                    }
                }
                tc_wait_st();
                tc_fence_before();
                mbar_arrive(&p_full[qt]);
            }
            if (ok) {
                ok = tc_wait(drain, 0u, p.status, abort_flag);
                ok = __all_sync(0xffffffffu, ok);
            }
            if (ok) {
                tc_fence_after();
                const bool sees = valid && pos >= T0;                  // of this partition, anything
                const float out_mul = fast_exp2(e_ref - 6.f) * (kFp8 ? 256.f : 1.f) / l;
                const size_t at = (size_t)(q0 + token) * p.num_q_heads + kvh * G + (row - token * G);
                const size_t part = at * p.max_parts + blockIdx.x;
                if (sees && p.max_parts > 1) {
                    p.max_logits[part] = m;
                    p.exp_sums[part] = l;
                }
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    tc_ld32(obuf + c, o);
                    tc_wait_ld();
                    float f[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(o[e]) * out_mul;
                    if (sees && p.max_parts > 1) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4*>(p.tmp_out + part * D + c + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
                    } else if (sees) {
                        uint16_t* orow = static_cast<uint16_t*>(p.out) + at * D + c;
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            uint4 v;
                            if (p.bf16)
                                v = make_uint4(pack2<__nv_bfloat16>(f[e], f[e + 1]), pack2<__nv_bfloat16>(f[e + 2], f[e + 3]),
                                               pack2<__nv_bfloat16>(f[e + 4], f[e + 5]), pack2<__nv_bfloat16>(f[e + 6], f[e + 7]));
                            else
                                v = make_uint4(pack2<__half>(f[e], f[e + 1]), pack2<__half>(f[e + 2], f[e + 3]),
                                               pack2<__half>(f[e + 4], f[e + 5]), pack2<__half>(f[e + 6], f[e + 7]));
                            *reinterpret_cast<uint4*>(orow + e) = v;
                        }
                    }
                    __syncwarp();
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kTcMmaWarp) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(Sh::kTmemCols) : "memory");
    }
}

template <typename CT, int D, bool kTwoTerms>
cudaError_t launch_scaled_prefill_terms(const ScaledAttnParams& p, cudaStream_t stream) {
    auto kernel = scaled_prefill_kernel<CT, D, kTwoTerms>;
    cudaError_t e = ensure_smem_attribute(reinterpret_cast<const void*>(kernel), SpShape<D>::kAlloc);
    if (e != cudaSuccess) return e;
    return launch_overlapped(kernel, p, dim3(p.max_parts, p.num_kv_heads * p.row_tiles, p.num_seqs), kTcThreadsFp8, SpShape<D>::kAlloc, stream);
}

template <typename CT, int D>
cudaError_t launch_scaled_prefill(const ScaledAttnParams& p, cudaStream_t stream) {
    return p.bf16 ? launch_scaled_prefill_terms<CT, D, false>(p, stream) : launch_scaled_prefill_terms<CT, D, true>(p, stream);
}

}  // namespace pagedkv
