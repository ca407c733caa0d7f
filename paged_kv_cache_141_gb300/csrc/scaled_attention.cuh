// scaled_attention.cuh -- causal attention over a paged cache of 8-bit codes with a
// scale for each (block, KV head): one query token per sequence (decode) or
// several (drafts, chunks). With codes c and scales a (keys) and b (values) of the
// block that holds position t,
//     s_t = scale a_t <q, c_t>,   out = sum_t softmax(s)_t b_t c_t.
//
// Work unit: (sequence, KV head, 8 NT query rows, partition of the context). Rows
// are (query token, head of the group) pairs, token-major, so a group's heads and a
// sequence's drafts read each key once. Four warps of a CTA take the partition's 32-token
// stages in turn, each with a ring of its own that it fills by 16-byte asynchronous copies
// (any block size: a lane finds a token's block, the rows' addresses go round by
// shuffles); no barrier but the warp's own. Per stage:
//   S (16 tokens x 8 rows) = C_K Q^T on binary16 warp-level MMAs, the codes widened in
//     registers, exactly: integers by the bits of 1024 + (c + 128), less 1152; E4M3 by
//     moving the exponent field (values times 2^-8);
//   softmax against a reference that moves only when a logit passes it by 2^8;
//   O^T += C_V^T P^T, with the value scales in the weights.
//
// Precision. The query meets the codes in binary16 under a power of two for each row
// that brings its largest component into [1, 2): exact for bfloat16 and binary16 but for
// components more than 2^14 below the row's largest. Scores, statistics and sums are
// binary32. A weight p b is rounded to binary16 (2^-11, below half a step of the codes)
// under a power of two shared by the stage's blocks, which follows the largest value
// scale seen: 2^-14 of the largest weight before its bits thin out, 2^-25 of it before it
// vanishes.
//
// Several partitions: normalised partial outputs with their maximum and sum go to the
// workspace, and a second kernel merges them (M = max m_p, sum of l_p exp(m_p - M) o_p).
#pragma once

#include "decode_mma.cuh"

namespace pagedkv {

struct int8_code_t {
    int8_t bits;
};

constexpr int kScaledWarps = 4;
constexpr int kScaledThreads = kScaledWarps * 32;
constexpr int kScaledStage = 32;                   // tokens

template <int D, int NT>
struct ScaledShape {
    static constexpr int KS = D / 16;
    static constexpr int kRows = 8 * NT;
    static constexpr int kTile = kScaledStage * D;                     // bytes of a stage's keys (values)
    static constexpr int kStageBytes = 2 * kTile + 2 * kScaledStage * 4;   // and its scales
    static constexpr int NST = D == 64 ? 6 : (D == 128 ? 3 : 2);
    static constexpr int kRing = kScaledWarps * NST * kStageBytes;
    static constexpr int kOutStride = D + 8;
    static constexpr int kCombine = kScaledWarps * kRows * (kOutStride + 2) * 4;
    static constexpr int kQOff = (kRing > kCombine ? kRing : kCombine);
    static constexpr int kMulOff = kQOff + NT * KS * 256;
    static constexpr int kBytes = kMulOff + kRows * 4;
    static constexpr bool kQReg = NT * KS <= 16;                       // the query's fragments in registers
};

// One sequence's part of the call. False: nothing to do (a fault is reported by one thread).
__device__ __forceinline__ bool scaled_sequence(const ScaledAttnParams& p, int s, bool report, int& L, int& q0, int& Q) {
    L = p.context_lens[s];
    q0 = s;
    Q = 1;
    int64_t end = (int64_t)s + 1;
    if (p.query_start) {
        q0 = p.query_start[s];
        end = p.query_start[s + 1];
        Q = (int)(end - q0);
    }
    const int64_t tab = (int64_t)p.max_blocks * p.block_size;
    if (L < 0 || L > p.max_context_len || L > tab || q0 < 0 || end < q0 || end > p.num_queries || end - q0 > p.max_queries ||
        (p.query_start && Q > L)) {
        if (report && p.status) atomicOr(p.status, PA_DEV_BAD_LEN);
        return false;
    }
    return Q > 0;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Byte offset of 16-byte chunk c of row r in a stage tile: within each 128-byte line the
// chunks change places by the row, so that the same chunk of eight rows lies in all banks.
template <int D>
__device__ __forceinline__ int tile_at(int r, int c) {
    if constexpr (D == 64) return (r >> 1) * 128 + (((((r & 1) << 2) | c) ^ ((r >> 1) & 7)) << 4);
    else return r * D + ((c >> 3) << 7) + (((c & 7) ^ (r & 7)) << 4);
}

// Two codes of a word to a binary16 pair. The bytes named by sel's digits 0 and 2.
template <typename CT>
__device__ __forceinline__ uint32_t widen2(uint32_t w, uint32_t sel) {
    if constexpr (std::is_same<CT, e4m3_t>::value) {
        return e4m3x2_to_f16x2_scaled(__byte_perm(w, 0u, sel));
    } else {
        const uint32_t u = __byte_perm(w, 0x64646464u, sel);           // 1024 + (c + 128)
        const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&u), __half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480)));
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}
template <typename CT>
__device__ __forceinline__ uint32_t biased(uint32_t w) {
    return std::is_same<CT, e4m3_t>::value ? w : w ^ 0x80808080u;
}

template <typename CT, int D, int NT>
__global__ void __launch_bounds__(kScaledThreads)
scaled_attention_kernel(const __grid_constant__ ScaledAttnParams p) {
    begin_overlapped();
    using S = ScaledShape<D, NT>;
    using Ops = MmaOps<__half>;
    constexpr bool kFp8 = std::is_same<CT, e4m3_t>::value;
    constexpr int KS = S::KS, NST = S::NST, W = kScaledWarps;
    constexpr int CPR = D / 16;                    // 16-byte chunks of a row
    constexpr int RPP = 32 / CPR;                  // rows of a copy pass
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t4 = lane & 3;
    const int mi = lane >> 3, r8 = lane & 7;
    const int s = blockIdx.z;
    const int kvh = blockIdx.y / p.row_tiles, tile = blockIdx.y - kvh * p.row_tiles;
    const int G = p.group, B = p.block_size;
    int L, q0, Q;
    if (!scaled_sequence(p, s, threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0, L, q0, Q)) return;
    const int row0 = tile * S::kRows, rows = min(S::kRows, Q * G - row0);
    if (rows <= 0) return;
    const int first_pos = L - Q;                   // of query token 0
    const int seen = first_pos + (row0 + rows - 1) / G + 1;            // keys that the tile's last row sees
    const int T0 = blockIdx.x * p.partition_size;
    if (T0 >= seen) {
        if (L == 0 && p.max_parts == 1) {          // an empty context
            for (int i = threadIdx.x; i < rows * D; i += kScaledThreads) {
                const size_t o = ((size_t)q0 * p.num_q_heads + kvh * G + row0 + i / D) * D + i % D;
                if (p.bf16) static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(0.f);
                else static_cast<__half*>(p.out)[o] = __float2half_rn(0.f);
            }
        }
        return;
    }
    const int Tend = min(T0 + p.partition_size, seen);
    const int n_st = (Tend - T0 + kScaledStage - 1) / kScaledStage;

    // ------------------------------------------------------------ this warp's ring
    uint8_t* ring = smem + warp * NST * S::kStageBytes;
    const uint32_t ring_u32 = smem_u32(ring);
    const int32_t* table = p.block_tables + (size_t)s * p.max_blocks;
    const int cr = lane / CPR, cc = lane % CPR;
    // the block of this lane's token in stage k, read a stage ahead of its use
    auto block_of = [&](int k) {
        const int t = T0 + k * kScaledStage + lane;
        return k < n_st && t < Tend ? table[t / B] : -1;
    };
    int next_block = block_of(warp);
    auto issue = [&](int k, int slot) {
        if (k < n_st) {
            const int t = T0 + k * kScaledStage + lane;
            const int blk = next_block;
            next_block = block_of(k + W);
            bool there = t < Tend;
            if (there && (blk < 0 || blk >= p.num_blocks)) {
                if (p.status) atomicOr(p.status, PA_DEV_BAD_BLOCK_ID);
                there = false;
            }
            const int64_t slab = there ? (int64_t)blk * p.num_kv_heads + kvh : 0;
            const int64_t row = there ? slab * B + (t - t / B * B) : -1;
            const uint32_t st = ring_u32 + slot * S::kStageBytes;
            cp_async4(st + 2 * S::kTile + lane * 4, p.k_scales + slab, there);
            cp_async4(st + 2 * S::kTile + (kScaledStage + lane) * 4, p.v_scales + slab, there);
#pragma unroll
            for (int i = 0; i < CPR; ++i) {
                const int r = i * RPP + cr;
                const int64_t src = __shfl_sync(0xffffffffu, row, r);
                const size_t off = (size_t)max(src, (int64_t)0) * D + cc * 16;
                const uint32_t d = st + tile_at<D>(r, cc);
                cp_async16(d, p.k_cache + off, src >= 0);
                cp_async16(d + S::kTile, p.v_cache + off, src >= 0);
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < NST - 1; ++i) issue(warp + i * W, i);

    // ------------------------------------------------------------ the query, as B fragments
    uint2* qf = reinterpret_cast<uint2*>(smem + S::kQOff);             // [NT][KS][32]
    float* mul = reinterpret_cast<float*>(smem + S::kMulOff);          // [rows]
    for (int nt = warp; nt < NT; nt += W) {
        const int r = 8 * nt + g;
        const int row = row0 + r;
        const bool there = r < rows;
        const size_t at = there ? ((size_t)(q0 + row / G) * p.num_q_heads + kvh * G + row % G) * D : 0;
        float x[KS][4], mx = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            uint2 w = make_uint2(0u, 0u);
            if (there) w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.query) + at + 16 * ks + 4 * t4);
            float2 a, b;
            if (p.bf16) {
                a = MmaOps<__nv_bfloat16>::unpack(w.x);
                b = MmaOps<__nv_bfloat16>::unpack(w.y);
            } else {
                a = Ops::unpack(w.x);
                b = Ops::unpack(w.y);
            }
            x[ks][0] = a.x; x[ks][1] = a.y; x[ks][2] = b.x; x[ks][3] = b.y;
            mx = fmaxf(mx, fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(b.x), fabsf(b.y))));
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // a power of two in the range whose reciprocal is a normal number
        const uint32_t ex = min(max(__float_as_uint(mx) >> 23, 1u), 252u);
        const float unit = mx > 0.f && mx < INFINITY ? __uint_as_float(ex << 23) : 1.f;
        const float inv = 1.f / unit;                                  // exact
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
            qf[(nt * KS + ks) * 32 + lane] = make_uint2(Ops::pack(x[ks][0] * inv, x[ks][1] * inv), Ops::pack(x[ks][2] * inv, x[ks][3] * inv));
        if (t4 == 0) mul[r] = p.q_mul * unit * (kFp8 ? 256.f : 1.f);
    }
    __syncthreads();
    uint2 qr[S::kQReg ? NT * KS : 1];
    if constexpr (S::kQReg) {
#pragma unroll
        for (int i = 0; i < NT * KS; ++i) qr[i] = qf[i * 32 + lane];
    }
    float hm[NT][2], m_ref[NT][2], l_run[NT][2];
    int lim[NT][2];                                // of the partition's tokens, those that the row sees
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = 8 * nt + 2 * t4 + j;
            hm[nt][j] = mul[r];
            lim[nt][j] = r < rows ? first_pos + (row0 + r) / G + 1 - T0 : 0;
            m_ref[nt][j] = -INFINITY;
            l_run[nt][j] = 0.f;
        }
    const int all_see = first_pos + row0 / G + 1 - T0;                 // tokens below it are seen by every row
    float acc[NT][KS][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[nt][i][j] = 0.f;
    int e_ref = -120;                              // value scales below 2^(e_ref + 1) fit the weights' range

    int slot = 0;
    for (int k = warp; k < n_st; k += W) {
        cp_async_wait<NST - 2>();
        __syncwarp();
        issue(k + (NST - 1) * W, slot == 0 ? NST - 1 : slot - 1);
        const uint8_t* Kst = ring + slot * S::kStageBytes;
        const uint8_t* Vst = Kst + S::kTile;
        const float* scales = reinterpret_cast<const float*>(Kst + 2 * S::kTile);

        // ---- S = C_K Q^T
        float sc[NT][2][4];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j) sc[nt][mt][j] = 0.f;
            const int row = 16 * mt + (mi & 1) * 8 + r8;
#pragma unroll
            for (int kp = 0; kp < KS / 2; ++kp) {
                uint32_t x[4];
                ldmatrix_x4(x, Kst + tile_at<D>(row, 2 * kp + (mi >> 1)));
#pragma unroll
                for (int h2 = 0; h2 < 2; ++h2) {
                    const uint32_t x0 = biased<CT>(x[2 * h2]), x1 = biased<CT>(x[2 * h2 + 1]);
                    uint32_t a[4];
                    a[0] = widen2<CT>(x0, 0x4140);
                    a[1] = widen2<CT>(x1, 0x4140);
                    a[2] = widen2<CT>(x0, 0x4342);
                    a[3] = widen2<CT>(x1, 0x4342);
                    const int ks = 2 * kp + h2;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint2 q = S::kQReg ? qr[nt * KS + ks] : qf[(nt * KS + ks) * 32 + lane];
                        Ops::mma(sc[nt][mt], a, q.x, q.y);
                    }
                }
            }
        }

        // ---- weights; this lane: tokens g, g + 8, g + 16, g + 24, rows 2 t4 and 2 t4 + 1 of each n-tile
        float ka[4], vb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ka[i] = scales[g + 8 * i];
            vb[i] = scales[kScaledStage + g + 8 * i];
        }
        const int vexp = (int)(__reduce_max_sync(0xffffffffu, __float_as_uint(scales[kScaledStage + lane]) << 1 >> 24)) - 127;
        const bool masked = (k + 1) * kScaledStage > all_see;
        bool move = vexp > e_ref;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float mx = -INFINITY;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float v = sc[nt][i >> 1][2 * (i & 1) + j] * ka[i] * hm[nt][j];
                    if (masked && k * kScaledStage + g + 8 * i >= lim[nt][j]) v = -INFINITY;
                    sc[nt][i >> 1][2 * (i & 1) + j] = v;
                    mx = fmaxf(mx, v);
                }
                move |= mx > m_ref[nt][j] + 8.f;
            }
        if (__any_sync(0xffffffffu, move)) {
            const int e_new = max(e_ref, vexp > e_ref ? vexp + 2 : e_ref);
            const float drop = fast_exp2((float)(e_ref - e_new));
            e_ref = e_new;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float alpha[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float mx = fmaxf(fmaxf(sc[nt][0][j], sc[nt][0][2 + j]), fmaxf(sc[nt][1][j], sc[nt][1][2 + j]));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                    const float m_new = fmaxf(m_ref[nt][j], mx);
                    const float al = m_new == -INFINITY || m_ref[nt][j] == -INFINITY ? 1.f : fast_exp2(m_ref[nt][j] - m_new);
                    m_ref[nt][j] = m_new;
                    l_run[nt][j] *= al;
                    alpha[j] = al * drop;
                }
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    acc[nt][i][0] *= alpha[0];
                    acc[nt][i][1] *= alpha[1];
                    acc[nt][i][2] *= alpha[0];
                    acc[nt][i][3] *= alpha[1];
                }
            }
        }
        const float lift = __uint_as_float((uint32_t)(127 + 6 - e_ref) << 23);
#pragma unroll
        for (int i = 0; i < 4; ++i) vb[i] *= lift;
        uint32_t pb[NT][2][2];                     // P^T fragments
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float w[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float m = m_ref[nt][j] == -INFINITY ? 0.f : m_ref[nt][j];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float e = fast_exp2(sc[nt][i >> 1][2 * (i & 1) + j] - m);
                    l_run[nt][j] += e;
                    w[j][i] = e * vb[i];
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) pb[nt][i >> 1][i & 1] = movmatrix_trans(Ops::pack(w[0][i], w[1][i]));
        }

        // ---- O^T += C_V^T P^T: a chunk is 16 components of all 32 tokens; fragment
        // row g is component 2 g, row g + 8 component 2 g + 1
#pragma unroll
        for (int md = 0; md < KS; ++md) {
            uint32_t y[4];
            ldmatrix_x4_trans(y, Vst + tile_at<D>(8 * mi + r8, md));
#pragma unroll
            for (int kt = 0; kt < 2; ++kt) {
                const uint32_t lo = biased<CT>(y[2 * kt]), hi = biased<CT>(y[2 * kt + 1]);
                uint32_t a[4];
                a[0] = widen2<CT>(lo, 0x4240);
                a[1] = widen2<CT>(lo, 0x4341);
                a[2] = widen2<CT>(hi, 0x4240);
                a[3] = widen2<CT>(hi, 0x4341);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) Ops::mma(acc[nt][md], a, pb[nt][kt][0], pb[nt][kt][1]);
            }
        }
        slot = slot + 1 == NST ? 0 : slot + 1;
    }

    // ------------------------------------------------------------ join the four warps
    cp_async_wait<0>();
    __syncthreads();                               // the rings are free
    float* cm = reinterpret_cast<float*>(smem);                        // [W][rows]
    float* cl = cm + W * S::kRows;                                     // [W][rows]
    float* co = cl + W * S::kRows;                                     // [W][rows][kOutStride]
    const float fall = __uint_as_float((uint32_t)(127 + e_ref - 6) << 23) * (kFp8 ? 256.f : 1.f);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float l = l_run[nt][j];
            l += __shfl_xor_sync(0xffffffffu, l, 4);
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            const int r = warp * S::kRows + 8 * nt + 2 * t4 + j;
            if (g == 0) {
                cm[r] = m_ref[nt][j];
                cl[r] = l;
            }
#pragma unroll
            for (int md = 0; md < KS; ++md)
                *reinterpret_cast<float2*>(co + r * S::kOutStride + 16 * md + 2 * g) =
                    make_float2(acc[nt][md][j] * fall, acc[nt][md][2 + j] * fall);
        }
    __syncthreads();
    for (int i = threadIdx.x; i < rows * (D / 4); i += kScaledThreads) {
        const int r = i / (D / 4), d = (i - r * (D / 4)) * 4;
        const int row = row0 + r, token = row / G, head = kvh * G + row - token * G;
        if (first_pos + token + 1 <= T0) continue;                     // sees nothing of this partition
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < W; ++w) M = fmaxf(M, cm[w * S::kRows + r]);
        float sum = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float mw = cm[w * S::kRows + r];
            const float f = mw == -INFINITY ? (cl[w * S::kRows + r] == 0.f ? 0.f : 1.f) : fast_exp2(mw - M);
            sum = fmaf(f, cl[w * S::kRows + r], sum);
            const float4 v = *reinterpret_cast<const float4*>(co + (w * S::kRows + r) * S::kOutStride + d);
            o.x = fmaf(f, v.x, o.x);
            o.y = fmaf(f, v.y, o.y);
            o.z = fmaf(f, v.z, o.z);
            o.w = fmaf(f, v.w, o.w);
        }
        const float inv = __fdiv_rn(1.f, sum);
        o.x *= inv; o.y *= inv; o.z *= inv; o.w *= inv;
        const size_t at = (size_t)(q0 + token) * p.num_q_heads + head;
        if (p.max_parts == 1) {
            uint2 w;
            if (p.bf16) w = make_uint2(MmaOps<__nv_bfloat16>::pack(o.x, o.y), MmaOps<__nv_bfloat16>::pack(o.z, o.w));
            else w = make_uint2(Ops::pack(o.x, o.y), Ops::pack(o.z, o.w));
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at * D + d) = w;
        } else {
            const size_t part = at * p.max_parts + blockIdx.x;
            *reinterpret_cast<float4*>(p.tmp_out + part * D + d) = o;
            if (d == 0) {
                p.max_logits[part] = M;
                p.exp_sums[part] = sum;
            }
        }
    }
}

// The merge of a row's partitions: 32 or 64 threads per (query token, head) hold four
// components each, eight rows of them a CTA taking partitions in turn.
constexpr int kScaledMergeThreads = 256;
constexpr int kScaledMergeParts = 512;             // weights at a time

template <int D>
__global__ void __launch_bounds__(kScaledMergeThreads)
scaled_merge_kernel(const __grid_constant__ ScaledAttnParams p) {
    begin_overlapped();
    constexpr int LANES = D / 4, SLICES = kScaledMergeThreads / LANES;
    __shared__ float weight[kScaledMergeParts];
    __shared__ float red[32];
    __shared__ float4 part_sum[kScaledMergeThreads];
    const int s = blockIdx.z, token = blockIdx.y, head = blockIdx.x;
    int L, q0, Q;
    if (!scaled_sequence(p, s, false, L, q0, Q) || token >= Q) return;
    const int seen = L - Q + token + 1;
    const int n = (seen + p.partition_size - 1) / p.partition_size;
    const size_t at = (size_t)(q0 + token) * p.num_q_heads + head;
    const float* ml = p.max_logits + at * p.max_parts;
    const float* es = p.exp_sums + at * p.max_parts;
    const float4* to = reinterpret_cast<const float4*>(p.tmp_out + at * p.max_parts * D);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float M = -INFINITY;
    for (int i = threadIdx.x; i < n; i += kScaledMergeThreads) M = fmaxf(M, ml[i]);
#pragma unroll
    for (int m = 16; m; m >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, m));
    if (lane == 0) red[warp] = M;
    __syncthreads();
    M = red[0];
#pragma unroll
    for (int w = 1; w < kScaledMergeThreads / 32; ++w) M = fmaxf(M, red[w]);
    const int slice = threadIdx.x / LANES, c = threadIdx.x % LANES;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
    for (int base = 0; base < n; base += kScaledMergeParts) {
        const int count = min(kScaledMergeParts, n - base);
        __syncthreads();
        for (int i = threadIdx.x; i < count; i += kScaledMergeThreads) {
            const float m = ml[base + i], l = es[base + i];
            const float w = m == -INFINITY ? l : l * fast_exp2(m - M);
            weight[i] = w;
            sum += w;
        }
        __syncthreads();
#pragma unroll 4
        for (int i = slice; i < count; i += SLICES) {
            const float w = weight[i];
            const float4 v = to[(size_t)(base + i) * LANES + c];
            o.x = fmaf(w, v.x, o.x);
            o.y = fmaf(w, v.y, o.y);
            o.z = fmaf(w, v.z, o.z);
            o.w = fmaf(w, v.w, o.w);
        }
    }
#pragma unroll
    for (int m = 16; m; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    part_sum[threadIdx.x] = o;
    __syncthreads();
    if (lane == 0) red[warp] = sum;
    __syncthreads();
    if (threadIdx.x >= LANES) return;
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < kScaledMergeThreads / 32; ++w) sum += red[w];
#pragma unroll
    for (int i = 1; i < SLICES; ++i) {
        const float4 v = part_sum[i * LANES + c];
        o.x += v.x; o.y += v.y; o.z += v.z; o.w += v.w;
    }
    const float inv = n > 0 ? __fdiv_rn(1.f, sum) : 0.f;               // no token: zeros
    o.x *= inv; o.y *= inv; o.z *= inv; o.w *= inv;
    uint2 w;
    if (p.bf16) w = make_uint2(MmaOps<__nv_bfloat16>::pack(o.x, o.y), MmaOps<__nv_bfloat16>::pack(o.z, o.w));
    else w = make_uint2(MmaOps<__half>::pack(o.x, o.y), MmaOps<__half>::pack(o.z, o.w));
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at * D + 4 * c) = w;
}

// scaled_prefill.cuh, instantiated in files of its own.
template <typename CT, int D>
cudaError_t launch_scaled_prefill(const ScaledAttnParams& p, cudaStream_t stream);

template <typename CT, int D, int NT>
cudaError_t launch_scaled_rows(const ScaledAttnParams& p, cudaStream_t stream) {
    using S = ScaledShape<D, NT>;
    auto kernel = scaled_attention_kernel<CT, D, NT>;
    cudaError_t e = ensure_smem_attribute(reinterpret_cast<const void*>(kernel), S::kBytes);
    if (e != cudaSuccess) return e;
    return launch_overlapped(kernel, p, dim3(p.max_parts, p.num_kv_heads * p.row_tiles, p.num_seqs), kScaledThreads, S::kBytes, stream);
}

template <typename CT, int D>
cudaError_t launch_scaled_head(const ScaledAttnParams& p, cudaStream_t stream) {
    cudaError_t e;
    if (p.tile_rows == 256) {
        if constexpr (D < 256) e = launch_scaled_prefill<CT, D>(p, stream);
        else return cudaErrorInvalidValue;
    } else if (p.tile_rows == 8) e = launch_scaled_rows<CT, D, 1>(p, stream);
    else if (p.tile_rows == 16) e = launch_scaled_rows<CT, D, 2>(p, stream);
    else if constexpr (D < 256) e = launch_scaled_rows<CT, D, 4>(p, stream);
    else return cudaErrorInvalidValue;
    if (e != cudaSuccess || p.max_parts == 1) return e;
    return launch_overlapped(scaled_merge_kernel<D>, p, dim3(p.num_q_heads, p.max_queries, p.num_seqs), kScaledMergeThreads, 0, stream);
}

template <typename CT>
cudaError_t launch_scaled(const ScaledAttnParams& p, int head_size, cudaStream_t stream) {
    switch (head_size) {
    case 64: return launch_scaled_head<CT, 64>(p, stream);
    case 128: return launch_scaled_head<CT, 128>(p, stream);
    case 256: return launch_scaled_head<CT, 256>(p, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace pagedkv
