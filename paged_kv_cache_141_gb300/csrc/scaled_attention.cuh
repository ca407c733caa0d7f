// scaled_attention.cuh -- causal attention over a paged cache of 8-bit codes with a
// scale for each (block, KV head): one query token per sequence (decode) or
// several (drafts, chunks). With codes c and scales a (keys) and b (values) of the
// block that holds position t,
//     s_t = scale a_t <q, c_t>,   out = sum_t softmax(s)_t b_t c_t.
//
// Rows are (query token, head of the group) pairs, token-major, so a group's heads and
// a sequence's drafts read each key once; an item is a (sequence, KV head, 8 NT rows), and
// its context is cut into stages of 32 tokens. A stage is small against the latency of
// memory, and a partition's own start and end (lengths, table, first stage, joining of
// warps) cost as much as a dozen of them, so nothing starts or ends per partition: the
// stages of all items lie in one line, and every warp of one wave of CTAs takes an
// equal piece of it, from the sums of the sequences' stages that each CTA makes for
// itself. A warp fills a ring of its own by 16-byte asynchronous copies (any block size:
// a lane finds a token's block, the rows' addresses go round by shuffles), across the
// borders of items; no barrier but the warp's own. (64 contexts of 512-8192 tokens,
// 32/8 heads of 128: 96 us, 117 with CTAs of four warps for partitions of 1024-4096 tokens;
// one of 131072: 53, 64. That is 6.0 and 5.0 TB/s; without the join 91 and 47 us, 0.93 and
// 0.85 of what the bytes take at 6.78 TB/s. What is left is the last pieces' end, the join's
// launch, and issue slots: 758 instructions a stage, 973 at first.)
// Per stage:
//   S (16 tokens x 8 rows) = C_K Q^T on binary16 warp-level MMAs, the codes widened in
//     registers, exactly: integers by the bits of 1024 + (c + 128), less 1152; E4M3 by
//     moving the exponent field (values times 2^-8);
//   softmax against a reference that moves only when a logit passes it by 2^8 (both rows of a
//     lane at a time, in two-wide binary32 instructions);
//   O^T += C_V^T P^T, with the value scales in the weights.
//
// Precision. The query meets the codes in binary16 under a power of two for each row
// that brings its largest component into [1, 2): exact for bfloat16 and binary16 but for
// components more than 2^14 below the row's largest. Scores, statistics and sums are
// binary32. A weight p b is rounded to binary16 (2^-11, below half a step of the codes)
// under a power of two of the row's own, which follows the largest weight among the tokens
// that it sees: the largest stands between 2^5 and 2^15, so that 2^-19 of it keeps all its
// bits and 2^-30 of it vanishes. (One unit for all rows, by the largest value scale among
// the blocks read, would cost no more, but a block of large values that a row hardly attends
// to, or does not see, would take the bits from all others.) A bfloat16 output's own
// rounding is eight times coarser; a binary16 output's is no finer than the weights', and
// takes them in two terms (2^-22).
//
// An item within one warp's piece is written out by it. Pieces of others go to the
// workspace, two of a warp's at most (the end of an item that began before its piece, the
// beginning of one that goes on behind it), and a second kernel joins them
// (M = max m_w, sum of exp(m_w - M) (o_w, l_w)).
#pragma once

#include "decode_mma.cuh"

namespace pagedkv {

struct int8_code_t {
    int8_t bits;
};

constexpr int kScaledStage = 32;                   // tokens

template <int D, int NT>
struct ScaledShape {
    static constexpr int KS = D / 16;
    static constexpr int kRows = 8 * NT;
    static constexpr int kTile = kScaledStage * D;                     // bytes of a stage's keys (values)
    static constexpr int kStageBytes = 2 * kTile + 2 * kScaledStage * 4;   // and its scales
    static constexpr int NST = D == 64 ? 4 : 2;
    static constexpr bool kQReg = NT * KS <= 16;                       // the query's fragments in registers
    static constexpr int kQBytes = kQReg ? 0 : NT * KS * 256;
    static constexpr int kWarpBytes = NST * kStageBytes + kQBytes;
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
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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

__device__ __forceinline__ void ldmatrix_x4_at(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans_at(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
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

// The query rows of an item as B fragments, each under a power of two, into registers or
// shared memory; mul: the rows' units (lanes hold rows 2 t4, 2 t4 + 1 of each n-tile).
template <typename CT, int D, int NT>
__device__ __forceinline__ void scaled_query(const ScaledAttnParams& p, int q0, int kvh, int row0, int rows, int lane,
                                             uint2* qr, uint2* qf, float (&mul)[NT][2]) {
    using S = ScaledShape<D, NT>;
    using Ops = MmaOps<__half>;
    const int g = lane >> 2, t4 = lane & 3, G = p.group;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = 8 * nt + g, row = row0 + r;
        const bool there = r < rows;
        const size_t at = there ? ((size_t)(q0 + row / G) * p.num_q_heads + kvh * G + row % G) * D : 0;
        uint2 w[S::KS];
        uint32_t m2 = 0u;                          // 16-bit magnitudes order as integers
#pragma unroll
        for (int ks = 0; ks < S::KS; ++ks) {
            w[ks] = make_uint2(0u, 0u);
            if (there) w[ks] = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.query) + at + 16 * ks + 4 * t4);
        }
#pragma unroll
        for (int ks = 0; ks < S::KS; ++ks) m2 = __vmaxu2(m2, __vmaxu2(w[ks].x & 0x7fff7fffu, w[ks].y & 0x7fff7fffu));
        m2 = max(m2 & 0xffffu, m2 >> 16);
        m2 = max(m2, __shfl_xor_sync(0xffffffffu, m2, 1));
        m2 = max(m2, __shfl_xor_sync(0xffffffffu, m2, 2));
        const float mx = p.bf16 ? __uint_as_float(m2 << 16) : __half2float(__ushort_as_half((unsigned short)m2));
        // a power of two in the range whose reciprocal is a normal number
        const uint32_t ex = min(max(__float_as_uint(mx) >> 23, 1u), 252u);
        const float unit = mx > 0.f && mx < INFINITY ? __uint_as_float(ex << 23) : 1.f;
        const float inv = 1.f / unit;                                  // exact
#pragma unroll
        for (int ks = 0; ks < S::KS; ++ks) {
            float2 a, b;
            if (p.bf16) {
                a = MmaOps<__nv_bfloat16>::unpack(w[ks].x);
                b = MmaOps<__nv_bfloat16>::unpack(w[ks].y);
            } else {
                a = Ops::unpack(w[ks].x);
                b = Ops::unpack(w[ks].y);
            }
            const uint2 f = make_uint2(Ops::pack(a.x * inv, a.y * inv), Ops::pack(b.x * inv, b.y * inv));
            if constexpr (S::kQReg) qr[nt * S::KS + ks] = f;
            else qf[(nt * S::KS + ks) * 32 + lane] = f;
        }
        // (never zero: that must not meet a masked score)
        const float u = fmaxf(p.q_mul * unit * (std::is_same<CT, e4m3_t>::value ? 256.f : 1.f), 1.17549435e-38f);
        mul[nt][0] = __shfl_sync(0xffffffffu, u, 8 * t4);
        mul[nt][1] = __shfl_sync(0xffffffffu, u, 8 * t4 + 4);
    }
}

__device__ __forceinline__ void store_pair(const ScaledAttnParams& p, size_t at, float x, float y) {
    uint32_t w;
    if (p.bf16) w = MmaOps<__nv_bfloat16>::pack(x, y);
    else w = MmaOps<__half>::pack(x, y);
    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + at) = w;
}

// The unit of a row's weights, 2^(6 - d), as kWeightBias - d: a number whose lowest bits are
// the unit's exponent, so that a shift makes it. d: of the row's largest weight p b, from
// above, for p relative to the row's reference.
constexpr float kWeightBias = 12582912.f + 133.f;  // 1.5 * 2^23, and 127 + 6
constexpr float kLeastWeight = -110.f, kMostWeight = 128.f;
__device__ __forceinline__ float weight_unit(float w_ref) { return __uint_as_float(__float_as_uint(w_ref) << 23); }
__device__ __forceinline__ float weight_fall(float w_ref) { return __uint_as_float((254u << 23) - (__float_as_uint(w_ref) << 23)); }

// Stages of a sequence's context; 0 where the call has nothing to do for it.
__device__ __forceinline__ int scaled_stages(const ScaledAttnParams& p, int s, bool report, int& L, int& q0, int& Q) {
    return scaled_sequence(p, s, report, L, q0, Q) ? (L + kScaledStage - 1) / kScaledStage : 0;
}

// A place in the line of stages: stage k of row tile `tile` of KV head kvh of sequence s.
struct ScaledPlace {
    int s, kvh, tile, k, stages;                   // the sequence's stages
    int L, q0, Q;
    __device__ __forceinline__ void next(const ScaledAttnParams& p) {
        if (++k < stages) return;
        k = 0;
        if (++tile < p.row_tiles) return;
        tile = 0;
        if (++kvh < p.num_kv_heads) return;
        kvh = 0;
        do {
            ++s;
            stages = s < p.num_seqs ? scaled_stages(p, s, false, L, q0, Q) : 0;
        } while (stages == 0 && s < p.num_seqs);
    }
};

// kTwoTerms: weights as a binary16 number and the binary16 rest.
template <typename CT, int D, int NT, int W, bool kTwoTerms>
__global__ void __launch_bounds__(W * 32, NT == 1 && D < 256 ? 3 : (D < 256 ? 2 : 1))
scaled_attention_kernel(const __grid_constant__ ScaledAttnParams p) {
    begin_overlapped();
    using S = ScaledShape<D, NT>;
    using Ops = MmaOps<__half>;
    constexpr bool kFp8 = std::is_same<CT, e4m3_t>::value;
    constexpr int KS = S::KS, NST = S::NST;
    constexpr int CPR = D / 16;                    // 16-byte chunks of a row
    constexpr int RPP = 32 / CPR;                  // rows of a copy pass
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t s_sum[W];
    __shared__ int64_t s_before[W];                // of each warp's first sequence: stages before it,
    __shared__ int s_first[W];                     // and which it is
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t4 = lane & 3;
    const int mi = lane >> 3, r8 = lane & 7;
    const int G = p.group, B = p.block_size;

    // ------------------------------------------------------------ this warp's piece of the line
    const int per = (p.num_seqs + W * 32 - 1) / (W * 32);              // sequences a thread
    const int s_lo = min(p.num_seqs, (int)threadIdx.x * per), s_hi = min(p.num_seqs, s_lo + per);
    int64_t mine = 0;
    for (int s = s_lo; s < s_hi; ++s) {
        int L, q0, Q;
        const int n = scaled_stages(p, s, blockIdx.x == 0, L, q0, Q);
        mine += n;
        if (n == 0 && L == 0 && !p.query_start && s % gridDim.x == blockIdx.x)     // an empty context: zeros
            for (int i = 0; i < p.num_q_heads * D; i += 2) store_pair(p, (size_t)s * p.num_q_heads * D + i, 0.f, 0.f);
    }
    int64_t upto = mine;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, upto, m);
        if (lane >= m) upto += o;
    }
    if (lane == 31) s_sum[warp] = upto;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        if (w == warp) upto += total;
        total += s_sum[w];
    }
    const int64_t line = total * p.items;
    const int64_t piece = scaled_piece(line, p.workers);
    {
        // the thread whose sequences hold a warp's first stage finds the sequence
        const int64_t before = upto - mine;
        for (int w = 0; w < W; ++w) {
            const int64_t from = (blockIdx.x * W + w) * piece;
            const int64_t at = from < INT32_MAX ? (uint32_t)from / (uint32_t)p.items : from / p.items;
            if (at >= before && at < upto) {
                int64_t b = before;
                int s = s_lo;
                for (;;) {
                    int L, q0, Q;
                    const int n = scaled_stages(p, s, false, L, q0, Q);
                    if (at < b + n) break;
                    b += n;
                    ++s;
                }
                s_first[w] = s;
                s_before[w] = b;
            }
        }
        if (blockIdx.x == 0) {                     // for the kernel that joins the pieces
            int64_t b = before;
            for (int s = s_lo; s < s_hi; ++s) {
                int L, q0, Q;
                p.stages_before[s] = b;
                b += scaled_stages(p, s, false, L, q0, Q);
            }
            if (threadIdx.x == 0) p.stages_before[p.num_seqs] = total;
        }
    }
    __syncthreads();
    const int64_t begin = (int64_t)(blockIdx.x * W + warp) * piece;
    if (begin >= line) return;
    const int count = (int)(min(begin + piece, line) - begin);

    ScaledPlace now;
    now.s = s_first[warp];
    now.stages = scaled_stages(p, now.s, false, now.L, now.q0, now.Q);
    {
        const int64_t in = begin - s_before[warp] * p.items;
        const int item = (int)(in / now.stages);
        now.k = (int)(in - (int64_t)item * now.stages);
        now.kvh = item / p.row_tiles;
        now.tile = item - now.kvh * p.row_tiles;
    }

    // ------------------------------------------------------------ the ring
    uint8_t* ring = smem + warp * S::kWarpBytes;
    uint2* qf = reinterpret_cast<uint2*>(ring + NST * S::kStageBytes);
    const uint32_t ring_u32 = smem_u32(ring);
    const int cr = lane / CPR, cc = lane % CPR;
    const uint8_t* k_from = p.k_cache + cc * 16;
    const uint8_t* v_from = p.v_cache + cc * 16;
    // the next stage to copy; the place of this lane's token in it, found a stage ahead
    ScaledPlace ahead = now;
    int left = count;                              // stages not yet copied
    int next_block = -1, next_in = 0;
    auto find = [&] {
        const int t = ahead.k * kScaledStage + lane;
        const int j = (int)((uint64_t)(uint32_t)t * p.block_mul >> p.block_shift);      // t / B
        next_in = t - j * B;
        next_block = left > 0 && t < ahead.L ? p.block_tables[(size_t)ahead.s * p.max_blocks + j] : -1;
    };
    find();
    auto issue = [&](int slot) {
        if (left > 0) {
            const bool inside = ahead.k * kScaledStage + lane < ahead.L;
            const bool there = (uint32_t)next_block < (uint32_t)p.num_blocks;
            if (inside && !there && p.status) atomicOr(p.status, PA_DEV_BAD_BLOCK_ID);
            const uint32_t slab = there ? (uint32_t)next_block * p.num_kv_heads + ahead.kvh : 0u;
            const uint32_t row = slab * B + next_in;
            --left;
            ahead.next(p);
            find();
            const uint32_t st = ring_u32 + slot * S::kStageBytes;
            cp_async4(st + 2 * S::kTile + lane * 4, p.k_scales + slab, there);
            cp_async4(st + 2 * S::kTile + (kScaledStage + lane) * 4, p.v_scales + slab, there);
            const uint32_t all = __ballot_sync(0xffffffffu, there);
            if (all == 0xffffffffu) {
#pragma unroll
                for (int i = 0; i < CPR; ++i) {
                    const size_t off = (size_t)__shfl_sync(0xffffffffu, row, i * RPP + cr) * D;
                    const uint32_t d = st + tile_at<D>(i * RPP + cr, cc);
                    cp_async16(d, k_from + off);
                    cp_async16(d + S::kTile, v_from + off);
                }
            } else {                               // zeros where there is no token
#pragma unroll
                for (int i = 0; i < CPR; ++i) {
                    const int r = i * RPP + cr;
                    const bool here = all >> r & 1u;
                    const uint32_t from = __shfl_sync(0xffffffffu, row, r);
                    const size_t off = here ? (size_t)from * D : 0;
                    const uint32_t d = st + tile_at<D>(r, cc);
                    cp_async16(d, k_from + off, here);
                    cp_async16(d + S::kTile, v_from + off, here);
                }
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < NST - 1; ++i) issue(i);

    uint2 qr[S::kQReg ? NT * KS : 1];
    float hm[NT][2], m_ref[NT][2], l_run[NT][2];
    float w_ref[NT][2];                            // kWeightBias - d; weights are p b 2^(6 - d)
    float acc[NT][KS][4];
    int all_see = 0, kvh = 0, row0 = 0, rows = 0;
    bool whole = false;                            // from the item's first stage on
    // tokens that row r sees (worked out where a stage is cut, as few are: in registers they
    // would spill in the widest tiles)
    auto sees = [&](int r) {
        return r < rows ? now.L - now.Q + (int)((uint64_t)(uint32_t)(row0 + r) * p.group_mul >> p.group_shift) + 1 : 0;
    };
    int slot = 0;
    for (int i = 0; i < count; ++i) {
        if (i == 0 || now.k == 0) {
            // ---- an item begins
            kvh = now.kvh;
            row0 = now.tile * S::kRows;
            rows = max(0, min(S::kRows, now.Q * G - row0));
            whole = now.k == 0;
            scaled_query<CT, D, NT>(p, now.q0, kvh, row0, rows, lane, qr, qf, hm);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    m_ref[nt][j] = -INFINITY;
                    l_run[nt][j] = 0.f;
                    w_ref[nt][j] = kWeightBias - kLeastWeight;
                }
            all_see = now.L - now.Q + row0 / G + 1;    // tokens below it are seen by every row
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int md = 0; md < KS; ++md)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[nt][md][j] = 0.f;
        }
        cp_async_wait<NST - 2>();
        __syncwarp();
        issue(slot == 0 ? NST - 1 : slot - 1);
        const float* scales = reinterpret_cast<const float*>(ring + slot * S::kStageBytes + 2 * S::kTile);
        const uint32_t k_at = ring_u32 + slot * S::kStageBytes, v_at = k_at + S::kTile;
        const int key0 = now.k * kScaledStage;

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
                ldmatrix_x4_at(x, k_at + tile_at<D>(row, 2 * kp + (mi >> 1)));
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
        if (vexp == 128) {
            // a value scale that is no number goes with the key's: the rows that see the token get
            // its NaN by their scores, and the weights of others, which are zero, stay so
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (!(vb[i] < INFINITY)) {
                    ka[i] = NAN;
                    vb[i] = 0.f;
                }
        }
        const float v_room = kWeightBias + 8.f - (float)vexp;
        bool move = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float* x = &sc[nt][i >> 1][2 * (i & 1)];           // both rows
                const float2 y = __fmul2_rn(make_float2(x[0], x[1]), make_float2(ka[i], ka[i]));
                x[0] = y.x;
                x[1] = y.y;
            }
        if (__any_sync(0xffffffffu, key0 + kScaledStage > all_see)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int lim = sees(8 * nt + 2 * t4 + j);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (key0 + g + 8 * i >= lim) sc[nt][i >> 1][2 * (i & 1) + j] = -INFINITY;
                }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float mx = fmaxf(fmaxf(sc[nt][0][j], sc[nt][0][2 + j]), fmaxf(sc[nt][1][j], sc[nt][1][2 + j]));
                // no logit more than 2^8 above the reference, and no weight of 2^15, were
                // the largest logit's value scale the stage's largest
                move |= fmaf(mx, hm[nt][j], -m_ref[nt][j]) > fminf(8.f, v_room - w_ref[nt][j]);
            }
        if (__any_sync(0xffffffffu, move)) {
            float bx[4];                           // the value scales' exponents
#pragma unroll
            for (int i = 0; i < 4; ++i) bx[i] = (float)((int)(__float_as_uint(vb[i]) << 1 >> 24) - 127);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float alpha[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float mx = fmaxf(fmaxf(sc[nt][0][j], sc[nt][0][2 + j]), fmaxf(sc[nt][1][j], sc[nt][1][2 + j]));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                    // whole numbers, as d: what moves from one to the other is not rounded
                    const float m_new = fmaxf(m_ref[nt][j], ceilf(mx * hm[nt][j]));
                    // the largest weight, to an octave (masked ones are none: -infinity or NaN here)
                    float t = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 4; ++i) t = fmaxf(t, fmaf(sc[nt][i >> 1][2 * (i & 1) + j], hm[nt][j], -m_new) + bx[i]);
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
                    const float fell = m_ref[nt][j] - m_new;       // (NaN where the row has seen nothing)
                    const float d = kWeightBias - w_ref[nt][j], d_new = fminf(fmaxf(fmaxf(d + fell, ceilf(t)), kLeastWeight), kMostWeight);
                    const bool none = m_new == -INFINITY || m_ref[nt][j] == -INFINITY;
                    m_ref[nt][j] = m_new;
                    w_ref[nt][j] = kWeightBias - d_new;
                    l_run[nt][j] *= none ? 1.f : fast_exp2(fell);
                    alpha[j] = none ? 1.f : fast_exp2(fell + (d - d_new));
                }
#pragma unroll
                for (int i = 0; i < KS; ++i)
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        const float2 y = __fmul2_rn(make_float2(acc[nt][i][e], acc[nt][i][e + 1]), make_float2(alpha[0], alpha[1]));
                        acc[nt][i][e] = y.x;
                        acc[nt][i][e + 1] = y.y;
                    }
            }
        }
        uint32_t pb[NT][2][2], pl[kTwoTerms ? NT : 1][2][2];           // P^T fragments, and of the rests
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            // both rows at a time
            const float2 less = make_float2(m_ref[nt][0] == -INFINITY ? 0.f : -m_ref[nt][0], m_ref[nt][1] == -INFINITY ? 0.f : -m_ref[nt][1]);
            const float2 unit = make_float2(weight_unit(w_ref[nt][0]), weight_unit(w_ref[nt][1]));
            float2 sum = make_float2(l_run[nt][0], l_run[nt][1]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 t = __ffma2_rn(make_float2(sc[nt][k >> 1][2 * (k & 1)], sc[nt][k >> 1][2 * (k & 1) + 1]),
                                            make_float2(hm[nt][0], hm[nt][1]), less);
                const float2 e = make_float2(fast_exp2(t.x), fast_exp2(t.y));
                sum = __fadd2_rn(sum, e);
                const float2 w = __fmul2_rn(__fmul2_rn(e, unit), make_float2(vb[k], vb[k]));
                const uint32_t hi = Ops::pack(w.x, w.y);
                pb[nt][k >> 1][k & 1] = movmatrix_trans(hi);
                if constexpr (kTwoTerms) {
                    const float2 h = Ops::unpack(hi);
                    pl[nt][k >> 1][k & 1] = movmatrix_trans(Ops::pack(w.x - h.x, w.y - h.y));
                }
            }
            l_run[nt][0] = sum.x;
            l_run[nt][1] = sum.y;
        }

        // ---- O^T += C_V^T P^T: a chunk is 16 components of all 32 tokens; fragment
        // row g is component 2 g, row g + 8 component 2 g + 1
#pragma unroll
        for (int md = 0; md < KS; ++md) {
            uint32_t y[4];
            ldmatrix_x4_trans_at(y, v_at + tile_at<D>(8 * mi + r8, md));
#pragma unroll
            for (int kt = 0; kt < 2; ++kt) {
                const uint32_t lo = biased<CT>(y[2 * kt]), hi = biased<CT>(y[2 * kt + 1]);
                uint32_t a[4];
                a[0] = widen2<CT>(lo, 0x4240);
                a[1] = widen2<CT>(lo, 0x4341);
                a[2] = widen2<CT>(hi, 0x4240);
                a[3] = widen2<CT>(hi, 0x4341);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    Ops::mma(acc[nt][md], a, pb[nt][kt][0], pb[nt][kt][1]);
                    if constexpr (kTwoTerms) Ops::mma(acc[nt][md], a, pl[nt][kt][0], pl[nt][kt][1]);
                }
            }
        }
        slot = slot + 1 == NST ? 0 : slot + 1;

        const bool ends = now.k + 1 == now.stages;
        if (ends || i + 1 == count) {
            // ---- the item ends, or the piece does
            const bool done = whole && ends;
            // where it began in this piece it is the piece's last, else its first
            float* part = p.parts + ((size_t)(blockIdx.x * W + warp) * 2 + (whole ? 1 : 0)) * S::kRows * (D + 2);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float l = l_run[nt][j];
                    l += __shfl_xor_sync(0xffffffffu, l, 4);
                    l += __shfl_xor_sync(0xffffffffu, l, 8);
                    l += __shfl_xor_sync(0xffffffffu, l, 16);
                    const int r = 8 * nt + 2 * t4 + j;
                    if (r >= rows) continue;
                    const float fall = weight_fall(w_ref[nt][j]);
                    constexpr float kBack = kFp8 ? 256.f : 1.f;                // (apart: their product may pass the largest number)
                    if (done) {
                        const int row = row0 + r, token = row / G;
                        const size_t at = ((size_t)(now.q0 + token) * p.num_q_heads + kvh * G + row - token * G) * D;
                        const float inv = __fdiv_rn(fall, l);
#pragma unroll
                        for (int md = 0; md < KS; ++md)
                            store_pair(p, at + 16 * md + 2 * g, acc[nt][md][j] * kBack * inv, acc[nt][md][2 + j] * kBack * inv);
                    } else {
#pragma unroll
                        for (int md = 0; md < KS; ++md)
                            *reinterpret_cast<float2*>(part + r * D + 16 * md + 2 * g) = make_float2(acc[nt][md][j] * kBack * fall, acc[nt][md][2 + j] * kBack * fall);
                        if (g == 0) {
                            part[S::kRows * D + r] = m_ref[nt][j];
                            part[S::kRows * (D + 1) + r] = l;
                        }
                    }
                }
            __syncwarp();
        }
        now.next(p);
    }
    cp_async_wait<0>();
}

// Joins an item's pieces, a CTA for an item (or for some of its rows, where there are few
// items). Few pieces: a warp a row. Many (a long context alone on the device): all warps a
// row, and one of them joins their sums.
// (Its warps: one for each row of a batch's items, sixteen where few items have many pieces.)
constexpr int kScaledJoinWarps = 16;
constexpr int kScaledFewPieces = 16;

template <int D, int NT>
__global__ void __launch_bounds__(kScaledJoinWarps * 32)
scaled_join_kernel(const __grid_constant__ ScaledAttnParams p) {
    begin_overlapped();
    constexpr int ROWS = 8 * NT;
    constexpr int E = D / 32;                      // a lane's components, neighbours
    const int W = blockDim.x >> 5;
    __shared__ float s_max[kScaledJoinWarps], s_sum[kScaledJoinWarps];
    __shared__ float s_out[kScaledJoinWarps][D];
    const int s = blockIdx.y, item = blockIdx.x;
    // all that says where the pieces lie, in one round of loads
    const int64_t before = p.stages_before[s], after = p.stages_before[s + 1], total = p.stages_before[p.num_seqs];
    int L, q0, Q;
    const bool fine = scaled_sequence(p, s, false, L, q0, Q);
    const int stages = (int)(after - before);
    if (stages == 0 || !fine) return;
    const int64_t line = total * p.items;
    const int64_t piece = scaled_piece(line, p.workers);
    const int64_t first = before * p.items + (int64_t)item * stages;
    int64_t w0, w1;
    if (line < INT32_MAX) {
        w0 = (uint32_t)first / (uint32_t)piece;
        w1 = (uint32_t)(first + stages - 1) / (uint32_t)piece;
    } else {
        w0 = first / piece;
        w1 = (first + stages - 1) / piece;
    }
    if (w0 == w1) return;                          // whole, and written
    const int n = (int)(w1 - w0) + 1;
    const int kvh = item / p.row_tiles, row0 = (item - kvh * p.row_tiles) * ROWS;
    const int rows = min(ROWS, Q * p.group - row0);
    // the first piece of the item lies last among its warp's, the others first
    auto piece_of = [&](int i) { return p.parts + ((size_t)(w0 + i) * 2 + (i == 0 ? 1 : 0)) * ROWS * (D + 2); };
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // pieces i0, i0 + step, ..: their maximum, and sums under it; eight at a time, whose
    // loads are in flight together
    constexpr int kAtOnce = 8;
    auto gather = [&](int r, int i0, int step, float& M, float& sum, float (&o)[E]) {
        M = -INFINITY;
        sum = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = 0.f;
        for (int i = i0; i < n; i += kAtOnce * step) {
            float m[kAtOnce], l[kAtOnce], v[kAtOnce][E];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                m[k] = -INFINITY;
                l[k] = 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e) v[k][e] = 0.f;
                if (i + k * step < n) {
                    const float* part = piece_of(i + k * step);
                    m[k] = part[ROWS * D + r];
                    l[k] = part[ROWS * (D + 1) + r];
                    RowLoader<float, E>::load(part + r * D + lane * E, v[k]);
                }
            }
            float most = M;
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) most = fmaxf(most, m[k]);
            const float was = M == -INFINITY ? (sum == 0.f ? 0.f : 1.f) : fast_exp2(M - most);
            M = most;
            sum *= was;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] *= was;
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const float f = m[k] == -INFINITY ? (l[k] == 0.f ? 0.f : 1.f) : fast_exp2(m[k] - M);
                sum = fmaf(f, l[k], sum);
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] = fmaf(f, v[k][e], o[e]);
            }
        }
    };
    auto store = [&](int r, float sum, const float (&o)[E]) {
        const float inv = __fdiv_rn(1.f, sum);
        const int row = row0 + r, token = row / p.group, head = kvh * p.group + row - token * p.group;
        const size_t at = ((size_t)(q0 + token) * p.num_q_heads + head) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; e += 2) store_pair(p, at + e, o[e] * inv, o[e + 1] * inv);
    };
    float M, sum, o[E];
    if (n <= kScaledFewPieces) {
        for (int r = blockIdx.z * W + warp; r < rows; r += gridDim.z * W) {
            gather(r, 0, 1, M, sum, o);
            store(r, sum, o);
        }
        return;
    }
    for (int r = blockIdx.z; r < rows; r += gridDim.z) {
        gather(r, warp, W, M, sum, o);
        __syncthreads();                           // the row before has been read
        if (lane == 0) {
            s_max[warp] = M;
            s_sum[warp] = sum;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) s_out[warp][lane * E + e] = o[e];
        __syncthreads();
        if (warp == 0) {
            float most = -INFINITY;
            for (int w = 0; w < W; ++w) most = fmaxf(most, s_max[w]);
            sum = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll 4
            for (int w = 0; w < W; ++w) {
                const float f = s_max[w] == -INFINITY ? (s_sum[w] == 0.f ? 0.f : 1.f) : fast_exp2(s_max[w] - most);
                sum = fmaf(f, s_sum[w], sum);
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] = fmaf(f, s_out[w][lane * E + e], o[e]);
            }
            store(r, sum, o);
        }
    }
}

template <typename CT, int D, int NT, bool kTwoTerms>
cudaError_t launch_scaled_rows(const ScaledAttnParams& p, cudaStream_t stream) {
    using S = ScaledShape<D, NT>;
    constexpr int W = scaled_warps(D, 8 * NT);
    auto kernel = scaled_attention_kernel<CT, D, NT, W, kTwoTerms>;
    cudaError_t e = ensure_smem_attribute(reinterpret_cast<const void*>(kernel), W * S::kWarpBytes);
    if (e != cudaSuccess) return e;
    e = launch_overlapped(kernel, p, dim3(p.workers / W), W * 32, W * S::kWarpBytes, stream);
    if (e != cudaSuccess) return e;
    const int64_t all = (int64_t)p.items * p.num_seqs;
    const int64_t rows = (int64_t)p.max_queries * p.group < 8 * NT ? (int64_t)p.max_queries * p.group : 8 * NT;
    const bool batch = all >= 152;
    const int warps = batch ? (int)(rows < 8 ? rows : 8) : kScaledJoinWarps;
    return launch_overlapped(scaled_join_kernel<D, NT>, p, dim3(p.items, p.num_seqs, batch ? 1 : (unsigned)rows), warps * 32, 0, stream);
}

// Up to 32 rows a tile; by the output's type (a file for each, scaled_attention_*.cu).
template <typename CT, bool kTwoTerms>
cudaError_t launch_scaled_warps(const ScaledAttnParams& p, int head_size, cudaStream_t stream) {
    auto rows = [&](auto d) -> cudaError_t {
        constexpr int D = decltype(d)::value;
        if (p.tile_rows == 8) return launch_scaled_rows<CT, D, 1, kTwoTerms>(p, stream);
        if (p.tile_rows == 16) return launch_scaled_rows<CT, D, 2, kTwoTerms>(p, stream);
        if constexpr (D < 256)
            if (p.tile_rows == 32) return launch_scaled_rows<CT, D, 4, kTwoTerms>(p, stream);
        return cudaErrorInvalidValue;
    };
    switch (head_size) {
    case 64: return rows(std::integral_constant<int, 64>{});
    case 128: return rows(std::integral_constant<int, 128>{});
    case 256: return rows(std::integral_constant<int, 256>{});
    }
    return cudaErrorInvalidValue;
}

}  // namespace pagedkv
