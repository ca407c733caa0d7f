// sparse_select.cu -- which blocks a block-sparse decode reads. For a sequence
// of n blocks and each KV head h,
//     score(b) = max over the group's query heads g of
//                sum_d max(q_gd lo_bd, q_gd hi_bd),
// the largest value q_g . k can take for keys within block b's bounds. The
// first `first_blocks` and the newest `recent_blocks` blocks are always taken;
// of the others the num_select - first - recent of largest score (ties: the
// lowest index; a NaN score counts as +infinity, so that a NaN key is read and
// shows, as it would in the dense decode). n <= num_select: every block.
//
// The result is defined by the exact order of the scores. Almost every block's
// place is clear at far lower precision, so there are two steps:
//  - approximate scores on warp-level MMAs. max(q lo, q hi) = min(q,0) lo +
//    max(q,0) hi, so a block's scores for all heads are one product of its
//    bounds, read as one row of 2 D elements, with the query's two sides:
//    16 blocks x 2 D by 2 D x 8 heads. The products are exact in binary32; the
//    sums are taken to err by at most kScoreEps times sum |q_d bound_d|, which
//    a second product of the magnitudes gives.
//  - the threshold among those scores. Blocks whose distance to the other side
//    of it exceeds both errors are settled; the rest (usually none) are scored
//    again in binary64 and ranked.
// A cluster of CTAs takes one (sequence, KV head): all score, into the first
// CTA's shared memory, and the first one selects. Reading the bounds once
// (2 D elements per block) bounds the kernel for batches, the latency of the
// score-search-emit chain for few rows.
//
// The selection goes out as a table of slabs (block * Hkv + head) in ascending
// block order, so that only its last block, the newest, can be partial: the
// paged decode reads it as a block table of S * Hkv one-head sequences.
#include <cooperative_groups.h>

#include "decode_mma.cuh"
#include "launch.h"

namespace pagedkv {

namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kRankList = 256;          // ambiguous blocks ranked in shared memory
// Keys of up to this many blocks are kept in shared memory (two CTAs per SM);
// longer contexts' in the workspace.
constexpr int kSmemKeys = 24 * 1024;
// |approximate - exact score| <= kScoreEps * sum_d |q_d bound_d|: 2 D <= 512
// terms, each addition off by at most 2^-23 of the sum of magnitudes.
constexpr float kScoreEps = 6.2e-5f;    // > 2^-14

// The sequence's length as the decode takes it (clamped to what the table and
// the bound allow).
__device__ __forceinline__ int clamped_len(const SelectParams& p, int s, bool& bad) {
    const int L = p.context_lens[s];
    const int64_t tab = (int64_t)p.max_blocks * p.block_size;
    const int cap = tab < p.max_context_len ? (int)tab : p.max_context_len;
    bad = L < 0 || L > cap;
    return L < 0 ? 0 : (L > cap ? cap : L);
}

__device__ __forceinline__ uint32_t ordered(float x) {        // the order of the values
    const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);   // -0 and 0 are one value
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint64_t ordered64(double x) {
    const uint64_t u = (uint64_t)__double_as_longlong(x == 0.0 ? 0.0 : x);
    return u >> 63 ? ~u : u | (1ull << 63);
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The two sides of eight query elements: min(x, 0) or max(x, 0), NaN kept.
template <typename T>
__device__ __forceinline__ uint32_t side2(uint32_t w, bool positive) {
    if constexpr (std::is_same<T, __half>::value) {
        const __half2 x = *reinterpret_cast<const __half2*>(&w);
        const __half2 z = __float2half2_rn(0.f);
        const __half2 y = positive ? __hmax2_nan(x, z) : __hmin2_nan(x, z);
        return *reinterpret_cast<const uint32_t*>(&y);
    } else {
        const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&w);
        const __nv_bfloat162 z = __float2bfloat162_rn(0.f);
        const __nv_bfloat162 y = positive ? __hmax2_nan(x, z) : __hmin2_nan(x, z);
        return *reinterpret_cast<const uint32_t*>(&y);
    }
}

// The exact score of a block in binary64, by one warp.
template <typename T, int D>
__device__ double exact_score(const SelectParams& p, int s, int h, int64_t blk, int lane) {
    constexpr int E = D / 32;
    if (blk < 0 || blk >= p.num_blocks) return -INFINITY;
    const T* bounds = static_cast<const T*>(p.k_bounds) + ((size_t)blk * p.num_kv_heads + h) * 2 * D + lane * E;
    float lo[E], hi[E], q[E];
    RowLoader<T, E>::load(bounds, lo);
    RowLoader<T, E>::load(bounds + D, hi);
    double best = -INFINITY;
    for (int g = 0; g < p.group; ++g) {
        RowLoader<T, E>::load(static_cast<const T*>(p.query) +
                              ((size_t)s * p.num_q_heads + h * p.group + g) * D + lane * E, q);
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < E; ++i) sum += (double)q[i] * (double)(q[i] < 0.f ? lo[i] : hi[i]);
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
        if (isnan(sum)) sum = INFINITY;
        best = sum > best ? sum : best;
    }
    return best;
}

struct SelShared {
    float err[kMaxCluster];             // per CTA: the largest sum of magnitudes
    int part[2][kSelWarps];             // count(): per-warp sums, double-buffered
    float fpart[2][kSelWarps];
    int list_n;
    int list[kRankList];
    uint64_t list_key[kRankList];
};

// Sum over the CTA; one barrier (`turn` alternates the buffer).
__device__ __forceinline__ int cta_sum(SelShared& sh, int x, int& turn) {
    const int w = __reduce_add_sync(0xffffffffu, x);
    if ((threadIdx.x & 31) == 0) sh.part[turn][threadIdx.x >> 5] = w;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    const int y = __reduce_add_sync(0xffffffffu, lane < kSelWarps ? sh.part[turn][lane] : 0);
    turn ^= 1;
    return y;
}

// The largest P with count(key >= P) >= want over the candidates that `key`
// gives (i strided over the threads; skip(i) leaves one out). exact: whether
// count(key >= P) == want.
template <typename K, typename Key, typename Skip>
__device__ __forceinline__ K kth_largest(SelShared& sh, int n, int want, int& turn, bool& exact,
                                         Key key, Skip skip) {
    K prefix = 0;
    exact = false;
    for (int bit = (int)sizeof(K) * 8 - 1; bit >= 0; --bit) {
        const K cand = prefix | ((K)1 << bit);
        int c = 0;
        for (int i = threadIdx.x; i < n; i += kSelThreads) c += !skip(i) && key(i) >= cand;
        const int total = cta_sum(sh, c, turn);
        if (total >= want) prefix = cand;
        if (total == want) {
            exact = true;
            break;
        }
    }
    return prefix;
}

template <typename T, int D>
__global__ void __launch_bounds__(kSelThreads, 2)
select_blocks_kernel(const __grid_constant__ SelectParams p) {
    constexpr int STEPS = 2 * D / 32;                          // 64-byte steps of a bounds row (16-bit types)
    extern __shared__ __align__(16) uint8_t dyn[];
    __shared__ SelShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks();
    const int rank = (int)cluster.block_rank();
    const int row = blockIdx.x / C;
    const int s = row / p.num_kv_heads;
    const int h = row - s * p.num_kv_heads;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    bool bad;
    const int L = clamped_len(p, s, bad);
    if (bad && h == 0 && rank == 0 && threadIdx.x == 0 && p.status) atomicOr(p.status, PA_DEV_BAD_LEN);
    const int B = p.block_size;
    const int n = (L + B - 1) / B;
    const int32_t* table = p.block_tables + (size_t)s * p.max_blocks;
    const bool all = n <= p.num_select;
    const int want = p.num_select - p.first_blocks - p.recent_blocks;
    const int lo = p.first_blocks;
    const int nc = all ? 0 : n - p.recent_blocks - lo;         // candidates lo .. lo + nc - 1

    uint4* sides = reinterpret_cast<uint4*>(dyn);              // [n-tile][step][lane]
    const int ntiles = (p.group + 7) / 8;
    float* keys = p.keys_in_smem ? reinterpret_cast<float*>(dyn + p.side_bytes)
                                 : p.scores + (size_t)row * p.max_ctx_blocks;

    if (nc > 0 && want > 0) {
        // ------------------------------------------------ approximate scores
        cluster.sync();                                        // the first CTA runs: its memory may be written
        float* out_keys = p.keys_in_smem ? cluster.map_shared_rank(keys, 0) : keys;
        float worst = 0.f;
        if constexpr (std::is_same<T, float>::value) {
            constexpr int E = D / 32;
            for (int i = rank * kSelWarps + warp; i < nc; i += C * kSelWarps) {
                const int64_t blk = table[lo + i];
                float best = -INFINITY;
                if (blk >= 0 && blk < p.num_blocks) {
                    const float* bounds = static_cast<const float*>(p.k_bounds) +
                                          ((size_t)blk * p.num_kv_heads + h) * 2 * D + lane * E;
                    float bl[E], bh[E], q[E];
                    RowLoader<float, E>::load(bounds, bl);
                    RowLoader<float, E>::load(bounds + D, bh);
                    for (int g = 0; g < p.group; ++g) {
                        RowLoader<float, E>::load(static_cast<const float*>(p.query) +
                                                  ((size_t)s * p.num_q_heads + h * p.group + g) * D + lane * E, q);
                        float sum = 0.f, mag = 0.f;
#pragma unroll
                        for (int j = 0; j < E; ++j) {
                            const float t = q[j] * (q[j] < 0.f ? bl[j] : bh[j]);
                            sum += t;
                            mag += fabsf(t);
                        }
#pragma unroll
                        for (int m = 16; m > 0; m >>= 1) {
                            sum += __shfl_xor_sync(0xffffffffu, sum, m);
                            mag += __shfl_xor_sync(0xffffffffu, mag, m);
                        }
                        best = fmaxf(best, sum);
                        worst = max_nan(worst, mag);
                    }
                }
                if (lane == 0) out_keys[i] = best;
            }
        } else {
            using Ops = MmaOps<T>;
            for (int i = threadIdx.x; i < ntiles * STEPS * 32; i += kSelThreads) {
                const int l = i & 31, j = (i >> 5) % STEPS, nt = i / (32 * STEPS);
                const int g = nt * 8 + (l >> 2);
                const int e = 32 * j + 8 * (l & 3);
                const bool positive = e >= D;
                uint4 w = make_uint4(0, 0, 0, 0);
                if (g < p.group) {
                    w = *reinterpret_cast<const uint4*>(
                        static_cast<const T*>(p.query) +
                        ((size_t)s * p.num_q_heads + h * p.group + g) * D + (positive ? e - D : e));
                    w = make_uint4(side2<T>(w.x, positive), side2<T>(w.y, positive),
                                   side2<T>(w.z, positive), side2<T>(w.w, positive));
                }
                sides[i] = w;
            }
            __syncthreads();
            const int g = lane >> 2, t4 = lane & 3;
            const int tiles = (nc + 15) / 16;
            for (int tile = rank * kSelWarps + warp; tile < tiles; tile += C * kSelWarps) {
                // this lane's rows: blocks g and g + 8 of the tile
                const T* src[2];
                bool there[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int i = tile * 16 + g + 8 * r;
                    const int64_t blk = table[lo + (i < nc ? i : nc - 1)];
                    there[r] = blk >= 0 && blk < p.num_blocks;
                    src[r] = static_cast<const T*>(p.k_bounds) +
                             ((size_t)(there[r] ? blk : 0) * p.num_kv_heads + h) * 2 * D + 8 * t4;
                }
                float best[2] = {-INFINITY, -INFINITY}, mag[2] = {0.f, 0.f};
                for (int nt = 0; nt < ntiles; ++nt) {
                    float c[4] = {0.f, 0.f, 0.f, 0.f}, m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int j0 = 0; j0 < STEPS; j0 += 4) {
                        constexpr int U = 4;
                        uint4 x[U], y[U];
#pragma unroll
                        for (int j = 0; j < U; ++j) {
                            x[j] = __ldg(reinterpret_cast<const uint4*>(src[0] + 32 * (j0 + j)));
                            y[j] = __ldg(reinterpret_cast<const uint4*>(src[1] + 32 * (j0 + j)));
                        }
#pragma unroll
                        for (int j = 0; j < U; ++j) {
                            const uint4 q = sides[(nt * STEPS + j0 + j) * 32 + lane];
                            constexpr uint32_t kAbs = 0x7fff7fffu;
                            const uint32_t a0[4] = {x[j].x, y[j].x, x[j].y, y[j].y};
                            const uint32_t a1[4] = {x[j].z, y[j].z, x[j].w, y[j].w};
                            Ops::mma(c, a0, q.x, q.y);
                            Ops::mma(c, a1, q.z, q.w);
                            const uint32_t b0[4] = {x[j].x & kAbs, y[j].x & kAbs, x[j].y & kAbs, y[j].y & kAbs};
                            const uint32_t b1[4] = {x[j].z & kAbs, y[j].z & kAbs, x[j].w & kAbs, y[j].w & kAbs};
                            Ops::mma(m, b0, q.x & kAbs, q.y & kAbs);
                            Ops::mma(m, b1, q.z & kAbs, q.w & kAbs);
                        }
                    }
                    // this lane: heads 2 t4 and 2 t4 + 1 of blocks g and g + 8
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (nt * 8 + 2 * t4 + e < p.group) {
                                best[r] = fmaxf(best[r], c[2 * r + e]);
                                mag[r] = max_nan(mag[r], m[2 * r + e]);
                            }
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 1));
                    best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 2));
                    const int i = tile * 16 + g + 8 * r;
                    if (there[r]) worst = max_nan(worst, mag[r]);
                    if (t4 == 0 && i < nc) out_keys[i] = there[r] ? best[r] : -INFINITY;
                }
            }
        }
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) worst = max_nan(worst, __shfl_xor_sync(0xffffffffu, worst, m));
        if (lane == 0) sh.fpart[0][warp] = worst;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < kSelWarps; ++w) worst = max_nan(worst, sh.fpart[0][w]);
            *cluster.map_shared_rank(&sh.err[rank], 0) = worst;
        }
    }
    cluster.sync();
    if (rank != 0) return;

    int turn = 0;
    uint32_t thr = 0;                                          // taken candidates: ordered(key) >= thr
    if (nc > 0 && want > 0) {
        float mag = 0.f;
        for (int r = 0; r < C; ++r) mag = max_nan(mag, sh.err[r]);
        const double err2 = 2.0 * (double)kScoreEps * (double)mag;
        const bool finite = isfinite(mag);
        // Settled blocks: those that beat (or lose to) every block on the other
        // side of the threshold by more than both errors. in_above: taken for
        // certain above it; out_below: left out for certain below it.
        double in_above = INFINITY, out_below = -INFINITY;
        if (finite) {
            bool exact;
            thr = kth_largest<uint32_t>(sh, nc, want, turn, exact, [&](int i) { return ordered(keys[i]); },
                                        [](int) { return false; });
            float a = INFINITY, b = -INFINITY;                 // the smallest taken, the largest left out
            for (int i = threadIdx.x; i < nc; i += kSelThreads) {
                const float k = keys[i];
                if (ordered(k) >= thr) a = fminf(a, k);
                else b = fmaxf(b, k);
            }
#pragma unroll
            for (int m = 16; m > 0; m >>= 1) {
                a = fminf(a, __shfl_xor_sync(0xffffffffu, a, m));
                b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, m));
            }
            if (lane == 0) {
                sh.fpart[0][warp] = a;
                sh.fpart[1][warp] = b;
            }
            __syncthreads();
            for (int w = 0; w < kSelWarps; ++w) {
                a = fminf(a, sh.fpart[0][w]);
                b = fmaxf(b, sh.fpart[1][w]);
            }
            if (!exact) b = a;                                 // equal keys across the threshold
            in_above = (double)b + err2;
            out_below = (double)a - err2;
        }
        const float kOut = __uint_as_float(0xffffffffu);       // ordered() puts it below every value
        auto settled = [&](float k) { return finite && ((double)k > in_above || (double)k < out_below); };
        // count the certain ones and the unsettled
        int in = 0, open = 0;
        for (int i = threadIdx.x; i < nc; i += kSelThreads) {
            const float k = keys[i];
            if (!settled(k)) ++open;
            else in += (double)k > in_above;
        }
        in = cta_sum(sh, in, turn);
        open = cta_sum(sh, open, turn);
        const int left = want - in;                            // places for the unsettled
        if (!finite) thr = ordered(INFINITY);
        if (left < open) {
            // ------------------------------------------- exact scores of the unsettled
            const bool small = open <= kRankList;
            if (threadIdx.x == 0) sh.list_n = 0;
            __syncthreads();
            uint64_t* exact_keys = p.exact_keys + (size_t)row * p.max_ctx_blocks;
            for (int i0 = warp * 32; i0 < nc; i0 += kSelThreads) {
                const bool mine = i0 + lane < nc && !settled(keys[i0 + lane]);
                uint32_t votes = __ballot_sync(0xffffffffu, mine);
                while (votes) {
                    const int i = i0 + __ffs(votes) - 1;
                    votes &= votes - 1;
                    const uint64_t k = ordered64(exact_score<T, D>(p, s, h, table[lo + i], lane));
                    if (lane == 0) {
                        if (small) {
                            const int at = atomicAdd(&sh.list_n, 1);
                            sh.list[at] = i;
                            sh.list_key[at] = k;
                        } else {
                            exact_keys[i] = k;
                        }
                    }
                }
            }
            __syncthreads();
            if (small) {
                // the list's order varies, the ranks do not: (key, index) differ in every pair
                const int e = threadIdx.x;
                if (e < open) {
                    const uint64_t k = sh.list_key[e];
                    const int i = sh.list[e];
                    int before = 0;
                    for (int o = 0; o < open; ++o)
                        before += sh.list_key[o] > k || (sh.list_key[o] == k && sh.list[o] < i);
                    keys[i] = before < left ? INFINITY : kOut;
                }
            } else if (left > 0) {
                bool exact;
                const uint64_t t = kth_largest<uint64_t>(
                    sh, nc, left, turn, exact, [&](int i) { return exact_keys[i]; },
                    [&](int i) { return settled(keys[i]); });
                int above = 0;
                for (int i = threadIdx.x; i < nc; i += kSelThreads)
                    above += !settled(keys[i]) && exact_keys[i] > t;
                above = cta_sum(sh, above, turn);
                int ties = exact ? 0x7fffffff : left - above;  // places for keys equal to t, lowest first
                for (int i0 = 0; i0 < nc; i0 += kSelThreads) {
                    const int i = i0 + threadIdx.x;
                    const bool mine = i < nc && !settled(keys[i]);
                    const uint64_t k = mine ? exact_keys[i] : 0;
                    const bool tie = mine && k == t;
                    const uint32_t votes = __ballot_sync(0xffffffffu, tie);
                    if (lane == 0) sh.part[turn][warp] = __popc(votes);
                    __syncthreads();
                    int at = __popc(votes & ((1u << lane) - 1)), total = 0;
                    for (int w = 0; w < kSelWarps; ++w) {
                        if (w < warp) at += sh.part[turn][w];
                        total += sh.part[turn][w];
                    }
                    turn ^= 1;
                    if (mine) keys[i] = k > t || (tie && at < ties) ? INFINITY : kOut;
                    if (!exact) ties -= total < ties ? total : ties;
                }
            } else {
                for (int i = threadIdx.x; i < nc; i += kSelThreads)
                    if (!settled(keys[i])) keys[i] = kOut;
            }
            __syncthreads();
        } else {
            // every unsettled block is taken: they are the candidates from out_below on
            for (int i = threadIdx.x; i < nc; i += kSelThreads)
                if (!settled(keys[i])) keys[i] = INFINITY;
            __syncthreads();
        }
    }

    // -------------------------------------------------------- emit in block order
    int32_t* slabs = p.slab_tables + (size_t)row * p.table_width;
    int32_t* out = p.selected ? p.selected + (size_t)row * p.num_select : nullptr;
    auto taken = [&](int b) {
        if (b >= n) return false;
        if (all || b < lo || b >= lo + nc) return true;
        return want > 0 && ordered(keys[b - lo]) >= thr;
    };
    const int span = ((n + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;   // blocks per warp
    const int b_lo = warp * span, b_hi = min(b_lo + span, n);
    int mine = 0;
    for (int b = b_lo + lane; b < b_hi; b += 32) mine += taken(b);
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (lane == 0) sh.part[turn][warp] = mine;
    __syncthreads();
    int at = 0, total = 0;
    for (int w = 0; w < kSelWarps; ++w) {
        if (w < warp) at += sh.part[turn][w];
        total += sh.part[turn][w];
    }
    for (int b0 = b_lo; b0 < b_hi; b0 += 32) {
        const int b = b0 + lane;
        const bool take = b < b_hi && taken(b);
        const uint32_t votes = __ballot_sync(0xffffffffu, take);
        const int to = at + __popc(votes & ((1u << lane) - 1));
        if (take && to < p.table_width) {
            const int64_t blk = table[b];
            slabs[to] = blk >= 0 && blk < p.num_blocks ? (int32_t)(blk * p.num_kv_heads + h) : -1;
            if (out) out[to] = b;
        }
        at += __popc(votes);
    }
    if (threadIdx.x == 0) p.slab_lens[row] = total * B - (n * B - L);   // total = min(n, num_select)
    if (out)
        for (int i = total + threadIdx.x; i < p.num_select; i += kSelThreads) out[i] = -1;
}

template <typename T, int D>
cudaError_t launch_select(SelectParams p, cudaStream_t stream) {
    const int rows = p.num_seqs * p.num_kv_heads;
    // CTAs per row: enough for two on each of 152 SMs, each with a tile of 16
    // blocks per warp or more
    int C = 1;
    while (C < 8 && rows * C < 304 && p.max_ctx_blocks >= 2 * C * kSelWarps * 16) C *= 2;
    const int ntiles = (p.group + 7) / 8;
    p.side_bytes = std::is_same<T, float>::value ? 0 : ntiles * (2 * D / 32) * 512;
    const bool scored = p.max_ctx_blocks > p.num_select;
    p.keys_in_smem = p.max_ctx_blocks <= kSmemKeys && p.side_bytes <= 96 * 1024;
    if (p.side_bytes > 200 * 1024) return cudaErrorInvalidValue;
    const int smem = scored ? p.side_bytes + (p.keys_in_smem ? p.max_ctx_blocks * 4 : 0) : 0;
    auto kernel = select_blocks_kernel<T, D>;
    cudaError_t e = ensure_smem_attribute(reinterpret_cast<const void*>(kernel), 200 * 1024);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(rows * C);
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {(unsigned)C, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
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
