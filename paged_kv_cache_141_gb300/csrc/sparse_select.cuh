// sparse_select.cuh -- which blocks a block-sparse decode reads. For a sequence
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
//  - the threshold among those scores, from a histogram over their range.
//    Blocks whose distance to the other side of the threshold exceeds both
//    errors are settled; the rest (usually none) are scored again exactly and
//    ranked. Where the histogram's bin at the threshold holds too many
//    blocks (equal scores) or a score is not finite, a search over the key
//    bits takes its place.
// A cluster of CTAs takes one (sequence, KV head): all score, into the first
// CTA's shared memory, and the first one selects. Reading the bounds once
// (2 D elements per block) bounds the kernel for batches, the latency of the
// score-search-emit chain for few rows.
//
// Shared by the fused kernel (sparse_decode.cuh) and the selection kernel whose
// slab tables the paged decode reads (sparse_select.cu).
#pragma once

#include <cooperative_groups.h>

#include "decode_mma.cuh"
#include "launch.h"

namespace pagedkv {

namespace cg = cooperative_groups;

constexpr int kMaxCluster = 8;         // the portable size
// Keys of up to this many blocks are kept in shared memory (two CTAs per SM);
// longer contexts' in the workspace.
constexpr int kSmemKeys = 24 * 1024;
// |approximate - exact score| <= kScoreEps * sum_d |q_d bound_d|. An MMA adds 16
// exact products to its accumulator; taking each of the 17 terms to lose up to
// 2^-23 of the largest, a chain of four MMAs errs by at most 4 * 17 * 2^-23 of
// its own terms' magnitudes, and so do all chains together (chains are joined
// in binary32, eight additions at most). That is below 2^-16.8; 2^-16 leaves a
// factor of 1.7. Binary32 queries (a sum of 8 + 5 terms a lane and across) are
// well inside it. How an MMA rounds inside is not documented; measured over all
// types and head sizes (normal values, magnitudes spread over 2^16, one sign, sums
// that cancel; 25,000 blocks each) the largest error is 2^-21.1 of the sum, a
// thirtieth of this.
constexpr float kScoreEps = 1.0f / 65536;

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

// The two sides of a pair of query elements: min(x, 0) or max(x, 0), NaN kept;
// bfloat16 ones times 2^40, so that products of bfloat16's small numbers stay
// above binary32's smallest (binary16's do).
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
        const __nv_bfloat162 y = __hmul2(positive ? __hmax2_nan(x, z) : __hmin2_nan(x, z),
                                         __float2bfloat162_rn(0x1p40f));
        return *reinterpret_cast<const uint32_t*>(&y);
    }
}

// A block's score for one head of the group, by one warp, as an ordered key (NaN
// as +infinity): the exact sum where a pair of binary32 numbers holds it, else
// the sum in binary64. Products of 16-bit types are exact in binary32, and the
// pair (Knuth's two-sum, for the sum and for its collected errors) says by
// itself whether anything was lost; with 48 bits that is rare, and binary64
// runs at a small fraction of binary32's rate on this GPU.
template <typename T, int D>
__device__ uint64_t exact_head_score(const SelectParams& p, int s, int h, int g, int64_t blk, int lane) {
    constexpr int E = D / 32;
    if (blk < 0 || blk >= p.num_blocks) return ordered64(-INFINITY);
    const T* bounds = static_cast<const T*>(p.k_bounds) + ((size_t)blk * p.num_kv_heads + h) * 2 * D + lane * E;
    float lo[E], hi[E], q[E];
    RowLoader<T, E>::load(bounds, lo);
    RowLoader<T, E>::load(bounds + D, hi);
    RowLoader<T, E>::load(static_cast<const T*>(p.query) +
                          ((size_t)s * p.num_q_heads + h * p.group + g) * D + lane * E, q);
    if constexpr (!std::is_same<T, float>::value) {
        float sum = 0.f, err = 0.f;
        bool lost = false;
        // a + b = t + two_sum's result, exactly
        auto two_sum = [](float a, float b, float& t) {
            t = __fadd_rn(a, b);
            const float z = __fsub_rn(t, a);
            return __fadd_rn(__fsub_rn(a, __fsub_rn(t, z)), __fsub_rn(b, z));
        };
        auto collect = [&](float e) { lost |= two_sum(err, e, err) != 0.f; };
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const float b = q[i] < 0.f ? lo[i] : hi[i];
            const float x = __fmul_rn(q[i], b);
            lost |= !(fabsf(x) > 0x1p-100f && fabsf(x) < INFINITY) && q[i] != 0.f && b != 0.f;   // may be inexact
            collect(two_sum(sum, x, sum));
        }
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) {
            const float s2 = __shfl_xor_sync(0xffffffffu, sum, m);
            const float e2 = __shfl_xor_sync(0xffffffffu, err, m);
            collect(two_sum(sum, s2, sum));
            collect(e2);
        }
        // (an infinity or a NaN anywhere leaves NaN errors: lost)
        if (!__any_sync(0xffffffffu, lost)) return ordered64((double)sum + (double)err);
    }
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < E; ++i) sum += (double)q[i] * (double)(q[i] < 0.f ? lo[i] : hi[i]);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    return ordered64(isnan(sum) ? INFINITY : sum);
}

// The same over all heads of the group.
template <typename T, int D>
__device__ uint64_t exact_score(const SelectParams& p, int s, int h, int64_t blk, int lane) {
    uint64_t best = 0;
    for (int g = 0; g < p.group; ++g) {
        const uint64_t x = exact_head_score<T, D>(p, s, h, g, blk, lane);
        best = x > best ? x : best;
    }
    return best;
}

// Sixteen blocks' bounds rows, four 64-byte steps (a quarter: 128 elements) at
// a time: this lane's 16-byte chunks of blocks g and g + 8.
struct Quarter {
    uint4 x[4], y[4];
    template <typename T>
    __device__ __forceinline__ void load(const T* x_row, const T* y_row) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[j] = *reinterpret_cast<const uint4*>(x_row + 32 * j);
            y[j] = *reinterpret_cast<const uint4*>(y_row + 32 * j);
        }
    }
};

// Adds a quarter's products with the query sides (this lane's chunks, 32 lanes
// apart) to the scores c and magnitudes m: lane (g, t4) holds blocks g and
// g + 8, heads 2 t4 and 2 t4 + 1. A lane's eight consecutive elements stand
// for k = 2 t4, 2 t4 + 1, 2 t4 + 8, 2 t4 + 9 of two MMAs, in the bounds and the
// sides alike, so both are loaded as 16-byte vectors.
template <typename T>
__device__ __forceinline__ void add_quarter(const Quarter& b, const uint4* sides, float (&c)[4],
                                            float (&m)[4]) {
    using Ops = MmaOps<T>;
    constexpr uint32_t kAbs = 0x7fff7fffu;
    float c0[4] = {0.f, 0.f, 0.f, 0.f}, c1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint4 q = sides[32 * j];
        const uint32_t a0[4] = {b.x[j].x, b.y[j].x, b.x[j].y, b.y[j].y};
        const uint32_t a1[4] = {b.x[j].z, b.y[j].z, b.x[j].w, b.y[j].w};
        Ops::mma(c0, a0, q.x, q.y);
        Ops::mma(c1, a1, q.z, q.w);
        const uint32_t b0[4] = {a0[0] & kAbs, a0[1] & kAbs, a0[2] & kAbs, a0[3] & kAbs};
        const uint32_t b1[4] = {a1[0] & kAbs, a1[1] & kAbs, a1[2] & kAbs, a1[3] & kAbs};
        Ops::mma(m, b0, q.x & kAbs, q.y & kAbs);
        Ops::mma(m, b1, q.z & kAbs, q.w & kAbs);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] += c0[i] + c1[i];
}

template <int NT>
struct SelShared {
    static constexpr int kWarps = NT / 32;
    static constexpr int kRankList = NT;    // blocks ranked here, one per thread
    static constexpr int kBins = 4 * NT;    // of the score histogram
    float err[kMaxCluster];             // per CTA: the largest sum of magnitudes,
    float lowest[kMaxCluster];          // and the range of its finite scores
    float highest[kMaxCluster];
    float sum[kMaxCluster];             // of its finite scores
    int bins[kBins];
    int bin;                            // the threshold's, and the candidates above it
    int above;
    int part[2][kWarps];             // count(): per-warp sums, double-buffered
    float fpart[4][kWarps];
    uint64_t bits_all[kWarps], bits_any[kWarps];
    int list_n;
    int list[kRankList];
    float list_score[kRankList];
    uint64_t list_key[kRankList];
};

// Sum over the CTA; one barrier (`turn` alternates the buffer).
template <int NT>
__device__ __forceinline__ int cta_sum(SelShared<NT>& sh, int x, int& turn) {
    const int w = __reduce_add_sync(0xffffffffu, x);
    if ((threadIdx.x & 31) == 0) sh.part[turn][threadIdx.x >> 5] = w;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    const int y = __reduce_add_sync(0xffffffffu, lane < (NT / 32) ? sh.part[turn][lane] : 0);
    turn ^= 1;
    return y;
}

__device__ __forceinline__ float warp_min(float x) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) x = fminf(x, __shfl_xor_sync(0xffffffffu, x, m));
    return x;
}

template <int NT>
__device__ __forceinline__ float cta_min(SelShared<NT>& sh, float x) {
    x = warp_min(x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh.fpart[0][threadIdx.x >> 5] = x;
    __syncthreads();
    for (int w = 0; w < (NT / 32); ++w) x = fminf(x, sh.fpart[0][w]);
    return x;
}

// The largest P with count(key >= P) >= want over the candidates that `key`
// gives (i strided over the threads; skip(i) leaves one out). exact: whether
// count(key >= P) == want.
template <typename K, int NT, typename Key, typename Skip>
__device__ __forceinline__ K kth_largest(SelShared<NT>& sh, int n, int want, int& turn, bool& exact,
                                         Key key, Skip skip) {
    exact = false;
    // the bits that all keys share need no search
    K common = ~(K)0, any = 0;
    for (int i = threadIdx.x; i < n; i += NT)
        if (!skip(i)) {
            common &= key(i);
            any |= key(i);
        }
    uint64_t c64 = common, a64 = any;
    c64 = (uint64_t)__reduce_and_sync(0xffffffffu, (uint32_t)(c64 >> 32)) << 32 | __reduce_and_sync(0xffffffffu, (uint32_t)c64);
    a64 = (uint64_t)__reduce_or_sync(0xffffffffu, (uint32_t)(a64 >> 32)) << 32 | __reduce_or_sync(0xffffffffu, (uint32_t)a64);
    if ((threadIdx.x & 31) == 0) {
        sh.bits_all[threadIdx.x >> 5] = c64;
        sh.bits_any[threadIdx.x >> 5] = a64;
    }
    __syncthreads();
    for (int w = 0; w < NT / 32; ++w) {
        c64 &= sh.bits_all[w];
        a64 |= sh.bits_any[w];
    }
    const int top = 63 - __clzll((long long)(c64 ^ a64));      // -1: one value
    K prefix = (K)(top < 0 ? c64 : c64 >> top >> 1 << top << 1);
    for (int bit = top; bit >= 0; --bit) {
        const K cand = prefix | ((K)1 << bit);
        int c = 0;
        for (int i = threadIdx.x; i < n; i += NT) c += !skip(i) && key(i) >= cand;
        const int total = cta_sum(sh, c, turn);
        if (total >= want) prefix = cand;
        if (total == want) {
            exact = true;
            break;
        }
    }
    return prefix;
}

// Whether approximate scores with terms of up to mag may be relied on: far above
// what an underflow could drop. (A sum of 0 says nothing: all products may have
// underflowed.)
__device__ __forceinline__ bool reliable(float mag) { return isfinite(mag) && mag >= 0x1p-100f; }

// Whether all query elements of the row's group are zero (all threads, for all).
template <typename T, int D, int NT>
__device__ bool zero_query(const SelectParams& p, int s, int h) {
    const T* q = static_cast<const T*>(p.query) + ((size_t)s * p.num_q_heads + h * p.group) * D;
    bool any = false;
    for (int i = threadIdx.x; i < p.group * D; i += NT) any |= to_float(q[i]) != 0.f;
    return !__syncthreads_or(any);
}

// Whether all bounds of the candidates are zero (all threads, for all).
template <typename T, int D, int NT>
__device__ bool zero_bounds(const SelectParams& p, int h, const int32_t* table, int nc) {
    constexpr int W = 2 * D * (int)sizeof(T) / 16;             // 16-byte words of a block's row
    constexpr uint32_t kAbs = sizeof(T) == 2 ? 0x7fff7fffu : 0x7fffffffu;
    constexpr int kBatch = 8;                                  // blocks read before one is looked at
    const int lane = threadIdx.x & 31;
    bool any = false;
    for (int i0 = threadIdx.x >> 5; i0 < nc && !any; i0 += kBatch * (NT / 32)) {
        uint32_t bits = 0;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int i = i0 + j * (NT / 32);
            const int64_t blk = i < nc ? table[i] : -1;
            if (blk < 0 || blk >= p.num_blocks) continue;
            const uint4* row = reinterpret_cast<const uint4*>(static_cast<const T*>(p.k_bounds) +
                                                              ((size_t)blk * p.num_kv_heads + h) * 2 * D);
#pragma unroll
            for (int c = lane; c < W; c += 32) {
                const uint4 w = row[c];
                bits |= w.x | w.y | w.z | w.w;
            }
        }
        any = __any_sync(0xffffffffu, (bits & kAbs) != 0);
    }
    return !__syncthreads_or(any);
}

// The score that ordered() puts below every value: a block not taken.
__device__ __forceinline__ float out_key() { return __uint_as_float(0xffffffffu); }

// Marks the taken candidates in `taken` (a bit each, in words) where a histogram
// of the approximate scores over their range leaves few blocks near the
// threshold. False: not decided here.
template <typename T, int D, int NT>
__device__ bool take_by_histogram(const SelectParams& p, SelShared<NT>& sh, const float* keys,
                                  uint32_t* taken, int nc, int want, float mag, int C, int s, int h,
                                  const int32_t* table) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float lowest = INFINITY, highest = -INFINITY, mean = 0.f;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {                    // (unrolled: loads in flight together)
        lowest = fminf(lowest, r < C ? sh.lowest[r] : INFINITY);
        highest = fmaxf(highest, r < C ? sh.highest[r] : -INFINITY);
        mean += r < C ? sh.sum[r] : 0.f;
    }
    mean = __fdividef(mean, (float)nc);                        // only places the cut
    const float err2 = mag * (2.f * kScoreEps * 1.01f);        // both errors
    constexpr int kBatch = 8;                                  // keys read before one is used
    // Where few are taken, first only the scores a quarter of the way from the
    // mean to the highest: shared-memory atomics are what the pass costs.
    float cut = want < nc / 16 && isfinite(mean) ? mean + 0.25f * (highest - mean) : -INFINITY;
    float bottom, range, scale;
    // non-decreasing in k; what lies below the range goes to bin 0
    auto bin_of = [&](float k) {
        const int b = __float2int_rz((k - bottom) * scale);
        return b < 0 ? 0 : (b >= SelShared<NT>::kBins ? SelShared<NT>::kBins - 1 : b);
    };
    for (;;) {
        bottom = fmaxf(cut, lowest);
        range = highest - bottom;
        scale = (float)(SelShared<NT>::kBins - 1) / range;
        if (!(reliable(mag) && highest > bottom && isfinite(scale))) return false;
        for (int i = threadIdx.x; i < SelShared<NT>::kBins; i += NT) sh.bins[i] = 0;
        if (threadIdx.x == 0) {
            sh.list_n = 0;
            sh.bin = -1;
        }
        __syncthreads();
        for (int i0 = threadIdx.x; i0 < nc; i0 += kBatch * NT) {
            float k[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) k[j] = i0 + j * NT < nc ? keys[i0 + j * NT] : out_key();
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int b = bin_of(k[j]);
                if (k[j] >= cut) atomicAdd(&sh.bins[b], 1);    // (not the NaN)
            }
        }
        __syncthreads();
        // the bin where the count from the top reaches want: thread t has the
        // four bins below kBins - 4 t
        const int top = SelShared<NT>::kBins - 1 - 4 * (int)threadIdx.x;
        int c[4], sum = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) sum += c[j] = sh.bins[top - j];
        int run = sum;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, run, m);
            if (lane >= m) run += v;
        }
        if (lane == 31) sh.part[0][warp] = run;
        __syncthreads();
        for (int w = 0; w < warp; ++w) run += sh.part[0][w];
        int before = run - sum;
        if (before < want && run >= want) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (before < want && before + c[j] >= want) {
                    sh.bin = top - j;
                    sh.above = before;
                }
                before += c[j];
            }
        }
        __syncthreads();
        if (sh.bin >= 0) break;
        cut = -INFINITY;                                       // too few above the cut
        __syncthreads();
    }
    // Every block that can change sides is within err2 of that bin's range of
    // scores (to the rounding of bin_of and of the range's ends). Above: taken.
    const int bin = sh.bin;
    const float slack = err2 + range * 0x1p-20f + (fabsf(bottom) + fabsf(highest)) * 0x1p-21f;
    const float from = bin == 0 && cut == -INFINITY ? -INFINITY : bottom + (float)bin / scale - slack;
    const float to = bottom + (float)(bin + 1) / scale + slack;
    int near_above = 0;                                        // counted above the bin, but not settled
    for (int i0 = warp * 32; i0 < nc; i0 += kBatch * NT) {
        float k[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int i = i0 + j * NT + lane;
            k[j] = i < nc ? keys[i] : out_key();               // (NaN: in neither)
        }
        uint32_t word = 0, near = 0;                           // lane j: the words of keys j
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const uint32_t w = __ballot_sync(0xffffffffu, k[j] > to);
            if (lane == j) word = w;
            near |= (uint32_t)(k[j] >= from && k[j] <= to) << j;
        }
        if (lane < kBatch && i0 + lane * NT < nc) taken[(i0 + lane * NT) >> 5] = word;
        while (near) {
            const int j = __ffs(near) - 1;
            near &= near - 1;
            const int i = i0 + j * NT + lane;
            const float x = keys[i];
            const int at = atomicAdd(&sh.list_n, 1);
            if (at < SelShared<NT>::kRankList) {
                sh.list[at] = i;
                sh.list_score[at] = x;
            }
            near_above += bin_of(x) > bin;
        }
    }
    int turn = 0;
    const int left = want - (sh.above - cta_sum(sh, near_above, turn));       // the list's places
    const int m = sh.list_n;
    if (m > SelShared<NT>::kRankList) return false;
    // rank by approximate score (the list's order varies, the ranks do not)
    const int e = threadIdx.x;
    const bool mine = e < m;
    const float k = mine ? sh.list_score[e] : 0.f;
    const int i = mine ? sh.list[e] : 0;
    int before = 0;
    if (mine)
        for (int o = 0; o < m; ++o)
            before += sh.list_score[o] > k || (sh.list_score[o] == k && sh.list[o] < i);
    bool take = mine && before < left;
    // the smallest taken and the largest left out of a set of scores in the list
    auto border = [&](float x, float& a, float& b) {
        a = take ? x : INFINITY;
        b = mine && !take ? x : -INFINITY;
        if (m > 32) {
            a = cta_min(sh, a);
            b = -cta_min(sh, -b);
        } else {                                               // the list is in warp 0
            a = warp_min(a);
            b = -warp_min(-b);
            if (threadIdx.x == 0) {
                sh.fpart[0][0] = a;
                sh.fpart[1][0] = b;
            }
            __syncthreads();
            a = sh.fpart[0][0];
            b = sh.fpart[1][0];
        }
    };
    float a, b;
    border(k, a, b);
    if (a - b <= err2) {
        // the blocks within err2 of the other side, by their exact scores
        const bool open = mine && (take ? k <= b + err2 : k >= a - err2);
        int ahead = cta_sum(sh, mine && !open && take, turn);  // settled inside
        if (mine) sh.list_key[e] = open ? 1 : 0;               // below every key of a score
        __syncthreads();
        for (int w = warp; w < m * p.group; w += (NT / 32)) {  // a warp per (block, head)
            const int o = w / p.group;
            if (sh.list_key[o] == 0) continue;
            const uint64_t x = exact_head_score<T, D>(p, s, h, w - o * p.group, table[sh.list[o]], lane);
            if (lane == 0) atomicMax(reinterpret_cast<unsigned long long*>(&sh.list_key[o]), (unsigned long long)x);
        }
        __syncthreads();
        if (open) {
            const uint64_t x = sh.list_key[e];
            for (int o = 0; o < m; ++o) {
                const uint64_t y = sh.list_key[o];
                ahead += y > x || (y == x && sh.list[o] < i);
            }
            take = ahead < left;
        }
    }
    if (take) atomicOr(&taken[i >> 5], 1u << (i & 31));
    __syncthreads();
    return true;
}

// One (sequence, KV head) of the batch, as every CTA of its cluster sees it.
struct SelRow {
    int row, s, h;                      // row = s * num_kv_heads + h
    int L, n;                           // tokens, blocks
    int C, rank;                        // CTAs of the cluster, this one's
    int lo, nc, want;                   // candidates lo .. lo + nc - 1, and how many are taken
    bool all, scored;
    const int32_t* table;
    uint4* sides;                       // [n-tile][step][lane]
    float* keys;                        // the candidates' scores (of the first CTA, or in memory)
    uint32_t* taken;                    // a bit per candidate (the first CTA's)
    int ahead[2];                       // the blocks of this lane's rows of its first tile

    __device__ __forceinline__ SelRow(const SelectParams& p, cg::cluster_group& cluster, uint8_t* smem) {
        C = (int)cluster.num_blocks();
        rank = (int)cluster.block_rank();
        row = blockIdx.x / C;
        s = row / p.num_kv_heads;
        h = row - s * p.num_kv_heads;
        table = p.block_tables + (size_t)s * p.max_blocks;
        lo = p.first_blocks;
        // the first table entries, on their way while the length is
        const int tile = (rank * blockDim.x + threadIdx.x) >> 5;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int64_t i = (int64_t)lo + tile * 16 + ((threadIdx.x & 31) >> 2) + 8 * r;
            ahead[r] = table[i < p.max_blocks ? i : p.max_blocks - 1];
        }
        bool bad;
        L = clamped_len(p, s, bad);
        if (bad && h == 0 && rank == 0 && threadIdx.x == 0 && p.status) atomicOr(p.status, PA_DEV_BAD_LEN);
        n = (L + p.block_size - 1) / p.block_size;
        all = n <= p.num_select;
        want = p.num_select - p.first_blocks - p.recent_blocks;
        nc = all ? 0 : n - p.recent_blocks - lo;
        scored = nc > 0 && want > 0;
        sides = reinterpret_cast<uint4*>(smem);
        taken = reinterpret_cast<uint32_t*>(smem + p.side_bytes);
        keys = p.keys_in_smem ? reinterpret_cast<float*>(smem + p.side_bytes + p.taken_bytes)
                              : p.scores + (size_t)row * p.max_ctx_blocks;
    }
};

// Barrier over the cluster (over the CTA where it is one).
__device__ __forceinline__ void cluster_barrier(cg::cluster_group& cluster, int C) {
    if (C > 1) cluster.sync();
    else __syncthreads();
}

// The query's two sides as the MMAs' second operand, [n-tile][step][lane]:
// lane (g, t4) of step j has head g's elements 32 j + 8 t4 .. of (min(q, 0),
// max(q, 0)). Followed by a barrier before their use.
template <typename T, int D, int NT>
__device__ void stage_sides(const SelectParams& p, const SelRow& rw) {
    constexpr int STEPS = 2 * D / 32;
    const int ntiles = (p.group + 7) / 8;
    for (int i = threadIdx.x; i < ntiles * STEPS * 32; i += NT) {
        const int l = i & 31, j = (i >> 5) % STEPS, nt = i / (32 * STEPS);
        const int g = nt * 8 + (l >> 2);
        const int e = 32 * j + 8 * (l & 3);
        const bool positive = e >= D;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (g < p.group) {
            w = *reinterpret_cast<const uint4*>(
                static_cast<const T*>(p.query) +
                ((size_t)rw.s * p.num_q_heads + rw.h * p.group + g) * D + (positive ? e - D : e));
            w = make_uint4(side2<T>(w.x, positive), side2<T>(w.y, positive),
                           side2<T>(w.z, positive), side2<T>(w.w, positive));
        }
        rw.sides[i] = w;
    }
}

// Approximate scores of the candidates (all CTAs of the cluster) into the first
// CTA's keys, and what it needs to know of them (err, lowest, highest, sum).
template <typename T, int D, bool kOneTile, int NT>
__device__ __forceinline__ void score_candidates(const SelectParams& p, SelShared<NT>& sh,
                                                 cg::cluster_group& cluster, const SelRow& rw) {
    constexpr int STEPS = 2 * D / 32;                          // 64-byte steps of a bounds row (16-bit types)
    constexpr int NQ = STEPS / 4;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int C = rw.C, rank = rw.rank, s = rw.s, h = rw.h, nc = rw.nc, lo = rw.lo;
    const int32_t* table = rw.table;
    const uint4* sides = rw.sides;
    float* out_keys = p.keys_in_smem ? cluster.map_shared_rank(rw.keys, 0) : rw.keys;
    float worst = 0.f, lowest = INFINITY, highest = -INFINITY, total = 0.f;
    if constexpr (std::is_same<T, float>::value) {
        constexpr int E = D / 32;
        for (int i = rank * (NT / 32) + warp; i < nc; i += C * (NT / 32)) {
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
                lowest = fminf(lowest, best);
                highest = fmaxf(highest, best);
                if (lane == 0) total += best;
            }
            if (lane == 0) out_keys[i] = best;
        }
    } else {
        const int ntiles = (p.group + 7) / 8;
        const int g = lane >> 2, t4 = lane & 3;
        const int tiles = (nc + 15) / 16;
        const int stride = C * (NT / 32);
        // this lane's two blocks of a tile, and their bounds rows (block 0's
        // where the table names none)
        auto block_of = [&](int tile, int r) {
            const int i = tile * 16 + g + 8 * r;
            return table[lo + (i < nc ? i : nc - 1)];
        };
        auto there = [&](int blk) { return blk >= 0 && blk < p.num_blocks; };
        auto row_of = [&](int blk) {
            return static_cast<const T*>(p.k_bounds) +
                   ((size_t)(there(blk) ? blk : 0) * p.num_kv_heads + h) * 2 * D + 8 * t4;
        };
        auto finish = [&](int tile, const int (&blk)[2], float (&best)[2], float (&mag)[2]) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 1));
                best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 2));
                const int i = tile * 16 + g + 8 * r;
                const bool ok = there(blk[r]);
                if (ok && i < nc) {
                    worst = max_nan(worst, mag[r]);
                    lowest = fminf(lowest, best[r]);
                    highest = fmaxf(highest, best[r]);
                    if (t4 == 0) total += best[r];
                }
                if (t4 == 0 && i < nc) out_keys[i] = ok ? best[r] : -INFINITY;
            }
        };
        // maxima over the heads of one MMA tile
        auto over_heads = [&](int nt, const float (&c)[4], const float (&m)[4], float (&best)[2], float (&mag)[2]) {
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (nt * 8 + 2 * t4 + e < p.group) {
                        best[r] = fmaxf(best[r], c[2 * r + e]);
                        mag[r] = max_nan(mag[r], m[2 * r + e]);
                    }
        };
        int tile = rank * (NT / 32) + warp;
        if constexpr (kOneTile) {
            // Two quarters' loads are always in flight: a buffer is refilled as
            // soon as it is multiplied. Block ids come two tiles ahead.
            Quarter buf[2];
            auto after = [&](int t) { return t + stride < tiles ? t + stride : t; };
            int blk[2], next_blk[2];                           // this tile's blocks, the next one's
            if (tile < tiles) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    blk[r] = rw.ahead[r];                      // (past nc: any block, its score unused)
                    next_blk[r] = block_of(after(tile), r);
                }
                const T *x = row_of(blk[0]), *y = row_of(blk[1]);
                buf[0].load(x, y);
                if (NQ > 1) buf[1].load(x + 128, y + 128);
                else buf[1].load(row_of(next_blk[0]), row_of(next_blk[1]));
            }
            // one tile from buffers b0 (and b1), which it refills
            auto step = [&](Quarter& b0, Quarter& b1) {
                const int next = after(tile), far = after(next);
                const int far_blk[2] = {block_of(far, 0), block_of(far, 1)};
                const T *x = row_of(blk[0]), *y = row_of(blk[1]);
                float c[4] = {0.f, 0.f, 0.f, 0.f}, m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int q = 0; q < NQ; ++q) {
                    Quarter& b = q & 1 ? b1 : b0;
                    add_quarter<T>(b, sides + 128 * q + lane, c, m);
                    if (q + 2 < NQ) b.load(x + 128 * (q + 2), y + 128 * (q + 2));
                    else if (NQ > 1 && next != tile)
                        b.load(row_of(next_blk[0]) + 128 * (q + 2 - NQ), row_of(next_blk[1]) + 128 * (q + 2 - NQ));
                    else if (NQ == 1 && far != next) b.load(row_of(far_blk[0]), row_of(far_blk[1]));
                }
                float best[2] = {-INFINITY, -INFINITY}, mag[2] = {0.f, 0.f};
                over_heads(0, c, m, best, mag);
                finish(tile, blk, best, mag);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    blk[r] = next_blk[r];
                    next_blk[r] = far_blk[r];
                }
                tile += stride;
            };
            while (tile < tiles) {
                step(buf[0], buf[1]);
                if (NQ == 1 && tile < tiles) step(buf[1], buf[0]);
            }
        } else {
            for (; tile < tiles; tile += stride) {
                const int blk[2] = {block_of(tile, 0), block_of(tile, 1)};
                const T *x = row_of(blk[0]), *y = row_of(blk[1]);
                float best[2] = {-INFINITY, -INFINITY}, mag[2] = {0.f, 0.f};
                for (int nt = 0; nt < ntiles; ++nt) {
                    float c[4] = {0.f, 0.f, 0.f, 0.f}, m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int q = 0; q < NQ; ++q) {
                        Quarter b;
                        b.load(x + 128 * q, y + 128 * q);
                        add_quarter<T>(b, sides + (nt * STEPS + 4 * q) * 32 + lane, c, m);
                    }
                    over_heads(nt, c, m, best, mag);
                }
                finish(tile, blk, best, mag);
            }
        }
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) {
        worst = max_nan(worst, __shfl_xor_sync(0xffffffffu, worst, m));
        lowest = fminf(lowest, __shfl_xor_sync(0xffffffffu, lowest, m));
        highest = fmaxf(highest, __shfl_xor_sync(0xffffffffu, highest, m));
        total += __shfl_xor_sync(0xffffffffu, total, m);
    }
    if (lane == 0) {
        sh.fpart[0][warp] = worst;
        sh.fpart[1][warp] = lowest;
        sh.fpart[2][warp] = highest;
        sh.fpart[3][warp] = total;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < (NT / 32); ++w) {
            worst = max_nan(worst, sh.fpart[0][w]);
            lowest = fminf(lowest, sh.fpart[1][w]);
            highest = fmaxf(highest, sh.fpart[2][w]);
            total += sh.fpart[3][w];
        }
        *cluster.map_shared_rank(&sh.err[rank], 0) = worst;
        *cluster.map_shared_rank(&sh.lowest[rank], 0) = lowest;
        *cluster.map_shared_rank(&sh.highest[rank], 0) = highest;
        *cluster.map_shared_rank(&sh.sum[rank], 0) = total;
    }
}

// Marks the taken candidates where the histogram does not decide: a search over
// the bits of the approximate scores, exact scores of all that it leaves
// unsettled (every block where magnitudes are not reliable), and if those are
// many a search over the exact scores' bits.
template <typename T, int D, int NT>
__device__ __forceinline__ void take_by_search(const SelectParams& p, SelShared<NT>& sh, const SelRow& rw,
                                            float mag) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = rw.row, s = rw.s, h = rw.h, nc = rw.nc, want = rw.want, lo = rw.lo;
    const int32_t* table = rw.table;
    float* keys = rw.keys;
    int turn = 0;
    uint32_t thr = 0;                                      // taken candidates: ordered(key) >= thr
    const double err2 = 2.0 * (double)kScoreEps * (double)mag * 1.001;
    const bool finite = reliable(mag);
    // Settled blocks: those that beat (or lose to) every block on the other
    // side of the threshold by more than both errors. in_above: taken for
    // certain above it; out_below: left out for certain below it.
    double in_above = INFINITY, out_below = -INFINITY;
    if (finite) {
        bool exact;
        thr = kth_largest<uint32_t, NT>(sh, nc, want, turn, exact, [&](int i) { return ordered(keys[i]); },
                                    [](int) { return false; });
        float a = INFINITY, b = -INFINITY;                 // the smallest taken, the largest left out
        for (int i = threadIdx.x; i < nc; i += NT) {
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
        for (int w = 0; w < (NT / 32); ++w) {
            a = fminf(a, sh.fpart[0][w]);
            b = fmaxf(b, sh.fpart[1][w]);
        }
        if (!exact) b = a;                                 // equal keys across the threshold
        in_above = (double)b + err2;
        out_below = (double)a - err2;
    }
    const float kOut = out_key();
    auto settled = [&](float k) { return finite && ((double)k > in_above || (double)k < out_below); };
    // count the certain ones and the unsettled
    int in = 0, open = 0;
    for (int i = threadIdx.x; i < nc; i += NT) {
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
        // (A zero query, say of a padding row, or a pool of zeros makes every score
        // 0, exactly.)
        const bool zeros = mag == 0.f && (zero_query<T, D, NT>(p, s, h) || zero_bounds<T, D, NT>(p, h, table + lo, nc));
        const bool small = open <= SelShared<NT>::kRankList && !zeros;
        if (threadIdx.x == 0) sh.list_n = 0;
        __syncthreads();
        uint64_t* exact_keys = p.exact_keys + (size_t)row * p.max_ctx_blocks;
        if (zeros)
            for (int i = threadIdx.x; i < nc; i += NT) exact_keys[i] = ordered64(keys[i]);
        for (int i0 = zeros ? nc : warp * 32; i0 < nc; i0 += NT) {
            const bool mine = i0 + lane < nc && !settled(keys[i0 + lane]);
            uint32_t votes = __ballot_sync(0xffffffffu, mine);
            while (votes) {
                const int i = i0 + __ffs(votes) - 1;
                votes &= votes - 1;
                const uint64_t k = exact_score<T, D>(p, s, h, table[lo + i], lane);
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
            const uint64_t t = kth_largest<uint64_t, NT>(
                sh, nc, left, turn, exact, [&](int i) { return exact_keys[i]; },
                [&](int i) { return settled(keys[i]); });
            int above = 0;
            for (int i = threadIdx.x; i < nc; i += NT)
                above += !settled(keys[i]) && exact_keys[i] > t;
            above = cta_sum(sh, above, turn);
            int ties = exact ? 0x7fffffff : left - above;  // places for keys equal to t, lowest first
            for (int i0 = 0; i0 < nc; i0 += NT) {
                const int i = i0 + threadIdx.x;
                const bool mine = i < nc && !settled(keys[i]);
                const uint64_t k = mine ? exact_keys[i] : 0;
                const bool tie = mine && k == t;
                const uint32_t votes = __ballot_sync(0xffffffffu, tie);
                if (lane == 0) sh.part[turn][warp] = __popc(votes);
                __syncthreads();
                int at = __popc(votes & ((1u << lane) - 1)), total = 0;
                for (int w = 0; w < (NT / 32); ++w) {
                    if (w < warp) at += sh.part[turn][w];
                    total += sh.part[turn][w];
                }
                turn ^= 1;
                if (mine) keys[i] = k > t || (tie && at < ties) ? INFINITY : kOut;
                if (!exact) ties -= total < ties ? total : ties;
            }
        } else {
            for (int i = threadIdx.x; i < nc; i += NT)
                if (!settled(keys[i])) keys[i] = kOut;
        }
        __syncthreads();
    } else {
        // every unsettled block is taken: they are the candidates from out_below on
        for (int i = threadIdx.x; i < nc; i += NT)
            if (!settled(keys[i])) keys[i] = INFINITY;
        __syncthreads();
    }
    for (int i0 = warp * 32; i0 < nc; i0 += NT) {
        const uint32_t word = __ballot_sync(0xffffffffu, i0 + lane < nc && ordered(keys[i0 + lane]) >= thr);
        if (lane == 0) rw.taken[i0 >> 5] = word;
    }
    __syncthreads();
}

// Scores the candidates (all CTAs of the cluster) and marks the taken ones (the
// first CTA, in rw.taken). All CTAs meet at two cluster barriers if rw.scored,
// else at none; the sides have been staged. kOneTile: groups of at most eight
// heads, one MMA tile.
template <typename T, int D, bool kOneTile, int NT>
__device__ __forceinline__ void score_and_take(const SelectParams& p, SelShared<NT>& sh,
                                               cg::cluster_group& cluster, const SelRow& rw) {
    if (!rw.scored) return;
    cluster_barrier(cluster, rw.C);                            // the sides; the first CTA runs: its memory may be written
    score_candidates<T, D, kOneTile, NT>(p, sh, cluster, rw);
    cluster_barrier(cluster, rw.C);
    if (rw.rank != 0) return;
    float mag = 0.f;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) mag = max_nan(mag, r < rw.C ? sh.err[r] : 0.f);
    if (!take_by_histogram<T, D, NT>(p, sh, rw.keys, rw.taken, rw.nc, rw.want, mag, rw.C, rw.s, rw.h,
                                     rw.table + rw.lo))
        take_by_search<T, D, NT>(p, sh, rw, mag);
}

// Calls put(position, block) for every block the row takes, positions in block
// order (the first CTA, after score_and_take; any CTA where rw.all).
template <int NT, typename Put>
__device__ __forceinline__ void for_taken(SelShared<NT>& sh, const SelRow& rw, Put put) {
    if (rw.all) {
        for (int b = threadIdx.x; b < rw.n; b += NT) put(b, b);
        return;
    }
    for (int b = threadIdx.x; b < rw.lo; b += NT) put(b, b);
    const int recent = rw.n - rw.lo - rw.nc;
    for (int i = threadIdx.x; i < recent; i += NT) put(rw.lo + rw.want + i, rw.lo + rw.nc + i);
    if (!rw.scored) return;
    // each thread has consecutive words of the candidates' bits
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int words = (rw.nc + 31) / 32, per = (words + NT - 1) / NT;
    const int w0 = threadIdx.x * per, w1 = min(w0 + per, words);
    int mine = 0;
    for (int w = w0; w < w1; ++w) mine += __popc(rw.taken[w]);
    int run = mine;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, run, m);
        if (lane >= m) run += v;
    }
    __syncthreads();
    if (lane == 31) sh.part[0][warp] = run;
    __syncthreads();
    for (int w = 0; w < warp; ++w) run += sh.part[0][w];
    int at = rw.lo + run - mine;
    for (int w = w0; w < w1; ++w)
        for (uint32_t word = rw.taken[w]; word && at < rw.lo + rw.want; word &= word - 1)
            put(at++, rw.lo + 32 * w + __ffs(word) - 1);
}

// The slab of a row's block, or -1 where the table names none.
__device__ __forceinline__ int32_t slab_of(const SelectParams& p, const SelRow& rw, int block) {
    const int64_t blk = rw.table[block];
    return blk >= 0 && blk < p.num_blocks ? (int32_t)(blk * p.num_kv_heads + rw.h) : -1;
}

// ---------------------------------------------------------------- host side

// CTAs of 8 warps per row for the selection alone (the fused kernel has a rule of
// its own): as many as fit on 152 SMs with a tile of 16 blocks or more for every
// warp. For many rows one CTA each wins, two on an SM: their selections overlap
// other rows' scoring. Whole calls of groups of 16 heads of 128, bf16, with 1, 2, 4
// and 8 CTAs: 8 rows of 8192 blocks 235, 137, 83 and 56 us; 32 rows of 1024 blocks
// 56, 46, 40 and 40, of 500 blocks 42, 38, 36 and 38; 112 rows of 1170 blocks 80, 79,
// 87 and 99. Binary32, 8 rows of 8192: 766, 446, 237 and 132.
inline int select_cluster(int rows, int max_ctx_blocks) {
    int C = 1;
    while (C < kMaxCluster && rows <= 152 / (2 * C) && max_ctx_blocks >= 2 * C * 256) C *= 2;
    return C;
}

// Sets the launch's shared-memory fields; returns the bytes of sides and keys.
template <typename T, int D>
int select_smem(SelectParams& p) {
    const int ntiles = (p.group + 7) / 8;
    p.side_bytes = std::is_same<T, float>::value ? 0 : ntiles * (2 * D / 32) * 512;
    p.keys_in_smem = p.max_ctx_blocks <= kSmemKeys && p.side_bytes <= 64 * 1024;
    p.taken_bytes = (p.max_ctx_blocks + 127) / 128 * 16;
    if (p.max_ctx_blocks <= p.num_select) return 0;            // nothing is scored
    return p.side_bytes + p.taken_bytes + (p.keys_in_smem ? p.max_ctx_blocks * 4 : 0);
}

template <typename Params>
cudaError_t launch_cluster(void (*kernel)(Params), const Params& p, int grid, int cluster, int threads, int smem,
                           cudaStream_t stream) {
    cudaError_t e = ensure_smem_attribute(reinterpret_cast<const void*>(kernel), 200 * 1024);
    if (e != cudaSuccess) return e;
    return launch_overlapped(kernel, p, dim3(grid), threads, smem, stream, cluster);
}

}  // namespace pagedkv
