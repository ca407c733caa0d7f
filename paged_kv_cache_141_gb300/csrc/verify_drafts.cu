// verify_drafts.cu -- verification of drafted tokens against the target's
// probabilities, by given random numbers. Draft i of a request, token x_i drawn
// with probability q_i(x_i), is accepted while
//     u_i q_i(x_i) < p_i(x_i)
// holds for it and for all before it (the products in binary64, where they are
// exact). After a accepted drafts one more token is drawn: from the part of p_a
// that lies beyond q_a, w_j = max(p_a(j) - q_a(j), 0), where a draft was
// rejected (w = p_a where nothing lies beyond), or from w = p_a after the last
// draft; this makes the tokens' distribution the target's. The drawn token is the
// first j with w_0 + .. + w_j > u W, W the sum of all.
//
// The accept tests read one value of each row; the work is one row of p and of q
// for each request, read once: HBM-bound for a batch, latency for one request. A
// cluster of CTAs takes a request, each CTA a contiguous section of the row in
// tiles of 512, a warp a tile, whose sum stays in shared memory. The CTAs trade their
// totals, the one whose section holds u W finds the tile among its sums, and one warp
// reads that tile again (from L1 or L2) for the token. Sums are pairs of binary32 numbers, a
// tile's as a tree, a warp's tiles dealt to its lanes: with 64 tiles a lane, of 2^22 tokens,
// (99 + 3 64 + 3 8) 2^-48 of the sum at most, less than 2^-39 (added tile after tile in one
// pair that is not brought back to |lo| <= 2^-24 |hi|, they lost up to 2^-31). Binary64
// units would take five times as long as the reads; binary64 across the lanes alone took 85 us
// where pairs took 63, across a warp's tiles alone 30.5 where this takes 28 (64 requests), and
// whole tiles without a test for each value now take 50, 5.2 TB/s, for 256 requests of 128,256
// tokens; one request of 32,000 takes 9.5: launch, three cluster barriers and the loads between them.
// With 100,000 borders between tokens, sums to 2^-30 alone would draw another token in one
// request of 5,000.
#include <cooperative_groups.h>

#include "device_common.cuh"
#include "launch.h"

namespace pagedkv {

namespace {

namespace cg = cooperative_groups;

constexpr int kVerifyTile = 512;
constexpr int kVerifyPer = kVerifyTile / 32;       // of a tile, a lane's values
constexpr int kVerifyCluster = 8;
// Warps that run at once: 32 an SM, and in clusters of eight CTAs 1184 of four warps or 592 of
// eight (as the occupancy calculator says; four SMs' worth fit no whole cluster).
constexpr int kVerifyWave = 4736;

// Row weights: p alone, p beyond q, or p without one token.
struct Weights {
    const float* p;
    const float* q;                                // may be null
    int64_t without;                               // -1: none
};

// This lane's values of the tile at `at`: elements 32 i + lane, i < 16; zeros past the row.
__device__ __forceinline__ void load_tile(const Weights& w, int64_t at, int64_t V, int lane, float (&a)[kVerifyPer],
                                          float (&b)[kVerifyPer]) {
    const float *p = w.p + at + lane, *q = w.q + at + lane;
    if (at + kVerifyTile <= V && (w.without < at || w.without >= at + kVerifyTile)) {
#pragma unroll
        for (int i = 0; i < kVerifyPer; ++i) a[i] = p[32 * i];
        if (w.q) {
#pragma unroll
            for (int i = 0; i < kVerifyPer; ++i) b[i] = q[32 * i];
        } else {
#pragma unroll
            for (int i = 0; i < kVerifyPer; ++i) b[i] = 0.f;
        }
        return;
    }
    const int left = (int)min((int64_t)kVerifyTile, V - at) - lane, not_this = (int)(w.without - at) - lane;
#pragma unroll
    for (int i = 0; i < kVerifyPer; ++i) {
        a[i] = 32 * i < left && (w.without < 0 || 32 * i != not_this) ? p[32 * i] : 0.f;
        b[i] = w.q && 32 * i < left ? q[32 * i] : 0.f;
    }
}

// A sum as an unevaluated pair of binary32 numbers.
struct Pair {
    float hi, lo;
};
__device__ __forceinline__ Pair add(Pair x, Pair y) {
    const float s = x.hi + y.hi, t = s - x.hi;
    return {s, (x.lo + y.lo) + ((x.hi - (s - t)) + (y.hi - t))};
}
__device__ __forceinline__ double value(Pair x) { return (double)x.hi + (double)x.lo; }
// The same sum, |lo| <= 2^-24 |hi| again.
__device__ __forceinline__ Pair normal(Pair x) {
    const float s = x.hi + x.lo;
    return {s, x.lo - (s - x.hi)};
}

// The sum of max(a - b, 0) over the warp's values, as a tree; the differences keep their
// rounding errors, as the sums do. A NaN stays. At level k of the tree lo is at most
// (k + 1) 2^-24 of the sum, and its two roundings (2 k + 1) 2^-48: 99 2^-48 after 9 levels.
// (A sum of normal pairs is good to 3 2^-48.)
__device__ __forceinline__ Pair tile_sum(const float (&a)[kVerifyPer], const float (&b)[kVerifyPer]) {
    Pair l[kVerifyPer];
#pragma unroll
    for (int i = 0; i < kVerifyPer; ++i) {
        l[i].hi = a[i] - b[i];
        l[i].lo = (a[i] - l[i].hi) - b[i];                         // exact for a >= b >= 0
        if (l[i].hi <= 0.f) l[i].hi = l[i].lo = 0.f;
    }
#pragma unroll
    for (int m = kVerifyPer / 2; m; m >>= 1)
#pragma unroll
        for (int i = 0; i < m; ++i) l[i] = add(l[i], l[i + m]);
    Pair x = l[0];
#pragma unroll
    for (int m = 16; m; m >>= 1) x = add(x, {__shfl_xor_sync(0xffffffffu, x.hi, m), __shfl_xor_sync(0xffffffffu, x.lo, m)});
    return x;
}

template <int T>
__global__ void __launch_bounds__(T, 1024 / T)
verify_drafts_kernel(const __grid_constant__ VerifyParams p) {
    begin_overlapped();
    constexpr int kWarps = T / 32;
    extern __shared__ Pair tile_sums[];
    __shared__ int s_accepted;
    __shared__ Pair s_part[kWarps];
    __shared__ double s_totals[kVerifyCluster];
    const cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int s = blockIdx.x / ranks;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int K = p.max_drafts;
    const int64_t V = p.vocab;
    int64_t* out = p.out_tokens + (size_t)s * (K + 1);
    // the first drafts, next to the rows' starts
    const int64_t token0 = warp == 0 && lane < K ? p.draft_tokens[(size_t)s * K + lane] : -1;
    const float u0 = warp == 0 && lane < K ? p.uniforms[(size_t)s * (K + 1) + lane] : 0.f;
    const double u = p.uniforms[(size_t)s * (K + 1) + K];
    const int64_t row0 = p.query_start[s], rows = p.query_start[s + 1] - row0;
    const bool bad = rows < 0 || rows > K + 1 || row0 < 0 || row0 + rows > p.num_rows;
    if (bad || rows == 0) {                        // every CTA of the cluster alike
        if (rank == 0) {
            for (int i = threadIdx.x; i <= K; i += T) out[i] = -1;
            if (threadIdx.x == 0) {
                p.accepted[s] = 0;
                if (p.rejected) p.rejected[s] = 0;
                if (bad && p.status) atomicOr(p.status, PA_DEV_BAD_LEN);
            }
        }
        return;
    }
    const int n = (int)rows - 1;
    if (warp == 0) {
        int a = n;
        for (int i0 = 0; i0 < n; i0 += 32) {
            const int i = i0 + lane;
            bool fine = true;
            if (i < n) {
                const int64_t x = i0 ? p.draft_tokens[(size_t)s * K + i] : token0;
                const double ui = i0 ? p.uniforms[(size_t)s * (K + 1) + i] : u0;
                if (x < 0 || x >= V) {
                    fine = false;
                    if (rank == 0 && p.status) atomicOr(p.status, PA_DEV_BAD_TOKEN);
                } else {
                    const double q = p.draft_probs ? p.draft_probs[((size_t)s * K + i) * p.draft_stride + x] : 1.f;
                    const double t = p.target_probs[(row0 + i) * p.target_stride + x];
                    fine = ui * q < t;
                }
            }
            const uint32_t no = __ballot_sync(0xffffffffu, !fine);
            if (no) {
                a = i0 + __ffs(no) - 1;
                break;
            }
        }
        if (lane == 0) s_accepted = a;
    }
    __syncthreads();
    const int a = s_accepted;
    Weights w{p.target_probs + (row0 + a) * p.target_stride, nullptr, -1};
    if (a < n) {
        if (p.draft_probs) w.q = p.draft_probs + ((size_t)s * K + a) * p.draft_stride;
        else {
            const int64_t x = p.draft_tokens[(size_t)s * K + a];
            if (x < V) w.without = x;              // (one that is no token takes nothing away)
        }
    }
    auto started = cluster.barrier_arrive();       // every CTA of the cluster runs before its memory is written
    bool first_pass = true;
    const int tiles = (int)((V + kVerifyTile - 1) / kVerifyTile);
    const int per = (tiles + ranks - 1) / ranks;
    const int first = min(tiles, rank * per), mine = min(tiles, first + per) - first;
    for (;;) {
        Pair part{0.f, 0.f};                       // the warp's tiles, dealt to its lanes
        int turn = lane;
        for (int t = warp; t < mine; t += kWarps) {
            float a[kVerifyPer], b[kVerifyPer];
            load_tile(w, (int64_t)(first + t) * kVerifyTile, V, lane, a, b);
            const Pair total = tile_sum(a, b);
            if (lane == 0) tile_sums[t] = total;
            const Pair next = normal(add(part, total));
            if (turn == 0) part = next;
            turn = (turn + 31) & 31;
        }
        for (int m = 1; m < 32 && m * kWarps < mine; m <<= 1)      // (over the lanes that were dealt any)
            part = normal(add(part, {__shfl_xor_sync(0xffffffffu, part.hi, m), __shfl_xor_sync(0xffffffffu, part.lo, m)}));
        if (lane == 0) s_part[warp] = part;
        if (first_pass) cluster.barrier_wait(std::move(started));
        first_pass = false;
        __syncthreads();
        if (threadIdx.x < ranks) {
            Pair c[kWarps];
#pragma unroll
            for (int i = 0; i < kWarps; ++i) c[i] = s_part[i];
#pragma unroll
            for (int m = kWarps / 2; m; m >>= 1)
#pragma unroll
                for (int i = 0; i < m; ++i) c[i] = normal(add(c[i], c[i + m]));
            cluster.map_shared_rank(s_totals, threadIdx.x)[rank] = value(c[0]);
        }
        if (ranks > 1) cluster.sync();
        else __syncthreads();
        double before = 0, total = 0;
        for (int r = 0; r < ranks; ++r) {
            if (r < rank) before += s_totals[r];
            total += s_totals[r];
        }
        // nothing beyond q: from p itself (every CTA of the cluster alike)
        if (total == 0 && (w.q || w.without >= 0)) {
            w.q = nullptr;
            w.without = -1;
            if (ranks > 1) cluster.sync();         // the totals have been read
            else __syncthreads();
            continue;
        }
        const bool drawable = total > 0 && total < (double)INFINITY;
        const double goal = u * total;
        if (rank == 0 && threadIdx.x < 32) {
            for (int i = lane; i <= K; i += 32)
                if (i != a || !drawable) out[i] = i < a ? p.draft_tokens[(size_t)s * K + i] : -1;
            if (lane == 0) {
                p.accepted[s] = a;
                if (p.rejected) p.rejected[s] = n - a;
                if (!drawable && p.status) atomicOr(p.status, PA_DEV_BAD_PROB);
            }
        }
        // the section of the goal: the last one with any weight that starts at or below it
        int holder = -1;
        double start = 0;
        for (int r = 0; r < ranks; ++r) {
            if (s_totals[r] > 0 && (holder < 0 || start <= goal)) holder = r;
            start += s_totals[r];
        }
        if (!drawable || holder != rank || warp != 0) return;
        // its tile, alike
        int tile = -1;
        double run = before, base = before;
        for (int t0 = 0; t0 < mine; t0 += 32) {
            const double v = t0 + lane < mine ? value(tile_sums[t0 + lane]) : 0;
            double up = v;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const double o = __shfl_up_sync(0xffffffffu, up, m);
                if (lane >= m) up += o;
            }
            const uint32_t here = __ballot_sync(0xffffffffu, v > 0 && run + (up - v) <= goal);
            const uint32_t any = __ballot_sync(0xffffffffu, v > 0);
            const int at = here ? 31 - __clz(here) : (tile < 0 && any ? __ffs(any) - 1 : -1);
            if (at >= 0) {
                tile = t0 + at;
                base = run + __shfl_sync(0xffffffffu, up - v, at);
            }
            run += __shfl_sync(0xffffffffu, up, 31);
        }
        // and the token: the first whose sum passes the goal, or the tile's last with any
        // weight. A lane takes 16 neighbours.
        const int64_t at = (int64_t)(first + tile) * kVerifyTile + lane * kVerifyPer;
        Pair own[kVerifyPer], all{0.f, 0.f};
        int last = -1;
        float x[kVerifyPer], y[kVerifyPer];
#pragma unroll
        for (int i = 0; i < kVerifyPer; ++i) {
            x[i] = at + i < V && at + i != w.without ? w.p[at + i] : 0.f;
            y[i] = w.q && at + i < V ? w.q[at + i] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kVerifyPer; ++i) {
            if (x[i] > y[i]) {
                const float d = x[i] - y[i];
                all = add(all, {d, (x[i] - d) - y[i]});
                last = i;
            }
            if ((i & 3) == 3) all = normal(all);                   // sixteen additions in a row would be too many
            own[i] = all;
        }
        const double mine_all = value(all);
        double up = mine_all;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const double o = __shfl_up_sync(0xffffffffu, up, m);
            if (lane >= m) up += o;
        }
        // what is left of the goal at this lane's first value
        const double rest = goal - (base + (up - mine_all));
        const Pair r{(float)rest, (float)(rest - (double)(float)rest)};
        int here = kVerifyPer;
#pragma unroll
        for (int i = kVerifyPer - 1; i >= 0; --i)
            if (x[i] > y[i] && (own[i].hi - r.hi) + (own[i].lo - r.lo) > 0.f) here = i;
        const uint32_t past = __ballot_sync(0xffffffffu, here < kVerifyPer), any = __ballot_sync(0xffffffffu, last >= 0);
        const int who = past ? __ffs(past) - 1 : 31 - __clz(any);
        if (lane == who) out[a] = at + (past ? here : last);
        return;
    }
}

}  // namespace

namespace {

template <int T>
cudaError_t launch_threads(const VerifyParams& p, int cluster, cudaStream_t stream) {
    auto kernel = verify_drafts_kernel<T>;
    const int tiles = (p.vocab + kVerifyTile - 1) / kVerifyTile;
    const int smem = (tiles + cluster - 1) / cluster * (int)sizeof(Pair);
    cudaError_t e = ensure_smem_attribute(reinterpret_cast<const void*>(kernel), kMaxVerifyVocab / kVerifyTile * (int)sizeof(Pair));
    if (e != cudaSuccess) return e;
    return launch_overlapped(kernel, p, dim3(p.num_seqs * cluster), T, smem, stream, cluster);
}

}  // namespace

// Few requests: as many warps as tiles, in clusters of up to eight CTAs. A batch: small CTAs,
// several to a request, so that the SMs' shares are even. Clusters grow only as far as they all
// run at once (75 requests of 128,256 tokens in clusters of eight, one of which waits: 34.5 us,
// in clusters of four 27; 150: 44.6, 41.3). Small CTAs against large ones: 256 requests 51 us
// and 52; 96 of them 34 and 31, 64 of them 23 and 28, 16 of them 14 and 15, so the border in
// between is a rough one.
cudaError_t launch_verify_drafts(const VerifyParams& p, cudaStream_t stream) {
    const int tiles = (p.vocab + kVerifyTile - 1) / kVerifyTile;
    const bool batch = p.num_seqs > 76;
    const int warps = batch ? 4 : 8;
    int cluster = 1;
    while (cluster < kVerifyCluster && (long long)p.num_seqs * cluster * 2 * warps <= kVerifyWave && tiles > cluster * warps) cluster *= 2;
    return batch ? launch_threads<128>(p, cluster, stream) : launch_threads<256>(p, cluster, stream);
}

}  // namespace pagedkv
