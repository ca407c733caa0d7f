// step_tables.cu -- block tables and slot maps built on the device from request
// lengths, for a step whose lengths the host does not know (how many drafted
// tokens were accepted, which requests end): the growth of every request's table
// from a stack of free blocks, and its counterpart.
//
// Extend. With held_s = ceil(L_s / B) and need_s = ceil((L_s + n_s) / B) - held_s,
// exclusive sums over the requests in their order give the first token
// (query_start) and the first block (before_s) of each; block k of request s is
// entry F - 1 - (before_s + k) of the stack of F free blocks, and the token at
// position p has slot table[p / B] * B + p mod B.
// Trim. With d_s tokens dropped, blocks ceil((L_s - d_s) / B) .. held_s - 1 go back,
// in the reverse of the order in which extend would take them.
//
// One launch of one cluster. Every CTA makes the sums for itself (a few kilobytes
// of lengths, in shared memory from then on), meets the others once, so that the
// outputs may be the inputs' own memory, and then takes its share of the entries
// and slots, one a thread, found by binary search over the sums. The work is
// launch latency and two or three dependent loads; sums in a kernel of their own
// would cost a launch more. A prompt step's slots are too many for one cluster's
// eight SMs (some 130,000 of them took 23 us): from kSlotsApart on a second kernel
// fills the whole device with them, from the first one's outputs (9.4 us). 4 requests of a
// token each take 3.4 us, 512 of five 5.4, 512 trimmed 8 (each CTA sums all requests first).
#include <cooperative_groups.h>

#include "device_common.cuh"
#include "launch.h"

namespace pagedkv {

namespace {

namespace cg = cooperative_groups;

constexpr int kTablesThreads = 1024;
constexpr int kTablesCluster = 8;
constexpr int64_t kSlotsApart = 16384;             // slots from which they have a kernel of their own
constexpr int64_t kMaxTableTokens = INT32_MAX - 1024;      // lengths round up to blocks in 32 bits

// Sums of a and b over the CTA's threads before this one; totals in ta, tb.
__device__ __forceinline__ void scan_two(int64_t& a, int64_t& b, int64_t& ta, int64_t& tb, int64_t (*part)[2]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int64_t ia = a, ib = b;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int64_t xa = __shfl_up_sync(0xffffffffu, ia, m), xb = __shfl_up_sync(0xffffffffu, ib, m);
        if (lane >= m) {
            ia += xa;
            ib += xb;
        }
    }
    __syncthreads();                               // part is free
    if (lane == 31) {
        part[warp][0] = ia;
        part[warp][1] = ib;
    }
    __syncthreads();
    int64_t sa = lane < warps ? part[lane][0] : 0, sb = lane < warps ? part[lane][1] : 0;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int64_t xa = __shfl_up_sync(0xffffffffu, sa, m), xb = __shfl_up_sync(0xffffffffu, sb, m);
        if (lane >= m) {
            sa += xa;
            sb += xb;
        }
    }
    ta = __shfl_sync(0xffffffffu, sa, 31);
    tb = __shfl_sync(0xffffffffu, sb, 31);
    const int64_t pa = __shfl_sync(0xffffffffu, sa, (warp + 31) & 31), pb = __shfl_sync(0xffffffffu, sb, (warp + 31) & 31);
    a = ia - a + (warp ? pa : 0);
    b = ib - b + (warp ? pb : 0);
}

// The largest s in [0, n) with first[s] <= x; first[0] <= x. `top`: the largest power of
// two below n (0 for n = 1).
__device__ __forceinline__ int owner_of(const int32_t* first, int n, int top, int x) {
    int s = 0;
    for (int step = top; step; step >>= 1)
        if (s + step < n && first[s + step] <= x) s += step;
    return s;
}
__device__ __forceinline__ int top_step(int n) { return n > 1 ? 1 << (31 - __clz(n - 1)) : 0; }

__device__ __forceinline__ void flag(uint32_t* status, uint32_t bit) {
    if (status) atomicOr(status, bit);
}

// F, brought into the stack's capacity.
__device__ __forceinline__ int64_t free_count(const TablesParams& p, bool report) {
    const int64_t F = *p.num_free;
    if (F >= 0 && F <= p.free_capacity) return F;
    if (report && threadIdx.x == 0) flag(p.status, PA_DEV_BAD_BLOCK_ID);
    return F < 0 ? 0 : p.free_capacity;
}

__global__ void __launch_bounds__(kTablesThreads)
extend_tables_kernel(const __grid_constant__ TablesParams p) {
    begin_overlapped();
    extern __shared__ int32_t sums[];
    const int S = p.num_seqs;
    int32_t* len = sums;                           // [S]
    int32_t* tok = len + S;                        // [S] first token of each request
    int32_t* blk = tok + S;                        // [S] its first new block
    __shared__ int64_t part[32][2];
    const cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const bool lead = rank == 0;
    const int B = p.block_size;
    const int64_t room = (int64_t)p.max_blocks * B, T = p.max_tokens;
    const int64_t F = free_count(p, lead);
    int64_t asked = 0, needed = 0, tokens = 0, taken = 0;      // sums over the requests so far
    for (int s0 = 0; s0 < S; s0 += blockDim.x) {
        const int s = s0 + threadIdx.x;
        int64_t L = 0, n = 0;
        if (s < S) {
            L = p.context_lens[s];
            n = p.new_tokens[s];
            if (L < 0 || n < 0 || L + n > room || L + n > kMaxTableTokens) {
                if (lead) flag(p.status, PA_DEV_BAD_LEN);
                n = 0;
            }
        }
        const int64_t need = n ? (int)(L + n + B - 1) / B - (int)(L + B - 1) / B : 0;
        int64_t a = n, b = need, ta, tb;
        scan_two(a, b, ta, tb, part);
        // a request is served if its blocks and its places in the slot map are there
        // after those of the requests before it
        const bool blocks = need == 0 || needed + b + need <= F;
        const bool places = asked + a + n <= T;
        if (lead && n && !(blocks && places)) flag(p.status, blocks ? PA_DEV_BAD_LEN : PA_DEV_NO_BLOCKS);
        const int64_t got = blocks && places ? n : 0;
        // the sums over those served: the same ones where all are
        int64_t first = a, served = ta;
        const bool all = __syncthreads_and(got == n);
        if (!all) {
            int64_t unused = 0, none;
            first = got;
            scan_two(first, unused, served, none, part);
        }
        // blocks are taken by a leading run of the requests that need any: the sums
        // before a served one count served ones alone
        if (all) {
            if (tb) taken = needed + tb;
        } else {
            const int used = got && need ? (int)(needed + b + need) : 0;
            const int most = __reduce_max_sync(0xffffffffu, used);
            __syncthreads();
            if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5][0] = most;
            __syncthreads();
            for (int w = 0; w < (int)(blockDim.x >> 5); ++w) taken = max(taken, part[w][0]);
        }
        if (s < S) {
            len[s] = (int32_t)L;
            tok[s] = (int32_t)(tokens + first);
            blk[s] = (int32_t)min(needed + b, taken);
        }
        asked += ta;
        needed = min(needed + tb, (int64_t)INT32_MAX);
        tokens += served;
    }
    if (ranks > 1) cluster.sync();
    else __syncthreads();
    // from here on the inputs that the outputs may lie over have been read
    const int total = (int)tokens;
    auto new_tokens = [&](int s) { return (s + 1 < S ? tok[s + 1] : total) - tok[s]; };
    if (lead) {
        for (int s = threadIdx.x; s < S; s += blockDim.x) {
            p.query_start[s] = tok[s];
            p.new_lens[s] = len[s] + new_tokens(s);
        }
        if (threadIdx.x == 0) {
            p.query_start[S] = total;
            *p.new_num_free = (int32_t)(F - taken);
        }
    }
    const int me = rank * blockDim.x + threadIdx.x, threads = ranks * blockDim.x;
    const int top = top_step(S);
    // (`left` counts down: the step beyond the last may pass 2^31)
    for (int k = me, left = (int)taken - me; left > 0; left -= threads, k += left > 0 ? threads : 0) {
        // several requests may share a first block where all but the last need none
        const int s = owner_of(blk, S, top, k);
        p.block_tables[(size_t)s * p.max_blocks + (len[s] + B - 1) / B + (k - blk[s])] = p.free_blocks[F - 1 - k];
    }
    if (p.slots_apart) return;
    for (int64_t t = me; t < T; t += threads) {
        int64_t slot = -1, pos = 0;
        if (t < total) {
            const int s = owner_of(tok, S, top, (int)t);
            const int L = len[s], at = L + ((int)t - tok[s]);
            const int j = at / B, held = (L + B - 1) / B;
            const int64_t id = j < held ? p.block_tables[(size_t)s * p.max_blocks + j]
                                        : p.free_blocks[F - 1 - (blk[s] + (j - held))];
            slot = id * B + (at - j * B);
            pos = at;
        }
        p.slot_mapping[t] = slot;
        if (p.positions) p.positions[t] = pos;
    }
}

// The slots and positions of many tokens, from the starts, lengths and tables as extend
// left them: kSlotsPer neighbours a thread.
constexpr int kSlotsThreads = 256;
constexpr int kSlotsPer = 4;

__global__ void __launch_bounds__(kSlotsThreads)
fill_slots_kernel(const __grid_constant__ TablesParams p) {
    begin_overlapped();
    const int S = p.num_seqs, B = p.block_size;
    const int64_t T = p.max_tokens;
    const int64_t t0 = ((int64_t)blockIdx.x * kSlotsThreads + threadIdx.x) * kSlotsPer;
    if (t0 >= T) return;
    const int total = p.query_start[S];
    int64_t slot[kSlotsPer], pos[kSlotsPer];
#pragma unroll
    for (int i = 0; i < kSlotsPer; ++i) {
        slot[i] = -1;
        pos[i] = 0;
    }
    if (t0 < total) {
        int s = owner_of(p.query_start, S, top_step(S), (int)t0);
        int end = p.query_start[s + 1], ahead = p.new_lens[s] - end;       // a token's position less its row
        int j = -1;
        int64_t id = 0;
#pragma unroll
        for (int i = 0; i < kSlotsPer; ++i) {
            const int t = (int)t0 + i;
            if (t < total) {
                while (t >= end) {
                    ++s;
                    end = p.query_start[s + 1];
                    ahead = p.new_lens[s] - end;
                    j = -1;
                }
                const int at = t + ahead;
                if (at / B != j) {
                    j = at / B;
                    id = p.block_tables[(size_t)s * p.max_blocks + j];
                }
                slot[i] = id * B + (at - j * B);
                pos[i] = at;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kSlotsPer; ++i)
        if (t0 + i < T) {
            p.slot_mapping[t0 + i] = slot[i];
            if (p.positions) p.positions[t0 + i] = pos[i];
        }
}

__global__ void __launch_bounds__(kTablesThreads)
trim_tables_kernel(const __grid_constant__ TablesParams p) {
    begin_overlapped();
    extern __shared__ int32_t sums[];
    const int S = p.num_seqs;
    int32_t* len = sums;                           // [S] the new length
    int32_t* from = len + S;                       // [S] the first block given back
    int32_t* blk = from + S;                       // [S] its place among all that are
    __shared__ int64_t part[32][2];
    const cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const bool lead = rank == 0;
    const int B = p.block_size;
    const int64_t room = (int64_t)p.max_blocks * B;
    const int64_t F = free_count(p, lead);
    int64_t given = 0;
    for (int s0 = 0; s0 < S; s0 += blockDim.x) {
        const int s = s0 + threadIdx.x;
        int64_t L = 0, d = 0, keep = 0, count = 0;
        if (s < S) {
            L = p.context_lens[s];
            d = p.new_tokens[s];
            if (L < 0 || L > room || L > kMaxTableTokens || d < 0 || d > L) {
                if (lead) flag(p.status, PA_DEV_BAD_LEN);
                d = 0;
            }
            if (d) {
                keep = (int)(L - d + B - 1) / B;
                if (p.shared_blocks) keep = max(keep, (int64_t)p.shared_blocks[s]);
                count = max((int64_t)0, (int)(L + B - 1) / B - keep);
            }
        }
        int64_t a = count, unused = 0, ta, tb;
        scan_two(a, unused, ta, tb, part);
        if (s < S) {
            len[s] = (int32_t)(L - d);
            from[s] = (int32_t)keep;
            blk[s] = (int32_t)min(given + a, (int64_t)INT32_MAX);
        }
        given += ta;
    }
    const bool fits = F + given <= p.free_capacity;
    if (!fits && lead && threadIdx.x == 0) flag(p.status, PA_DEV_BAD_BLOCK_ID);
    if (ranks > 1) cluster.sync();
    else __syncthreads();
    if (lead) {
        // a stack that cannot take them back: nothing is dropped
        for (int s = threadIdx.x; s < S; s += blockDim.x) p.new_lens[s] = fits ? len[s] : p.context_lens[s];
        if (threadIdx.x == 0) *p.new_num_free = (int32_t)(fits ? F + given : F);
    }
    if (!fits) return;
    // a warp takes runs of neighbours, most often one request's: their first and last tell
    constexpr int kAtOnce = 4, kRun = 32 * kAtOnce;                // entries whose loads are in flight together
    const int lane = threadIdx.x & 31, warps = ranks * (int)(blockDim.x >> 5), top = top_step(S);
    // (unsigned: the run beyond the last may pass 2^31)
    for (uint32_t k0 = (rank * (blockDim.x >> 5) + (threadIdx.x >> 5)) * kRun; k0 < (uint32_t)given; k0 += warps * kRun) {
        const int left = (int)given - (int)k0;
        const int lo = owner_of(blk, S, top, (int)k0), hi = owner_of(blk, S, top, (int)k0 + min(kRun, left) - 1);
        int32_t id[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            if (32 * i + lane < left) {
                const int k = (int)k0 + 32 * i + lane;
                const int s = lo == hi ? lo : lo + owner_of(blk + lo, hi - lo + 1, top_step(hi - lo + 1), k);
                id[i] = p.block_tables[(size_t)s * p.max_blocks + from[s] + (k - blk[s])];
            }
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
            if (32 * i + lane < left) p.stack[F + given - 1 - (int)k0 - (32 * i + lane)] = id[i];
    }
}

}  // namespace

cudaError_t launch_tables(const TablesParams& tables, bool extend, cudaStream_t stream) {
    TablesParams p = tables;
    p.slots_apart = extend && p.max_tokens > kSlotsApart;
    // entries and slots to write, about: a request in four gives all its blocks back at worst
    const int64_t work = !extend ? (int64_t)p.num_seqs * p.max_blocks / 4
                                 : (p.slots_apart ? p.max_tokens / p.block_size : p.max_tokens);
    // Small calls in small CTAs: 4 requests of a token 3.3 us and 3.8 in 1,024 threads, 32 of four
    // 3.4 and 4.2, though 128 of four, at the border, 5.9 and 4.7. One CTA up to a slot a thread:
    // 512 requests of two 5.2 us and 5.4 in eight; of three 6.2 and 5.6. Slots apart: 512 requests
    // of 31 (15,872) 7.0 us in one kernel and 10.4 in two, 16 of 1,100 (17,600) 6.2 and 7.7, 64 of
    // 4,096 31 and 10.2.
    const int threads = p.num_seqs <= 128 && work <= 512 ? 128 : kTablesThreads;
    const int cluster = work <= kTablesThreads ? 1 : kTablesCluster;
    auto kernel = extend ? extend_tables_kernel : trim_tables_kernel;
    const int smem = 12 * p.num_seqs;
    cudaError_t e = ensure_smem_attribute(reinterpret_cast<const void*>(kernel), 12 * kMaxTableSeqs);
    if (e != cudaSuccess) return e;
    e = launch_overlapped(kernel, p, dim3(cluster), threads, smem, stream, cluster);
    if (e != cudaSuccess || !p.slots_apart) return e;
    const int64_t per = kSlotsThreads * kSlotsPer;
    return launch_overlapped(fill_slots_kernel, p, dim3((unsigned)((p.max_tokens + per - 1) / per)), kSlotsThreads, 0, stream);
}

}  // namespace pagedkv
