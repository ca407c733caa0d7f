// scaled_prefill.cuh -- attention over block-scaled 8-bit codes for many query rows
// (prompt chunks, large groups' drafts) on the 5th-generation tensor cores.
//
// Work unit: (sequence, KV head, two tiles of 128 query rows, partition of the
// context), one CTA on an SM. Rows are (query token, head of the group) pairs,
// token-major, as in scaled_attention.cuh, whose definitions hold here. Key tiles of
// 128. Two streams, each with scores, weights and an output of its own in TMEM, so
// that the tensor cores work for one while the other's softmax runs: the two query
// tiles over the same key tiles, or, where one tile holds all rows (drafts), the
// even and the odd key tiles, joined at the end. At head size 256 TMEM holds one output: one
// stream of one query tile, key tiles of 64, and scores in two places by turns, so that the
// next are on their way during a softmax (8 chunks of 512, 16/4 heads: 180-206 us by card, 668
// TFLOP/s at 206; 1,287 on warp-level tiles of 16 rows). Roles:
//   warps 0-3, 4-7   softmax of stream 0, 1: a thread a row;
//   warps 8-11       load K (12-14: V): codes from the cache's blocks into two staging slots
//                    of a warp's own by asynchronous copies, 32 keys at a time in two pieces,
//                    the next slice's under way; from there widened to binary16 -- exactly, as
//                    in scaled_attention.cuh -- into the swizzled tiles that the MMAs read;
//   warp 15          issues tcgen05.mma: S0, S1, then PV0, S0', PV1, S1', ...
// A softmax warp without rows (40 rows of drafts leave two of four) is a fourth for V.
// What bounds it is a stream's chain of scores, softmax and P V -- a warp gets an instruction
// in about eight cycles -- and the loaders' instructions beside it. Slices of 32 keys, whose
// bookkeeping is done once and the blocks looked up by a lane each, took drafts (64 contexts of
// 2304 tokens, 5 drafted each) from 147 us to 129 where 16 keys had taken 300 instructions; P V of
// half of the keys while the others' weights are made, 133 to 128 (two terms: 167 to 158; 155 with
// both terms in one store).
// The roles' loops together have to fit the instruction cache: loops of their own for K and V,
// unrolled over register buffers, and an issuer inlined three times had four in ten warps
// waiting for instructions: 482 us for 8 chunks of 512 that take 366 with one copy of each. A
// softmax holds 64 scores at a time for the same reason, and so that 16 warps of 128 registers
// do without a split of them by role. 17 warps of 96 registers and 16 scores at a time: 420 us;
// two threads a row (24 warps of 80): 387, though drafts in two terms gain 4 %.
// (The fence between the loaders' stores and the MMAs' reads is the issuer's, which waits
// for the tile: a loader's own waited for its loads in flight, 541 us for 510.)
//
// The scales stay out of the tiles. Blocks are multiples of kG = 16 or 8 tokens here, so a
// group of kG columns of S has one key scale a and one value scale b: with raw
// scores s and the row's unit u (scale, log2 e and the query's power of two),
//     weight = 2^(s (u a) + (log2 b - d + 6) - m),
// one fused multiply-add and one exponential a score; the maximum is taken over raw
// scores within a group (a >= 0) and the row's sum gets each group's weights divided by
// 2^(log2 b - d + 6) again. d follows the largest of s (u a) + log2 b - m among the keys
// that the row sees (one addition a group and row more than a unit for all rows by the
// largest value scale, 1 % of the chunks' time; but that one gave the bits of all weights
// to a block of large values that a row hardly attends to or does not see): the row's
// largest weight reaches the MMA between 2^5 and 2^14, rounded to binary16 (2^-11 of
// itself; with a binary16 output, whose own step is no larger, in two terms, 2^-22). A
// value scale below 2^(d - 60) counts as that: its weights vanish in binary16 either way.
//
// Every wait is bounded, as in prefill_tc.cuh.
#pragma once

#include "prefill_tc.cuh"
#include "scaled_attention.cuh"

namespace pagedkv {

constexpr int kSpThreads = 16 * 32;
constexpr int kSpMmaWarp = 15;
constexpr int kSpLoaders = 4;                      // warps for K, one less for V; and up to three softmax warps without rows
constexpr int kSpSlices = 4;                       // of a key tile, each a loader's at a time
constexpr int kSpRing = 8;                         // tiles whose scales are kept
constexpr float kSpMoveLog2 = 8.f;                 // a row's references move when a score, a weight, passes them by this
constexpr float kSpNoWeight = -1e4f;

template <int D>
struct SpShape {
    static constexpr bool kOne = D == 256;                             // one stream
    static constexpr int N = kOne ? 64 : 128;                          // keys of a tile
    static constexpr int kSlice = N / kSpSlices, kPiece = kSlice / 2;  // of a slice, of its pieces
    static constexpr int kRows = kOne ? kTcRows : 2 * kTcRows;
    static constexpr int kQBytes = kTcRows * D * 2;                    // a query tile
    static constexpr int kTile = N * D * 2;                            // a K (V) stage
    static constexpr int NSK = 2, NSV = 2;
    static constexpr int kKOff = kRows / kTcRows * kQBytes;
    static constexpr int kVOff = kKOff + NSK * kTile;
    static constexpr int kStagingOff = kVOff + NSV * kTile;            // two pieces of codes for each loader
    static constexpr int kSlot = kPiece * D;
    static constexpr int kBarOff = kStagingOff + (2 * kSpLoaders - !kOne) * 2 * kSlot;
    // k_full[NSK] k_empty[NSK] v_full[NSV] v_empty[NSV] scales[kSpRing] s_full[2] p_full[4] drain q_ready
    static constexpr int kNumBars = 2 * NSK + 2 * NSV + kSpRing + 8;
    static constexpr int kMiscOff = kBarOff + kNumBars * 8;            // tmem base, abort flag
    static constexpr int kScaleOff = (kMiscOff + 16 + 15) / 16 * 16;   // [kSpRing][N / kG] pairs (a, log2 b)
    static constexpr int kUnitOff = kScaleOff + kSpRing * (N / 8) * 8;     // [256] the rows' powers of two, biased exponents
    static constexpr int kBytes = kUnitOff + 256;
    static constexpr int kAlloc = kBytes + 1024;
    static constexpr int kTmemCols = 512;
    // S (then P) and O of each stream; of one stream, S twice and O
    static constexpr int kSCols = kOne ? N : N + D;                    // from one S to the other
    static constexpr int kOCol = kOne ? 2 * N : N;
    static_assert((kOne ? 2 * N + D : 2 * (N + D)) <= kTmemCols, "TMEM columns");
    static_assert(kOne || 2 * kSlot <= kQBytes, "a loader more has its slots in the second query tile's place");
    static_assert(2 * kTcRows * 4 <= kTile, "the streams trade maxima and sums in a K stage");
    static_assert(kAlloc <= kTcSmemLimit, "shared memory");
    // Scales live until both softmaxes have read them: a loader writes those of tile j once it
    // has passed the wait for tile j - 1's slot, so S of tile j - 1 - NSK (K) or P.V of tile
    // j - 1 - NSV (V) is done. S of a tile comes after the weights of the tile two before it.
    static_assert(kSpRing >= NSK + 3 && kSpRing >= NSV + 1, "scales");
};

// tcgen05.mma and its commit from a whole warp, issued by the lane whose `leader` is set. The
// warp stays together, so that descriptors and loop counts live in uniform registers, where the
// instruction takes them from; a lone lane moves each of them there (100 cycles an instruction).
__device__ __forceinline__ void sp_mma(uint32_t leader, uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(leader) : "memory");
}
__device__ __forceinline__ void sp_mma_ts(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate), "r"(leader) : "memory");
}
__device__ __forceinline__ void sp_commit(uint32_t leader, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
        ::"r"(smem_u32(bar)), "r"(leader) : "memory");
}

__device__ __forceinline__ float ld_shared(uint32_t at) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint4 ld_shared4(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}

// tcgen05.wait::ld, on which the loaded registers depend: no use moves above it. (Nothing that
// could move the registers themselves, a branch or a wait, stands between a load and this.)
__device__ __forceinline__ void tc_wait_ld32(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                   "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                   "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :: "memory");
}

// One loader warp's slices of an operand: slice n = 8 j + q is keys 16 q .. of tile j.
// Keys and values, and every warp that loads, run the same code, inlined once.
// At most kSpSlices warps load an operand, so that each has a slice of every tile: waiting for a
// stage's phase by parity needs that.
template <typename CT, int D, int kG>
__device__ __forceinline__ void sp_load(const ScaledAttnParams& p, bool keys, const uint8_t* staging, uint8_t* ring, int stages, float* scales,
                                        uint64_t* full, uint64_t* empty, uint64_t* scale_bar, int s, int kvh, int T0, int kend,
                                        int ntiles, int which, int loaders, int lane, volatile int* abort_flag) {
    using Sh = SpShape<D>;
    constexpr int CPR = D / 16;                    // 16-code chunks of a row
    constexpr int PER = Sh::kPiece * CPR / 32;       // of a lane's, of a piece
    constexpr int PARTS = Sh::kSlice / kG;           // runs of kG keys, in one block each
    constexpr int PIECE_PARTS = Sh::kPiece / kG, PER_PART = PER / PIECE_PARTS;
    const int32_t* table = p.block_tables + (size_t)s * p.max_blocks;
    const float* block_scales = keys ? p.k_scales : p.v_scales;
    const int B = p.block_size;
    const int last = kSpSlices * ntiles;
    // eight lanes that store together hold two rows of one 64-column span, in all banks
    const int chunk = D == 256 ? (lane & 3) + ((lane >> 3) << 2) : (D == 128 ? (lane & 3) + ((lane >> 1) & 4) : lane & 3);
    const int row0 = D == 256 ? (lane >> 2) & 1 : (D == 128 ? ((lane >> 2) & 1) + ((lane >> 4) << 1) : lane >> 2);
    constexpr int STEP = 32 / CPR;                 // rows of a pass
    const uint8_t* cache = (keys ? p.k_cache : p.v_cache) + chunk * 16;
    // Lane h, and those that repeat it, look up part h of the slices: table entry and row in
    // the block, which move on without a division.
    const int part = lane & (PARTS - 1);
    int left = kend - T0 - which * Sh::kSlice;       // keys from the slice to look up on
    int entry, in;
    {
        const int key = T0 + which * Sh::kSlice + part * kG;
        entry = (int)((uint64_t)(uint32_t)key * p.block_mul >> p.block_shift);
        in = key - entry * B;
    }
    const int entry_step = loaders * Sh::kSlice / B, in_step = loaders * Sh::kSlice % B;
    int blk = -1, blk_in = 0, blk_left = 0;
    auto look = [&] {
        blk_left = left;
        blk_in = in;
        blk = left > part * kG ? table[entry] : -1;
        entry += entry_step;
        in += in_step;
        if (in >= B) {
            in -= B;
            ++entry;
        }
        left -= loaders * Sh::kSlice;
    };
    // of the slice to copy: the part's first row in the pool (~0: none), its scale, keys left
    uint32_t row = ~0u;
    float scale = 0.f;
    int copy_left = 0;
    auto place = [&] {
        copy_left = blk_left;
        row = ~0u;
        scale = 0.f;
        if ((uint32_t)blk < (uint32_t)p.num_blocks) {
            const uint32_t slab = (uint32_t)blk * p.num_kv_heads + kvh;
            row = slab * B + blk_in;
            scale = block_scales[slab];
        } else if (lane < PARTS && copy_left > part * kG && p.status) {
            atomicOr(p.status, PA_DEV_BAD_BLOCK_ID);
        }
    };
    // a lane copies, and later widens, its own chunks: nothing of the staging slots is shared
    const uint32_t mine = smem_u32(staging) + lane * 16;
    auto fetch = [&](int piece, bool any) {
        if (any)
#pragma unroll
            for (int h = 0; h < PIECE_PARTS; ++h) {
                const uint32_t to = mine + piece * Sh::kSlot + h * PER_PART * 512;
                const uint32_t at = __shfl_sync(0xffffffffu, row, piece * PIECE_PARTS + h);
                const int here = copy_left - (piece * PIECE_PARTS + h) * kG;
                if (at != ~0u && here >= kG) {
                    const uint8_t* from = cache + (size_t)(at + row0) * D;
#pragma unroll
                    for (int i = 0; i < PER_PART; ++i) cp_async16(to + i * 512, from + i * STEP * D);
                } else {                           // the context's end, or a bad block: zeros
                    const int rows = at != ~0u ? here - row0 : 0;      // of this lane's, STEP apart
                    const uint8_t* from = cache + ((size_t)at + row0) * D;
#pragma unroll 1
                    for (int i = 0; i < PER_PART; ++i)
                        cp_async16(to + i * 512, i * STEP < rows ? from + i * STEP * D : cache, i * STEP < rows);
                }
            }
        cp_async_commit();
    };
    look();
    place();
    look();
    fetch(0, which < last);
    fetch(1, which < last);
    int tile = 0, st = 0;                          // of the slice to widen: key tile, its stage
    uint32_t phase = 1;                            // of its stage's `empty`; the first round waits for nothing
#pragma unroll 1
    for (int n = which; n < last; n += loaders) {
        const int q = n % kSpSlices;
        if (n / kSpSlices != tile) {
            ++tile;
            if (++st == stages) {
                st = 0;
                phase ^= 1u;
            }
        }
        const float now = scale;
        place();
        look();
        if (lane < PARTS) {
            float2* to = reinterpret_cast<float2*>(scales) + (tile % kSpRing) * (Sh::N / kG) + q * PARTS + lane;
            if (keys) to->x = now;
            else to->y = log2f(now);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&scale_bar[tile % kSpRing]);
        if (tile >= stages) {
            const bool ok = tc_wait(&empty[st], phase, p.status, abort_flag);
            if (!__all_sync(0xffffffffu, ok)) break;
        }
        uint8_t* to = ring + st * Sh::kTile + q * Sh::kSlice * 128;
#pragma unroll 1
        for (int piece = 0; piece < Sh::kSlice / Sh::kPiece; ++piece) {
            cp_async_wait<1>();
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const uint4 v = ld_shared4(mine + piece * Sh::kSlot + i * 512);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                uint32_t o[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t u = biased<CT>(w[k]);
                    o[2 * k] = widen2<CT>(u, 0x4140);
                    o[2 * k + 1] = widen2<CT>(u, 0x4342);
                }
                const int r = i * STEP + row0;
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    *reinterpret_cast<uint4*>(to + piece * Sh::kPiece * 128 + sw128_chunk<Sh::N>(r, 2 * chunk + h)) =
                        make_uint4(o[4 * h], o[4 * h + 1], o[4 * h + 2], o[4 * h + 3]);
            }
            fetch(piece, n + loaders < last);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[st]);     // the MMA issuer, which waits for it, has the fence between the proxies
    }
    cp_async_wait<0>();
}

// The sequence of this CTA: the longest contexts' first, so that what is left when SMs run
// out of work is short (64 contexts of 512-4096 tokens with 5 drafted: 121 us, 132 in their
// order; 8 chunks of 512 in contexts of 512-8192: 320 us, 366). With more than kSpSorted sequences there are waves enough for it not to matter.
constexpr int kSpSorted = 128;
__device__ __forceinline__ int sp_sequence(const int32_t* context_lens, int num_seqs, int* lens) {
    if (num_seqs == 1 || num_seqs > kSpSorted) return blockIdx.z;
    __shared__ int mine;
    const int t = threadIdx.x;
    int len = 0;
    if (t < kSpSorted) {
        len = t < num_seqs ? context_lens[t] : INT_MIN;
        lens[t] = len;
    }
    __syncthreads();
    if (t < num_seqs) {
        int longer = 0;
        for (int u = 0; u < num_seqs; u += 4) {
            const int4 v = *reinterpret_cast<const int4*>(lens + u);
            longer += (v.x > len || (v.x == len && u < t)) + (v.y > len || (v.y == len && u + 1 < t)) +
                      (v.z > len || (v.z == len && u + 2 < t)) + (v.w > len || (v.w == len && u + 3 < t));
        }
        if (longer == (int)blockIdx.z) mine = t;
    }
    __syncthreads();
    return mine;
}

template <typename CT, int D, int kG, bool kTwoTerms>
__global__ void __launch_bounds__(kSpThreads, 1)
scaled_prefill_kernel(const __grid_constant__ ScaledAttnParams p) {
    begin_overlapped();
    using Sh = SpShape<D>;
    constexpr bool kFp8 = std::is_same<CT, e4m3_t>::value;
    constexpr bool kOne = Sh::kOne;
    constexpr int N = Sh::N, NSK = Sh::NSK, NSV = Sh::NSV;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* k_full = reinterpret_cast<uint64_t*>(sm + Sh::kBarOff);
    uint64_t* k_empty = k_full + NSK;
    uint64_t* v_full = k_empty + NSK;
    uint64_t* v_empty = v_full + NSV;
    uint64_t* scale_bar = v_empty + NSV;           // [kSpRing]
    uint64_t* s_full = scale_bar + kSpRing;        // [2], by query tile
    uint64_t* p_full = s_full + 2;                 // [half of the keys][query tile]
    uint64_t* drain = p_full + 4;
    uint64_t* q_ready = drain + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + Sh::kMiscOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + Sh::kMiscOff + 4);
    float2* scales = reinterpret_cast<float2*>(sm + Sh::kScaleOff);
    uint8_t* units = sm + Sh::kUnitOff;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int s = sp_sequence(p.context_lens, p.num_seqs, reinterpret_cast<int*>(sm));
    const int pair = blockIdx.y / p.num_kv_heads, kvh = blockIdx.y - pair * p.num_kv_heads;
    int L, q0, Q;
    if (!scaled_sequence(p, s, tid == 0 && blockIdx.x == 0 && blockIdx.y == 0, L, q0, Q)) return;
    const int G = p.group;
    const int row0 = pair * Sh::kRows, rows = min(Sh::kRows, Q * G - row0);
    if (rows <= 0) return;
    const bool two = rows > kTcRows;               // query tiles; else the streams take alternate key tiles
    const int first_pos = L - Q;
    const int seen = first_pos + (row0 + rows - 1) / G + 1;
    const int T0 = blockIdx.x * p.partition_size;
    if (T0 >= seen) {
        // a token with an empty context: zeros (with partitions, from their merge)
        if (seen <= 0 && p.max_parts == 1) {
            uint4* to = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + ((size_t)q0 * p.num_q_heads + kvh * G + row0) * D);
            for (int i = tid; i < rows * (D / 8); i += kSpThreads) to[i] = make_uint4(0u, 0u, 0u, 0u);
        }
        return;
    }
    const int kend = min(T0 + p.partition_size, seen);
    const int ntiles = (kend - T0 + N - 1) / N;
    // stream t's steps, and the key tile of step i
    auto steps_of = [&](int t) { return kOne ? (t ? 0 : ntiles) : (two ? ntiles : (ntiles + 1 - t) / 2); };
    auto tile_of = [&](int t, int i) { return two || kOne ? i : 2 * i + t; };
    // softmax warps with rows in stream t
    auto warps_of = [&](int t) { return (min(kTcRows, two ? rows - t * kTcRows : rows) + 31) >> 5; };
    const bool join = !kOne && !two && ntiles > 1;          // the streams' results are one

    if (tid == kSpMmaWarp * 32) {
        for (int i = 0; i < NSK; ++i) {
            mbar_init(&k_full[i], kSpSlices);
            mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < NSV; ++i) {
            mbar_init(&v_full[i], kSpSlices);
            mbar_init(&v_empty[i], 1);
        }
        for (int i = 0; i < kSpRing; ++i) mbar_init(&scale_bar[i], 2 * kSpSlices);
        for (int t = 0; t < 2; ++t) {
            mbar_init(&s_full[t], 1);
            mbar_init(&p_full[t], max(1, warps_of(t)));
            mbar_init(&p_full[2 + t], max(1, warps_of(t)));
        }
        mbar_init(drain, 1);
        mbar_init(q_ready, kTcSoftmaxThreads / 32);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == kSpMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(tmem_slot)), "r"(Sh::kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == kSpMmaWarp) {
        const uint32_t leader = lane == 0;
        auto wait = [&](uint64_t* bar, int parity) {
            return __all_sync(0xffffffffu, tc_wait(bar, (uint32_t)(parity & 1), p.status, abort_flag)) != 0;
        };
        constexpr uint32_t idS = tc_idesc<__half>(kTcRows, N, 0);
        constexpr uint32_t idO = tc_idesc<__half>(kTcRows, D, 1);
        // the operands' descriptors; an address adds to their low bits (in units of 16 bytes)
        const uint64_t q_desc = tc_desc(smem_u32(sm), 16, 1024);
        const uint64_t k_desc = tc_desc(smem_u32(sm + Sh::kKOff), 16, 1024);
        const uint64_t v_desc = tc_desc(smem_u32(sm + Sh::kVOff), N * 128, 1024);
        // S of stream t's step i; of one stream, S into place t
        auto qk = [&](int t, int i) -> bool {
            const int j = tile_of(t, i), st = j % NSK;
            if (t == 0 || !two) {
                if (!wait(&k_full[st], j / NSK)) return false;
                fence_async_smem();
                tc_fence_after();
            }
            const uint64_t qa = q_desc + (two && t ? Sh::kQBytes >> 4 : 0);
            const uint64_t ka = k_desc + st * (Sh::kTile >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t q_off = ((kk >> 2) * (kTcRows * 128) + (kk & 3) * 32) >> 4;
                const uint32_t k_off = ((kk >> 2) * (N * 128) + (kk & 3) * 32) >> 4;
                sp_mma(leader, tmem + t * Sh::kSCols, qa + q_off, ka + k_off, idS, kk > 0);
            }
            if (t == 1 || !two) sp_commit(leader, &k_empty[st]);
            sp_commit(leader, &s_full[t]);
            return true;
        };
        auto pv = [&](int t, int i) -> bool {
            const int j = tile_of(t, i), st = j % NSV;
            const uint64_t va = v_desc + st * (Sh::kTile >> 4);
            const uint32_t pt = tmem + t * Sh::kSCols, ot = tmem + (kOne ? 0 : t * Sh::kSCols) + Sh::kOCol;
#pragma unroll 1
            for (int h = 0; h < N / 64; ++h) {                         // the first half while the second's weights are made
                if (!wait(&p_full[2 * h + t], kOne ? i >> 1 : i)) return false;
                if (h == 0 && (t == 0 || !two)) {
                    if (!wait(&v_full[st], j / NSV)) return false;
                    fence_async_smem();
                }
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                    for (int u = 0; u < (kTwoTerms ? 2 : 1); ++u)
                        sp_mma_ts(leader, ot, pt + h * 64 + (kk >> 1) * 32 + u * 16 + (kk & 1) * 8,
                                  va + (h * 4 + kk) * (2048 >> 4), idO, i > 0 || h > 0 || u > 0 || kk > 0);
            }
            if (t == 1 || !two) sp_commit(leader, &v_empty[st]);
            return true;
        };
        bool ok = wait(q_ready, 0);
        tc_fence_after();
        if constexpr (kOne) {
            // the next scores are on their way while a softmax runs
            ok = ok && qk(0, 0);
#pragma unroll 1
            for (int i = 0; i < ntiles && ok; ++i) {
                if (i + 1 < ntiles) ok = qk((i + 1) & 1, i + 1);
                if (ok) ok = pv(i & 1, i);
            }
        } else {
#pragma unroll 1
            for (int i = -1; i < steps_of(0) && ok; ++i)
#pragma unroll 1
                for (int t = 0; t < 2 && ok; ++t) {
                    if (i >= 0 && i < steps_of(t)) ok = pv(t, i);
                    if (ok && i + 1 < steps_of(t)) ok = qk(t, i + 1);
                }
        }
        // everything issued ends before the epilogue reads O and before TMEM is freed
        sp_commit(leader, drain);
        mbar_wait_bounded(drain, 0, p.status);
    } else {
        const int qt = warp >> 2;                                      // the stream
        auto over_group = [&](int r) { return (int)((uint64_t)(uint32_t)r * p.group_mul >> p.group_shift); };
        const int r = tid & (kTcRows - 1);
        // ---- the query, under a power of two for each row: a group of lanes a row
        if (warp < kTcSoftmaxThreads / 32) {
            constexpr int CPR = D / 8;                                 // 16-byte chunks of a row
            constexpr int RPW = 32 / CPR;                              // rows at a time
            const int c = lane % CPR;
            constexpr int ROWS = Sh::kRows / 8;                        // of a warp
            uint4 v[ROWS / RPW];
#pragma unroll
            for (int i = 0; i < ROWS / RPW; ++i) {
                const int rr = warp * ROWS + i * RPW + lane / CPR, row = row0 + rr;
                v[i] = make_uint4(0u, 0u, 0u, 0u);
                if (rr < rows) {
                    const int token = over_group(row);
                    v[i] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.query) +
                                                           ((size_t)(q0 + token) * p.num_q_heads + kvh * G + row - token * G) * D + c * 8);
                }
            }
#pragma unroll
            for (int i = 0; i < ROWS / RPW; ++i) {
                const int rr = warp * ROWS + i * RPW + lane / CPR;
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
                if (rr < kTcRows || two) {                             // (else its place is a loader's)
                    *reinterpret_cast<uint4*>(sm + (rr >> 7) * Sh::kQBytes + sw128_chunk<kTcRows>(rr & (kTcRows - 1), c)) = make_uint4(w[0], w[1], w[2], w[3]);
                    if (c == 0) units[rr] = (uint8_t)(__float_as_uint(unit) >> 23);
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_ready);
            if (!two) named_barrier(4, kTcSoftmaxThreads);             // both streams read the first tile's units
        }
        // ---- loaders: warps 8-14, and a softmax warp without rows
        const bool spare = kOne ? warp == 4 : warp < 8 && !two && (warp & 3) >= warps_of(qt);
        const int steps = warp < 8 ? steps_of(qt) : 0;
        if (warp >= 8 || spare) {
            const bool keys = !spare && warp < 8 + kSpLoaders;
            const bool more = kOne || (!two && warps_of(1) < 4);       // a fourth for V: the first such warp of stream 1
            if (!spare || warp == 4 + (kOne ? 0 : warps_of(1)))
                sp_load<CT, D, kG>(p, keys, !spare ? sm + Sh::kStagingOff + (warp - 8) * 2 * Sh::kSlot
                                                   : (kOne ? sm + Sh::kStagingOff + 7 * 2 * Sh::kSlot : sm + Sh::kQBytes),
                                   sm + (keys ? Sh::kKOff : Sh::kVOff), keys ? NSK : NSV, reinterpret_cast<float*>(scales),
                                   keys ? k_full : v_full, keys ? k_empty : v_empty, scale_bar, s, kvh, T0, kend, ntiles,
                                   spare ? 3 : warp & 3, keys || more ? kSpLoaders : kSpLoaders - 1, lane, abort_flag);
            if (spare && join) named_barrier(3, kTcSoftmaxThreads);
        } else if (steps > 0 && (warp & 3) < warps_of(qt)) {
            const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16) + qt * Sh::kSCols;
            const uint32_t obuf = lanes + Sh::kOCol;
            const int rr = (two ? qt * kTcRows : 0) + r;
            const bool valid = rr < rows;
            const int row = row0 + min(rr, rows - 1);
            const int token = over_group(row);
            const int pos = first_pos + token;                         // the last key that the row sees
            const float hm = p.q_mul * __uint_as_float((uint32_t)units[rr] << 23) * (kFp8 ? 256.f : 1.f);
            float m = -INFINITY, l = 0.f;
            float d = kSpNoWeight;                                     // weights are p b 2^(6 - d), p relative to m
            bool ok = true;
            for (int i = 0; i < steps; ++i) {
                const int j = tile_of(qt, i);
                const uint32_t sbuf = lanes + (kOne ? (i & 1) * N : 0);
                ok = tc_wait(&scale_bar[j % kSpRing], (uint32_t)((j / kSpRing) & 1), p.status, abort_flag) &&
                     tc_wait(&s_full[kOne ? i & 1 : qt], (uint32_t)((kOne ? i >> 1 : i) & 1), p.status, abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const float2* sp = scales + (j % kSpRing) * (N / kG);         // broadcast reads
                // the group's scale on the row's scores; zero must not meet a masked one
                auto on_row = [&](float a, bool past) {
                    const float k = a * hm;
                    return past | (k == 0.f) ? 1.17549435e-38f : k;
                };
                // keys of this tile that the row sees (at or below 0: none)
                const int sees = pos + 1 - (T0 + j * N);
                const bool cut = __any_sync(0xffffffffu, sees < N);
                auto mask = [&](uint32_t (&x)[32], int c0) {
                    if (__builtin_expect(cut, 0)) {
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            if (c0 + c >= sees) x[c] = 0xff800000u;    // -infinity
                    }
                };
                // ---- the maximum
                float m_cand = m, w_cand = -INFINITY;                  // of the logits, and of logit + log2 b
                uint32_t xa[32], xb[32];
                auto largest = [&](uint32_t (&x)[32], int h) {
                    mask(x, 32 * h);
#pragma unroll
                    for (int g = 0; g < 32 / kG; ++g) {
                        auto at = [&](int c) { return __uint_as_float(x[kG * g + c]); };
                        float y = fmax3(at(0), at(1), at(2)), z = fmax3(at(3), at(4), at(5));
                        y = fmax3(y, at(6), at(7));
                        if constexpr (kG == 16) {
                            z = fmax3(z, at(8), at(9));
                            y = fmax3(y, at(10), at(11));
                            z = fmax3(z, at(12), at(13));
                            y = fmax3(y, at(14), at(15));
                        }
                        const float2 ab = sp[32 / kG * h + g];
                        y = fmaxf(y, z) * on_row(ab.x, false);
                        m_cand = fmaxf(m_cand, y);
                        w_cand = fmaxf(w_cand, y + ab.y);
                    }
                };
                tc_ld32(sbuf, xa);
#pragma unroll 1
                for (int h = 0; h < N / 32; h += 2) {
                    tc_wait_ld32(xa);
                    tc_ld32(sbuf + 32 * h + 32, xb);
                    largest(xa, h);
                    tc_wait_ld32(xb);
                    if (h + 2 < N / 32) tc_ld32(sbuf + 32 * h + 64, xa);
                    largest(xb, h + 1);
                }
                const bool moved = m_cand > m + kSpMoveLog2;
                const float m_use = moved ? m_cand : m;
                const float m_sub = m_use == -INFINITY ? 0.f : m_use;
                const float fell = m == -INFINITY ? 0.f : m - m_use;
                // d falls by what m rises, and rises to the row's largest weight
                float d_use = fmaxf(d + fell, kSpNoWeight);
                const float w_most = w_cand - m_sub;
                const bool wider = w_most > d_use + kSpMoveLog2;
                if (wider) d_use = ceilf(w_most);
                l *= fast_exp2(fell);
                const float alpha = fast_exp2(fell + (d - d_use));
                d = d_use;
                m = m_use;
                if (i > 0 && __any_sync(0xffffffffu, moved || wider)) {
                    // O holds the tiles before this one: S of this tile came after their P.V, of
                    // one stream after all but the last
                    if constexpr (kOne) {
                        ok = __all_sync(0xffffffffu, tc_wait(&v_empty[(i - 1) % NSV], (uint32_t)((i - 1) / NSV & 1), p.status, abort_flag));
                        if (!ok) break;
                        tc_fence_after();
                    }
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t o[32];
                        tc_ld32(obuf + c, o);
                        tc_wait_ld32(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        tc_st32(obuf + c, o);
                    }
                }
                // ---- the weights, 32 keys at a time, their scores read again: a loop of few
                // instructions and registers, the next scores under way. Weights lie over their
                // scores: those of keys 32 h .. in columns 32 h .., their second terms in 32 h + 16 ..
                auto weigh = [&](uint32_t (&x)[32], int h) {
                    uint32_t w2[kTwoTerms ? 32 : 16];                  // first terms, second terms
                    mask(x, 32 * h);
#pragma unroll
                    for (int g = 0; g < 32 / kG; ++g) {
                        const float2 ab = sp[32 / kG * h + g];
                        // (of a group that the row does not see the scales may be no numbers)
                        const bool past = 32 * h + kG * g >= sees;
                        const float lift = (past | (ab.y < d - 60.f) ? -60.f : ab.y - d) + 6.f;
                        const float k1 = on_row(ab.x, past);
                        const float2 k2 = make_float2(k1, k1);
                        const float2 c2 = make_float2(lift - m_sub, lift - m_sub);
                        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                        for (int c = 0; c < kG; c += 2) {
                            const float2 t = __ffma2_rn(make_float2(__uint_as_float(x[kG * g + c]), __uint_as_float(x[kG * g + c + 1])), k2, c2);
                            const float2 e = make_float2(fast_exp2(t.x), fast_exp2(t.y));
                            sum[(c >> 1) & 1] = __fadd2_rn(sum[(c >> 1) & 1], e);
                            const uint32_t w = pack2<__half>(e.x, e.y);
                            w2[kG / 2 * g + c / 2] = w;
                            if constexpr (kTwoTerms) {
                                const float2 rest = __ffma2_rn(unpack2<__half>(w), make_float2(-1.f, -1.f), e);
                                w2[16 + kG / 2 * g + c / 2] = pack2<__half>(rest.x, rest.y);
                            }
                        }
                        sum[0] = __fadd2_rn(sum[0], sum[1]);
                        l = fmaf(sum[0].x + sum[0].y, fast_exp2(-lift), l);
                    }
                    tc_st_n<kTwoTerms ? 32 : 16>(sbuf + 32 * h, w2);
                };
                tc_ld32(sbuf, xa);
#pragma unroll 1
                for (int h = 0; h < N / 32; h += 2) {
                    tc_wait_ld32(xa);
                    tc_ld32(sbuf + 32 * h + 32, xb);
                    weigh(xa, h);
                    tc_wait_ld32(xb);
                    if (h + 2 < N / 32) tc_ld32(sbuf + 64, xa);
                    weigh(xb, h + 1);
                    tc_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    // (of one stream by turns: a warp may be a tile ahead of another)
                    if (lane == 0) mbar_arrive(&p_full[h + (kOne ? i & 1 : qt)]);
                }
            }
            if (ok) {
                ok = tc_wait(drain, 0u, p.status, abort_flag);
                ok = __all_sync(0xffffffffu, ok);
            }
            float fall = fast_exp2(d - (kFp8 ? -2.f : 6.f));
            // two streams of one query tile: the second hands its rows to the first, in the
            // queries' place (every MMA is done, and every slice widened)
            float* other = reinterpret_cast<float*>(sm);               // [128][D], columns turned by the row
            float* other_m = reinterpret_cast<float*>(sm + Sh::kKOff);
            float* other_l = other_m + kTcRows;
            if (join && qt == 1) {
                if (ok) {
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t o[32];
                        tc_ld32(obuf + c, o);
                        tc_wait_ld32(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) other[r * D + ((c + e + r) & (D - 1))] = __uint_as_float(o[e]) * fall;
                    }
                    other_m[r] = m;
                    other_l[r] = l;
                }
                named_barrier(3, kTcSoftmaxThreads);
                ok = false;
            }
            float from_other = 0.f;
            if (join && qt == 0) {
                named_barrier(3, kTcSoftmaxThreads);
                const float m1 = other_m[r], l1 = other_l[r];
                const float most = fmaxf(m, m1);
                const float f0 = m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : fast_exp2(m - most);
                from_other = m1 == -INFINITY ? (l1 == 0.f ? 0.f : 1.f) : fast_exp2(m1 - most);
                l = l * f0 + l1 * from_other;
                fall *= f0;
                m = most;
            }
            if (ok) {
                tc_fence_after();
                const bool sees = valid && pos >= T0;                  // anything of this partition
                const float inv = 1.f / l;
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
                    tc_wait_ld32(o);
                    float f[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        f[e] = __uint_as_float(o[e]) * fall;
                        if (join) f[e] = fmaf(other[r * D + ((c + e + r) & (D - 1))], from_other, f[e]);
                        f[e] *= inv;
                    }
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
    if (warp == kSpMmaWarp) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(Sh::kTmemCols) : "memory");
    }
}

template <typename CT, int D, int kG, bool kTwoTerms>
cudaError_t launch_scaled_prefill_terms(const ScaledAttnParams& p, cudaStream_t stream) {
    auto kernel = scaled_prefill_kernel<CT, D, kG, kTwoTerms>;
    cudaError_t e = ensure_smem_attribute(reinterpret_cast<const void*>(kernel), SpShape<D>::kAlloc);
    if (e != cudaSuccess) return e;
    return launch_overlapped(kernel, p, dim3(p.max_parts, p.num_kv_heads * p.row_tiles, p.num_seqs), kSpThreads, SpShape<D>::kAlloc, stream);
}

// The merge of a row's partitions: 16 or 32 threads hold four components each, and the others
// of a (query token, head)'s CTA take partitions in turn.
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

template <typename CT, int D, bool kTwoTerms>
cudaError_t launch_scaled_prefill_head(const ScaledAttnParams& p, cudaStream_t stream) {
    const cudaError_t e = D < 256 && p.block_size % 16 == 0 ? launch_scaled_prefill_terms<CT, D, D < 256 ? 16 : 8, kTwoTerms>(p, stream)
                                                 : launch_scaled_prefill_terms<CT, D, 8, kTwoTerms>(p, stream);
    if (e != cudaSuccess || p.max_parts == 1) return e;
    return launch_overlapped(scaled_merge_kernel<D>, p, dim3(p.num_q_heads, p.max_queries, p.num_seqs), kScaledMergeThreads, 0, stream);
}

// By the output's type, a file for each (scaled_prefill_*.cu).
template <typename CT, bool kTwoTerms>
cudaError_t launch_scaled_prefill(const ScaledAttnParams& p, int head_size, cudaStream_t stream) {
    switch (head_size) {
    case 64: return launch_scaled_prefill_head<CT, 64, kTwoTerms>(p, stream);
    case 128: return launch_scaled_prefill_head<CT, 128, kTwoTerms>(p, stream);
    case 256: return launch_scaled_prefill_head<CT, 256, kTwoTerms>(p, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace pagedkv
