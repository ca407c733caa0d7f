// sparse_decode.cuh -- the block-sparse decode in one kernel: a cluster of CTAs
// takes one (sequence, KV head), scores its blocks and selects (see
// sparse_select.cuh), and then attends to the selection:
//     out_h = sum_i softmax_i(scale q_h . k_i) v_i   over the selected tokens.
// While one row's first CTA selects, other rows' CTAs on the SM score or
// attend, so the memory system has work throughout; nothing goes through
// memory between the two parts, and few rows pay one launch.
//
// Attention: each warp of the cluster in turn takes a tile of 16 tokens (a block, or a part
// of one). Both products run on warp-level MMAs, straight from global memory
// to registers, as no element is used twice but by the group's heads:
//   S (16 tokens x 8 heads) = K (16 x D) . Q^T, a lane's 16-byte chunk of a key
//     row standing for k = 2 t4, 2 t4 + 1, 2 t4 + 8, 2 t4 + 9 of two steps;
//   O^T (D x 8 heads) += V^T (D x 16 tokens) . P^T: a lane loads the 16-byte
//     chunks of the four tokens it holds as k (2 t4, 2 t4 + 1, 2 t4 + 8,
//     2 t4 + 9) and pairs them component by component with byte permutes; the
//     components of a chunk are spread over the tiles' rows g and g + 8.
// The next tile's keys are loaded while this tile's softmax and P.V run, its
// values while the next scores run. The softmax reference moves only when a
// score passes it by 2^8 (weights up to 256 are as good as those up to 1), so
// most tiles need no maximum across lanes. Weights are sums of 16-bit terms, each
// with its own MMA: three of bfloat16, all 24 bits, or two of binary16, 22 bits
// (times 2^7, so that what binary16 cannot hold is below 2^-31 of the reference's
// weight). The sums use exactly the weights that the products use. Fewer terms
// would be a little faster on E4M3 caches (one: 120 us for 123 on the batch below)
// and no faster on 16-bit ones, which the loads bound. E4M3 codes convert to
// binary16, NaN codes to NaN: a NaN key or value shows in the output (the integer
// widening of the dense decode, which reads those as +-480, took 117 us for 120). A
// 16-bit query meets them scaled by a power of two to at most 2 in magnitude, exact
// but for components more than 2^14 below the head's largest. Partial results are
// joined in shared memory across the warps, and through the cluster's across CTAs.
//
// Measured in a graph (32/8 heads of 128, block size 16): 64 bf16 contexts of 8k to
// 32k tokens with 64 blocks selected 113 us, 5.4 TB/s of bounds, keys and values,
// where bare gathers of such chunks reach 5.2 (512 bytes) to 5.9 (4 KB) TB/s: bound
// by them. One context of 131072 with 128 selected 27 us: bound by the latencies
// of score, select, attend and the cluster's barriers in a row. E4M3 (64/8 heads,
// 128 contexts of 100 to 8k, 96 selected) 124 us, 4.4 TB/s: bound by latency at 16
// warps per SM (loads, the conversions' chain, the selection's barriers).
#pragma once

#include "sparse_select.cuh"

namespace pagedkv {

// A tile's keys of tokens g and g + 8 (this lane's chunks), and values of
// tokens 2 t4, 2 t4 + 1, 2 t4 + 8, 2 t4 + 9.
template <typename CT, int D>
struct Tile16 {                                     // 16-bit caches
    static constexpr int KJ = D / 32, VU = D / 64;
    uint4 x[KJ], y[KJ];
    uint4 v[4][VU];
};

template <int D>
struct Tile16<e4m3_t, D> {
    static constexpr int KJ = D / 64, VW = D / 32;  // D / 8 codes a lane and token
    uint4 x[KJ], y[KJ];
    uint32_t v[4][VW];
};

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

struct Joined {                                     // one CTA's result, read by the cluster
    float m[8], l[8];
};

template <typename QT, typename CT, int D, int NT>
__global__ void __launch_bounds__(NT, D == 256 ? 1 : 512 / NT)
sparse_decode_kernel(const __grid_constant__ SparseParams sp) {
    begin_overlapped();
    constexpr bool kFp8 = std::is_same<CT, e4m3_t>::value;
    using MT = typename MathType<CT>::T;            // the MMAs' type
    // weights: bfloat16 terms of 8 bits, or binary16 ones of 11, those times 2^7
    constexpr bool kThreeTerms = std::is_same<MT, __nv_bfloat16>::value;
    constexpr float kUp = kThreeTerms ? 0.f : 7.f;
    using Ops = MmaOps<MT>;
    using OutOps = MmaOps<QT>;
    using Tile = Tile16<CT, D>;
    constexpr int MD = D / 16;                      // O^T row tiles
    constexpr int NW = NT / 32;
    const SelectParams& p = sp.sel;
    extern __shared__ __align__(16) uint8_t dyn[];
    __shared__ SelShared<NT> sh;
    __shared__ Joined joined;
    __shared__ float wm[NW][8], wl[NW][8], wf[NW][8], q_unit[8];
    __shared__ float sh_m[8 * kMaxCluster], sh_l[8 * kMaxCluster];
    int32_t* list = reinterpret_cast<int32_t*>(dyn);                   // the row's slabs
    uint4* qf = reinterpret_cast<uint4*>(dyn + sp.list_bytes);         // query fragments: D * 16 bytes
    uint8_t* work = dyn + sp.list_bytes + 16 * D;                      // selection, then the warps' O
    cg::cluster_group cluster = cg::this_cluster();
    const int G = p.group, B = p.block_size;
    // this thread's eight query elements, before anything waits for the length
    constexpr int kChunks = D / 8;                  // chunks of a head
    const int q_head = threadIdx.x / kChunks, q_chunk = threadIdx.x % kChunks;
    uint4 q_words = make_uint4(0, 0, 0, 0);
    if (q_head < G) {                               // rows of a sequence's heads are contiguous
        const size_t row = blockIdx.x / cluster.num_blocks();
        q_words = *reinterpret_cast<const uint4*>(static_cast<const QT*>(p.query) + (row * G + q_head) * D + 8 * q_chunk);
    }
    const SelRow rw(p, cluster, work);
    const int C = rw.C;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t4 = lane & 3;
    QT* out = static_cast<QT*>(sp.out) + ((size_t)rw.s * p.num_q_heads + rw.h * G) * D;

    for (int i = threadIdx.x; i < p.table_width; i += NT) list[i] = -1;
    // The query in two forms, from one load: its sides for the scores, and the
    // fragments for S (head g's elements as the keys' chunks hold them). A
    // thread has eight elements, a head D / 8 neighbouring threads.
    if (threadIdx.x < D) {
        constexpr int N = kChunks;
        const int hd = q_head, c = q_chunk;
        const uint4 w = q_words;
        const int l = 4 * hd + (c & 3);                        // the lane, in step c / 4
        if (rw.scored) {
#pragma unroll
            for (int side = 0; side < 2; ++side)
                rw.sides[(side * (D / 32) + c / 4) * 32 + l] =
                    make_uint4(side2<QT>(w.x, side), side2<QT>(w.y, side), side2<QT>(w.z, side), side2<QT>(w.w, side));
        }
        if constexpr (!kFp8) {
            qf[(c / 4) * 32 + l] = w;
        } else {
            float x[8], mx = 0.f;
            widen16<QT>(w, x);
#pragma unroll
            for (int k = 0; k < 8; ++k) mx = fmaxf(mx, fabsf(x[k]));
#pragma unroll
            for (int m = N / 2; m > 0; m >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, m));
            // a power of two that brings the largest magnitude into [1, 2),
            // kept to the range whose reciprocal is a normal number
            const uint32_t ex = min(max(__float_as_uint(mx) >> 23, 1u), 252u);
            const float unit = mx > 0.f && mx < INFINITY ? __uint_as_float(ex << 23) : 1.f;
            if (c == 0) q_unit[hd] = unit;
            const float r = 1.f / unit;                        // exact
            // 64 elements a step, 16 a lane: this chunk is half c & 1 of lane
            // c / 2 & 3
            qf[((c / 8) * 32 + 4 * hd + (c / 2 & 3)) * 2 + (c & 1)] =
                make_uint4(Ops::pack(x[0] * r, x[1] * r), Ops::pack(x[2] * r, x[3] * r),
                           Ops::pack(x[4] * r, x[5] * r), Ops::pack(x[6] * r, x[7] * r));
        }
    }

    // ------------------------------------------------------------ selection
    if (!rw.scored) __syncthreads();                // else at the scoring's first barrier
    score_and_take<QT, D, true, NT>(p, sh, cluster, rw);
    int32_t* selected = p.selected ? p.selected + (size_t)rw.row * p.num_select : nullptr;
    const int total = rw.n < p.num_select ? rw.n : p.num_select;
    if (rw.rank == 0 || rw.all) {                   // with every block taken each CTA lists them itself
        for_taken(sh, rw, [&](int at, int b) { list[at] = b; });
        __syncthreads();
        for (int i = threadIdx.x; i < total; i += NT) {
            const int b = list[i];
            const int slab = b < 0 ? -1 : slab_of(p, rw, b);
            if (rw.rank == 0) {
                if (selected) selected[i] = b;
                if (slab < 0 && p.status) atomicOr(p.status, PA_DEV_BAD_BLOCK_ID);
            }
            list[i] = slab;
        }
        if (rw.rank == 0 && selected)
            for (int i = total + threadIdx.x; i < p.num_select; i += NT) selected[i] = -1;
    }
    // (the others read the first one's list in place)
    if (C > 1 && !rw.all) cluster.sync();
    else __syncthreads();
    const int32_t* slabs = C > 1 && !rw.all ? cluster.map_shared_rank(list, 0) : list;

    // ------------------------------------------------------------ attention
    const int len = total * B - (rw.n * B - rw.L);  // the selection's tokens
    const int tiles = (len + 15) / 16;
    const int per_block = B / 16;                   // B is a multiple of 16
    float acc[MD][4];
#pragma unroll
    for (int i = 0; i < MD; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
    float m_ref[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
    const float unit0 = kFp8 && 2 * t4 < G ? q_unit[2 * t4] : 1.f;
    const float unit1 = kFp8 && 2 * t4 + 1 < G ? q_unit[2 * t4 + 1] : 1.f;
    const float q_mul[2] = {sp.q_mul * unit0, sp.q_mul * unit1};

    Tile tl;
    constexpr int kRowBytes = D * (int)sizeof(CT);
    // byte offset of a tile's first token in the caches; -1: no such block
    auto tile_at = [&](int tile) -> int64_t {
        const int j = per_block == 1 ? tile : tile / per_block;
        const int slab = slabs[j];
        return slab < 0 ? -1 : ((int64_t)slab * B + (tile - j * per_block) * 16) * kRowBytes;
    };
    auto load_keys = [&](int64_t at) {
        const uint8_t* k = static_cast<const uint8_t*>(sp.k_cache) + (at < 0 ? 0 : at) + g * kRowBytes + 16 * t4;
#pragma unroll
        for (int j = 0; j < Tile::KJ; ++j) {
            tl.x[j] = *reinterpret_cast<const uint4*>(k + 64 * j);
            tl.y[j] = *reinterpret_cast<const uint4*>(k + 8 * kRowBytes + 64 * j);
        }
    };
    // rows from nvalid on are zeroed: their weights are 0, and 0 x NaN is not
    auto load_values = [&](int64_t at, int nvalid) {
        const uint8_t* v = static_cast<const uint8_t*>(sp.v_cache) + (at < 0 ? 0 : at);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int tok = 2 * t4 + (r & 1) + 8 * (r >> 1);
            const uint8_t* row = v + tok * kRowBytes;
            const bool there = tok < nvalid;
            if constexpr (kFp8) {
                const uint8_t* codes = row + g * (D / 8);
                if constexpr (D == 64) {
                    const uint2 w = there ? *reinterpret_cast<const uint2*>(codes) : make_uint2(0, 0);
                    tl.v[r][0] = w.x;
                    tl.v[r][1] = w.y;
                } else {
#pragma unroll
                    for (int u = 0; u < Tile::VW; u += 4) {
                        uint4 w = make_uint4(0, 0, 0, 0);
                        if (there) w = *reinterpret_cast<const uint4*>(codes + 4 * u);
                        tl.v[r][u] = w.x;
                        tl.v[r][u + 1] = w.y;
                        tl.v[r][u + 2] = w.z;
                        tl.v[r][u + 3] = w.w;
                    }
                }
            } else {
#pragma unroll
                for (int u = 0; u < Tile::VU; ++u) {
                    uint4 w = make_uint4(0, 0, 0, 0);
                    if (there) w = *reinterpret_cast<const uint4*>(row + 128 * u + 16 * g);
                    tl.v[r][u] = w;
                }
            }
        }
    };
    const int stride = C * NW;
    int tile = rw.rank * NW + warp;
    int64_t at = -1;
    int nvalid = 0;
    auto valid_of = [&](int64_t a, int tile) { return a < 0 ? 0 : min(16, len - tile * 16); };
    if (tile < tiles) {
        at = tile_at(tile);
        nvalid = valid_of(at, tile);
        load_keys(at);
        load_values(at, nvalid);
    }
    while (tile < tiles) {
        // ---- scores: tokens g, g + 8 x heads 2 t4, 2 t4 + 1
        float sc[4] = {0.f, 0.f, 0.f, 0.f};
        if constexpr (kFp8) {
#pragma unroll
            for (int j = 0; j < Tile::KJ; ++j)
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    const uint4 q = qf[(j * 32 + lane) * 2 + part];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t wx = word_of(tl.x[j], 2 * part + k), wy = word_of(tl.y[j], 2 * part + k);
                        const uint32_t a[4] = {e4m3x2_to_f16x2(wx), e4m3x2_to_f16x2(wy), e4m3x2_to_f16x2(wx >> 16),
                                               e4m3x2_to_f16x2(wy >> 16)};
                        Ops::mma(sc, a, k ? q.z : q.x, k ? q.w : q.y);
                    }
                }
        } else {
#pragma unroll
            for (int j = 0; j < Tile::KJ; ++j) {
                const uint4 q = qf[j * 32 + lane];
                const uint32_t a0[4] = {tl.x[j].x, tl.y[j].x, tl.x[j].y, tl.y[j].y};
                const uint32_t a1[4] = {tl.x[j].z, tl.y[j].z, tl.x[j].w, tl.y[j].w};
                Ops::mma(sc, a0, q.x, q.y);
                Ops::mma(sc, a1, q.z, q.w);
            }
        }
        const int next = tile + stride;
        const int64_t next_at = next < tiles ? tile_at(next) : -1;
        if (next < tiles) load_keys(next_at);

        // ---- softmax weights
        bool over = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float v = sc[i] * q_mul[i & 1];
            sc[i] = g + 8 * (i >> 1) < nvalid ? v : -INFINITY;         // select, never multiply
            over |= sc[i] > m_ref[i & 1] + 8.f;
        }
        if (__any_sync(0xffffffffu, over)) {
            float alpha[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float mx = fmaxf(sc[j], sc[j + 2]);
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                const float m_new = fmaxf(m_ref[j], mx);
                alpha[j] = m_new == -INFINITY ? 1.f : (m_ref[j] == -INFINITY ? 0.f : fast_exp2(m_ref[j] - m_new));
                m_ref[j] = m_new;
                l_run[j] *= alpha[j];
            }
#pragma unroll
            for (int i = 0; i < MD; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] *= alpha[j & 1];
        }
        const float ref[2] = {m_ref[0] - kUp, m_ref[1] - kUp};
        uint32_t hi[2], lo[2], low[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float w0 = sc[2 * r] == -INFINITY ? 0.f : fast_exp2(sc[2 * r] - ref[0]);
            const float w1 = sc[2 * r + 1] == -INFINITY ? 0.f : fast_exp2(sc[2 * r + 1] - ref[1]);
            const uint32_t h = Ops::pack(w0, w1);
            const float2 hf = Ops::unpack(h);
            const uint32_t l = Ops::pack(w0 - hf.x, w1 - hf.y);
            const float2 lf = Ops::unpack(l);
            if constexpr (kThreeTerms) low[r] = movmatrix_trans(Ops::pack(w0 - hf.x - lf.x, w1 - hf.y - lf.y));
            l_run[0] += kThreeTerms ? w0 : hf.x + lf.x;
            l_run[1] += kThreeTerms ? w1 : hf.y + lf.y;
            hi[r] = movmatrix_trans(h);
            lo[r] = movmatrix_trans(l);
        }

        // ---- O^T += V^T P^T
        if constexpr (kFp8) {
#pragma unroll
            for (int i = 0; i < MD; ++i) {
                // codes 2 i and 2 i + 1 of each token's chunk: rows g and g + 8
                const uint32_t sel = i & 1 ? 0x7362 : 0x5140;
                const uint32_t v01 = __byte_perm(tl.v[0][i / 2], tl.v[1][i / 2], sel);
                const uint32_t v23 = __byte_perm(tl.v[2][i / 2], tl.v[3][i / 2], sel);
                const uint32_t a[4] = {e4m3x2_to_f16x2(v01), e4m3x2_to_f16x2(v01 >> 16), e4m3x2_to_f16x2(v23),
                                       e4m3x2_to_f16x2(v23 >> 16)};
                Ops::mma(acc[i], a, hi[0], hi[1]);
                Ops::mma(acc[i], a, lo[0], lo[1]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < MD; ++i) {
                const int u = i / 4, w = i % 4;
                const uint32_t v0 = word_of(tl.v[0][u], w), v1 = word_of(tl.v[1][u], w);
                const uint32_t v2 = word_of(tl.v[2][u], w), v3 = word_of(tl.v[3][u], w);
                const uint32_t a[4] = {__byte_perm(v0, v1, 0x5410), __byte_perm(v0, v1, 0x7632),
                                       __byte_perm(v2, v3, 0x5410), __byte_perm(v2, v3, 0x7632)};
                Ops::mma(acc[i], a, hi[0], hi[1]);
                Ops::mma(acc[i], a, lo[0], lo[1]);
                if constexpr (kThreeTerms) Ops::mma(acc[i], a, low[0], low[1]);
            }
        }
        tile = next;
        if (tile < tiles) {
            at = next_at;
            nvalid = valid_of(at, tile);
            load_values(at, nvalid);
        }
    }

    // ------------------------------------------------------------ join the warps
    // O of a warp: [head][D + 4] (the padding spreads the heads over the banks)
    constexpr int kPitch = D + 4;
    float* wo = reinterpret_cast<float*>(work);
    __syncthreads();                                // the selection's use of this memory is over
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int m = 4; m < 32; m <<= 1) l_run[j] += __shfl_xor_sync(0xffffffffu, l_run[j], m);
        const int hd = 2 * t4 + j;
        if (g == 0) {
            wm[warp][hd] = m_ref[j];
            wl[warp][hd] = l_run[j];
        }
        float* o = wo + (warp * 8 + hd) * kPitch;
#pragma unroll
        for (int i = 0; i < MD; ++i) {
            const int d = kFp8 ? (D / 8) * g + 2 * i : 64 * (i / 4) + 8 * g + 2 * (i % 4);
            *reinterpret_cast<float2*>(o + d) = make_float2(acc[i][j], acc[i][2 + j]);
        }
    }
    __syncthreads();
    // each warp's factor relative to the CTA's maximum (a single CTA: over the sum)
    if (threadIdx.x < NW * 8) {
        const int w = threadIdx.x >> 3, hd = threadIdx.x & 7;
        float M = -INFINITY, l = 0.f;
#pragma unroll
        for (int v = 0; v < NW; ++v) M = fmaxf(M, wm[v][hd]);
#pragma unroll
        for (int v = 0; v < NW; ++v) l += wm[v][hd] == -INFINITY ? 0.f : fast_exp2(wm[v][hd] - M) * wl[v][hd];
        float f = wm[w][hd] == -INFINITY ? 0.f : fast_exp2(wm[w][hd] - M);
        if (C == 1) f *= l > 0.f || l != l ? sp.v_mul / l : 0.f;       // no tokens: zero; NaN stays
        wf[w][hd] = f;
        if (w == 0) {
            joined.m[hd] = M;
            joined.l[hd] = l;
        }
    }
    __syncthreads();
    // four elements of a head a thread
    for (int e = threadIdx.x; e < G * (D / 4); e += NT) {
        const int hd = e / (D / 4), d = 4 * (e - hd * (D / 4));
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float f = wf[w][hd];
            const float4 x = *reinterpret_cast<const float4*>(wo + (w * 8 + hd) * kPitch + d);
            o.x += f * x.x;
            o.y += f * x.y;
            o.z += f * x.z;
            o.w += f * x.w;
        }
        if (C == 1) {
            *reinterpret_cast<uint2*>(out + hd * D + d) = make_uint2(OutOps::pack(o.x, o.y), OutOps::pack(o.z, o.w));
        } else {
            // into warp 0's place, which only this thread reads for these elements
            *reinterpret_cast<float4*>(wo + hd * kPitch + d) = o;
        }
    }
    if (C == 1) return;
    cluster.sync();
    // ------------------------------------------------------------ join the CTAs
    // each CTA's factor relative to the row's maximum, over the sum
    if (threadIdx.x < 8 * C) {
        const Joined* jr = cluster.map_shared_rank(&joined, threadIdx.x >> 3);
        sh_m[threadIdx.x] = jr->m[threadIdx.x & 7];
        sh_l[threadIdx.x] = jr->l[threadIdx.x & 7];
    }
    __syncthreads();
    float f = 0.f;
    if (threadIdx.x < 8 * C) {
        const int hd = threadIdx.x & 7;
        float M = -INFINITY, l = 0.f;
        for (int r = 0; r < C; ++r) M = fmaxf(M, sh_m[8 * r + hd]);
        for (int r = 0; r < C; ++r)
            l += sh_m[8 * r + hd] == -INFINITY ? 0.f : fast_exp2(sh_m[8 * r + hd] - M) * sh_l[8 * r + hd];
        f = sh_m[threadIdx.x] == -INFINITY ? 0.f : fast_exp2(sh_m[threadIdx.x] - M);
        f *= l > 0.f || l != l ? sp.v_mul / l : 0.f;
    }
    __syncthreads();
    if (threadIdx.x < 8 * C) sh_m[threadIdx.x] = f;
    __syncthreads();
    for (int e = rw.rank + C * threadIdx.x; e < G * (D / 4); e += C * NT) {
        const int hd = e / (D / 4), d = 4 * (e - hd * (D / 4));
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int r = 0; r < C; ++r) {
            const float4 x = *reinterpret_cast<const float4*>(cluster.map_shared_rank(wo + hd * kPitch + d, r));
            const float w = sh_m[8 * r + hd];
            o.x += w * x.x;
            o.y += w * x.y;
            o.z += w * x.z;
            o.w += w * x.w;
        }
        *reinterpret_cast<uint2*>(out + hd * D + d) = make_uint2(OutOps::pack(o.x, o.y), OutOps::pack(o.z, o.w));
    }
    cluster.sync();                                 // no CTA leaves while its memory is read
}

// CTAs per row: as many as find room, for contexts long enough to score together
// or where a single CTA's warps would each attend to more than three tiles of 16
// tokens; what a cluster costs is about 3 us. Up to 152 CTAs have an SM each; 256
// of clusters of 8 share them in pairs. Measured with 1, 2, 4 and 8 CTAs (bf16,
// head size 128, block size 16): 8 rows of 8192 blocks 69, 44, 31, 25 us (the
// selection alone); 8 rows of 170 blocks with 117 selected 26, 22, 19, 17, with
// 64 selected 19, 18, 17, 17, with 32 selected 15, 17, 17, 17; 32 rows of 500
// blocks with 64 selected 22, 21, 19, 17; 64 rows of it 25, 23, 22, 34; 104 rows
// 26, 28, 40, 50.
template <int D>
int decode_cluster(int rows, int max_ctx_blocks, int num_select, int block_size) {
    constexpr int kWarps = D < 256 ? 16 : 8;
    const int64_t tiles = (int64_t)(num_select < max_ctx_blocks ? num_select : max_ctx_blocks) * (block_size / 16);
    if (max_ctx_blocks < 512 && tiles <= 3 * kWarps) return 1;
    constexpr int kMost[] = {76, 38, D < 256 ? 32 : 14};       // rows for 2, 4 and 8
    int C = 1;
    for (int most : kMost) {
        if (rows > most) break;
        C *= 2;
    }
    return C;
}

template <typename QT, typename CT, int D>
cudaError_t launch_sparse(SparseParams sp, cudaStream_t stream) {
    const int rows = sp.sel.num_seqs * sp.sel.num_kv_heads;
    const int C = decode_cluster<D>(rows, sp.sel.max_ctx_blocks, sp.sel.num_select, sp.sel.block_size);
    // An SM for every CTA: 16 warps each, else two CTAs of 8 an SM (head size
    // 256: a tile's fragments take the registers of one CTA of 8 warps). Not
    // every GPC has 16 SMs for two clusters of 8 that fill theirs: of 16 clusters
    // one waits for a second wave (2 contexts of 131072: 49 us, 33 us with 8
    // warps; head size 256 in clusters of 8 and 4: 53 and 41 us).
    const bool placed = rows * C <= (C == kMaxCluster ? 112 : 152);
    const bool wide = D < 256 && placed;
    const int select = select_smem<QT, D>(sp.sel);
    const int join = (wide ? 16 : 8) * 8 * (D + 4) * (int)sizeof(float);
    sp.list_bytes = (sp.sel.table_width * 4 + 15) / 16 * 16;
    const int smem = sp.list_bytes + 16 * D + (select > join ? select : join);
    if constexpr (D < 256) {
        if (wide) return launch_cluster(sparse_decode_kernel<QT, CT, D, 512>, sp, rows * C, C, 512, smem, stream);
    }
    return launch_cluster(sparse_decode_kernel<QT, CT, D, 256>, sp, rows * C, C, 256, smem, stream);
}

template <typename QT, typename CT>
cudaError_t launch_sparse_types(const SparseParams& sp, int head_size, cudaStream_t stream) {
    switch (head_size) {
    case 64: return launch_sparse<QT, CT, 64>(sp, stream);
    case 128: return launch_sparse<QT, CT, 128>(sp, stream);
    default: return launch_sparse<QT, CT, 256>(sp, stream);
    }
}

}  // namespace pagedkv
