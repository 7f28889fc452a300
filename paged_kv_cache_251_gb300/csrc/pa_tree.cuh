// Tree attention over the paged cache: what its kernels share, the kernel for
// fp32 caches, and the merge of its partitions.
//
// Sequence s has L = context_lens[s] cached tokens, the last T_s of them
// drafted.  Row r = i * G + g of a (sequence, kv head) is query head g of
// drafted token i (G query heads share the kv head), so all T * G rows read
// the same K/V rows: cached token t is attended by row r when
//   t < L - T_s   (committed), or bit t - (L - T_s) of mask[s][i] is set.
// Work unit: (sequence, kv head, row tile, context partition); partitions are
// merged by log-sum-exp as in the other decodes.  A partition's partial is
// column-major over the rows of its (sequence, kv head): accumulators
// [D][T * G], then (running max, denominator) pairs [T * G] in their own array.
#pragma once

#include "pa_decode.cuh"

namespace pa {

struct TreeParams : DecodeParams {
    const int32_t *draft_lens;  // [num_seqs] or nullptr (num_draft everywhere)
    const uint64_t *mask;       // [num_seqs][num_draft][words] or nullptr (chain)
    int num_draft, words;
    int row_tiles;  // tiles of rows a (sequence, kv head)
    int4 *cuts;     // tensor-core kernel: two records a CTA for the merge, or nullptr
};

// Cached tokens and drafted tokens of sequence s, clamped.
struct TreeSeq {
    int len, drafted;
    bool bad;  // a value had to be clamped
};
__device__ inline TreeSeq tree_seq(const TreeParams &p, int s) {
    TreeSeq q;
    const int len = ld_nc_i32(p.context_lens + s);
    q.len = max(0, min(len, p.max_len));
    const int want = p.draft_lens ? ld_nc_i32(p.draft_lens + s) : p.num_draft;
    q.drafted = max(0, min(want, min(p.num_draft, q.len)));
    q.bad = len > p.max_len || want != q.drafted;
    return q;
}

// The 64 cached tokens [tok, tok + 64) that a row attends, blocks aside:
// committed tokens, then the row's drafted ones.  The mask words come in one
// round trip (two 64-bit words cover 64 bits at any offset).
__device__ inline uint64_t first_bits(int n) { return n <= 0 ? 0ull : (n >= 64 ? ~0ull : (1ull << n) - 1ull); }

__device__ inline uint64_t tree_bits64(const TreeParams &p, int s, int committed, int drafted, int i, int tok) {
    const int j = tok - committed;  // drafted index of the first token (negative: committed tokens first)
    const int up = max(-j, 0), j0 = max(j, 0);
    uint64_t d = 0;  // bit e: drafted token j0 + e
    if (j > -64 && j < drafted) {
        if (p.mask) {
            const uint64_t *row = p.mask + (static_cast<long long>(s) * p.num_draft + i) * p.words + (j0 >> 6);
            const int sh = j0 & 63;
            const uint64_t lo = row[0], hi = (j0 >> 6) + 1 < p.words ? row[1] : 0ull;
            d = sh ? (lo >> sh) | (hi << (64 - sh)) : lo;
        } else {  // a chain
            d = first_bits(i + 1 - j0);
        }
        d &= first_bits(drafted - j0);
    }
    return up >= 64 ? ~0ull : first_bits(up) | (d << up);
}

// ---------------------------------------------------------------------------
// fp32 caches: on the CUDA cores.  A CTA of 128 threads takes 16 R rows, 8 lanes a
// row and R rows a thread, and 64 tokens at a time in shared memory (one round trip
// a tile).  Scores: lane l of a row has tokens l, l + 8, ... with whole dot products,
// no exchange; one maximum and one rescale a tile; then the weights go through shared
// memory and lane l sums its D / 8 elements of the output over the attended tokens
// (others are never multiplied).
// Shared memory's rate bounds it at many rows: with R = 2 each K or V element read
// there serves two.  R = 2 above 16 rows (12 drafted, 32 / 8 heads of 128, 64 contexts
// spread evenly from 32 to 2048 tokens: 750 us, 992 with R = 1); up to 16 half of its
// rows would be empty.  4 rows of 64 elements, 8 kv heads, two contexts of 8000 and
// 16000 tokens: 71 us, 1.4 TB/s; a 5-token tree over a hundred tokens: 11 us.

constexpr int kTreeThreads = 128;
constexpr int kTreeRows = kTreeThreads / 8;  // rows of a CTA, times R
constexpr int kTreeTile = 64;
constexpr int kTreePartition = 256;  // tokens of a context partition

template <int D, int R> struct TreeSmem {
    float k[kTreeTile][D + 4];  // (+ 4: rows of a lane's tokens on different banks)
    float v[kTreeTile][D];
    float q[R * kTreeRows][D + 4];
    float w[R * kTreeRows][kTreeTile + 4];
    int phys[kTreePartition / 8];  // blocks of the partition, -1: left out
};

template <int D, int R>
__global__ void __launch_bounds__(kTreeThreads) pa_tree_kernel(const TreeParams p) {
    pdl_launch_dependents();
    pdl_wait();
    constexpr int E = D / 8;
    constexpr int V = 4;  // elements per 16-byte load
    constexpr int kPer = kTreeTile / 8;  // tokens of a lane
    extern __shared__ __align__(16) char smem[];
    TreeSmem<D, R> *sh = reinterpret_cast<TreeSmem<D, R> *>(smem);
    const int G = p.num_heads / p.num_kv_heads;
    const int rows = p.num_draft * G;
    const int rl = threadIdx.x >> 3, l8 = threadIdx.x & 7;
    const int bs = p.block_size, tile_blocks = kTreeTile / bs;
    const long long total = static_cast<long long>(p.num_seqs) * p.max_parts * p.num_kv_heads * p.row_tiles;
    for (long long w = blockIdx.x; w < total; w += gridDim.x) {
        long long f = w;
        const int rt = static_cast<int>(f % p.row_tiles);
        f /= p.row_tiles;
        const int kvh = static_cast<int>(f % p.num_kv_heads);
        f /= p.num_kv_heads;
        const int part = static_cast<int>(f % p.max_parts);
        const int s = static_cast<int>(f / p.max_parts);
        const TreeSeq q = tree_seq(p, s);
        const SeqSpan sp = seq_span(q.len, p.max_len, 0, bs, p.bpp);
        if (part >= sp.nparts)
            continue;
        if (q.bad && part == 0 && kvh == 0 && rt == 0 && threadIdx.x == 0 && p.err)
            atomicOr(p.err, PA_DEVERR_BAD_LEN);
        const int committed = q.len - q.drafted;
        // the thread's rows: rl + 16 y of the row tile
        const int r0 = rt * kTreeRows * R + rl;
        bool mine[R], live[R];
        int i[R];
        long long orow[R];
        float acc[R][E], m[R], l[R];
        __syncthreads();  // (the item before is done with shared memory)
#pragma unroll
        for (int y = 0; y < R; ++y) {
            const int r = r0 + kTreeRows * y;
            mine[y] = r < rows;
            i[y] = mine[y] ? r / G : 0;
            live[y] = mine[y] && i[y] < q.drafted;
            orow[y] = (static_cast<long long>(s) * p.num_draft + i[y]) * p.num_heads + kvh * G + (mine[y] ? r % G : 0);
            m[y] = -INFINITY, l[y] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int c = l8 + 8 * e;
                sh->q[rl + kTreeRows * y][c] =
                    live[y] ? static_cast<const float *>(p.q)[orow[y] * D + c] * p.scale_log2 : 0.f;
                acc[y][e] = 0.f;
            }
        }
        const int b_lo = part * p.bpp, b_hi = min(b_lo + p.bpp, sp.nblk);
        if (static_cast<int>(threadIdx.x) < b_hi - b_lo) {  // (at most 32 blocks a partition)
            int phys =
                ld_nc_i32(p.block_tables + static_cast<long long>(s) * p.max_blocks_per_seq + b_lo + threadIdx.x);
            if (phys < 0 || phys >= p.num_blocks) {
                phys = -1;
                if (p.err)
                    atomicOr(p.err, PA_DEVERR_BAD_BLOCK);
            }
            sh->phys[threadIdx.x] = phys;
        }
        for (int b = b_lo; b < b_hi; b += tile_blocks) {
            __syncthreads();
            // 16-byte pieces of the tile's rows, the loads of eight of a thread (K and V)
            // in flight: one after another they took 6000 cycles a tile
            constexpr int kAhead = 8;
            for (int c0 = threadIdx.x; c0 < kTreeTile * D / V; c0 += kAhead * kTreeThreads) {
                float4 kx[kAhead], vx[kAhead];
                bool on[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int c = c0 + u * kTreeThreads, t = c / (D / V), e = (c - t * (D / V)) * V;
                    const int blk = b + t / bs;
                    const int phys = t < kTreeTile && blk < b_hi ? sh->phys[blk - b_lo] : -1;
                    on[u] = phys >= 0;
                    if (on[u]) {
                        const long long at =
                            ((static_cast<long long>(phys) * p.num_kv_heads + kvh) * bs + t % bs) * D + e;
                        kx[u] = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.k_cache) + at);
                        vx[u] = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.v_cache) + at);
                    }
                }
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int c = c0 + u * kTreeThreads, t = c / (D / V), e = (c - t * (D / V)) * V;
                    if (on[u]) {
                        *reinterpret_cast<float4 *>(&sh->k[t][e]) = kx[u];
                        *reinterpret_cast<float4 *>(&sh->v[t][e]) = vx[u];
                    }
                }
            }
            __syncthreads();
            const int tok0 = b * bs;
            uint64_t allow[R];
#pragma unroll
            for (int y = 0; y < R; ++y)
                allow[y] = live[y] ? tree_bits64(p, s, committed, q.drafted, i[y], tok0) : 0ull;
            uint64_t blocks = ~0ull;
            for (int k = 0; k < tile_blocks; ++k)
                if (b + k >= b_hi || sh->phys[b - b_lo + k] < 0)
                    blocks &= ~(first_bits(bs) << (k * bs));
            float x[R][kPer] = {};
#pragma unroll 4
            for (int e = 0; e < D; e += 4) {
                float4 a[R];
#pragma unroll
                for (int y = 0; y < R; ++y)
                    a[y] = *reinterpret_cast<const float4 *>(&sh->q[rl + kTreeRows * y][e]);
#pragma unroll
                for (int k = 0; k < kPer; ++k) {
                    const float4 c = *reinterpret_cast<const float4 *>(&sh->k[l8 + 8 * k][e]);
#pragma unroll
                    for (int y = 0; y < R; ++y)
                        x[y][k] = fmaf(a[y].x, c.x,
                                       fmaf(a[y].y, c.y, fmaf(a[y].z, c.z, fmaf(a[y].w, c.w, x[y][k]))));
                }
            }
#pragma unroll
            for (int y = 0; y < R; ++y) {
                allow[y] &= blocks;
                float mt = -INFINITY;
#pragma unroll
                for (int k = 0; k < kPer; ++k) {
                    x[y][k] = (allow[y] >> (l8 + 8 * k)) & 1u ? x[y][k] : -INFINITY;
                    mt = fmaxf(mt, x[y][k]);
                }
#pragma unroll
                for (int o = 1; o < 8; o <<= 1)
                    mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
                const float mn = fmaxf(m[y], mt);
                const float alpha = mn == -INFINITY ? 1.f : exp2f(m[y] - mn);
                l[y] *= alpha;
#pragma unroll
                for (int e = 0; e < E; ++e)
                    acc[y][e] *= alpha;
                m[y] = mn;
#pragma unroll
                for (int k = 0; k < kPer; ++k) {
                    // (a NaN score stays one)
                    const float pw = x[y][k] == -INFINITY ? 0.f : exp2f(x[y][k] - mn);
                    l[y] += pw;
                    sh->w[rl + kTreeRows * y][l8 + 8 * k] = pw;
                }
            }
            __syncwarp();
            // attended tokens in order, kAtOnce at a time that some row of the warp attends; lane l8
            // sums elements 32 c + 4 l8 .. + 3 of the output (a walk over a row's own bits took
            // 140 cycles a token, this 20)
            constexpr int kAtOnce = R == 1 ? 8 : 4;
#pragma unroll 1
            for (int t0 = 0; t0 < kTreeTile; t0 += kAtOnce) {
                uint32_t bits[R], any = 0;
                float pw[R][kAtOnce];
#pragma unroll
                for (int y = 0; y < R; ++y) {
                    bits[y] = static_cast<uint32_t>(allow[y] >> t0) & ((1u << kAtOnce) - 1u);
                    any |= bits[y];
                }
                if (!__any_sync(0xffffffffu, any))
                    continue;
#pragma unroll
                for (int y = 0; y < R; ++y)
#pragma unroll
                    for (int u = 0; u < kAtOnce; u += 4)
                        *reinterpret_cast<float4 *>(&pw[y][u]) =
                            *reinterpret_cast<const float4 *>(&sh->w[rl + kTreeRows * y][t0 + u]);
#pragma unroll
                for (int u = 0; u < kAtOnce; ++u) {
#pragma unroll
                    for (int e = 0; e < E; e += 4) {
                        const float4 c = *reinterpret_cast<const float4 *>(&sh->v[t0 + u][8 * e + 4 * l8]);
#pragma unroll
                        for (int y = 0; y < R; ++y) {
                            if ((bits[y] >> u) & 1u) {
                                acc[y][e] = fmaf(pw[y][u], c.x, acc[y][e]);
                                acc[y][e + 1] = fmaf(pw[y][u], c.y, acc[y][e + 1]);
                                acc[y][e + 2] = fmaf(pw[y][u], c.z, acc[y][e + 2]);
                                acc[y][e + 3] = fmaf(pw[y][u], c.w, acc[y][e + 3]);
                            }
                        }
                    }
                }
            }
            __syncwarp();
        }
#pragma unroll
        for (int y = 0; y < R; ++y) {
#pragma unroll
            for (int o = 1; o < 8; o <<= 1)
                l[y] += __shfl_xor_sync(0xffffffffu, l[y], o);
            if (!mine[y])
                continue;
            if (sp.nparts == 1) {
                // (a NaN denominator is the row's own: it stays)
#pragma unroll
                for (int e = 0; e < E; ++e)
                    store_out(p.out, p.out_dtype, orow[y] * D + 8 * (e & ~3) + 4 * l8 + (e & 3),
                              l[y] == 0.f ? 0.f : acc[y][e] / l[y]);
            } else {
                const int r = r0 + kTreeRows * y;
                const long long item = (static_cast<long long>(s) * p.num_kv_heads + kvh) * p.max_parts + part;
#pragma unroll
                for (int e = 0; e < E; ++e)
                    p.part_acc[(item * D + 8 * (e & ~3) + 4 * l8 + (e & 3)) * rows + r] = acc[y][e];
                if (l8 == 0)
                    reinterpret_cast<float2 *>(p.part_ml)[item * rows + r] = make_float2(m[y], l[y]);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Merge of the partitions of every row of a multi-partition sequence.  A CTA
// takes RB rows of a (sequence, kv head) and 16 * 32 / RB columns (RB: 32, or
// the next power of two of fewer rows): lane = (row, column), so partials are
// read as whole lines.  Its 8 warps take every eighth partition each (one round
// trip of 17 loads a partition, few in sequence however long the context), and
// their states meet in shared memory.  A partition in which a row attends
// nothing (l == 0) left no accumulator.  `steps` column chunks a CTA: all of them
// when there are rows enough for every SM (a CTA of a single-partition sequence
// only reads its length and leaves, and 8192 such cost 20 us), one when few.
constexpr int kTreeMergeThreads = 256;
constexpr int kTreeMergeWarps = kTreeMergeThreads / 32;
constexpr int kTreeMergeCols = 16;  // columns of a lane

// log2 of RB for `rows` rows: at most 32, and at least what leaves the CTA's columns within D
__host__ __device__ inline int tree_merge_log_rows(int rows, int D) {
    int l = D == 64 ? 3 : 2;
    while (l < 5 && (1 << l) < rows)
        ++l;
    return l;
}

template <int D>
__global__ void __launch_bounds__(kTreeMergeThreads, 3) pa_tree_merge_kernel(const TreeParams p, int steps) {
    pdl_launch_dependents();
    pdl_wait();
    constexpr int E = kTreeMergeCols;
    __shared__ float acc[kTreeMergeWarps][E][33];  // [warp][element][lane]
    __shared__ float2 state[kTreeMergeWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int G = p.num_heads / p.num_kv_heads;
    const int rows = p.num_draft * G;
    const int lrb = tree_merge_log_rows(rows, D);
    const int RB = 1 << lrb, CB = 32 >> lrb;  // rows, and columns a step
    const int chunks = (rows + RB - 1) >> lrb;
    const int col_groups = D / (E * CB * steps);
    long long f = blockIdx.x;
    const int group0 = static_cast<int>(f % col_groups) * (E * CB * steps);
    f /= col_groups;
    const int r0 = static_cast<int>(f % chunks) << lrb;
    const long long seq_head = f / chunks;
    const int s = static_cast<int>(seq_head / p.num_kv_heads);
    const int kvh = static_cast<int>(seq_head - static_cast<long long>(s) * p.num_kv_heads);
    const int r = r0 + (lane & (RB - 1));
    const SeqSpan sp = seq_span(ld_nc_i32(p.context_lens + s), p.max_len, 0, p.block_size, p.bpp);
    if (sp.nparts <= 1)
        return;
    for (int step = 0; step < steps; ++step) {
        const int col0 = group0 + step * (E * CB);
        float M = -INFINITY, den = 0.f, num[E];
#pragma unroll
        for (int e = 0; e < E; ++e)
            num[e] = 0.f;
        if (r < rows) {
            const float2 *ml = reinterpret_cast<const float2 *>(p.part_ml) + seq_head * p.max_parts * rows + r;
            const float *a = p.part_acc + (seq_head * p.max_parts * D + col0 + (lane >> lrb)) * rows + r;
            for (int q = warp; q < sp.nparts; q += kTreeMergeWarps) {
                const float2 v = ml[static_cast<long long>(q) * rows];
                const float *aq = a + static_cast<long long>(q) * D * rows;
                float x[E];
#pragma unroll
                for (int e = 0; e < E; ++e)
                    x[e] = aq[static_cast<long long>(e * CB) * rows];
                if (v.y == 0.f)
                    continue;
                const float mn = fmaxf(M, v.x);
                const float keep = M == -INFINITY ? 0.f : exp2f(M - mn), add = exp2f(v.x - mn);
                den = den * keep + v.y * add;
#pragma unroll
                for (int e = 0; e < E; ++e)
                    num[e] = num[e] * keep + x[e] * add;
                M = mn;
            }
        }
        state[warp][lane] = make_float2(M, den);
#pragma unroll
        for (int e = 0; e < E; ++e)
            acc[warp][e][lane] = num[e];
        __syncthreads();
        // output o of the CTA: row o / (E CB), column o % (E CB)
        for (int o = threadIdx.x; o < 32 * E; o += kTreeMergeThreads) {
            const int rr = o / (E * CB), c = o - rr * (E * CB);
            if (r0 + rr >= rows)
                break;
            const int e = c / CB, ln = ((c - e * CB) << lrb) + rr;
            float m = -INFINITY;
#pragma unroll
            for (int w = 0; w < kTreeMergeWarps; ++w)
                if (state[w][ln].y != 0.f)
                    m = fmaxf(m, state[w][ln].x);
            float n = 0.f, d = 0.f;
#pragma unroll
            for (int w = 0; w < kTreeMergeWarps; ++w) {
                const float2 v = state[w][ln];
                if (v.y != 0.f) {
                    const float sc = v.x == m ? 1.f : exp2f(v.x - m);
                    d = fmaf(v.y, sc, d);
                    n = fmaf(acc[w][e][ln], sc, n);
                }
            }
            const int i = (r0 + rr) / G, h = kvh * G + (r0 + rr) % G;
            const long long orow = (static_cast<long long>(s) * p.num_draft + i) * p.num_heads + h;
            store_out(p.out, p.out_dtype, orow * D + col0 + c, d == 0.f ? 0.f : n / d);
        }
        __syncthreads();
    }
}

}  // namespace pa
