// Tree attention over the paged cache: what its kernels share, the general
// kernel, and the merge of partitions.
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
    int4 *cuts;     // tensor-core kernel: a record per CTA for the merge, or nullptr
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

// Whether query i attends drafted token j (both below the sequence's drafted count).
__device__ inline bool tree_bit(const TreeParams &p, int s, int i, int j) {
    if (!p.mask)
        return j <= i;
    const uint64_t w = p.mask[(static_cast<long long>(s) * p.num_draft + i) * p.words + (j >> 6)];
    return (w >> (j & 63)) & 1u;
}

// ---------------------------------------------------------------------------
// General kernel: any dtype, on the CUDA cores.  A CTA of 128 threads takes 16
// rows: 8 lanes a row, lane l holding elements l, l + 8, ... of its query and
// accumulator.  K and V of one block at a time are widened to fp32 in shared
// memory; every row then walks the block's tokens with an online softmax.

constexpr int kTreeRows = 16;
constexpr int kTreeThreads = kTreeRows * 8;

template <typename T, int D>
__global__ void __launch_bounds__(kTreeThreads) pa_tree_kernel(const TreeParams p) {
    pdl_launch_dependents();
    pdl_wait();
    constexpr int E = D / 8;
    constexpr int V = 16 / sizeof(T);  // elements per 16-byte load
    extern __shared__ __align__(16) float kv[];
    float *ks = kv, *vs = kv + p.block_size * D;
    const int G = p.num_heads / p.num_kv_heads;
    const int rows = p.num_draft * G;
    const int rl = threadIdx.x >> 3, l8 = threadIdx.x & 7;
    const int bs = p.block_size;
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
        const int r = rt * kTreeRows + rl;
        const bool mine = r < rows;
        const int i = mine ? r / G : 0;
        const int h = kvh * G + (mine ? r % G : 0);
        const bool live = mine && i < q.drafted;
        const long long orow = (static_cast<long long>(s) * p.num_draft + i) * p.num_heads + h;
        float qf[E], acc[E], m = -INFINITY, l = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            qf[e] = live ? static_cast<float>(static_cast<const T *>(p.q)[orow * D + l8 + 8 * e]) * p.scale_log2 : 0.f;
            acc[e] = 0.f;
        }
        const int b_lo = part * p.bpp, b_hi = min(b_lo + p.bpp, sp.nblk);
        for (int b = b_lo; b < b_hi; ++b) {
            const int phys = ld_nc_i32(p.block_tables + static_cast<long long>(s) * p.max_blocks_per_seq + b);
            if (phys < 0 || phys >= p.num_blocks) {  // (uniform over the CTA)
                if (threadIdx.x == 0 && p.err)
                    atomicOr(p.err, PA_DEVERR_BAD_BLOCK);
                continue;
            }
            const long long tile = (static_cast<long long>(phys) * p.num_kv_heads + kvh) * bs * D;
            __syncthreads();
            for (int c = threadIdx.x; c < bs * D / V; c += kTreeThreads) {
                Elt<T>::unpack(reinterpret_cast<const uint4 *>(static_cast<const T *>(p.k_cache) + tile)[c],
                               ks + c * V);
                Elt<T>::unpack(reinterpret_cast<const uint4 *>(static_cast<const T *>(p.v_cache) + tile)[c],
                               vs + c * V);
            }
            __syncthreads();
            const int hi = min(bs, q.len - b * bs);
            for (int u = 0; u < hi; ++u) {
                const int j = b * bs + u - committed;
                const bool ok = live && (j < 0 || tree_bit(p, s, i, j));
                float x = 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e)
                    x = fmaf(qf[e], ks[u * D + l8 + 8 * e], x);
                x += __shfl_xor_sync(0xffffffffu, x, 1);
                x += __shfl_xor_sync(0xffffffffu, x, 2);
                x += __shfl_xor_sync(0xffffffffu, x, 4);
                if (ok) {
                    const float mn = fmaxf(m, x);
                    const float alpha = mn == -INFINITY ? 1.f : exp2f(m - mn);
                    const float pw = x == -INFINITY ? 0.f : exp2f(x - mn);  // (a NaN score stays one)
                    l = fmaf(l, alpha, pw);
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        acc[e] = fmaf(acc[e], alpha, pw * vs[u * D + l8 + 8 * e]);
                    m = mn;
                }
            }
        }
        if (!mine)
            continue;
        if (sp.nparts == 1) {
            // (a NaN denominator is the row's own: it stays)
#pragma unroll
            for (int e = 0; e < E; ++e)
                store_out(p.out, p.out_dtype, orow * D + l8 + 8 * e, l == 0.f ? 0.f : acc[e] / l);
        } else {
            const long long item = (static_cast<long long>(s) * p.num_kv_heads + kvh) * p.max_parts + part;
#pragma unroll
            for (int e = 0; e < E; ++e)
                p.part_acc[(item * D + l8 + 8 * e) * rows + r] = acc[e];
            if (l8 == 0)
                reinterpret_cast<float2 *>(p.part_ml)[item * rows + r] = make_float2(m, l);
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
