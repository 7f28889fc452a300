// Tree attention over the paged cache: what its kernels share, the general
// kernel, and the merge of partitions.
//
// Sequence s has L = context_lens[s] cached tokens, the last T_s of them
// drafted.  Row r = i * G + g of a (sequence, kv head) is query head g of
// drafted token i (G query heads share the kv head), so all T * G rows read
// the same K/V rows: cached token t is attended by row r when
//   t < L - T_s   (committed), or bit t - (L - T_s) of mask[s][i] is set.
// Work unit: (sequence, kv head, row tile, context partition); partitions are
// merged by log-sum-exp as in the other decodes.
#pragma once

#include "pa_decode.cuh"

namespace pa {

struct TreeParams : DecodeParams {
    const int32_t *draft_lens;  // [num_seqs] or nullptr (num_draft everywhere)
    const uint64_t *mask;       // [num_seqs][num_draft][words] or nullptr (chain)
    int num_draft, words;
    int row_tiles;  // tiles of rows a (sequence, kv head)
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
            const long long pr = orow * p.max_parts + part;
#pragma unroll
            for (int e = 0; e < E; ++e)
                p.part_acc[pr * D + l8 + 8 * e] = acc[e];
            if (l8 == 0) {
                p.part_ml[pr * 2] = m;
                p.part_ml[pr * 2 + 1] = l;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Merge of the partitions of every row of a multi-partition sequence, a warp a
// row; a partition in which the row attends nothing (l == 0) left no
// accumulator.
constexpr int kTreeMergeThreads = 128;

template <int D>
__global__ void __launch_bounds__(kTreeMergeThreads) pa_tree_merge_kernel(const TreeParams p) {
    pdl_launch_dependents();
    pdl_wait();
    constexpr int kPer = D / 32;
    const int lane = threadIdx.x & 31;
    const long long row = static_cast<long long>(blockIdx.x) * (kTreeMergeThreads / 32) + (threadIdx.x >> 5);
    if (row >= static_cast<long long>(p.num_seqs) * p.num_draft * p.num_heads)
        return;
    const int s = static_cast<int>(row / (static_cast<long long>(p.num_draft) * p.num_heads));
    const SeqSpan sp = seq_span(ld_nc_i32(p.context_lens + s), p.max_len, 0, p.block_size, p.bpp);
    if (sp.nparts <= 1)
        return;
    const float2 *ml = reinterpret_cast<const float2 *>(p.part_ml) + row * p.max_parts;
    const float *a = p.part_acc + row * p.max_parts * D + lane * kPer;
    float M = -INFINITY, den = 0.f, num[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e)
        num[e] = 0.f;
    for (int q = 0; q < sp.nparts; ++q) {
        const float2 v = ml[q];
        if (v.y == 0.f)
            continue;
        const float mn = fmaxf(M, v.x);
        const float keep = M == -INFINITY ? 0.f : exp2f(M - mn), add = exp2f(v.x - mn);
        den = den * keep + v.y * add;
#pragma unroll
        for (int e = 0; e < kPer; ++e)
            num[e] = num[e] * keep + a[static_cast<long long>(q) * D + e] * add;
        M = mn;
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e)
        store_out(p.out, p.out_dtype, row * D + lane * kPer + e, den == 0.f ? 0.f : num[e] / den);
}

}  // namespace pa
