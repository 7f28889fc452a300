// Eviction by accumulated score: which cached tokens to keep, and the
// movement of their rows.
//
// Selection.  For each (sequence, kv head) the `recent` last tokens stay, and
// of the C tokens before them the k = budget - recent with the largest
// scores, of equal scores the lowest index.  A score's order is that of the
// unsigned image of its bits (sign bit flipped, negatives complemented; -0 as
// +0, NaN on top).  The k-th largest image is found by a radix search, one
// byte at a time from the top: a histogram of the next byte over the scores
// that share the bytes found so far, then the byte whose suffix count passes
// k.  One ordered pass then writes the kept indices: those above the k-th
// image, and the first (lowest-index) of those equal to it that are needed.
//
// Movement.  A row moves to an equal or lower place: place i takes token
// j >= i.  In place, a CTA owns the same 16-byte columns of every row of a
// (sequence, kv head) and walks the places upward, a chunk at a time: all
// loads of a chunk happen before its stores, and a later chunk only reads at
// or above its own first place, which the stores before it never reach.
// Into other blocks there is nothing to order, and the rows are split over
// more CTAs.
#include <cuda_runtime.h>

#include "pa_device.cuh"
#include "pa_evict.h"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;

__device__ inline uint32_t order_of(float x) {
    const uint32_t u = __float_as_uint(x);
    if ((u & 0x7fffffffu) > 0x7f800000u)
        return 0xffffffffu;  // NaN
    if (u == 0x80000000u)
        return 0x80000000u;  // -0 as +0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive prefix of `v` over the CTA (two packed 16-bit counts), and the total.
__device__ inline uint32_t cta_scan(uint32_t v, uint32_t *warp_sum, uint32_t &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o)
            x += y;
    }
    __syncthreads();  // the sums of the scan before are read
    if (lane == 31)
        warp_sum[warp] = x;
    __syncthreads();
    uint32_t before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) {
        const uint32_t t = warp_sum[w];
        before += w < warp ? t : 0;
        total += t;
    }
    return before + x - v;
}

// grid: (kv heads, sequences)
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectParams p) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ uint32_t hist[256];
    __shared__ uint32_t warp_sum[kSelWarps];
    __shared__ uint32_t found_byte, found_above;
    const int s = blockIdx.y, h = blockIdx.x, tid = threadIdx.x;
    int L = ld_nc_i32(p.context_lens + s);
    if (L > p.max_len) {
        if (p.err && tid == 0 && h == 0)
            atomicOr(p.err, PA_DEVERR_BAD_LEN);
        L = static_cast<int>(p.max_len);
    }
    L = max(L, 0);
    const int n = min(L, p.budget);
    const long long row = static_cast<long long>(s) * p.num_kv_heads + h;
    const float *in = p.scores + row * p.stride;
    float *out = p.scores_out ? p.scores_out + row * p.stride : nullptr;
    int32_t *keep = p.keep + row * p.budget;
    if (h == 0 && tid == 0)
        p.new_lens[s] = n;
    const int C = L > p.budget ? L - p.recent : 0;  // candidates
    const int k = L > p.budget ? p.budget - p.recent : 0;
    uint32_t kth = 0, above = 0;  // the k-th largest image, scores above it
    if (k > 0) {
        uint32_t need = k;
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += kSelThreads)
                hist[i] = 0;
            __syncthreads();
            const uint32_t high = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
            for (int t = tid; t < C; t += kSelThreads) {
                const uint32_t u = order_of(in[t]);
                if ((u & high) == (kth & high))
                    atomicAdd(&hist[(u >> shift) & 255], 1u);
            }
            __syncthreads();
            if (tid < 32) {  // suffix counts of 8 bins a lane, from the top
                uint32_t mine = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    mine += hist[255 - tid * 8 - i];
                uint32_t x = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
                    if (tid >= o)
                        x += y;
                }
                uint32_t before = x - mine;
                if (before < need && x >= need) {
                    int b = 255 - tid * 8;
                    while (before + hist[b] < need)
                        before += hist[b--];
                    found_byte = static_cast<uint32_t>(b);
                    found_above = before;
                }
            }
            __syncthreads();
            kth |= found_byte << shift;
            above += found_above;
            need -= found_above;
            __syncthreads();
        }
    }
    const uint32_t equal = k - above;  // scores equal to the k-th that are kept: the first ones
    // the ordered pass; a thread takes one token a round.  In place (scores_out
    // is scores), a score moves to an equal or lower index: a round's loads
    // come before its stores, and later rounds read higher indices only.
    uint32_t kept_above = 0, seen_equal = 0;
    for (int t0 = 0; t0 < C; t0 += kSelThreads) {
        const int t = t0 + tid;
        float x = 0.f;
        uint32_t u = 0;
        bool gt = false, eq = false;
        if (t < C) {
            x = in[t];
            u = order_of(x);
            gt = k > 0 && u > kth;
            eq = k > 0 && u == kth;
        }
        uint32_t total;
        const uint32_t pre = cta_scan((gt ? 1u : 0u) | (eq ? 0x10000u : 0u), warp_sum, total);
        const uint32_t eq_before = seen_equal + (pre >> 16);
        const uint32_t place = kept_above + (pre & 0xffffu) + min(eq_before, equal);
        if (gt || (eq && eq_before < equal)) {
            keep[place] = t;
            if (out)
                out[place] = x;
        }
        kept_above += total & 0xffffu;
        seen_equal += total >> 16;
    }
    __syncthreads();
    // the tokens kept for being recent (or all of a short context)
    const int from = C, head = k;
    for (int i0 = 0; i0 < L - from; i0 += kSelThreads) {
        const int i = i0 + tid;
        float x = 0.f;
        if (i < L - from)
            x = in[from + i];
        __syncthreads();
        if (i < L - from) {
            keep[head + i] = from + i;
            if (out)
                out[head + i] = x;
        }
    }
    __syncthreads();
    for (int i = n + tid; i < p.budget; i += kSelThreads)
        keep[i] = -1;
    if (out)
        for (long long i = n + tid; i < p.stride; i += kSelThreads)
            out[i] = 0.f;
}

constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 4;

// A thread moves one 16-byte column of kMoveUnroll rows a chunk.  grid.x:
// column segments x row splits, grid.y: kv heads x {K, V}, grid.z: sequences
// (65535 at a time).
template <bool InPlace>
__global__ void __launch_bounds__(kMoveThreads) compact_kernel(const CompactParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int s = blockIdx.z;
    const bool is_v = blockIdx.y >= static_cast<unsigned>(p.num_kv_heads);
    const int h = static_cast<int>(blockIdx.y) - (is_v ? p.num_kv_heads : 0);
    const int seg = static_cast<int>(blockIdx.x) % p.segs, split = static_cast<int>(blockIdx.x) / p.segs;
    const int rows = kMoveThreads / p.seg_chunks;  // rows a pass
    const int r = threadIdx.x / p.seg_chunks;
    const int col = seg * p.seg_chunks + threadIdx.x % p.seg_chunks;  // 16-byte column of a row
    const bool report = p.err && !is_v && seg == 0 && threadIdx.x % p.seg_chunks == 0;
    uint4 *cache = static_cast<uint4 *>(is_v ? p.v_cache : p.k_cache);
    const long long max_tok = static_cast<long long>(p.max_blocks) * p.block_size;
    const long long dst_tok = static_cast<long long>(p.dst_max_blocks) * p.block_size;
    const int n = min(max(ld_nc_i32(p.keep_lens + s), 0), p.keep_stride);
    const long long base = p.base_lens ? ld_nc_i32(p.base_lens + s) : 0;
    const int32_t *keep = p.keep + (static_cast<long long>(s) * p.keep_heads + (p.keep_heads > 1 ? h : 0)) *
                                       p.keep_stride;
    const int32_t *src_row = p.block_tables + static_cast<long long>(s) * p.max_blocks;
    const int32_t *dst_row = p.dst_block_tables + static_cast<long long>(s) * p.dst_max_blocks;
    // the 16-byte chunk of a token's row in the cache, -1 (flagged) when it has none
    auto chunk_of = [&](const int32_t *table, long long tok) -> long long {
        const int blk = static_cast<int>(tok / p.block_size);
        const int phys = ld_nc_i32(table + blk);
        if (phys < 0 || phys >= p.num_blocks) {
            if (report)
                atomicOr(p.err, PA_DEVERR_BAD_BLOCK);
            return -1;
        }
        const long long tile = static_cast<long long>(phys) * p.num_kv_heads + h;
        return (tile * p.block_size + (tok - static_cast<long long>(blk) * p.block_size)) * p.row_chunks + col;
    };
    const int chunk = rows * kMoveUnroll;
    for (int i0 = split * chunk; i0 < n; i0 += p.splits * chunk) {
        uint4 v[kMoveUnroll];
        long long to[kMoveUnroll];
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u) {
            const int i = i0 + u * rows + r;
            to[u] = -1;
            if (r < rows && i < n) {
                const int j = ld_nc_i32(keep + i);
                if (j < (InPlace ? i : 0) || base < 0 || base + j >= max_tok || base + i >= dst_tok) {
                    if (report)
                        atomicOr(p.err, PA_DEVERR_BAD_INDEX);
                } else if (!InPlace || j != i) {
                    const long long from = chunk_of(src_row, base + j);
                    const long long dst = chunk_of(dst_row, base + i);
                    if (from >= 0 && dst >= 0) {
                        v[u] = cache[from];
                        to[u] = dst;
                    }
                }
            }
        }
        if (InPlace)
            __syncthreads();  // every load of the chunk before its first store
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u)
            if (to[u] >= 0)
                cache[to[u]] = v[u];
        if (InPlace)
            __syncthreads();  // (the compiler keeps later loads behind this chunk's)
    }
}

}  // namespace

cudaError_t launch_select(SelectParams p, cudaStream_t stream) {
    for (int s0 = 0; s0 < p.num_seqs; s0 += 65535) {
        SelectParams c = p;
        const int n = p.num_seqs - s0 < 65535 ? p.num_seqs - s0 : 65535;
        const long long rows = static_cast<long long>(s0) * p.num_kv_heads;
        c.context_lens += s0;
        c.new_lens += s0;
        c.keep += rows * p.budget;
        c.scores += rows * p.stride;
        if (c.scores_out)
            c.scores_out += rows * p.stride;
        void *args[] = {&c};
        const cudaError_t e = launch_dependent(reinterpret_cast<const void *>(&select_kernel),
                                               dim3(p.num_kv_heads, n), dim3(kSelThreads), args, 0, stream);
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

cudaError_t launch_compact(CompactParams p, bool in_place, int num_sms, cudaStream_t stream) {
    p.seg_chunks = p.row_chunks < 4 ? p.row_chunks : 4;  // 64-byte column segments
    p.segs = p.row_chunks / p.seg_chunks;
    p.splits = 1;
    if (!in_place) {
        const int chunk = kMoveThreads / p.seg_chunks * kMoveUnroll;
        p.splits = (p.keep_stride + chunk - 1) / chunk;
        const long long ctas = static_cast<long long>(p.segs) * p.num_kv_heads * 2 * p.num_seqs;
        const long long most = (64LL * num_sms + ctas - 1) / ctas;
        if (p.splits > most)
            p.splits = static_cast<int>(most);
    }
    for (int s0 = 0; s0 < p.num_seqs; s0 += 65535) {
        CompactParams c = p;
        const int n = p.num_seqs - s0 < 65535 ? p.num_seqs - s0 : 65535;
        c.keep += static_cast<long long>(s0) * p.keep_heads * p.keep_stride;
        c.keep_lens += s0;
        if (c.base_lens)
            c.base_lens += s0;
        c.block_tables += static_cast<long long>(s0) * p.max_blocks;
        c.dst_block_tables += static_cast<long long>(s0) * p.dst_max_blocks;
        void *args[] = {&c};
        const void *fn = in_place ? reinterpret_cast<const void *>(&compact_kernel<true>)
                                  : reinterpret_cast<const void *>(&compact_kernel<false>);
        const cudaError_t e = launch_dependent(fn, dim3(p.segs * p.splits, 2 * p.num_kv_heads, n), dim3(kMoveThreads),
                                               args, 0, stream);
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

}  // namespace pa
