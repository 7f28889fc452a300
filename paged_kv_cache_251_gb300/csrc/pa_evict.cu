// Eviction by accumulated score: which cached tokens to keep, and the
// movement of their rows.
//
// Selection.  For each (sequence, kv head) the `recent` last tokens stay, and
// of the C tokens before them the k = budget - recent with the largest
// scores, of equal scores the lowest index.  A score's order is that of the
// unsigned image of its bits (sign bit flipped, negatives complemented; -0 as
// +0, NaN on top).  The k-th largest image is found by a radix search from the
// top, 11 + 11 + 10 bits: a histogram of the digit over the scores that share
// the digits found so far, then the digit whose suffix count passes k (2048
// bins: the first digit holds the exponent and two bits of mantissa, so scores of
// one magnitude do not all meet in one counter).  One ordered pass then writes
// the kept indices: the recent ones, those above the k-th image, and the first
// (lowest-index) of those equal to it that are needed.  A row is shared by the
// CTAs of a cluster, each holding a slice of it in shared memory (the scores are
// read from memory once); histograms and counts are exchanged through
// distributed shared memory.  Few long rows thus use many SMs.
//
// Movement.  A row moves to an equal or lower place: place i takes token
// j >= i.  A warp takes 32 places at a time, one a lane: kept index, both table
// entries and both addresses are found once a row, then whole rows of K and V
// go through the warp, addresses by shuffle.  Into other blocks there is nothing
// to order.  In place, a CTA owns all rows of a (sequence, kv head) of K or of V
// and walks the places upward, a chunk at a time: all loads of a chunk happen
// before its stores, and a later chunk only reads at or above its own first
// place, which the stores before it never reach.
//
// Measured: 64 contexts of 2049 to 8192 tokens, 8 kv heads of 128, bf16, cut to
// 2048: selection 26 us (latency of its passes over shared memory), movement 157 us,
// 6.5 TB/s (HBM).  Two contexts of 65537 to 131072 tokens cut to 16001: selection 28
// us (8 CTAs a row: 17 us of it loads and counting, the rest cluster barriers),
// movement 39 us, 6.7 TB/s.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "pa_device.cuh"
#include "pa_evict.h"
#include "pa_host.h"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;

// A score as it is compared and written: -0 as +0, any NaN as the one whose bits
// are largest.  Its order is then that of the image below.
__device__ inline float canonical(float x) { return x != x ? __int_as_float(0x7fffffff) : x + 0.f; }
__device__ inline uint32_t order_of(float canonical_x) {
    const int u = __float_as_int(canonical_x);
    return static_cast<uint32_t>(u ^ ((u >> 31) | static_cast<int>(0x80000000u)));
}

constexpr int kSelBins = 2048;
constexpr int kSelPer = 8;                        // tokens of a thread and round of the ordered pass
constexpr int kSelRound = kSelThreads * kSelPer;  // tokens of a round: 256 consecutive ones a warp
constexpr int kSelMaxSlice = 48 * 1024;           // scores a CTA holds in shared memory
constexpr int kSelMaxCluster = 8;

struct SelectShared {
    uint32_t hist[kSelBins];  // of this CTA's slice
    uint32_t all[kSelBins];   // of the row (clusters)
    uint32_t part[kSelBins];  // every CTA's counts of this CTA's share of the bins (clusters)
    uint32_t warp_sum[kSelWarps];
    uint32_t warp_count[2][kSelWarps];  // by round parity: kept surely | equal << 16
    uint32_t digit, above;
    uint32_t count[2];  // of the slice: kept surely, equal to the k-th
};

// One count more where `on`, without a branch (a taken branch an element cost 20
// cycles of a warp's 32, the atomic itself 5).
__device__ inline void count_if(bool on, uint32_t *bin) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t@p red.shared.add.u32 [%0], 1;\n\t}" ::"r"(
            static_cast<uint32_t>(__cvta_generic_to_shared(bin))),
        "r"(static_cast<uint32_t>(on))
        : "memory");
}

// grid: (kv heads x cluster, sequences); a cluster of p.cluster CTAs takes a
// row.  Cached: the slices are in shared memory.  Otherwise (rows longer than
// the cluster's shared memory) one CTA reads the row from memory in every pass.
template <bool Cached>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectParams p) {
    namespace cg = cooperative_groups;
    pdl_launch_dependents();
    pdl_wait();
    extern __shared__ __align__(16) char smem[];
    SelectShared *sh = reinterpret_cast<SelectShared *>(smem);
    float *slice = reinterpret_cast<float *>(smem + sizeof(SelectShared));
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = Cached ? static_cast<int>(cluster.block_rank()) : 0;
    const int ranks = Cached ? p.cluster : 1;
    const int s = blockIdx.y, h = blockIdx.x / ranks, tid = threadIdx.x;
    int L = ld_nc_i32(p.context_lens + s);
    if (L > p.max_len) {
        if (p.err && tid == 0 && h == 0 && rank == 0)
            atomicOr(p.err, PA_DEVERR_BAD_LEN);
        L = static_cast<int>(p.max_len);
    }
    L = max(L, 0);
    const int n = min(L, p.budget);
    const long long row = static_cast<long long>(s) * p.num_kv_heads + h;
    const float *in = p.scores + row * p.stride;
    float *out = p.scores_out ? p.scores_out + row * p.stride : nullptr;
    int32_t *keep = p.keep + row * p.budget;
    if (h == 0 && tid == 0 && rank == 0)
        p.new_lens[s] = n;
    const int C = L > p.budget ? L - p.recent : 0;  // candidates
    const int k = L > p.budget ? p.budget - p.recent : 0;
    // this CTA's tokens [lo, hi): slices of whole 16-byte groups
    const int per = Cached ? ((L + ranks - 1) / ranks + 3) & ~3 : L;
    const int lo = min(L, rank * per), hi = min(L, lo + per);
    const int chi = max(lo, min(hi, C));  // the slice's candidates: [lo, chi)
    for (int i = tid; i < kSelBins; i += kSelThreads)
        sh->hist[i] = 0;
    __syncthreads();
    if (Cached) {
        // the slice, canonical; its first histogram on the way (unless nothing is chosen: chi == lo)
        auto first = [&](int t, float x) { count_if(t < chi, &sh->hist[order_of(x) >> 21]); };
        int i = tid, n4 = 0;
        if ((reinterpret_cast<uintptr_t>(in + lo) & 15u) == 0) {
            n4 = (hi - lo) / 4;
            constexpr int kAhead = 4;  // loads of a thread in flight
            const float4 *in4 = reinterpret_cast<const float4 *>(in + lo);
            for (; i < n4; i += kAhead * kSelThreads) {
                float4 v[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u)
                    if (i + u * kSelThreads < n4)
                        v[u] = in4[i + u * kSelThreads];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int j = i + u * kSelThreads;
                    if (j < n4) {
                        const float4 c = make_float4(canonical(v[u].x), canonical(v[u].y), canonical(v[u].z),
                                                     canonical(v[u].w));
                        reinterpret_cast<float4 *>(slice)[j] = c;
                        first(lo + 4 * j, c.x);
                        first(lo + 4 * j + 1, c.y);
                        first(lo + 4 * j + 2, c.z);
                        first(lo + 4 * j + 3, c.w);
                    }
                }
            }
        }
        for (int j = n4 * 4 + tid; j < hi - lo; j += kSelThreads) {
            const float c = canonical(in[lo + j]);
            slice[j] = c;
            first(lo + j, c);
        }
    }
    auto score = [&](int t) -> float { return Cached ? slice[t - lo] : canonical(in[t]); };

    uint32_t kth = 0, above = 0;  // the k-th largest image, scores above it
    // of this slice: scores above the k-th (in the thread's bins), and equal to it
    // (one thread has them)
    uint32_t own_above = 0, own_equal = 0;
    if (k > 0) {
        uint32_t need = k;
#pragma unroll
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
            const uint32_t high = pass == 0 ? 0u : 0xffffffffu << (pass == 1 ? 21 : 10);
            const uint32_t digits = pass == 2 ? 1023u : 2047u;
            uint32_t *hist = sh->hist, *all = ranks > 1 ? sh->all : hist;
            auto count = [&](float x) {
                const uint32_t u = order_of(x);
                count_if((u & high) == (kth & high), &hist[(u >> shift) & digits]);
            };
            if (Cached && pass > 0) {
                const int n4 = (chi - lo) / 4;
#pragma unroll 2
                for (int i = tid; i < n4; i += kSelThreads) {
                    const float4 x = reinterpret_cast<const float4 *>(slice)[i];
                    count(x.x);
                    count(x.y);
                    count(x.z);
                    count(x.w);
                }
                if (tid < chi - lo - 4 * n4)
                    count(slice[4 * n4 + tid]);
            } else if (!Cached) {
#pragma unroll 4
                for (int t = lo + tid; t < chi; t += kSelThreads)
                    count(score(t));
            }
            const int top = kSelBins - 1 - 4 * tid;  // thread tid: bins top, top - 1, top - 2, top - 3
            if (ranks > 1) {
                // The row's histogram in every CTA: rank r sums bins [r, r + 1) 2048 / ranks over the
                // slices, and gives its sums to all.  One 16-byte access of a thread to another CTA's
                // memory each way (counts added there by remote atomics took 13000 cycles a pass
                // with many digits in use).
                cluster.sync();  // every slice is counted
                const int quads = kSelThreads / ranks, q = tid % quads, r = tid / quads;
                const int share = rank * (kSelBins / ranks) + 4 * q;
                reinterpret_cast<uint4 *>(sh->part)[tid] =
                    *reinterpret_cast<const uint4 *>(cluster.map_shared_rank(hist, r) + share);
                __syncthreads();
                uint4 sum = make_uint4(0, 0, 0, 0);
                for (int i = 0; i < ranks; ++i) {
                    const uint4 v = reinterpret_cast<const uint4 *>(sh->part)[i * quads + q];
                    sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
                }
                *reinterpret_cast<uint4 *>(cluster.map_shared_rank(all, r) + share) = sum;
                cluster.sync();
            } else {
                __syncthreads();
            }
            // suffix counts, from the top
            const uint4 v = *reinterpret_cast<const uint4 *>(all + top - 3);
            const uint4 ov = *reinterpret_cast<const uint4 *>(hist + top - 3);
            const uint32_t c[4] = {v.w, v.z, v.y, v.x}, own[4] = {ov.w, ov.z, ov.y, ov.x};
            const uint32_t mine = c[0] + c[1] + c[2] + c[3];
            // (counts up to 2^31: a plain scan, not the packed one)
            uint32_t x = mine;
            const int lane = tid & 31, warp = tid >> 5;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o)
                    x += y;
            }
            if (lane == 31)
                sh->warp_sum[warp] = x;
            __syncthreads();
            uint32_t before = x - mine;
#pragma unroll
            for (int w = 0; w < kSelWarps; ++w)
                before += w < warp ? sh->warp_sum[w] : 0;
            if (before < need && before + mine >= need) {
                int b = 0;
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    if (b == i && before + c[i] < need)
                        before += c[i], b = i + 1;
                sh->digit = static_cast<uint32_t>(top - b);
                sh->above = before;
            }
            if (pass < 2)  // for the next pass (everyone has read the counts)
                *reinterpret_cast<uint4 *>(hist + top - 3) = make_uint4(0, 0, 0, 0);
            __syncthreads();
            const uint32_t digit = sh->digit;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                own_above += static_cast<uint32_t>(top - i) > digit ? own[i] : 0;
                if (pass == 2 && static_cast<uint32_t>(top - i) == digit)
                    own_equal = own[i];
            }
            kth |= digit << shift;
            above += sh->above;
            need -= sh->above;
        }
    }
    const uint32_t equal = k - above;  // scores equal to the k-th that are kept: the first ones
    // a token is kept surely when it is recent (or the context short), or above the k-th
    auto classify = [&](int t, bool &sure, bool &eq, float &x) {
        x = 0.f;
        sure = eq = false;
        if (t < hi) {
            x = score(t);
            const uint32_t u = order_of(x);
            sure = t >= C || (k > 0 && u > kth);
            eq = !sure && k > 0 && u == kth;
        }
    };
    const int lane = tid & 31, warp = tid >> 5;
    uint32_t kept = 0, seen = 0;  // in the tokens before: kept surely, equal
    if (ranks > 1) {
        if (tid == 0) {
            sh->count[0] = max(0, hi - max(lo, C));  // recent ones (of a short context: all)
            sh->count[1] = 0;
        }
        __syncthreads();
        own_above = __reduce_add_sync(0xffffffffu, own_above);
        if (lane == 0 && own_above)
            atomicAdd(&sh->count[0], own_above);
        if (own_equal)
            sh->count[1] = own_equal;
        // (also: every slice is in shared memory before any score is written, which may be over them)
        cluster.sync();
        for (int r = 0; r < rank; ++r) {
            const uint32_t *rc = cluster.map_shared_rank(sh->count, r);
            kept += rc[0];
            seen += rc[1];
        }
    } else {
        __syncthreads();
    }
    // The ordered pass: a warp takes 256 consecutive tokens a round, a lane every
    // 32nd of them, so that places follow from ballots and the kept tokens of a
    // step go to adjacent places.  One barrier a round: the loads (and counts) of a
    // round come before it, its stores after it.  Without a cached slice and in
    // place, a score moves to an equal or lower index, and later rounds read higher
    // indices only.
    for (int t0 = lo, round = 0; t0 < hi; t0 += kSelRound, ++round) {
        const int t1 = t0 + warp * (32 * kSelPer) + lane;
        float x[kSelPer];
        uint32_t sure_bits = 0, eq_bits = 0, mine = 0;
#pragma unroll
        for (int i = 0; i < kSelPer; ++i) {
            bool sure, eq;
            classify(t1 + 32 * i, sure, eq, x[i]);
            sure_bits |= (sure ? 1u : 0u) << i;
            eq_bits |= (eq ? 1u : 0u) << i;
        }
        mine = __reduce_add_sync(0xffffffffu, __popc(sure_bits) | (__popc(eq_bits) << 16));
        uint32_t *count = sh->warp_count[round & 1];
        if (lane == 0)
            count[warp] = mine;
        __syncthreads();
        const uint32_t c = lane < kSelWarps ? count[lane] : 0;
        const uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? c : 0);
        const uint32_t total = __reduce_add_sync(0xffffffffu, c);
        uint32_t place_sure = kept + (before & 0xffffu), rank_eq = seen + (before >> 16);
        if ((mine >> 16) == 0) {  // (of the warp's tokens none is equal to the k-th: nearly always)
            place_sure += min(rank_eq, equal);
#pragma unroll
            for (int i = 0; i < kSelPer; ++i) {
                const bool sure = (sure_bits >> i) & 1u;
                const uint32_t sures = __ballot_sync(0xffffffffu, sure);
                if (sure) {
                    const uint32_t place = place_sure + __popc(sures & ((1u << lane) - 1u));
                    keep[place] = t1 + 32 * i;
                    if (out)
                        out[place] = x[i];
                }
                place_sure += __popc(sures);
            }
            mine = 0;
        }
#pragma unroll
        for (int i = 0; i < kSelPer && mine; ++i) {
            const bool sure = (sure_bits >> i) & 1u, eq = (eq_bits >> i) & 1u;
            const uint32_t sures = __ballot_sync(0xffffffffu, sure), eqs = __ballot_sync(0xffffffffu, eq);
            const uint32_t below = (1u << lane) - 1u;
            const uint32_t my_eq = rank_eq + __popc(eqs & below);
            if (sure || (eq && my_eq < equal)) {
                const uint32_t place = place_sure + __popc(sures & below) + min(my_eq, equal);
                keep[place] = t1 + 32 * i;
                if (out)
                    out[place] = x[i];
            }
            place_sure += __popc(sures);
            rank_eq += __popc(eqs);
        }
        kept += total & 0xffffu;
        seen += total >> 16;
    }
    __syncthreads();
    for (int i = n + rank * kSelThreads + tid; i < p.budget; i += ranks * kSelThreads)
        keep[i] = -1;
    if (out) {
        // up to a 16-byte boundary, four at a time, the rest
        const int head = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(out + n) & 15u)) & 15u) / 4;
        const long long from = min(static_cast<long long>(n + head), p.stride);
        const long long n4 = (p.stride - from) / 4, rest = from + 4 * n4;
        if (rank == 0 && tid < from - n)
            out[n + tid] = 0.f;
        for (long long j = rank * kSelThreads + tid; j < n4; j += ranks * kSelThreads)
            reinterpret_cast<float4 *>(out + from)[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (rank == 0 && tid < p.stride - rest)
            out[rest + tid] = 0.f;
    }
    if (ranks > 1)
        cluster.sync();  // no CTA leaves while another may read its counts
}

constexpr int kMoveThreads = 256;
constexpr int kMoveWarps = kMoveThreads / 32;
constexpr int kMoveUnroll = 4;

// The move of place i of (sequence s, kv head h): the 16-byte chunk where the
// source row starts, and the destination's; -1 when nothing moves.
struct Move {
    long long from, to;
};
template <bool InPlace>
__device__ inline Move find_move(const CompactParams &p, int s, int h, int i, int n, long long base, bool report) {
    Move m = {-1, -1};
    if (i >= n)
        return m;
    const int j = ld_nc_i32(p.keep + (static_cast<long long>(s) * p.keep_heads + (p.keep_heads > 1 ? h : 0)) *
                                         p.keep_stride + i);
    const long long src = base + j, dst = base + i;
    if (j < (InPlace ? i : 0) || base < 0 || src >= static_cast<long long>(p.max_blocks) << p.log_block ||
        dst >= static_cast<long long>(p.dst_max_blocks) << p.log_block) {
        if (report)
            atomicOr(p.err, PA_DEVERR_BAD_INDEX);
        return m;
    }
    if (InPlace && j == i)
        return m;
    const int sb = ld_nc_i32(p.block_tables + static_cast<long long>(s) * p.max_blocks + (src >> p.log_block));
    const int db = ld_nc_i32(p.dst_block_tables + static_cast<long long>(s) * p.dst_max_blocks + (dst >> p.log_block));
    if (sb < 0 || sb >= p.num_blocks || db < 0 || db >= p.num_blocks) {
        if (report)
            atomicOr(p.err, PA_DEVERR_BAD_BLOCK);
        return m;
    }
    const int mask = (1 << p.log_block) - 1;
    m.from = ((((static_cast<long long>(sb) * p.num_kv_heads + h) << p.log_block) + (src & mask)) * p.row_chunks);
    m.to = ((((static_cast<long long>(db) * p.num_kv_heads + h) << p.log_block) + (dst & mask)) * p.row_chunks);
    return m;
}

// Into other blocks.  Lpr lanes a row (16 bytes each).  grid.x: 32-row batches
// (8 a CTA), grid.y: kv heads, grid.z: sequences.
template <int Lpr>
__global__ void __launch_bounds__(kMoveThreads) compact_kernel(const CompactParams p) {
    pdl_launch_dependents();
    pdl_wait();
    constexpr int kRows = 32 / Lpr;  // rows of a warp access
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int s = blockIdx.z, h = blockIdx.y;
    const int n = min(max(ld_nc_i32(p.keep_lens + s), 0), p.keep_stride);
    const int i0 = (blockIdx.x * kMoveWarps + warp) * 32;
    if (i0 >= n)
        return;
    const long long base = p.base_lens ? ld_nc_i32(p.base_lens + s) : 0;
    const Move m = find_move<false>(p, s, h, i0 + lane, n, base, p.err != nullptr);
    uint4 *k = static_cast<uint4 *>(p.k_cache), *v = static_cast<uint4 *>(p.v_cache);
    const int sub = lane / Lpr, col = lane % Lpr;
#pragma unroll 1
    for (int r = 0; r < 32; r += kRows * kMoveUnroll) {
        uint4 kx[kMoveUnroll], vx[kMoveUnroll];
        long long to[kMoveUnroll];
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u) {
            const int rr = r + u * kRows + sub;
            const long long from = __shfl_sync(0xffffffffu, m.from, rr & 31);
            to[u] = __shfl_sync(0xffffffffu, m.to, rr & 31);
            if (rr >= 32 || from < 0)
                to[u] = -1;
            if (to[u] >= 0) {
                kx[u] = k[from + col];
                vx[u] = v[from + col];
            }
        }
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u)
            if (to[u] >= 0) {
                k[to[u] + col] = kx[u];
                v[to[u] + col] = vx[u];
            }
    }
}

// In place.  A CTA takes K or V of a (sequence, kv head), 32 rows a warp and
// chunk.  grid.x: kv heads, grid.y: {K, V}, grid.z: sequences.
template <int Lpr>
__global__ void __launch_bounds__(kMoveThreads) compact_in_place_kernel(const CompactParams p) {
    pdl_launch_dependents();
    pdl_wait();
    constexpr int kRows = 32 / Lpr;
    constexpr int kHold = 16;                 // 16-byte pieces a lane holds
    constexpr int kBatch = kHold * kRows;     // rows of a warp and chunk (at most 32)
    constexpr int kBatchRows = kBatch < 32 ? kBatch : 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int s = blockIdx.z, h = blockIdx.x;
    const int n = min(max(ld_nc_i32(p.keep_lens + s), 0), p.keep_stride);
    const long long base = p.base_lens ? ld_nc_i32(p.base_lens + s) : 0;
    uint4 *c = static_cast<uint4 *>(blockIdx.y ? p.v_cache : p.k_cache);
    const int sub = lane / Lpr, col = lane % Lpr;
    for (int i0 = 0; i0 < n; i0 += kMoveWarps * kBatchRows) {
        const int i = i0 + warp * kBatchRows + lane;
        const Move m = lane < kBatchRows ? find_move<true>(p, s, h, i, n, base, p.err && blockIdx.y == 0)
                                         : Move{-1, -1};
        uint4 x[kBatchRows / kRows];
#pragma unroll
        for (int u = 0; u < kBatchRows / kRows; ++u) {
            const long long from = __shfl_sync(0xffffffffu, m.from, u * kRows + sub);
            if (from >= 0)
                x[u] = c[from + col];
        }
        __syncthreads();  // every load of the chunk before its first store
#pragma unroll
        for (int u = 0; u < kBatchRows / kRows; ++u) {
            const long long to = __shfl_sync(0xffffffffu, m.to, u * kRows + sub);
            if (to >= 0)
                c[to + col] = x[u];
        }
        __syncthreads();  // (later loads stay behind)
    }
}

}  // namespace

cudaError_t launch_select(SelectParams p, int num_sms, cudaStream_t stream) {
    // a cluster a row: enough CTAs that a slice fits shared memory, and (for few
    // rows) that every SM has one, down to 2048 scores a CTA
    const long long rows = static_cast<long long>(p.num_seqs) * p.num_kv_heads;
    int cluster = 1;
    while (cluster < kSelMaxCluster &&
           ((p.max_len + cluster - 1) / cluster > kSelMaxSlice ||
            (rows * cluster < num_sms && (p.max_len + cluster - 1) / cluster > 2048)))
        cluster *= 2;
    const bool cached = (p.max_len + cluster - 1) / cluster <= kSelMaxSlice;
    if (!cached)
        cluster = 1;
    p.cluster = cluster;
    const void *fn = cached ? reinterpret_cast<const void *>(&select_kernel<true>)
                            : reinterpret_cast<const void *>(&select_kernel<false>);
    const size_t slice = cached ? static_cast<size_t>((p.max_len + cluster - 1) / cluster + 3) / 4 * 16 : 0;
    const size_t smem = sizeof(SelectShared) + slice;
    int dev = 0, sms = 0, per_sm = 0;
    cudaError_t e = device_sms(&dev, &sms);
    if (e == cudaSuccess)
        e = prepare_kernel(dev, fn, smem, kSelThreads, &per_sm);
    if (e != cudaSuccess)
        return e;
    for (int s0 = 0; s0 < p.num_seqs; s0 += 65535) {
        SelectParams c = p;
        const int n = p.num_seqs - s0 < 65535 ? p.num_seqs - s0 : 65535;
        const long long r0 = static_cast<long long>(s0) * p.num_kv_heads;
        c.context_lens += s0;
        c.new_lens += s0;
        c.keep += r0 * p.budget;
        c.scores += r0 * p.stride;
        if (c.scores_out)
            c.scores_out += r0 * p.stride;
        void *args[] = {&c};
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(p.num_kv_heads * cluster, n);
        cfg.blockDim = dim3(kSelThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = cluster;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        e = cudaLaunchKernelExC(&cfg, fn, args);
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

cudaError_t launch_compact(CompactParams p, bool in_place, cudaStream_t stream) {
    p.log_block = p.block_size == 8 ? 3 : (p.block_size == 16 ? 4 : 5);
    const void *fn;
    if (in_place)
        fn = p.row_chunks == 8    ? reinterpret_cast<const void *>(&compact_in_place_kernel<8>)
             : p.row_chunks == 16 ? reinterpret_cast<const void *>(&compact_in_place_kernel<16>)
                                  : reinterpret_cast<const void *>(&compact_in_place_kernel<32>);
    else
        fn = p.row_chunks == 8    ? reinterpret_cast<const void *>(&compact_kernel<8>)
             : p.row_chunks == 16 ? reinterpret_cast<const void *>(&compact_kernel<16>)
                                  : reinterpret_cast<const void *>(&compact_kernel<32>);
    const int batches = (p.keep_stride + kMoveWarps * 32 - 1) / (kMoveWarps * 32);
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
        const dim3 grid = in_place ? dim3(p.num_kv_heads, 2, n) : dim3(batches, p.num_kv_heads, n);
        const cudaError_t e = launch_dependent(fn, grid, dim3(kMoveThreads), args, 0, stream);
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

}  // namespace pa
