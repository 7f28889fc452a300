// Block tables and reference counts on the device: the tables of a next step
// (rows kept, forked, cut, freed and grown, shared last blocks copied on write), the
// used blocks of a pool moved to its front, and the copies that both ask for.
// ("PagedAttention — 把 KV cache 当虚拟内存页来管理", 案例 3: reference counts,
// copy-on-write, one block is the copy unit.)
//
// A block is free when its count is 0; free blocks are handed out in ascending
// order, row by row, so the result is a function of the inputs alone.
//
// The first two are bound by latency: a few dependent passes over arrays of some
// hundred KB, each needing the whole of the one before.  Both are a single kernel of
// one cluster of CTAs, its barriers between the passes (a launch a pass would cost
// more than a pass).  Ordered ranks (which free block is the k-th) are a count a CTA,
// exchanged through shared memory, and a scan within it.
//
// Measured on the GPU, copies included: a step of 256 rows over a pool of 25000 blocks
// 16 us (four barriers 3, the tables' rows 3, the rest dependent reads of 0.4 us), 32
// prompts of 8 forked beams 18 to 19 us, a pool of 38000 blocks with 12000 moves of 16 KB,
// K and V, 111 us (the copies 97, 6.3 TB/s; floor of the whole 91).
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <atomic>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_pages.h"

namespace cg = cooperative_groups;

namespace pa {

namespace {

constexpr int kPageThreads = 1024;
constexpr int kPageWarps = kPageThreads / 32;
static_assert(kPageWarps == 32, "block_scan: a lane a warp's sum");
constexpr int kPageMaxCluster = 16;  // 8 where the GPU holds no cluster of 16
constexpr int kCopied = 1 << 31;
// Rows up to which a CTA holds their parents and kept blocks in shared memory, and looks for an old
// row's children there: a step of 256 rows 13.4 us, else 15.9; of 1024 22.4 and 24.2; of 2048
// 38.8 and 29.2; 2048 forked beams 36.6 and 26.9.
constexpr int kRowsHeld = 1024;

struct PagesShared {
    int warp[kPageWarps];
    int sum;                              // of block_sum
    long long total[3][kPageMaxCluster];  // every CTA's counts
    int parent[kRowsHeld], kept[kRowsHeld];
};

// Exclusive prefix of `x` over the CTA's threads; *all gets the sum.
__device__ inline int block_scan(int x, PagesShared *sh, int *all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o)
            incl += y;
    }
    __syncthreads();  // (the last call's sums were read)
    if (lane == 31)
        sh->warp[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        int w = sh->warp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o)
                w += y;
        }
        sh->warp[lane] = w;
    }
    __syncthreads();
    *all = sh->warp[kPageWarps - 1];
    return incl - x + (warp ? sh->warp[warp - 1] : 0);
}

// Sum of `x` over the CTA's threads, added to sh->sum (zero before; read after a barrier).
__device__ inline void block_sum(int x, PagesShared *sh) {
    x = __reduce_add_sync(0xffffffffu, x);
    if ((threadIdx.x & 31) == 0 && x)
        atomicAdd(&sh->sum, x);
}

__device__ inline int blocks_of(long long tokens, int block_size) {
    return static_cast<int>((tokens + block_size - 1) / block_size);
}

// A row of the update, from its inputs.
struct Row {
    int parent;  // -1: none
    int keep, grow;  // tokens
    int kept, total;  // blocks
    int last;  // the last kept block if tokens are written behind its kept ones, else -1
};

__device__ inline int held_len(const PagesUpdateParams &p, int row) {
    const long long most = static_cast<long long>(p.max_blocks) * p.block_size;
    const int n = p.lens[row];
    return n < 0 ? 0 : (n > most ? static_cast<int>(most) : n);
}

__device__ inline Row row_of(const PagesUpdateParams &p, int i) {
    const long long most = static_cast<long long>(p.max_blocks) * p.block_size;
    Row r;
    r.parent = p.parents ? p.parents[i] : i;
    if (r.parent < 0 || r.parent >= p.old_rows)
        r.parent = -1;
    const int have = r.parent >= 0 ? held_len(p, r.parent) : 0;
    const int keep = p.keep[i];
    r.keep = keep < 0 ? 0 : (keep > have ? have : keep);
    const long long grow = p.grow[i];
    r.grow = grow > most ? static_cast<int>(most) : (grow < r.keep ? r.keep : static_cast<int>(grow));
    r.kept = blocks_of(r.keep, p.block_size);
    r.total = blocks_of(r.grow, p.block_size);
    r.last = -1;
    if (r.grow > r.keep && r.keep % p.block_size != 0) {
        const int b = p.tables[static_cast<long long>(r.parent) * p.max_blocks + r.kept - 1];
        if (b >= 0 && b < p.num_blocks)
            r.last = b;
    }
    return r;
}

// Entries that a warp loads before it uses the first.
constexpr int kAhead = 8;

// Adds `by` to the counts of entries [j0, j1) of an old row (a warp).
__device__ inline void count_entries(const PagesUpdateParams &p, int row, int j0, int j1, int by, int lane) {
    const int32_t *t = p.tables + static_cast<long long>(row) * p.max_blocks;
    bool bad = false;
    for (int j = j0 + lane; j < j1; j += 32 * kAhead) {
        int b[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            b[k] = j + 32 * k < j1 ? t[j + 32 * k] : 0;
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (j + 32 * k < j1) {
                if (b[k] >= 0 && b[k] < p.num_blocks)
                    atomicAdd(p.count + b[k], by);
                else
                    bad = true;
            }
    }
    if (bad && p.err)
        atomicOr(p.err, PA_DEVERR_BAD_BLOCK);
}

// Four consecutive counts, those from `end` on as `none`.
__device__ inline void load_counts(const int32_t *from, int b, int end, int none, int *c) {
    if (b + 4 <= end && (reinterpret_cast<uintptr_t>(from + b) & 15u) == 0) {
        const int4 x = __ldcg(reinterpret_cast<const int4 *>(from + b));
        c[0] = x.x, c[1] = x.y, c[2] = x.z, c[3] = x.w;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            c[k] = b + k < end ? __ldcg(from + b + k) : none;
    }
}

// Of four consecutive blocks with counts c: where they are, ~ that of those without a count.
__device__ inline void store_places(int32_t *to, int b, int end, const int *c) {
    int x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        x[k] = c[k] > 0 ? b + k : ~(b + k);
    if (b + 4 <= end && (reinterpret_cast<uintptr_t>(to + b) & 15u) == 0) {
        *reinterpret_cast<int4 *>(to + b) = make_int4(x[0], x[1], x[2], x[3]);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (b + k < end)
                to[b + k] = x[k];
    }
}

constexpr int kTile = 4 * kPageThreads;  // counts of a CTA at once

// A CTA's share of the blocks: whole groups of four.
__device__ inline void block_share(int num_blocks, int rank, int ranks, int *b0, int *b1) {
    const long long share = (static_cast<long long>(num_blocks) + 4 * ranks - 1) / (4 * ranks) * 4;
    *b0 = static_cast<int>(min(rank * share, static_cast<long long>(num_blocks)));
    *b1 = static_cast<int>(min((rank + 1) * share, static_cast<long long>(num_blocks)));
}

// Parts of a row of tables, a warp each, such that every warp has one (of 128 entries at least:
// 32 or 1024 measure the same at 256 to 2048 rows of 64 to 128 entries).
__device__ inline int row_part(int max_blocks, int rows, int warps, int *parts) {
    const int want = max(1, min(warps / max(rows, 1), (max_blocks + 127) / 128));
    const int part = ((max_blocks + want - 1) / want + 31) / 32 * 32;
    *parts = (max_blocks + part - 1) / part;
    return part;
}

// What the entries that the update's rows keep tell of: blocks outside the pool, and blocks that no
// reference counts any more, which go out as free ones, too.  The warps of a CTA take rows from the
// last warp on (the first have needs to find meanwhile).  Only calls with an error word pay for it:
// with 256 rows 0.6 to 1 us, with 1024 or 2048 4 to 5 (a gather of every entry's count).
__device__ inline uint32_t kept_errors(const PagesUpdateParams &p, int rank, int ranks, int warp, int lane) {
    uint32_t bad = 0;
    int parts;
    const int warps = ranks * kPageWarps, part = row_part(p.max_blocks, p.rows, warps, &parts);
    const long long items = static_cast<long long>(p.rows) * parts;
    for (long long u = rank + ranks * (kPageWarps - 1 - warp); u < items; u += warps) {
        const int i = static_cast<int>(u / parts), j0 = static_cast<int>(u % parts) * part;
        const int kept = __ldcg(p.kept + i), parent = p.parents ? p.parents[i] : i, j1 = min(kept, j0 + part);
        const int32_t *from = p.tables + static_cast<long long>(kept ? parent : 0) * p.max_blocks;
        for (int j = j0 + lane; j < j1; j += 32 * kAhead) {
            int b[kAhead], c[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                b[k] = j + 32 * k < j1 ? from[j + 32 * k] : -1;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const bool inside = b[k] >= 0 && b[k] < p.num_blocks;
                bad |= inside || j + 32 * k >= j1 ? 0u : PA_DEVERR_BAD_BLOCK;
                c[k] = inside ? __ldcg(p.count + b[k]) : 1;
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                bad |= c[k] > 0 ? 0u : PA_DEVERR_BAD_COUNT;
        }
    }
    return bad;
}

// The children of an old row (a warp): how many, and how many blocks all of them keep.
struct Children {
    int count, kept;  // kept 0 without any
};
__device__ inline Children children_of(const PagesUpdateParams &p, const PagesShared *sh, int row, int lane) {
    int n = 0, least = 0x7fffffff;
    for (int i = lane; i < p.rows; i += 32)
        if (sh->parent[i] == row) {
            ++n;
            least = min(least, sh->kept[i]);
        }
    n = __reduce_add_sync(0xffffffffu, n);
    least = __reduce_min_sync(0xffffffffu, least);
    return {n, n ? least : 0};
}

__global__ void __launch_bounds__(kPageThreads, 1) pages_update_kernel(const PagesUpdateParams p) {
    __shared__ PagesShared shared;
    PagesShared *sh = &shared;
    pdl_launch_dependents();
    pdl_wait();
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank()), ranks = static_cast<int>(cluster.num_blocks());
    const int tid = threadIdx.x, lane = tid & 31;
    const int gtid = rank * kPageThreads + tid, gthreads = ranks * kPageThreads;
    const int gwarp = gtid >> 5, gwarps = gthreads >> 5;
    const long long most = static_cast<long long>(p.max_blocks) * p.block_size;
    const int rows_share = (p.rows + ranks - 1) / ranks;
    const int i0 = min(rank * rows_share, p.rows), i1 = min(i0 + rows_share, p.rows);
    int b0, b1, all;
    block_share(p.num_blocks, rank, ranks, &b0, &b1);
    const bool one_tile = b1 - b0 <= kTile;

    // counts to work on; what the rows keep and get; a clean slate where writers will meet
    int c[4];
    load_counts(p.refs, b0 + 4 * tid, b1, 0, c);
    if (tid < 3 * kPageMaxCluster)
        (&sh->total[0][0])[tid] = 0;
    for (int i = i0 + tid; i < i1; i += kPageThreads) {
        const Row r = row_of(p, i);
        p.kept[i] = r.kept;
        p.total[i] = r.total;
        p.base[i] = r.last;  // (until it is known)
        if (r.last >= 0) {
            p.first[r.last] = p.rows;
            p.writers[r.last] = 0;
        }
        const int given = p.parents ? p.parents[i] : i;
        if (p.err && given >= p.old_rows)
            atomicOr(p.err, PA_DEVERR_BAD_INDEX);
        if (p.err && p.grow[i] > most)
            atomicOr(p.err, PA_DEVERR_BAD_LEN);
    }
    for (int t0 = b0; t0 < b1; t0 += kTile) {
        const int b = t0 + 4 * tid;
        if (t0 != b0)
            load_counts(p.refs, b, b1, 0, c);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (b + k < b1)
                p.count[b + k] = c[k];
    }
    if (tid == 0)
        sh->sum = 0;
    cluster.sync();

    // writers of the last blocks
    for (int i = i0 + tid; i < i1; i += kPageThreads) {
        const int last = __ldcg(p.base + i);
        if (last >= 0) {
            atomicMin(p.first + last, i);
            atomicAdd(p.writers + last, 1);
        }
    }
    // References: an old row lets go of its blocks, a new row holds what it keeps.  What all
    // children of a row keep is counted once, with their number: nothing for an only child.
    const bool held = p.rows <= kRowsHeld;
    if (held) {
        for (int i = tid; i < p.rows; i += kPageThreads) {
            const int parent = p.parents ? p.parents[i] : i;
            sh->parent[i] = parent < p.old_rows ? parent : -1;
            sh->kept[i] = __ldcg(p.kept + i);
        }
        __syncthreads();
    }
    const int both = max(p.rows, p.old_rows);
    int parts;
    const int part = row_part(p.max_blocks, both, gwarps, &parts);
    for (long long x = gwarp; x < static_cast<long long>(both) * parts; x += gwarps) {
        const int r = static_cast<int>(x / parts), j0 = static_cast<int>(x % parts) * part, j1 = j0 + part;
        if (r < p.old_rows) {
            const int len = p.lens[r];
            if (lane == 0 && j0 == 0 && p.err && (len < 0 || len > most))
                atomicOr(p.err, PA_DEVERR_BAD_LEN);
            const int n = blocks_of(held_len(p, r), p.block_size);
            Children ch = {0, 0};
            if (held)
                ch = children_of(p, sh, r, lane);
            if (ch.count != 1)
                count_entries(p, r, j0, min(ch.kept, j1), ch.count - 1, lane);
            count_entries(p, r, max(ch.kept, j0), min(n, j1), -1, lane);
        }
        if (r < p.rows) {
            const int parent = held ? sh->parent[r] : (p.parents ? p.parents[r] : r);
            if (parent >= 0 && parent < p.old_rows) {
                const int from = held ? children_of(p, sh, parent, lane).kept : 0;
                const int kept = held ? sh->kept[r] : __ldcg(p.kept + r);
                count_entries(p, parent, max(from, j0), min(kept, j1), 1, lane);
            }
        }
    }
    cluster.sync();

    // what each row needs, and how many blocks are free, a share a CTA
    load_counts(p.count, b0 + 4 * tid, b1, 1, c);
    uint32_t bad = 0;
    if (p.err)
        bad = kept_errors(p, rank, ranks, tid >> 5, lane);
    long long needs = 0;
    int copies = 0;
    for (int at = i0; at < i1; at += kPageThreads) {
        const int i = at + tid;
        int need = 0;
        if (i < i1) {
            const int last = __ldcg(p.base + i);
            // a last block stays where all its holders write to it, with the first of them
            bool copied = false;
            if (last >= 0) {
                const int writers = __ldcg(p.writers + last), holders = __ldcg(p.count + last);
                copied = !(writers == holders && __ldcg(p.first + last) == i);
                bad |= writers > holders ? PA_DEVERR_BAD_COUNT : 0u;
            }
            need = __ldcg(p.total + i) - __ldcg(p.kept + i) + copied;
            copies += copied;
            p.need[i] = need | (copied ? kCopied : 0);
        }
        const int before = block_scan(need, sh, &all);
        if (i < i1)
            p.base[i] = static_cast<int>(needs) + before;  // within the CTA's rows
        needs += all;
    }
    block_sum(copies, sh);
    long long spare = 0;
    int place = 0;  // free blocks of the CTA before the thread's four (of its last tile)
    for (int t0 = b0; t0 < b1; t0 += kTile) {
        if (t0 != b0)
            load_counts(p.count, t0 + 4 * tid, b1, 1, c);
        place = block_scan((c[0] == 0) + (c[1] == 0) + (c[2] == 0) + (c[3] == 0), sh, &all);
        spare += all;
        bad |= min(min(c[0], c[1]), min(c[2], c[3])) < 0 ? PA_DEVERR_BAD_COUNT : 0u;
    }
    if (bad && p.err)
        atomicOr(p.err, bad);
    __syncthreads();
    if (tid < ranks) {
        PagesShared *to = cluster.map_shared_rank(sh, tid);
        to->total[0][rank] = needs;
        to->total[1][rank] = spare;
        to->total[2][rank] = sh->sum;
    }
    cluster.sync();

    long long needed = 0, free = 0, copied_all = 0, need_before = 0, free_before = 0;
#pragma unroll
    for (int r = 0; r < kPageMaxCluster; ++r) {  // (zeros beyond the last CTA)
        if (r == rank) {
            need_before = needed;
            free_before = free;
        }
        needed += sh->total[0][r];
        free += sh->total[1][r];
        copied_all += sh->total[2][r];
    }
    const bool done = needed <= free;
    if (gtid == 0) {
        p.status[0] = done;
        p.status[1] = needed > 0x7fffffff ? 0x7fffffff : static_cast<int>(needed);
        p.status[2] = static_cast<int>(done ? free - needed : free);
        p.status[3] = done ? static_cast<int>(copied_all) : 0;
    }
    if (!done) {  // nothing changes
        for (int i = gtid; i < p.rows; i += gthreads) {
            p.pairs[2 * static_cast<long long>(i)] = -1;
            p.pairs[2 * static_cast<long long>(i) + 1] = -1;
        }
        return;
    }
    // the free blocks in order, as far as they are needed, and the counts (copied blocks
    // lose their holder later)
    {
        long long at = free_before;
        for (int t0 = b0; t0 < b1; t0 += kTile) {
            const int b = t0 + 4 * tid;
            if (!one_tile) {  // (else the counts and places are those of above)
                load_counts(p.count, b, b1, 1, c);
                place = block_scan((c[0] == 0) + (c[1] == 0) + (c[2] == 0) + (c[3] == 0), sh, &all);
            }
            long long k0 = at + place;
            at += all;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (b + k < b1) {
                    if (c[k] == 0 && k0++ < needed) {
                        p.free_list[k0 - 1] = b + k;
                        c[k] = 1;
                    }
                    p.new_refs[b + k] = c[k];
                }
        }
    }
    // places in the whole list
    for (int i = i0 + tid; i < i1; i += kPageThreads)
        p.base[i] += static_cast<int>(need_before);
    cluster.sync();

    for (int i = gtid; i < p.rows; i += gthreads) {
        int64_t src = -1, dst = -1;
        if (__ldcg(p.need + i) & kCopied) {
            dst = __ldcg(p.free_list + __ldcg(p.base + i));
            src = p.tables[static_cast<long long>(p.parents ? p.parents[i] : i) * p.max_blocks + __ldcg(p.kept + i) - 1];
            atomicAdd(p.new_refs + src, -1);
        }
        p.pairs[2 * static_cast<long long>(i)] = src;
        p.pairs[2 * static_cast<long long>(i) + 1] = dst;
    }
    const int out_part = row_part(p.max_blocks, p.rows, gwarps, &parts);
    for (long long u = gwarp; u < static_cast<long long>(p.rows) * parts; u += gwarps) {
        const int i = static_cast<int>(u / parts), j0 = static_cast<int>(u % parts) * out_part;
        const int j1 = min(p.max_blocks, j0 + out_part);
        const int parent = p.parents ? p.parents[i] : i;
        const int kept = __ldcg(p.kept + i), total = __ldcg(p.total + i), base = __ldcg(p.base + i);
        const bool copied = __ldcg(p.need + i) & kCopied;
        const int32_t *from = p.tables + static_cast<long long>(kept ? parent : 0) * p.max_blocks;
        int32_t *to = p.new_tables + static_cast<long long>(i) * p.max_blocks;
        for (int j = j0 + lane; j < j1; j += 32 * kAhead) {
            int b[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int at = j + 32 * k;
                b[k] = -1;
                if (at < j1 && at < kept)
                    b[k] = copied && at == kept - 1 ? __ldcg(p.free_list + base) : from[at];
                else if (at < j1 && at < total && base + copied + (at - kept) < needed)
                    b[k] = __ldcg(p.free_list + base + copied + (at - kept));
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (j + 32 * k < j1)
                    to[j + 32 * k] = b[k];
        }
    }
}

__device__ inline int held_len(const PagesCompactParams &p, int row) {
    const long long most = static_cast<long long>(p.max_blocks) * p.block_size;
    const int n = p.lens[row];
    return n < 0 ? 0 : (n > most ? static_cast<int>(most) : n);
}

// With U blocks in use, a used block b >= U that has k used blocks above it goes
// to the k-th free block below U (there are as many).
__global__ void __launch_bounds__(kPageThreads, 1) pages_compact_kernel(const PagesCompactParams p) {
    __shared__ PagesShared shared;
    PagesShared *sh = &shared;
    pdl_launch_dependents();
    pdl_wait();
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank()), ranks = static_cast<int>(cluster.num_blocks());
    const int tid = threadIdx.x, lane = tid & 31;
    const int gtid = rank * kPageThreads + tid, gthreads = ranks * kPageThreads;
    const int gwarp = gtid >> 5, gwarps = gthreads >> 5;
    int b0, b1, all;
    block_share(p.num_blocks, rank, ranks, &b0, &b1);
    if (tid == 0)
        sh->sum = 0;
    if (tid < 2 * kPageMaxCluster)
        (&sh->total[0][0])[tid] = 0;
    cluster.sync();  // (before another CTA's count)
    {
        int mine = 0;
        for (int t0 = b0; t0 < b1; t0 += kTile) {
            int c[4];
            load_counts(p.refs, t0 + 4 * tid, b1, 0, c);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                mine += c[k] > 0;
                if (c[k] < 0 && p.err)
                    atomicOr(p.err, PA_DEVERR_BAD_COUNT);
            }
        }
        block_sum(mine, sh);
        __syncthreads();
        if (tid < ranks)
            cluster.map_shared_rank(sh, tid)->total[0][rank] = sh->sum;
    }
    cluster.sync();
    if (tid == 0)
        sh->sum = 0;  // (read before the barrier; added to behind a block_scan's)
    long long used = 0, before = 0;
#pragma unroll
    for (int r = 0; r < kPageMaxCluster; ++r) {
        if (r == rank)
            before = used;
        used += sh->total[0][r];
    }
    int movers = 0;
    for (int t0 = b0; t0 < b1; t0 += kTile) {
        const int b = t0 + 4 * tid;
        int c[4], n = 0;
        load_counts(p.refs, b, b1, 0, c);
        if (p.err)
            store_places(p.place, b, b1, c);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            n += c[k] > 0;
        long long below = before + block_scan(n, sh, &all);  // used blocks below b + k
        before += all;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (b + k >= b1)
                continue;
            p.new_refs[b + k] = c[k];
            p.remap[b + k] = b + k;
            if (c[k] > 0) {
                if (b + k >= used) {
                    const long long place = used - 1 - below;
                    if (place <= p.max_moves)  // (one more: the highest that stays)
                        p.src_list[place] = b + k;
                    ++movers;
                }
                ++below;
            } else if (b + k < used && b + k - below < p.max_moves) {
                p.dst_list[b + k - below] = b + k;
            }
        }
    }
    block_sum(movers, sh);
    __syncthreads();
    if (tid < ranks)
        cluster.map_shared_rank(sh, tid)->total[1][rank] = sh->sum;
    cluster.sync();
    long long total = 0;
#pragma unroll
    for (int r = 0; r < kPageMaxCluster; ++r)
        total += sh->total[1][r];
    const int moves = total < p.max_moves ? static_cast<int>(total) : p.max_moves;
#pragma unroll 2
    for (int k = gtid; k < p.max_moves; k += gthreads) {
        int src = -1, dst = -1;
        if (k < moves) {
            src = __ldcg(p.src_list + k);
            dst = __ldcg(p.dst_list + k);
            p.remap[src] = dst;
            if (p.err)
                p.place[src] = dst;
            p.new_refs[dst] = __ldcg(p.new_refs + src);
            p.new_refs[src] = 0;
        }
        p.pairs[2 * static_cast<long long>(k)] = src;
        p.pairs[2 * static_cast<long long>(k) + 1] = dst;
    }
    cluster.sync();
    int parts;
    const int part = row_part(p.max_blocks, p.rows, gwarps, &parts);
    const long long most = static_cast<long long>(p.max_blocks) * p.block_size;
    // (with an error word: blocks without a count, free ones to all others, are told of where a row
    // holds them; 0.2 to 0.6 us)
    const int32_t *place = p.err ? p.place : p.remap;
    for (long long u = gwarp; u < static_cast<long long>(p.rows) * parts; u += gwarps) {
        const int i = static_cast<int>(u / parts), j0 = static_cast<int>(u % parts) * part;
        const int j1 = min(p.max_blocks, j0 + part);
        const int len = p.lens[i], n = blocks_of(held_len(p, i), p.block_size);
        uint32_t bad = len < 0 || len > most ? PA_DEVERR_BAD_LEN : 0u;
        const int32_t *from = p.tables + static_cast<long long>(i) * p.max_blocks;
        int32_t *to = p.new_tables + static_cast<long long>(i) * p.max_blocks;
        for (int j = j0 + lane; j < j1; j += 32 * kAhead) {
            int b[kAhead];
            unsigned inside = 0;
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                b[k] = j + 32 * k < j1 && j + 32 * k < n ? from[j + 32 * k] : -1;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (b[k] >= 0 && b[k] < p.num_blocks) {
                    b[k] = __ldcg(place + b[k]);
                    inside |= 1u << k;
                } else if (j + 32 * k < j1 && j + 32 * k < n) {
                    bad |= PA_DEVERR_BAD_BLOCK;
                }
            }
            if (p.err) {
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
                    if (inside >> k & 1 && b[k] < 0) {
                        b[k] = ~b[k];
                        bad |= PA_DEVERR_BAD_COUNT;
                    }
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (j + 32 * k < j1)
                    to[j + 32 * k] = b[k];
        }
        if (p.err && bad)
            atomicOr(p.err, bad);
    }
    if (gtid == 0) {
        p.status[0] = moves;
        p.status[1] = static_cast<int>(used);
        p.status[2] = total > moves ? __ldcg(p.src_list + moves) + 1 : static_cast<int>(used);
        p.status[3] = static_cast<int>(total);
    }
}

constexpr int kCopyThreads = 256;
constexpr int kCopyFlight = 4;

template <typename V>
__device__ inline void copy_block(V *dst, const V *src, long long n) {
    const long long step = static_cast<long long>(gridDim.x) * kCopyThreads * kCopyFlight;
    for (long long base = static_cast<long long>(blockIdx.x) * kCopyThreads * kCopyFlight + threadIdx.x; base < n;
         base += step) {
        V r[kCopyFlight];
#pragma unroll
        for (int u = 0; u < kCopyFlight; ++u)
            if (base + u * kCopyThreads < n)
                r[u] = __ldcs(src + base + u * kCopyThreads);
#pragma unroll
        for (int u = 0; u < kCopyFlight; ++u)
            if (base + u * kCopyThreads < n)
                __stcs(dst + base + u * kCopyThreads, r[u]);
    }
}

// grid.x: parts of a block, grid.y: pairs (strided), grid.z: pools.
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const CopyPagesParams p) {
    pdl_launch_dependents();
    pdl_wait();
    char *pool = p.pool[blockIdx.z];
    const long long bytes = p.block_bytes[blockIdx.z];
    const bool wide = bytes % 16 == 0 && (reinterpret_cast<uintptr_t>(pool) & 15u) == 0;
    for (int i = blockIdx.y; i < p.num_pairs; i += gridDim.y) {
        const long long src = p.pairs[2 * static_cast<long long>(i)], dst = p.pairs[2 * static_cast<long long>(i) + 1];
        if (src < 0)
            continue;  // padding
        if (src >= p.num_blocks || dst < 0 || dst >= p.num_blocks) {
            if (p.err && blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0)
                atomicOr(p.err, PA_DEVERR_BAD_PAIR);
            continue;
        }
        if (wide)
            copy_block(reinterpret_cast<uint4 *>(pool + dst * bytes), reinterpret_cast<const uint4 *>(pool + src * bytes),
                       bytes / 16);
        else
            copy_block(reinterpret_cast<uint32_t *>(pool + dst * bytes),
                       reinterpret_cast<const uint32_t *>(pool + src * bytes), bytes / 4);
    }
}

// One cluster of 16 CTAs where the device holds one (asked once a device and kernel), else of 8
// (a step of 256 rows: 18 us instead of 21).
cudaError_t launch_cluster(const void *fn, int which, void **args, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kPageThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    constexpr int kDevices = 64;
    static std::atomic<int> known[2][kDevices];  // 0: not asked yet
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    int size = dev < kDevices ? known[which][dev].load(std::memory_order_relaxed) : 8;
    if (size == 0) {
        size = 8;
        int clusters = 0;
        attr[0].val.clusterDim.x = kPageMaxCluster;
        cfg.gridDim = dim3(kPageMaxCluster);
        cfg.numAttrs = 1;
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
            cudaOccupancyMaxActiveClusters(&clusters, fn, &cfg) == cudaSuccess && clusters > 0)
            size = kPageMaxCluster;
        else
            cudaGetLastError();
        known[which][dev].store(size, std::memory_order_relaxed);
    }
    attr[0].val.clusterDim.x = size;
    cfg.gridDim = dim3(size);
    cfg.numAttrs = 2;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace

cudaError_t launch_pages_update(PagesUpdateParams p, cudaStream_t stream) {
    void *args[] = {&p};
    return launch_cluster(reinterpret_cast<const void *>(&pages_update_kernel), 0, args, stream);
}

cudaError_t launch_pages_compact(PagesCompactParams p, cudaStream_t stream) {
    void *args[] = {&p};
    return launch_cluster(reinterpret_cast<const void *>(&pages_compact_kernel), 1, args, stream);
}

cudaError_t launch_copy_pages(CopyPagesParams p, int num_sms, cudaStream_t stream) {
    long long most = 0;
    for (int i = 0; i < p.num_pools; ++i)
        most = p.block_bytes[i] > most ? p.block_bytes[i] : most;
    const long long per_cta = 16LL * kCopyThreads * kCopyFlight;
    long long gx = (most + per_cta - 1) / per_cta;
    const long long cap = static_cast<long long>(num_sms) * 8;
    if (gx > cap)
        gx = cap;
    long long gy = cap / (gx * p.num_pools);
    gy = gy < 1 ? 1 : (gy > p.num_pairs ? p.num_pairs : gy);
    if (gy > 65535)
        gy = 65535;
    void *args[] = {&p};
    return launch_dependent(reinterpret_cast<const void *>(&copy_pages_kernel),
                            dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy), p.num_pools),
                            dim3(kCopyThreads), args, 0, stream);
}

}  // namespace pa
