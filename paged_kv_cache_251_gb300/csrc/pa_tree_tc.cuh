// Tree attention on the 5th-generation tensor cores (tcgen05, accumulators in
// tensor memory), for 16-bit K/V.
//
// The T drafted tokens x G query heads of a (sequence, kv head) are the rows
// of a 128-row operand (row r = i * G + g), a tile is 128 cached tokens:
//   S = Q . K^T    M = 128 rows, N = 128 tokens, K = head_dim
//   O += P . V     M = 128 rows, N = head_dim,   K = 128 tokens
// Q, K, V come from shared memory, P from tensor memory (it overwrites S in
// place), so shared memory feeds one operand of P V only.  A thread owns a row
// of S: its softmax needs no exchange between lanes.  O accumulates in tensor
// memory over the tiles of an item; a row whose maximum grows by more than 2^8
// (fp16: 2^4) rescales its O (rare after the first tiles), a smaller growth is
// left in the exponents (larger weights, fp32 sums), which changes nothing in
// the quotient.
//
// With at most 128 rows (Units = 1) warpgroup w takes tokens 64 w .. 64 w + 63
// of every tile, with its own running state and O, merged once per item; it has
// two S buffers of 64 columns, so that the next S is made while it works.  With
// more rows (Units = 2) each warpgroup takes one of two row tiles and all 128
// tokens of a tile: one S of 128 columns each fills tensor memory (an S of 64
// tokens would cost three quarters of one of 128, as it rereads Q, and the
// tensor cores are the scarce part there).  P overwrites S, and goes to its
// product in halves of 64 tokens.
//
// P's rounding (Parts): a 16-bit output takes P rounded once to the type of V
// (the output is rounded as coarsely: against 64 bits 2.2e-3 instead of 1.7e-3 in
// bf16, 2.9e-4 instead of 2.1e-4 in fp16); an fp32 output takes hi + lo parts
// (hi = round(p), lo = round(p - hi)), two accumulating products.  Two parts for
// 16-bit outputs as well cost 234 -> 293, 72 -> 89 and 306 -> 433 us on the three
// calls measured below (fp32 outputs: 279, 87 and 455); a caller who wants them
// asks for fp32.  In fp16 weights are lifted above its small numbers (kTcLift).
//
// Work is split evenly over the CTAs, one per SM: the tiles of all pairs
// (sequence, kv head, row tile) in order, each pair counted with kTcPairCost
// tiles more for what it costs whatever its length, are cut into gridDim.x equal
// spans.  A CTA's items are the parts of pairs in its span; a pair inside one
// span is finished there, one cut by a boundary leaves a partial in each CTA it
// touches (at most two a CTA: the first and the last of its span), merged by a
// second kernel.  Partials number a few hundred however long the contexts are
// (fixed partitions of 1024 tokens wrote and read back a quarter of the K/V bytes
// at 256 rows), and no CTA is left with a long item at the end.
//
// Warp roles (384 threads, persistent over the CTA's items):
//   warp 0      K producer: the items of the span, block-table slices in
//               registers, K of each tile by TMA (one copy per block), and a
//               record of the tile's blocks for the V producer;
//   warp 1      V producer, from the records;
//   warp 2      tensor-memory allocation, the queries' TMA, S products;
//   warp 3      P V products;
//   warps 4-7, 8-11  softmax and epilogue, warpgroups 0 and 1.
//
// Masks.  A tile whose blocks are all valid and whose tokens are all committed
// needs none.  Elsewhere each row builds its 128 allowed bits from the
// committed count, its mask words and the valid blocks, and masked scores are
// replaced, never multiplied.  V rows of tokens outside the context or behind
// a bad table entry are zeroed in shared memory (their weight is 0, and 0 x
// NaN is not).  A drafted token whose V row holds an infinity or NaN must not
// reach the rows that do not attend it: its contribution is added to the
// attending rows' O by the softmax threads, and its V row is then zeroed.
// Every wait is bounded (PA_DEVERR_TIMEOUT); bad table entries are never
// dereferenced (PA_DEVERR_BAD_BLOCK).
//
// Measured (calls, with their merge; head_dim 128, block size 16): 64 sequences of
// 512 to 2048 tokens, 8 drafted, 40 heads, fp16: 234 us, 6.3 TB/s of K/V.  64 of 16
// to 8192 tokens, 16 drafted, 32 / 8 heads, bf16: 72 us, 5.2 TB/s; the CTAs' ends
// spread over 15 us.  Both are bound by HBM while every CTA works.  4 of 65536 to
// 131072 tokens, 64 drafted, 32 / 8 heads, bf16: 303 us at 2070 MHz, 5.2 TB/s and 1.0
// PFLOP/s of drafted rows (1.3 with the padding rows of the two row tiles), 332 us
// (4.7 TB/s) in a long run under the power limit: the two row tiles' chains of S,
// exponentials and P V on one tensor core, 62 % active.  With 128 drafted (512 rows,
// K/V read by two pairs of row tiles): 585 us.
#pragma once

#include "pa_decode_gqa.cuh"
#include "pa_tree.cuh"

namespace pa {

constexpr int kTcThreads = 12 * 32;
constexpr int kTcItems = 4;      // item ring
constexpr int kTcRecords = 3;    // record ring of the V producer
// valid-block masks of the last tiles: the K producer of tile t has seen all S of tile t - kSK finish, the last of
// which was issued after the softmax of the sub-unit four before it was done, so no reader lags by more than
// kSK + 1 <= 7 tiles
constexpr int kTcMeta = 8;
constexpr int kTcMaxBpt = 16;    // blocks per tile at block size 8
constexpr uint32_t kTcEnd = 0xFFFFFFFFu;
// kTcLazy: growth of a row's maximum (base 2) that rescales its O.  kTcLift: weights are
// carried 2^kTcLift times larger, numerator and denominator alike.  Above the maximum in
// use they reach 2^(kTcLazy + kTcLift).  fp16 ends at 2^16 and loses what is below 2^-25:
// lifted, that is 2^-36 of the maximum (not lifted, 2^-25: 131072 tokens behind a dominant
// one lost up to 2^-8 of the mass from the numerator alone).  bf16 has fp32's exponents.
template <typename T> constexpr float kTcLazy = 8.0f;
template <> constexpr float kTcLazy<__half> = 4.0f;
template <typename T> constexpr float kTcLift = 0.0f;
template <> constexpr float kTcLift<__half> = 11.0f;

template <int D, int Units> struct TcCfg {
    static constexpr int kHalves = D / 64;
    static constexpr int kGroup = 1024 * kHalves;      // 8 token rows
    static constexpr int kTile = 16 * kGroup;          // 128 tokens of K or V
    static constexpr int kRow = D * 2;
    static constexpr int kQ = 128 * kRow;              // one row tile of queries
    // measured on the tree over long contexts and the ragged batch: as many
    // tiles as shared memory holds beside the queries
    static constexpr int kSK = D == 64 ? 6 : (Units == 1 ? 3 : 2);
    static constexpr int kSV = D == 64 ? 6 : 3;
    static constexpr int kOffK = Units * kQ;
    static constexpr int kOffV = kOffK + kSK * kTile;
    static constexpr int kOffMisc = kOffV + kSV * kTile;
};

struct TcItem {
    int s, kvh, rt;
    int slot;  // -1: the whole context, final rows; else this CTA's partial 0 or 1
    int tile0, ntiles, t_first;
    int len, committed, drafted, end;
};

// Small shared-memory state, behind the operand buffers.
struct TcMisc {
    uint64_t kfull[6], kempty[6], vfull[6], vempty[6];
    uint64_t zfull[kTcRecords], zfree[kTcRecords];
    uint64_t ifull[kTcItems], iempty[kTcItems];
    uint64_t qfull, qempty, sfull[4], pfull[4], pvdone[4], odone, ofree, xbar, pz[2], fin, done;
    TcItem items[kTcItems];
    uint32_t meta[kTcMeta];
    uint32_t zmask[kTcRecords];
    int32_t zid[kTcRecords][kTcMaxBpt];
    // votes of the warps of a warpgroup, by tile parity: a warp may be a tile ahead of
    // another of its warpgroup, not two (the S after next waits for all of them)
    uint32_t poison[2][2][4];
    int oinit[2];
    uint32_t tmem;
    float2 ml[2][128];
};

template <int D, int Units> __host__ __device__ constexpr int tc_smem() {
    return TcCfg<D, Units>::kOffMisc + static_cast<int>(sizeof(TcMisc));
}
static_assert(tc_smem<128, 1>() <= 232448 && tc_smem<128, 2>() <= 232448 && tc_smem<64, 2>() <= 232448,
              "shared memory of one CTA");

// MMAs issued by a converged warp, one elected lane executing (`lead`): the
// operands stay warp-uniform, so the compiler keeps descriptors in uniform
// registers (a divergent lane paid about 90 cycles an MMA for moving them).
__device__ inline uint32_t elect_lane() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p;
}
// D (tensor memory) (+)= A (shared memory) . B (shared memory)
__device__ inline void tc_mma_ss(uint32_t lead, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                 int accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(lead)
        : "memory");
}
// D (tensor memory) (+)= A (tensor memory) . B (shared memory)
__device__ inline void tc_mma_ts(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                 int accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(lead)
        : "memory");
}
__device__ inline void tc_commit_lead(uint32_t lead, uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar)),
        "r"(lead)
        : "memory");
}

template <> __device__ inline void tmem_ld<32>(uint32_t taddr, float *v) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 32; ++i)
        v[i] = __uint_as_float(r[i]);
}
__device__ inline void tmem_st16(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ inline void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ inline void tma_load_3d(void *dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
        : "memory");
}

// Two 16-bit values of one word (lo element first), rounded to nearest even.
template <typename T> __device__ inline uint32_t pack2(float lo, float hi);
template <> __device__ inline uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <> __device__ inline uint32_t pack2<__half>(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <typename T> __device__ inline void unpack2(uint32_t w, float &lo, float &hi);
template <> __device__ inline void unpack2<__nv_bfloat16>(uint32_t w, float &lo, float &hi) {
    lo = __uint_as_float(w << 16), hi = __uint_as_float(w & 0xffff0000u);
}
template <> __device__ inline void unpack2<__half>(uint32_t w, float &lo, float &hi) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    lo = f.x, hi = f.y;
}
// Whether a phase has completed, without waiting (try_wait may suspend the
// thread for a while when it has not).
__device__ inline bool mbar_test_wait(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// Two fp32 operations of one instruction.
__device__ inline float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(*reinterpret_cast<uint64_t *>(&d))
        : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)),
          "l"(*reinterpret_cast<uint64_t *>(&c)));
    return d;
}
__device__ inline float2 add2(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(*reinterpret_cast<uint64_t *>(&d))
        : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)));
    return d;
}

// Whether either 16-bit value of a word is an infinity or NaN.
template <typename T> __device__ inline bool non_finite2(uint32_t w) {
    constexpr uint32_t e = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
    return (w & e) == e || ((w >> 16) & e) == e;
}

// ---------------------------------------------------------------------------
// The even split

// In tiles.  An item costs its start, its masked last tile and its epilogue beside
// its tiles: 2.8 tiles' time in a fit of the CTAs' end times on contexts of 512 to
// 2048 tokens, 3.6 on contexts of 16 to 8192.  Those take 234 and 72 us with a cost
// of 3, 238 and 72 with 4; costs of 1 and 12 lost a third and a tenth on the ragged ones.
constexpr int kTcPairCost = 3;

__device__ inline int tc_tiles(const TreeParams &p, int s) {
    const int len = max(0, min(ld_nc_i32(p.context_lens + s), p.max_len));
    return (len >> 7) + ((len & 127) != 0);
}

// Span `part` of `parts` (warp-collective): the sequence of its first unit, the
// units before that sequence, and all units.  No more spans than units: `parts`
// is cut to that, so no span is empty; a span past it has no sequence.
struct TcFind {
    int s;
    long long before, total, parts;
    __device__ long long bound(long long b) const { return total * b / parts; }  // first unit of span b
};
__device__ inline TcFind tc_find(const TreeParams &p, int pairs_per_seq, int part, int parts) {
    const int lane = threadIdx.x & 31;
    TcFind f = {p.num_seqs, 0, 0, 1};
    long long sum = 0;
#pragma unroll 4
    for (int s = lane; s < p.num_seqs; s += 32)
        sum += tc_tiles(p, s) + kTcPairCost;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
    f.total = sum * pairs_per_seq;
    f.parts = min(static_cast<long long>(parts), max(f.total, 1LL));
    if (part >= f.parts)
        return f;
    const long long u = f.bound(part);
    long long run = 0;
    for (int s0 = 0; s0 < p.num_seqs; s0 += 32) {
        const int s = s0 + lane;
        const long long mine =
            s < p.num_seqs ? static_cast<long long>(tc_tiles(p, s) + kTcPairCost) * pairs_per_seq : 0;
        long long incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o)
                incl += v;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, run + incl > u);
        if (hit) {
            const int j = __ffs(hit) - 1;
            f.s = s0 + j;
            f.before = run + __shfl_sync(0xffffffffu, incl - mine, j);
            return f;
        }
        run += __shfl_sync(0xffffffffu, incl, 31);
    }
    return f;
}

// Tiles of a pair below unit u (the pair's units start at `start`; its cost
// comes before its tiles).
__device__ inline int tc_tiles_below(long long u, long long start, int tiles) {
    const long long x = u - start - kTcPairCost;
    return static_cast<int>(x < 0 ? 0 : (x > tiles ? tiles : x));
}

// ---------------------------------------------------------------------------
// Producers

// The items of a CTA's span, in chunks whose table slice fits the registers of
// a warp (256 entries); every call gives the next chunk with its entries loaded.
struct TcChunk {
    int s = -1, kvh, rt, slot;
    int tile0, ntiles;  // of the item
    int lo, hi;         // of the chunk, in tiles of the sequence
    int first, parts;   // slots 0 and 1: the CTA that begins the pair, and how many hold a part of it
    int nblk;           // blocks of the sequence
    int tb[kMaxBpp / 32];
};
struct TcWalk {
    long long u0, u1, start;  // the span; first unit of the pair at hand
    long long total, spans;
    int s, j, tiles;
    int lo, hi, at;  // the item at hand (tiles) and the next chunk's first tile
    bool open;       // an item is being cut into chunks

    __device__ void begin(const TreeParams &p, int pairs_per_seq) {
        const TcFind f = tc_find(p, pairs_per_seq, blockIdx.x, gridDim.x);
        u0 = f.bound(blockIdx.x);
        u1 = f.bound(blockIdx.x + 1);
        total = f.total;
        spans = f.parts;
        s = f.s;
        open = false;
        j = 0;
        tiles = 0;
        start = f.before;
        if (s < p.num_seqs) {
            tiles = tc_tiles(p, s);
            j = static_cast<int>((u0 - start) / (tiles + kTcPairCost));
            start += static_cast<long long>(j) * (tiles + kTcPairCost);
        }
    }
    __device__ void next(const TreeParams &p, int pairs_per_seq, TcChunk &c) {
        const int lane = threadIdx.x & 31;
        const int bpt = 128 / p.block_size;
        c.s = -1;
        while (!open) {
            if (s >= p.num_seqs || start >= u1)
                return;
            lo = tc_tiles_below(u0, start, tiles);
            hi = tc_tiles_below(u1, start, tiles);
            // (an empty context is the item of the CTA that has its first unit)
            open = hi > lo || (tiles == 0 && start >= u0);
            if (open)
                at = lo;
            else
                step(p, pairs_per_seq);
        }
        c.s = s;
        c.kvh = j / p.row_tiles;
        c.rt = j - c.kvh * p.row_tiles;
        c.slot = hi - lo == tiles ? -1 : (lo > 0 ? 0 : 1);
        if (c.slot >= 0) {  // from the CTA of the pair's first tile to that of its last
            const long long one = start + kTcPairCost, last = one + tiles - 1;
            c.first = static_cast<int>(((one + 1) * spans - 1) / total);
            c.parts = static_cast<int>(((last + 1) * spans - 1) / total) - c.first + 1;
        }
        c.tile0 = lo;
        c.ntiles = hi - lo;
        c.lo = at;
        c.hi = min(hi, at + kMaxBpp / bpt);
        const int len = max(0, min(ld_nc_i32(p.context_lens + s), p.max_len));
        c.nblk = len / p.block_size + (len % p.block_size != 0);
        const int32_t *row = p.block_tables + static_cast<long long>(s) * p.max_blocks_per_seq + c.lo * bpt;
        const int n = min(c.hi * bpt, c.nblk) - c.lo * bpt;
#pragma unroll
        for (int i = 0; i < kMaxBpp / 32; ++i)
            c.tb[i] = lane + 32 * i < n ? ld_nc_i32(row + lane + 32 * i) : -1;
        at = c.hi;
        if (at >= hi) {
            open = false;
            step(p, pairs_per_seq);
        }
    }
    __device__ void step(const TreeParams &p, int pairs_per_seq) {
        start += tiles + kTcPairCost;
        if (++j == pairs_per_seq) {
            j = 0;
            if (++s < p.num_seqs)
                tiles = tc_tiles(p, s);
        }
    }
};

template <int D, int Units>
__device__ inline void tc_kproducer(const TreeParams &p, const CUtensorMap *tmk, char *smem, TcMisc *M) {
    using C = TcCfg<D, Units>;
    const int lane = threadIdx.x & 31;
    const int bs = p.block_size, bpt = 128 / bs;
    const uint32_t block_bytes = static_cast<uint32_t>(bs) * C::kRow;
    const uint64_t policy = policy_evict_first();
    if (lane == 0)
        prefetch_tensormap(tmk);
    const int pairs_per_seq = p.num_kv_heads * p.row_tiles;
    TcWalk walk;
    TcChunk cur, nxt;
    walk.begin(p, pairs_per_seq);
    // the merge's records of this CTA: the pairs of its partials 0 and 1, or zeros
    uint32_t cuts = 0;
    walk.next(p, pairs_per_seq, cur);
    uint32_t t = 0, k = 0;
    bool ok = true;
    for (;;) {
        if (cur.s < 0 || cur.lo == cur.tile0) {  // an item starts, or the span is done
            const int slot = static_cast<int>(k % kTcItems);
            if (!mbar_wait_bounded(&M->iempty[slot], ((k / kTcItems) & 1u) ^ 1u)) {
                ok = false;
                break;
            }
            ++k;
            if (cur.s < 0) {
                if (lane == 0) {
                    M->items[slot].end = 1;
                    mbar_arrive(&M->ifull[slot]);
                }
                __syncwarp();
                break;
            }
            if (cur.slot >= 0) {
                cuts |= 1u << cur.slot;
                if (lane == 0)
                    p.cuts[2 * blockIdx.x + cur.slot] =
                        make_int4(cur.s, cur.kvh * p.row_tiles + cur.rt, cur.first, cur.parts);
            }
            if (lane == 0) {
                const TreeSeq q = tree_seq(p, cur.s);
                if (q.bad && cur.tile0 == 0 && cur.kvh == 0 && cur.rt == 0 && p.err)
                    atomicOr(p.err, PA_DEVERR_BAD_LEN);
                TcItem it;
                it.s = cur.s;
                it.kvh = cur.kvh;
                it.rt = cur.rt;
                it.slot = cur.slot;
                it.tile0 = cur.tile0;
                it.ntiles = cur.ntiles;
                it.t_first = static_cast<int>(t);
                it.len = q.len;
                it.committed = q.len - q.drafted;
                it.drafted = q.drafted;
                it.end = 0;
                M->items[slot] = it;
                mbar_arrive(&M->ifull[slot]);
            }
            __syncwarp();
        }
        walk.next(p, pairs_per_seq, nxt);  // its entries arrive while this chunk is issued
        for (int tile = cur.lo; tile < cur.hi; ++tile, ++t) {
            const int stage = static_cast<int>(t % C::kSK), rec = static_cast<int>(t % kTcRecords);
            if (!mbar_wait_bounded(&M->kempty[stage], ((t / C::kSK) & 1u) ^ 1u) ||
                !mbar_wait_bounded(&M->zfree[rec], ((t / kTcRecords) & 1u) ^ 1u)) {
                ok = false;
                break;
            }
            // lane j takes block j of the tile: its entry is in lane (index % 32) of the slice registers
            const int b0 = (tile - cur.lo) * bpt;  // (a tile's entries share one register: bpt divides 32)
            int entry = -1;
#pragma unroll
            for (int i = 0; i < kMaxBpp / 32; ++i) {
                const int e = __shfl_sync(0xffffffffu, cur.tb[i], (b0 + lane) & 31);
                if (i == b0 >> 5)
                    entry = e;
            }
            const bool in = lane < bpt && tile * bpt + lane < cur.nblk;
            const bool mine = in && entry >= 0 && entry < p.num_blocks;
            if (in && !mine && p.err)
                atomicOr(p.err, PA_DEVERR_BAD_BLOCK);
            const uint32_t mask = __ballot_sync(0xffffffffu, mine);
            const int z = mine ? entry * p.num_kv_heads + cur.kvh : 0;
            if (lane < kTcMaxBpt)
                M->zid[rec][lane] = z;
            if (lane == 0) {
                M->meta[t % kTcMeta] = mask;
                M->zmask[rec] = mask;
                if (mask)
                    mbar_arrive_expect_tx(&M->kfull[stage], __popc(mask) * block_bytes);
                else
                    mbar_arrive(&M->kfull[stage]);
            }
            __syncwarp();
            if (mine)
                tma_load_5d(smem + C::kOffK + stage * C::kTile + lane * block_bytes, tmk, z, &M->kfull[stage], policy);
            if (lane == 0)
                mbar_arrive(&M->zfull[rec]);
            __syncwarp();
        }
        if (!ok)
            break;
        cur = nxt;
    }
    if (p.cuts && lane < 2 && !((cuts >> lane) & 1u))
        p.cuts[2 * blockIdx.x + lane] = make_int4(0, 0, 0, 0);
    // no more tiles for the V producer (after a failed wait too)
    if (lane == 0) {
        const int rec = static_cast<int>(t % kTcRecords);
        if (!mbar_wait_bounded(&M->zfree[rec], ((t / kTcRecords) & 1u) ^ 1u))
            ok = false;
        M->zmask[rec] = kTcEnd;
        mbar_arrive(&M->zfull[rec]);
    }
    if (!ok && lane == 0) {
        if (p.err)
            atomicOr(p.err, PA_DEVERR_TIMEOUT);
        const uint32_t first = t > static_cast<uint32_t>(C::kSK) ? t - C::kSK : 0;
        for (uint32_t u = first; u < t; ++u)
            (void)mbar_wait_bounded(&M->kfull[u % C::kSK], (u / C::kSK) & 1u);
    }
    __syncwarp();
}

template <int D, int Units>
__device__ inline void tc_vproducer(const TreeParams &p, const CUtensorMap *tmv, char *smem, TcMisc *M) {
    using C = TcCfg<D, Units>;
    const int lane = threadIdx.x & 31;
    const uint32_t block_bytes = static_cast<uint32_t>(p.block_size) * C::kRow;
    const uint64_t policy = policy_evict_first();
    if (lane == 0)
        prefetch_tensormap(tmv);
    bool ok = true;
    uint32_t t = 0;
    for (;; ++t) {
        const int stage = static_cast<int>(t % C::kSV), rec = static_cast<int>(t % kTcRecords);
        if (!mbar_wait_bounded(&M->zfull[rec], (t / kTcRecords) & 1u)) {
            ok = false;
            break;
        }
        const uint32_t mask = M->zmask[rec];
        if (mask == kTcEnd)
            break;
        const int z = lane < kTcMaxBpt ? M->zid[rec][lane] : 0;
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&M->zfree[rec]);  // the record is in registers
        if (!mbar_wait_bounded(&M->vempty[stage], ((t / C::kSV) & 1u) ^ 1u)) {
            ok = false;
            break;
        }
        if (lane == 0) {
            if (mask)
                mbar_arrive_expect_tx(&M->vfull[stage], __popc(mask) * block_bytes);
            else
                mbar_arrive(&M->vfull[stage]);
        }
        __syncwarp();
        if ((mask >> lane) & 1u)
            tma_load_5d(smem + C::kOffV + stage * C::kTile + lane * block_bytes, tmv, z, &M->vfull[stage], policy);
        __syncwarp();
    }
    if (!ok && lane == 0) {
        if (p.err)
            atomicOr(p.err, PA_DEVERR_TIMEOUT);
        const uint32_t first = t > static_cast<uint32_t>(C::kSV) ? t - C::kSV : 0;
        for (uint32_t u = first; u < t; ++u)
            (void)mbar_wait_bounded(&M->vfull[u % C::kSV], (u / C::kSV) & 1u);
    }
    __syncwarp();
}

// ---------------------------------------------------------------------------
// The two issuing warps.  Each is converged, one elected lane executing.  The S
// warp runs up to four sub-units ahead of the P V warp (across items too); one
// warp issuing both took about 1000 cycles a sub-unit in waits and issue alone.

// S / P buffer of warpgroup w for tile t, and the phase of that use: Units = 1
// has two a warpgroup (2 (t & 1) + w), Units = 2 one (w).
template <int Units> __device__ inline uint32_t tc_buf(uint32_t t, uint32_t w) {
    return Units == 2 ? w : 2 * (t & 1u) + w;
}
template <int Units> __device__ inline uint32_t tc_phase(uint32_t t) { return (Units == 2 ? t : t >> 1) & 1u; }
// First column of a buffer: a warpgroup's are adjacent.
__device__ inline uint32_t tc_buf_col(uint32_t b) { return (b & 1u) * 128 + (b >> 1) * 64; }

// S = Q . K^T of every tile, and the item's query rows: row tile(s) of 128
// rows = 128 / G drafted tokens x G heads; rows past the last drafted token of
// the batch read zeros, rows of the next sequence are computed and never stored.
template <typename T, int D, int Units>
__device__ inline bool tc_s_warp(const TreeParams &p, const CUtensorMap *tmq, char *smem, TcMisc *M, uint32_t tmem) {
    using C = TcCfg<D, Units>;
    // a negative scale is the sign of Q (bit 13: A negated), so the softmax
    // takes maxima of raw scores
    const uint32_t id_qk = idesc_f16<T>(128, Units == 2 ? 128 : 64, 0, 0) | (p.scale_log2 < 0.f ? 1u << 13 : 0u);
    constexpr uint32_t kHalf = 8 * C::kGroup >> 4;  // 64 tokens of a tile, in descriptor units
    const uint32_t lead = elect_lane();
    const bool lane0 = (threadIdx.x & 31) == 0;
    // descriptors of the first Q row tile and the first K stage; steps along a
    // buffer are added to the address field (16-byte units)
    const uint64_t q_desc = sdesc(smem, 16, 1024);
    const uint64_t k_desc = sdesc(smem + C::kOffK, 16, C::kGroup);
    const int G = p.num_heads / p.num_kv_heads;
    if (lane0)
        prefetch_tensormap(tmq);
    uint32_t t = 0;             // tiles so far
    uint32_t ke = 0;            // items with tiles
    uint32_t kst = 0, kph = 0;  // K stage, phase of its use
    for (uint32_t k = 0;; ++k) {
        const int slot = static_cast<int>(k % kTcItems);
        if (!mbar_wait_bounded(&M->ifull[slot], (k / kTcItems) & 1u))
            return false;
        const TcItem it = M->items[slot];
        __syncwarp();
        if (lane0)
            mbar_arrive(&M->iempty[slot]);
        if (it.end)
            return true;
        const int ntiles = it.ntiles;
        if (ntiles == 0)
            continue;
        // the Q buffer: free once the last S of the item before has finished
        if (ke > 0 && !mbar_wait_bounded(&M->qempty, (ke - 1) & 1u))
            return false;
        if (lane0) {
            mbar_arrive_expect_tx(&M->qfull, Units * C::kQ);
#pragma unroll
            for (int u = 0; u < Units; ++u) {
                const int z = it.s * p.num_draft + (it.rt * Units + u) * (128 / G);
#pragma unroll
                for (int hf = 0; hf < C::kHalves; ++hf)
                    tma_load_3d(smem + u * C::kQ + hf * (128 * 128), tmq, hf * 64, it.kvh * G, z, &M->qfull);
            }
        }
        __syncwarp();
        if (!mbar_wait_bounded(&M->qfull, ke & 1u))
            return false;
        for (int ti = 0; ti < ntiles; ++ti) {
            if (!mbar_wait_bounded(&M->kfull[kst], kph))
                return false;
#pragma unroll
            for (uint32_t e = 0; e < 2; ++e) {
                // S shares its columns with the P of their last use: two tiles ago (Units = 1), or one
                const uint32_t b = tc_buf<Units>(t, e);
                if (t >= (Units == 2 ? 1 : 2) && !mbar_wait_bounded(&M->pvdone[b], tc_phase<Units>(t) ^ 1u))
                    return false;
                tc_fence_after();
                const uint64_t qd = q_desc + (Units == 2 ? e * (C::kQ >> 4) : 0u);
                const uint64_t kd = k_desc + kst * (C::kTile >> 4) + (Units == 2 ? 0u : e * kHalf);
                const uint32_t d = tmem + tc_buf_col(b);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    tc_mma_ss(lead, d, qd + ((kk >> 2) * (128 * 128 >> 4) + (kk & 3) * 2),
                              kd + ((kk >> 2) * (1024 >> 4) + (kk & 3) * 2), id_qk, kk > 0);
                tc_commit_lead(lead, &M->sfull[b]);
            }
            ++t;
            tc_commit_lead(lead, &M->kempty[kst]);
            if (ti == ntiles - 1)
                tc_commit_lead(lead, &M->qempty);
            if (++kst == C::kSK)
                kst = 0, kph ^= 1u;
        }
        ++ke;
    }
}

// O += P . V of every tile, 64 tokens at a time.  With two row tiles the product of
// the second is left out where it has no drafted token (its buffers change hands all
// the same): four contexts of 65536 to 131072 tokens, 24 of 64 queries drafted, 280
// -> 261 us (leaving out its S as well costs full trees 2 to 5 %).
template <typename T, int D, int Parts, int Units>
__device__ inline bool tc_pv_warp(const TreeParams &p, char *smem, TcMisc *M, uint32_t tmem) {
    using C = TcCfg<D, Units>;
    constexpr uint32_t kIdPV = idesc_f16<T>(128, D, 0, 1);
    constexpr uint32_t kHalf = 8 * C::kGroup >> 4;
    const uint32_t lead = elect_lane();
    const bool lane0 = (threadIdx.x & 31) == 0;
    // V, MN-major: 64-column halves 1024 bytes apart, 8-token groups kGroup apart
    const uint64_t v_desc = sdesc(smem + C::kOffV, 1024, C::kGroup);
    const int G = p.num_heads / p.num_kv_heads;
    uint32_t t = 0, ke = 0, vst = 0, vph = 0;
    for (uint32_t k = 0;; ++k) {
        const int slot = static_cast<int>(k % kTcItems);
        if (!mbar_wait_bounded(&M->ifull[slot], (k / kTcItems) & 1u))
            return false;
        const int ntiles = M->items[slot].ntiles, end = M->items[slot].end;
        const bool both = Units == 1 || M->items[slot].drafted * G > M->items[slot].rt * 256 + 128;
        __syncwarp();
        if (lane0)
            mbar_arrive(&M->iempty[slot]);
        if (end)
            return true;
        if (ntiles == 0)
            continue;
        for (int ti = 0; ti < ntiles; ++ti, ++t) {
            // Units = 1: tokens 64 w of the tile, from warpgroup w; Units = 2: both halves
            // of row tile 0, then of row tile 1 (the warpgroups settle half a tile apart,
            // one's exponentials beside the other's products)
#pragma unroll
            for (uint32_t e = 0; e < 2 * Units; ++e) {
                const uint32_t w = Units == 2 ? e >> 1 : e, half = e & 1u;
                const uint32_t b = tc_buf<Units>(t, w);
                if (!mbar_wait_bounded(&M->pfull[Units == 2 ? 2 * half + w : b], tc_phase<Units>(t)))
                    return false;
                // O is free once the item before has been written out
                if (e == 0 && ti == 0 && ke > 0 && !mbar_wait_bounded(&M->ofree, (ke - 1) & 1u))
                    return false;
                if (e == 0 && !mbar_wait_bounded(&M->vfull[vst], vph))
                    return false;
                tc_fence_after();
                const int keep =
                    ti == 0 && (Units == 1 || half == 0) ? *reinterpret_cast<volatile int *>(&M->oinit[w]) : 1;
                const uint64_t vd = v_desc + vst * (C::kTile >> 4) + half * kHalf;
                const uint32_t o = tmem + 256 + w * D;
                const uint32_t pt = tmem + tc_buf_col(b) + (Units == 2 ? half * 64 : 0u);
                if (Units == 1 || w == 0 || both) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                        for (int part = 0; part < Parts; ++part)
                            tc_mma_ts(lead, o, pt + (kk >> 1) * 32 + part * 16 + (kk & 1) * 8,
                                      vd + kk * (2 * C::kGroup >> 4), kIdPV, (kk | part) ? 1 : keep);
                }
                if (Units == 1 || half == 1)
                    tc_commit_lead(lead, &M->pvdone[b]);
            }
            tc_commit_lead(lead, &M->vempty[vst]);
            if (++vst == C::kSV)
                vst = 0, vph ^= 1u;
        }
        tc_commit_lead(lead, &M->odone);
        ++ke;
    }
}

// ---------------------------------------------------------------------------
// Softmax and epilogue

// N columns of an accumulator row to the output (a multiple of 8).
template <int N> __device__ inline void store_cols(void *out, int dtype, long long idx, const float *v) {
    if (dtype == PA_F32) {
        float *o = static_cast<float *>(out) + idx;
        if ((reinterpret_cast<uintptr_t>(o) & 15u) == 0) {
#pragma unroll
            for (int i = 0; i < N; i += 4)
                *reinterpret_cast<float4 *>(o + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                o[i] = v[i];
        }
        return;
    }
    uint16_t *o = static_cast<uint16_t *>(out) + idx;
    uint32_t w[N / 2];
#pragma unroll
    for (int e = 0; e < N / 2; ++e)
        w[e] = dtype == PA_F16 ? pack2<__half>(v[2 * e], v[2 * e + 1]) : pack2<__nv_bfloat16>(v[2 * e], v[2 * e + 1]);
    if ((reinterpret_cast<uintptr_t>(o) & 15u) == 0) {
#pragma unroll
        for (int i = 0; i < N / 8; ++i)
            reinterpret_cast<uint4 *>(o)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else {
#pragma unroll
        for (int e = 0; e < N / 2; ++e)
            o[2 * e] = static_cast<uint16_t>(w[e]), o[2 * e + 1] = static_cast<uint16_t>(w[e] >> 16);
    }
}

// Rows of a partial: those of the row tile(s) a CTA takes.
template <int Units> __host__ __device__ inline int tc_slot_rows(int rows) {
    return rows < 128 * Units ? rows : 128 * Units;
}

template <int N> __device__ inline float max_of(const float *v) {
    float m[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
    for (int e = 4; e + 8 <= N; e += 8)
#pragma unroll
        for (int c = 0; c < 4; ++c)
            m[c] = fmaxf(fmaxf(m[c], v[e + c]), v[e + 4 + c]);
#pragma unroll
    for (int c = 0; c < 4; ++c)
        m[c] = fmaxf(m[c], v[N - 4 + c]);
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// Whether token u of the warpgroup's share of a tile has a non-finite V row:
// word q holds the votes of the warpgroup's warp q (Units = 1: two threads a token).
template <int Units> __device__ inline bool tc_poison(const uint32_t *votes, int u) {
    const uint32_t w = Units == 2 ? votes[u >> 5] : votes[u >> 5] | votes[2 + (u >> 5)];
    return (w >> (u & 31)) & 1u;
}

// The weights 2^(s sc - me) of 32 scores of this thread's row: summed, and as
// the P operand over the columns the scores came from (hi parts in the first
// 16, lo parts behind them).
template <typename T, int Parts>
__device__ inline void weights32(const float *s, float sc, float me, uint32_t addr, float2 &sum) {
    const float2 sc2 = make_float2(sc, sc), me2 = make_float2(-me, -me);
    uint32_t w[16], wl[16];
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
        float2 x = fma2(make_float2(s[e], s[e + 1]), sc2, me2);
        x.x = fast_exp2(x.x), x.y = fast_exp2(x.y);
        sum = add2(sum, x);
        w[e / 2] = pack2<T>(x.x, x.y);
        if constexpr (Parts == 2) {
            float h0, h1;
            unpack2<T>(w[e / 2], h0, h1);
            wl[e / 2] = pack2<T>(x.x - h0, x.y - h1);
        }
    }
    tmem_st16(addr, w);
    if constexpr (Parts == 2)
        tmem_st16(addr + 16, wl);
}

template <typename T, int D, int Parts, int Units>
__device__ inline bool tc_softmax(const TreeParams &p, char *smem, TcMisc *M, uint32_t tmem) {
    using C = TcCfg<D, Units>;
    constexpr int kTok = 64 * Units;  // tokens of a tile that a warpgroup takes
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int wg = (warp >> 2) - 1;
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;  // row of the 128
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t o_addr = tmem + lanes + 256 + wg * D;
    const int bs = p.block_size, bpt = 128 / bs;
    const int G = p.num_heads / p.num_kv_heads;
    const int lg = G == 1 ? 0 : (G == 2 ? 1 : (G == 4 ? 2 : 3));
    const int lbs = bs == 8 ? 3 : (bs == 16 ? 4 : 5);
    // (a scale of 0 as one too small to matter: a masked -inf times 0 would be NaN)
    const float sc = fmaxf(fabsf(p.scale_log2), 1e-30f);
    uint64_t *pzbar = Units == 1 ? &M->pz[wg] : &M->pz[0];
    // V rows of the warpgroup's tokens: 128 / kTok threads a token, each with its
    // share of the row's 16-byte chunks
    const int tk = row & (kTok - 1), vpart = row / kTok;
    constexpr int kShare = C::kHalves * 8 * kTok / 128;  // chunks of a thread: 16, 8 or 4
    const uint32_t sub_bpt = static_cast<uint32_t>(bpt) / (128 / kTok), sub_full = (1u << sub_bpt) - 1u;
    uint32_t t = 0;  // tiles so far
    uint32_t pzc = 0, ke = 0;

    auto arrive_wait = [&](uint64_t *bar, uint32_t phase) -> bool {
        __syncwarp();
        if (lane == 0)
            mbar_arrive(bar);
        return mbar_wait_bounded(bar, phase & 1u);
    };

    for (uint32_t k = 0;; ++k) {
        const int slot = static_cast<int>(k % kTcItems);
        if (!mbar_wait_bounded(&M->ifull[slot], (k / kTcItems) & 1u))
            return false;
        const TcItem it = M->items[slot];
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&M->iempty[slot]);
        if (it.end)
            return true;
        const int ntiles = it.ntiles;
        // this thread's row of the (sequence, kv head)
        const int r = (it.rt * Units + (Units == 2 ? wg : 0)) * 128 + row;
        const int i = r >> lg;
        const bool stored = i < p.num_draft, live = i < it.drafted;
        const bool warp_live = __any_sync(0xffffffffu, live);
        const long long orow =
            (static_cast<long long>(it.s) * p.num_draft + i) * p.num_heads + it.kvh * G + (r & (G - 1));
        float m = -INFINITY, l = 0.f;
        bool first = true;
        // the scores at hand, and their maximum; `ready`: loaded during the tile
        // before (Units = 1, interior tiles: nothing masked)
        float sv[kTok], top = -INFINITY;
        bool ready = false;
        for (int ti = 0; ti < ntiles; ++ti, ++t) {
            const int half = Units == 2 ? 0 : wg;
            const uint32_t buf = tc_buf<Units>(t, wg);
            const uint32_t s_addr = tmem + lanes + tc_buf_col(buf);
            const int tok0 = (it.tile0 + ti) * 128 + half * 64;
            uint64_t allow[Units];
            bool masked = false, poisoned = false;
            if (!ready) {
                const bool drafts = it.drafted > 0 && tok0 + kTok > it.committed && tok0 < it.len;
#pragma unroll
                for (int u = 0; u < Units; ++u) {
                    allow[u] = ~0ull;
                    if (tok0 + kTok > it.committed)  // (the mask's round trip overlaps the wait for S)
                        allow[u] = tree_bits64(p, it.s, it.committed, live ? it.drafted : 0, live ? i : 0,
                                               tok0 + 64 * u);
                }
                if (!mbar_wait_bounded(&M->sfull[buf], tc_phase<Units>(t)))
                    return false;
                tc_fence_after();
                if (warp_live) {
#pragma unroll
                    for (int c = 0; c < kTok; c += 32)
                        tmem_ld<32>(s_addr + c, sv + c);
                }
                // the tokens' blocks, bit e: block e of them
                const uint32_t blocks = (M->meta[t % kTcMeta] >> (half * sub_bpt)) & sub_full;
                const bool whole = blocks == sub_full;
                masked = !whole || tok0 + kTok > it.committed;
                if (masked) {
                    const int vstage = static_cast<int>(t % C::kSV);
                    const char *vhalf = smem + C::kOffV + vstage * C::kTile + half * (8 * C::kGroup);
                    char *vrow = const_cast<char *>(vhalf) + (tk >> 3) * C::kGroup + (tk & 7) * 128;
                    // chunk c of this thread's share, in an order rotated by the row (the lanes of an access then
                    // cover all banks)
                    auto chunk = [&](int c) -> char * {
                        const int at = vpart * kShare + ((c + tk) & (kShare - 1));
                        return vrow + (at >> 3) * 1024 + (at & 7) * 16;
                    };
                    if (!whole) {
#pragma unroll
                        for (int u = 0; u < Units; ++u)
#pragma unroll
                            for (int e = 0; e < 8; ++e)  // 8-token pieces
                                if (!((blocks >> ((64 * u + 8 * e) >> lbs)) & 1u))
                                    allow[u] &= ~(0xffull << (8 * e));
                    }
                    const int tok = tok0 + tk;
                    const bool valid = ((blocks >> (tk >> lbs)) & 1u) && tok < it.len;
                    uint32_t *poison = M->poison[t & 1u][wg];
                    bool drop = !valid;  // this token's V row must not be multiplied
                    if (__any_sync(0xffffffffu, drop) || drafts)
                        if (!mbar_wait_bounded(&M->vfull[vstage], (t / C::kSV) & 1u))
                            return false;
                    if (drafts) {
                        bool bad = false;
                        if (valid && tok >= it.committed) {
#pragma unroll
                            for (int c = 0; c < kShare; ++c) {
                                const uint4 x = ld_shared_v4(chunk(c));
                                bad = bad || non_finite2<T>(x.x) || non_finite2<T>(x.y) || non_finite2<T>(x.z) ||
                                      non_finite2<T>(x.w);
                            }
                        }
                        const uint32_t votes = __ballot_sync(0xffffffffu, bad);
                        if (lane == 0)
                            poison[quarter] = votes;
                        if (!arrive_wait(pzbar, pzc++))
                            return false;
                        poisoned =
                            (poison[0] | poison[1] | poison[2] | poison[3]) != 0;
                        drop = drop || tc_poison<Units>(poison, tk);
                    }
                    if (warp_live) {
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < kTok; ++e)
                            sv[e] = (allow[e >> 6] >> (e & 63)) & 1u ? sv[e] : -INFINITY;
                        top = max_of<kTok>(sv);
                    }
                    if (poisoned) {
                        // drafted tokens with non-finite V: added to the rows that attend them, before
                        // their V rows are zeroed; the row's maximum in use, and O's scale, are settled first
                        if (!first && !mbar_wait_bounded(&M->pvdone[tc_buf<Units>(t - 1, wg)], tc_phase<Units>(t - 1)))
                            return false;
                        // (with two row tiles only this warpgroup reads its O)
                        if (Units == 1 && first && ke > 0 && !mbar_wait_bounded(&M->ofree, (ke - 1) & 1u))
                            return false;
                        tc_fence_after();
                        if (warp_live) {
                            const float mx = fmaxf(m, top == -INFINITY ? -INFINITY : top * sc);
                            const float mn = first || mx > m + kTcLazy<T> ? mx : m;  // (as below)
                            const float alpha = first || (m == -INFINITY && mn != m) ? 0.f : fast_exp2(m - mn);
                            const float me = (mn == -INFINITY ? 0.f : mn) - kTcLift<T>;
                            for (int c = 0; c < D; c += 16) {
                                float o[16];
                                tmem_ld<16>(o_addr + c, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    o[e] = !first && mn == m ? o[e] : (alpha == 0.f ? 0.f : o[e] * alpha);
                                for (int u = 0; u < kTok; ++u) {
                                    if (!tc_poison<Units>(poison, u))
                                        continue;
                                    float x[2];
                                    tmem_ld<2>(s_addr + (u & ~1), x);
                                    tmem_wait_ld();
                                    const float sx = u & 1 ? x[1] : x[0];
                                    if (((Units == 2 && u >= 64 ? allow[Units - 1] : allow[0]) >> (u & 63)) & 1u) {
                                        const float pw = fast_exp2(fmaf(sx, sc, -me));
                                        const char *vr = vhalf + (u >> 3) * C::kGroup + (u & 7) * 128 + (c >> 6) * 1024;
#pragma unroll
                                        for (int e = 0; e < 16; e += 2) {
                                            const int ch = ((c & 63) + e) >> 3;  // 16-byte chunk, swizzled by the row
                                            float v0, v1;
                                            unpack2<T>(ld_shared_u32(vr + ((ch ^ (u & 7)) << 4) + (e & 7) * 2), v0, v1);
                                            o[e] = fmaf(pw, v0, o[e]);
                                            o[e + 1] = fmaf(pw, v1, o[e + 1]);
                                        }
                                    }
                                }
                                __syncwarp();
                                uint32_t w[16];
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    w[e] = __float_as_uint(o[e]);
                                tmem_st16(o_addr + c, w);
                            }
                            l *= mn == m ? 1.f : alpha;
                            m = mn;
                            tmem_wait_st();
                        }
                        if (!arrive_wait(pzbar, pzc++))  // every row has read the V rows that are zeroed now
                            return false;
                    }
                    if (drop) {
#pragma unroll
                        for (int c = 0; c < kShare; ++c)
                            *reinterpret_cast<uint4 *>(chunk(c)) = make_uint4(0, 0, 0, 0);
                    }
                    fence_async_smem();
                } else if (warp_live) {
                    tmem_wait_ld();
                    top = max_of<kTok>(sv);
                }
            }
            if (first && quarter == 0 && lane == 0)
                M->oinit[wg] = poisoned ? 1 : 0;
            ready = false;
            if (warp_live) {
                // the row's maximum (raw scores; sc >= 0)
                const float mt = top == -INFINITY ? -INFINITY : top * sc;
                // O scales with the maximum in use; it changes only when the row's
                // maximum passed it by kTcLazy
                const float mn = fmaxf(m, mt);
                const bool grow = first ? false : mn > m + kTcLazy<T>;
                if (__any_sync(0xffffffffu, grow)) {
                    // every product into this O so far is done once the last one is
                    if (!mbar_wait_bounded(&M->pvdone[tc_buf<Units>(t - 1, wg)], tc_phase<Units>(t - 1)))
                        return false;
                    tc_fence_after();
                    const float alpha = grow ? (m == -INFINITY ? 0.f : fast_exp2(m - mn)) : 1.f;
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        float o[16];
                        tmem_ld<16>(o_addr + c, o);
                        tmem_wait_ld();
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            w[e] = __float_as_uint(alpha == 1.f ? o[e] : o[e] * alpha);
                        tmem_st16(o_addr + c, w);
                    }
                    l *= alpha;
                    tmem_wait_st();
                }
                if (first || grow)
                    m = mn;
                const float me = (m == -INFINITY ? 0.f : m) - kTcLift<T>;
                // (a masked score is -inf: its weight is exactly 0)
                float2 l2 = make_float2(0.f, 0.f);
                weights32<T, Parts>(sv, sc, me, s_addr, l2);
                if constexpr (Units == 2) {
                    weights32<T, Parts>(sv + 32, sc, me, s_addr + 32, l2);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&M->pfull[wg]);  // the first half
                    weights32<T, Parts>(sv + 64, sc, me, s_addr + 64, l2);
                    weights32<T, Parts>(sv + 96, sc, me, s_addr + 96, l2);
                } else {
                    // the next tile's scores replace this one's as they are used up, when its
                    // S is there and nothing of it is masked
                    const uint32_t nbuf = tc_buf<Units>(t + 1, wg);
                    const uint32_t n_addr = tmem + lanes + tc_buf_col(nbuf);
                    if (ti + 1 < ntiles && tok0 + 128 + kTok <= it.committed)
                        ready = __all_sync(0xffffffffu, mbar_test_wait(&M->sfull[nbuf], tc_phase<Units>(t + 1))) &&
                                ((M->meta[(t + 1) % kTcMeta] >> (half * sub_bpt)) & sub_full) == sub_full;
                    if (ready) {
                        tc_fence_after();
                        tmem_ld<32>(n_addr, sv);
                    }
                    weights32<T, Parts>(sv + 32, sc, me, s_addr + 32, l2);
                    if (ready) {
                        tmem_ld<32>(n_addr + 32, sv + 32);
                        tmem_wait_ld();
                        top = max_of<kTok>(sv);
                    }
                }
                l += l2.x + l2.y;
                tmem_wait_st();
            } else if (Units == 2) {
                __syncwarp();  // (lanes may have zeroed V rows of the first half)
                if (lane == 0)
                    mbar_arrive(&M->pfull[wg]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&M->pfull[Units == 2 ? 2 + wg : buf]);
            first = false;
        }
        // ---- the item's output: final rows, or a partial per row
        const bool direct = it.slot < 0;
        if (!live)  // padding rows in a warp with live ones: they attend nothing
            m = -INFINITY, l = 0.f;
        float f0 = 1.f, f1 = 0.f, den = l, mx = m;
        if (ntiles > 0) {
            if (!mbar_wait_bounded(&M->odone, ke & 1u))
                return false;
            tc_fence_after();
            if (Units == 1) {
                // both warpgroups hold a state of the same rows: this one stores columns [wg D / 2, + D / 2)
                M->ml[wg][row] = make_float2(m, l);
                if (!arrive_wait(&M->xbar, ke))
                    return false;
                const float2 a = M->ml[0][row], b = M->ml[1][row];
                mx = fmaxf(a.x, b.x);
                // (a state that saw nothing has l == 0 and no accumulator; a NaN denominator stays)
                f0 = a.y == 0.f ? 0.f : (a.x == mx ? 1.f : fast_exp2(a.x - mx));
                f1 = b.y == 0.f ? 0.f : (b.x == mx ? 1.f : fast_exp2(b.x - mx));
                den = a.y * f0 + b.y * f1;
            }
        }
        // final rows row by row, partials column by column (the lanes' rows are
        // adjacent there: whole lines without any exchange)
        constexpr int kCols = Units == 1 ? D / 2 : D;
        const int col0 = Units == 1 ? wg * kCols : 0;
        const int rows = tc_slot_rows<Units>(p.num_draft << lg);
        const int ir = r - it.rt * Units * 128;  // row of the row tile(s)
        const long long item = static_cast<long long>(blockIdx.x) * 2 + it.slot;
        if (__any_sync(0xffffffffu, stored)) {
            if (direct) {
                const float inv = den == 0.f ? 0.f : __fdividef(1.f, den);
                f0 = den == 0.f ? 0.f : f0 * inv;  // (a factor of 0 is a row that saw nothing: 0, not 0 x garbage)
                f1 = den == 0.f ? 0.f : f1 * inv;
            }
#pragma unroll 1
            for (int c = col0; c < col0 + kCols; c += 32) {
                float o[32];
                if (ntiles > 0 && warp_live) {
                    tmem_ld<32>(tmem + lanes + 256 + (Units == 1 ? 0 : wg * D) + c, o);
                    if (Units == 1) {
                        float x[32];
                        tmem_ld<32>(tmem + lanes + 256 + D + c, x);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = (f0 == 0.f ? 0.f : o[e] * f0) + (f1 == 0.f ? 0.f : x[e] * f1);
                    } else {
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = f0 == 0.f ? 0.f : o[e] * f0;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        o[e] = 0.f;
                }
                if (direct) {
                    if (stored)
                        store_cols<32>(p.out, p.out_dtype, orow * D + c, o);
                } else if (stored && den != 0.f) {
                    float *a = p.part_acc + (item * D + c) * rows + ir;
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        a[static_cast<long long>(e) * rows] = o[e];
                }
            }
        }
        if (stored && !direct && col0 == 0)
            reinterpret_cast<float2 *>(p.part_ml)[item * rows + ir] = make_float2(mx, den);
        if (ntiles > 0) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&M->ofree);
            ++ke;
        }
    }
}

template <typename T, int D, int Parts, int Units>
__global__ void __launch_bounds__(kTcThreads, 1)
    pa_tree_tc_kernel(const TreeParams p, const __grid_constant__ CUtensorMap tmk,
                      const __grid_constant__ CUtensorMap tmv, const __grid_constant__ CUtensorMap tmq) {
    pdl_launch_dependents();
    pdl_wait();
    using C = TcCfg<D, Units>;
    extern __shared__ __align__(1024) char smem_raw[];
    char *smem = smem_raw;
    // the operand buffers need 1024-byte alignment (the swizzle); dynamic
    // shared memory starts there when a kernel has no other.  Refused otherwise.
    if (smem_addr(smem) & 1023u) {
        if (threadIdx.x == 0 && p.err)
            atomicOr(p.err, PA_DEVERR_BAD_LAUNCH);
        if (threadIdx.x < 2 && p.cuts)
            p.cuts[2 * blockIdx.x + threadIdx.x] = make_int4(0, 0, 0, 0);
        return;
    }
    TcMisc *M = reinterpret_cast<TcMisc *>(smem + C::kOffMisc);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 6; ++i) {
            mbar_init(&M->kfull[i], 1);
            mbar_init(&M->kempty[i], 1);
            mbar_init(&M->vfull[i], 1);
            mbar_init(&M->vempty[i], 1);
        }
        for (int i = 0; i < kTcRecords; ++i) {
            mbar_init(&M->zfull[i], 1);
            mbar_init(&M->zfree[i], 1);
        }
        for (int i = 0; i < kTcItems; ++i) {
            mbar_init(&M->ifull[i], 1);
            mbar_init(&M->iempty[i], 10);  // S warp, P V warp, softmax warps
        }
        mbar_init(&M->qfull, 1);
        mbar_init(&M->qempty, 1);
        for (int i = 0; i < 4; ++i) {
            mbar_init(&M->sfull[i], 1);
            mbar_init(&M->pfull[i], 4);
            mbar_init(&M->pvdone[i], 1);
        }
        for (int i = 0; i < 2; ++i)
            mbar_init(&M->pz[i], Units == 1 ? 4 : 8);
        mbar_init(&M->odone, 1);
        mbar_init(&M->ofree, 8);
        mbar_init(&M->xbar, 8);
        mbar_init(&M->fin, 1);
        mbar_init(&M->done, 9);  // softmax warps, P V warp
        fence_mbar_init();
    }
    if (warp == 2) {
        tmem_alloc(&M->tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(&M->tmem);

    // registers: 384 x 168 = 128 x 88 + 256 x 208
    bool ok = true;
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == 0) {
            tc_kproducer<D, Units>(p, &tmk, smem, M);
        } else if (warp == 1) {
            tc_vproducer<D, Units>(p, &tmv, smem, M);
        } else if (warp == 2) {
            ok = tc_s_warp<T, D, Units>(p, &tmq, smem, M, tmem);
            // every S has finished, and everyone is done with tensor memory, before it goes
            tc_commit_lead(elect_lane(), &M->fin);
            (void)mbar_wait_bounded(&M->fin, 0);
            (void)mbar_wait_bounded(&M->done, 0);
            __syncwarp();
            tc_fence_after();
            tmem_dealloc(tmem, 512);
        } else {
            ok = tc_pv_warp<T, D, Parts, Units>(p, smem, M, tmem);
            // done once its products have finished
            tc_commit_lead(elect_lane(), &M->done);
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        ok = tc_softmax<T, D, Parts, Units>(p, smem, M, tmem);
        tc_fence_before();
        __syncwarp();
        if ((threadIdx.x & 31) == 0)
            mbar_arrive(&M->done);
    }
    if (!ok && (threadIdx.x & 31) == 0 && p.err)
        atomicOr(p.err, PA_DEVERR_TIMEOUT);
}

// ---------------------------------------------------------------------------
// Merge of the pairs that a span boundary cuts: CTA f's second partial begins
// such a pair, the first partials of CTAs f + 1 .. f + P - 1 continue it.  The
// work goes back to the P CTAs (grid.x) that made the parts: the j-th takes every
// P-th column group, so each reads about as much as it wrote, in one or two round
// trips whatever P is (one CTA of a pair for all its columns, or for 16 of them
// with warps over the parts, took 14 us on the ragged batch and 22 us on
// the long contexts, against 5 and 13).  grid.y: chunks of RB rows, grid.z: the
// CTA's first or second partial.  A warp's lanes are RB rows x 32 / RB column
// groups of kTcMergeCols columns (whole lines of the column-major partials); the 8
// warps take different groups, or, when there are fewer, share the parts of one
// and meet in shared memory.
constexpr int kTcMergeThreads = 256;
constexpr int kTcMergeWarps = kTcMergeThreads / 32;
constexpr int kTcMergeCols = 8;

// log2 of RB for `rows` rows: at most 32, and no less than what a warp's columns within D leave
__host__ __device__ inline int tc_merge_log_rows(int rows, int D) {
    int l = D == 64 ? 2 : 1;
    while (l < 5 && (1 << l) < rows)
        ++l;
    return l;
}

// The state of a row over some parts: running maximum, denominator, numerators.
struct TcMergeState {
    float m = -INFINITY, den = 0.f, num[kTcMergeCols] = {};
    // x, v: a part's accumulators and (maximum, denominator); one that attended
    // nothing (v.y == 0) left no accumulators
    __device__ inline void add(float2 v, const float *x) {
        if (v.y == 0.f)
            return;
        const float mn = fmaxf(m, v.x);
        const float keep = m == -INFINITY ? 0.f : exp2f(m - mn), w = exp2f(v.x - mn);
        den = den * keep + v.y * w;
#pragma unroll
        for (int e = 0; e < kTcMergeCols; ++e)
            num[e] = num[e] * keep + x[e] * w;
        m = mn;
    }
};

template <int D, int Units>
__global__ void __launch_bounds__(kTcMergeThreads, 4) pa_tree_tc_merge_kernel(const TreeParams p) {
    pdl_launch_dependents();
    pdl_wait();
    constexpr int E = kTcMergeCols;
    __shared__ float acc[kTcMergeWarps][E + 2][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int4 cut = p.cuts[2 * blockIdx.x + blockIdx.z];
    const int parts = cut.w, first = cut.z;
    if (parts == 0)
        return;
    const int G = p.num_heads / p.num_kv_heads;
    const int all_rows = p.num_draft * G, rows = tc_slot_rows<Units>(all_rows);
    const int lrb = tc_merge_log_rows(rows, D);
    const int groups = (D / E) >> (5 - lrb);  // column groups of a warp's width
    const int r = (blockIdx.y << lrb) + (lane & ((1 << lrb) - 1));
    const int j = static_cast<int>(blockIdx.x) - first;
    const int mine = groups > j ? (groups - j + parts - 1) / parts : 0;
    if (mine == 0)
        return;
    int cw = 1;  // warps over column groups; the others over parts
    while (cw < kTcMergeWarps && cw < mine)
        cw *= 2;
    const int pw = kTcMergeWarps / cw;
    const int full = cut.y % p.row_tiles * Units * 128 + r;  // row of the (sequence, kv head)
    const bool live = r < rows && full < all_rows;
    const long long orow = (static_cast<long long>(cut.x) * p.num_draft + full / G) * p.num_heads +
                           cut.y / p.row_tiles * G + full % G;
    // (one turn when warps share parts: cw >= mine then)
    for (int k0 = 0; k0 < mine; k0 += cw) {
        const int k = k0 + warp % cw;
        const int col = (((j + k * parts) << (5 - lrb)) + (lane >> lrb)) * E;
        TcMergeState st;
        if (live && k < mine) {
            // part 0: the first CTA's partial 1; part q: partial 0 of the q-th CTA after it
            for (int q = warp / cw; q < parts; q += 2 * pw) {
                float2 v[2];
                float x[2][E];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int part = q + u * pw;
                    v[u] = make_float2(0.f, 0.f);
                    if (part < parts) {
                        const long long slot = 2LL * (first + part) + (part == 0);
                        v[u] = reinterpret_cast<const float2 *>(p.part_ml)[slot * rows + r];
                        const float *a = p.part_acc + (slot * D + col) * rows + r;
#pragma unroll
                        for (int e = 0; e < E; ++e)
                            x[u][e] = a[static_cast<long long>(e) * rows];
                    }
                }
                st.add(v[0], x[0]);
                st.add(v[1], x[1]);
            }
        }
        if (pw > 1) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                acc[warp][e][lane] = st.num[e];
            acc[warp][E][lane] = st.m;
            acc[warp][E + 1][lane] = st.den;
            __syncthreads();
            if (warp < cw)
                for (int w = warp + cw; w < kTcMergeWarps; w += cw) {
                    float x[E];
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        x[e] = acc[w][e][lane];
                    st.add(make_float2(acc[w][E][lane], acc[w][E + 1][lane]), x);
                }
        }
        if (live && k < mine && (pw == 1 || warp < cw)) {
            const float inv = st.den == 0.f ? 0.f : 1.f / st.den;
#pragma unroll
            for (int e = 0; e < E; ++e)
                st.num[e] = st.den == 0.f ? 0.f : st.num[e] * inv;
            store_cols<E>(p.out, p.out_dtype, orow * D + col, st.num);
        }
    }
}

}  // namespace pa
