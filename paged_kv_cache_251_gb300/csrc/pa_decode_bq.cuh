// Decode attention over a block-scaled 8-bit cache (one scale for each block and
// kv head, K and V apart).
//
// HBM-bound: a code byte is worth 2 G flops (G query heads a kv head).  What it needs
// beside the bytes in flight is few instructions a byte: codes go to shared memory by
// asynchronous copies of whole lines, two iterations ahead, and from there straight to the
// registers of mma fragments.
// A warp works alone on a run of 16-token tiles of one (sequence, kv head):
//
//   S = K Q^T    m16n8k16, rows = tokens, columns = heads.  The contraction runs over
//                head_dim in any order that K and Q share, so a lane's fragment of
//                four k-steps is 16 adjacent code bytes of a row: one load.
//   O^T += V^T P m16n8k16, rows = dims, columns = heads.  A lane holds 16 (8) adjacent
//                dims of four tokens, and pairs tokens by byte permutation.
//
// The tensor work is small (8 + 8 mma of 4 KB at head_dim 128), so the legacy mma
// with its register operands is the right one here: tcgen05 wants both operands of
// 16 bits in shared memory, and the codes are 8.
//
// Codes become fp16 exactly.  INT8: the low byte of 1024 + 128 + code, less 1152.  E4M3:
// converted by the hardware.
//
// The eight columns are four heads twice.  For S both halves hold the same
// queries, scaled to fp16 by a power of two a row (fp16 and bf16 queries: exact to
// 2^-40 of the row's largest element); fp32 queries as three fp16 terms, the halves'
// sums added.  For P the halves hold the weight's fp16 value and 2^11 times what that
// leaves.  Groups of eight heads fill the columns: fp32 queries are then three sets of
// them, and what fp16 leaves of a weight is a second product.  K scales multiply the scores.
// V scales multiply the weights before they are rounded, as a power of two that O is kept
// in, moved when a scale exceeds it or lies 2^4 below (down only while O stays below 2^120),
// and a factor of at most 1.  Blocks of one iteration whose scales lie further apart are
// taken one by one.  So a weight is off by 2^-22 of itself, or, being small, by 2^-39 of the
// largest so far (four heads: steps of 2^-35 below 2^7, a scale 2^-4 of the unit) or 2^-34
// (eight: of 2^-24 below 2^13).
//
// The running maximum is kept as it was until a score exceeds it by 2^8 (eight heads: 2^2),
// so a tile normally needs one vote of the warp and no shuffles.
//
// Work: the tiles of all (sequence, kv head) pieces in one line, cut evenly over all
// warps of the grid; a piece counts kPieceCost iterations more (its start and end).
// A warp whose cut lies inside a piece leaves a partial (O, max, sum) in shared
// memory, where the CTA's warps join them; what is cut between CTAs goes to
// the workspace, two partials a CTA at most, and the join kernel joins those.  Where
// every piece can have a CTA and is short (kByPieceIters), each takes one: nothing is
// cut between CTAs, nothing counted first and no second kernel.
//
// Measured, 64 x 8192 tokens of 32 / 8 heads of 128, bf16 queries (1.07 GB of codes): E4M3
// 169 us, INT8 170 us, 6.3 TB/s, 93 % of the copy bandwidth (loads alone by the same
// copies: 6.8); issue slots half busy, tensor pipe 16 %.  Fragment-shaped loads of 64-byte
// pieces, to registers or shared memory, end at 4.8 TB/s whatever the occupancy.  16
// warps an SM (128 registers, spills) 5.8 to 5.9 TB/s, three stages 6.0.  Groups of eight
// heads: 64 sequences of 1024 to 8192 tokens, 32 / 4 heads, 52 us (two sets of
// duplicated columns: 68).  A short batch is bound by a piece's start (queries, table,
// scales, first codes: about 3 us in sequence).
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "pa_block_quant.h"
#include "pa_device.cuh"
#include "pa_quant.cuh"

namespace pa {

// (2 or 6, and 4 as the least share, measure the same to 1 %.)
constexpr int kPieceCost = 3;   // iterations that a piece costs beside its own
constexpr int kMinShare = 8;    // iterations of a warp at least
// 16 a warp.  A CTA a piece and the even cut, 32 / 8 heads of 128, on the GPU: 4 contexts of 128
// tokens 6 and 10 us, of 1024 14 and 17, of 2048 23 and 19, of 8192 76 and 22; 40 of 512 14
// and 22, of 1024 22 and 25, of 2048 39 and 39, up to 2048 32 and 23.
constexpr int kByPieceIters = 64;
// log2 by which scores may exceed the running maximum, and of the weight at the running maximum (groups of
// four heads and of eight): together 15, so weights are within fp16.  What fp16 leaves of eight heads'
// weights is not scaled up, ends at 2^-25, and needs them large.
constexpr float kMaxSlack4 = 8, kMaxSlack8 = 2;
constexpr float kPTop4 = 7, kPTop8 = 13;
constexpr float kPLow = 2048;   // the low part of a weight is kept times this
constexpr float kLowScale = 1.f / 16;    // V scales this far below O's unit move it
constexpr float kNoMax = -3.4028234e38f;  // (finite: less it, a score of -inf stays -inf)

struct BqSpan {
    int start, end;  // attended tokens
    int b0;          // first block
    int tiles;       // 16-token tiles from b0's first token on
};

__device__ inline BqSpan bq_span(const DecodeBqParams &p, int L) {
    BqSpan sp;
    L = L < 0 ? 0 : (L > p.max_len ? p.max_len : L);
    sp.end = L;
    sp.start = p.window > 0 && L > p.window ? L - p.window : 0;
    sp.b0 = sp.start >> p.log_block;
    sp.tiles = L > sp.start ? (L - (sp.b0 << p.log_block) + 15) >> 4 : 0;
    return sp;
}

// 16 bytes to shared memory, asynchronously; the copies so far as a group; until all
// but the newest N groups are there.
__device__ inline void copy16(uint32_t to, const uint8_t *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ inline void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ inline void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// N words (2 or 4) of shared memory.
template <int N> __device__ inline void ld_words(uint32_t from, uint32_t *r) {
    if constexpr (N == 4)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(from)
                     : "memory");
    else
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(from) : "memory");
}

// The two codes of the low (or high) half of w as a pair of fp16.
__device__ inline uint32_t e4m3_pair(uint32_t w, bool high) {
    uint32_t y;
    if (high)
        asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, h;}" : "=r"(y) : "r"(w));
    else
        asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, l;}" : "=r"(y) : "r"(w));
    return y;
}

// Codes + 128 in the low bytes of two fp16 of 1024 + 128, to the codes, exactly.
__device__ inline uint32_t unbias(uint32_t w) {
    const __half2 bias = __half2(__half_raw{0x6480}, __half_raw{0x6480});
    const __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&w), bias);
    return *reinterpret_cast<const uint32_t *>(&x);
}

// K: four adjacent codes as two pairs of fp16.  E4M3: dims (0, 1), (2, 3).  INT8: dims
// (0, 2), (1, 3).
template <int Fmt> __device__ inline void k_pairs(uint32_t w, uint32_t &a, uint32_t &b) {
    if (Fmt == kFmtI8) {
        a = unbias((w & 0x00ff00ffu) ^ 0x64806480u);
        b = unbias(__byte_perm(w, 0, 0x4341) ^ 0x64806480u);
    } else {
        a = e4m3_pair(w, false);
        b = e4m3_pair(w, true);
    }
}
template <int Fmt> __device__ constexpr int k_dim(int pair, int i) {  // dim of pair's element i
    return Fmt == kFmtI8 ? 2 * i + pair : 2 * pair + i;
}

// V: dims 2i and 2i + 1 (i = half) of four of tokens a and b, each as the pair (a, b).
template <int Fmt> __device__ inline void v_pairs(uint32_t wa, uint32_t wb, int half, uint32_t &x, uint32_t &y) {
    if (Fmt == kFmtI8) {
        const uint32_t z = __byte_perm(wa, wb, half ? 0x7632 : 0x5410);  // a, a', b, b'
        x = unbias((z & 0x00ff00ffu) ^ 0x64806480u);
        y = unbias(__byte_perm(z, 0, 0x4341) ^ 0x64806480u);
    } else {
        const uint32_t z = __byte_perm(wa, wb, half ? 0x7362 : 0x5140);  // a, b, a', b'
        x = e4m3_pair(z, false);
        y = e4m3_pair(z, true);
    }
}

// d = a b + c (d may be c).
__device__ inline void mma16(float *d, const uint32_t *a, uint32_t b0, uint32_t b1, const float *c) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, "
        "%12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
__device__ inline uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ inline float ex2(float x) {
    float y;
    asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ inline uint32_t pack_half(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// N consecutive query elements from element `at` on, as fp32.
template <int N> __device__ inline void load_query(const DecodeBqParams &p, long long at, float *x) {
    if (p.q_dtype == PA_F32) {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            Elt<float>::unpack(*reinterpret_cast<const uint4 *>(static_cast<const float *>(p.q) + at + i), x + i);
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 8) {
            const uint4 r = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.q) + at + i);
            if (p.q_dtype == PA_F16)
                Elt<__half>::unpack(r, x + i);
            else
                Elt<__nv_bfloat16>::unpack(r, x + i);
        }
    }
}

// Units (iterations and piece costs) of a sequence's kv head.
template <int U> __device__ inline long long bq_units(const BqSpan &sp) { return (sp.tiles + U - 1) / U + kPieceCost; }

// A warp's partials in shared memory: slot 0 of a piece that began in an earlier warp,
// slot 1 of one that goes on in the next.  Behind them, for each slot:
struct BqSlot {
    int seq, head;
    int valid, ends;  // ends: (slot 0) the piece ends in this warp
};
inline __host__ __device__ constexpr int bq_part_floats(int group, int head_dim) {
    return group * head_dim + (2 * group + 3) / 4 * 4;  // (whole float4s)
}
// Of a warp: two iterations' codes, 2 KB of K and of V each.
constexpr int kBqStage = 2048;
constexpr int kBqStages = 2;
inline size_t bq_smem(int group, int head_dim) {
    return static_cast<size_t>(kDecodeBqWarps) *
           (2 * kBqStages * kBqStage + 2 * bq_part_floats(group, head_dim) * sizeof(float));
}

// (Three CTAs an SM: 168 registers a thread.  Three sets of queries of eight heads do not fit
// in those.)
template <int D, bool B8, int Fmt, int QT, bool Wide, int U>
__global__ void __launch_bounds__(kDecodeBqThreads, Wide && QT == 3 ? 2 : kDecodeBqCtas)
    decode_bq_kernel(const DecodeBqParams p) {
    constexpr int KW = D / 16;       // words of a K row a lane holds: one a k-step of S
    constexpr int KC = D / 64;       // its 16-byte chunks
    constexpr int VW = D / 32;       // words of a V row a lane holds (4 dims each)
    constexpr int MT = D / 16;       // row tiles of O^T
    constexpr int NB = B8 ? 2 : 1;   // blocks of a tile
    // column sets of queries; three terms: (hi, mid), (lo, 0), or a set each where the columns are eight heads
    constexpr int QS = QT == 1 ? 1 : (Wide ? 3 : 2);
    __shared__ long long prefix[kDecodeBqThreads + 1];
    __shared__ long long warp_units[kDecodeBqWarps];
    __shared__ BqSlot slots[kDecodeBqWarps][2];
    __shared__ int last_cta[kDecodeBqWarps];  // of a slot 1's piece
    extern __shared__ __align__(128) float4 dynamic[];  // [warps][stages] codes of K and of V, then
    // [warps][2]: [group][D] accumulators, [group][2] (max, sum)
    float *const all_parts = reinterpret_cast<float *>(dynamic) + kDecodeBqWarps * 2 * kBqStages * kBqStage / 4;
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    // the lane's place in a K tile (row g) and in a V tile (row 2t)
    const uint8_t *const k_lane = p.k_cache + lane * 16, *const v_lane = p.v_cache + lane * 16;
    // A stage is 16 lines of 128 bytes, copied as they lie in the pool (whole lines a warp
    // instruction), the 16-byte chunks of line i at their place xor i (head_dim 128; a line
    // is a row) or xor 2 i (64; two rows), modulo 8, so that no fragment's read meets a
    // bank twice.
    const uint32_t stages = smem_addr(dynamic) + warp * 2 * kBqStages * kBqStage;
    const uint32_t copy_to = stages + (lane >> 3) * 128 + ((lane & 7) ^ ((lane >> 3) * (128 / D))) * 16;
    // (lines 4 on: xor 4, of rows of 128)
    const uint32_t copy_odd = D == 128 ? copy_to ^ 64 : copy_to;
    const uint32_t k_read = stages + (D == 128 ? g * 128 + ((2 * t) ^ g) * 16
                                               : (g >> 1) * 128 + (((g & 1) * 4 + t) ^ (2 * (g >> 1))) * 16);
    const uint32_t v_read = stages + kBqStages * kBqStage +
                            (D == 128 ? 2 * t * 128 + (g ^ (2 * t)) * 16
                                      : t * 128 + ((g >> 1) ^ (2 * t)) * 16 + (g & 1) * 8);
    const float take = t < 2 ? 0.f : -kPLow, mul = t < 2 ? 1.f : kPLow;
    const int hkv = p.num_kv_heads, G = p.num_heads / hkv;
    const int wid = blockIdx.x * kDecodeBqWarps + warp, nwarps = gridDim.x * kDecodeBqWarps;

    if (lane < 2)
        slots[warp][lane].valid = 0;
    __syncwarp();
    int seq = 0, head = 0;
    BqSpan sp;
    long long units, piece = 0;  // of the piece: its units, its first one
    long long u0, u1, share;     // the warp's units
    bool works;
    if (p.by_piece) {
        // the CTA's piece, its iterations shared by the warps
        seq = blockIdx.x / hkv;
        head = blockIdx.x % hkv;
        const int L = p.context_lens[seq];
        if (L > p.max_len && p.err && tid == 0)
            atomicOr(p.err, PA_DEVERR_BAD_LEN);
        sp = bq_span(p, L);
        units = bq_units<U>(sp);
        share = (units - kPieceCost + kDecodeBqWarps - 1) / kDecodeBqWarps;
        u0 = warp == 0 ? 0 : kPieceCost + warp * share;
        u1 = min(kPieceCost + (warp + 1) * share, units);
        works = u0 < units;
    } else {
        // every thread's sequences and the units before them
        const int per = (p.num_seqs + kDecodeBqThreads - 1) / kDecodeBqThreads;
        long long mine = 0;
        for (int k = 0; k < per; ++k) {
            const int s = tid * per + k;
            if (s < p.num_seqs) {
                const int L = p.context_lens[s];
                if (L > p.max_len && p.err && blockIdx.x == 0)
                    atomicOr(p.err, PA_DEVERR_BAD_LEN);
                mine += hkv * bq_units<U>(bq_span(p, L));
            }
        }
        long long incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o)
                incl += y;
        }
        if (lane == 31)
            warp_units[warp] = incl;
        __syncthreads();
        long long before = 0, total = 0;
#pragma unroll
        for (int w = 0; w < kDecodeBqWarps; ++w) {
            if (w < warp)
                before += warp_units[w];
            total += warp_units[w];
        }
        prefix[tid] = before + incl - mine;
        if (tid == 0) {
            prefix[kDecodeBqThreads] = total;
            p.records[blockIdx.x] = make_int4(0, 0, 0, 0);
        }
        __syncthreads();

        share = (total + nwarps - 1) / nwarps;
        if (share < kMinShare + kPieceCost)
            share = kMinShare + kPieceCost;
        u0 = wid * share;
        u1 = u0 + share < total ? u0 + share : total;
        works = u0 < total;
        // the sequence that holds unit u0
        long long at = 0;  // the first unit of the sequence
        if (works) {
            int a = 0, b = kDecodeBqThreads;  // prefix[a] <= u0 < prefix[b]
            while (b - a > 1) {
                const int m = (a + b) >> 1;
                if (prefix[m] <= u0)
                    a = m;
                else
                    b = m;
            }
            seq = a * per;
            at = prefix[a];
        }
        sp = bq_span(p, p.context_lens[seq]);
        units = bq_units<U>(sp);
        while (works && at + hkv * units <= u0) {
            at += hkv * units;
            sp = bq_span(p, p.context_lens[++seq]);
            units = bq_units<U>(sp);
        }
        head = works ? static_cast<int>((u0 - at) / units) : 0;
        piece = at + head * units;
    }

    while (works) {
        // this warp's iterations of the piece
        const int iters = static_cast<int>(units) - kPieceCost;
        const long long i0 = u0 - piece - kPieceCost, i1 = u1 - piece - kPieceCost;
        const int k0 = i0 > 0 ? static_cast<int>(i0 < iters ? i0 : iters) : 0;
        const int k1 = i1 < iters ? static_cast<int>(i1 > 0 ? i1 : 0) : iters;
        const long long out_row = static_cast<long long>(seq) * p.num_heads + static_cast<long long>(head) * G;

        if (iters == 0 && u0 <= piece) {  // nothing attended
            for (int j = lane; j < G * D; j += 32)
                store_out(p.out, p.out_dtype, out_row * D + j, 0.f);
        }
        if (k0 < k1) {
            // queries as fragments; their power of two
            uint32_t qf[QS][KW][2];
            float qs[2];     // of the lane's two columns: scale * log2 e / the power of two
            {
                const int h = Wide ? g : g & 3;
                float x[KW * 4], top = 0.f;
                load_query<KW * 4>(p, (out_row + (h < G ? h : 0)) * D + t * (KW * 4), x);
#pragma unroll
                for (int c = 0; c < KW * 4; ++c) {
                    x[c] = h < G ? x[c] : 0.f;
                    top = fmaxf(top, fabsf(x[c]));
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // 2^e <= top < 2^(e + 1); queries times 2^(14 - e)
                int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
                e = e < -100 ? -100 : (e > 100 ? 100 : e);
                const float up = __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23);
                const float down =
                    __uint_as_float(static_cast<uint32_t>(e - 14 + 127) << 23) * p.scale_log2;
#pragma unroll
                for (int ks = 0; ks < KW; ++ks)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        float y[QS][2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float z = x[ks * 4 + k_dim<Fmt>(b, i)] * up;
                            if constexpr (QT == 1) {
                                y[0][i] = z;
                            } else {
                                const float hi = __half2float(__float2half_rn(z)), r = z - hi;
                                const float mid = __half2float(__float2half_rn(r));
                                if constexpr (Wide) {
                                    y[0][i] = hi;
                                    y[1][i] = mid;
                                    y[2][i] = r - mid;
                                } else {
                                    y[0][i] = g < 4 ? hi : mid;
                                    y[1][i] = g < 4 ? r - mid : 0.f;
                                }
                            }
                        }
#pragma unroll
                        for (int q = 0; q < QS; ++q)
                            qf[q][ks][b] = pack_half(y[q][0], y[q][1]);
                    }
                // columns 2t, 2t + 1 are those of lanes g = 2t, 2t + 1 (of four heads: modulo 4)
                const int from = Wide ? 2 * t : 2 * (t & 1);
                qs[0] = __shfl_sync(0xffffffffu, down, from << 2);
                qs[1] = __shfl_sync(0xffffffffu, down, (from + 1) << 2);
            }
            constexpr float kMaxSlack = Wide ? kMaxSlack8 : kMaxSlack4, kPTop = Wide ? kPTop8 : kPTop4;
            // base: the running maximum less kPTop
            float base[2] = {kNoMax, kNoMax}, l[2] = {0.f, 0.f}, o[MT][4];
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    o[i][c] = 0.f;

            // Blocks of the piece, a lane an entry, 32 at a time: those in use, with their
            // scales; the next 32, their scales on the way; and the entries after them.
            const int32_t *table = p.block_tables + static_cast<long long>(seq) * p.max_blocks;
            const int end_block = (sp.end + p.block_size - 1) >> p.log_block;
            const int tile_shift = p.log_block - 4;  // (not B8) tiles of a block: 1 or 2
            const int first = sp.b0 + (B8 ? 2 * k0 * U : (k0 * U) >> tile_shift);
            int group = 0;
            int phys, phys_next, entry_next;
            float gks, gvs, gks_next, gvs_next;
            auto entry = [&](int i) { return first + i + lane < end_block ? table[first + i + lane] : -1; };
            auto scales = [&](int &e, int i, float &a, float &b) {  // of entry e, the i-th and so on
                const bool ok = e >= 0 && e < p.num_blocks;
                if (!ok && first + i + lane < end_block && p.err)
                    atomicOr(p.err, PA_DEVERR_BAD_BLOCK);
                e = ok ? e : -1;
                const long long pair = static_cast<long long>(ok ? e : 0) * hkv + head;
                a = ok ? __ldg(p.k_scales + pair) : 0.f;
                b = ok ? __ldg(p.v_scales + pair) : 0.f;
            };
            phys = entry(0);
            phys_next = entry(32);
            entry_next = entry(64);
            scales(phys, 0, gks, gvs);
            scales(phys_next, 32, gks_next, gvs_next);

            // V scales as a power of two (of o) and a factor of the weights
            float v_unit = 1.f, v_inv = 1.f;
            auto unit_for = [](float top) {  // its exponent: 2^(e - 127) >= top
                const int e = static_cast<int>(__float_as_uint(top) >> 23) + 1;
                return e > 252 ? 252 : (e < 2 ? 2 : e);
            };
            // (lowered no further than O stays below 2^120, whatever its heads hold)
            auto set_unit = [&](float top) {
                if (!(top < INFINITY))
                    return;
                const int e = unit_for(top);
                const int from = static_cast<int>(__float_as_uint(v_unit) >> 23);
                int shift = from - e;  // log2 of O's factor
                uint32_t most = 0;  // (a head that is NaN or infinite must not hold the others)
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t x = __float_as_uint(o[i][c]) & 0x7fffffffu;
                        most = max(most, x < 0x7f800000u ? x : 1u);
                    }
                most = __reduce_max_sync(0xffffffffu, most);
                const int room = 127 + 120 - static_cast<int>(most >> 23);
                if (most >= 0x00800000u && shift > room)
                    shift = room > 0 ? room : 0;
                v_unit = __uint_as_float(static_cast<uint32_t>(from - shift) << 23);
                v_inv = __uint_as_float(static_cast<uint32_t>(254 - from + shift) << 23);
                if (most == 0)
                    return;
                // (in two steps: fp32 holds no 2^250)
                const int half = shift / 2;
                const float f0 = __uint_as_float(static_cast<uint32_t>(127 + half) << 23);
                const float f1 = __uint_as_float(static_cast<uint32_t>(127 + shift - half) << 23);
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        o[i][c] = o[i][c] * f0 * f1;
            };

            // The copies run two iterations ahead: K of one is started when K of the one two
            // before was used, V likewise.  Scales and places of the two on the way:
            struct Ahead {
                long long off[U][NB];  // the block's start in either pool, plus the tile's
                float ks[U][NB], vs[U][NB];
                unsigned ok;  // bit u * NB + b: the block is in the pool
            } now, next, after;

            // A stage's lines 0 - 7 and 8 - 15 from `lo` and `hi`.
            auto copy_stage = [&](uint32_t to, const uint8_t *lo, const uint8_t *hi) {
                copy16(copy_to + to, lo);
                copy16(copy_odd + to + 512, lo + 512);
                copy16(copy_to + to + 1024, hi);
                copy16(copy_odd + to + 1536, hi + 512);
            };
            // Halves of a stage: the blocks or halves of a tile (head_dim 128), two tiles (64; of
            // blocks of 8 each half is two pieces of 512 bytes).
            auto copy_halves = [&](uint32_t to, const uint8_t *pool, const Ahead &a) {
                if constexpr (D == 128) {
                    copy_stage(to, pool + a.off[0][0], pool + a.off[0][NB - 1] + (B8 ? 0 : 1024));
                } else {
                    copy16(copy_to + to, pool + a.off[0][0]);
                    copy16(copy_to + to + 512, pool + a.off[0][NB - 1] + (B8 ? 0 : 512));
                    copy16(copy_to + to + 1024, pool + a.off[1][0]);
                    copy16(copy_to + to + 1536, pool + a.off[1][NB - 1] + (B8 ? 0 : 512));
                }
            };
            auto copy_k = [&](int it) {  // K of iteration it; `after` gets its scales and places
                after.ok = 0;
#pragma unroll
                for (int u = 0; u < U; ++u) {
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const int tile = it * U + u;
                        const int e = sp.b0 + (B8 ? 2 * tile + b : tile >> tile_shift) - first;
                        if ((e >> 5) != group) {  // the same for the whole warp, and all of an iteration
                            ++group;
                            phys = phys_next, gks = gks_next, gvs = gvs_next;
                            phys_next = entry_next;
                            entry_next = entry(32 * (group + 2));
                            scales(phys_next, 32 * (group + 1), gks_next, gvs_next);
                        }
                        const int ph = __shfl_sync(0xffffffffu, phys, e & 31);
                        after.ks[u][b] = __shfl_sync(0xffffffffu, gks, e & 31);
                        after.vs[u][b] = __shfl_sync(0xffffffffu, gvs, e & 31);
                        const long long pair = static_cast<long long>(ph < 0 ? 0 : ph) * hkv + head;
                        long long off = (pair << p.log_block) * D;
                        if (!B8 && (tile & ((1 << tile_shift) - 1)))
                            off += 16 * D;
                        after.off[u][b] = off;
                        after.ok |= static_cast<unsigned>(ph >= 0) << (u * NB + b);
                    }
                }
                copy_halves((it & 1) * kBqStage, k_lane, after);
            };
            auto copy_v = [&](int it, const Ahead &a) {
                copy_halves((kBqStages + (it & 1)) * kBqStage, v_lane, a);
            };
            auto scale_range = [&](float &top, float &low) {  // of the present iteration's V scales but 0
                top = 0.f, low = INFINITY;
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const float vs = fabsf(now.vs[u][b]);
                        top = fmaxf(top, vs);
                        if (U * NB > 1)
                            low = fminf(low, vs > 0 ? vs : INFINITY);
                    }
            };
            auto inside = [&](int tok, bool ok) { return tok >= sp.start && tok < sp.end && ok; };

            copy_k(k0);
            now = after;
            copy_commit();
            copy_v(k0, now);
            copy_commit();
            if (k0 + 1 < k1)
                copy_k(k0 + 1);
            next = after;
            copy_commit();
            if (k0 + 1 < k1)
                copy_v(k0 + 1, next);
            copy_commit();
            {
                float top, low;
                scale_range(top, low);
                if (top > 0 && top < INFINITY) {
                    v_unit = __uint_as_float(static_cast<uint32_t>(unit_for(top)) << 23);
                    v_inv = __uint_as_float(static_cast<uint32_t>(254 - unit_for(top)) << 23);
                }
            }
            // Of an iteration whose blocks' V scales lie so far apart that one's weights would be lost
            // beside another's: the block of this pass over it; else -1.  (A second copy of the loop's
            // body for them costs all other iterations 2 to 4 %, a loop around half of it 3 to 16, this 0 to 2.)
            constexpr int kBlocks = U * NB;
            int only = -1;
            for (int it = k0; it < k1;) {
                float x[U][4];
                bool full[U];
                copy_wait<3>();  // K of this iteration is there (V, and K and V of the next, may not be)
                __syncwarp();
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    uint32_t kr[2][KW];
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int c = 0; c < KC; ++c)
                            ld_words<4>((k_read ^ (c * 16)) + (it & 1) * kBqStage + u * 1024 + r * (8 * D), kr[r] + c * 4);
#pragma unroll
                    for (int ks = 0; ks < KW; ++ks) {
                        uint32_t a[4];
                        if (ks == 0)
                            x[u][0] = x[u][1] = x[u][2] = x[u][3] = 0.f;
                        k_pairs<Fmt>(kr[0][ks], a[0], a[2]);
                        k_pairs<Fmt>(kr[1][ks], a[1], a[3]);
#pragma unroll
                        for (int q = 0; q < QS; ++q)
                            mma16(x[u], a, qf[q][ks][0], qf[q][ks][1], x[u]);
                    }
                    const float ks0 = now.ks[u][0], ks1 = now.ks[u][NB - 1];
                    if (QT == 3 && !Wide) {  // the terms' halves
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            x[u][c] += __shfl_xor_sync(0xffffffffu, x[u][c], 2);
                    }
                    x[u][0] *= ks0 * qs[0];
                    x[u][1] *= ks0 * qs[1];
                    x[u][2] *= ks1 * qs[0];
                    x[u][3] *= ks1 * qs[1];
                    // tokens outside the context, or of blocks outside the pool
                    const int tok = (sp.b0 << p.log_block) + (it * U + u) * 16;
                    const unsigned ok = now.ok >> (u * NB);
                    full[u] = tok >= sp.start && tok + 16 <= sp.end && (ok & ((1 << NB) - 1)) == (1 << NB) - 1;
                    if (!full[u]) {
                        const bool in0 = inside(tok + g, ok & 1);
                        const bool in1 = inside(tok + g + 8, ok >> (NB - 1) & 1);
                        x[u][0] = in0 ? x[u][0] : -INFINITY;
                        x[u][1] = in0 ? x[u][1] : -INFINITY;
                        x[u][2] = in1 ? x[u][2] : -INFINITY;
                        x[u][3] = in1 ? x[u][3] : -INFINITY;
                    }
                }
                // V scales: whether O's unit has to move
                float top, low;
                scale_range(top, low);
                const bool apart = kBlocks > 1 && low < top * kLowScale;
                if (apart) {
                    only = only < 0 ? 0 : only;
#pragma unroll
                    for (int i = 0; i < kBlocks; ++i)
                        top = only == i ? fabsf(now.vs[i / NB][i % NB]) : top;
                }
                const bool moves = top > v_unit || (top < v_unit * kLowScale && top > 0);
                const bool last = !apart || only == kBlocks - 1;  // pass over the iteration
                __syncwarp();  // (every lane has read this iteration's K)
                if (it + 2 < k1 && last)
                    copy_k(it + 2);
                copy_commit();
                // the running maximum moves only when it is exceeded by kMaxSlack
                float t0 = x[0][0], t1 = x[0][1];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    t0 = fmaxf(t0, fmaxf(x[u][0], x[u][2]));
                    t1 = fmaxf(t1, fmaxf(x[u][1], x[u][3]));
                }
                if (__any_sync(0xffffffffu,
                               t0 > base[0] + (kMaxSlack + kPTop) || t1 > base[1] + (kMaxSlack + kPTop))) {
#pragma unroll
                    for (int s = 4; s < 32; s <<= 1) {
                        t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, s));
                        t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, s));
                    }
                    t0 = fmaxf(t0 - kPTop, base[0]);
                    t1 = fmaxf(t1 - kPTop, base[1]);
                    const float f0 = ex2(base[0] - t0), f1 = ex2(base[1] - t1);
                    base[0] = t0;
                    base[1] = t1;
                    l[0] *= f0;
                    l[1] *= f1;
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        o[i][0] *= f0;
                        o[i][1] *= f1;
                        o[i][2] *= f0;
                        o[i][3] *= f1;
                    }
                }
                copy_wait<3>();  // V is there
                __syncwarp();
                if (moves)  // (behind the maximum: O has lost what that makes nothing of)
                    set_unit(top);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float r0 = now.vs[u][0] * v_inv, r1 = now.vs[u][NB - 1] * v_inv;
                    if (kBlocks > 1 && only >= 0) {
                        r0 = only == u * NB ? r0 : 0.f;
                        r1 = only == u * NB + NB - 1 ? r1 : 0.f;
                    }
                    // weights as the second product's operand: tokens 2t.. and 2t + 8..
                    uint32_t pf[Wide ? 2 : 1][2];
                    {
                        float e[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            e[c] = ex2(x[u][c] - base[c & 1]);
                        if (kBlocks == 1 || only <= 0) {
                            l[0] += e[0] + e[2];
                            l[1] += e[1] + e[3];
                        }
                        e[0] *= r0, e[1] *= r0, e[2] *= r1, e[3] *= r1;
                        const uint32_t h0 = pack_half(e[0], e[1]), h1 = pack_half(e[2], e[3]);
                        const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&h0));
                        const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&h1));
                        if constexpr (Wide) {  // what fp16 leaves of a weight, as a product of its own
                            pf[0][0] = transpose8x8(h0);
                            pf[0][1] = transpose8x8(h1);
                            pf[1][0] = transpose8x8(pack_half(e[0] - a.x, e[1] - a.y));
                            pf[1][1] = transpose8x8(pack_half(e[2] - b.x, e[3] - b.y));
                        } else {  // columns 0 to 3: the weight itself; 4 to 7: kPLow times what fp16 leaves of it
                            pf[0][0] = transpose8x8(pack_half(fmaf(a.x, take, e[0] * mul), fmaf(a.y, take, e[1] * mul)));
                            pf[0][1] = transpose8x8(pack_half(fmaf(b.x, take, e[2] * mul), fmaf(b.y, take, e[3] * mul)));
                        }
                    }
                    uint32_t vr[4][VW];
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        ld_words<VW>((v_read ^ ((r & 1) * (D == 128 ? 16 : 64))) + (D == 128 ? (r & 1) * 128 : 0) +
                                         (it & 1) * kBqStage + u * 1024 + (r >> 1) * (8 * D),
                                     vr[r]);
                    if (Fmt == kFmtE4M3 && !full[u]) {  // (a NaN code outside must not meet its weight of 0)
                        const int tok = (sp.b0 << p.log_block) + (it * U + u) * 16;
                        const unsigned ok = now.ok >> (u * NB);
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (!inside(tok + 2 * t + (r & 1) + 8 * (r >> 1), ok >> (B8 ? r >> 1 : 0) & 1))
#pragma unroll
                                for (int w = 0; w < VW; ++w)
                                    vr[r][w] = 0;
                    }
#pragma unroll
                    for (int w = 0; w < VW; ++w)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t a[4];
                            v_pairs<Fmt>(vr[0][w], vr[1][w], i, a[0], a[1]);
                            v_pairs<Fmt>(vr[2][w], vr[3][w], i, a[2], a[3]);
                            mma16(o[2 * w + i], a, pf[0][0], pf[0][1], o[2 * w + i]);
                            if constexpr (Wide)
                                mma16(o[2 * w + i], a, pf[1][0], pf[1][1], o[2 * w + i]);
                        }
                }
                __syncwarp();
                if (it + 2 < k1 && last)
                    copy_v(it + 2, after);
                copy_commit();
                if (!last) {
                    ++only;
                    continue;
                }
                only = -1;
                now = next;
                next = after;
                ++it;
            }

            // Of four heads: the low parts of the weights join the high ones and the lane gets one
            // head.  Of eight: the lane has two.  Dims g * D / 8 .. + D / 8.
            const bool whole = k0 == 0 && k1 == iters;
#pragma unroll
            for (int s = 4; s < 32; s <<= 1) {
                l[0] += __shfl_xor_sync(0xffffffffu, l[0], s);
                l[1] += __shfl_xor_sync(0xffffffffu, l[1], s);
            }
#pragma unroll
            for (int n = 0; n < (Wide ? 2 : 1); ++n) {
                const int h = Wide ? 2 * t + n : 2 * (t & 1) + (t >> 1);
                const float sum = (Wide ? n == 0 : t < 2) ? l[0] : l[1];
                const float top = (Wide ? n == 0 : t < 2) ? base[0] : base[1];
                float y[D / 8];
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        if constexpr (Wide) {
                            y[2 * i + c] = v_unit * o[i][2 * c + n];
                        } else {
                            const float got = __shfl_xor_sync(0xffffffffu, t < 2 ? o[i][2 * c + 1] : o[i][2 * c], 2);
                            y[2 * i + c] = v_unit * (t < 2 ? fmaf(got, 1.f / kPLow, o[i][2 * c])
                                                           : fmaf(o[i][2 * c + 1], 1.f / kPLow, got));
                        }
                    }
                if (h >= G)
                    continue;
                if (whole) {
                    const float inv = sum > 0 ? 1.f / sum : (sum == 0 ? 0.f : sum);  // (NaN stays)
                    const long long to = (out_row + h) * D + g * (D / 8);
                    if (p.out_dtype == PA_F32) {
#pragma unroll
                        for (int i = 0; i < D / 8; ++i)
                            static_cast<float *>(p.out)[to + i] = y[i] * inv;
                    } else {
#pragma unroll
                        for (int i = 0; i < D / 8; ++i)
                            store_out(p.out, p.out_dtype, to + i, y[i] * inv);
                    }
                } else {
                    float *part = all_parts + (warp * 2 + (k0 == 0)) * bq_part_floats(G, D);
                    float4 *to = reinterpret_cast<float4 *>(part + h * D + g * (D / 8));
#pragma unroll
                    for (int i = 0; i < D / 32; ++i)
                        to[i] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
                    if (g == 0)
                        reinterpret_cast<float2 *>(part + G * D)[h] = make_float2(top, sum);
                }
            }
            if (!whole && lane == 0) {
                slots[warp][k0 == 0] = BqSlot{seq, head, 1, k1 == iters};
                if (k0 == 0)
                    last_cta[warp] = static_cast<int>((piece + units - 1) / share / kDecodeBqWarps);
            }
        }
        // the next piece
        piece += units;
        if (piece >= u1)
            break;
        if (++head == hkv) {
            head = 0;
            sp = bq_span(p, p.context_lens[++seq]);
            units = bq_units<U>(sp);
        }
    }
    __syncthreads();

    // The pieces cut between the CTA's warps: warp w joins the one that begins in it, and
    // warp 0 also the one that comes from the CTA before.
    for (int from = warp == 0 ? 0 : 1; from < 2; ++from) {
        const BqSlot slot = slots[warp][from];
        if (!slot.valid)
            continue;
        int n = 1;  // warps of the piece
        bool ends = from == 0 && slot.ends;
        while (!ends && warp + n < kDecodeBqWarps) {
            ends = slots[warp + n][0].ends;
            ++n;
        }
        const bool final = from == 1 && ends;
        const int floats = bq_part_floats(G, D);
        const float *parts = all_parts + warp * 2 * floats;
        const long long out_row = static_cast<long long>(slot.seq) * p.num_heads + static_cast<long long>(slot.head) * G;
        if (!final && from == 1 && lane == 0)
            p.records[blockIdx.x] = make_int4(slot.seq, slot.head, last_cta[warp], 1);
        for (int h = 0; h < G; ++h) {
            float top = -INFINITY;
            for (int i = 0; i < n; ++i)
                top = fmaxf(top, parts[(2 * i + (i ? 0 : from)) * floats + G * D + 2 * h]);
            float sum = 0.f;
            float y[D / 32];
#pragma unroll
            for (int c = 0; c < D / 32; ++c)
                y[c] = 0.f;
            for (int i = 0; i < n; ++i) {
                const float *part = parts + (2 * i + (i ? 0 : from)) * floats;
                const float f = ex2(part[G * D + 2 * h] - top);
                sum = fmaf(f, part[G * D + 2 * h + 1], sum);
#pragma unroll
                for (int c = 0; c < D / 32; ++c)
                    y[c] = fmaf(f, part[h * D + 32 * c + lane], y[c]);
            }
            if (final) {
                const float inv = sum > 0 ? 1.f / sum : (sum == 0 ? 0.f : sum);
#pragma unroll
                for (int c = 0; c < D / 32; ++c)
                    store_out(p.out, p.out_dtype, (out_row + h) * D + 32 * c + lane, y[c] * inv);
            } else {
                const long long part = (static_cast<long long>(blockIdx.x) * 2 + from) * G + h;
#pragma unroll
                for (int c = 0; c < D / 32; ++c)
                    p.part_acc[part * D + 32 * c + lane] = y[c];
                if (lane == 0)
                    reinterpret_cast<float2 *>(p.part_ml)[part] = make_float2(top, sum);
            }
        }
    }
}

template <int D, int Fmt> const void *decode_bq_kernel(bool wide, bool f32, bool b8) {
    constexpr int U = 128 / D;
    if (wide) {
        if (f32)
            return b8 ? reinterpret_cast<const void *>(&decode_bq_kernel<D, true, Fmt, 3, true, U>)
                      : reinterpret_cast<const void *>(&decode_bq_kernel<D, false, Fmt, 3, true, U>);
        return b8 ? reinterpret_cast<const void *>(&decode_bq_kernel<D, true, Fmt, 1, true, U>)
                  : reinterpret_cast<const void *>(&decode_bq_kernel<D, false, Fmt, 1, true, U>);
    }
    if (f32)
        return b8 ? reinterpret_cast<const void *>(&decode_bq_kernel<D, true, Fmt, 3, false, U>)
                  : reinterpret_cast<const void *>(&decode_bq_kernel<D, false, Fmt, 3, false, U>);
    return b8 ? reinterpret_cast<const void *>(&decode_bq_kernel<D, true, Fmt, 1, false, U>)
              : reinterpret_cast<const void *>(&decode_bq_kernel<D, false, Fmt, 1, false, U>);
}

}  // namespace pa
