// Decode attention over a block-scaled 8-bit cache (one scale for each block and
// kv head, K and V apart).
//
// HBM-bound: a code byte is worth 2 G flops (G query heads a kv head).  What it needs
// beside the bytes in flight is few instructions a byte: codes go from global
// memory straight to the registers of mma fragments, no shared memory between.
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
// Codes become fp16 exactly: INT8 as the low byte of 1024 + 128 + code, less 1152;
// E4M3 by moving its bits (the value times 2^-8; a NaN code, which no append
// writes, reads as 480 times its sign).  So no code is infinite or NaN, and rows
// behind the context cannot spoil a product with a weight of 0.
//
// The eight columns are four heads twice.  For S both halves hold the same
// queries, scaled to fp16 by a power of two a row (fp16 and bf16 queries: exact to
// 2^-40 of the row's largest element); fp32 queries as three fp16 terms, the halves'
// sums added.  For P the halves hold the weight's fp16 value and 2^11 times what that
// leaves (22 bits together, down to 2^-50 of the largest weight).  Groups of eight
// heads take two such column sets.  K scales multiply the scores, V scales each tile's
// product, in fp32: O += v_scale * (V^T P of the block).
//
// The running maximum is kept as it was until a score exceeds it by 2^8, so a tile
// normally needs one vote of the warp and no shuffles.
//
// Work: the tiles of all (sequence, kv head) pieces in one line, cut evenly over all
// warps of the grid; a piece counts kPieceCost iterations more (its start and end).
// A warp whose cut lies inside a piece leaves a partial (O, max, sum) in shared
// memory, where the CTA's warps join them; what is cut between CTAs goes to
// the workspace, two partials a CTA at most, and the merge kernel joins those.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "pa_block_quant.h"
#include "pa_device.cuh"
#include "pa_quant.cuh"

namespace pa {

constexpr int kPieceCost = 3;   // iterations that a piece costs beside its own
constexpr int kMinShare = 8;    // iterations of a warp at least
constexpr float kMaxSlack = 8;  // log2 by which scores may exceed the running maximum
constexpr float kPTop = 7;      // weights are at most 2^(kMaxSlack + kPTop): within fp16
constexpr float kPLow = 2048;   // the low part of a weight is kept times this

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

__device__ inline uint4 ld_codes16(const uint8_t *p) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}
__device__ inline uint2 ld_codes8(const uint8_t *p) {
    uint2 r;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
    return r;
}

// Two codes, the bytes `Lo` and `Lo` + 1 of w, as a pair of fp16 (E4M3: times 2^-8).
template <int Fmt, int Lo> __device__ inline uint32_t code_pair(uint32_t w) {
    if (Fmt == kFmtI8) {
        // w's bytes are code + 128 (see code_bias)
        const uint32_t x = __byte_perm(w, 0x64646464u, Lo == 0 ? 0x4140 : 0x4342);
        const __half2 y = __hsub2(*reinterpret_cast<const __half2 *>(&x), __half2(__half_raw{0x6480}, __half_raw{0x6480}));
        return *reinterpret_cast<const uint32_t *>(&y);
    }
    const uint32_t x = __byte_perm(w, 0u, Lo == 0 ? 0x1404 : 0x3424);
    return (x & 0x80008000u) | ((x >> 1) & 0x3f803f80u);
}
template <int Fmt> __device__ inline uint32_t code_bias(uint32_t w) { return Fmt == kFmtI8 ? w ^ 0x80808080u : w; }
template <int Fmt> __host__ __device__ constexpr float code_unit() { return Fmt == kFmtI8 ? 1.f : 256.f; }

__device__ inline void mma16(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ inline void mma8(float *c, uint32_t a0, uint32_t a1, uint32_t b) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(b));
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
inline size_t bq_smem(int group, int head_dim) {
    return static_cast<size_t>(kDecodeBqWarps) * 2 * bq_part_floats(group, head_dim) * sizeof(float);
}

template <int D, bool B8, int Fmt, int QT, int NG, int U>
__global__ void __launch_bounds__(kDecodeBqThreads, NG == 1 && QT == 1 ? kDecodeBqCtas : 1)
    decode_bq_kernel(const DecodeBqParams p) {
    constexpr int KC = D / 64;       // 16-byte chunks of a K row a lane holds
    constexpr int KS = D / 16;       // k-steps of S
    constexpr int VW = D / 32;       // words of a V row a lane holds (4 dims each)
    constexpr int MT = D / 16;       // row tiles of O^T
    constexpr int NB = B8 ? 2 : 1;   // blocks of a tile
    constexpr int QS = QT == 1 ? 1 : 2;  // column sets of queries: (hi, mid), (lo, 0)
    __shared__ long long prefix[kDecodeBqThreads + 1];
    __shared__ long long warp_units[kDecodeBqWarps];
    __shared__ BqSlot slots[kDecodeBqWarps][2];
    __shared__ int last_cta[kDecodeBqWarps];  // of a slot 1's piece
    extern __shared__ float4 parts4[];        // [warps][2]: [group][D] accumulators, [group][2] (max, sum)
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int hkv = p.num_kv_heads, G = p.num_heads / hkv;
    const int wid = blockIdx.x * kDecodeBqWarps + warp, nwarps = gridDim.x * kDecodeBqWarps;

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
    if (tid == 0)
        prefix[kDecodeBqThreads] = total;
    __syncthreads();

    long long share = (total + nwarps - 1) / nwarps;
    if (share < kMinShare + kPieceCost)
        share = kMinShare + kPieceCost;
    const long long u0 = wid * share, u1 = u0 + share < total ? u0 + share : total;
    if (lane < 2)
        slots[warp][lane].valid = 0;
    if (tid == 0)
        p.records[blockIdx.x] = make_int4(0, 0, 0, 0);
    __syncwarp();

    // the sequence that holds unit u0
    int seq = 0;
    long long at = 0;  // the first unit of the sequence
    const bool works = u0 < total;
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
    BqSpan sp = bq_span(p, p.context_lens[seq]);
    long long units = bq_units<U>(sp);
    while (works && at + hkv * units <= u0) {
        at += hkv * units;
        sp = bq_span(p, p.context_lens[++seq]);
        units = bq_units<U>(sp);
    }
    int head = works ? static_cast<int>((u0 - at) / units) : 0;
    long long piece = at + head * units;  // first unit of the piece

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
            uint32_t qf[NG][QS][KS][2];
            float qs[NG][2];  // of the lane's two columns: scale * log2 e / the power of two
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                const int h = 4 * n + (g & 3);
                const bool there = h < G;
                const int elt = p.q_dtype == PA_F32 ? 4 : 2;
                const char *row = static_cast<const char *>(p.q) + (out_row + (there ? h : 0)) * D * elt;
                float top = 0.f;
                for (int c = 0; c < KC * 16; ++c) {
                    const float x = there ? fabsf(load_elt(row, p.q_dtype, (c >> 4) * 64 + t * 16 + (c & 15))) : 0.f;
                    top = fmaxf(top, x);
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // 2^e <= top < 2^(e + 1); queries times 2^(14 - e)
                int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
                e = e < -100 ? -100 : (e > 100 ? 100 : e);
                const float up = __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23);
                const float down = __uint_as_float(static_cast<uint32_t>(e - 14 + 127) << 23) * p.scale_log2;
                // the lane's columns 2t, 2t + 1 are the heads of lanes g = 2t, 2t + 1 (modulo 4)
                qs[n][0] = __shfl_sync(0xffffffffu, down, (2 * (t & 1)) << 2);
                qs[n][1] = __shfl_sync(0xffffffffu, down, (2 * (t & 1) + 1) << 2);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const int d = (ks >> 2) * 64 + t * 16 + (ks & 3) * 4 + 2 * b;
                        float x[2], y[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            x[i] = there ? load_elt(row, p.q_dtype, d + i) * up : 0.f;
                            y[i] = 0.f;
                            if (QT == 3) {
                                const float hi = __half2float(__float2half_rn(x[i]));
                                const float r = x[i] - hi;
                                const float mid = __half2float(__float2half_rn(r));
                                x[i] = g < 4 ? hi : mid;
                                y[i] = g < 4 ? r - mid : 0.f;
                            }
                        }
                        qf[n][0][ks][b] = pack_half(x[0], x[1]);
                        if (QT == 3)
                            qf[n][QS - 1][ks][b] = pack_half(y[0], y[1]);
                    }
            }
            float m[NG][2], l[NG][2], o[NG][MT][4];
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                m[n][0] = m[n][1] = -INFINITY;
                l[n][0] = l[n][1] = 0.f;
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        o[n][i][c] = 0.f;
            }

            // blocks of the piece, 32 table entries at a time (and the next 32)
            const int32_t *table = p.block_tables + static_cast<long long>(seq) * p.max_blocks;
            const int end_block = (sp.end + p.block_size - 1) >> p.log_block;
            const int tile_shift = p.log_block - 4;  // (not B8) tiles of a block: 1 or 2
            const int first = sp.b0 + (B8 ? 2 * k0 * U : (k0 * U) >> tile_shift);
            int group = 0;
            int entries = first + lane < end_block ? table[first + lane] : -1;
            int entries_next = first + 32 + lane < end_block ? table[first + 32 + lane] : -1;

            uint4 kr[U][2][KC];
            uint32_t vr[U][4][VW];
            long long off[U][NB];       // of the next tiles: bytes from the pool's start
            float ks_next[U][NB], vs_next[U][NB];
            unsigned ok_next = 0;       // bit u * NB + b: the block is in the pool

            auto locate = [&](int it) {  // the tiles of iteration it
                ok_next = 0;
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const int tile = it * U + u;
                        const int e = sp.b0 + (B8 ? 2 * tile + b : tile >> tile_shift) - first;
                        if ((e >> 5) != group) {  // the same for the whole warp
                            ++group;
                            entries = entries_next;
                            const int x = first + 32 * (group + 1) + lane;
                            entries_next = x < end_block ? table[x] : -1;
                        }
                        const int phys = __shfl_sync(0xffffffffu, entries, e & 31);
                        const bool ok = phys >= 0 && phys < p.num_blocks;
                        if (!ok && first + e < end_block && lane == 0 && p.err)
                            atomicOr(p.err, PA_DEVERR_BAD_BLOCK);
                        const long long pair = static_cast<long long>(ok ? phys : 0) * hkv + head;
                        ks_next[u][b] = __ldg(p.k_scales + pair);
                        vs_next[u][b] = __ldg(p.v_scales + pair);
                        off[u][b] = (pair << p.log_block) * D;
                        if (!B8 && (tile & ((1 << tile_shift) - 1)))
                            off[u][b] += 16 * D;
                        ok_next |= static_cast<unsigned>(ok) << (u * NB + b);
                    }
            };
            auto load_k = [&]() {
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const uint8_t *row = p.k_cache + off[u][B8 ? r : 0] + (g + (B8 ? 0 : 8 * r)) * D + t * 16;
#pragma unroll
                        for (int c = 0; c < KC; ++c)
                            kr[u][r][c] = ld_codes16(row + c * 64);
                    }
            };
            auto load_v = [&]() {  // tokens 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const uint8_t *row = p.v_cache + off[u][B8 ? r >> 1 : 0] +
                                             (2 * t + (r & 1) + (B8 ? 0 : 8 * (r >> 1))) * D + g * (D / 8);
                        if constexpr (VW == 4) {
                            const uint4 x = ld_codes16(row);
                            vr[u][r][0] = x.x, vr[u][r][1] = x.y, vr[u][r][2] = x.z, vr[u][r][3] = x.w;
                        } else {
                            const uint2 x = ld_codes8(row);
                            vr[u][r][0] = x.x, vr[u][r][1] = x.y;
                        }
                    }
            };

            locate(k0);
            load_k();
            load_v();
            for (int it = k0; it < k1; ++it) {
                const unsigned ok = ok_next;
                float vs[U][NB];
                float x[U][NG][4];
#pragma unroll
                for (int u = 0; u < U; ++u) {
#pragma unroll
                    for (int n = 0; n < NG; ++n)
                        x[u][n][0] = x[u][n][1] = x[u][n][2] = x[u][n][3] = 0.f;
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        const uint4 r0 = kr[u][0][ks >> 2], r1 = kr[u][1][ks >> 2];
                        const uint32_t w0 = code_bias<Fmt>((&r0.x)[ks & 3]), w1 = code_bias<Fmt>((&r1.x)[ks & 3]);
                        const uint32_t a[4] = {code_pair<Fmt, 0>(w0), code_pair<Fmt, 0>(w1), code_pair<Fmt, 2>(w0),
                                               code_pair<Fmt, 2>(w1)};
#pragma unroll
                        for (int n = 0; n < NG; ++n)
#pragma unroll
                            for (int q = 0; q < QS; ++q)
                                mma16(x[u][n], a, qf[n][q][ks][0], qf[n][q][ks][1]);
                    }
                    float ks0 = ks_next[u][0] * code_unit<Fmt>(), ks1 = B8 ? ks_next[u][NB - 1] * code_unit<Fmt>() : ks0;
#pragma unroll
                    for (int b = 0; b < NB; ++b)
                        // (a block outside the pool stands for block 0, whose scale may be anything)
                        vs[u][b] = (ok >> (u * NB + b) & 1) ? vs_next[u][b] * code_unit<Fmt>() : 0.f;
                    const int tok = (sp.b0 << p.log_block) + (it * U + u) * 16 + g;
                    const bool in0 = tok >= sp.start && tok < sp.end && (ok >> (u * NB) & 1);
                    const bool in1 = tok + 8 >= sp.start && tok + 8 < sp.end && (ok >> (u * NB + NB - 1) & 1);
#pragma unroll
                    for (int n = 0; n < NG; ++n) {
                        if (QT == 3) {  // the terms' halves
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                x[u][n][c] += __shfl_xor_sync(0xffffffffu, x[u][n][c], 2);
                        }
                        x[u][n][0] = in0 ? x[u][n][0] * (ks0 * qs[n][0]) : -INFINITY;
                        x[u][n][1] = in0 ? x[u][n][1] * (ks0 * qs[n][1]) : -INFINITY;
                        x[u][n][2] = in1 ? x[u][n][2] * (ks1 * qs[n][0]) : -INFINITY;
                        x[u][n][3] = in1 ? x[u][n][3] * (ks1 * qs[n][1]) : -INFINITY;
                    }
                }
                if (it + 1 < k1) {
                    locate(it + 1);
                    load_k();
                }
                // the running maximum moves only when it is exceeded by kMaxSlack
#pragma unroll
                for (int n = 0; n < NG; ++n) {
                    float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        t0 = fmaxf(t0, fmaxf(x[u][n][0], x[u][n][2]));
                        t1 = fmaxf(t1, fmaxf(x[u][n][1], x[u][n][3]));
                    }
                    if (__any_sync(0xffffffffu, t0 > m[n][0] + kMaxSlack || t1 > m[n][1] + kMaxSlack)) {
#pragma unroll
                        for (int s = 4; s < 32; s <<= 1) {
                            t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, s));
                            t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, s));
                        }
                        t0 = fmaxf(t0, m[n][0]);
                        t1 = fmaxf(t1, m[n][1]);
                        const float f0 = t0 == -INFINITY ? 1.f : ex2(m[n][0] - t0);
                        const float f1 = t1 == -INFINITY ? 1.f : ex2(m[n][1] - t1);
                        m[n][0] = t0;
                        m[n][1] = t1;
                        l[n][0] *= f0;
                        l[n][1] *= f1;
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            o[n][i][0] *= f0;
                            o[n][i][1] *= f1;
                            o[n][i][2] *= f0;
                            o[n][i][3] *= f1;
                        }
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    uint32_t pf[NG][2];  // weights as the second product's operand: tokens 2t.. and 2t + 8..
#pragma unroll
                    for (int n = 0; n < NG; ++n) {
                        // (no token yet: every weight of the column is exp2(-inf) = 0)
                        const float m0 = m[n][0] == -INFINITY ? 0.f : m[n][0] - kPTop;
                        const float m1 = m[n][1] == -INFINITY ? 0.f : m[n][1] - kPTop;
                        const float e0 = ex2(x[u][n][0] - m0), e1 = ex2(x[u][n][1] - m1);
                        const float e2 = ex2(x[u][n][2] - m0), e3 = ex2(x[u][n][3] - m1);
                        l[n][0] += e0 + e2;
                        l[n][1] += e1 + e3;
                        uint32_t h0 = pack_half(e0, e1), h1 = pack_half(e2, e3);
                        if (t >= 2) {
                            const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&h0));
                            const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&h1));
                            h0 = pack_half((e0 - a.x) * kPLow, (e1 - a.y) * kPLow);
                            h1 = pack_half((e2 - b.x) * kPLow, (e3 - b.y) * kPLow);
                        }
                        pf[n][0] = transpose8x8(h0);
                        pf[n][1] = transpose8x8(h1);
                    }
#pragma unroll
                    for (int w = 0; w < VW; ++w) {
                        // [token pair][dims 0 and 1, dims 2 and 3]: bytes (a, b, a, b)
                        uint32_t z[2][2];
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            z[r][0] = code_bias<Fmt>(__byte_perm(vr[u][2 * r][w], vr[u][2 * r + 1][w], 0x5140));
                            z[r][1] = code_bias<Fmt>(__byte_perm(vr[u][2 * r][w], vr[u][2 * r + 1][w], 0x7362));
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t a[4] = {code_pair<Fmt, 0>(z[0][i]), code_pair<Fmt, 2>(z[0][i]),
                                                   code_pair<Fmt, 0>(z[1][i]), code_pair<Fmt, 2>(z[1][i])};
#pragma unroll
                            for (int n = 0; n < NG; ++n) {
                                float *acc = o[n][2 * w + i];
                                float y[4] = {0.f, 0.f, 0.f, 0.f};
                                if constexpr (B8) {
                                    float y1[4] = {0.f, 0.f, 0.f, 0.f};
                                    mma8(y, a[0], a[1], pf[n][0]);
                                    mma8(y1, a[2], a[3], pf[n][1]);
#pragma unroll
                                    for (int c = 0; c < 4; ++c)
                                        acc[c] = fmaf(vs[u][NB - 1], y1[c], acc[c]);
                                } else {
                                    mma16(y, a, pf[n][0], pf[n][1]);
                                }
#pragma unroll
                                for (int c = 0; c < 4; ++c)
                                    acc[c] = fmaf(vs[u][0], y[c], acc[c]);
                            }
                        }
                    }
                }
                if (it + 1 < k1)
                    load_v();
            }

            // The low parts of the weights join the high ones: the lane gets one head,
            // dims g * D / 8 .. + D / 8.
            const bool whole = k0 == 0 && k1 == iters;
            const int hc = 2 * (t & 1) + (t >> 1);  // the lane's head of each four
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                float lsum[2] = {l[n][0], l[n][1]};
#pragma unroll
                for (int s = 4; s < 32; s <<= 1) {
                    lsum[0] += __shfl_xor_sync(0xffffffffu, lsum[0], s);
                    lsum[1] += __shfl_xor_sync(0xffffffffu, lsum[1], s);
                }
                const float sum = t < 2 ? lsum[0] : lsum[1];
                const float top = t < 2 ? m[n][0] : m[n][1];
                float y[D / 8];
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float send = t < 2 ? o[n][i][2 * c + 1] : o[n][i][2 * c];
                        const float got = __shfl_xor_sync(0xffffffffu, send, 2);
                        y[2 * i + c] = t < 2 ? fmaf(got, 1.f / kPLow, o[n][i][2 * c])
                                             : fmaf(o[n][i][2 * c + 1], 1.f / kPLow, got);
                    }
                const int h = 4 * n + hc;
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
                    float *part = reinterpret_cast<float *>(parts4) + (warp * 2 + (k0 == 0)) * bq_part_floats(G, D);
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
        const float *parts = reinterpret_cast<const float *>(parts4) + warp * 2 * floats;
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
                const float f = top == -INFINITY ? 1.f : ex2(part[G * D + 2 * h] - top);
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
            return b8 ? reinterpret_cast<const void *>(&decode_bq_kernel<D, true, Fmt, 3, 2, U>)
                      : reinterpret_cast<const void *>(&decode_bq_kernel<D, false, Fmt, 3, 2, U>);
        return b8 ? reinterpret_cast<const void *>(&decode_bq_kernel<D, true, Fmt, 1, 2, U>)
                  : reinterpret_cast<const void *>(&decode_bq_kernel<D, false, Fmt, 1, 2, U>);
    }
    if (f32)
        return b8 ? reinterpret_cast<const void *>(&decode_bq_kernel<D, true, Fmt, 3, 1, U>)
                  : reinterpret_cast<const void *>(&decode_bq_kernel<D, false, Fmt, 3, 1, U>);
    return b8 ? reinterpret_cast<const void *>(&decode_bq_kernel<D, true, Fmt, 1, 1, U>)
              : reinterpret_cast<const void *>(&decode_bq_kernel<D, false, Fmt, 1, 1, U>);
}

}  // namespace pa
