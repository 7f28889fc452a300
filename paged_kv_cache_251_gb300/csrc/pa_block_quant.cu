// Append to a block-scaled 8-bit cache: every (block, kv head) of K and of V has
// one fp32 scale, and an element is code * scale.
//
//   scale = amax / Q over the rows that the call writes to the block (Q = 127 INT8,
//           448 E4M3; one IEEE division); at least the scale of before, unless the
//           call writes row 0, which starts the block anew
//   code  = x / scale (IEEE) rounded to the nearest code, ties to even, saturating
// and where the scale grew, the rows of before are coded again: code * old scale
// (rounded to fp32) / scale, rounded the same way.
// ("KV Cache与长上下文管理": the cache stored in 8 bits halves its size.)
//
// A (block, kv head) of K or V is a unit, taken whole by one warp, whichever of its rows
// the call writes: the scale needs them all.  A block's tokens may stand anywhere in the
// call.  A few tokens (a decode step): every warp looks at all slots.  Many: a first kernel
// writes each slot's token into a map of the pool's slots, which needs no clearing: an entry
// is believed only if the token that it names has that very slot.  A second lists the
// blocks, each by the window of tokens that holds its lowest written row, and a third goes over
// all units of the list, evenly, the next unit's tokens on their way meanwhile.
//
// HBM-bound: a row is read, its codes written.  A lane takes eight elements of a row, and
// holds its share of the unit's rows in registers, all loads in flight together, between the
// scale and the codes (fp32 rows of blocks of 32 at head_dim 128 are read twice).
// Divisions: the correctly rounded quotient from the correctly rounded reciprocal by two
// residual corrections (Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990), where no step can leave the normal range; else the plain one.
//
// Measured on the GPU: 24000 tokens of ragged prompts, 8 kv heads of 128, bf16 to E4M3: 28 us,
// 5.4 TB/s (floor 22 us; the map and the list 5); blocks looked for by the CTAs that store them
// 33 us, by their warps 45; plain divisions and rows read twice 72.  64 tokens of a
// decode step: 3.3 us.
#include <cuda_runtime.h>

#include "pa_block_quant.h"
#include "pa_device.cuh"
#include "pa_f32x2.cuh"
#include "pa_internal.h"
#include "pa_quant.cuh"

namespace pa {

namespace {

constexpr int kBqThreads = 256;
constexpr int kBqWarps = kBqThreads / 32;
// Tokens of a warp that lists blocks: with 8, 4, 2 the prompts above take 27.9, 28.1, 29.1 us,
// 1024 tokens of as many blocks 17.4, 14.4, 12.6.
constexpr int kListWindow = 4;

// Which token has a slot; no blocks listed yet.
__global__ void __launch_bounds__(kBqThreads) map_tokens_kernel(const AppendBqParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int i = blockIdx.x * kBqThreads + threadIdx.x;
    if (i == 0)
        *p.listed = 0;
    if (i < p.num_tokens) {
        const long long slot = p.slots[i];
        if (slot >= 0 && slot < p.pool_slots)
            p.token_of[slot] = i;
    }
}

// Eight elements of a row, as they are.
template <typename T> struct Raw {
    uint4 r[sizeof(T) / 2];
    __device__ inline void load(const T *p) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
            r[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
    }
    __device__ inline void get(float *f) const {
        constexpr int E = 16 / sizeof(T);
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
            Elt<T>::unpack(r[i], f + i * E);
    }
    // The largest magnitude so far, as bits (which order magnitudes, infinities and NaN
    // above all numbers): of two halves for 16-bit types.
    __device__ inline uint32_t peak(uint32_t top) const {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) {
            const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
                top = sizeof(T) == 4 ? max(top, w[k] & 0x7fffffffu) : __vmaxu2(top, w[k] & 0x7fff7fffu);
        }
        return top;
    }
};
// Of a warp's peaks: the largest magnitude.
template <typename T> __device__ inline float peak_value(uint32_t top) {
    if (sizeof(T) == 2)
        top = max(top >> 16, top & 0xffffu);
    top = __reduce_max_sync(0xffffffffu, top);
    if (sizeof(T) == 4)
        return __uint_as_float(top);
    return Elt<T>::kCode == PA_F16 ? __half2float(__ushort_as_half(static_cast<unsigned short>(top)))
                                   : __uint_as_float(top << 16);
}

// Codes of eight elements.  Plain: any elements and scale.  Otherwise all finite, the
// scale in [2^-60, 2^100], magnitudes up to about Q scales: a quotient's corrections
// then lose nothing, unless it is below 2^-40 and coded 0 whatever they do.
template <int Fmt, bool Plain> __device__ inline uint2 code8(const float *f, float scale, float inv) {
    float y[8];
    if (Plain) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            y[e] = __fdiv_rn(f[e], scale);
            y[e] = y[e] != y[e] ? 0.f : y[e];
        }
    } else {
        const F2 s = f2(-scale, -scale), r = f2(inv, inv);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const F2 x = f2(f[e], f[e + 1]);
            F2 q = f2_mul(x, r);
            q = f2_fma(f2_fma(q, s, x), r, q);
            q = f2_fma(f2_fma(q, s, x), r, q);
            const float2 z = f2_get(q);
            y[e] = z.x;
            y[e + 1] = z.y;
        }
    }
    uint32_t w[2];
    if (Fmt == kFmtI8) {
        // clamped, then rounded to the low bits of 1.5 * 2^23
        uint32_t b[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            b[e] = __float_as_uint(__fadd_rn(fminf(fmaxf(y[e], -127.f), 127.f), 12582912.f));
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[i] = __byte_perm(__byte_perm(b[4 * i], b[4 * i + 1], 0x0040), __byte_perm(b[4 * i + 2], b[4 * i + 3], 0x0040),
                               0x5410);
    } else {
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            h[i] = __nv_cvt_float2_to_fp8x2(make_float2(y[2 * i], y[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
        w[0] = h[0] | h[1] << 16;
        w[1] = h[2] | h[3] << 16;
    }
    return make_uint2(w[0], w[1]);
}

// One kv head of K or V (unit u) of a block, by a warp.  token: lane r's is row r's, -1 where
// the call does not write it; written: those rows.
template <typename T, int D, int BS, int Fmt>
__device__ inline void store_unit(const AppendBqParams &p, long long block, int token, unsigned written, int u, int lane) {
    constexpr int kRowLanes = D / 8;
    constexpr int kRows = 32 / kRowLanes;  // rows of a warp at once
    constexpr int kIters = BS / kRows;
    constexpr bool kHeld = kIters * static_cast<int>(sizeof(T)) <= 32;  // 64 registers
    const int r_lane = lane / kRowLanes, c = lane % kRowLanes * 8;
    const long long stride = static_cast<long long>(p.num_kv_heads) * D;
    const unsigned mine_written = written >> r_lane;  // bit r * kRows: of the lane's r-th row
    const bool is_v = u >= p.num_kv_heads;
    const int h = is_v ? u - p.num_kv_heads : u;
    const T *x = static_cast<const T *>(is_v ? p.v : p.k) + static_cast<long long>(h) * D + c;
    const long long tile = block * p.num_kv_heads + h;
    float *scale_at = (is_v ? p.v_scales : p.k_scales) + tile;
    uint8_t *codes = (is_v ? p.v_cache : p.k_cache) + tile * BS * D + r_lane * D + c;
    const bool fresh = written & 1;
    const float old = __shfl_sync(0xffffffffu, lane == 0 ? *scale_at : 0.f, 0);  // (lane 0 writes it too)
    Raw<T> raw[kHeld ? kIters : 1];
    uint32_t top = 0;
    if (kHeld) {
#pragma unroll
        for (int r = 0; r < kIters; ++r) {
            const int j = __shfl_sync(0xffffffffu, token, r * kRows + r_lane);
            if (j >= 0)
                raw[r].load(x + j * stride);
        }
#pragma unroll
        for (int r = 0; r < kIters; ++r)
            if (mine_written >> (r * kRows) & 1)
                top = raw[r].peak(top);
    } else {
#pragma unroll 4
        for (int r = 0; r < kIters; ++r) {
            const int j = __shfl_sync(0xffffffffu, token, r * kRows + r_lane);
            if (j >= 0) {
                raw[0].load(x + j * stride);
                top = raw[0].peak(top);
            }
        }
    }
    float amax = peak_value<T>(top);
    const bool plain_rows = !(amax < INFINITY);
    if (plain_rows) {  // infinities and NaN do not count
        amax = 0.f;
        for (int r = 0; r < kIters; ++r) {
            const int j = __shfl_sync(0xffffffffu, token, r * kRows + r_lane);
            if (j >= 0) {
                Raw<T> again;
                float f[8];
                again.load(x + j * stride);
                again.get(f);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    amax = fabsf(f[e]) < INFINITY ? fmaxf(amax, fabsf(f[e])) : amax;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    }
    const float mine = __fdiv_rn(amax, Q8<Fmt>::kQmax);
    const bool grew = !fresh && mine > old;
    const float scale = fresh || !(mine <= old) ? mine : old;
    if (lane == 0 && !(old == scale))
        *scale_at = scale;
    const bool plain = plain_rows || !(scale >= 8.7e-19f && scale <= 1.2e30f);  // 2^-60, 2^100
    const float inv = __frcp_rn(scale);
    auto code = [&](const float *f) {
        if (plain)
            return scale > 0 ? code8<Fmt, true>(f, scale, inv) : make_uint2(0, 0);
        return code8<Fmt, false>(f, scale, inv);
    };
#pragma unroll
    for (int r = 0; r < kIters; ++r) {
        const int j = kHeld ? 0 : __shfl_sync(0xffffffffu, token, r * kRows + r_lane);
        if (mine_written >> (r * kRows) & 1) {
            float f[8];
            if (!kHeld)
                raw[0].load(x + j * stride);
            raw[kHeld ? r : 0].get(f);
            *reinterpret_cast<uint2 *>(codes + r * kRows * D) = code(f);
        }
    }
    if (grew) {  // the other rows are coded again
#pragma unroll 1
        for (int r = 0; r < kIters; ++r)
            if (!(mine_written >> (r * kRows) & 1)) {
                uint2 *at = reinterpret_cast<uint2 *>(codes + r * kRows * D);
                const uint2 before = *at;
                float f[8];
                Q8<Fmt>::widen4(before.x, f);
                Q8<Fmt>::widen4(before.y, f + 4);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    f[e] = __fmul_rn(f[e], old);
                    if (Fmt == kFmtE4M3)  // (NaN codes, which only a pool of any contents holds)
                        f[e] = f[e] != f[e] ? 0.f : f[e];
                }
                *at = code(f);
            }
    }
}

// The blocks that tokens [first, first + count) (a warp, 32 at most) write and whose lowest
// written row is theirs: use(block, the rows' tokens, the rows).
template <int BS, typename Rows, typename Use>
__device__ inline void for_blocks(const AppendBqParams &p, long long first, int count, bool flag, int lane, Rows rows,
                                  Use use) {
    // a token whose predecessor in the call has the row before it has not the lowest
    long long slot = -1;
    bool may_lead = false;
    if (lane < count) {
        const long long i = first + lane;
        slot = p.slots[i];
        const long long before = i > 0 ? p.slots[i - 1] : -1;
        if (slot >= p.pool_slots) {
            if (flag && p.err)
                atomicOr(p.err, PA_DEVERR_BAD_SLOT);
        } else if (slot >= 0) {
            may_lead = slot % BS == 0 || before != slot - 1;
        }
    }
    // every block is looked up once
    const unsigned same = __match_any_sync(0xffffffffu, static_cast<unsigned>(slot / BS));
    const unsigned leads = __ballot_sync(0xffffffffu, may_lead);
    const bool looks = may_lead && __ffs(same & leads) - 1 == lane;
    for (unsigned todo = __ballot_sync(0xffffffffu, looks); todo; todo &= todo - 1) {
        const long long block = __shfl_sync(0xffffffffu, slot, __ffs(todo) - 1) / BS;
        const int token = rows(block * BS);
        const unsigned written = __ballot_sync(0xffffffffu, token >= 0);
        const int lowest = __shfl_sync(0xffffffffu, token, written ? __ffs(written) - 1 : 0);
        if (lowest >= first && lowest < first + count)
            use(block, token, written);
    }
}

// Few tokens: a warp a token and every parts-th unit of its block; the warps of a token
// look for its block each for itself, so none waits for another.
template <typename T, int D, int BS, int Fmt>
__global__ void __launch_bounds__(kBqThreads, 2) append_few_kernel(const AppendBqParams p) {
    __shared__ int32_t found[kBqWarps][32];  // a block's tokens
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long at = static_cast<long long>(blockIdx.x) * kBqWarps + warp;
    const long long first = at / p.parts;
    const int part = static_cast<int>(at % p.parts);
    if (first >= p.num_tokens)
        return;
    auto rows = [&](long long base) {  // of two tokens of one slot the later one counts
        found[warp][lane] = -1;
        __syncwarp();
        for (int j = lane; j < p.num_tokens; j += 32) {
            const long long off = p.slots[j] - base;
            if (off >= 0 && off < BS)
                atomicMax(&found[warp][off], j);
        }
        __syncwarp();
        const int token = found[warp][lane];
        __syncwarp();
        return token;
    };
    for_blocks<BS>(p, first, 1, part == 0, lane, rows, [&](long long block, int token, unsigned written) {
        for (int u = part; u < 2 * p.num_kv_heads; u += p.parts)
            store_unit<T, D, BS, Fmt>(p, block, token, written, u, lane);
    });
}

// Many: first a list of the blocks, the map's entries of theirs set to -1 where the call does not
// write the row.
template <int BS> __global__ void __launch_bounds__(kBqThreads) list_blocks_kernel(const AppendBqParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long first = (static_cast<long long>(blockIdx.x) * kBqWarps + (threadIdx.x >> 5)) * kListWindow;
    if (first >= p.num_tokens)
        return;
    const int count = static_cast<int>(min(static_cast<long long>(kListWindow), p.num_tokens - first));
    auto rows = [&](long long base) {
        int token = lane < BS ? __ldcg(p.token_of + base + lane) : -1;
        if (token < 0 || token >= p.num_tokens || p.slots[token] != base + lane)
            token = -1;
        return token;
    };
    for_blocks<BS>(p, first, count, true, lane, rows, [&](long long block, int token, unsigned) {
        if (lane == 0)
            p.list[atomicAdd(p.listed, 1)] = static_cast<int32_t>(block);
        if (lane < BS)
            p.token_of[block * BS + lane] = token;
    });
}

// Then all units of all blocks in one line, warp by warp; a unit's tokens and the block after the
// next unit's are on their way while the one before is stored.
template <typename T, int D, int BS, int Fmt>
__global__ void __launch_bounds__(kBqThreads, 3) append_listed_kernel(const AppendBqParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int units = 2 * p.num_kv_heads;
    const int warps = gridDim.x * kBqWarps, me = blockIdx.x * kBqWarps + (threadIdx.x >> 5);
    const int step_block = warps / units, step_unit = warps % units;
    const int blocks = __ldcg(p.listed);
    long long i = me / units;
    int u = me % units;
    auto block_at = [&](long long k) { return k < blocks ? __ldcg(p.list + k) : -1; };
    auto token_at = [&](int block) {
        return block >= 0 && lane < BS ? __ldcg(p.token_of + static_cast<long long>(block) * BS + lane) : -1;
    };
    auto advance = [&]() {
        i += step_block;
        u += step_unit;
        if (u >= units) {
            u -= units;
            ++i;
        }
    };
    int block = block_at(i), unit = u;
    int token = token_at(block);
    advance();
    int block_next = block_at(i), unit_next = u;
    while (block >= 0) {
        const int token_next = token_at(block_next);
        advance();
        const int block_after = block_at(i);
        store_unit<T, D, BS, Fmt>(p, block, token, __ballot_sync(0xffffffffu, token >= 0), unit, lane);
        block = block_next, token = token_next, unit = unit_next;
        block_next = block_after, unit_next = u;
    }
}

template <typename T, int D, int BS> const void *append_bq_fn(int fmt, bool few) {
    if (fmt == PA_I8)
        return few ? reinterpret_cast<const void *>(&append_few_kernel<T, D, BS, kFmtI8>)
                   : reinterpret_cast<const void *>(&append_listed_kernel<T, D, BS, kFmtI8>);
    return few ? reinterpret_cast<const void *>(&append_few_kernel<T, D, BS, kFmtE4M3>)
               : reinterpret_cast<const void *>(&append_listed_kernel<T, D, BS, kFmtE4M3>);
}
template <typename T> const void *append_bq_fn(int head_dim, int block_size, int fmt, bool few) {
    if (head_dim == 128)
        return block_size == 8    ? append_bq_fn<T, 128, 8>(fmt, few)
               : block_size == 16 ? append_bq_fn<T, 128, 16>(fmt, few)
                                  : append_bq_fn<T, 128, 32>(fmt, few);
    return block_size == 8    ? append_bq_fn<T, 64, 8>(fmt, few)
           : block_size == 16 ? append_bq_fn<T, 64, 16>(fmt, few)
                              : append_bq_fn<T, 64, 32>(fmt, few);
}

}  // namespace

cudaError_t launch_append_bq(AppendBqParams p, int dtype, int cache_dtype, int head_dim, int num_sms,
                             cudaStream_t stream) {
    const bool few = p.num_tokens <= kAppendBqFew;
    const void *fn = dtype == PA_F32   ? append_bq_fn<float>(head_dim, p.block_size, cache_dtype, few)
                     : dtype == PA_F16 ? append_bq_fn<__half>(head_dim, p.block_size, cache_dtype, few)
                                       : append_bq_fn<__nv_bfloat16>(head_dim, p.block_size, cache_dtype, few);
    const int units = 2 * p.num_kv_heads;
    void *args[] = {&p};
    const dim3 threads(kBqThreads);
    if (few) {
        p.parts = units < 512 ? units : 512;
        const int warps = p.num_tokens * p.parts;
        return launch_dependent(fn, dim3((warps + kBqWarps - 1) / kBqWarps), threads, args, 0, stream);
    }
    const void *list = p.block_size == 8    ? reinterpret_cast<const void *>(&list_blocks_kernel<8>)
                       : p.block_size == 16 ? reinterpret_cast<const void *>(&list_blocks_kernel<16>)
                                            : reinterpret_cast<const void *>(&list_blocks_kernel<32>);
    cudaError_t e = launch_dependent(reinterpret_cast<const void *>(&map_tokens_kernel),
                                     dim3((p.num_tokens + kBqThreads - 1) / kBqThreads), threads, args, 0, stream);
    constexpr int kListed = kListWindow * kBqWarps;
    if (e == cudaSuccess)
        e = launch_dependent(list, dim3((p.num_tokens + kListed - 1) / kListed), threads, args, 0, stream);
    if (e != cudaSuccess)
        return e;
    // (two CTAs an SM 31 us, four 28.5, for the prompts above)
    return launch_dependent(fn, dim3(3 * num_sms), threads, args, 0, stream);
}

}  // namespace pa
