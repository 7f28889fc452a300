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
// A block is taken whole by one CTA, whichever of its rows the call writes: the
// scale needs them all.  Its tokens may stand anywhere in the call.  A few tokens
// (a decode step): every CTA looks at all slots.  Many: a first kernel writes each
// slot's token into a map of the pool's slots, which needs no clearing: an entry is
// believed only if the token that it names has that very slot.  The CTA of a block is
// the one whose window of tokens holds the block's lowest written row.
//
// HBM-bound: a row is read, its codes written.  A warp takes one kv head of K or V of
// a block; a lane eight elements of a row, and holds its share of the block's
// rows in registers, all loads in flight together, between the scale and the codes (fp32
// rows of blocks of 32 at head_dim 128 are read twice).  Divisions: the correctly
// rounded quotient from the correctly rounded reciprocal by two residual corrections
// (Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990), where no step can leave the normal range; else the plain one.
//
// Measured: 24000 tokens of ragged prompts, 8 kv heads of 128, bf16 to E4M3: 33 us with the
// map (2 us), 4.6 TB/s (floor 22 us): a CTA's search for its blocks is three dependent
// reads, its rows a fourth, and 24 warps an SM do not cover them; plain divisions
// 72 us (with rows read twice).  64 tokens of a decode step: 3.5 us on the GPU.
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
constexpr int kBqMaxWindow = 64;

__global__ void __launch_bounds__(kBqThreads) map_tokens_kernel(const int64_t *__restrict__ slots, int32_t *token_of,
                                                                int num_tokens, long long pool_slots) {
    pdl_launch_dependents();
    pdl_wait();
    const int i = blockIdx.x * kBqThreads + threadIdx.x;
    if (i < num_tokens) {
        const long long slot = slots[i];
        if (slot >= 0 && slot < pool_slots)
            token_of[slot] = i;
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

// grid: (windows, unit_split).
template <typename T, int D, int BS, int Fmt>
__global__ void __launch_bounds__(kBqThreads, 2) append_bq_kernel(const AppendBqParams p) {
    constexpr int kRowLanes = D / 8;
    constexpr int kRows = 32 / kRowLanes;  // rows of a warp at once
    constexpr int kIters = BS / kRows;
    constexpr bool kHeld = kIters * static_cast<int>(sizeof(T)) <= 32;  // 64 registers
    __shared__ int32_t rows[kBqMaxWindow][BS];  // of a candidate's block: every row's token, -1: not written
    __shared__ long long block_at[kBqMaxWindow];
    __shared__ int32_t candidate[kBqMaxWindow], lead[kBqMaxWindow];
    __shared__ int candidates, leads;
    __shared__ long long slots[kAppendBqFew];  // of a call of few tokens
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int first = blockIdx.x * p.window;
    const int count = p.num_tokens - first < p.window ? p.num_tokens - first : p.window;
    const bool few = p.token_of == nullptr;
    if (tid == 0)
        candidates = leads = 0;
    if (few) {
        for (int j = tid; j < p.num_tokens; j += kBqThreads)
            slots[j] = p.slots[j];
        for (int j = tid; j < count * BS; j += kBqThreads)
            (&rows[0][0])[j] = -1;
    }
    __syncthreads();
    // a token whose predecessor in the call has the row before it does not lead its block
    if (tid < count) {
        const int i = first + tid;
        const long long slot = p.slots[i], before = i > 0 && slot % BS != 0 ? p.slots[i - 1] : -1;
        if (slot >= p.pool_slots) {
            if (blockIdx.y == 0 && p.err)
                atomicOr(p.err, PA_DEVERR_BAD_SLOT);
        } else if (slot >= 0 && (slot % BS == 0 || before != slot - 1)) {
            const int n = atomicAdd(&candidates, 1);
            candidate[n] = i;
            block_at[n] = slot / BS;
        }
    }
    __syncthreads();
    for (int n = warp; n < candidates; n += kBqWarps) {
        const int i = candidate[n];
        const long long base = block_at[n] * BS;
        if (few) {  // of two tokens of one slot the later one counts
            for (int j = lane; j < p.num_tokens; j += 32) {
                const long long off = slots[j] - base;
                if (off >= 0 && off < BS)
                    atomicMax(&rows[n][off], j);
            }
            __syncwarp();
        } else if (lane < BS) {
            int j = p.token_of[base + lane];
            if (j < 0 || j >= p.num_tokens || p.slots[j] != base + lane)
                j = -1;
            rows[n][lane] = j;
        }
        // the token of the lowest written row leads
        const int j = lane < BS ? rows[n][lane] : -1;
        const unsigned any = __ballot_sync(0xffffffffu, j >= 0);
        const int lowest = __shfl_sync(0xffffffffu, j, any ? __ffs(any) - 1 : 0);
        if (lane == 0 && any != 0 && lowest == i)
            lead[atomicAdd(&leads, 1)] = n;
    }
    __syncthreads();
    const int units = 2 * p.num_kv_heads;
    const int r_lane = lane / kRowLanes, c = lane % kRowLanes * 8;
    const long long stride = static_cast<long long>(p.num_kv_heads) * D;
    const long long all = static_cast<long long>(units) * leads;
    for (long long k = warp + kBqWarps * blockIdx.y; k < all; k += kBqWarps * gridDim.y) {
        const int w = lead[static_cast<int>(k / units)], u = static_cast<int>(k % units);
        const bool is_v = u >= p.num_kv_heads;
        const int h = is_v ? u - p.num_kv_heads : u;
        const T *x = static_cast<const T *>(is_v ? p.v : p.k) + static_cast<long long>(h) * D + c;
        const long long tile = block_at[w] * p.num_kv_heads + h;
        float *scale_at = (is_v ? p.v_scales : p.k_scales) + tile;
        uint8_t *codes = (is_v ? p.v_cache : p.k_cache) + tile * BS * D + r_lane * D + c;
        const bool fresh = rows[w][0] >= 0;
        const float old = __shfl_sync(0xffffffffu, lane == 0 ? *scale_at : 0.f, 0);  // (lane 0 writes it too)
        Raw<T> raw[kHeld ? kIters : 1];
        uint32_t top = 0;
        if (kHeld) {
#pragma unroll
            for (int r = 0; r < kIters; ++r) {
                const int j = rows[w][r * kRows + r_lane];
                if (j >= 0)
                    raw[r].load(x + j * stride);
            }
#pragma unroll
            for (int r = 0; r < kIters; ++r)
                if (rows[w][r * kRows + r_lane] >= 0)
                    top = raw[r].peak(top);
        } else {
#pragma unroll 4
            for (int r = 0; r < kIters; ++r) {
                const int j = rows[w][r * kRows + r_lane];
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
                const int j = rows[w][r * kRows + r_lane];
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
            const int j = rows[w][r * kRows + r_lane];
            if (j >= 0) {
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
                if (rows[w][r * kRows + r_lane] < 0) {
                    uint2 *at = reinterpret_cast<uint2 *>(codes + r * kRows * D);
                    const uint2 before = *at;
                    float f[8];
                    Q8<Fmt>::widen4(before.x, f);
                    Q8<Fmt>::widen4(before.y, f + 4);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        f[e] = __fmul_rn(f[e], old);
                    *at = code(f);
                }
        }
    }
}

template <typename T, int D, int BS> const void *append_bq_fn(int fmt) {
    return fmt == PA_I8 ? reinterpret_cast<const void *>(&append_bq_kernel<T, D, BS, kFmtI8>)
                        : reinterpret_cast<const void *>(&append_bq_kernel<T, D, BS, kFmtE4M3>);
}
template <typename T> const void *append_bq_fn(int head_dim, int block_size, int fmt) {
    if (head_dim == 128)
        return block_size == 8    ? append_bq_fn<T, 128, 8>(fmt)
               : block_size == 16 ? append_bq_fn<T, 128, 16>(fmt)
                                  : append_bq_fn<T, 128, 32>(fmt);
    return block_size == 8    ? append_bq_fn<T, 64, 8>(fmt)
           : block_size == 16 ? append_bq_fn<T, 64, 16>(fmt)
                              : append_bq_fn<T, 64, 32>(fmt);
}

}  // namespace

cudaError_t launch_append_bq(AppendBqParams p, int dtype, int cache_dtype, int head_dim, int num_sms,
                             cudaStream_t stream) {
    const bool few = p.num_tokens <= kAppendBqFew;
    if (few)
        p.token_of = nullptr;
    const void *fn = dtype == PA_F32   ? append_bq_fn<float>(head_dim, p.block_size, cache_dtype)
                     : dtype == PA_F16 ? append_bq_fn<__half>(head_dim, p.block_size, cache_dtype)
                                       : append_bq_fn<__nv_bfloat16>(head_dim, p.block_size, cache_dtype);
    if (!few) {
        const int ctas = (p.num_tokens + kBqThreads - 1) / kBqThreads;
        void *args[] = {&p.slots, &p.token_of, &p.num_tokens, &p.pool_slots};
        const cudaError_t e = launch_dependent(reinterpret_cast<const void *>(&map_tokens_kernel),
                                               dim3(static_cast<unsigned>(ctas)), dim3(kBqThreads), args, 0, stream);
        if (e != cudaSuccess)
            return e;
    }
    // windows as long as they leave eight CTAs an SM (24000 tokens: 33 us; four or sixteen CTAs
    // 36 to 37); CTAs share a window's heads where there are still too few
    const int want = 8 * num_sms;
    p.window = 1;
    while (p.window < kBqMaxWindow && p.num_tokens / (p.window * 2) >= want)
        p.window *= 2;
    const int windows = (p.num_tokens + p.window - 1) / p.window;
    int split = 1;
    while (windows * split < want && 2 * p.num_kv_heads > kBqWarps * split)
        ++split;
    void *args[] = {&p};
    return launch_dependent(fn, dim3(static_cast<unsigned>(windows), static_cast<unsigned>(split)), dim3(kBqThreads),
                            args, 0, stream);
}

}  // namespace pa
