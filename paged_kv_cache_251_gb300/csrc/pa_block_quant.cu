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
// a block; a lane eight elements of a row.  The rows are read twice (the scale comes
// before the codes), the second time from L1.
#include <cuda_runtime.h>

#include "pa_block_quant.h"
#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_quant.cuh"

namespace pa {

namespace {

constexpr int kBqThreads = 256;
constexpr int kBqWarps = kBqThreads / 32;
constexpr int kBqMaxWindow = 64;
constexpr int kBqMaxBlock = 32;

__device__ inline long long div_block(long long slot, int block_size) {  // 8, 16 or 32
    return slot >> (block_size == 8 ? 3 : (block_size == 16 ? 4 : 5));
}

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

// Eight elements of a row as fp32.
template <typename T> __device__ inline void load8(const T *p, float *f) {
    if constexpr (sizeof(T) == 4) {
        Elt<T>::unpack(*reinterpret_cast<const uint4 *>(p), f);
        Elt<T>::unpack(*reinterpret_cast<const uint4 *>(p + 4), f + 4);
    } else {
        Elt<T>::unpack(*reinterpret_cast<const uint4 *>(p), f);
    }
}

template <int Fmt> __device__ inline uint32_t code_of(float x, float scale) {
    const float y = __fdiv_rn(x, scale);
    return y != y ? 0u : Q8<Fmt>::encode(y);  // (NaN, or 0 / 0: code 0)
}

template <int Fmt> __device__ inline uint2 code8(const float *f, float scale) {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        w[e >> 2] |= code_of<Fmt>(f[e], scale) << (8 * (e & 3));
    return make_uint2(w[0], w[1]);
}

// grid: (windows, unit_split).
template <typename T, int D, int Fmt, bool Few>
__global__ void __launch_bounds__(kBqThreads) append_bq_kernel(const AppendBqParams p) {
    constexpr int kRowLanes = D / 8;
    constexpr int kRows = 32 / kRowLanes;  // rows of a warp at once
    __shared__ int32_t rows[kBqMaxWindow][kBqMaxBlock];  // token of every row of a block, -1: not written
    __shared__ long long block_at[kBqMaxWindow];         // block of the window's token if it leads it, else -1
    __shared__ long long few[Few ? kAppendBqFew : 1];
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int first = blockIdx.x * p.window;
    const int count = p.num_tokens - first < p.window ? p.num_tokens - first : p.window;
    const int bs = p.block_size;
    if (Few) {
        for (int j = tid; j < p.num_tokens; j += kBqThreads)
            few[j] = p.slots[j];
        for (int j = tid; j < count * kBqMaxBlock; j += kBqThreads)
            (&rows[0][0])[j] = -1;
        __syncthreads();
    }
    for (int w = warp; w < count; w += kBqWarps) {
        const int i = first + w;
        const long long slot = Few ? few[i] : p.slots[i];
        long long block = -1;
        if (slot >= p.pool_slots) {
            if (lane == 0 && blockIdx.y == 0 && p.err)
                atomicOr(p.err, PA_DEVERR_BAD_SLOT);
        } else if (slot >= 0) {
            block = div_block(slot, bs);
            const long long base = block * bs;
            if (Few) {  // of two tokens of one slot the later one counts
                for (int j = lane; j < p.num_tokens; j += 32) {
                    const long long off = few[j] - base;
                    if (off >= 0 && off < bs)
                        atomicMax(&rows[w][off], j);
                }
                __syncwarp();
            } else if (lane < bs) {
                int j = p.token_of[base + lane];
                if (j < 0 || j >= p.num_tokens || p.slots[j] != base + lane)
                    j = -1;
                rows[w][lane] = j;
            }
            const int j = lane < bs ? rows[w][lane] : -1;
            const unsigned any = __ballot_sync(0xffffffffu, j >= 0);
            // the token of the lowest written row leads
            if (any == 0 || __shfl_sync(0xffffffffu, j, any ? __ffs(any) - 1 : 0) != i)
                block = -1;
        }
        if (lane == 0)
            block_at[w] = block;
    }
    __syncthreads();
    const int units = 2 * p.num_kv_heads;
    const int r_lane = lane / kRowLanes, c = lane % kRowLanes * 8;
    const long long stride = static_cast<long long>(p.num_kv_heads) * D;
    for (int u = warp + kBqWarps * blockIdx.y; u < units; u += kBqWarps * gridDim.y) {
        const bool is_v = u >= p.num_kv_heads;
        const int h = is_v ? u - p.num_kv_heads : u;
        const T *x = static_cast<const T *>(is_v ? p.v : p.k) + static_cast<long long>(h) * D + c;
        for (int w = 0; w < count; ++w) {
            const long long block = block_at[w];
            if (block < 0)
                continue;
            const long long tile = block * p.num_kv_heads + h;
            float *scale_at = (is_v ? p.v_scales : p.k_scales) + tile;
            uint8_t *codes = (is_v ? p.v_cache : p.k_cache) + tile * bs * D + c;
            const float old = __shfl_sync(0xffffffffu, lane == 0 ? *scale_at : 0.f, 0);  // (lane 0 writes it too)
            float amax = 0.f;
#pragma unroll 4
            for (int r0 = 0; r0 < bs; r0 += kRows) {
                const int j = rows[w][r0 + r_lane];
                if (j >= 0) {
                    float f[8];
                    load8(x + j * stride, f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float a = fabsf(f[e]);
                        amax = a < INFINITY ? fmaxf(amax, a) : amax;  // infinities saturate, NaN is coded 0
                    }
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            const float mine = __fdiv_rn(amax, Q8<Fmt>::kQmax);
            const bool fresh = rows[w][0] >= 0;
            const bool grew = !fresh && mine > old;
            const float scale = fresh || !(mine <= old) ? mine : old;
            if (lane == 0 && (fresh || grew || !(old == scale)))
                *scale_at = scale;
#pragma unroll 4
            for (int r0 = 0; r0 < bs; r0 += kRows) {
                const int r = r0 + r_lane, j = rows[w][r];
                if (j < 0 && !grew)
                    continue;
                float f[8];
                uint2 *at = reinterpret_cast<uint2 *>(codes + static_cast<long long>(r) * D);
                if (j >= 0) {
                    load8(x + j * stride, f);
                } else {
                    const uint2 old8 = *at;
                    Q8<Fmt>::widen4(old8.x, f);
                    Q8<Fmt>::widen4(old8.y, f + 4);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        f[e] = __fmul_rn(f[e], old);
                }
                *at = scale > 0 ? code8<Fmt>(f, scale) : make_uint2(0, 0);
            }
            __syncwarp();
        }
    }
}

template <typename T, int D> const void *append_bq_fn(int fmt, bool few) {
    if (fmt == PA_I8)
        return few ? reinterpret_cast<const void *>(&append_bq_kernel<T, D, kFmtI8, true>)
                   : reinterpret_cast<const void *>(&append_bq_kernel<T, D, kFmtI8, false>);
    return few ? reinterpret_cast<const void *>(&append_bq_kernel<T, D, kFmtE4M3, true>)
               : reinterpret_cast<const void *>(&append_bq_kernel<T, D, kFmtE4M3, false>);
}

}  // namespace

cudaError_t launch_append_bq(AppendBqParams p, int dtype, int cache_dtype, int head_dim, int num_sms,
                             cudaStream_t stream) {
    const bool few = p.num_tokens <= kAppendBqFew;
    const void *fn;
    if (dtype == PA_F32)
        fn = head_dim == 128 ? append_bq_fn<float, 128>(cache_dtype, few) : append_bq_fn<float, 64>(cache_dtype, few);
    else if (dtype == PA_F16)
        fn = head_dim == 128 ? append_bq_fn<__half, 128>(cache_dtype, few) : append_bq_fn<__half, 64>(cache_dtype, few);
    else
        fn = head_dim == 128 ? append_bq_fn<__nv_bfloat16, 128>(cache_dtype, few)
                             : append_bq_fn<__nv_bfloat16, 64>(cache_dtype, few);
    if (!few) {
        const int ctas = (p.num_tokens + kBqThreads - 1) / kBqThreads;
        void *args[] = {&p.slots, &p.token_of, &p.num_tokens, &p.pool_slots};
        const cudaError_t e = launch_dependent(reinterpret_cast<const void *>(&map_tokens_kernel),
                                               dim3(static_cast<unsigned>(ctas)), dim3(kBqThreads), args, 0, stream);
        if (e != cudaSuccess)
            return e;
    }
    // windows as long as they leave four CTAs an SM; CTAs share a window's heads
    // where there are still too few
    const int want = 4 * num_sms;
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
