// The score pass of the scored decode: from every query head's scores (base-2
// units) and its partitions' running maxima and denominators to softmax
// weights, added to the accumulated scores of the kv head:
//   M = max_p m_p, den = sum_p 2^(m_p - M) l_p,
//   scores_out[s][kvh][t] = scores_in[s][kvh][t] + sum_g 2^(x_gt - M_g) / den_g.
// It reads G + 1 floats and writes one per (kv head, token): HBM-bound (the
// scores were written just before and partly sit in L2).  The decode cannot
// form the weights itself: a token's weight needs the whole row's maximum and
// denominator, known only when its last partition is done.
#include <cuda_runtime.h>

#include "pa_decode.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kScoreThreads = 256;
constexpr int kScoreTokens = 1024;  // tokens of a CTA
constexpr int kMaxGroup = 8;

// grid: (token chunks, kv heads, sequences)
__global__ void __launch_bounds__(kScoreThreads) score_kernel(const DecodeParams p, const float *in, float *out,
                                                              long long stride) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ float top[kMaxGroup], inv[kMaxGroup];
    const int s = blockIdx.z, kvh = blockIdx.y;
    const int G = p.num_heads / p.num_kv_heads;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const SeqSpan sp = seq_span(ld_nc_i32(p.context_lens + s), p.max_len, 0, p.block_size, p.bpp);
    const int t0 = blockIdx.x * kScoreTokens;
    if (t0 >= sp.end)
        return;
    const long long row0 = static_cast<long long>(s) * p.num_heads + static_cast<long long>(kvh) * G;
    if (warp < G) {
        const float2 *ml = reinterpret_cast<const float2 *>(p.part_ml) + (row0 + warp) * p.max_parts;
        float m = -INFINITY;
        for (int q = lane; q < sp.nparts; q += 32)
            m = fmaxf(m, ml[q].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        float den = 0.f;
        for (int q = lane; q < sp.nparts; q += 32) {
            const float2 v = ml[q];
            den += v.x == -INFINITY ? 0.f : v.y * exp2f(v.x - m);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            den += __shfl_xor_sync(0xffffffffu, den, o);
        if (lane == 0) {
            top[warp] = m == -INFINITY ? 0.f : m;
            inv[warp] = den == 0.f ? 0.f : 1.f / den;
        }
    }
    __syncthreads();
    const float *x = p.logits + row0 * p.logits_stride;
    const long long at = (static_cast<long long>(s) * p.num_kv_heads + kvh) * stride;
#pragma unroll
    for (int i = 0; i < kScoreTokens / kScoreThreads; ++i) {
        const int t = t0 + i * kScoreThreads + threadIdx.x;
        if (t < sp.end) {
            float w = 0.f;
            for (int g = 0; g < G; ++g)
                w += exp2f(x[g * p.logits_stride + t] - top[g]) * inv[g];
            out[at + t] = in ? in[at + t] + w : w;
        }
    }
}

}  // namespace

cudaError_t launch_scores(DecodeParams &p, const float *in, float *out, long long stride, cudaStream_t stream) {
    const int chunks = (p.max_len + kScoreTokens - 1) / kScoreTokens;
    // sequences on z, 65535 at a time
    for (int s0 = 0; s0 < p.num_seqs; s0 += 65535) {
        DecodeParams c = p;
        const int n = p.num_seqs - s0 < 65535 ? p.num_seqs - s0 : 65535;
        const long long rows = static_cast<long long>(s0) * p.num_heads;
        c.context_lens += s0;
        c.part_ml += rows * p.max_parts * 2;
        c.logits += rows * p.logits_stride;
        const long long at = static_cast<long long>(s0) * p.num_kv_heads * stride;
        const float *ci = in ? in + at : nullptr;
        float *co = out + at;
        void *args[] = {&c, &ci, &co, &stride};
        const cudaError_t e = launch_dependent(reinterpret_cast<const void *>(&score_kernel),
                                               dim3(chunks, p.num_kv_heads, n), dim3(kScoreThreads), args, 0, stream);
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

}  // namespace pa
