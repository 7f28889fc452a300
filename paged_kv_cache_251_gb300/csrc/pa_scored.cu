// The score pass of the scored decode: from every query head's scores (base-2
// units) and its partitions' running maxima and denominators to softmax
// weights, added to the accumulated scores of the kv head:
//   M = max_p m_p, den = sum_p 2^(m_p - M) l_p,
//   scores_out[s][kvh][t] = scores_in[s][kvh][t] + sum_g 2^(x_gt - M_g) / den_g.
// It reads G + 1 floats and writes one per (kv head, token): HBM-bound (the
// scores were written just before and partly sit in L2).  The decode cannot
// form the weights itself: a token's weight needs the whole row's maximum and
// denominator, known only when its last partition is done.  Measured: 256 contexts of
// 16 to 8192 tokens, 32 / 8 heads, bf16: 19 us for 66 MB, of a call of 250 us.
#include <cuda_runtime.h>

#include "pa_decode.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kScoreThreads = 256;
constexpr int kScorePer = 4;                                // tokens of a thread
constexpr int kScoreTokens = kScoreThreads * kScorePer;     // tokens of a CTA

// grid: (token chunks, kv heads, sequences); a CTA takes every gridDim.x-th chunk
// of its context.  The first chunk's loads go out before the row states are
// formed (two round trips in all: the length, then the rest).
template <int G>
__global__ void __launch_bounds__(kScoreThreads) score_kernel(const DecodeParams p, const float *in, float *out,
                                                              long long stride) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ float top[G], inv[G];
    const int s = blockIdx.z, kvh = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const SeqSpan sp = seq_span(ld_nc_i32(p.context_lens + s), p.max_len, 0, p.block_size, p.bpp);
    if (static_cast<int>(blockIdx.x) * kScoreTokens >= sp.end)
        return;
    const long long row0 = static_cast<long long>(s) * p.num_heads + static_cast<long long>(kvh) * G;
    // (rows of scores are whole blocks, so four at a time stay inside and aligned)
    const float *x = p.logits + row0 * p.logits_stride;
    const long long at = (static_cast<long long>(s) * p.num_kv_heads + kvh) * stride;
    const bool in16 = (reinterpret_cast<uintptr_t>(in + at) & 15u) == 0;
    const bool out16 = (reinterpret_cast<uintptr_t>(out + at) & 15u) == 0;
    bool first = true;
    for (int t = blockIdx.x * kScoreTokens + threadIdx.x * kScorePer; first || t < sp.end;
         t += gridDim.x * kScoreTokens) {
        const int n = min(kScorePer, sp.end - t);
        float4 v[G];
        float base[kScorePer] = {0.f, 0.f, 0.f, 0.f};
        if (n > 0) {
#pragma unroll
            for (int g = 0; g < G; ++g)
                v[g] = *reinterpret_cast<const float4 *>(x + g * p.logits_stride + t);
            if (in) {
                if (n == kScorePer && in16) {
                    const float4 b = *reinterpret_cast<const float4 *>(in + at + t);
                    base[0] = b.x, base[1] = b.y, base[2] = b.z, base[3] = b.w;
                } else {
                    for (int i = 0; i < n; ++i)
                        base[i] = in[at + t + i];
                }
            }
        }
        if (first) {
            if (warp < G) {
                const float2 *ml = reinterpret_cast<const float2 *>(p.part_ml) + (row0 + warp) * p.max_parts;
                float m = -INFINITY, den = 0.f;
                for (int q = lane; q < sp.nparts; q += 32) {
                    const float2 a = ml[q];
                    if (a.x == -INFINITY && a.y == 0.f)
                        continue;
                    const float mn = fmaxf(m, a.x);
                    den = (m == -INFINITY ? 0.f : den * exp2f(m - mn)) + a.y * exp2f(a.x - mn);
                    m = mn;
                }
                float M = m;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
                den = m == -INFINITY ? den : den * exp2f(m - M);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    den += __shfl_xor_sync(0xffffffffu, den, o);
                if (lane == 0) {
                    top[warp] = M == -INFINITY ? 0.f : M;
                    inv[warp] = den == 0.f ? 0.f : 1.f / den;
                }
            }
            __syncthreads();
            first = false;
        }
        if (n <= 0)
            return;
        float w[kScorePer] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const float m = top[g], r = inv[g];
            w[0] += exp2f(v[g].x - m) * r;
            w[1] += exp2f(v[g].y - m) * r;
            w[2] += exp2f(v[g].z - m) * r;
            w[3] += exp2f(v[g].w - m) * r;
        }
        if (n == kScorePer && out16) {
            *reinterpret_cast<float4 *>(out + at + t) =
                make_float4(base[0] + w[0], base[1] + w[1], base[2] + w[2], base[3] + w[3]);
        } else {
            for (int i = 0; i < n; ++i)
                out[at + t + i] = base[i] + w[i];
        }
    }
}

const void *score_fn(int G) {
    return G == 1   ? reinterpret_cast<const void *>(&score_kernel<1>)
           : G == 2 ? reinterpret_cast<const void *>(&score_kernel<2>)
           : G == 4 ? reinterpret_cast<const void *>(&score_kernel<4>)
                    : reinterpret_cast<const void *>(&score_kernel<8>);
}

}  // namespace

cudaError_t launch_scores(DecodeParams &p, const float *in, float *out, long long stride, int sms,
                          cudaStream_t stream) {
    // enough CTAs a context to fill the SMs twice over, no more: one without a chunk
    // costs nearly as much as one with (a chunk a CTA: 7.5 us more on 256 contexts of
    // 16 to 8192 tokens)
    const long long pairs = static_cast<long long>(p.num_seqs) * p.num_kv_heads;
    const long long most = (p.max_len + kScoreTokens - 1) / kScoreTokens;
    long long chunks = (16LL * sms + pairs - 1) / pairs;
    chunks = chunks < most ? chunks : most;
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
        const cudaError_t e = launch_dependent(score_fn(p.num_heads / p.num_kv_heads),
                                               dim3(static_cast<unsigned>(chunks), p.num_kv_heads, n), dim3(kScoreThreads), args, 0,
                                               stream);
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

}  // namespace pa
