// Launch of the block-scaled decode, and the kernel that joins the pieces cut
// between its CTAs.
#include <climits>

#include "pa_decode_bq.cuh"
#include "pa_host.h"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kJoinThreads = 512;
constexpr int kJoinWarps = kJoinThreads / 32;

// A CTA a record: the partials of CTAs blockIdx.x (slot 1) .. last (slot 0).  A warp
// takes one head and every kJoinWarps / heads-th partial; D / 32 columns a lane.
template <int D> __global__ void __launch_bounds__(kJoinThreads) join_bq_kernel(const DecodeBqParams p) {
    constexpr int C = D / 32;
    __shared__ float acc[kJoinWarps][D];
    pdl_launch_dependents();
    pdl_wait();
    const int4 rec = p.records[blockIdx.x];
    if (rec.w == 0)
        return;
    const int G = p.num_heads / p.num_kv_heads;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int h = warp % G, sub = warp / G, subs = kJoinWarps / G;  // G: 1, 2, 4 or 8
    const int first = blockIdx.x, n = rec.z - first + 1;
    const float2 *ml = reinterpret_cast<const float2 *>(p.part_ml);
    auto part_of = [&](int i) { return (static_cast<long long>(first + i) * 2 + (i == 0)) * G + h; };
    // the first partials are on their way while the largest maximum is found
    constexpr int kAhead = 4;
    float ahead[kAhead][C];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
        const int i = sub + k * subs;
#pragma unroll
        for (int c = 0; c < C; ++c)
            ahead[k][c] = i < n ? p.part_acc[part_of(i) * D + 32 * c + lane] : 0.f;
    }
    float2 mine = lane < n ? ml[part_of(lane)] : make_float2(kNoMax, 0.f);
    float top = mine.x;
    for (int i = lane + 32; i < n; i += 32)
        top = fmaxf(top, ml[part_of(i)].x);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
    float sum = ex2(mine.x - top) * mine.y;
    for (int i = lane + 32; i < n; i += 32) {
        const float2 x = ml[part_of(i)];
        sum = fmaf(ex2(x.x - top), x.y, sum);
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, s);
    float y[C];
#pragma unroll
    for (int c = 0; c < C; ++c)
        y[c] = 0.f;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
        const int i = sub + k * subs;
        const float f = i < n ? ex2(ml[part_of(i)].x - top) : 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c)
            y[c] = fmaf(f, ahead[k][c], y[c]);
    }
#pragma unroll 4
    for (int i = sub + kAhead * subs; i < n; i += subs) {
        const long long part = part_of(i);
        const float f = ex2(ml[part].x - top);
#pragma unroll
        for (int c = 0; c < C; ++c)
            y[c] = fmaf(f, p.part_acc[part * D + 32 * c + lane], y[c]);
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
        acc[warp][32 * c + lane] = y[c];
    __syncthreads();
    if (sub != 0)
        return;
    const float inv = sum > 0 ? 1.f / sum : (sum == 0 ? 0.f : sum);
    const long long row = static_cast<long long>(rec.x) * p.num_heads + static_cast<long long>(rec.y) * G + h;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        float v = 0.f;
        for (int s = 0; s < subs; ++s)
            v += acc[s * G + h][32 * c + lane];
        store_out(p.out, p.out_dtype, row * D + 32 * c + lane, v * inv);
    }
}

}  // namespace

int decode_bq_ctas(int num_seqs, int num_kv_heads, int max_len) {
    // pieces of 16-token iterations at most, kMinShare of them a warp at least
    const long long iters = (static_cast<long long>(max_len) + 15) / 16 + kPieceCost;
    const long long pieces = static_cast<long long>(num_seqs) * num_kv_heads;
    const long long per_cta = static_cast<long long>(kDecodeBqWarps) * (kMinShare + kPieceCost);
    if (pieces > kDecodeBqMaxCtas * per_cta / iters)
        return kDecodeBqMaxCtas;
    return static_cast<int>((pieces * iters + per_cta - 1) / per_cta);
}

cudaError_t launch_decode_bq(DecodeBqParams p, int cache_dtype, int head_dim, int num_sms, cudaStream_t stream) {
    const int group = p.num_heads / p.num_kv_heads;
    const bool wide = group > 4, f32 = p.q_dtype == PA_F32, b8 = p.block_size == 8;
    const void *fn = cache_dtype == PA_I8
                         ? (head_dim == 128 ? decode_bq_kernel_i8_128(wide, f32, b8) : decode_bq_kernel_i8_64(wide, f32, b8))
                         : (head_dim == 128 ? decode_bq_kernel_e4m3_128(wide, f32, b8)
                                            : decode_bq_kernel_e4m3_64(wide, f32, b8));
    const size_t smem = bq_smem(group, head_dim);
    int dev = 0, sms = 0, per_sm = 0;
    cudaError_t e = device_sms(&dev, &sms);
    if (e == cudaSuccess)
        e = prepare_kernel(dev, fn, smem, kDecodeBqThreads, &per_sm);
    if (e != cudaSuccess)
        return e;
    if (per_sm > kDecodeBqCtas)
        per_sm = kDecodeBqCtas;
    const int most = (num_sms < kDecodeBqSms ? num_sms : kDecodeBqSms) * (per_sm < 1 ? 1 : per_sm);
    const long long pieces = static_cast<long long>(p.num_seqs) * p.num_kv_heads;
    const int tokens = 16 * (128 / head_dim);  // of an iteration
    p.by_piece = pieces <= most && p.max_len <= kByPieceIters * tokens;
    int ctas = p.by_piece ? static_cast<int>(pieces) : decode_bq_ctas(p.num_seqs, p.num_kv_heads, p.max_len);
    if (ctas > most)
        ctas = most;
    void *args[] = {&p};
    e = launch_dependent(fn, dim3(static_cast<unsigned>(ctas)), dim3(kDecodeBqThreads), args, smem, stream);
    if (e != cudaSuccess || p.by_piece || ctas == 1)
        return e;
    return launch_dependent(head_dim == 128 ? reinterpret_cast<const void *>(&join_bq_kernel<128>)
                                            : reinterpret_cast<const void *>(&join_bq_kernel<64>),
                            dim3(static_cast<unsigned>(ctas)), dim3(kJoinThreads), args, 0, stream);
}

}  // namespace pa
