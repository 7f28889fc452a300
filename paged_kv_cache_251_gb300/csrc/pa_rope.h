// Parameters of the rotary kernel (pa_rope.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pa {

struct RopeParams {
    const void *q;       // rows of num_heads * head_dim, q_stride elements apart
    void *q_out;         // the same, q_out_stride apart
    const void *k, *v;   // rows of num_kv_heads * head_dim (num_kv_heads 0: none)
    const int32_t *positions;
    const double *freqs;
    const int64_t *slots;
    void *k_cache, *v_cache;
    uint32_t *err;
    long long num_tokens, q_stride, q_out_stride, k_stride, v_stride;
    int num_heads, num_kv_heads, head_dim, rot, block_size, num_blocks, direction;
    float mscale;
    int tok;  // tokens per CTA (set by the launch)
};

cudaError_t launch_rope(RopeParams p, int dtype, int interleaved, int num_sms, cudaStream_t stream);

}  // namespace pa
