// Scored-decode kernel instantiations for __nv_bfloat16 caches: the decode kernels with
// every token's score written out (general kernel: head_dim 64, query groups
// 2/4/8; one query head per kv head: head_dim 64/128, block 8/16/32;
// tensor-core grouped heads: head_dim 128, block 8/16/32, query groups 2/4/8).
#include "pa_decode_gqa.cuh"
#include "pa_internal.h"

namespace pa {

const void *scored_kernel_bf16(int head_dim, int group) {
#define PA_CASE(D, G)                                                    \
    if (head_dim == D && group == G)                                     \
        return reinterpret_cast<const void *>(&pa_decode_kernel<__nv_bfloat16, D, G, true>);
    PA_CASE(64, 2) PA_CASE(64, 4) PA_CASE(64, 8)
#undef PA_CASE
    return nullptr;
}

const void *scored_mha_kernel_bf16(int head_dim, int block_size) {
#define PA_CASE(D, BS)                                                   \
    if (head_dim == D && block_size == BS)                               \
        return reinterpret_cast<const void *>(&pa_decode_mha_kernel<__nv_bfloat16, D, BS, true>);
    PA_CASE(64, 8) PA_CASE(64, 16) PA_CASE(64, 32)
    PA_CASE(128, 8) PA_CASE(128, 16) PA_CASE(128, 32)
#undef PA_CASE
    return nullptr;
}

const void *scored_gqa_kernel_bf16(int block_size, int group) {
#define PA_CASE(BS, G)                                                   \
    if (block_size == BS && group == G)                                  \
        return reinterpret_cast<const void *>(&pa_decode_gqa_kernel<__nv_bfloat16, BS, G, true>);
    PA_CASE(8, 2) PA_CASE(8, 4) PA_CASE(8, 8)
    PA_CASE(16, 2) PA_CASE(16, 4) PA_CASE(16, 8)
    PA_CASE(32, 2) PA_CASE(32, 4) PA_CASE(32, 8)
#undef PA_CASE
    return nullptr;
}

}  // namespace pa
