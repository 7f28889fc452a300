// Scored-decode kernel instantiations for float caches: the decode kernels with
// every token's score written out (general kernel: head_dim 64/128, query
// groups 2/4/8; one query head per kv head: head_dim 64/128, block 8/16/32).
#include "pa_decode_mha.cuh"
#include "pa_internal.h"

namespace pa {

const void *scored_kernel_f32(int head_dim, int group) {
#define PA_CASE(D, G)                                                    \
    if (head_dim == D && group == G)                                     \
        return reinterpret_cast<const void *>(&pa_decode_kernel<float, D, G, true>);
    PA_CASE(64, 2) PA_CASE(64, 4) PA_CASE(64, 8)
    PA_CASE(128, 2) PA_CASE(128, 4) PA_CASE(128, 8)
#undef PA_CASE
    return nullptr;
}

const void *scored_mha_kernel_f32(int head_dim, int block_size) {
#define PA_CASE(D, BS)                                                   \
    if (head_dim == D && block_size == BS)                               \
        return reinterpret_cast<const void *>(&pa_decode_mha_kernel<float, D, BS, true>);
    PA_CASE(64, 8) PA_CASE(64, 16) PA_CASE(64, 32)
    PA_CASE(128, 8) PA_CASE(128, 16) PA_CASE(128, 32)
#undef PA_CASE
    return nullptr;
}

}  // namespace pa
