// Tensor-core tree attention instantiations for __nv_bfloat16 caches (head_dim
// 64/128, one or two row tiles a CTA, P in one or two parts).
#include "pa_internal.h"
#include "pa_tree_tc.cuh"

namespace pa {

const void *tree_tc_kernel_bf16(int head_dim, int parts, int units, size_t *smem) {
#define PA_CASE(D, PARTS, UNITS)                                                                    \
    if (head_dim == D && parts == PARTS && units == UNITS) {                                        \
        *smem = tc_smem<D, UNITS>();                                                                \
        return reinterpret_cast<const void *>(&pa_tree_tc_kernel<__nv_bfloat16, D, PARTS, UNITS>);           \
    }
    PA_CASE(64, 1, 1) PA_CASE(64, 1, 2) PA_CASE(64, 2, 1) PA_CASE(64, 2, 2)
    PA_CASE(128, 1, 1) PA_CASE(128, 1, 2) PA_CASE(128, 2, 1) PA_CASE(128, 2, 2)
#undef PA_CASE
    return nullptr;
}

}  // namespace pa
