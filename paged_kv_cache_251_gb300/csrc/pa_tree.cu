// Tree attention: launches (the kernels: pa_tree.cuh).
#include "pa_tree.cuh"

#include "pa_host.h"
#include "pa_internal.h"
#include "pa_step.h"

namespace pa {

namespace {

template <typename T> const void *tree_fn(int head_dim) {
    return head_dim == 64 ? reinterpret_cast<const void *>(&pa_tree_kernel<T, 64>)
                          : reinterpret_cast<const void *>(&pa_tree_kernel<T, 128>);
}

}  // namespace

pa_status launch_tree(TreeParams &p, int dtype, int head_dim, cudaStream_t stream) {
    int dev = 0, sms = 0, per_sm = 0;
    cudaError_t e = device_sms(&dev, &sms);
    if (e != cudaSuccess)
        return cuda_fail(e, "device query");
    const int G = p.num_heads / p.num_kv_heads;
    p.row_tiles = (p.num_draft * G + kTreeRows - 1) / kTreeRows;
    const void *fn = dtype == PA_F32   ? tree_fn<float>(head_dim)
                     : dtype == PA_F16 ? tree_fn<__half>(head_dim)
                                       : tree_fn<__nv_bfloat16>(head_dim);
    const size_t smem = static_cast<size_t>(2) * p.block_size * head_dim * sizeof(float);
    e = prepare_kernel(dev, fn, smem, kTreeThreads, &per_sm);
    if (e != cudaSuccess)
        return cuda_fail(e, "tree kernel set-up");
    const long long items =
        static_cast<long long>(p.num_seqs) * p.max_parts * p.num_kv_heads * p.row_tiles;
    const long long grid = items < (1 << 30) ? items : (1 << 30);
    void *args[] = {&p};
    e = launch_dependent(fn, dim3(static_cast<unsigned>(grid)), dim3(kTreeThreads), args, smem, stream);
    if (e != cudaSuccess)
        return cuda_fail(e, "tree launch");
    if (p.max_parts > 1) {
        const long long rows = static_cast<long long>(p.num_seqs) * p.num_draft * p.num_heads;
        constexpr int kRows = kTreeMergeThreads / 32;
        const void *mf = head_dim == 64 ? reinterpret_cast<const void *>(&pa_tree_merge_kernel<64>)
                                        : reinterpret_cast<const void *>(&pa_tree_merge_kernel<128>);
        e = launch_dependent(mf, dim3(static_cast<unsigned>((rows + kRows - 1) / kRows)), dim3(kTreeMergeThreads),
                             args, 0, stream);
        if (e != cudaSuccess)
            return cuda_fail(e, "tree merge launch");
    }
    return PA_OK;
}

}  // namespace pa
