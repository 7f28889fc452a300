// Tree attention: launches (the kernels: pa_tree.cuh).
#include <climits>

#include "pa_tree_tc.cuh"

#include "pa_host.h"
#include "pa_internal.h"
#include "pa_step.h"

namespace pa {

namespace {

template <int R> const void *tree_fn(int head_dim, size_t *smem) {
    *smem = head_dim == 64 ? sizeof(TreeSmem<64, R>) : sizeof(TreeSmem<128, R>);
    return head_dim == 64 ? reinterpret_cast<const void *>(&pa_tree_kernel<64, R>)
                          : reinterpret_cast<const void *>(&pa_tree_kernel<128, R>);
}

pa_status launch_f32(TreeParams &p, int head_dim, int dev, cudaStream_t stream) {
    const int rows = p.num_draft * (p.num_heads / p.num_kv_heads);
    const int R = rows > kTreeRows ? 2 : 1;
    p.row_tiles = (rows + R * kTreeRows - 1) / (R * kTreeRows);
    size_t smem = 0;
    const void *fn = R == 1 ? tree_fn<1>(head_dim, &smem) : tree_fn<2>(head_dim, &smem);
    int per_sm = 0;
    cudaError_t e = prepare_kernel(dev, fn, smem, kTreeThreads, &per_sm);
    if (e != cudaSuccess)
        return cuda_fail(e, "tree kernel set-up");
    const long long items = static_cast<long long>(p.num_seqs) * p.max_parts * p.num_kv_heads * p.row_tiles;
    const long long grid = items < (1 << 30) ? items : (1 << 30);
    void *args[] = {&p};
    e = launch_dependent(fn, dim3(static_cast<unsigned>(grid)), dim3(kTreeThreads), args, smem, stream);
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "tree launch");
}

// 16-bit caches: the tensor-core kernel.  More than 128 rows a kv head: two
// row tiles a CTA, which read each K/V tile once.
pa_status launch_tc(TreeParams &p, int dtype, int head_dim, int dev, int sms, cudaStream_t stream) {
    const int G = p.num_heads / p.num_kv_heads;
    const int rows = p.num_draft * G;
    const int units = rows > 128 ? 2 : 1;
    p.row_tiles = (rows + 128 * units - 1) / (128 * units);
    const int parts = p.out_dtype == PA_F32 ? 2 : 1;
    size_t smem = 0;
    const void *fn = dtype == PA_F16 ? tree_tc_kernel_f16(head_dim, parts, units, &smem)
                                     : tree_tc_kernel_bf16(head_dim, parts, units, &smem);
    if (!fn)
        return fail(PA_ERR_UNSUPPORTED, "no tree kernel for this dtype / head_dim");
    CUtensorMap tmk, tmv, tmq;
    const long long tiles = static_cast<long long>(p.num_blocks) * p.num_kv_heads;
    pa_status st = kv_tensor_map_groups(&tmk, p.k_cache, dtype, p.block_size, tiles, 1, head_dim);
    if (st == PA_OK)
        st = kv_tensor_map_groups(&tmv, p.v_cache, dtype, p.block_size, tiles, 1, head_dim);
    if (st == PA_OK)
        st = tree_q_tensor_map(&tmq, p.q, dtype, head_dim, p.num_heads,
                               static_cast<long long>(p.num_seqs) * p.num_draft, G);
    if (st != PA_OK)
        return st;
    int per_sm = 0;
    cudaError_t e = prepare_kernel(dev, fn, smem, kTcThreads, &per_sm);
    if (e != cudaSuccess)
        return cuda_fail(e, "tree kernel set-up");
    if (per_sm < 1)
        return fail(PA_ERR_UNSUPPORTED, "tree kernel does not fit on an SM");
    const int grid = tree_tc_ctas(p.num_seqs, p.num_kv_heads, rows, p.max_len, sms);
    void *args[] = {&p, &tmk, &tmv, &tmq};
    e = launch_dependent(fn, dim3(grid), dim3(kTcThreads), args, smem, stream);
    if (e != cudaSuccess)
        return cuda_fail(e, "tree launch");
    // a context of one tile is never cut
    if (grid > 1 && p.max_len > 128) {
        const int slot_rows = units == 2 ? tc_slot_rows<2>(rows) : tc_slot_rows<1>(rows);
        const int lrb = tc_merge_log_rows(slot_rows, head_dim);
        const dim3 mgrid(grid, (slot_rows + (1 << lrb) - 1) >> lrb, 2);
        const void *mf = head_dim == 64 ? (units == 2 ? reinterpret_cast<const void *>(&pa_tree_tc_merge_kernel<64, 2>)
                                                      : reinterpret_cast<const void *>(&pa_tree_tc_merge_kernel<64, 1>))
                                        : (units == 2 ? reinterpret_cast<const void *>(&pa_tree_tc_merge_kernel<128, 2>)
                                                      : reinterpret_cast<const void *>(&pa_tree_tc_merge_kernel<128, 1>));
        void *margs[] = {&p};
        e = launch_dependent(mf, mgrid, dim3(kTcMergeThreads), margs, 0, stream);
        if (e != cudaSuccess)
            return cuda_fail(e, "tree merge launch");
    }
    return PA_OK;
}

}  // namespace

// One CTA per SM, no more than there can be units of work.
int tree_tc_ctas(int num_seqs, int num_kv_heads, int rows, int max_len, int sms) {
    const int tile_rows = rows > 128 ? 256 : 128;
    const long long pairs =
        static_cast<long long>(num_seqs) * num_kv_heads * ((rows + tile_rows - 1) / tile_rows);
    const long long tiles = pairs * ((static_cast<long long>(max_len) + 127) / 128);  // (at least)
    const int most = sms < kTreeSms ? sms : kTreeSms;
    return static_cast<int>(tiles < most ? (tiles < 1 ? 1 : tiles) : most);
}

size_t tree_tc_workspace(int num_seqs, int num_kv_heads, int rows, int head_dim, int max_len) {
    const int ctas = tree_tc_ctas(num_seqs, num_kv_heads, rows, max_len, kTreeSms);
    const size_t slot_rows = static_cast<size_t>(rows < 256 ? rows : 256);
    // two partials a CTA, each with a merge record
    return ctas > 1 && max_len > 128
               ? 2 * static_cast<size_t>(ctas) * (slot_rows * (head_dim + 2) * sizeof(float) + sizeof(int4))
               : 0;
}

pa_status launch_tree(TreeParams &p, int dtype, int head_dim, cudaStream_t stream) {
    int dev = 0, sms = 0;
    cudaError_t e = device_sms(&dev, &sms);
    if (e != cudaSuccess)
        return cuda_fail(e, "device query");
    const bool tensor_cores = dtype != PA_F32;
    const pa_status st = tensor_cores ? launch_tc(p, dtype, head_dim, dev, sms, stream)
                                      : launch_f32(p, head_dim, dev, stream);
    if (st != PA_OK)
        return st;
    if (!tensor_cores && p.max_parts > 1) {
        const int rows = p.num_draft * (p.num_heads / p.num_kv_heads);
        const int lrb = tree_merge_log_rows(rows, head_dim);
        const int col_chunks = head_dim / (kTreeMergeCols * (32 >> lrb));  // a power of two
        const long long groups = static_cast<long long>(p.num_seqs) * p.num_kv_heads * ((rows + (1 << lrb) - 1) >> lrb);
        int steps = col_chunks;
        while (steps > 1 && groups * (col_chunks / steps) < 4LL * sms)
            steps /= 2;
        const long long ctas = groups * (col_chunks / steps);
        if (ctas > INT_MAX)
            return fail(PA_ERR_UNSUPPORTED, "num_seqs * num_draft * num_heads too large");
        const void *mf = head_dim == 64 ? reinterpret_cast<const void *>(&pa_tree_merge_kernel<64>)
                                        : reinterpret_cast<const void *>(&pa_tree_merge_kernel<128>);
        void *margs[] = {&p, &steps};
        e = launch_dependent(mf, dim3(static_cast<unsigned>(ctas)), dim3(kTreeMergeThreads), margs, 0, stream);
        if (e != cudaSuccess)
            return cuda_fail(e, "tree merge launch");
    }
    return PA_OK;
}

}  // namespace pa
