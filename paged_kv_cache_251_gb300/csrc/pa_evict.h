// Parameters of the eviction kernels (pa_evict.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pa {

struct SelectParams {
    int32_t *keep;      // [num_seqs][num_kv_heads][budget]
    int32_t *new_lens;  // [num_seqs]
    float *scores_out;  // [num_seqs][num_kv_heads][stride] or nullptr
    const float *scores;
    const int32_t *context_lens;
    uint32_t *err;
    long long stride, max_len;  // max_len: the longest context a row holds
    int num_seqs, num_kv_heads, budget, recent;
    int cluster;  // CTAs of a row (set by the launch)
};

struct CompactParams {
    void *k_cache, *v_cache;
    const int32_t *keep, *keep_lens, *base_lens, *block_tables, *dst_block_tables;
    uint32_t *err;
    int num_seqs, keep_heads, keep_stride, num_kv_heads, block_size, max_blocks, dst_max_blocks, num_blocks;
    int row_chunks;  // 16-byte chunks of a row: 8, 16 or 32
    int log_block;   // set by the launch
};

cudaError_t launch_select(SelectParams p, int num_sms, cudaStream_t stream);
cudaError_t launch_compact(CompactParams p, bool in_place, cudaStream_t stream);

}  // namespace pa
