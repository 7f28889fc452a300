// Parameters of the page-table kernels (pa_pages.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pa {

struct PagesUpdateParams {
    int32_t *new_tables;  // [rows][max_blocks]
    int32_t *new_refs;    // [num_blocks]; may be refs
    int64_t *pairs;       // [rows][2]
    int32_t *status;      // [4]
    const int32_t *tables, *refs, *lens, *parents, *keep, *grow;
    // workspace
    int32_t *count, *first, *writers, *free_list;  // [num_blocks]
    int32_t *kept, *total;                         // [rows]: blocks kept, blocks in all
    int32_t *need;                                 // [rows]; bit 31: the last kept block is copied
    int32_t *base;                                 // [rows]: the row's first place in free_list
    uint32_t *err;
    int rows, old_rows, max_blocks, num_blocks, block_size;
};

struct PagesCompactParams {
    int32_t *new_tables;  // [rows][max_blocks]; may be tables
    int32_t *new_refs;    // [num_blocks]; may be refs
    int32_t *remap;       // [num_blocks]
    int64_t *pairs;       // [max_moves][2]
    int32_t *status;      // [4]
    const int32_t *tables, *refs, *lens;
    int32_t *src_list, *dst_list;  // workspace, [num_blocks] each
    int32_t *place;                // workspace, [num_blocks] (with err): remap, ~b of blocks without a count
    uint32_t *err;
    int rows, max_blocks, num_blocks, block_size, max_moves;
};

constexpr int kMaxPools = 8;

struct CopyPagesParams {
    const int64_t *pairs;
    char *pool[kMaxPools];
    long long block_bytes[kMaxPools];
    uint32_t *err;
    long long num_blocks;
    int num_pairs, num_pools;
};

cudaError_t launch_pages_update(PagesUpdateParams p, cudaStream_t stream);
cudaError_t launch_pages_compact(PagesCompactParams p, cudaStream_t stream);
cudaError_t launch_copy_pages(CopyPagesParams p, int num_sms, cudaStream_t stream);

}  // namespace pa
