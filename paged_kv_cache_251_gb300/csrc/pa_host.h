// Host helpers shared by the translation units that hold C entry points:
// errors, argument checks, launch planning, tensor maps.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <string>

#include "pa.h"

namespace pa {

struct DecodeParams;

// The detail text of the last error on the calling thread.
extern thread_local std::string g_detail;
pa_status fail(pa_status st, const std::string &why);
pa_status cuda_fail(cudaError_t e, const char *what);

inline int elt_bytes(int dtype) { return dtype == PA_F32 ? 4 : 2; }
inline bool dtype_ok(int dtype) { return dtype == PA_F32 || dtype == PA_F16 || dtype == PA_BF16; }
inline bool code_dtype_ok(int dtype) { return dtype == PA_I8 || dtype == PA_E4M3; }
inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool block_size_ok(int bs) { return bs == 8 || bs == 16 || bs == 32; }
inline bool head_dim_ok(int d) { return d == 64 || d == 128; }

// The current device and its SM count.
cudaError_t device_sms(int *dev, int *sms);
// Shared-memory opt-in and resident CTAs per SM of a kernel (cached).
cudaError_t prepare_kernel(int dev, const void *fn, size_t smem, int threads, int *blocks_per_sm);

// Tensor maps (see their definitions).
pa_status kv_tensor_map(CUtensorMap *map, const void *base, int dtype, int head_dim, int block_size,
                        long long tiles);
pa_status kv_tensor_map_groups(CUtensorMap *map, const void *base, int dtype, int block_size, long long tiles,
                               int box_tiles = 1, int head_dim = 128);
pa_status tree_q_tensor_map(CUtensorMap *map, const void *base, int dtype, int head_dim, int heads, long long tokens,
                            int group);

// Context partitions of a decode.
struct DecodePlan {
    int bpp = 0;
    int max_parts = 0;
    size_t workspace = 0;
};

constexpr int kDefaultPartition = 512;
// The tensor-core kernels (grouped heads over 16-bit K/V, and over E4M3
// pages) pay more per item (query load, the merge of the quarters, partials):
// their default partition is twice as long.  pa_decode_workspace_size(..., 0) sizes for the shorter one, which
// needs at least as much.
constexpr int kGqaDefaultPartition = 1024;

pa_status plan_decode(int num_seqs, int num_heads, int head_dim, int block_size, int max_blocks_per_seq, int window,
                      int partition_size, DecodePlan *plan);
bool gqa_tensor_core_path(int num_heads, int num_kv_heads, int head_dim, int dtype);
cudaError_t launch_reduce(DecodeParams &p, int head_dim, long long rows, cudaStream_t cs);

}  // namespace pa
