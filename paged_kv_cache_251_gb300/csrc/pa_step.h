// Launches of the serving-step operators (pa_step_api.cu calls them).
#pragma once

#include <cuda_runtime.h>

#include "pa.h"

namespace pa {

struct DecodeParams;
struct TreeParams;

// The score pass of the scored decode, after the decode and its merge.
cudaError_t launch_scores(DecodeParams &p, const float *in, float *out, long long stride, int sms,
                          cudaStream_t stream);

// CTAs of the tensor-core tree attention: one per SM, at most this many (the
// workspace is sized for them).
constexpr int kTreeSms = 152;

// How many CTAs the tree attention of 16-bit caches has on a device of `sms`
// SMs, and its workspace (two partials for each of kTreeSms CTAs).
int tree_tc_ctas(int num_seqs, int num_kv_heads, int rows, int max_len, int sms);
size_t tree_tc_workspace(int num_seqs, int num_kv_heads, int rows, int head_dim, int max_len);

// The tree attention of filled-in parameters (the row tiles are set there).
pa_status launch_tree(TreeParams &p, int dtype, int head_dim, cudaStream_t stream);

}  // namespace pa
