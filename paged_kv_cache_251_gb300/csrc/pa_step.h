// Launches of the serving-step operators (pa_step_api.cu calls them).
#pragma once

#include <cuda_runtime.h>

#include "pa.h"

namespace pa {

struct DecodeParams;
struct TreeParams;

// The score pass of the scored decode, after the decode and its merge.
cudaError_t launch_scores(DecodeParams &p, const float *in, float *out, long long stride, cudaStream_t stream);

// The tree attention of filled-in parameters (the row tiles are set there).
pa_status launch_tree(TreeParams &p, int dtype, int head_dim, cudaStream_t stream);

}  // namespace pa
