// Parameters of the verification of drafted tokens (pa_verify.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pa {

constexpr int kVerifyMaxDraft = 256;

struct VerifyParams {
    int32_t *accept_lens;  // [num_seqs]
    int32_t *accepted;     // [num_seqs][num_draft]
    int32_t *tokens;       // [num_seqs][num_draft + 1]
    const void *target;    // [num_seqs][num_draft + 1] rows, target_stride elements apart
    const void *draft;     // [num_seqs][num_draft] rows, draft_stride elements apart, or nullptr
    const int32_t *draft_tokens;
    const int32_t *draft_lens;  // [num_seqs] or nullptr
    const int32_t *parents;     // [num_seqs][num_draft] or nullptr
    const float *uniforms;      // [num_seqs][num_draft + 1]
    uint32_t *err;
    long long target_stride, draft_stride;
    int num_seqs, num_draft, vocab;
    int cluster;  // CTAs of a sequence (set by the launch)
    int slice;    // entries of a warp (set by the launch)
};

cudaError_t launch_verify(VerifyParams p, int dtype, int num_sms, cudaStream_t stream);

}  // namespace pa
