// Parameters of the block-scaled 8-bit cache: append (pa_block_quant.cu) and
// decode (pa_decode_bq.cuh).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pa {

struct AppendBqParams {
    const void *k, *v;  // [num_tokens][num_kv_heads][head_dim]
    const int64_t *slots;
    uint8_t *k_cache, *v_cache;  // [num_blocks][num_kv_heads][block_size][head_dim]
    float *k_scales, *v_scales;  // [num_blocks][num_kv_heads]
    // workspace (many tokens only)
    int32_t *token_of;      // [num_blocks * block_size]
    int32_t *list, *listed;  // [min(num_tokens, num_blocks)] blocks that the call writes; their number
    uint32_t *err;
    long long pool_slots;
    int num_tokens, num_kv_heads, block_size;
    int parts;  // (few tokens) warps that share a token's (kv head, K or V) units (set by the launch)
};

// Tokens up to which an append finds the tokens of a block by looking at all of
// them (no workspace, two kernels less).  bf16, 8 heads of 128, on the GPU, so and with the
// list: 64 single rows 3.3 and 8.0 us, 256 5.6 and 9.4, 512 10.2 and 11.1, 1024 18.3 and
// 14.4; a prompt of 512 6.0 and 6.5, of 1024 8.8 and 7.0.
constexpr int kAppendBqFew = 512;

cudaError_t launch_append_bq(AppendBqParams p, int dtype, int cache_dtype, int head_dim, int num_sms,
                             cudaStream_t stream);

struct DecodeBqParams {
    void *out;
    const void *q;
    const uint8_t *k_cache, *v_cache;
    const float *k_scales, *v_scales;
    const int32_t *block_tables, *context_lens;
    // workspace: two partials a CTA, and a record a CTA
    int4 *records;    // [CTAs]: {sequence, kv head, last CTA, 1} of a cut piece that begins there, else {.., 0}
    float *part_acc;  // [CTAs][2][group][head_dim]
    float *part_ml;   // [CTAs][2][group][2]
    uint32_t *err;
    int num_seqs, num_heads, num_kv_heads, block_size, log_block, window, max_blocks, max_len, num_blocks;
    int q_dtype, out_dtype;
    int by_piece;      // a CTA a (sequence, kv head), none cut between CTAs (set by the launch)
    float scale_log2;  // scale * log2 e
};

// CTAs of the block-scaled decode: kDecodeBqCtas an SM, of at most kDecodeBqSms SMs
// (the workspace is sized for them).
constexpr int kDecodeBqThreads = 128;
constexpr int kDecodeBqWarps = kDecodeBqThreads / 32;
constexpr int kDecodeBqCtas = 3;
constexpr int kDecodeBqSms = 152;
constexpr int kDecodeBqMaxCtas = kDecodeBqSms * kDecodeBqCtas;

// Kernel of (group <= 4 or 8, fp32 queries or not, block size 8 or not).
const void *decode_bq_kernel_i8_64(bool wide, bool f32, bool b8);
const void *decode_bq_kernel_i8_128(bool wide, bool f32, bool b8);
const void *decode_bq_kernel_e4m3_64(bool wide, bool f32, bool b8);
const void *decode_bq_kernel_e4m3_128(bool wide, bool f32, bool b8);

// Sequences times kv heads times the table's tokens bound the CTAs of a call.
int decode_bq_ctas(int num_seqs, int num_kv_heads, int max_len);

cudaError_t launch_decode_bq(DecodeBqParams p, int cache_dtype, int head_dim, int num_sms, cudaStream_t stream);

}  // namespace pa
