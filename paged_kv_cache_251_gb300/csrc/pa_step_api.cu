// C entry points of the serving-step operators: rotary positions, tree
// attention, scored decode, eviction.  Argument checks and launch planning;
// the operations are documented in include/pa.h.
#include <climits>
#include <cmath>

#include "pa.h"
#include "pa_evict.h"
#include "pa_host.h"
#include "pa_internal.h"
#include "pa_rope.h"
#include "pa_step.h"
#include "pa_tree.cuh"

using namespace pa;

namespace {

cudaStream_t stream_of(pa_stream_t stream) { return reinterpret_cast<cudaStream_t>(stream); }

bool elt_aligned(const void *p, int dtype) {
    return (reinterpret_cast<uintptr_t>(p) & (elt_bytes(dtype) - 1)) == 0;
}

// Positions along a context, a score row or a list of kept tokens are 32 bits in
// the kernels, with room for a tile past the end.
constexpr long long kMaxTokens = 1LL << 30;

size_t round16(size_t x) { return (x + 15) & ~static_cast<size_t>(15); }

pa_status rope_args(int num_tokens, int num_heads, int head_dim, int rot_dim, float mscale, int dtype) {
    if (num_tokens < 0 || num_heads <= 0)
        return fail(PA_ERR_INVALID_ARGUMENT, "num_tokens or num_heads out of range");
    if (!head_dim_ok(head_dim))
        return fail(PA_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
    if (rot_dim < 2 || rot_dim > head_dim || rot_dim % 2 != 0)
        return fail(PA_ERR_INVALID_ARGUMENT, "rot_dim must be even and in [2, head_dim]");
    if (!std::isfinite(mscale))
        return fail(PA_ERR_INVALID_ARGUMENT, "mscale must be finite");
    if (!dtype_ok(dtype))
        return fail(PA_ERR_INVALID_ARGUMENT, "unknown dtype");
    return PA_OK;
}

// Checks shared by the decodes of this file, in pa_decode's order.
pa_status decode_args(const void *out, const void *q, const void *k_cache, const void *v_cache,
                      const int32_t *block_tables, const int32_t *context_lens, int num_heads, int num_kv_heads,
                      float scale, int dtype, int out_dtype, int num_blocks) {
    if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens)
        return fail(PA_ERR_INVALID_ARGUMENT, "null pointer");
    if (num_kv_heads <= 0 || num_heads % num_kv_heads != 0)
        return fail(PA_ERR_INVALID_ARGUMENT, "num_heads must be a multiple of num_kv_heads");
    const int G = num_heads / num_kv_heads;
    if (G != 1 && G != 2 && G != 4 && G != 8)
        return fail(PA_ERR_UNSUPPORTED, "num_heads / num_kv_heads must be 1, 2, 4 or 8");
    if (!dtype_ok(dtype) || !dtype_ok(out_dtype))
        return fail(PA_ERR_INVALID_ARGUMENT, "unknown dtype");
    if (num_blocks <= 0)
        return fail(PA_ERR_INVALID_ARGUMENT, "num_blocks must be positive");
    if (!std::isfinite(scale))
        return fail(PA_ERR_INVALID_ARGUMENT, "scale must be finite");
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache))
        return fail(PA_ERR_INVALID_ARGUMENT, "q, k_cache and v_cache must be 16-byte aligned");
    if (!elt_aligned(out, out_dtype))
        return fail(PA_ERR_INVALID_ARGUMENT, "out is not aligned to its element size");
    return PA_OK;
}

void fill_decode(DecodeParams &p, void *out, const void *q, const void *k_cache, const void *v_cache,
                 const int32_t *block_tables, const int32_t *context_lens, int num_seqs, int num_heads,
                 int num_kv_heads, int block_size, float scale, int dtype, int out_dtype, int max_blocks_per_seq,
                 int num_blocks, const DecodePlan &plan, uint32_t *err_word) {
    p.out = out;
    p.q = q;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.part_acc = nullptr;
    p.part_ml = nullptr;
    p.err = err_word;
    p.num_seqs = num_seqs;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.block_size = block_size;
    p.window = 0;
    p.max_blocks_per_seq = max_blocks_per_seq;
    const long long max_len = static_cast<long long>(max_blocks_per_seq) * block_size;
    p.max_len = static_cast<int>(max_len < INT_MAX ? max_len : INT_MAX);
    p.num_blocks = num_blocks;
    p.bpp = plan.bpp;
    p.max_parts = plan.max_parts;
    p.out_dtype = out_dtype;
    p.stages = 0;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.start_tok = nullptr;
    p.force_partial = 0;
    p.q_dtype = dtype;
}

constexpr int kMaxDraft = 256;

// The partitions of the fp32 kernel, and the workspace of the kernel that takes
// the call.
pa_status plan_tree(int num_seqs, int num_draft, int num_heads, int num_kv_heads, int head_dim, int block_size,
                    int max_blocks_per_seq, int dtype, DecodePlan *plan) {
    if (num_draft < 1 || num_draft > kMaxDraft)
        return fail(PA_ERR_INVALID_ARGUMENT, "num_draft must be 1 .. 256");
    if (num_kv_heads <= 0 || num_heads <= 0 || num_heads % num_kv_heads != 0)
        return fail(PA_ERR_INVALID_ARGUMENT, "num_heads must be a positive multiple of num_kv_heads");
    if (!dtype_ok(dtype))
        return fail(PA_ERR_INVALID_ARGUMENT, "unknown dtype");
    const pa_status st = plan_decode(num_seqs, num_heads, head_dim, block_size, max_blocks_per_seq, 0, kTreePartition,
                                     plan);
    if (st != PA_OK)
        return st;
    if (dtype != PA_F32) {
        const long long max_len = static_cast<long long>(max_blocks_per_seq) * block_size;
        plan->workspace =
            tree_tc_workspace(num_seqs, num_kv_heads, num_draft * (num_heads / num_kv_heads), head_dim,
                              static_cast<int>(max_len < INT_MAX ? max_len : INT_MAX));
    } else {
        plan->workspace = plan->max_parts > 1 ? static_cast<size_t>(num_seqs) * num_draft * num_heads *
                                                    plan->max_parts * (head_dim + 2) * sizeof(float)
                                              : 0;
    }
    return PA_OK;
}

// Sizes of the scored decode's workspace: partials, every row's (max,
// denominator) pairs, every query head's scores.
struct ScoredPlan {
    DecodePlan decode;
    size_t acc = 0, ml = 0, logits = 0;
    size_t total() const { return acc + ml + logits; }
};

pa_status plan_scored(int num_seqs, int num_heads, int head_dim, int block_size, int max_blocks_per_seq,
                      int partition_size, ScoredPlan *plan) {
    const pa_status st = plan_decode(num_seqs, num_heads, head_dim, block_size, max_blocks_per_seq, 0, partition_size,
                                     &plan->decode);
    if (st != PA_OK)
        return st;
    const size_t rows = static_cast<size_t>(num_seqs) * num_heads;
    const size_t parts = static_cast<size_t>(plan->decode.max_parts);
    plan->acc = parts > 1 ? rows * parts * head_dim * sizeof(float) : 0;
    plan->ml = round16(rows * parts * 2 * sizeof(float));
    plan->logits = rows * max_blocks_per_seq * block_size * sizeof(float);
    return PA_OK;
}

}  // namespace

extern "C" {

pa_status pa_rope_frequencies(double *freqs, int rot_dim, double base, pa_rope_scaling scaling, double factor,
                              double original_len, double low, double high) {
    g_detail.clear();
    if (!freqs)
        return fail(PA_ERR_INVALID_ARGUMENT, "null pointer");
    if (rot_dim < 2 || rot_dim % 2 != 0)
        return fail(PA_ERR_INVALID_ARGUMENT, "rot_dim must be even and positive");
    if (!(base > 0) || !std::isfinite(base) || !(factor > 0) || !std::isfinite(factor))
        return fail(PA_ERR_INVALID_ARGUMENT, "base and factor must be positive and finite");
    if (scaling != PA_ROPE_PLAIN && scaling != PA_ROPE_LINEAR && scaling != PA_ROPE_BASE && scaling != PA_ROPE_RAMP)
        return fail(PA_ERR_INVALID_ARGUMENT, "unknown scaling");
    if (scaling == PA_ROPE_RAMP &&
        (!(original_len > 0) || !std::isfinite(original_len) || !(low >= 0) || !(high > low) || !std::isfinite(high)))
        return fail(PA_ERR_INVALID_ARGUMENT, "PA_ROPE_RAMP needs original_len > 0 and 0 <= low < high");
    constexpr double kPi = 3.14159265358979323846;
    if (scaling == PA_ROPE_BASE && rot_dim > 2)
        base *= std::pow(factor, static_cast<double>(rot_dim) / (rot_dim - 2));
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rot_dim);
        if (scaling == PA_ROPE_LINEAR) {
            f /= factor;
        } else if (scaling == PA_ROPE_RAMP) {
            const double turns = original_len * f / (2 * kPi);
            double keep = (turns - low) / (high - low);
            keep = keep < 0 ? 0 : (keep > 1 ? 1 : keep);
            f *= keep + (1 - keep) / factor;
        }
        freqs[i] = f;
    }
    return PA_OK;
}

pa_status pa_rope(void *out, const void *x, const int32_t *positions, const double *freqs, int num_tokens,
                  int num_heads, int head_dim, int rot_dim, long long x_stride, long long out_stride, int interleaved,
                  int direction, float mscale, pa_dtype dtype, pa_stream_t stream) {
    g_detail.clear();
    const pa_status st = rope_args(num_tokens, num_heads, head_dim, rot_dim, mscale, dtype);
    if (st != PA_OK)
        return st;
    if (direction != 1 && direction != -1)
        return fail(PA_ERR_INVALID_ARGUMENT, "direction must be 1 or -1");
    const long long width = static_cast<long long>(num_heads) * head_dim;
    if (x_stride < width || out_stride < width)
        return fail(PA_ERR_INVALID_ARGUMENT, "a row stride is smaller than num_heads * head_dim");
    if (num_tokens == 0)
        return PA_OK;
    if (!out || !x || !positions || !freqs)
        return fail(PA_ERR_INVALID_ARGUMENT, "null pointer");
    if (!elt_aligned(out, dtype) || !elt_aligned(x, dtype))
        return fail(PA_ERR_INVALID_ARGUMENT, "x or out is not aligned to its element size");
    if (out == x && out_stride != x_stride)
        return fail(PA_ERR_INVALID_ARGUMENT, "in place needs equal strides");
    RopeParams p = {};
    p.q = x;
    p.q_out = out;
    p.positions = positions;
    p.freqs = freqs;
    p.num_tokens = num_tokens;
    p.q_stride = x_stride;
    p.q_out_stride = out_stride;
    p.num_heads = num_heads;
    p.head_dim = head_dim;
    p.rot = rot_dim;
    p.direction = direction;
    p.mscale = mscale;
    p.block_size = 1;
    int dev = 0, sms = 0;
    cudaError_t e = device_sms(&dev, &sms);
    if (e != cudaSuccess)
        return cuda_fail(e, "device query");
    e = launch_rope(p, dtype, interleaved, sms, stream_of(stream));
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "rope launch");
}

pa_status pa_rope_append_kv(void *q_out, const void *q, const void *k, const void *v, const int32_t *positions,
                            const int64_t *slot_mapping, const double *freqs, void *k_cache, void *v_cache,
                            int num_tokens, int num_heads, int num_kv_heads, int head_dim, int rot_dim,
                            long long q_stride, long long k_stride, long long v_stride, int block_size,
                            int num_blocks, int interleaved, float mscale, pa_dtype dtype, uint32_t *err_word,
                            pa_stream_t stream) {
    g_detail.clear();
    const pa_status st = rope_args(num_tokens, num_heads, head_dim, rot_dim, mscale, dtype);
    if (st != PA_OK)
        return st;
    if (num_kv_heads <= 0 || num_blocks <= 0)
        return fail(PA_ERR_INVALID_ARGUMENT, "num_kv_heads or num_blocks out of range");
    if (!block_size_ok(block_size))
        return fail(PA_ERR_UNSUPPORTED, "block_size must be 8, 16 or 32");
    const long long width = static_cast<long long>(num_heads) * head_dim;
    const long long kv_width = static_cast<long long>(num_kv_heads) * head_dim;
    if (q_stride < width || k_stride < kv_width || v_stride < kv_width)
        return fail(PA_ERR_INVALID_ARGUMENT, "a row stride is smaller than the row");
    if (num_tokens == 0)
        return PA_OK;
    if (!q_out || !q || !k || !v || !positions || !slot_mapping || !freqs || !k_cache || !v_cache)
        return fail(PA_ERR_INVALID_ARGUMENT, "null pointer");
    if (!aligned16(k_cache) || !aligned16(v_cache))
        return fail(PA_ERR_INVALID_ARGUMENT, "the caches must be 16-byte aligned");
    if (!elt_aligned(q_out, dtype) || !elt_aligned(q, dtype) || !elt_aligned(k, dtype) || !elt_aligned(v, dtype))
        return fail(PA_ERR_INVALID_ARGUMENT, "q, k, v or q_out is not aligned to its element size");
    if ((reinterpret_cast<uintptr_t>(slot_mapping) & 7u) != 0)
        return fail(PA_ERR_INVALID_ARGUMENT, "slot_mapping must be 8-byte aligned");
    if (q_out == q && q_stride != width)
        return fail(PA_ERR_INVALID_ARGUMENT, "q_out may be q only when q is dense");
    RopeParams p = {};
    p.q = q;
    p.q_out = q_out;
    p.k = k;
    p.v = v;
    p.positions = positions;
    p.freqs = freqs;
    p.slots = slot_mapping;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.err = err_word;
    p.num_tokens = num_tokens;
    p.q_stride = q_stride;
    p.q_out_stride = width;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.head_dim = head_dim;
    p.rot = rot_dim;
    p.block_size = block_size;
    p.num_blocks = num_blocks;
    p.direction = 1;
    p.mscale = mscale;
    int dev = 0, sms = 0;
    cudaError_t e = device_sms(&dev, &sms);
    if (e != cudaSuccess)
        return cuda_fail(e, "device query");
    e = launch_rope(p, dtype, interleaved, sms, stream_of(stream));
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "rope append launch");
}

size_t pa_decode_tree_workspace_size(int num_seqs, int num_draft, int num_heads, int num_kv_heads, int head_dim,
                                     int block_size, int max_blocks_per_seq, pa_dtype dtype) {
    DecodePlan plan;
    if (plan_tree(num_seqs, num_draft, num_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq, dtype,
                  &plan) != PA_OK)
        return 0;
    return plan.workspace;
}

pa_status pa_decode_tree(void *out, const void *q, const void *k_cache, const void *v_cache,
                         const int32_t *block_tables, const int32_t *context_lens, const int32_t *draft_lens,
                         const uint64_t *tree_mask, int num_seqs, int num_draft, int num_heads, int num_kv_heads,
                         int head_dim, int block_size, float scale, pa_dtype dtype, pa_dtype out_dtype,
                         int max_blocks_per_seq, int num_blocks, void *workspace, size_t workspace_bytes,
                         uint32_t *err_word, pa_stream_t stream) {
    g_detail.clear();
    DecodePlan plan;
    pa_status st = plan_tree(num_seqs, num_draft, num_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq,
                             dtype, &plan);
    if (st != PA_OK)
        return st;
    if (num_seqs == 0)
        return PA_OK;
    st = decode_args(out, q, k_cache, v_cache, block_tables, context_lens, num_heads, num_kv_heads, scale, dtype,
                     out_dtype, num_blocks);
    if (st != PA_OK)
        return st;
    if (static_cast<long long>(max_blocks_per_seq) * block_size > kMaxTokens)
        return fail(PA_ERR_UNSUPPORTED, "max_blocks_per_seq * block_size is above 2^30");
    // the tensor maps of 16-bit caches address (block, kv head) tiles by 32 bits
    if (dtype != PA_F32 && static_cast<long long>(num_blocks) * num_kv_heads > INT_MAX)
        return fail(PA_ERR_UNSUPPORTED, "num_blocks * num_kv_heads is above 2^31 - 1");
    if ((reinterpret_cast<uintptr_t>(tree_mask) & 7u) != 0)
        return fail(PA_ERR_INVALID_ARGUMENT, "tree_mask must be 8-byte aligned");
    if (plan.workspace > 0 && (workspace == nullptr || workspace_bytes < plan.workspace))
        return fail(PA_ERR_WORKSPACE_TOO_SMALL, "workspace smaller than pa_decode_tree_workspace_size()");
    if (plan.workspace > 0 && !aligned16(workspace))
        return fail(PA_ERR_INVALID_ARGUMENT, "workspace must be 16-byte aligned");
    const long long rows = static_cast<long long>(num_seqs) * num_draft * num_heads;
    if (rows > INT_MAX)
        return fail(PA_ERR_UNSUPPORTED, "num_seqs * num_draft * num_heads too large");
    TreeParams p;
    fill_decode(p, out, q, k_cache, v_cache, block_tables, context_lens, num_seqs, num_heads, num_kv_heads, block_size,
                scale, dtype, out_dtype, max_blocks_per_seq, num_blocks, plan, err_word);
    p.draft_lens = draft_lens;
    p.mask = tree_mask;
    p.num_draft = num_draft;
    p.words = (num_draft + 63) / 64;
    p.row_tiles = 0;
    p.cuts = nullptr;
    if (plan.workspace > 0) {
        if (dtype != PA_F32) {
            // merge records, accumulators, (max, denominator) pairs
            const int tree_rows = num_draft * (num_heads / num_kv_heads);
            const size_t ctas = tree_tc_ctas(num_seqs, num_kv_heads, tree_rows, p.max_len, kTreeSms);
            p.cuts = static_cast<int4 *>(workspace);
            p.part_acc = reinterpret_cast<float *>(p.cuts + 2 * ctas);
            p.part_ml = p.part_acc + 2 * ctas * (tree_rows < 256 ? tree_rows : 256) * head_dim;
        } else {
            p.part_acc = static_cast<float *>(workspace);
            p.part_ml = p.part_acc + rows * plan.max_parts * head_dim;
        }
    }
    return launch_tree(p, dtype, head_dim, stream_of(stream));
}

size_t pa_decode_scored_workspace_size(int num_seqs, int num_heads, int head_dim, int block_size,
                                       int max_blocks_per_seq, int partition_size) {
    ScoredPlan plan;
    if (plan_scored(num_seqs, num_heads, head_dim, block_size, max_blocks_per_seq, partition_size, &plan) != PA_OK)
        return 0;
    return plan.total();
}

pa_status pa_decode_scored(void *out, float *scores_out, const float *scores_in, const void *q, const void *k_cache,
                           const void *v_cache, const int32_t *block_tables, const int32_t *context_lens,
                           int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size, float scale,
                           long long scores_stride, pa_dtype dtype, pa_dtype out_dtype, int max_blocks_per_seq,
                           int num_blocks, int partition_size, void *workspace, size_t workspace_bytes,
                           uint32_t *err_word, pa_stream_t stream) {
    g_detail.clear();
    ScoredPlan need;  // of the workspace: partition_size 0 sizes for the shorter default, which covers both
    pa_status st = plan_scored(num_seqs, num_heads, head_dim, block_size, max_blocks_per_seq, partition_size, &need);
    if (st != PA_OK)
        return st;
    if (partition_size == 0 && gqa_tensor_core_path(num_heads, num_kv_heads, head_dim, dtype))
        partition_size = kGqaDefaultPartition;
    ScoredPlan plan;
    st = plan_scored(num_seqs, num_heads, head_dim, block_size, max_blocks_per_seq, partition_size, &plan);
    if (st != PA_OK)
        return st;
    if (num_seqs == 0)
        return PA_OK;
    st = decode_args(out, q, k_cache, v_cache, block_tables, context_lens, num_heads, num_kv_heads, scale, dtype,
                     out_dtype, num_blocks);
    if (st != PA_OK)
        return st;
    const long long max_len = static_cast<long long>(max_blocks_per_seq) * block_size;
    if (!scores_out || !elt_aligned(scores_out, PA_F32) || !elt_aligned(scores_in, PA_F32))
        return fail(PA_ERR_INVALID_ARGUMENT, "scores_out is null, or a score array is not 4-byte aligned");
    if (max_len > kMaxTokens)
        return fail(PA_ERR_UNSUPPORTED, "max_blocks_per_seq * block_size is above 2^30");
    if (scores_stride < max_len)
        return fail(PA_ERR_INVALID_ARGUMENT, "scores_stride smaller than max_blocks_per_seq * block_size");
    if (num_kv_heads > 65535)
        return fail(PA_ERR_UNSUPPORTED, "num_kv_heads too large");
    // the tensor maps address (block, kv head) tiles and query rows by 32 bits
    if (static_cast<long long>(num_blocks) * num_kv_heads > INT_MAX)
        return fail(PA_ERR_UNSUPPORTED, "num_blocks * num_kv_heads is above 2^31 - 1");
    if (static_cast<long long>(num_seqs) * num_heads > INT_MAX)
        return fail(PA_ERR_UNSUPPORTED, "num_seqs * num_heads is above 2^31 - 1");
    if (workspace == nullptr || workspace_bytes < need.total())
        return fail(PA_ERR_WORKSPACE_TOO_SMALL, "workspace smaller than pa_decode_scored_workspace_size()");
    if (!aligned16(workspace))
        return fail(PA_ERR_INVALID_ARGUMENT, "workspace must be 16-byte aligned");
    DecodeParams p;
    fill_decode(p, out, q, k_cache, v_cache, block_tables, context_lens, num_seqs, num_heads, num_kv_heads, block_size,
                scale, dtype, out_dtype, max_blocks_per_seq, num_blocks, plan.decode, err_word);
    char *ws = static_cast<char *>(workspace);
    p.part_acc = plan.acc ? reinterpret_cast<float *>(ws) : nullptr;
    p.part_ml = reinterpret_cast<float *>(ws + plan.acc);
    p.logits = reinterpret_cast<float *>(ws + plan.acc + plan.ml);
    p.logits_stride = max_len;
    const cudaStream_t cs = stream_of(stream);
    st = launch_decode_kernel(p, dtype, head_dim, num_heads / num_kv_heads, cs);
    if (st != PA_OK)
        return st;
    int dev = 0, sms = 0;
    cudaError_t e = device_sms(&dev, &sms);
    if (e == cudaSuccess && plan.decode.max_parts > 1)
        e = launch_reduce(p, head_dim, static_cast<long long>(num_seqs) * num_heads, cs);
    if (e == cudaSuccess)
        e = launch_scores(p, scores_in, scores_out, scores_stride, sms, cs);
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "score launch");
}

pa_status pa_evict_select(int32_t *keep, int32_t *new_lens, float *scores_out, const float *scores,
                          const int32_t *context_lens, int num_seqs, int num_kv_heads, int budget, int recent,
                          long long scores_stride, uint32_t *err_word, pa_stream_t stream) {
    g_detail.clear();
    if (num_seqs < 0 || num_kv_heads <= 0 || scores_stride <= 0)
        return fail(PA_ERR_INVALID_ARGUMENT, "num_seqs, num_kv_heads or scores_stride out of range");
    if (budget < 1 || recent < 0 || recent > budget)
        return fail(PA_ERR_INVALID_ARGUMENT, "budget must be positive and recent in [0, budget]");
    if (scores_stride > kMaxTokens || budget > kMaxTokens)
        return fail(PA_ERR_UNSUPPORTED, "scores_stride or budget is above 2^30");
    if (num_seqs == 0)
        return PA_OK;
    if (!keep || !new_lens || !scores || !context_lens)
        return fail(PA_ERR_INVALID_ARGUMENT, "null pointer");
    if (!elt_aligned(scores, PA_F32) || !elt_aligned(scores_out, PA_F32) || !elt_aligned(keep, PA_F32) ||
        !elt_aligned(new_lens, PA_F32))
        return fail(PA_ERR_INVALID_ARGUMENT, "an array is not 4-byte aligned");
    SelectParams p = {};
    p.keep = keep;
    p.new_lens = new_lens;
    p.scores_out = scores_out;
    p.scores = scores;
    p.context_lens = context_lens;
    p.err = err_word;
    p.stride = scores_stride;
    p.max_len = scores_stride;
    p.num_seqs = num_seqs;
    p.num_kv_heads = num_kv_heads;
    p.budget = budget;
    p.recent = recent;
    int dev = 0, sms = 0;
    cudaError_t e = device_sms(&dev, &sms);
    if (e != cudaSuccess)
        return cuda_fail(e, "device query");
    e = launch_select(p, sms, stream_of(stream));
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "select launch");
}

pa_status pa_compact_kv(void *k_cache, void *v_cache, const int32_t *keep, const int32_t *keep_lens,
                        const int32_t *base_lens, const int32_t *block_tables, const int32_t *dst_block_tables,
                        int num_seqs, int keep_heads, int keep_stride, int num_kv_heads, int head_dim, int block_size,
                        int max_blocks_per_seq, int dst_max_blocks_per_seq, int num_blocks, pa_dtype dtype,
                        uint32_t *err_word, pa_stream_t stream) {
    g_detail.clear();
    if (num_seqs < 0 || num_kv_heads <= 0 || keep_stride < 0 || max_blocks_per_seq <= 0 || num_blocks <= 0)
        return fail(PA_ERR_INVALID_ARGUMENT,
                    "num_seqs, num_kv_heads, keep_stride, max_blocks_per_seq or num_blocks out of range");
    if (keep_heads != 1 && keep_heads != num_kv_heads)
        return fail(PA_ERR_INVALID_ARGUMENT, "keep_heads must be 1 or num_kv_heads");
    if (!block_size_ok(block_size))
        return fail(PA_ERR_UNSUPPORTED, "block_size must be 8, 16 or 32");
    if (!head_dim_ok(head_dim))
        return fail(PA_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
    if (!dtype_ok(dtype))
        return fail(PA_ERR_INVALID_ARGUMENT, "unknown dtype");
    if (dst_block_tables && dst_max_blocks_per_seq <= 0)
        return fail(PA_ERR_INVALID_ARGUMENT, "dst_max_blocks_per_seq must be positive");
    if (num_kv_heads > 65535)
        return fail(PA_ERR_UNSUPPORTED, "num_kv_heads too large");
    if (keep_stride > kMaxTokens)
        return fail(PA_ERR_UNSUPPORTED, "keep_stride is above 2^30");
    if (num_seqs == 0 || keep_stride == 0)
        return PA_OK;
    if (!k_cache || !v_cache || !keep || !keep_lens || !block_tables)
        return fail(PA_ERR_INVALID_ARGUMENT, "null pointer");
    if (!aligned16(k_cache) || !aligned16(v_cache))
        return fail(PA_ERR_INVALID_ARGUMENT, "the caches must be 16-byte aligned");
    CompactParams p = {};
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.keep = keep;
    p.keep_lens = keep_lens;
    p.base_lens = base_lens;
    p.block_tables = block_tables;
    const bool in_place = dst_block_tables == nullptr || dst_block_tables == block_tables;
    p.dst_block_tables = in_place ? block_tables : dst_block_tables;
    p.err = err_word;
    p.num_seqs = num_seqs;
    p.keep_heads = keep_heads;
    p.keep_stride = keep_stride;
    p.num_kv_heads = num_kv_heads;
    p.block_size = block_size;
    p.max_blocks = max_blocks_per_seq;
    p.dst_max_blocks = in_place ? max_blocks_per_seq : dst_max_blocks_per_seq;
    p.num_blocks = num_blocks;
    p.row_chunks = head_dim * elt_bytes(dtype) / 16;
    const cudaError_t e = launch_compact(p, in_place, stream_of(stream));
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "compact launch");
}

}  // extern "C"
