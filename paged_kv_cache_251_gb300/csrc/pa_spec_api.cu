// C entry points of the verification of drafted tokens, the block-scaled 8-bit
// cache, and the page tables on the device.  Argument checks and launch planning;
// the operations are documented in include/pa.h.
#include <climits>
#include <cmath>

#include "pa.h"
#include "pa_block_quant.h"
#include "pa_host.h"
#include "pa_internal.h"
#include "pa_pages.h"
#include "pa_verify.h"

using namespace pa;

namespace {

cudaStream_t stream_of(pa_stream_t stream) { return reinterpret_cast<cudaStream_t>(stream); }

bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

size_t round16(size_t x) { return (x + 15) & ~static_cast<size_t>(15); }

// Positions along a context or a vocabulary are 32 bits in the kernels, with room
// for a tile past the end.
constexpr long long kMaxTokens = 1LL << 30;
// What 1024 rows need is summed in 32 bits.
constexpr int kMaxRowBlocks = (1 << 21) - 1;

// Counts of the pages' lists and tables are 32 bits, rows times blocks 64.
constexpr int kPagesArrays = 4;  // of num_blocks (and as many of num_rows)

pa_status pages_args(int num_rows, int max_blocks_per_seq, int block_size, int num_blocks) {
    if (num_rows < 0 || max_blocks_per_seq <= 0 || block_size <= 0 || num_blocks <= 0)
        return fail(PA_ERR_INVALID_ARGUMENT, "num_rows, max_blocks_per_seq, block_size or num_blocks out of range");
    if (static_cast<long long>(max_blocks_per_seq) * block_size > kMaxTokens)
        return fail(PA_ERR_UNSUPPORTED, "max_blocks_per_seq * block_size is above 2^30");
    if (max_blocks_per_seq > kMaxRowBlocks)
        return fail(PA_ERR_UNSUPPORTED, "max_blocks_per_seq is above 2^21 - 1");
    if (num_rows > kMaxTokens || num_blocks > kMaxTokens)
        return fail(PA_ERR_UNSUPPORTED, "num_rows or num_blocks is above 2^30");
    return PA_OK;
}

// Whether [a, a + n) and [b, b + m) have bytes in common.
bool overlap(const void *a, long long n, const void *b, long long m) {
    const char *x = static_cast<const char *>(a), *y = static_cast<const char *>(b);
    return n > 0 && m > 0 && x < y + m && y < x + n;
}

bool int32_aligned(const void *a, const void *b = nullptr, const void *c = nullptr, const void *d = nullptr,
                   const void *e = nullptr) {
    return aligned(a, 4) && aligned(b, 4) && aligned(c, 4) && aligned(d, 4) && aligned(e, 4);
}

}  // namespace

extern "C" {

pa_status pa_verify_drafts(int32_t *accept_lens, int32_t *accepted, int32_t *tokens, const void *target_probs,
                           const void *draft_probs, const int32_t *draft_tokens, const int32_t *draft_lens,
                           const int32_t *parents, const float *uniforms, int num_seqs, int num_draft, int vocab_size,
                           long long target_stride, long long draft_stride, pa_dtype dtype, uint32_t *err_word,
                           pa_stream_t stream) {
    g_detail.clear();
    if (num_seqs < 0)
        return fail(PA_ERR_INVALID_ARGUMENT, "num_seqs out of range");
    if (num_draft < 1 || num_draft > kVerifyMaxDraft)
        return fail(PA_ERR_INVALID_ARGUMENT, "num_draft must be 1 .. 256");
    if (vocab_size < 1)
        return fail(PA_ERR_INVALID_ARGUMENT, "vocab_size must be positive");
    if (vocab_size > kMaxTokens)
        return fail(PA_ERR_UNSUPPORTED, "vocab_size is above 2^30");
    if (!dtype_ok(dtype))
        return fail(PA_ERR_INVALID_ARGUMENT, "unknown dtype");
    if (target_stride < vocab_size || (draft_probs && draft_stride < vocab_size))
        return fail(PA_ERR_INVALID_ARGUMENT, "a row stride is smaller than vocab_size");
    if (num_seqs > INT_MAX / 16)
        return fail(PA_ERR_UNSUPPORTED, "num_seqs too large");
    if (num_seqs == 0)
        return PA_OK;
    if (!accept_lens || !accepted || !tokens || !target_probs || !draft_tokens || !uniforms)
        return fail(PA_ERR_INVALID_ARGUMENT, "null pointer");
    const size_t elt = elt_bytes(dtype);
    if (!aligned(target_probs, elt) || !aligned(draft_probs, elt))
        return fail(PA_ERR_INVALID_ARGUMENT, "target_probs or draft_probs is not aligned to its element size");
    if (!int32_aligned(accept_lens, accepted, tokens) ||
        !int32_aligned(draft_tokens, draft_lens, parents, uniforms, err_word))
        return fail(PA_ERR_INVALID_ARGUMENT, "an array is not 4-byte aligned");
    VerifyParams p = {};
    p.accept_lens = accept_lens;
    p.accepted = accepted;
    p.tokens = tokens;
    p.target = target_probs;
    p.draft = draft_probs;
    p.draft_tokens = draft_tokens;
    p.draft_lens = draft_lens;
    p.parents = parents;
    p.uniforms = uniforms;
    p.err = err_word;
    p.target_stride = target_stride;
    p.draft_stride = draft_probs ? draft_stride : 0;
    p.num_seqs = num_seqs;
    p.num_draft = num_draft;
    p.vocab = vocab_size;
    int dev = 0, sms = 0;
    cudaError_t e = device_sms(&dev, &sms);
    if (e != cudaSuccess)
        return cuda_fail(e, "device query");
    e = launch_verify(p, dtype, sms, stream_of(stream));
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "verify launch");
}

size_t pa_append_kv_block_quant_workspace_size(int num_tokens, int block_size, int num_blocks) {
    if (num_tokens <= kAppendBqFew || !block_size_ok(block_size) || num_blocks <= 0)
        return 0;
    const size_t blocks = num_tokens < num_blocks ? num_tokens : num_blocks;
    return (static_cast<size_t>(num_blocks) * block_size + blocks + 1) * sizeof(int32_t);
}

pa_status pa_append_kv_block_quant(const void *k, const void *v, const int64_t *slot_mapping, void *k_cache,
                                   void *v_cache, float *k_scales, float *v_scales, int num_tokens, int num_kv_heads,
                                   int head_dim, int block_size, int num_blocks, pa_dtype dtype, pa_dtype cache_dtype,
                                   void *workspace, size_t workspace_bytes, uint32_t *err_word, pa_stream_t stream) {
    g_detail.clear();
    if (num_tokens < 0 || num_kv_heads <= 0 || num_blocks <= 0)
        return fail(PA_ERR_INVALID_ARGUMENT, "num_tokens, num_kv_heads or num_blocks out of range");
    if (!block_size_ok(block_size))
        return fail(PA_ERR_UNSUPPORTED, "block_size must be 8, 16 or 32");
    if (!head_dim_ok(head_dim))
        return fail(PA_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
    if (!dtype_ok(dtype))
        return fail(PA_ERR_INVALID_ARGUMENT, "k and v must be PA_F32, PA_F16 or PA_BF16");
    if (!code_dtype_ok(cache_dtype))
        return fail(PA_ERR_INVALID_ARGUMENT, "cache_dtype must be PA_I8 or PA_E4M3");
    if (num_kv_heads > kMaxTokens / 2)
        return fail(PA_ERR_UNSUPPORTED, "num_kv_heads is above 2^29");
    if (num_tokens > kMaxTokens)
        return fail(PA_ERR_UNSUPPORTED, "num_tokens is above 2^30");
    if (num_tokens == 0)
        return PA_OK;
    if (!k || !v || !slot_mapping || !k_cache || !v_cache || !k_scales || !v_scales)
        return fail(PA_ERR_INVALID_ARGUMENT, "null pointer");
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache))
        return fail(PA_ERR_INVALID_ARGUMENT, "k, v and the caches must be 16-byte aligned");
    if (!aligned(slot_mapping, 8))
        return fail(PA_ERR_INVALID_ARGUMENT, "slot_mapping must be 8-byte aligned");
    if (!int32_aligned(k_scales, v_scales, workspace, err_word))
        return fail(PA_ERR_INVALID_ARGUMENT, "a scale array, the workspace or err_word is not 4-byte aligned");
    const size_t need = pa_append_kv_block_quant_workspace_size(num_tokens, block_size, num_blocks);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need))
        return fail(PA_ERR_WORKSPACE_TOO_SMALL, "workspace smaller than pa_append_kv_block_quant_workspace_size()");
    AppendBqParams p = {};
    p.k = k;
    p.v = v;
    p.slots = slot_mapping;
    p.k_cache = static_cast<uint8_t *>(k_cache);
    p.v_cache = static_cast<uint8_t *>(v_cache);
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    if (need > 0) {
        p.token_of = static_cast<int32_t *>(workspace);
        p.listed = p.token_of + static_cast<size_t>(num_blocks) * block_size;
        p.list = p.listed + 1;
    }
    p.err = err_word;
    p.pool_slots = static_cast<long long>(num_blocks) * block_size;
    p.num_tokens = num_tokens;
    p.num_kv_heads = num_kv_heads;
    p.block_size = block_size;
    int dev = 0, sms = 0;
    cudaError_t e = device_sms(&dev, &sms);
    if (e != cudaSuccess)
        return cuda_fail(e, "device query");
    e = launch_append_bq(p, dtype, cache_dtype, head_dim, sms, stream_of(stream));
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "append launch");
}

size_t pa_decode_block_quant_workspace_size(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                            int block_size, int max_blocks_per_seq) {
    const long long max_len = static_cast<long long>(max_blocks_per_seq) * block_size;
    if (num_seqs <= 0 || num_kv_heads <= 0 || num_heads <= 0 || num_heads % num_kv_heads != 0 ||
        !head_dim_ok(head_dim) || !block_size_ok(block_size) || max_blocks_per_seq <= 0 || max_len > kMaxTokens)
        return 0;
    const int group = num_heads / num_kv_heads;
    const size_t ctas = decode_bq_ctas(num_seqs, num_kv_heads, static_cast<int>(max_len));
    return ctas * sizeof(int4) + ctas * 2 * group * (head_dim + 2) * sizeof(float);
}

pa_status pa_decode_block_quant(void *out, const void *q, const void *k_cache, const void *v_cache,
                                const float *k_scales, const float *v_scales, const int32_t *block_tables,
                                const int32_t *context_lens, int num_seqs, int num_heads, int num_kv_heads,
                                int head_dim, int block_size, float scale, int window, pa_dtype dtype,
                                pa_dtype cache_dtype, pa_dtype out_dtype, int max_blocks_per_seq, int num_blocks,
                                void *workspace, size_t workspace_bytes, uint32_t *err_word, pa_stream_t stream) {
    g_detail.clear();
    if (num_seqs < 0 || num_heads <= 0 || max_blocks_per_seq <= 0 || window < 0)
        return fail(PA_ERR_INVALID_ARGUMENT, "num_seqs, num_heads, max_blocks_per_seq or window out of range");
    if (!head_dim_ok(head_dim))
        return fail(PA_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
    if (!block_size_ok(block_size))
        return fail(PA_ERR_UNSUPPORTED, "block_size must be 8, 16 or 32");
    if (num_kv_heads <= 0 || num_heads % num_kv_heads != 0)
        return fail(PA_ERR_INVALID_ARGUMENT, "num_heads must be a multiple of num_kv_heads");
    const int group = num_heads / num_kv_heads;
    if (group != 1 && group != 2 && group != 4 && group != 8)
        return fail(PA_ERR_UNSUPPORTED, "num_heads / num_kv_heads must be 1, 2, 4 or 8");
    if (!dtype_ok(dtype) || !dtype_ok(out_dtype))
        return fail(PA_ERR_INVALID_ARGUMENT, "unknown dtype");
    if (!code_dtype_ok(cache_dtype))
        return fail(PA_ERR_INVALID_ARGUMENT, "cache_dtype must be PA_I8 or PA_E4M3");
    if (num_blocks <= 0)
        return fail(PA_ERR_INVALID_ARGUMENT, "num_blocks must be positive");
    if (!std::isfinite(scale))
        return fail(PA_ERR_INVALID_ARGUMENT, "scale must be finite");
    if (num_seqs == 0)
        return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !k_scales || !v_scales || !block_tables || !context_lens)
        return fail(PA_ERR_INVALID_ARGUMENT, "null pointer");
    const long long max_len = static_cast<long long>(max_blocks_per_seq) * block_size;
    if (max_len > kMaxTokens)
        return fail(PA_ERR_UNSUPPORTED, "max_blocks_per_seq * block_size is above 2^30");
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache))
        return fail(PA_ERR_INVALID_ARGUMENT, "q, k_cache and v_cache must be 16-byte aligned");
    if (!aligned(out, elt_bytes(out_dtype)))
        return fail(PA_ERR_INVALID_ARGUMENT, "out is not aligned to its element size");
    if (!int32_aligned(k_scales, v_scales, block_tables, context_lens, err_word))
        return fail(PA_ERR_INVALID_ARGUMENT, "an array is not 4-byte aligned");
    const size_t need = pa_decode_block_quant_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                                                             max_blocks_per_seq);
    if (workspace == nullptr || workspace_bytes < need)
        return fail(PA_ERR_WORKSPACE_TOO_SMALL, "workspace smaller than pa_decode_block_quant_workspace_size()");
    if (!aligned16(workspace))
        return fail(PA_ERR_INVALID_ARGUMENT, "workspace must be 16-byte aligned");
    DecodeBqParams p = {};
    p.out = out;
    p.q = q;
    p.k_cache = static_cast<const uint8_t *>(k_cache);
    p.v_cache = static_cast<const uint8_t *>(v_cache);
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    const size_t ctas = decode_bq_ctas(num_seqs, num_kv_heads, static_cast<int>(max_len));
    p.records = static_cast<int4 *>(workspace);
    p.part_acc = reinterpret_cast<float *>(p.records + ctas);
    p.part_ml = p.part_acc + ctas * 2 * group * head_dim;
    p.err = err_word;
    p.num_seqs = num_seqs;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.block_size = block_size;
    p.log_block = block_size == 8 ? 3 : (block_size == 16 ? 4 : 5);
    p.window = window;
    p.max_blocks = max_blocks_per_seq;
    p.max_len = static_cast<int>(max_len);
    p.num_blocks = num_blocks;
    p.q_dtype = dtype;
    p.out_dtype = out_dtype;
    p.scale_log2 = scale * 1.4426950408889634f;
    int dev = 0, sms = 0;
    cudaError_t e = device_sms(&dev, &sms);
    if (e != cudaSuccess)
        return cuda_fail(e, "device query");
    e = launch_decode_bq(p, cache_dtype, head_dim, sms, stream_of(stream));
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "decode launch");
}

size_t pa_pages_workspace_size(int num_rows, int num_blocks) {
    if (num_rows < 0 || num_blocks <= 0)
        return 0;
    return kPagesArrays * (static_cast<size_t>(num_rows) + num_blocks) * sizeof(int32_t);
}

pa_status pa_pages_update(int32_t *new_tables, int32_t *new_ref_counts, int64_t *pairs, int32_t *status,
                          const int32_t *tables, const int32_t *ref_counts, const int32_t *lens,
                          const int32_t *parents, const int32_t *keep_lens, const int32_t *grow_lens, int num_rows,
                          int old_rows, int max_blocks_per_seq, int block_size, int num_blocks, void *workspace,
                          size_t workspace_bytes, uint32_t *err_word, pa_stream_t stream) {
    g_detail.clear();
    pa_status st = pages_args(num_rows, max_blocks_per_seq, block_size, num_blocks);
    if (st == PA_OK)
        st = pages_args(old_rows, max_blocks_per_seq, block_size, num_blocks);
    if (st != PA_OK)
        return st;
    if (!parents && num_rows > old_rows)
        return fail(PA_ERR_INVALID_ARGUMENT, "without parents num_rows must not exceed old_rows");
    if (!new_ref_counts || !status || !ref_counts ||
        (num_rows > 0 && (!new_tables || !pairs || !keep_lens || !grow_lens)) || (old_rows > 0 && (!tables || !lens)))
        return fail(PA_ERR_INVALID_ARGUMENT, "null pointer");
    if (!int32_aligned(new_tables, new_ref_counts, status, tables, ref_counts) ||
        !int32_aligned(lens, parents, keep_lens, grow_lens, workspace) || !aligned(err_word, 4))
        return fail(PA_ERR_INVALID_ARGUMENT, "an array is not 4-byte aligned");
    if (!aligned(pairs, 8))
        return fail(PA_ERR_INVALID_ARGUMENT, "pairs must be 8-byte aligned");
    const long long row = 4LL * max_blocks_per_seq, counts = 4LL * num_blocks;
    if (overlap(new_tables, num_rows * row, tables, old_rows * row))
        return fail(PA_ERR_INVALID_ARGUMENT, "new_tables overlaps tables");
    if (new_ref_counts != ref_counts && overlap(new_ref_counts, counts, ref_counts, counts))
        return fail(PA_ERR_INVALID_ARGUMENT, "new_ref_counts overlaps ref_counts and is not the same");
    const int rows = num_rows > old_rows ? num_rows : old_rows;
    if (workspace == nullptr || workspace_bytes < pa_pages_workspace_size(rows, num_blocks))
        return fail(PA_ERR_WORKSPACE_TOO_SMALL, "workspace smaller than pa_pages_workspace_size()");
    PagesUpdateParams p = {};
    p.new_tables = new_tables;
    p.new_refs = new_ref_counts;
    p.pairs = pairs;
    p.status = status;
    p.tables = tables;
    p.refs = ref_counts;
    p.lens = lens;
    p.parents = parents;
    p.keep = keep_lens;
    p.grow = grow_lens;
    const size_t nb = num_blocks, nr = rows;
    p.count = static_cast<int32_t *>(workspace);
    p.first = p.count + nb;
    p.writers = p.first + nb;
    p.free_list = p.writers + nb;
    p.kept = p.free_list + nb;
    p.total = p.kept + nr;
    p.need = p.total + nr;
    p.base = p.need + nr;
    p.err = err_word;
    p.rows = num_rows;
    p.old_rows = old_rows;
    p.max_blocks = max_blocks_per_seq;
    p.num_blocks = num_blocks;
    p.block_size = block_size;
    const cudaError_t e = launch_pages_update(p, stream_of(stream));
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "pages update launch");
}

pa_status pa_pages_compact(int32_t *new_tables, int32_t *new_ref_counts, int32_t *remap, int64_t *pairs,
                           int32_t *status, const int32_t *tables, const int32_t *ref_counts, const int32_t *lens,
                           int num_rows, int max_blocks_per_seq, int block_size, int num_blocks, int max_moves,
                           void *workspace, size_t workspace_bytes, uint32_t *err_word, pa_stream_t stream) {
    g_detail.clear();
    const pa_status st = pages_args(num_rows, max_blocks_per_seq, block_size, num_blocks);
    if (st != PA_OK)
        return st;
    if (max_moves < 0)
        return fail(PA_ERR_INVALID_ARGUMENT, "max_moves must not be negative");
    if (max_moves > kMaxTokens)
        return fail(PA_ERR_UNSUPPORTED, "max_moves is above 2^30");
    if (!new_ref_counts || !remap || !status || !ref_counts || (num_rows > 0 && (!new_tables || !tables || !lens)) ||
        (max_moves > 0 && !pairs))
        return fail(PA_ERR_INVALID_ARGUMENT, "null pointer");
    if (!int32_aligned(new_tables, new_ref_counts, remap, status, tables) ||
        !int32_aligned(ref_counts, lens, workspace, err_word))
        return fail(PA_ERR_INVALID_ARGUMENT, "an array is not 4-byte aligned");
    if (!aligned(pairs, 8))
        return fail(PA_ERR_INVALID_ARGUMENT, "pairs must be 8-byte aligned");
    const long long bytes = 4LL * max_blocks_per_seq * num_rows, counts = 4LL * num_blocks;
    if ((new_tables != tables && overlap(new_tables, bytes, tables, bytes)) ||
        (new_ref_counts != ref_counts && overlap(new_ref_counts, counts, ref_counts, counts)))
        return fail(PA_ERR_INVALID_ARGUMENT, "an output overlaps its input and is not the same");
    if (workspace == nullptr || workspace_bytes < pa_pages_workspace_size(num_rows, num_blocks))
        return fail(PA_ERR_WORKSPACE_TOO_SMALL, "workspace smaller than pa_pages_workspace_size()");
    PagesCompactParams p = {};
    p.new_tables = new_tables;
    p.new_refs = new_ref_counts;
    p.remap = remap;
    p.pairs = pairs;
    p.status = status;
    p.tables = tables;
    p.refs = ref_counts;
    p.lens = lens;
    p.src_list = static_cast<int32_t *>(workspace);
    p.dst_list = p.src_list + num_blocks;
    p.place = p.dst_list + num_blocks;
    p.err = err_word;
    p.rows = num_rows;
    p.max_blocks = max_blocks_per_seq;
    p.num_blocks = num_blocks;
    p.block_size = block_size;
    p.max_moves = max_moves;
    const cudaError_t e = launch_pages_compact(p, stream_of(stream));
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "pages compact launch");
}

pa_status pa_copy_pages(const int64_t *src_dst_pairs, int num_pairs, void *const *pools, const long long *block_bytes,
                        int num_pools, int num_blocks, uint32_t *err_word, pa_stream_t stream) {
    g_detail.clear();
    if (num_pairs < 0 || num_blocks <= 0)
        return fail(PA_ERR_INVALID_ARGUMENT, "num_pairs or num_blocks out of range");
    if (num_pools < 1 || num_pools > kMaxPools)
        return fail(PA_ERR_INVALID_ARGUMENT, "num_pools must be 1 .. 8");
    if (num_pairs > kMaxTokens)
        return fail(PA_ERR_UNSUPPORTED, "num_pairs is above 2^30");
    if (!pools || !block_bytes)
        return fail(PA_ERR_INVALID_ARGUMENT, "null pointer");
    CopyPagesParams p = {};
    for (int i = 0; i < num_pools; ++i) {
        if (block_bytes[i] <= 0 || block_bytes[i] % 4 != 0)
            return fail(PA_ERR_INVALID_ARGUMENT, "block_bytes must be positive multiples of 4");
        if (block_bytes[i] > LLONG_MAX / num_blocks)
            return fail(PA_ERR_UNSUPPORTED, "a pool is too large");
        if (num_pairs > 0 && (!pools[i] || !aligned(pools[i], 4)))
            return fail(PA_ERR_INVALID_ARGUMENT, "a pool is null or not 4-byte aligned");
        p.pool[i] = static_cast<char *>(pools[i]);
        p.block_bytes[i] = block_bytes[i];
    }
    if (num_pairs == 0)
        return PA_OK;
    if (!src_dst_pairs || !aligned(src_dst_pairs, 8) || !aligned(err_word, 4))
        return fail(PA_ERR_INVALID_ARGUMENT, "src_dst_pairs is null, or an array is not aligned to its element size");
    p.pairs = src_dst_pairs;
    p.err = err_word;
    p.num_blocks = num_blocks;
    p.num_pairs = num_pairs;
    p.num_pools = num_pools;
    int dev = 0, sms = 0;
    cudaError_t e = device_sms(&dev, &sms);
    if (e != cudaSuccess)
        return cuda_fail(e, "device query");
    e = launch_copy_pages(p, sms, stream_of(stream));
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "copy launch");
}

}  // extern "C"
