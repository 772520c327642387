// extern "C" entry points of the operators around the paged cache (declared in
// include/q4_search.h).  Every argument is checked here, before any HIP call.

#include "q4_search.h"

#include "q4_abi_checks.h"
#include "q4_search_internal.h"

namespace {

using namespace q4_abi;

constexpr int64_t kMaxTableWidth = int64_t(1) << 20, kMaxBlocks = int64_t(1) << 24, kMaxSequences = 65535;

bool beams_ok(int64_t groups, int64_t beams, int64_t V) {
    return groups >= 0 && groups <= 65535 && beams >= 1 && beams <= q4::kMaxBeams && groups * beams <= 65535 && V >= 1 &&
           V <= (int64_t(1) << 24);
}

bool table_ok(int64_t rows, int64_t width, int64_t num_blocks) {
    return rows >= 0 && rows <= kMaxSequences && width >= 1 && width <= kMaxTableWidth && rows * width < (int64_t(1) << 31) &&
           num_blocks >= 1 && num_blocks <= kMaxBlocks;
}

// Sizes of the selection, without its memory.
q4::SelectArgs select_args(const q4_kv_cache *cache, const q4_kv_batch *batch) {
    q4::SelectArgs a = {};
    a.kv = view(cache, batch);
    a.max_rows = static_cast<int32_t>(batch->max_rows);
    a.max_blocks = static_cast<int32_t>((batch->max_length + q4::kKvBlock - 1) / q4::kKvBlock);
    return a;
}

}  // namespace

extern "C" {

size_t q4_beam_select_workspace(int64_t groups, int64_t beams, int64_t V) {
    if (!beams_ok(groups, beams, V) || groups == 0) return 0;
    return q4::beam_workspace(groups * beams, V);
}

q4_status q4_beam_select(const float *logits, int64_t groups, int64_t beams, int64_t V, const float *scores,
                         const int32_t *finished, int32_t pad, int64_t keep, int32_t *parents, int32_t *tokens,
                         float *out_scores, void *workspace, size_t workspace_bytes, void *stream) {
    if (!beams_ok(groups, beams, V) || keep < 1 || keep > q4::kMaxKeep || pad < 0) return Q4_ERR_RANGE;
    if (groups == 0) return Q4_OK;
    if (!logits || !scores || !parents || !tokens || !out_scores || !workspace) return Q4_ERR_NULL;
    if (!aligned(logits, 4) || !aligned(scores, 4) || !aligned(finished, 4) || !aligned(parents, 4) || !aligned(tokens, 4) ||
        !aligned(out_scores, 4) || !aligned(workspace, 16))
        return Q4_ERR_ALIGN;
    if (workspace_bytes < q4::beam_workspace(groups * beams, V)) return Q4_ERR_RANGE;
    q4::BeamArgs a;
    a.logits = logits;
    a.groups = static_cast<int32_t>(groups);
    a.beams = static_cast<int32_t>(beams);
    a.V = static_cast<int32_t>(V);
    a.scores = scores;
    a.finished = finished;
    a.pad = pad;
    a.keep = static_cast<int32_t>(keep);
    a.parents = parents;
    a.tokens = tokens;
    a.out_scores = out_scores;
    a.workspace = workspace;
    return from_hip(q4::launch_beam_select(a, as_stream(stream)));
}

q4_status q4_beam_advance(const int32_t *sequences, int64_t rows, int64_t width, const int32_t *lengths,
                          const int32_t *finished, const int32_t *parents, const int32_t *tokens, int64_t n_out,
                          int32_t eos, int32_t pad, int32_t *out_sequences, int32_t *out_lengths,
                          int32_t *out_finished, void *stream) {
    if (rows < 0 || rows > kMaxRows || n_out < 0 || n_out > kMaxRows || width < 1 || width > (int64_t(1) << 24)) return Q4_ERR_RANGE;
    if (n_out == 0) return Q4_OK;
    if ((rows && (!sequences || !lengths)) || !parents || !tokens || !out_sequences || !out_lengths || !out_finished) return Q4_ERR_NULL;
    if (!aligned(sequences, 4) || !aligned(lengths, 4) || !aligned(finished, 4) || !aligned(parents, 4) || !aligned(tokens, 4) ||
        !aligned(out_sequences, 4) || !aligned(out_lengths, 4) || !aligned(out_finished, 4))
        return Q4_ERR_ALIGN;
    q4::AdvanceArgs a;
    a.sequences = sequences;
    a.lengths = lengths;
    a.finished = finished;
    a.parents = parents;
    a.tokens = tokens;
    a.rows = static_cast<int32_t>(rows);
    a.width = static_cast<int32_t>(width);
    a.n_out = static_cast<int32_t>(n_out);
    a.eos = eos;
    a.pad = pad;
    a.out_sequences = out_sequences;
    a.out_lengths = out_lengths;
    a.out_finished = out_finished;
    return from_hip(q4::launch_beam_advance(a, as_stream(stream)));
}

size_t q4_kv_fork_workspace(int64_t n_out, int64_t num_blocks) {
    if (!table_ok(n_out, 1, num_blocks)) return 0;
    return q4::fork_workspace(n_out, num_blocks);
}

q4_status q4_kv_fork(const int32_t *block_table, int64_t rows, int64_t table_width, const int32_t *lengths,
                     const int32_t *parents, int64_t n_out, const int32_t *grow, int64_t grow_each,
                     const int32_t *held, int64_t num_blocks, int32_t *out_table, int32_t *out_lengths,
                     int32_t *refs, int32_t *src, int32_t *dst, int32_t *short_of, void *workspace,
                     size_t workspace_bytes, void *stream) {
    if (!table_ok(rows, table_width, num_blocks) || !table_ok(n_out, table_width, num_blocks)) return Q4_ERR_RANGE;
    if (!grow && (grow_each < 0 || grow_each > (int64_t(1) << 25))) return Q4_ERR_RANGE;
    if (!refs || !workspace || (rows && (!block_table || !lengths))) return Q4_ERR_NULL;
    if (n_out && (!parents || !out_table || !out_lengths || !src || !dst || !short_of)) return Q4_ERR_NULL;
    if (!aligned(block_table, 4) || !aligned(lengths, 4) || !aligned(parents, 4) || !aligned(grow, 4) || !aligned(held, 4) ||
        !aligned(out_table, 4) || !aligned(out_lengths, 4) || !aligned(refs, 4) || !aligned(src, 4) || !aligned(dst, 4) ||
        !aligned(short_of, 4) || !aligned(workspace, 16))
        return Q4_ERR_ALIGN;
    if (workspace_bytes < q4::fork_workspace(n_out, num_blocks)) return Q4_ERR_RANGE;
    q4::ForkArgs a;
    a.table = block_table;
    a.lengths = lengths;
    a.parents = parents;
    a.grow = grow;
    a.held = held;
    a.rows = static_cast<int32_t>(rows);
    a.width = static_cast<int32_t>(table_width);
    a.n_out = static_cast<int32_t>(n_out);
    a.grow_each = static_cast<int32_t>(grow ? 0 : grow_each);
    a.num_blocks = static_cast<int32_t>(num_blocks);
    a.out_table = out_table;
    a.out_lengths = out_lengths;
    a.refs = refs;
    a.src = src;
    a.dst = dst;
    a.short_of = short_of;
    a.workspace = static_cast<int32_t *>(workspace);
    return from_hip(q4::launch_kv_fork(a, as_stream(stream)));
}

size_t q4_kv_compact_workspace(int64_t num_blocks) {
    if (!table_ok(0, 1, num_blocks)) return 0;
    return q4::compact_workspace(num_blocks);
}

q4_status q4_kv_compact(const int32_t *block_table, int64_t rows, int64_t table_width, const int32_t *lengths,
                        const int32_t *held, int64_t num_blocks, int32_t *out_table, int32_t *src, int32_t *dst,
                        int32_t *live, void *workspace, size_t workspace_bytes, void *stream) {
    if (!table_ok(rows, table_width, num_blocks)) return Q4_ERR_RANGE;
    if (!src || !dst || !live || !workspace || (rows && (!block_table || !lengths || !out_table))) return Q4_ERR_NULL;
    if (!aligned(block_table, 4) || !aligned(lengths, 4) || !aligned(held, 4) || !aligned(out_table, 4) || !aligned(src, 4) ||
        !aligned(dst, 4) || !aligned(live, 4) || !aligned(workspace, 16))
        return Q4_ERR_ALIGN;
    if (workspace_bytes < q4::compact_workspace(num_blocks)) return Q4_ERR_RANGE;
    q4::CompactArgs a;
    a.table = block_table;
    a.lengths = lengths;
    a.held = held;
    a.rows = static_cast<int32_t>(rows);
    a.width = static_cast<int32_t>(table_width);
    a.num_blocks = static_cast<int32_t>(num_blocks);
    a.out_table = out_table;
    a.src = src;
    a.dst = dst;
    a.live = live;
    a.workspace = static_cast<int32_t *>(workspace);
    return from_hip(q4::launch_kv_compact(a, as_stream(stream)));
}

q4_status q4_kv_copy_blocks(const q4_kv_cache *cache, void *const *data, void *const *summaries, int64_t layers,
                            const int32_t *src, const int32_t *dst, int64_t n, void *stream) {
    if (!cache) return Q4_ERR_NULL;
    if (!cache_ok(cache->num_blocks, cache->kv_heads, cache->head_dim) || layers < 0 || layers > 1024 || n < 0 ||
        n > (int64_t(1) << 24))
        return Q4_ERR_RANGE;
    if (n == 0 || layers == 0) return Q4_OK;
    if (!data || !src || !dst) return Q4_ERR_NULL;
    if (!aligned(src, 4) || !aligned(dst, 4)) return Q4_ERR_ALIGN;
    for (int64_t l = 0; l < layers; ++l) {
        if (!data[l] || (summaries && !summaries[l])) return Q4_ERR_NULL;
        if (!aligned(data[l], 16) || (summaries && !aligned(summaries[l], 16))) return Q4_ERR_ALIGN;
    }
    q4::CopyArgs a;
    a.num_blocks = static_cast<int32_t>(cache->num_blocks);
    a.kv_heads = cache->kv_heads;
    a.head_dim = cache->head_dim;
    a.n = static_cast<int32_t>(n);
    a.src = src;
    a.dst = dst;
    for (int64_t first = 0; first < layers; first += q4::kLayersAtOnce) {
        a.layers = static_cast<int32_t>(layers - first < q4::kLayersAtOnce ? layers - first : q4::kLayersAtOnce);
        for (int l = 0; l < q4::kLayersAtOnce; ++l) {
            a.data[l] = l < a.layers ? static_cast<uint8_t *>(data[first + l]) : nullptr;
            a.summary[l] = l < a.layers && summaries ? static_cast<uint8_t *>(summaries[first + l]) : nullptr;
        }
        if (const q4_status st = from_hip(q4::launch_kv_copy(a, as_stream(stream)))) return st;
    }
    return Q4_OK;
}

size_t q4_kv_summary_bytes(int64_t num_blocks, int64_t kv_heads, int64_t head_dim) {
    if (!cache_ok(num_blocks, kv_heads, head_dim)) return 0;
    return static_cast<size_t>(num_blocks) * kv_heads * 2 * head_dim;
}

q4_status q4_kv_summarize(const q4_kv_cache *cache, const q4_kv_batch *batch, void *summary, void *stream) {
    if (!cache || !batch) return Q4_ERR_NULL;
    if (const q4_status st = check_shape(cache, batch, cache->kv_heads)) return st;
    if (batch->batch == 0 || batch->rows == 0) return Q4_OK;
    if (const q4_status st = check_memory(cache, batch)) return st;
    if (!summary) return Q4_ERR_NULL;
    if (!aligned(summary, 16)) return Q4_ERR_ALIGN;
    q4::SelectArgs a = select_args(cache, batch);
    a.summary = static_cast<int8_t *>(summary);
    return from_hip(q4::launch_kv_summarize(a, cache->head_dim, as_stream(stream)));
}

size_t q4_kv_select_workspace(const q4_kv_cache *cache, const q4_kv_batch *batch) {
    if (!cache || !batch || check_shape(cache, batch, cache->kv_heads) != Q4_OK || batch->batch == 0 || batch->rows == 0) return 0;
    const q4::SelectArgs a = select_args(cache, batch);
    return (static_cast<size_t>(batch->rows) * cache->kv_heads * a.max_blocks * sizeof(float) + 15) / 16 * 16;
}

q4_status q4_kv_select(const q4_kv_cache *cache, const q4_kv_batch *batch, const void *summary, const void *q,
                       int64_t q_heads, int64_t keep, int64_t first, int64_t recent, int32_t *chosen,
                       void *workspace, size_t workspace_bytes, void *stream) {
    if (const q4_status st = check_shape(cache, batch, q_heads)) return st;
    if (keep < 1 || keep > (int64_t(1) << 16) || first < 0 || recent < 0 || first > keep || recent > keep || first + recent > keep)
        return Q4_ERR_RANGE;
    if (batch->batch == 0 || batch->rows == 0) return Q4_OK;
    if (const q4_status st = check_memory(cache, batch)) return st;
    if (!summary || !q || !chosen || !workspace) return Q4_ERR_NULL;
    if (!aligned(summary, 16) || !aligned(q, 16) || !aligned(chosen, 4) || !aligned(workspace, 16)) return Q4_ERR_ALIGN;
    if (workspace_bytes < q4_kv_select_workspace(cache, batch)) return Q4_ERR_RANGE;
    q4::SelectArgs a = select_args(cache, batch);
    a.summary = static_cast<int8_t *>(const_cast<void *>(summary));
    a.q = static_cast<const uint16_t *>(q);
    a.q_heads = static_cast<int32_t>(q_heads);
    a.group = static_cast<int32_t>(q_heads / cache->kv_heads);
    a.keep = static_cast<int32_t>(keep);
    a.first = static_cast<int32_t>(first);
    a.recent = static_cast<int32_t>(recent);
    a.chosen = chosen;
    a.scores = static_cast<float *>(workspace);
    return from_hip(q4::launch_kv_select(a, cache->head_dim, as_stream(stream)));
}

size_t q4_kv_attention_blocks_workspace(const q4_kv_cache *cache, const q4_kv_batch *batch, int64_t q_heads,
                                        int64_t keep) {
    if (check_shape(cache, batch, q_heads) != Q4_OK || keep < 1 || keep > (int64_t(1) << 16) || batch->batch == 0 || batch->rows == 0)
        return 0;
    q4::AttentionArgs a = {};
    a.kv = view(cache, batch);
    a.q_heads = static_cast<int32_t>(q_heads);
    a.group = static_cast<int32_t>(q_heads / cache->kv_heads);
    return q4::attention_blocks_workspace(a, static_cast<int>(keep), cache->head_dim);
}

q4_status q4_kv_attention_blocks(const q4_kv_cache *cache, const q4_kv_batch *batch, const void *q, int64_t q_heads,
                                 const int32_t *chosen, int64_t keep, float scale, void *out, int out_dtype,
                                 void *workspace, size_t workspace_bytes, void *stream) {
    if (const q4_status st = check_shape(cache, batch, q_heads)) return st;
    if (!is_dtype(out_dtype) || !isfinite(scale) || keep < 1 || keep > (int64_t(1) << 16)) return Q4_ERR_RANGE;
    if (batch->batch == 0 || batch->rows == 0) return Q4_OK;
    if (const q4_status st = check_memory(cache, batch)) return st;
    if (!q || !chosen || !out) return Q4_ERR_NULL;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(chosen, 4) || !aligned(workspace, 16)) return Q4_ERR_ALIGN;
    q4::AttentionArgs a = {};
    a.kv = view(cache, batch);
    a.q = static_cast<const uint16_t *>(q);
    a.out = out;
    a.q_heads = static_cast<int32_t>(q_heads);
    a.group = static_cast<int32_t>(q_heads / cache->kv_heads);
    a.scale_log2 = scale_log2_of(scale);
    a.out_bf16 = out_dtype == Q4_BF16;
    a.max_rows = static_cast<int32_t>(batch->max_rows);
    a.workspace = static_cast<float *>(workspace);
    const size_t need = q4::attention_blocks_workspace(a, static_cast<int>(keep), cache->head_dim);
    if (need && !workspace) return Q4_ERR_NULL;
    if (workspace_bytes < need) return Q4_ERR_RANGE;
    return from_hip(q4::launch_kv_attention_blocks(a, chosen, static_cast<int>(keep), cache->head_dim, as_stream(stream)));
}

}  // extern "C"
