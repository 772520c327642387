// extern "C" entry points of the decoder operators (declared in
// include/q4_decoder.h).  Every argument is checked here, before any HIP call.

#include "q4_decoder.h"

#include <math.h>

#include "q4_decoder_internal.h"

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 20;
constexpr int64_t kMaxCols = int64_t(1) << 20;

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool is_dtype(int t) { return t == Q4_F32 || t == Q4_BF16; }

q4_status from_hip(hipError_t e) { return e == hipSuccess ? Q4_OK : Q4_ERR_HIP; }

hipStream_t as_stream(void *s) { return reinterpret_cast<hipStream_t>(s); }

bool cache_ok(int64_t num_blocks, int64_t kv_heads, int64_t head_dim) {
    return num_blocks >= 1 && num_blocks <= (int64_t(1) << 24) && kv_heads >= 1 && kv_heads <= 256 &&
           (head_dim == 64 || head_dim == 128);
}

q4_status check_shape(const q4_kv_cache *c, const q4_kv_batch *b, int64_t q_heads) {
    if (!c || !b) return Q4_ERR_NULL;
    if (!cache_ok(c->num_blocks, c->kv_heads, c->head_dim)) return Q4_ERR_RANGE;
    if (q_heads < 1 || q_heads % c->kv_heads || q_heads / c->kv_heads > 64) return Q4_ERR_RANGE;
    if (b->batch < 0 || b->batch > 65535 || b->rows < 0 || b->rows > kMaxRows) return Q4_ERR_RANGE;
    if (b->table_width < 1 || b->table_width > (int64_t(1) << 20)) return Q4_ERR_RANGE;
    if (b->max_rows < 1 || b->max_rows > kMaxRows || b->max_length < 1 || b->max_length > (int64_t(1) << 25))
        return Q4_ERR_RANGE;
    if (!b->cu_rows && b->batch && b->rows % b->batch) return Q4_ERR_RANGE;
    return Q4_OK;
}

q4_status check_memory(const q4_kv_cache *c, const q4_kv_batch *b) {
    if (!c->data || !b->block_table || !b->lengths) return Q4_ERR_NULL;
    if (!aligned(c->data, 16) || !aligned(b->block_table, 4) || !aligned(b->lengths, 4) || !aligned(b->cu_rows, 4))
        return Q4_ERR_ALIGN;
    return Q4_OK;
}

q4::KvView view(const q4_kv_cache *c, const q4_kv_batch *b) {
    q4::KvView v;
    v.data = static_cast<uint8_t *>(c->data);
    v.exps = reinterpret_cast<int8_t *>(v.data + c->num_blocks * c->kv_heads * 2 * q4::kKvBlock * c->head_dim);
    v.num_blocks = static_cast<int32_t>(c->num_blocks);
    v.kv_heads = c->kv_heads;
    v.table = b->block_table;
    v.lengths = b->lengths;
    v.cu_rows = b->cu_rows;
    v.table_width = static_cast<int32_t>(b->table_width);
    v.rows = static_cast<int32_t>(b->rows);
    v.rows_each = b->batch ? static_cast<int32_t>(b->rows / b->batch) : 0;
    v.batch = static_cast<int32_t>(b->batch);
    return v;
}

}  // namespace

extern "C" {

size_t q4_kv_cache_bytes(int64_t num_blocks, int64_t kv_heads, int64_t head_dim) {
    if (!cache_ok(num_blocks, kv_heads, head_dim)) return 0;
    return static_cast<size_t>(num_blocks) * kv_heads * 2 * (q4::kKvBlock * head_dim + 1);
}

q4_status q4_kv_append(const q4_kv_cache *cache, const q4_kv_batch *batch, const void *q, int64_t q_stride,
                       int64_t q_heads, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                       int dtype, const float *rope, int64_t positions, int64_t rot, int interleaved,
                       void *q_out, void *stream) {
    if (const q4_status st = check_shape(cache, batch, q_heads)) return st;
    const int64_t D = cache->head_dim, HD = cache->kv_heads * D, QD = q_heads * D;
    if (!is_dtype(dtype) || (interleaved != 0 && interleaved != 1)) return Q4_ERR_RANGE;
    if (rot < 0 || rot > D || rot % 32) return Q4_ERR_RANGE;
    if (rot && (positions < 1 || positions > (int64_t(1) << 25))) return Q4_ERR_RANGE;
    if (q_stride < QD || k_stride < HD || v_stride < HD) return Q4_ERR_RANGE;
    if (batch->batch == 0 || batch->rows == 0) return Q4_OK;
    if (const q4_status st = check_memory(cache, batch)) return st;
    if (!q || !k || !v || !q_out || (rot && !rope)) return Q4_ERR_NULL;
    const int64_t per16 = dtype == Q4_BF16 ? 8 : 4;   // elements of 16 bytes
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || !aligned(rope, 16))
        return Q4_ERR_ALIGN;
    if (q_stride % per16 || k_stride % per16 || v_stride % per16) return Q4_ERR_ALIGN;
    q4::AppendArgs a;
    a.kv = view(cache, batch);
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_heads = static_cast<int32_t>(q_heads);
    a.rope = rope;
    a.positions = static_cast<int32_t>(positions);
    a.rot = static_cast<int32_t>(rot);
    a.interleaved = interleaved;
    a.q_out = static_cast<uint16_t *>(q_out);
    a.max_rows = static_cast<int32_t>(batch->max_rows);
    return from_hip(q4::launch_kv_append(a, cache->head_dim, dtype, as_stream(stream)));
}

size_t q4_kv_attention_workspace(const q4_kv_cache *cache, const q4_kv_batch *batch, int64_t q_heads) {
    if (check_shape(cache, batch, q_heads) != Q4_OK || batch->batch == 0 || batch->rows == 0) return 0;
    q4::AttentionArgs a = {};
    a.kv = view(cache, batch);
    a.q_heads = static_cast<int32_t>(q_heads);
    a.group = static_cast<int32_t>(q_heads / cache->kv_heads);
    a.max_rows = static_cast<int32_t>(batch->max_rows);
    a.max_length = static_cast<int32_t>(batch->max_length);
    return q4::attention_workspace(a, cache->head_dim);
}

q4_status q4_kv_attention_plan(const q4_kv_cache *cache, const q4_kv_batch *batch, int64_t q_heads, int64_t window,
                               int32_t *rows, int32_t *waves, int32_t *parts) {
    if (const q4_status st = check_shape(cache, batch, q_heads)) return st;
    if (window < 0 || window > (int64_t(1) << 30)) return Q4_ERR_RANGE;
    if (!rows || !waves || !parts) return Q4_ERR_NULL;
    q4::AttentionArgs a = {};
    a.kv = view(cache, batch);
    a.q_heads = static_cast<int32_t>(q_heads);
    a.group = static_cast<int32_t>(q_heads / cache->kv_heads);
    a.window = static_cast<int32_t>(window);
    a.max_rows = static_cast<int32_t>(batch->max_rows);
    a.max_length = static_cast<int32_t>(batch->max_length);
    q4::attention_plan(a, cache->head_dim, rows, waves, parts);
    return Q4_OK;
}

q4_status q4_kv_attention(const q4_kv_cache *cache, const q4_kv_batch *batch, const void *q, int64_t q_heads,
                          float scale, int64_t window, void *out, int out_dtype, void *workspace,
                          size_t workspace_bytes, void *stream) {
    if (const q4_status st = check_shape(cache, batch, q_heads)) return st;
    if (!is_dtype(out_dtype) || !isfinite(scale) || window < 0 || window > (int64_t(1) << 30)) return Q4_ERR_RANGE;
    if (batch->batch == 0 || batch->rows == 0) return Q4_OK;
    if (const q4_status st = check_memory(cache, batch)) return st;
    if (!q || !out) return Q4_ERR_NULL;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 16)) return Q4_ERR_ALIGN;
    q4::AttentionArgs a;
    a.kv = view(cache, batch);
    a.q = static_cast<const uint16_t *>(q);
    a.out = out;
    a.q_heads = static_cast<int32_t>(q_heads);
    a.group = static_cast<int32_t>(q_heads / cache->kv_heads);
    a.group_inverse = a.group > 1 ? static_cast<uint32_t>(((uint64_t(1) << 32) + a.group - 1) / a.group) : 0;
    a.scale_log2 = scale * 1.44269504088896340736f;
    // The kernels give a token that is not seen a score of -inf * |scale| * 2^eK,
    // so that product is held to fp32's normal numbers: 2^-94, with the smallest
    // eK of -32, which is 0 to any q . k below 2^70.
    constexpr float least = 0x1p-94f;
    if (fabsf(a.scale_log2) < least) a.scale_log2 = least;
    a.window = static_cast<int32_t>(window);
    a.out_bf16 = out_dtype == Q4_BF16;
    a.max_rows = static_cast<int32_t>(batch->max_rows);
    a.max_length = static_cast<int32_t>(batch->max_length);
    a.workspace = static_cast<float *>(workspace);
    const size_t need = q4::attention_workspace(a, cache->head_dim);
    if (need && !workspace) return Q4_ERR_NULL;
    if (workspace_bytes < need) return Q4_ERR_RANGE;
    return from_hip(q4::launch_kv_attention(a, cache->head_dim, as_stream(stream)));
}

q4_status q4_add_rmsnorm(const void *residual, int residual_dtype, const void *y, int y_dtype, int64_t M, int64_t C,
                         const float *weight, const float *post_weight, const float *gate, int64_t gate_rows,
                         float scale, const float *modulation, int64_t modulation_rows, float eps,
                         void *residual_out, void *x, int x_dtype, void *stream) {
    if (!is_dtype(residual_dtype) || !is_dtype(y_dtype) || !is_dtype(x_dtype)) return Q4_ERR_RANGE;
    if (M < 0 || M > kMaxRows || C < 32 || C > kMaxCols || C % 32) return Q4_ERR_RANGE;
    if (!isfinite(eps) || eps < 0 || !isfinite(scale)) return Q4_ERR_RANGE;
    if (!y && (post_weight || gate)) return Q4_ERR_RANGE;
    if (M == 0) return Q4_OK;
    if (gate && (gate_rows < 1 || gate_rows > M || M % gate_rows)) return Q4_ERR_RANGE;
    if (modulation && (modulation_rows < 1 || modulation_rows > M || M % modulation_rows)) return Q4_ERR_RANGE;
    if (!residual || !weight || !x || (y && !residual_out)) return Q4_ERR_NULL;
    if (!aligned(residual, 16) || !aligned(y, 16) || !aligned(weight, 16) || !aligned(post_weight, 16) ||
        !aligned(gate, 16) || !aligned(modulation, 16) || !aligned(residual_out, 16) || !aligned(x, 16))
        return Q4_ERR_ALIGN;
    q4::NormArgs a;
    a.residual = residual;
    a.y = y;
    a.M = M;
    a.C = static_cast<int32_t>(C);
    a.weight = weight;
    a.post_weight = post_weight;
    a.gate = gate;
    a.modulation = modulation;
    a.gate_run = gate ? static_cast<int32_t>(M / gate_rows) : 1;
    a.modulation_run = modulation ? static_cast<int32_t>(M / modulation_rows) : 1;
    a.scale = scale;
    a.eps = eps;
    a.residual_out = residual_out;
    a.x = x;
    return from_hip(q4::launch_add_rmsnorm(a, residual_dtype, y_dtype, x_dtype, as_stream(stream)));
}

q4_status q4_logits_adjust(const float *logits, int64_t M, int64_t V, const int32_t *history,
                           const int32_t *cu_history, int64_t history_size, const int32_t *prompt_lengths,
                           const float *repetition, const float *frequency, const float *presence,
                           const int32_t *bias_ids, const float *bias, const int32_t *cu_bias, int64_t bias_size,
                           const uint32_t *mask, float *out, void *stream) {
    if (M < 0 || M > 65535 || V < 1 || V > (int64_t(1) << 24)) return Q4_ERR_RANGE;
    if (history_size < 0 || history_size >= (int64_t(1) << 31) || bias_size < 0 || bias_size >= (int64_t(1) << 31))
        return Q4_ERR_RANGE;
    if (M == 0) return Q4_OK;
    if (!logits || !out || (history_size && (!history || !cu_history))) return Q4_ERR_NULL;
    if (bias_size && (!bias_ids || !bias || !cu_bias)) return Q4_ERR_NULL;
    if (!aligned(logits, 16) || !aligned(out, 16) || !aligned(history, 4) || !aligned(cu_history, 4) ||
        !aligned(prompt_lengths, 4) || !aligned(repetition, 4) || !aligned(frequency, 4) || !aligned(presence, 4) ||
        !aligned(bias_ids, 4) || !aligned(bias, 4) || !aligned(cu_bias, 4) || !aligned(mask, 4))
        return Q4_ERR_ALIGN;
    q4::LogitsArgs a;
    a.logits = logits;
    a.M = static_cast<int32_t>(M);
    a.V = static_cast<int32_t>(V);
    a.history = history;
    a.cu_history = cu_history;
    a.history_size = static_cast<int32_t>(history_size);
    a.prompt_lengths = prompt_lengths;
    a.repetition = repetition;
    a.frequency = frequency;
    a.presence = presence;
    a.bias_ids = bias_ids;
    a.bias = bias;
    a.cu_bias = cu_bias;
    a.bias_size = static_cast<int32_t>(bias_size);
    a.mask = mask;
    a.out = out;
    return from_hip(q4::launch_logits_adjust(a, as_stream(stream)));
}

}  // extern "C"
