// Checks of arguments that the C entry points of the decoder's operators share.
#pragma once

#include <math.h>

#include "q4_decoder_internal.h"

namespace q4_abi {

constexpr int64_t kMaxRows = int64_t(1) << 20;
constexpr int64_t kMaxCols = int64_t(1) << 20;

inline bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline bool is_dtype(int t) { return t == Q4_F32 || t == Q4_BF16; }

inline q4_status from_hip(hipError_t e) { return e == hipSuccess ? Q4_OK : Q4_ERR_HIP; }

inline hipStream_t as_stream(void *s) { return reinterpret_cast<hipStream_t>(s); }

inline bool cache_ok(int64_t num_blocks, int64_t kv_heads, int64_t head_dim) {
    return num_blocks >= 1 && num_blocks <= (int64_t(1) << 24) && kv_heads >= 1 && kv_heads <= 256 &&
           (head_dim == 64 || head_dim == 128);
}

inline q4_status check_shape(const q4_kv_cache *c, const q4_kv_batch *b, int64_t q_heads) {
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

inline q4_status check_memory(const q4_kv_cache *c, const q4_kv_batch *b) {
    if (!c->data || !b->block_table || !b->lengths) return Q4_ERR_NULL;
    if (!aligned(c->data, 16) || !aligned(b->block_table, 4) || !aligned(b->lengths, 4) || !aligned(b->cu_rows, 4))
        return Q4_ERR_ALIGN;
    return Q4_OK;
}

inline q4::KvView view(const q4_kv_cache *c, const q4_kv_batch *b) {
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

// The kernels give a token that is not seen a score of -inf * |scale| * 2^eK,
// so that product is held to fp32's normal numbers: 2^-94, with the smallest
// eK of -32, which is 0 to any q . k below 2^70.
inline float scale_log2_of(float scale) {
    constexpr float least = 0x1p-94f;
    const float c = scale * 1.44269504088896340736f;
    return fabsf(c) < least ? least : c;
}

}  // namespace q4_abi
