// Internal declarations of the decoder operators (public ABI:
// include/q4_decoder.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q4_decoder.h"

namespace q4 {

constexpr int kKvBlock = Q4_KV_BLOCK;
constexpr int kExpMin = -32, kExpMax = 32;   // range of a block's stored exponent
constexpr float kE4m3Max = 448.0f;

// A cache and a batch as the kernels see them (checked on the host).
struct KvView {
    uint8_t *data;
    int8_t *exps;
    int32_t num_blocks;
    int32_t kv_heads;
    const int32_t *table;
    const int32_t *lengths;
    const int32_t *cu_rows;
    int32_t table_width;
    int32_t rows;
    int32_t rows_each;      // rows of every sequence where cu_rows is null
    int32_t batch;
};

#ifdef __HIPCC__
// One sequence of a batch: its first row, its number of rows, and the
// position of row 0 (negative where the sequence has more rows than tokens).
struct KvSequence {
    int32_t row0, rows, length, pos0;
};

__device__ __forceinline__ KvSequence kv_sequence(const KvView &c, int b) {
    KvSequence s;
    if (c.cu_rows) {
        const int32_t lo = c.cu_rows[b], hi = c.cu_rows[b + 1];
        s.row0 = lo < 0 ? 0 : lo > c.rows ? c.rows : lo;
        const int32_t end = hi < s.row0 ? s.row0 : hi > c.rows ? c.rows : hi;
        s.rows = end - s.row0;
    } else {
        s.row0 = b * c.rows_each;
        s.rows = c.rows_each;
    }
    const int32_t n = c.lengths[b];
    s.length = n < 0 ? 0 : n;
    s.pos0 = s.length - s.rows;
    return s;
}

// Block id of tokens [32 i, 32 i + 32) of sequence b, or -1 where the table
// has none inside the cache.
__device__ __forceinline__ int32_t kv_block_id(const KvView &c, int b, int i) {
    if (i < 0 || i >= c.table_width) return -1;
    const int32_t id = c.table[static_cast<int64_t>(b) * c.table_width + i];
    return id >= 0 && id < c.num_blocks ? id : -1;
}
#endif

struct AppendArgs {
    KvView kv;
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;   // elements
    int32_t q_heads;
    const float *rope;
    int32_t positions, rot, interleaved;
    uint16_t *q_out;
    int32_t max_rows;
};
hipError_t launch_kv_append(const AppendArgs &a, int head_dim, int dtype, hipStream_t s);

struct AttentionArgs {
    KvView kv;
    const uint16_t *q;
    void *out;
    int32_t q_heads, group;
    uint32_t group_inverse;  // 2^32 / group, rounded up: i / group = i * it >> 32 up to 2^26
    float scale_log2;        // softmax scale times log2(e)
    int32_t window;          // 0: none
    int32_t out_bf16;
    int32_t max_rows, max_length;
    float *workspace;
};
size_t attention_workspace(const AttentionArgs &a, int head_dim);
void attention_plan(const AttentionArgs &a, int head_dim, int32_t *rows, int32_t *waves, int32_t *parts);
hipError_t launch_kv_attention(const AttentionArgs &a, int head_dim, hipStream_t s);

struct NormArgs {
    const void *residual, *y;
    int64_t M;
    int32_t C;
    const float *weight, *post_weight, *gate, *modulation;
    int32_t gate_run, modulation_run;   // rows that share a row of gate / modulation
    float scale, eps;
    void *residual_out, *x;
};
hipError_t launch_add_rmsnorm(const NormArgs &a, int residual_dtype, int y_dtype, int x_dtype, hipStream_t s);

struct LogitsArgs {
    const float *logits;
    int32_t M, V;
    const int32_t *history, *cu_history;
    int32_t history_size;
    const int32_t *prompt_lengths;
    const float *repetition, *frequency, *presence;
    const int32_t *bias_ids;
    const float *bias;
    const int32_t *cu_bias;
    int32_t bias_size;
    const uint32_t *mask;
    float *out;
};
hipError_t launch_logits_adjust(const LogitsArgs &a, hipStream_t s);

}  // namespace q4
