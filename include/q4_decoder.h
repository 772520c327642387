/*
 * q4_decoder.h -- C ABI of libq4amd's decoder operators for AMD Instinct
 * MI355X (gfx950): what a decoder computes between the 4-bit linears of
 * q4_0.h.
 *
 *   q4_kv_append      rotates q and k by their positions, quantizes k and v to
 *                     8 bits and appends them to a paged cache;
 *   q4_kv_attention   attention over that cache, for single tokens, a few
 *                     tokens and prompts;
 *   q4_add_rmsnorm    the norm after a block, its gate and residual scale, the
 *                     residual add and the norm before the next block;
 *   q4_logits_adjust  penalties for repeated tokens, biases and a grammar mask
 *                     on the LM head's logits.
 *
 * The conventions of q4_0.h hold: device pointers, the caller's buffers and
 * stream, every argument checked before any HIP call, nothing allocated,
 * results equal bit for bit from call to call.  Sizes, flags and pointers are
 * checked on the host (Q4_ERR_NULL, Q4_ERR_RANGE, Q4_ERR_ALIGN); what lies in
 * device memory (lengths, row bounds, block ids, token ids) is checked by the
 * kernels, which never read or write out of range for it: what they do
 * instead is stated with each call.  Unless stated otherwise outputs must not
 * overlap inputs.
 */
#ifndef Q4_DECODER_H
#define Q4_DECODER_H

#include "q4_0.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of activations. */
enum { Q4_F32 = 0, Q4_BF16 = 1 };

/*
 * The cache.  A block holds Q4_KV_BLOCK tokens.  For a block, a kv head and
 * each of K and V there are 32 * head_dim 8-bit codes (e4m3: sign, 4 exponent
 * bits of bias 7, 3 fraction bits, 0x7F and 0xFF not a number) and one int8
 * exponent e; the value of a code is code * 2^e.  e is the smallest exponent
 * with max |value| <= 448 * 2^e over the finite values of the block and head,
 * held to -32 .. 32 (-32 where all are zero); larger values saturate at
 * 448 * 2^32, and what is not finite becomes not a number.
 *
 * Layout of `data` (q4_kv_cache_bytes, 16-byte aligned):
 *   data plane [num_blocks][kv_heads][K | V][32 * head_dim] codes, then
 *   exponent plane [num_blocks][kv_heads][K | V] int8.
 *   K codes: token s, dimension d at
 *     ((((s / 16) * (D / 64) + d / 64) * 4 + d / 16 % 4) * 16 + s % 16) * 16 + d % 16,
 *   V codes: at
 *     (((d / 32 * 4 + s / 4 % 4) * 16 + d % 16) * 2 + d / 16 % 2) * 8 + s / 16 * 4 + s % 4,
 * so that lane l of a 64-lane wave reading 16 bytes at 16 l gets its operand
 * slices of two 16x16x32 matrix products, for K as for V transposed, and the
 * products' results need no exchange between lanes from the first to the
 * second.
 */
#define Q4_KV_BLOCK 32

typedef struct {
    void *data;
    int64_t num_blocks;   /* 1 .. 2^24 */
    int32_t kv_heads;     /* 1 .. 256  */
    int32_t head_dim;     /* 64 or 128 */
} q4_kv_cache;

size_t q4_kv_cache_bytes(int64_t num_blocks, int64_t kv_heads, int64_t head_dim);   /* 0 if invalid */

/*
 * The sequences of a call.  Sequence b has rows cu_rows[b] .. cu_rows[b + 1]
 * of q, k, v and of the outputs, and after the call's append lengths[b] tokens
 * in the cache, its rows the last of them: with n rows, row t is at position
 * lengths[b] - n + t, and its token is in slot position % 32 of block
 * block_table[b][position / 32].  Rows whose position would be negative have
 * no token (an idle slot of a batch is a sequence of length 0 with one row).
 * cu_rows may be NULL: every sequence has rows / batch rows.
 *
 * max_rows and max_length are what the launch is shaped for, the largest
 * number of rows and length of a sequence; larger ones are computed too, only
 * slower.  Row bounds are held to 0 .. rows, lengths to 0 .. table_width * 32
 * for what is read through the table.  Rows that belong to no sequence are not
 * written.
 */
typedef struct {
    const int32_t *block_table;   /* device [batch, table_width] */
    const int32_t *lengths;       /* device [batch]              */
    const int32_t *cu_rows;       /* device [batch + 1] or NULL  */
    int64_t table_width;          /* 1 .. 2^20                   */
    int64_t batch;                /* 0 .. 65535                  */
    int64_t rows;                 /* 0 .. 2^20                   */
    int64_t max_rows;             /* 1 .. 2^20                   */
    int64_t max_length;           /* 1 .. 2^25                   */
} q4_kv_batch;

/*
 * Appends the rows' keys and values and returns the rotated queries.
 *
 * q [rows, q_heads * D], k and v [rows, kv_heads * D], all of type `dtype`
 * (Q4_F32, as q4_0_linear_multi writes them, or Q4_BF16), device, 16-byte
 * aligned, a row's elements contiguous and rows `q_stride`, `k_stride`,
 * `v_stride` elements apart (a multiple of 16 bytes, no less than the row).
 * rope: fp32 [positions, rot / 2, 2] (device, 16-byte aligned), the cosine and
 * sine of the angle of pair i at a position; rot is 0 (no rotation, rope may
 * be NULL) or a multiple of 32 up to D.  Pair i is dimensions i and
 * i + rot / 2, or, with `interleaved`, 2 i and 2 i + 1:
 *     y_a = x_a cos - x_b sin,   y_b = x_b cos + x_a sin      (fp32);
 * dimensions from rot on stay as they are.  q_out: bf16 [rows, q_heads * D]
 * (device, contiguous), the rotated q rounded to nearest even.
 *
 * A block whose slot 0 is written by the call starts anew: its exponent comes
 * from the written values alone.  In another block the exponent never falls;
 * where it rises from e to e', the block's codes become
 * e4m3(code * 2^(e - e')), which is exact unless a value falls below 2^-6 of
 * the new scale.  Writing the same rows again gives the same cache.
 *
 * Rows without a position, or past the rope table, and ids outside the cache:
 * q_out is 0 for a row without a position, and past the table not a number in
 * the dimensions that are turned (so are the codes of k); a block whose id is outside [0, num_blocks) or past
 * table_width is not written.  Two sequences of one call must not write the
 * same block.
 */
q4_status q4_kv_append(const q4_kv_cache *cache, const q4_kv_batch *batch, const void *q, int64_t q_stride,
                       int64_t q_heads, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                       int dtype, const float *rope, int64_t positions, int64_t rot, int interleaved,
                       void *q_out, void *stream);

/*
 * o[row, head] = sum_j w_j v_j,  w = softmax over the visible tokens j of
 * scale * (q . k_j), kv head = head / (q_heads / kv_heads).  A row at position
 * p sees tokens j <= p, with window > 0 only j > p - window.  A row that sees
 * nothing gives 0.
 *
 * q: bf16 [rows, q_heads * D], out: [rows, q_heads * D] fp32 or bf16 by
 * out_dtype (device, 16-byte aligned, contiguous).  q_heads is a multiple of
 * kv_heads, at most 64 times.  Products of q with the codes of k are exact and
 * summed in fp32, the softmax's maximum and sum are fp32; the weights, times
 * the scale of their token's v, are rounded to fp16 for their products with the
 * codes of v, which are summed in fp32: within 2^-11 of each, or 2^-32 of the
 * row's largest where that is more.  Within fp32's range an output is finite
 * where the formula's is, and not a number where that is not: a token that a
 * row does not see has no effect on it, whatever its codes are, and one that it
 * sees has, however small its weight.  A token in a block whose id is outside
 * [0, num_blocks), or past table_width, counts as not a number.
 *
 * workspace: device, 16-byte aligned, q4_kv_attention_workspace bytes for the
 * same batch (0: may be NULL; never more than 2^18 * (head_dim + 2), 34 MB for
 * heads of 128), its content free before and after.  A max_length or max_rows
 * larger than the sequences' costs time (the splits that it asks for have
 * nothing to do, and are joined) and workspace.
 */
size_t q4_kv_attention_workspace(const q4_kv_cache *cache, const q4_kv_batch *batch, int64_t q_heads);
q4_status q4_kv_attention(const q4_kv_cache *cache, const q4_kv_batch *batch, const void *q, int64_t q_heads,
                          float scale, int64_t window, void *out, int out_dtype, void *workspace,
                          size_t workspace_bytes, void *stream);

/*
 * The launch that q4_kv_attention takes for these sizes: how many rows (times
 * the heads of a kv head) a workgroup has, its waves, and into how many parts
 * the tokens of its rows are divided.  No pointer of the cache or the batch is
 * read but for whether cu_rows is NULL.
 */
q4_status q4_kv_attention_plan(const q4_kv_cache *cache, const q4_kv_batch *batch, int64_t q_heads, int64_t window,
                               int32_t *rows, int32_t *waves, int32_t *parts);

/*
 * One residual step:
 *     u = y;  u = u / rms(u) * post_weight  (post_weight given);
 *     u = gate * u                          (gate given);
 *     r' = residual + scale * u;
 *     x = r' / rms(r') * weight;  x = x * (1 + modulation)  (modulation given)
 * with rms(a) = sqrt(mean(a^2) + eps) over a row, all in fp32; x uses r'
 * before its rounding to the residual's type.
 *
 * residual, residual_out [M, C] of type residual_dtype, y [M, C] of type
 * y_dtype (NULL: x is the norm of residual, residual_out is not written and
 * may be NULL, and post_weight and gate must be NULL), x [M, C] of type
 * x_dtype.  residual_out may be residual itself.  weight, post_weight fp32
 * [C]; gate and modulation fp32 [gate_rows, C] and [modulation_rows, C], their
 * row for row m being m / (M / rows): 1 shares one row, M gives each row its
 * own, and a number between, which must divide M, one per run of rows.
 * All device, contiguous, 16-byte aligned.  0 <= M <= 2^20, 32 <= C <= 2^20,
 * C % 32 == 0; eps and scale finite, eps >= 0.
 */
q4_status q4_add_rmsnorm(const void *residual, int residual_dtype, const void *y, int y_dtype, int64_t M, int64_t C,
                         const float *weight, const float *post_weight, const float *gate, int64_t gate_rows,
                         float scale, const float *modulation, int64_t modulation_rows, float eps,
                         void *residual_out, void *x, int x_dtype, void *stream);

/*
 * Adjusts logits z [M, V] (fp32, row-major, device) of each row's next token:
 *     z1 = z / rho if z > 0 else z * rho   for tokens in the row's history
 *     z2 = z1 - frequency * n - presence * [n > 0],  n = how often the token
 *          is in the history after its first prompt_lengths[row] ids
 *     z3 = z2 + the row's biases for the token
 *     out = z3 where the mask allows the token, else -inf.
 * history: int32 ids, row m's from cu_history[m] to cu_history[m + 1];
 * prompt_lengths int32 [M] (NULL: 0); repetition (rho), frequency, presence
 * fp32 [M], each may be NULL (1, 0, 0).  history may be NULL with cu_history
 * (none).  bias_ids int32 and bias fp32, row m's from cu_bias[m] to
 * cu_bias[m + 1] (all three NULL: none); repeated ids add up, in their order.
 * mask: 32-bit words [M, ceil(V / 32)], bit t % 32 of word t / 32 set where
 * token t is allowed (NULL: all are).  out may be logits itself.
 * Ids outside [0, V) are passed over; row bounds are held to
 * 0 .. history_size and 0 .. bias_size.  0 <= M <= 2^16 - 1, 1 <= V <= 2^24,
 * 0 <= history_size, bias_size < 2^31.  logits and out 16-byte aligned, the
 * others 4-byte aligned.
 */
q4_status q4_logits_adjust(const float *logits, int64_t M, int64_t V, const int32_t *history,
                           const int32_t *cu_history, int64_t history_size, const int32_t *prompt_lengths,
                           const float *repetition, const float *frequency, const float *presence,
                           const int32_t *bias_ids, const float *bias, const int32_t *cu_bias, int64_t bias_size,
                           const uint32_t *mask, float *out, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* Q4_DECODER_H */
