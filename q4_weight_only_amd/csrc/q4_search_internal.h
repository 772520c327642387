// Internal declarations of the operators around the paged cache (public ABI:
// include/q4_search.h).
#pragma once

#include "q4_decoder_internal.h"
#include "q4_search.h"

namespace q4 {

constexpr int kMaxBeams = 64, kMaxKeep = 128;
constexpr int kBeamSegment = 32;   // tokens of a segment of a row of logits

struct BeamArgs {
    const float *logits;
    int32_t groups, beams, V;
    const float *scores;
    const int32_t *finished;
    int32_t pad, keep;
    int32_t *parents, *tokens;
    float *out_scores;
    void *workspace;
};
size_t beam_workspace(int64_t rows, int64_t V);
hipError_t launch_beam_select(const BeamArgs &a, hipStream_t s);

struct AdvanceArgs {
    const int32_t *sequences, *lengths, *finished, *parents, *tokens;
    int32_t rows, width, n_out, eos, pad;
    int32_t *out_sequences, *out_lengths, *out_finished;
};
hipError_t launch_beam_advance(const AdvanceArgs &a, hipStream_t s);

struct ForkArgs {
    const int32_t *table, *lengths, *parents, *grow, *held;
    int32_t rows, width, n_out, grow_each, num_blocks;
    int32_t *out_table, *out_lengths, *refs, *src, *dst, *short_of;
    int32_t *workspace;
};
size_t fork_workspace(int64_t n_out, int64_t num_blocks);
hipError_t launch_kv_fork(const ForkArgs &a, hipStream_t s);

struct CompactArgs {
    const int32_t *table, *lengths, *held;
    int32_t rows, width, num_blocks;
    int32_t *out_table, *src, *dst, *live;
    int32_t *workspace;
};
size_t compact_workspace(int64_t num_blocks);
hipError_t launch_kv_compact(const CompactArgs &a, hipStream_t s);

constexpr int kLayersAtOnce = 32;   // caches of one launch: their addresses are its arguments

struct CopyArgs {
    uint8_t *data[kLayersAtOnce];
    uint8_t *summary[kLayersAtOnce];   // null: none
    int32_t layers, num_blocks, kv_heads, head_dim, n;
    const int32_t *src, *dst;
};
hipError_t launch_kv_copy(const CopyArgs &a, hipStream_t s);

struct SelectArgs {
    KvView kv;
    int8_t *summary;
    const uint16_t *q;
    int32_t q_heads, group;
    int32_t keep, first, recent;
    int32_t max_rows, max_blocks;
    int32_t *chosen;
    float *scores;           // [rows][kv_heads][max_blocks]
};
hipError_t launch_kv_summarize(const SelectArgs &a, int head_dim, hipStream_t s);
hipError_t launch_kv_select(const SelectArgs &a, int head_dim, hipStream_t s);

size_t attention_blocks_workspace(const AttentionArgs &a, int keep, int head_dim);
hipError_t launch_kv_attention_blocks(const AttentionArgs &a, const int32_t *chosen, int keep, int head_dim, hipStream_t s);

#ifdef __HIPCC__
// Sum over the lanes before this one, and over all: within 16 lanes by shifts, then the last lane
// of 16 to the next 16, and of 32 to the next 32.
template <typename T>
__device__ __forceinline__ T scan_wave(T v, T &total) {
    int sum = static_cast<int>(v);
    sum += __builtin_amdgcn_update_dpp(0, sum, 0x111, 0xF, 0xF, true);    // row_shr:1
    sum += __builtin_amdgcn_update_dpp(0, sum, 0x112, 0xF, 0xF, true);
    sum += __builtin_amdgcn_update_dpp(0, sum, 0x114, 0xF, 0xF, true);
    sum += __builtin_amdgcn_update_dpp(0, sum, 0x118, 0xF, 0xF, true);
    sum += __builtin_amdgcn_update_dpp(0, sum, 0x142, 0xA, 0xF, false);   // row_bcast:15 into rows 1 and 3
    sum += __builtin_amdgcn_update_dpp(0, sum, 0x143, 0xC, 0xF, false);   // row_bcast:31 into rows 2 and 3
    total = static_cast<T>(__builtin_amdgcn_readlane(sum, 63));
    return static_cast<T>(sum) - v;
}

// The same over a workgroup of WAVES waves.  `sums` may be used again after the
// caller's next barrier.
template <typename T, int WAVES>
__device__ __forceinline__ T scan_group(T v, T (&sums)[WAVES], T &total) {
    const int wave = threadIdx.x >> 6;
    T mine;
    const T before = scan_wave(v, mine);
    if ((threadIdx.x & 63) == 0) sums[wave] = mine;
    __syncthreads();
    T front = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        front += w < wave ? sums[w] : 0;
        total += sums[w];
    }
    return front + before;
}
#endif

}  // namespace q4
