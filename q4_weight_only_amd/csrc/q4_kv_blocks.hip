// Attention over chosen blocks of the paged 8-bit cache (include/q4_search.h).
// The mathematics is that of q4_kv_attention.hip; what differs is where the
// blocks come from, and that the rows of a sequence do not share them: a tile
// has the heads of one row that share a kv head.

#include "q4_kv_tile.h"
#include "q4_search_internal.h"

namespace q4 {
namespace {

constexpr int kBlocksWaves = 4;
constexpr int kTileHeads = 16;

// How a launch is shaped: a row's list is divided into `splits` chunks, the last of which
// has the rest of the list.
struct BlocksPlan {
    int tiles;            // of 16 heads, of a group
    int chunk, splits;
};

// Partial results, as for attention over all blocks: {m, l} [row][head][split],
// then O [row][head][split][D].  A split that saw nothing has {kLowest, kUnseen}
// and no O.
constexpr float kUnseen = -1.0f;   // no sum of weights

struct BlocksPartials {
    floatx2 *ml;
    float *o;
};
__device__ __forceinline__ BlocksPartials blocks_partials(const AttentionArgs &a, const BlocksPlan &p) {
    BlocksPartials w;
    w.ml = reinterpret_cast<floatx2 *>(a.workspace);
    w.o = a.workspace + (static_cast<int64_t>(a.kv.rows) * a.q_heads * p.splits * 2 + 3) / 4 * 4;   // 16-byte aligned
    return w;
}

// A workgroup has one row, up to 16 heads of a kv head, and one chunk of the
// row's list; its waves take the entries in turn.  A block goes from memory to the
// registers of one wave as its operand slices; the next block's codes are on their
// way while one is worked on (past the last block a resource of size 0 is read,
// which costs no memory traffic and needs no branch).
//
// What bounds it is memory where there are rows enough: 31 rows of 8 kv heads, 96 blocks,
// 195 MB, 33.5 us or 5.8 TB/s; one row, lengths, list, table and codes one after the other,
// 5.6 us; many rows of few heads, 61 of 8 with 40 blocks that are shared and so in the caches,
// the instructions for 16 heads of which few are there, 12.0 us (256 rows, 96 blocks: 71 us, 11 TB/s).
template <int D>
__global__ __launch_bounds__(64 * kBlocksWaves, 2) void attention_blocks_kernel(AttentionArgs a, BlocksPlan plan, const int32_t *chosen, int keep) {
    constexpr int W = kBlocksWaves, KQ = D / 32, DT = D / 16;
    __shared__ float part_m[W][16], part_l[W][16];
    __shared__ int part_seen[W];
    __shared__ floatx4 part_o[W][DT][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g4 = lane >> 4;
    const int b = blockIdx.z, head = blockIdx.x / plan.tiles, first_head = blockIdx.x % plan.tiles * kTileHeads;
    const int split = plan.splits == 1 ? 0 : blockIdx.y % plan.splits;
    const int grid_rows = plan.splits == 1 ? gridDim.y : gridDim.y / plan.splits;
    const KvSequence s = kv_sequence(a.kv, b);
    const int heads = a.group - first_head < kTileHeads ? a.group - first_head : kTileHeads;
    const int e0 = split * plan.chunk, e1 = split + 1 < plan.splits ? e0 + plan.chunk : keep;
    for (int t = plan.splits == 1 ? blockIdx.y : blockIdx.y / plan.splits; t < s.rows; t += grid_rows) {
        const int pos = s.pos0 + t;
        const int64_t row = s.row0 + t;
        const bool live = r < heads;
        const int64_t q_head = row * a.q_heads + head * a.group + first_head + (live ? r : heads - 1);
        const int32_t *list = chosen + (row * a.kv.kv_heads + head) * keep;
        bf16x8 q[KQ];
        load_q<D>(a, q_head * D, g4, q);
        Tile<D> tile[1];
        tile[0].clear();
        int seen_blocks = 0;
        for (int first = e0 + wave; first < e1; first += 64 * W) {
            const int entry = first + lane * W;
            const int my_block = entry < e1 ? list[entry] : -1;
            const bool visible = my_block >= 0 && my_block <= pos / kKvBlock && pos >= 0;
            const int my_id = visible ? kv_block_id(a.kv, b, my_block) : -1;
            const int my_exps =
                reinterpret_cast<const uint16_t *>(a.kv.exps)[static_cast<int64_t>(my_id < 0 ? 0 : my_id) * a.kv.kv_heads + head];
            uint64_t left = __ballot(visible);
            if (!left) continue;
            seen_blocks += __builtin_popcountll(left);
            u32x4 codes[2][2 * KQ];
            const auto fetch = [&](int i, bool more, u32x4(&to)[2 * KQ]) {   // K's slices are [0, KQ), V's follow
                const int id = __builtin_amdgcn_readlane(my_id, i);
                const int64_t plane = (static_cast<int64_t>(id < 0 ? 0 : id) * a.kv.kv_heads + head) * 2;
                const __amdgpu_buffer_rsrc_t src = __builtin_amdgcn_make_buffer_rsrc(
                    a.kv.data + plane * (kKvBlock * D), 0, more ? 2 * kKvBlock * D : 0, 0x00020000);
#pragma unroll
                for (int j = 0; j < 2 * KQ; ++j)
                    to[j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(src, lane * 16, 1024 * j, 2));   // streaming
            };
            const auto work = [&](int i, u32x4(&kc)[2 * KQ]) {
                const BlockScales scales = block_scales(a, __builtin_amdgcn_readlane(my_exps, i));
                const bool known = __builtin_amdgcn_readlane(my_id, i) >= 0;
                floatx4 st[1][2];
#pragma unroll
                for (int tt = 0; tt < 2; ++tt) {
                    st[0][tt] = (floatx4){0, 0, 0, 0};
#pragma unroll
                    for (int k = 0; k < KQ; ++k) {
                        const u32x4 w = kc[tt * (KQ / 2) + k / 2];
                        const bf16x8 kf = k % 2 ? codes_bf16(w.z, w.w) : codes_bf16(w.x, w.y);
                        st[0][tt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, q[k], st[0][tt], 0, 0, 0);
                    }
                    if (!known) st[0][tt] = (floatx4){kNan, kNan, kNan, kNan};
                }
                const int start = __builtin_amdgcn_readlane(my_block, i) * kKvBlock;
                if (start + kKvBlock - 1 > pos) {   // the row does not see some token
                    const int tok = start + 4 * g4;
                    hide_unseen(st[0], tok, 0, static_cast<uint32_t>(pos) + 1);
                    // bytes that it does not see may hold anything, and what is not
                    // a number must not meet a weight of 0: noted, a bit each, and cleared
                    const uint32_t in0 = bytes_in(tok, 0, pos + 1), in1 = bytes_in(tok + 16, 0, pos + 1);
                    uint32_t bad[2] = {0, 0};
#pragma unroll
                    for (int j = 0; j < 4 * KQ; ++j) {
                        const uint32_t v = kc[KQ + j / 4][j % 4] & (j % 2 ? in1 : in0), n = nan_bytes(v) >> 7;
                        bad[j / 8] |= n << (j % 8);
                        kc[KQ + j / 4][j % 4] = v & ~(n * 0xFFu);
                    }
                    if (__any((bad[0] | bad[1]) != 0)) {
                        const halfx8 seen = seen_tokens(tok, 0, static_cast<uint32_t>(pos) + 1);
#pragma unroll
                        for (int d = 0; d < DT; ++d) {
                            const uint32_t n0 = bad[d / 4] >> (d % 4 * 2), n1 = n0 >> 1;
                            tile[0].mark_nans(d, n0 & 0x01010101u, n1 & 0x01010101u, seen);
                        }
                    }
                }
                halfx8 wf[1];
                block_weights<D, 1>(tile, st, scales, wf);
#pragma unroll
                for (int d = 0; d < DT; ++d) {
                    const u32x4 v = kc[KQ + d / 2];
                    const halfx8 vf = d % 2 ? codes_f16(v.z, v.w) : codes_f16(v.x, v.y);
                    tile[0].o[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, wf[0], tile[0].o[d], 0, 0, 0);
                }
            };
            int now = __builtin_ctzll(left);
            left &= left - 1;
            fetch(now, true, codes[0]);
            asm volatile("" ::"v"(my_exps));   // has arrived before the loop, whose waits are for codes alone
            for (bool more = true; more;) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    more = left != 0;
                    const int next = more ? __builtin_ctzll(left) : now;
                    left &= left - 1;
                    fetch(next, more, codes[u ^ 1]);
                    work(now, codes[u]);
                    now = next;
                    if (!more) break;
                }
            }
        }
        // join the waves
        const float sum = row_sum(tile[0].l);
        __syncthreads();   // the row before has been read
        if (g4 == 0) {
            part_m[wave][r] = tile[0].m;
            part_l[wave][r] = sum;
        }
        if (lane == 0) part_seen[wave] = seen_blocks;
#pragma unroll
        for (int i = 0; i < DT; ++i) part_o[wave][i][lane] = tile[0].o[i];
        __syncthreads();
        float top = part_m[0][r];
        int seen = part_seen[0];
#pragma unroll
        for (int w = 1; w < W; ++w) {
            top = fmaxf(top, part_m[w][r]);
            seen += part_seen[w];
        }
        float f[W], total = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            f[w] = __builtin_amdgcn_exp2f(part_m[w][r] - top);
            total += f[w] * part_l[w][r];
        }
        if (!live) continue;
        const BlocksPartials ws = blocks_partials(a, plan);
        const int64_t at = q_head * plan.splits + split;
        if (plan.splits > 1 && seen == 0) {
            if (wave == 0 && g4 == 0) ws.ml[at] = (floatx2){kLowest, kUnseen};
            continue;
        }
        // nothing seen gives 0; a total of 0 otherwise means scores of -inf alone, whose softmax is not a number
        const float inv = seen == 0 ? 0.0f : 1.0f / total;
#pragma unroll
        for (int i = 0; i < DT / W; ++i) {
            const int tile_i = wave * (DT / W) + i, d = 16 * tile_i + 4 * g4;
            floatx4 acc = part_o[0][tile_i][lane] * f[0];
#pragma unroll
            for (int w = 1; w < W; ++w) acc = acc + part_o[w][tile_i][lane] * f[w];
            if (plan.splits > 1) *reinterpret_cast<floatx4 *>(ws.o + at * D + d) = acc;
            else if (a.out_bf16)
                *reinterpret_cast<bf16x4 *>(static_cast<__bf16 *>(a.out) + q_head * D + d) = __builtin_convertvector(acc * inv, bf16x4);
            else *reinterpret_cast<floatx4 *>(static_cast<float *>(a.out) + q_head * D + d) = acc * inv;
        }
        if (plan.splits > 1 && wave == 0 && g4 == 0) ws.ml[at] = (floatx2){top, total};
    }
}

// Joins the splits of a row's head: a wave each, whose lanes have D / 4 sets of four
// dimensions, and 256 / D of such sets the splits side by side.  All loads, for up to
// kJoinAhead splits a set, are on their way together.  (At most 64 splits: plan_blocks.)
constexpr int kJoinAhead = 8;

template <int D>
__global__ __launch_bounds__(256) void blocks_join_kernel(AttentionArgs a, BlocksPlan plan) {
    constexpr int LANES = D / 4, SETS = 64 / LANES;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int x = lane % LANES, set = lane / LANES;
    const int b = blockIdx.z, q_head = blockIdx.x * 4 + wave;
    if (q_head >= a.q_heads) return;
    const KvSequence s = kv_sequence(a.kv, b);
    const BlocksPartials ws = blocks_partials(a, plan);
    for (int t = blockIdx.y; t < s.rows; t += gridDim.y) {
        const int64_t at = static_cast<int64_t>(s.row0 + t) * a.q_heads + q_head;
        const floatx2 ml = lane < plan.splits ? ws.ml[at * plan.splits + lane] : (floatx2){kLowest, kUnseen};
        const floatx4 *o = reinterpret_cast<const floatx4 *>(ws.o + at * plan.splits * D) + x;
        floatx4 acc = {0, 0, 0, 0};
        float top = ml.x, f = 0.0f;
        for (int i0 = 0; i0 < plan.splits; i0 += SETS * kJoinAhead) {
            floatx4 part[kJoinAhead];
#pragma unroll
            for (int k = 0; k < kJoinAhead; ++k) {
                const int i = i0 + SETS * k + set;
                part[k] = o[(i < plan.splits ? i : 0) * LANES];
            }
            if (i0 == 0) {
#pragma unroll
                for (int i = 1; i < 64; i *= 2) top = fmaxf(top, __shfl_xor(top, i));
                f = ml.y != kUnseen ? __builtin_amdgcn_exp2f(ml.x - top) : kUnseen;
            }
#pragma unroll
            for (int k = 0; k < kJoinAhead; ++k) {
                const int i = i0 + SETS * k + set;
                const float fi = __shfl(f, i & 63);
                // (a split that saw nothing has no O: what was read for it is not used)
                if (i < plan.splits && fi != kUnseen) acc = acc + part[k] * fi;
            }
        }
        float total = ml.y != kUnseen ? f * ml.y : 0.0f;
        const bool some = __ballot(ml.y != kUnseen) != 0;   // (what is not a number is not kUnseen)
#pragma unroll
        for (int i = 1; i < 64; i *= 2) total += __shfl_xor(total, i);
#pragma unroll
        for (int i = LANES; i < 64; i *= 2)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[k] += __shfl_xor(acc[k], i);
        acc = acc * (some ? 1.0f / total : 0.0f);
        if (set != 0) continue;
        if (a.out_bf16) reinterpret_cast<bf16x4 *>(static_cast<__bf16 *>(a.out) + at * D)[x] = __builtin_convertvector(acc, bf16x4);
        else reinterpret_cast<floatx4 *>(static_cast<float *>(a.out) + at * D)[x] = acc;
    }
}

// Entries of a chunk at least, one for each wave; what a join has to save, as for
// attention over all blocks; and the most splits, one a lane of the join.  (One row of 8
// kv heads, 24 blocks 8.4 us, split 8.3; 32 blocks 9.7 and 8.1; 96 blocks 20.6 and 8.6.  8 rows,
// 24 blocks 8.8 and 9.2; 96 blocks 21.4 and 14.6.)
constexpr int kChunkLeast = kBlocksWaves, kSavedEntries = 22, kMostSplits = 64;

int64_t splits_wanted(const AttentionArgs &a, int64_t tiles) {
    const int64_t work = static_cast<int64_t>(a.kv.rows) * a.kv.kv_heads * tiles;
    const int64_t splits = work < 256 ? 256 / (work < 1 ? 1 : work) : 1;
    return splits < kMostSplits ? splits : kMostSplits;
}

// For lists with `entries` to divide.
BlocksPlan plan_blocks(const AttentionArgs &a, int64_t entries) {
    BlocksPlan p;
    p.tiles = (a.group + kTileHeads - 1) / kTileHeads;
    const int64_t splits = splits_wanted(a, p.tiles);
    int64_t chunk = (entries + splits - 1) / splits;
    if (chunk < kChunkLeast) chunk = kChunkLeast;
    if (entries - chunk < kSavedEntries + static_cast<int64_t>(a.kv.rows) * a.q_heads / 128) chunk = entries;
    p.chunk = static_cast<int>(chunk);
    p.splits = static_cast<int>((entries + chunk - 1) / chunk);
    return p;
}

template <int D>
hipError_t launch(const AttentionArgs &a, const int32_t *chosen, int keep, hipStream_t s) {
    // A list that kv_select made has its blocks in front, no more than the table has: so many are
    // divided.  (Another list may have more; the last chunk then takes longer.  Lists of 64 with 10 blocks
    // 6.8 us, divided as if they were full 8.2; 16 rows of them 6.9 and 10.1.)
    const BlocksPlan p = plan_blocks(a, keep < a.kv.table_width ? keep : a.kv.table_width);
    int rows = a.max_rows;   // the kernels loop where a launch cannot hold them all
    if (static_cast<int64_t>(rows) * p.splits > 65535) rows = 65535 / p.splits;
    const dim3 grid(a.kv.kv_heads * p.tiles, rows * p.splits, a.kv.batch);
    hipLaunchKernelGGL((attention_blocks_kernel<D>), grid, dim3(64 * kBlocksWaves), 0, s, a, p, chosen, keep);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    hipLaunchKernelGGL((blocks_join_kernel<D>), dim3((a.q_heads + 3) / 4, rows, a.kv.batch), dim3(256), 0, s, a, p);
    return hipGetLastError();
}

}  // namespace

size_t attention_blocks_workspace(const AttentionArgs &a, int keep, int head_dim) {
    // whatever the table's width: what is divided for a list is divided for a longer one
    const BlocksPlan p = plan_blocks(a, keep);
    if (p.splits == 1) return 0;
    const int64_t most = (keep + kChunkLeast - 1) / kChunkLeast, wanted = splits_wanted(a, p.tiles);
    const size_t parts = static_cast<size_t>(a.kv.rows) * a.q_heads * (most < wanted ? most : wanted);   // as in blocks_partials()
    return ((parts * 2 + 3) / 4 * 4 + parts * head_dim) * sizeof(float);
}

hipError_t launch_kv_attention_blocks(const AttentionArgs &a, const int32_t *chosen, int keep, int head_dim, hipStream_t s) {
    return head_dim == 128 ? launch<128>(a, chosen, keep, s) : launch<64>(a, chosen, keep, s);
}

}  // namespace q4
