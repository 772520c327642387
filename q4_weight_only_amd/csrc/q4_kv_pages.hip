// The pages of the paged cache: tables that go on from others, moving blocks
// together, and the copies that both ask for (include/q4_search.h).
//
// Who holds a block is counted anew from the tables in each call.  That reads
// all of them, which a fork does in any case, and leaves no counters that could go wrong
// beside them.  The counts are whole numbers, so the order of the atomics does not
// matter; every other step has one writer for each place.

#include "q4_search_internal.h"

namespace q4 {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ int32_t held_to(int32_t v, int32_t lo, int32_t hi) { return v < lo ? lo : v > hi ? hi : v; }

// ------------------------------------------------------------------- fork
// The workspace: for each block how many new sequences go on in it and the last of
// these; for each new sequence how many free blocks it and those before it
// want; the free blocks in their order, as far as they are wanted.
struct ForkSpace {
    int32_t *writers, *keeper;   // [num_blocks]
    int32_t *wanted;             // [n_out]
    int32_t *free;               // [num_blocks]
};
ForkSpace fork_space(int32_t *w, int64_t n_out, int64_t num_blocks) {
    ForkSpace s;
    s.writers = w;
    s.keeper = w + num_blocks;
    s.free = w + 2 * num_blocks;
    s.wanted = w + 3 * num_blocks;
    (void)n_out;
    return s;
}

__global__ __launch_bounds__(256) void fork_clear_kernel(ForkArgs a, ForkSpace w) {
    for (int64_t i = blockIdx.x * int64_t(256) + threadIdx.x; i < a.num_blocks; i += gridDim.x * int64_t(256)) {
        const int32_t h = a.held ? a.held[i] : 0;
        a.refs[i] = h > 0 ? h : 0;
        w.writers[i] = 0;
        w.keeper[i] = -1;
    }
}

// A new sequence before its blocks are handed out.
struct NewSequence {
    int32_t parent, was, grow, have, need;   // need: blocks with the tokens to come
    bool goes_on;                            // in a partly filled block, its last
};
__device__ __forceinline__ NewSequence new_sequence(const ForkArgs &a, int i) {
    NewSequence s;
    s.parent = a.parents[i];
    if (s.parent < 0 || s.parent >= a.rows) s.parent = -1;
    s.was = s.parent < 0 ? 0 : held_to(a.lengths[s.parent], 0, a.width * kKvBlock);
    s.grow = s.parent < 0 ? 0 : held_to(a.grow ? a.grow[i] : a.grow_each, 0, 1 << 25);
    s.have = (s.was + kKvBlock - 1) / kKvBlock;
    s.need = (s.was + s.grow + kKvBlock - 1) / kKvBlock;
    s.goes_on = s.was % kKvBlock != 0 && s.grow > 0;
    return s;
}

// A workgroup has 1024 entries of one new table row: they are copied and counted.
constexpr int kForkEntries = 1024;

__global__ __launch_bounds__(256) void fork_gather_kernel(ForkArgs a, ForkSpace w) {
    const int i = blockIdx.y;
    const NewSequence s = new_sequence(a, i);
    const int32_t *from = a.table + static_cast<int64_t>(s.parent < 0 ? 0 : s.parent) * a.width;
    int32_t *to = a.out_table + static_cast<int64_t>(i) * a.width;
#pragma unroll
    for (int k = 0; k < kForkEntries / 256; ++k) {
        const int t = blockIdx.x * kForkEntries + k * 256 + threadIdx.x;
        if (t >= a.width) break;
        int32_t id = -1;
        if (t < s.have) {
            id = from[t];
            if (id >= 0 && id < a.num_blocks) {
                atomicAdd(&a.refs[id], 1);
                if (t == s.have - 1 && s.goes_on) {
                    atomicAdd(&w.writers[id], 1);
                    atomicMax(&w.keeper[id], i);
                }
            }
        }
        to[t] = id;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) a.out_lengths[i] = s.was + s.grow;
}

// Whether new sequence i gets a copy of its last block: others hold it that do not
// go on in it, or it is not the last of those that do.
__device__ __forceinline__ bool gets_copy(const ForkArgs &a, const ForkSpace &w, const NewSequence &s, int i, int32_t &last) {
    last = -1;
    if (!s.goes_on) return false;
    last = a.table[static_cast<int64_t>(s.parent) * a.width + s.have - 1];
    if (last < 0 || last >= a.num_blocks) return false;
    return w.keeper[last] != i || a.refs[last] > w.writers[last];
}

// One workgroup: how many blocks each new sequence wants, the free ones, and
// their handing out.
constexpr int kHandThreads = 1024;

__global__ __launch_bounds__(kHandThreads) void fork_hand_kernel(ForkArgs a, ForkSpace w) {
    __shared__ int32_t sums[2][kHandThreads / 64];
    const int tid = threadIdx.x;
    int32_t want_all = 0;
    for (int i0 = 0, turn = 0; i0 < a.n_out; i0 += kHandThreads, turn ^= 1) {
        const int i = i0 + tid;
        int32_t want = 0;
        if (i < a.n_out) {
            const NewSequence s = new_sequence(a, i);
            int32_t last;
            const bool copy = gets_copy(a, w, s, i, last);
            // blocks for which the table has no room take none
            want = copy + (s.need < a.width ? s.need : a.width) - s.have;
        }
        int32_t total;
        const int32_t before = scan_group(want, sums[turn], total);
        if (i < a.n_out) w.wanted[i] = want_all + before + want;
        want_all += total;
    }
    // the first want_all free blocks
    constexpr int kEach = 4;
    int32_t found = 0;
    __syncthreads();
    for (int b0 = 0, turn = 0; b0 < a.num_blocks && found < want_all; b0 += kHandThreads * kEach, turn ^= 1) {
        const int b = b0 + tid * kEach;
        bool free[kEach];
        int32_t n = 0;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            free[k] = b + k < a.num_blocks && a.refs[b + k] == 0;
            n += free[k];
        }
        int32_t total;
        int32_t at = found + scan_group(n, sums[turn], total);
#pragma unroll
        for (int k = 0; k < kEach; ++k)
            if (free[k] && at < want_all) w.free[at++] = b + k;
        found += total;
    }
    __syncthreads();
    if (found > want_all) found = want_all;
    for (int i = tid; i < a.n_out; i += kHandThreads) {
        const NewSequence s = new_sequence(a, i);
        int32_t last;
        const bool copy = gets_copy(a, w, s, i, last);
        const int32_t at = i ? w.wanted[i - 1] : 0, upto = w.wanted[i];
        int32_t dst = -1;
        if (copy) {
            if (at < found) dst = w.free[at];
            a.out_table[static_cast<int64_t>(i) * a.width + s.have - 1] = dst;
        }
        a.src[i] = dst >= 0 ? last : -1;
        a.dst[i] = dst;
        a.short_of[i] = (upto > found ? upto - (at > found ? at : found) : 0) + (s.need > a.width ? s.need - a.width : 0);
    }
    // new blocks, one a thread: the sequence by bisection
    for (int k = tid; k < want_all; k += kHandThreads) {
        int lo = 0, hi = a.n_out - 1;   // the first with wanted > k
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (w.wanted[mid] > k) hi = mid;
            else lo = mid + 1;
        }
        const NewSequence s = new_sequence(a, lo);
        int32_t last;
        const bool copy = gets_copy(a, w, s, lo, last);
        const int32_t place = k - (lo ? w.wanted[lo - 1] : 0) - copy;
        if (place >= 0) a.out_table[static_cast<int64_t>(lo) * a.width + s.have + place] = k < found ? w.free[k] : -1;
    }
    __syncthreads();   // refs has been read
    for (int i = tid; i < a.n_out; i += kHandThreads) {
        const NewSequence s = new_sequence(a, i);
        int32_t last;
        if (!s.goes_on) continue;
        last = a.table[static_cast<int64_t>(s.parent) * a.width + s.have - 1];
        if (last < 0 || last >= a.num_blocks || w.keeper[last] != i) continue;
        // the last of those that go on in a block takes all copies from its count
        const int32_t kept = a.refs[last] > w.writers[last] ? 0 : 1;
        a.refs[last] -= w.writers[last] - kept;
    }
    for (int k = tid; k < found; k += kHandThreads) a.refs[w.free[k]] = 1;
}

// ---------------------------------------------------------------- compact
// The workspace: a byte for each block that a table names; for each tile of
// blocks how many are live and how many of these may move; where blocks went.
constexpr int kTileBlocksHeld = 4096, kTileThreads = 256, kTileEach = kTileBlocksHeld / kTileThreads;

struct CompactSpace {
    int32_t *named;     // [num_blocks]: not 0 where a sequence holds the block
    int32_t *moved;     // [num_blocks]: where it goes
    int32_t *live, *movable;   // [tiles]
    int32_t tiles;
};
int64_t tiles_of(int64_t num_blocks) { return (num_blocks + kTileBlocksHeld - 1) / kTileBlocksHeld; }
CompactSpace compact_space(int32_t *w, int64_t num_blocks) {
    CompactSpace s;
    s.tiles = static_cast<int32_t>(tiles_of(num_blocks));
    s.named = w;
    s.moved = w + num_blocks;
    s.live = w + 2 * num_blocks;
    s.movable = s.live + s.tiles;
    return s;
}

__global__ __launch_bounds__(256) void compact_clear_kernel(CompactArgs a, CompactSpace w) {
    const int64_t half = a.num_blocks / 2 > 1 ? a.num_blocks / 2 : 1;
    for (int64_t i = blockIdx.x * int64_t(256) + threadIdx.x; i < a.num_blocks; i += gridDim.x * int64_t(256)) {
        w.named[i] = 0;
        if (i < half) {
            a.src[i] = -1;
            a.dst[i] = -1;
        }
    }
}

__global__ __launch_bounds__(256) void compact_mark_kernel(CompactArgs a, CompactSpace w) {
    const int row = blockIdx.y;
    const int32_t n = held_to(a.lengths[row], 0, a.width * kKvBlock), have = (n + kKvBlock - 1) / kKvBlock;
    const int32_t *from = a.table + static_cast<int64_t>(row) * a.width;
    for (int t = blockIdx.x * 256 + threadIdx.x; t < have; t += gridDim.x * 256) {
        const int32_t id = from[t];
        if (id >= 0 && id < a.num_blocks) w.named[id] = 1;   // whoever writes it writes the same
    }
}

__device__ __forceinline__ void block_state(const CompactArgs &a, const CompactSpace &w, int b, bool &live, bool &movable) {
    live = movable = false;
    if (b >= a.num_blocks) return;
    const bool pinned = a.held && a.held[b] > 0;
    live = pinned || w.named[b] != 0;
    movable = live && !pinned;
}

__global__ __launch_bounds__(kTileThreads) void compact_count_kernel(CompactArgs a, CompactSpace w) {
    __shared__ int32_t sums[2][kTileThreads / 64];
    int32_t live = 0, movable = 0;
    for (int k = 0; k < kTileEach; ++k) {
        bool l, m;
        block_state(a, w, blockIdx.x * kTileBlocksHeld + k * kTileThreads + threadIdx.x, l, m);
        live += l;
        movable += m;
    }
    int32_t all_live, all_movable;
    scan_group(live, sums[0], all_live);
    scan_group(movable, sums[1], all_movable);
    if (threadIdx.x == 0) {
        w.live[blockIdx.x] = all_live;
        w.movable[blockIdx.x] = all_movable;
    }
}

// Every workgroup works out L and what lies before its tile from all tiles'
// counts; of the tile that L falls into it counts the blocks itself.
__global__ __launch_bounds__(kTileThreads) void compact_list_kernel(CompactArgs a, CompactSpace w) {
    __shared__ int32_t sums[6][kTileThreads / 64];
    const int tid = threadIdx.x, tile = blockIdx.x;
    int32_t all = 0;
    for (int i = tid; i < w.tiles; i += kTileThreads) all += w.live[i];
    int32_t limit;
    scan_group(all, sums[0], limit);
    const int border = limit / kTileBlocksHeld;   // L's tile (past the last where all blocks are live)
    // free blocks below L in the tiles before, and blocks that move in them
    int32_t slots_before = 0, moves_before = 0;
    for (int i = tid; i < tile && i < w.tiles; i += kTileThreads) {
        if (i < border) slots_before += kTileBlocksHeld - w.live[i];
        if (i > border) moves_before += w.movable[i];
    }
    if (tile > border) {
        for (int k = 0; k < kTileEach; ++k) {
            const int b = border * kTileBlocksHeld + k * kTileThreads + tid;
            bool l, m;
            block_state(a, w, b, l, m);
            moves_before += m && b >= limit;
            slots_before += !l && b < limit;
        }
    }
    int32_t slots, moves;
    scan_group(slots_before, sums[1], slots);
    scan_group(moves_before, sums[2], moves);
    const int half = a.num_blocks / 2 > 1 ? a.num_blocks / 2 : 1;
    const int first = tile * kTileBlocksHeld + tid * kTileEach;
    int32_t my_slots = 0, my_moves = 0;
    uint32_t slot_bits = 0, move_bits = 0;
#pragma unroll
    for (int k = 0; k < kTileEach; ++k) {
        bool l, m;
        block_state(a, w, first + k, l, m);
        const bool slot = first + k < limit && !l, move = first + k >= limit && m;
        my_slots += slot;
        my_moves += move;
        slot_bits |= static_cast<uint32_t>(slot) << k;
        move_bits |= static_cast<uint32_t>(move) << k;
    }
    int32_t total;
    int32_t slot_at = slots + scan_group(my_slots, sums[3], total), move_at = moves + scan_group(my_moves, sums[4], total);
#pragma unroll
    for (int k = 0; k < kTileEach; ++k) {
        if (slot_bits >> k & 1) {
            if (slot_at < half) a.dst[slot_at] = first + k;
            ++slot_at;
        }
        if (move_bits >> k & 1) {
            if (move_at < half) a.src[move_at] = first + k;
            ++move_at;
        }
    }
    if (tile == 0 && tid == 0) *a.live = limit;
}

// There may be more free blocks below L than blocks that move: the rest of dst
// is cleared.  And where each block went.
__global__ __launch_bounds__(256) void compact_map_kernel(CompactArgs a, CompactSpace w) {
    const int half = a.num_blocks / 2 > 1 ? a.num_blocks / 2 : 1;
    for (int i = blockIdx.x * 256 + threadIdx.x; i < half; i += gridDim.x * 256) {
        const int32_t src = a.src[i];
        if (src < 0) a.dst[i] = -1;
        else w.moved[src] = a.dst[i];
    }
}

__global__ __launch_bounds__(256) void compact_table_kernel(CompactArgs a, CompactSpace w) {
    const int row = blockIdx.y, limit = *a.live;
    const int32_t n = held_to(a.lengths[row], 0, a.width * kKvBlock), have = (n + kKvBlock - 1) / kKvBlock;
    const int64_t at = static_cast<int64_t>(row) * a.width;
    for (int t = blockIdx.x * 256 + threadIdx.x; t < a.width; t += gridDim.x * 256) {
        int32_t id = t < have ? a.table[at + t] : -1;
        if (id < 0 || id >= a.num_blocks) id = -1;
        else if (id >= limit && !(a.held && a.held[id] > 0)) id = w.moved[id];
        a.out_table[at + t] = id;
    }
}

// ------------------------------------------------------------------- copy
// A wave has a piece of 4 KB of the blocks of one layer, for some of the pairs: it
// reads their ids at once and copies the piece of those that there are.
constexpr int kPiece = 4096;

__global__ __launch_bounds__(256) void copy_kernel(CopyArgs a, int pieces, int pairs_each) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t chunk = blockIdx.x * int64_t(4) + wave;
    const int layer = blockIdx.y / pieces, piece = blockIdx.y % pieces;
    const int64_t first = chunk * pairs_each;
    if (first >= a.n) return;
    int32_t src = -1, dst = -1;
    if (lane < pairs_each && first + lane < a.n) {
        src = a.src[first + lane];
        dst = a.dst[first + lane];
    }
    const bool some = src >= 0 && src < a.num_blocks && dst >= 0 && dst < a.num_blocks;
    const int64_t block_bytes = static_cast<int64_t>(a.kv_heads) * 2 * kKvBlock * a.head_dim;   // a multiple of kPiece
    uint8_t *data = a.data[layer];
    uint8_t *exps = data + a.num_blocks * block_bytes;
    for (uint64_t left = __ballot(some); left; left &= left - 1) {
        const int i = __builtin_ctzll(left);
        const int64_t from = __builtin_amdgcn_readlane(src, i), to = __builtin_amdgcn_readlane(dst, i);
        const u32x4 *p = reinterpret_cast<const u32x4 *>(data + from * block_bytes + piece * int64_t(kPiece)) + lane;
        u32x4 *q = reinterpret_cast<u32x4 *>(data + to * block_bytes + piece * int64_t(kPiece)) + lane;
        u32x4 v[kPiece / 1024];
#pragma unroll
        for (int k = 0; k < kPiece / 1024; ++k) v[k] = p[64 * k];
#pragma unroll
        for (int k = 0; k < kPiece / 1024; ++k) q[64 * k] = v[k];
        if (piece == 0) {
            const int n = a.kv_heads * 2;
            for (int k = lane; k < n; k += 64) exps[to * n + k] = exps[from * n + k];
        }
        if (uint8_t *summary = a.summary[layer]) {   // its pieces are a 32nd of the codes': one of 128 bytes
            const int64_t bytes = static_cast<int64_t>(a.kv_heads) * 2 * a.head_dim, part = kPiece / kKvBlock;
            if (lane < part / 16)
                reinterpret_cast<u32x4 *>(summary + to * bytes + piece * part)[lane] =
                    reinterpret_cast<const u32x4 *>(summary + from * bytes + piece * part)[lane];
        }
    }
}

uint32_t blocks_of(int64_t n, int64_t each, int64_t most) {
    const int64_t b = (n + each - 1) / each;
    return static_cast<uint32_t>(b < 1 ? 1 : b > most ? most : b);
}

}  // namespace

size_t fork_workspace(int64_t n_out, int64_t num_blocks) {
    return (static_cast<size_t>(3 * num_blocks + n_out) * 4 + 15) / 16 * 16;
}

hipError_t launch_kv_fork(const ForkArgs &a, hipStream_t s) {
    const ForkSpace w = fork_space(a.workspace, a.n_out, a.num_blocks);
    hipLaunchKernelGGL(fork_clear_kernel, dim3(blocks_of(a.num_blocks, 256, 2048)), dim3(256), 0, s, a, w);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (a.n_out) {
        hipLaunchKernelGGL(fork_gather_kernel, dim3((a.width + kForkEntries - 1) / kForkEntries, a.n_out), dim3(256), 0, s, a, w);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(fork_hand_kernel, dim3(1), dim3(kHandThreads), 0, s, a, w);
        e = hipGetLastError();
    }
    return e;
}

size_t compact_workspace(int64_t num_blocks) {
    return (static_cast<size_t>(2 * num_blocks + 2 * tiles_of(num_blocks)) * 4 + 15) / 16 * 16;
}

hipError_t launch_kv_compact(const CompactArgs &a, hipStream_t s) {
    const CompactSpace w = compact_space(a.workspace, a.num_blocks);
    const dim3 tables(blocks_of(a.width, 256, 64), a.rows), blocks(blocks_of(a.num_blocks, 256, 2048));
    hipLaunchKernelGGL(compact_clear_kernel, blocks, dim3(256), 0, s, a, w);
    if (a.rows) hipLaunchKernelGGL(compact_mark_kernel, tables, dim3(256), 0, s, a, w);
    hipLaunchKernelGGL(compact_count_kernel, dim3(w.tiles), dim3(kTileThreads), 0, s, a, w);
    hipLaunchKernelGGL(compact_list_kernel, dim3(w.tiles), dim3(kTileThreads), 0, s, a, w);
    hipLaunchKernelGGL(compact_map_kernel, blocks, dim3(256), 0, s, a, w);
    if (a.rows) hipLaunchKernelGGL(compact_table_kernel, tables, dim3(256), 0, s, a, w);
    return hipGetLastError();
}

hipError_t launch_kv_copy(const CopyArgs &a, hipStream_t s) {
    const int pieces = a.kv_heads * 2 * kKvBlock * a.head_dim / kPiece;
    // a wave for each piece while there is room for that many, then up to 64 pairs a wave
    const int64_t all = static_cast<int64_t>(a.n) * pieces * a.layers;
    int64_t each = all / 8192;
    each = each < 1 ? 1 : each > 64 ? 64 : each;
    const int64_t chunks = (a.n + each - 1) / each;
    const int64_t rows = static_cast<int64_t>(pieces) * a.layers;   // at most 256 * 2 * 128 / 128 * 32
    hipLaunchKernelGGL(copy_kernel, dim3(static_cast<uint32_t>((chunks + 3) / 4), static_cast<uint32_t>(rows)), dim3(256), 0, s, a,
                       pieces, static_cast<int>(each));
    return hipGetLastError();
}

}  // namespace q4
