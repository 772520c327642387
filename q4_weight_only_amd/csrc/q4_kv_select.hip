// Bounds of the keys of a cache's blocks, and the blocks that matter most to a
// row by them (include/q4_search.h).
//
// The mathematics.  q . k <= sum_d max(q_d hi_d, q_d lo_d) for every key k between
// lo and hi, and that is max(q, 0) . hi + min(q, 0) . lo.  Summed over the heads of a
// group the bound is linear in Q+ = sum max(q_h, 0) and Q- = sum min(q_h, 0), so
// a group of heads costs as much as one.  With Q in 14 bits, as two parts of 7 on
// 8-bit matrix products, and bounds in 8, the sums are exact whole numbers, and what
// is chosen does not depend on the order in which anything is added.

#include "q4_search_internal.h"

namespace q4 {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef float floatx2 __attribute__((ext_vector_type(2)));

// ------------------------------------------------------------------ bounds
// The smaller or larger over the 16 lanes of a row of lanes.
template <int CTRL, bool MAX>
__device__ __forceinline__ int pick_dpp(int v) {
    const int other = __builtin_amdgcn_update_dpp(v, v, CTRL, 0xF, 0xF, false);
    return MAX ? (other > v ? other : v) : (other < v ? other : v);
}
template <bool MAX>
__device__ __forceinline__ int pick_of_16(int v) {
    v = pick_dpp<0xB1, MAX>(v);     // lane ^ 1
    v = pick_dpp<0x4E, MAX>(v);     // lane ^ 2
    v = pick_dpp<0x141, MAX>(v);    // 7 - lane, within 8
    return pick_dpp<0x140, MAX>(v); // 15 - lane, within 16
}

// A code's place in the order of the values: a code of sign and magnitude as a whole number.
__device__ __forceinline__ int place_of(uint32_t code) { return code & 0x80 ? -static_cast<int>(code & 0x7F) : static_cast<int>(code & 0x7F); }

// The value at that place, over 4.
__device__ __forceinline__ float quarter_of(int place) {
    const uint32_t code = place < 0 ? 0x80u | static_cast<uint32_t>(-place) : static_cast<uint32_t>(place);
    return __builtin_amdgcn_cvt_f32_fp8(code, 0) * 0.25f;
}

constexpr int kNanPlace = 127;   // of 0x7F; -127 of 0xFF

// A wave has the keys of one block and kv head.  Lane l of a 1 KB piece has 16
// dimensions, l / 16, of one token, l % 16.
template <int D>
__global__ __launch_bounds__(256) void summarize_kernel(SelectArgs a) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int b = blockIdx.z, head = blockIdx.x * 4 + wave;
    if (head >= a.kv.kv_heads) return;
    const KvSequence s = kv_sequence(a.kv, b);
    if (s.rows == 0 || s.length == 0) return;
    const int begin = (s.pos0 < 0 ? 0 : s.pos0) / kKvBlock, end = (s.length + kKvBlock - 1) / kKvBlock;
    for (int block = begin + blockIdx.y; block < end; block += gridDim.y) {
        const int32_t id = kv_block_id(a.kv, b, block);
        if (id < 0) continue;
        const int64_t plane = static_cast<int64_t>(id) * a.kv.kv_heads + head;
        const u32x4 *src = reinterpret_cast<const u32x4 *>(a.kv.data + plane * (2 * kKvBlock * D));
        u32x4 codes[2][D / 64];   // of both halves of the tokens
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < D / 64; ++j) codes[h][j] = src[(h * (D / 64) + j) * 64 + lane];
        const int tokens = s.length - block * kKvBlock;   // 32 and more: all
        const bool there[2] = {(lane & 15) < tokens, (lane & 15) + 16 < tokens};
        int8_t *out = a.summary + plane * (2 * D);
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
            uint32_t hi[4] = {0, 0, 0, 0}, lo[4] = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                int top = -128, low = 128;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int p = place_of(codes[h][j][i / 4] >> (i % 4 * 8) & 0xFF);
                    if (there[h]) {
                        top = p > top ? p : top;
                        low = p < low ? p : low;
                    }
                }
                top = pick_of_16<true>(top);
                low = pick_of_16<false>(low);
                const bool bad = top == kNanPlace || low == -kNanPlace;
                const int up = bad ? 127 : static_cast<int>(ceilf(quarter_of(top)));
                const int down = bad ? -127 : static_cast<int>(floorf(quarter_of(low)));
                hi[i / 4] |= static_cast<uint32_t>(up & 0xFF) << (i % 4 * 8);
                lo[i / 4] |= static_cast<uint32_t>(down & 0xFF) << (i % 4 * 8);
            }
            if (lane % 16 == 0) {
                const int d = 64 * j + lane;   // 16 * (lane / 16)
                *reinterpret_cast<u32x4 *>(out + d) = (u32x4){hi[0], hi[1], hi[2], hi[3]};
                *reinterpret_cast<u32x4 *>(out + D + d) = (u32x4){lo[0], lo[1], lo[2], lo[3]};
            }
        }
    }
}

// ------------------------------------------------------------------ scores
constexpr int kScoreTiles = 2;   // of 16 blocks, of a wave at a time
constexpr int kScoreWaves = 4;

// A workgroup has 16 rows of one sequence and kv head and some of its blocks; a
// wave's product is 16 rows x 16 blocks, the bounds straight from memory to operand
// registers: lane l has 16 bytes at 16 (l / 16) of each 64 of block l % 16.
template <int D>
__global__ __launch_bounds__(64 * kScoreWaves) void score_kernel(SelectArgs a, int blocks_each) {
    constexpr int KK = 2 * D / 64, kStride = 2 * D + 16;   // bytes of a row of q in LDS
    __shared__ __align__(16) uint8_t parts[2][16][kStride];   // high and low 7 bits of Q+ and Q-
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int b = blockIdx.z, head = blockIdx.x % a.kv.kv_heads, begin = blockIdx.x / a.kv.kv_heads * blocks_each;
    const KvSequence s = kv_sequence(a.kv, b);
    for (int t0 = blockIdx.y * 16; t0 < s.rows; t0 += gridDim.y * 16) {
        const int rows = s.rows - t0 < 16 ? s.rows - t0 : 16;
        const int last = s.pos0 + t0 + rows - 1;   // position of the last row
        int end = last < 0 ? 0 : last / kKvBlock + 1;
        end = end < a.max_blocks ? end : a.max_blocks;
        if (begin >= end) continue;                // the same for the workgroup
        __syncthreads();                           // the rows before have been read
        {   // D / 2 lanes have a row, a pair of dimensions each
            constexpr int kLanes = D / 2, kAtOnce = 64 * kScoreWaves / kLanes;
            const int pair = threadIdx.x % kLanes;
#pragma unroll
            for (int i = 0; i < 16 / kAtOnce; ++i) {
                const int row = i * kAtOnce + threadIdx.x / kLanes;
                if (i > 0 && i * kAtOnce >= rows) {   // no row of these
                    for (int p = 0; p < 2; ++p) {
                        *reinterpret_cast<uint16_t *>(&parts[p][row][2 * pair]) = 0;
                        *reinterpret_cast<uint16_t *>(&parts[p][row][D + 2 * pair]) = 0;
                    }
                    continue;
                }
                double up[2] = {0, 0}, down[2] = {0, 0};
                if (row < rows) {
                    const uint32_t *q = reinterpret_cast<const uint32_t *>(
                        a.q + (static_cast<int64_t>(s.row0 + t0 + row) * a.q_heads + head * a.group) * D) + pair;
                    for (int h = 0; h < a.group; ++h) {
                        const uint32_t v = q[h * (D / 2)];
                        const float x[2] = {__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u)};
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            // what is not a number goes into both
                            up[k] += x[k] < 0.0f ? 0.0f : x[k];
                            down[k] += x[k] > 0.0f ? 0.0f : x[k];
                        }
                    }
                }
                double top = fmax(fmax(up[0], up[1]), -fmin(down[0], down[1]));
                bool fine = __builtin_isfinite(up[0]) && __builtin_isfinite(up[1]) && __builtin_isfinite(down[0]) && __builtin_isfinite(down[1]);
#pragma unroll
                for (int m = 1; m < kLanes; m *= 2) top = fmax(top, __shfl_xor(top, m));
                const uint64_t all = __ballot(fine);
                fine = kLanes == 64 ? all == ~uint64_t(0) : static_cast<uint32_t>(lane < 32 ? all : all >> 32) == ~0u;
                const int e = static_cast<int>(static_cast<uint64_t>(__double_as_longlong(top)) >> 52 & 0x7FF) - 1022;   // top < 2^e
                uint32_t high[2] = {0, 0}, low[2] = {0, 0};
                if (fine && top > 0.0) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int v = static_cast<int>(__builtin_rint(__builtin_ldexp(k < 2 ? up[k & 1] : down[k & 1], 13 - e)));
                        high[k / 2] |= static_cast<uint32_t>((v >> 7) & 0xFF) << (k % 2 * 8);
                        low[k / 2] |= static_cast<uint32_t>(v & 0x7F) << (k % 2 * 8);
                    }
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    *reinterpret_cast<uint16_t *>(&parts[0][row][k * D + 2 * pair]) = static_cast<uint16_t>(high[k]);
                    *reinterpret_cast<uint16_t *>(&parts[1][row][k * D + 2 * pair]) = static_cast<uint16_t>(low[k]);
                }
            }
        }
        __syncthreads();
        i32x4 qa[2][KK];
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int k = 0; k < KK; ++k) qa[p][k] = *reinterpret_cast<const i32x4 *>(&parts[p][r][64 * k + 16 * g]);
        const int stop = begin + blocks_each < end ? begin + blocks_each : end;
        for (int first = begin + wave * 16 * kScoreTiles; first < stop; first += kScoreWaves * 16 * kScoreTiles) {
            int32_t id[kScoreTiles];
            i32x4 bounds[kScoreTiles][KK];
            int e[kScoreTiles];
#pragma unroll
            for (int t = 0; t < kScoreTiles; ++t) id[t] = first + 16 * t + r < stop ? kv_block_id(a.kv, b, first + 16 * t + r) : -1;
#pragma unroll
            for (int t = 0; t < kScoreTiles; ++t) {
                const int64_t plane = static_cast<int64_t>(id[t] < 0 ? 0 : id[t]) * a.kv.kv_heads + head;
                e[t] = a.kv.exps[plane * 2];
                const i32x4 *src = reinterpret_cast<const i32x4 *>(a.summary + plane * (2 * D)) + g;
#pragma unroll
                for (int k = 0; k < KK; ++k) bounds[t][k] = __builtin_nontemporal_load(src + 4 * k);
            }
#pragma unroll
            for (int t = 0; t < kScoreTiles; ++t) {
                i32x4 high = {0, 0, 0, 0}, low = {0, 0, 0, 0};
#pragma unroll
                for (int k = 0; k < KK; ++k) {
                    high = __builtin_amdgcn_mfma_i32_16x16x64_i8(qa[0][k], bounds[t][k], high, 0, 0, 0);
                    low = __builtin_amdgcn_mfma_i32_16x16x64_i8(qa[1][k], bounds[t][k], low, 0, 0, 0);
                }
                const int block = first + 16 * t + r;
                if (block >= stop) continue;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int row = 4 * g + j;
                    if (row >= rows) break;
                    const float sum = static_cast<float>(high[j] * 128 + low[j]);   // below 2^28, rounded once
                    a.scores[(static_cast<int64_t>(s.row0 + t0 + row) * a.kv.kv_heads + head) * a.max_blocks + block] =
                        id[t] < 0 ? -__builtin_inff() : __builtin_ldexpf(sum, e[t]);
                }
            }
        }
    }
}

// --------------------------------------------------------------- selection
// Scores in the order of unsigned numbers; 0 is below every score's.
__device__ __forceinline__ uint32_t ordered(float s) {
    const uint32_t w = __float_as_uint(s);
    return w >> 31 ? ~w : w | 0x80000000u;
}

// A workgroup has one row and kv head.  The m-th largest of the scores between the
// first and the last blocks is found bit by bit, each time counting how many
// scores are no less, until that is m; then those are written in their order.
// LOOP: more scores than the workgroup's registers hold, read each time.
template <int THREADS, int EACH, bool LOOP>
__global__ __launch_bounds__(THREADS) void choose_kernel(SelectArgs a) {
    constexpr int WAVES = THREADS / 64, kHeld = THREADS * EACH;
    __shared__ int32_t counter[3];
    __shared__ uint32_t folded[2][WAVES];
    __shared__ int32_t sums[2][WAVES];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int b = blockIdx.z, head = blockIdx.x;
    const KvSequence s = kv_sequence(a.kv, b);
    for (int t = blockIdx.y; t < s.rows; t += gridDim.y) {
        const int pos = s.pos0 + t;
        const int count = pos < 0 || pos / kKvBlock >= a.max_blocks ? 0 : pos / kKvBlock + 1;
        const int64_t set = static_cast<int64_t>(s.row0 + t) * a.kv.kv_heads + head;
        int32_t *out = a.chosen + set * a.keep;
        if (count <= a.keep) {   // the same for the workgroup
            for (int i = tid; i < a.keep; i += THREADS) out[i] = i < count ? i : -1;
            continue;
        }
        const int lo = a.first, n = count - a.recent - lo, m = a.keep - a.first - a.recent;   // m of n
        for (int i = tid; i < a.first; i += THREADS) out[i] = i;
        for (int i = tid; i < a.recent; i += THREADS) out[a.keep - a.recent + i] = count - a.recent + i;
        if (m == 0) continue;
        const float *scores = a.scores + set * a.max_blocks + lo;
        const int turns = LOOP ? (n + kHeld - 1) / kHeld : 1;
        uint32_t key[EACH];
        const auto load = [&](int turn) {
#pragma unroll
            for (int k = 0; k < EACH; ++k) {
                const int i = turn * kHeld + tid * EACH + k;
                key[k] = i < n ? ordered(scores[i]) : 0;
            }
        };
        if (!LOOP) load(0);
        // the bits that all keys share
        uint32_t all_and = ~0u, all_or = 0;
        for (int turn = 0; turn < turns; ++turn) {
            if (LOOP) load(turn);
#pragma unroll
            for (int k = 0; k < EACH; ++k)
                if (turn * kHeld + tid * EACH + k < n) {
                    all_and &= key[k];
                    all_or |= key[k];
                }
        }
#pragma unroll
        for (int i = 1; i < 64; i *= 2) {
            all_and &= __shfl_xor(all_and, i);
            all_or |= __shfl_xor(all_or, i);
        }
        __syncthreads();   // the row before is done
        if (lane == 0) {
            folded[0][wave] = all_and;
            folded[1][wave] = all_or;
        }
        if (tid < 3) counter[tid] = 0;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            all_and &= folded[0][w];
            all_or |= folded[1][w];
        }
        const uint32_t differ = all_and ^ all_or;
        int bit = differ ? 31 - __builtin_clz(differ) : -1;
        uint32_t least = bit < 31 ? all_and >> (bit + 1) << (bit + 1) : 0;   // (bit 31: no common bits)
        int reach = n;   // how many keys are at least `least`
        for (int step = 0; bit >= 0 && reach != m; --bit, ++step) {
            const uint32_t probe = least | 1u << bit;
            int c = 0;
            for (int turn = 0; turn < turns; ++turn) {
                if (LOOP) load(turn);
#pragma unroll
                for (int k = 0; k < EACH; ++k) c += __builtin_popcountll(__ballot(key[k] >= probe));
            }
            // three counters in turn: one barrier a step
            if (lane == 0) atomicAdd(&counter[step % 3], c);
            if (tid == 0) counter[(step + 1) % 3] = 0;
            __syncthreads();
            c = counter[step % 3];
            if (c >= m) {
                least = probe;
                reach = c;
            }
        }
        // all above `least`, and of those equal to it the first; where m are at
        // least that, all of these
        int above = 0, equal = 0;
        const bool whole = reach == m;
        int need = 0;   // of the equal ones
        if (!whole) {
            int c = 0;
            for (int turn = 0; turn < turns; ++turn) {
                if (LOOP) load(turn);
#pragma unroll
                for (int k = 0; k < EACH; ++k) c += key[k] > least;
            }
            int32_t total;
            __syncthreads();
            scan_group(c, sums[0], total);
            need = m - total;
            __syncthreads();
        }
        for (int turn = 0; turn < turns; ++turn) {
            if (LOOP) load(turn);
            int mine = 0;   // both counts in one word: 16 bits each hold kHeld
#pragma unroll
            for (int k = 0; k < EACH; ++k) {
                const bool up = whole ? key[k] >= least && key[k] != 0 : key[k] > least;
                mine += up ? 0x10000 : !whole && key[k] == least && key[k] != 0 ? 1 : 0;
            }
            int32_t total;
            const uint32_t before = static_cast<uint32_t>(scan_group(mine, sums[turn & 1], total));
            int up_at = above + static_cast<int>(before >> 16), equal_at = equal + static_cast<int>(before & 0xFFFF);
#pragma unroll
            for (int k = 0; k < EACH; ++k) {
                const bool up = whole ? key[k] >= least && key[k] != 0 : key[k] > least;
                const bool same = !up && !whole && key[k] == least && key[k] != 0;
                const int at = up_at + (equal_at < need ? equal_at : need);
                if (up || (same && equal_at < need)) out[a.first + at] = lo + turn * kHeld + tid * EACH + k;
                up_at += up;
                equal_at += same;
            }
            above += static_cast<int>(static_cast<uint32_t>(total) >> 16);
            equal += total & 0xFFFF;
        }
    }
}

template <int D>
hipError_t launch_select(const SelectArgs &a, hipStream_t s) {
    const int64_t tiles = (static_cast<int64_t>(a.max_rows) + 15) / 16, sets = a.kv.kv_heads * static_cast<int64_t>(a.kv.batch) * tiles;
    // blocks of a workgroup: as many as leave four workgroups for every compute unit
    constexpr int kLeast = kScoreWaves * 16 * kScoreTiles;
    int64_t ranges = 1024 / sets;
    const int64_t most = (a.max_blocks + kLeast - 1) / kLeast;
    ranges = ranges < 1 ? 1 : ranges > most ? most : ranges;
    const int64_t each = ((a.max_blocks + ranges - 1) / ranges + kLeast - 1) / kLeast * kLeast;
    ranges = (a.max_blocks + each - 1) / each;
    const dim3 grid(static_cast<uint32_t>(a.kv.kv_heads * ranges), static_cast<uint32_t>(tiles < 65535 ? tiles : 65535), a.kv.batch);
    hipLaunchKernelGGL((score_kernel<D>), grid, dim3(64 * kScoreWaves), 0, s, a, static_cast<int>(each));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const dim3 rows(a.kv.kv_heads, a.max_rows < 65535 ? a.max_rows : 65535, a.kv.batch);
    if (a.max_blocks <= 1024) hipLaunchKernelGGL((choose_kernel<256, 4, false>), rows, dim3(256), 0, s, a);
    else if (a.max_blocks <= 4096) hipLaunchKernelGGL((choose_kernel<1024, 4, false>), rows, dim3(1024), 0, s, a);
    else if (a.max_blocks <= 16384) hipLaunchKernelGGL((choose_kernel<1024, 16, false>), rows, dim3(1024), 0, s, a);
    else hipLaunchKernelGGL((choose_kernel<1024, 16, true>), rows, dim3(1024), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_summarize(const SelectArgs &a, int head_dim, hipStream_t s) {
    // blocks that a sequence's rows lie in
    const int blocks = (a.max_rows + kKvBlock - 2) / kKvBlock + 1;
    const dim3 grid((a.kv.kv_heads + 3) / 4, blocks < 65535 ? blocks : 65535, a.kv.batch);
    if (head_dim == 128) hipLaunchKernelGGL((summarize_kernel<128>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((summarize_kernel<64>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_kv_select(const SelectArgs &a, int head_dim, hipStream_t s) {
    return head_dim == 128 ? launch_select<128>(a, s) : launch_select<64>(a, s);
}

}  // namespace q4
