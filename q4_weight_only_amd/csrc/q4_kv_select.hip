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
typedef _Float16 halfx2 __attribute__((ext_vector_type(2)));

// ------------------------------------------------------------------ bounds
// Codes two at a time as fp16, which holds every value of theirs, and not a number as
// such: the larger or smaller of two is not a number where one is not.
__device__ __forceinline__ uint32_t pair_of(uint32_t word, bool high) {
    return __builtin_bit_cast(uint32_t, high ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(word, 1.0f, true)
                                             : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(word, 1.0f, false));
}
template <bool MAX>
__device__ __forceinline__ uint32_t pick(uint32_t x, uint32_t y) {
    const halfx2 a = __builtin_bit_cast(halfx2, x), b = __builtin_bit_cast(halfx2, y);
    return __builtin_bit_cast(uint32_t, MAX ? __builtin_elementwise_maximum(a, b) : __builtin_elementwise_minimum(a, b));
}
constexpr uint32_t kLeast = 0xFC00FC00u, kMost = 0x7C007C00u;   // -inf and inf, two each

// One step of picking over lanes: a lane and its mate, CTRL, have 2 N words each, and
// each is left with N of them, the mate's picked in: the upper ones where `upper`.
template <int CTRL, bool MAX, int N>
__device__ __forceinline__ void halve(uint32_t (&v)[8], bool upper) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint32_t keep = upper ? v[N + i] : v[i], send = upper ? v[i] : v[N + i];
        v[i] = pick<MAX>(keep, __builtin_amdgcn_mov_dpp(send, CTRL, 0xF, 0xF, true));
    }
}
// Over 16 lanes, of 16 values in 8 words: the lane is left with its value in the
// low half, that of place_of_lane.
template <bool MAX>
__device__ __forceinline__ uint32_t pick_of_16(uint32_t (&v)[8], int lane) {
    halve<0x140, MAX, 4>(v, lane & 8);   // 15 - lane
    halve<0x141, MAX, 2>(v, lane & 4);   // 7 - lane, within 8
    halve<0x4E, MAX, 1>(v, lane & 2);    // lane ^ 2
    const uint32_t mine = lane & 1 ? v[0] >> 16 : v[0] & 0xFFFF, other = lane & 1 ? v[0] & 0xFFFF : v[0] >> 16;
    return pick<MAX>(mine, __builtin_amdgcn_mov_dpp(other, 0xB1, 0xF, 0xF, true));
}
__device__ __forceinline__ int place_of_lane(int lane) { return lane & 15; }   // the steps above take its bits from the top

// A wave has the keys of one block and kv head.  Lane l of a 1 KB piece has 16
// dimensions, l / 16, of one token, l % 16; after four steps over 16 lanes, in each of
// which a lane hands on half of what it has, it has one dimension of all tokens.  (All
// 16 dimensions in every lane: 7.5 us for one token of each of 8 heads, which is
// the time that its code takes to arrive; so it is 2.6, the launch and three waits.)
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
            uint32_t top[8], low[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t x = pair_of(codes[0][j][i / 2], i % 2), y = pair_of(codes[1][j][i / 2], i % 2);
                top[i] = pick<true>(there[0] ? x : kLeast, there[1] ? y : kLeast);
                low[i] = pick<false>(there[0] ? x : kMost, there[1] ? y : kMost);
            }
            const uint32_t most = pick_of_16<true>(top, lane), least = pick_of_16<false>(low, lane);
            const float up = static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(most)));
            const float down = static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(least)));
            const int d = 64 * j + (lane & 48) + place_of_lane(lane);
            const bool bad = !(up - down < __builtin_inff());   // not a number among them
            out[d] = static_cast<int8_t>(bad ? 127 : static_cast<int>(ceilf(up * 0.25f)));
            out[D + d] = static_cast<int8_t>(bad ? -127 : static_cast<int>(floorf(down * 0.25f)));
        }
    }
}

// ------------------------------------------------------------------ scores
constexpr int kScoreWaves = 4, kScoreBlocks = 16 * kScoreWaves;   // of a workgroup

// What `join` makes of the values of each LANES lanes (32 or 64), in all of them.
template <int CTRL>
__device__ __forceinline__ uint32_t from_lane(uint32_t v) {
    return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), CTRL, 0xF, 0xF, true));
}
template <int LANES, typename Join>
__device__ __forceinline__ uint32_t fold(uint32_t v, Join join) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    v = join(v, from_lane<0xB1>(v));    // lane ^ 1
    v = join(v, from_lane<0x4E>(v));    // lane ^ 2
    v = join(v, from_lane<0x141>(v));   // 7 - lane, within 8
    v = join(v, from_lane<0x140>(v));   // 15 - lane, within 16
    const u32x2 x = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(v, v, false, false));
    v = join(x.x, x.y);
    if (LANES == 64) {
        const u32x2 y = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(v, v, false, false));
        v = join(y.x, y.y);
    }
    return v;
}

// How the workgroups divide: units of 16 rows of a sequence and a range of its
// blocks, each for every kv head.
struct ScorePlan {
    int tiles;     // of 16 rows, of the sequence with most of them
    int ranges;    // of 16 blocks for each wave
    int units;     // tiles * ranges * sequences
};

// A workgroup has 16 rows of one sequence and kv head and a range of its blocks; a
// wave's product is 16 rows x 16 blocks, the bounds straight from memory to operand
// registers: lane l has 16 bytes at 16 (l / 16) of each 64 of block l % 16.  They are on
// their way while the rows' sums are formed, or the blocks before are worked on.
//
// What bounds it is memory: 31 sequences of up to 2047 blocks and 8 heads, 84 MB of bounds
// and exponents, in 18.2 us or 4.6 TB/s.  A block's exponents of all heads are in one line, so
// a unit's heads are given to one of the 8 dies, one after the other.
template <int D>
__global__ __launch_bounds__(64 * kScoreWaves) void score_kernel(SelectArgs a, ScorePlan plan) {
    constexpr int KK = 2 * D / 64, kStride = 2 * D + 16;   // bytes of a row of q in LDS
    __shared__ __align__(16) uint8_t parts[2][16][kStride];   // high and low 7 bits of Q+ and Q-
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int head = blockIdx.x / 8, unit = blockIdx.y * 8 + blockIdx.x % 8;   // workgroups are dealt to the dies in turn
    if (unit >= plan.units) return;
    const int range = unit % plan.ranges, b = unit / plan.ranges / plan.tiles, tile = unit / plan.ranges % plan.tiles;
    const KvSequence s = kv_sequence(a.kv, b);
    for (int t0 = tile * 16; t0 < s.rows; t0 += plan.tiles * 16) {
        const int rows = s.rows - t0 < 16 ? s.rows - t0 : 16;
        const int last = s.pos0 + t0 + rows - 1;   // position of the last row
        int end = last < 0 ? 0 : last / kKvBlock + 1;
        end = end < a.max_blocks ? end : a.max_blocks;
        // a wave's blocks of a range: their ids two ranges ahead, their bounds one
        const int step = plan.ranges * kScoreBlocks;
        const auto id_of = [&](int begin) {
            const int block = begin + 16 * wave + r;
            return block < end ? kv_block_id(a.kv, b, block) : -1;
        };
        int begin = range * kScoreBlocks;
        if (begin >= end) continue;   // the same for the workgroup
        int32_t id[2];
        i32x4 bounds[2][KK];
        int exps[2];
        const auto fetch = [&](int u) {
            const int64_t plane = static_cast<int64_t>(id[u] < 0 ? 0 : id[u]) * a.kv.kv_heads + head;
            const i32x4 *src = reinterpret_cast<const i32x4 *>(a.summary + plane * (2 * D)) + g;
#pragma unroll
            for (int k = 0; k < KK; ++k) bounds[u][k] = src[4 * k];   // a line is two of them: not nontemporal
            exps[u] = a.kv.exps[plane * 2];
        };
        id[0] = id_of(begin);
        // D / 2 lanes have a row of q, a pair of dimensions each; the first rows' first heads are read ahead of the bounds
        constexpr int kLanes = D / 2, kAtOnce = 64 * kScoreWaves / kLanes;
        const int pair = threadIdx.x % kLanes;
        const uint32_t *q = reinterpret_cast<const uint32_t *>(
            a.q + (static_cast<int64_t>(s.row0 + t0 + threadIdx.x / kLanes) * a.q_heads + head * a.group) * D) + pair;
        const int64_t q_step = static_cast<int64_t>(kAtOnce) * a.q_heads * (D / 2);
        const auto heads_of = [&](int i, int h0, uint32_t(&v)[4]) {   // (what is past the rows or the group is 0)
            const bool there = i * kAtOnce + static_cast<int>(threadIdx.x) / kLanes < rows;
#pragma unroll
            for (int h = 0; h < 4; ++h) v[h] = there && h0 + h < a.group ? q[i * q_step + (h0 + h) * (D / 2)] : 0;
        };
        uint32_t v[4];
        heads_of(0, 0, v);
        fetch(0);
        id[1] = id_of(begin + step);
        for (int i = 0; i < 16 / kAtOnce; ++i) {
            const int row = i * kAtOnce + threadIdx.x / kLanes;
            double up[2] = {0, 0}, down[2] = {0, 0};
            for (int h0 = 0; h0 < a.group; h0 += 4) {
                if (i + h0 > 0) heads_of(i, h0, v);
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const float x[2] = {__uint_as_float(v[h] << 16), __uint_as_float(v[h] & 0xFFFF0000u)};
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        // what is not a number goes into both
                        up[k] += x[k] < 0.0f ? 0.0f : x[k];
                        down[k] += x[k] > 0.0f ? 0.0f : x[k];
                    }
                }
            }
            const double most = fmax(fmax(up[0], up[1]), -fmin(down[0], down[1]));
            const bool fine = __builtin_isfinite(up[0] + up[1] - down[0] - down[1]);
            // most < 2^(e2 - 1022)
            const int e2 = static_cast<int>(fold<kLanes>(static_cast<uint32_t>(static_cast<uint64_t>(__double_as_longlong(most)) >> 52 & 0x7FF),
                                                         [](uint32_t x, uint32_t y) { return x > y ? x : y; }));
            const uint64_t all = __ballot(fine);
            const bool every = kLanes == 64 ? all == ~uint64_t(0) : static_cast<uint32_t>(lane < 32 ? all : all >> 32) == ~0u;
            uint32_t high[2] = {0, 0}, low[2] = {0, 0};
            if (every && e2 > 0) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int x = static_cast<int>(__builtin_rint(__builtin_ldexp(k < 2 ? up[k & 1] : down[k & 1], 13 + 1022 - e2)));
                    high[k / 2] |= static_cast<uint32_t>((x >> 7) & 0xFF) << (k % 2 * 8);
                    low[k / 2] |= static_cast<uint32_t>(x & 0x7F) << (k % 2 * 8);
                }
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                *reinterpret_cast<uint16_t *>(&parts[0][row][k * D + 2 * pair]) = static_cast<uint16_t>(high[k]);
                *reinterpret_cast<uint16_t *>(&parts[1][row][k * D + 2 * pair]) = static_cast<uint16_t>(low[k]);
            }
            if ((i + 1) * kAtOnce >= rows) break;   // rows past the last hold anything: their sums are not used
        }
        __syncthreads();
        for (bool more = true; more;) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int block = begin + 16 * wave + r;
                const int32_t now = id[u];
                more = begin + step < end;
                if (more) {
                    fetch(u ^ 1);
                    id[u] = id_of(begin + 2 * step);
                }
                i32x4 sum[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
                for (int k = 0; k < KK; ++k)
#pragma unroll
                    for (int p = 0; p < 2; ++p)
                        sum[p] = __builtin_amdgcn_mfma_i32_16x16x64_i8(*reinterpret_cast<const i32x4 *>(&parts[p][r][64 * k + 16 * g]), bounds[u][k], sum[p], 0, 0, 0);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int row = 4 * g + j;
                    if (block >= end || row >= rows) break;
                    const float total = static_cast<float>(sum[0][j] * 128 + sum[1][j]);   // below 2^28, rounded once
                    a.scores[(static_cast<int64_t>(s.row0 + t0 + row) * a.kv.kv_heads + head) * a.max_blocks + block] =
                        now < 0 ? -__builtin_inff() : __builtin_ldexpf(total, exps[u]);
                }
                begin += step;
                if (!more) break;
            }
        }
        __syncthreads();   // the rows' sums have been read
    }
}

// --------------------------------------------------------------- selection
// Scores in the order of unsigned numbers; 0 is below every score's.
__device__ __forceinline__ uint32_t ordered(float s) {
    const uint32_t w = __float_as_uint(s);
    return w >> 31 ? ~w : w | 0x80000000u;
}

__device__ __forceinline__ float unordered(uint32_t key) { return __uint_as_float(key >> 31 ? key & 0x7FFFFFFFu : ~key); }

constexpr uint32_t kLowestKey = 0x007FFFFF;   // of -inf
constexpr int kBins = 1024, kBinListed = 64;   // kBinListed: scores of a bin that may be ranked, one a lane

// A workgroup has one row and kv head.  The scores between the first and the last
// blocks are counted in bins of equal width; in the bin that the m-th largest falls
// into, the scores are ranked one by one (where they are too many, because they are equal
// or nearly so, the m-th is found two bits at a time, each time counting how many
// are no less).  Then the m largest are written in their order.  A thread has EACH / 4
// times four scores next to each other, THREADS * 4 apart.  LOOP: more scores than
// the workgroup's registers hold, read each time.
//
// What bounds it is one step after the other: lengths, scores, six barriers.  1024 blocks
// 4.7 us, 4096 6.2.  (Two bits at a time alone, some ten counts with a barrier each: 9.8 us
// for 4096 blocks; but of 250 scores that all fall into one bin, next to one that is far above
// them, both kernels take 9.5 us that way, and 34.7 ranked one by one.)
template <int THREADS, int EACH, bool LOOP>
__global__ __launch_bounds__(THREADS) void choose_kernel(SelectArgs a) {
    constexpr int WAVES = THREADS / 64, kHeld = THREADS * EACH, SETS = EACH / 4;
    typedef float floatx4_any __attribute__((ext_vector_type(4), aligned(4)));
    __shared__ int32_t counter[3][3];   // of a step, for each of its values
    __shared__ uint32_t folded[2][WAVES];
    __shared__ int32_t sums[2][2][SETS][WAVES];
    __shared__ __align__(16) int32_t bins[kBins];
    __shared__ uint32_t list_key[kBinListed];
    __shared__ int32_t list_index[kBinListed];
    __shared__ int32_t found[4];        // the bin, what is still wanted of it, how many it has, and of these listed
    __shared__ uint32_t found_key;      // all above it are chosen,
    __shared__ int32_t found_need;      // and so many of those equal to it
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
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
        const float *scores = a.scores + set * a.max_blocks + lo;
        const int turns = LOOP ? (n + kHeld - 1) / kHeld : 1;
        const auto index = [&](int turn, int k) { return turn * kHeld + (k / 4 * THREADS + tid) * 4 + k % 4; };
        uint32_t key[EACH];   // 0 past the last
        const auto load = [&](int turn) {
#pragma unroll
            for (int k = 0; k < EACH; k += 4) {
                const int i = index(turn, k);
                float v[4] = {0, 0, 0, 0};
                if (i + 4 <= n) {
                    const floatx4_any x = *reinterpret_cast<const floatx4_any *>(scores + i);
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[j] = x[j];
                } else {
#pragma unroll
                    for (int j = 0; j < 3; ++j)
                        if (i + j < n) v[j] = scores[i + j];
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) key[k + j] = i + j < n ? ordered(v[j]) : 0;
            }
        };
        if (!LOOP) load(0);
        for (int i = tid; i < a.first; i += THREADS) out[i] = i;
        for (int i = tid; i < a.recent; i += THREADS) out[a.keep - a.recent + i] = count - a.recent + i;
        if (m == 0) continue;
        // the smallest and the largest score, but for -inf
        uint32_t low = ~0u, high = 0;
        for (int turn = 0; turn < turns; ++turn) {
            if (LOOP) load(turn);
#pragma unroll
            for (int k = 0; k < EACH; ++k) {
                const uint32_t least = key[k] > kLowestKey ? key[k] : ~0u;
                low = least < low ? least : low;
                high = key[k] > high ? key[k] : high;
            }
        }
        low = fold<64>(low, [](uint32_t x, uint32_t y) { return x < y ? x : y; });
        high = fold<64>(high, [](uint32_t x, uint32_t y) { return x > y ? x : y; });
        __syncthreads();   // the row before is done
        if (lane == 0) {
            folded[0][wave] = low;
            folded[1][wave] = high;
        }
        for (int i = tid; i < kBins / 4; i += THREADS) reinterpret_cast<i32x4 *>(bins)[i] = (i32x4){0, 0, 0, 0};
        if (tid < 9) counter[tid / 3][tid % 3] = 0;
        if (tid == 0) found[0] = -1, found[3] = 0;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            low = folded[0][w] < low ? folded[0][w] : low;
            high = folded[1][w] > high ? folded[1][w] : high;
        }
        // bins 1 .. kBins - 1 from the smallest to the largest, -inf in 0; rounding does not change the order
        const float from = unordered(low), scale = (kBins - 2) / (unordered(high) - from);
        const bool spread = low < high && scale > 0.0f && scale < __builtin_inff();   // the same for the workgroup
        const auto bin_of = [&](uint32_t x) {
            const int bin = static_cast<int>(fmaxf((unordered(x) - from) * scale, 0.0f)) + 1;
            return x <= kLowestKey ? 0 : bin < kBins ? bin : kBins - 1;
        };
        uint32_t above = 0;   // all scores above it are chosen,
        int need = 0;         // and so many of those equal to it, the first ones
        if (spread) {
            for (int turn = 0; turn < turns; ++turn) {
                if (LOOP) load(turn);
#pragma unroll
                for (int k = 0; k < EACH; ++k)
                    if (key[k]) atomicAdd(&bins[bin_of(key[k])], 1);
            }
            __syncthreads();
            if (wave == 0) {   // from the last bin down, 16 a lane
                constexpr int kOf = kBins / 64;
                static_assert(kOf == 16, "a lane's bins are those of 16 lanes");
                int all = 0;
#pragma unroll
                for (int i = 0; i < kOf; i += 4) {
                    const i32x4 x = *reinterpret_cast<const i32x4 *>(&bins[kBins - kOf * (lane + 1) + i]);
                    all += (x[0] + x[1]) + (x[2] + x[3]);
                }
                int32_t total;
                const int before = scan_wave(all, total);
                // the lane whose bins reach m, and of these, a lane each, the one that does
                const int at = __builtin_ctzll(__ballot(before + all >= m)), last = kBins - 1 - kOf * at;
                const int mine = lane < kOf ? bins[last - (lane & (kOf - 1))] : 0;
                const int above = __builtin_amdgcn_readlane(before, at) + scan_wave(mine, total);
                const int bin = __builtin_ctzll(__ballot(above + mine >= m));
                if (lane == bin) {
                    found[0] = last - lane;
                    found[1] = m - above;
                    found[2] = mine;
                }
            }
            __syncthreads();
        }
        const int border = found[0], wanted = found[1], size = found[2];
        if (spread && size <= kBinListed) {   // the same for the workgroup
            for (int turn = 0; turn < turns; ++turn) {
                if (LOOP) load(turn);
#pragma unroll
                for (int k = 0; k < EACH; ++k)
                    if (key[k] && bin_of(key[k]) == border) {
                        const int i = atomicAdd(&found[3], 1);
                        list_key[i] = key[k];
                        list_index[i] = index(turn, k);
                    }
            }
            __syncthreads();
            // a wave has one of them at a time, its lanes those that may be in front
            const uint32_t other = lane < size ? list_key[lane] : 0;
            const int other_at = list_index[lane < size ? lane : 0];
            for (int i = wave; i < size; i += WAVES) {
                const uint32_t mine = __builtin_amdgcn_readlane(other, i);
                const int at = __builtin_amdgcn_readlane(other_at, i);
                const bool same = other == mine;
                const int higher = __builtin_popcountll(__ballot(other > mine));
                const int equal = __builtin_popcountll(__ballot(same));
                const int front = __builtin_popcountll(__ballot(same && other_at < at));
                if (lane == 0 && higher + front == wanted - 1) {   // the last one that is chosen
                    const bool whole = wanted - higher == equal;   // all that are equal to it are
                    found_key = whole ? mine - 1 : mine;
                    found_need = whole ? 0 : wanted - higher;
                }
            }
            __syncthreads();
            above = found_key;
            need = found_need;
        } else {
            uint32_t least = 0;
            int reach = n;   // how many keys are at least `least`
            // two bits a step: of the three values that they may add, the largest that m keys reach
            for (int bit = 31, step = 0; bit >= 0 && reach != m; bit -= 2, ++step) {
                const uint32_t unit = 1u << (bit - 1);
                int c[3] = {0, 0, 0};
                for (int turn = 0; turn < turns; ++turn) {
                    if (LOOP) load(turn);
#pragma unroll
                    for (int k = 0; k < EACH; ++k)
#pragma unroll
                        for (int i = 0; i < 3; ++i) c[i] += __builtin_popcountll(__ballot(key[k] >= least + (i + 1) * unit));
                }
                // three sets of counters in turn: one barrier a step
                if (lane < 3) atomicAdd(&counter[step % 3][lane], lane == 0 ? c[0] : lane == 1 ? c[1] : c[2]);
                if (tid < 3) counter[(step + 1) % 3][tid] = 0;
                __syncthreads();
                int add = 0;
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    const int all = counter[step % 3][i];
                    if (all >= m) {
                        add = i + 1;
                        reach = all;
                    }
                }
                least += add * unit;
            }
            // where m are at least that, all of these; otherwise the first of those equal to it
            above = reach == m ? least - 1 : least;
            if (reach != m) {
                int c = 0;
                for (int turn = 0; turn < turns; ++turn) {
                    if (LOOP) load(turn);
#pragma unroll
                    for (int k = 0; k < EACH; ++k) c += __builtin_popcountll(__ballot(key[k] > above));
                }
                __syncthreads();
                if (lane == 0) folded[0][wave] = c;
                __syncthreads();
                need = m;
#pragma unroll
                for (int w = 0; w < WAVES; ++w) need -= static_cast<int>(folded[0][w]);
            }
        }
        int up_before = 0, equal_before = 0;   // of the turns before
        for (int turn = 0; turn < turns; ++turn) {
            if (LOOP) load(turn);
            // for each set: how many the lanes before have, and the waves
            int up_at[SETS], equal_at[SETS];
#pragma unroll
            for (int k = 0; k < SETS; ++k) {
                int up = 0, equal = 0;
                up_at[k] = equal_at[k] = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint64_t u = __ballot(key[4 * k + j] > above);
                    up += __builtin_popcountll(u);
                    up_at[k] = __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(u >> 32), __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(u), up_at[k]));
                    if (need > 0) {
                        const uint64_t e = __ballot(key[4 * k + j] == above);
                        equal += __builtin_popcountll(e);
                        equal_at[k] = __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(e >> 32), __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(e), equal_at[k]));
                    }
                }
                if (lane == 0) {
                    sums[turn & 1][0][k][wave] = up;
                    sums[turn & 1][1][k][wave] = equal;
                }
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < SETS; ++k) {
                int at = up_before, same_at = equal_before;
#pragma unroll
                for (int w = 0; w < WAVES; ++w) {
                    const int u = sums[turn & 1][0][k][w], e = sums[turn & 1][1][k][w];
                    if (w < wave) {
                        at += u;
                        same_at += e;
                    }
                    up_before += u;
                    equal_before += e;
                }
                at += up_at[k];
                same_at += equal_at[k];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool up = key[4 * k + j] > above, same = need > 0 && key[4 * k + j] == above;
                    if (up || (same && same_at < need)) out[a.first + at + (same_at < need ? same_at : need)] = lo + index(turn, 4 * k + j);
                    at += up;
                    same_at += same;
                }
            }
        }
    }
}

// Workgroups that are wanted, four on each compute unit: where there are more ranges, a workgroup
// takes several, with the rows' sums formed once.  (31 sequences of up to 2047 blocks, both kernels, with
// 512, 1024, 2048 and any number of them 28.3, 25.9, 26.6 and 31.8 us; 32 of 1875, 20 heads of 64, 39.4, 39.6,
// 39.4 and, with the sums for each range, 45.6.)
constexpr int64_t kScoreGroups = 1024;

// The kernels loop where a launch cannot hold all units.
constexpr int64_t kMostUnits = 8 * 65535;

template <int D>
hipError_t launch_select(const SelectArgs &a, hipStream_t s) {
    ScorePlan p;
    const int64_t batch = a.kv.batch;
    int64_t ranges = (a.max_blocks + kScoreBlocks - 1) / kScoreBlocks, tiles = (static_cast<int64_t>(a.max_rows) + 15) / 16;
    const int64_t others = batch * tiles * a.kv.kv_heads;
    if (ranges * others > kScoreGroups) ranges = others < kScoreGroups ? kScoreGroups / others : 1;
    if (ranges * batch > kMostUnits) ranges = kMostUnits / batch;
    if (tiles * ranges * batch > kMostUnits) tiles = kMostUnits / (ranges * batch);
    p.tiles = static_cast<int>(tiles);
    p.ranges = static_cast<int>(ranges);
    p.units = static_cast<int>(tiles * ranges * batch);
    if (a.max_blocks > a.keep) {   // otherwise rows have all of their blocks, and no score is looked at
        hipLaunchKernelGGL((score_kernel<D>), dim3(8 * a.kv.kv_heads, (p.units + 7) / 8), dim3(64 * kScoreWaves), 0, s, a, p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const dim3 rows(a.kv.kv_heads, a.max_rows < 65535 ? a.max_rows : 65535, a.kv.batch);
    // the fewest waves whose registers hold the scores, 8 a thread while there are threads (both kernels: 61 rows of
    // 938 blocks 10.3 us, with 512 threads 12.0; 2 of 4096 13.3, with 256 threads 15.2, with 1024 of 16 scores 19.2)
    if (a.max_blocks <= 1024) hipLaunchKernelGGL((choose_kernel<256, 4, false>), rows, dim3(256), 0, s, a);
    else if (a.max_blocks <= 4096) hipLaunchKernelGGL((choose_kernel<512, 8, false>), rows, dim3(512), 0, s, a);
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
