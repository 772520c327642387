// Attention over the paged 8-bit cache (include/q4_decoder.h).
//
// The mathematics.  For a query row r and the tokens j it sees,
//     s_j = c * 2^eK * (q . k_j),   o = sum_j 2^s_j 2^eV v_j / sum_j 2^s_j
// with c = scale * log2(e), k_j and v_j the codes and eK, eV the exponents of
// token j's block.  The kernels work with t_j = s_j + eV, the exponent of
// token j's weight on its codes: with m at least about max_j t_j,
//     w_j = 2^(t_j - m + 7),   o = sum_j w_j v_j / sum_j w_j 2^-eV,
// so the codes go into the matrix products as they are.  m and the sums are
// fp32 and are carried over the tokens in one pass.  m is only raised when some
// t_j passes it by 8, so that most blocks need no rescaling (by 4: a prompt of
// 2048 49.9 us instead of 49.3, by 2: 51.8).  w is rounded to fp16 for the
// products with V alone (bf16, as fast, would keep 8 bits of it, fp32 products
// take many times as long): the largest is at least 2^7 and at most 2^15, so
// w is within 2^-11 of itself down to 2^-21 of the largest, within 2^-32 of
// the largest below, and lost below that.  Such weights matter where one token
// leads a great many others and has values close to 0; 2^7 keeps them to a
// 128th of what 1 would, and cancels between the two sums.
//
// Rows.  The rows of a sequence and the heads that share a kv head are one
// axis: row t, head g of the group is t * group + g, so a group of heads
// reads its kv head once.
//
// The products.  S^T = K Q^T on 16x16x32 bf16 MFMAs (e4m3 codes are exact in
// bf16), O^T += V^T W^T on 16x16x32 fp16 MFMAs (exact in fp16).  A lane's
// results of the first product -- 4 consecutive tokens of each half block for
// one row -- are its operand of the second in the cache's order of tokens, so
// the weights never leave their lane.

#include "q4_decoder_internal.h"

namespace q4 {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef float floatx2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 halfx2 __attribute__((ext_vector_type(2)));
typedef _Float16 halfx8 __attribute__((ext_vector_type(8)));

constexpr float kNan = __builtin_nanf("");
constexpr float kLowest = -3.402823466e38f;
constexpr float kSlack = 8.0f;   // how far a score may pass m before m is raised
constexpr float kUp = 7.0f;      // the weight of a score of m is 2^kUp; 2^(kSlack + kUp) is within fp16
// The rounding of an m below this moves a weight by 2^(2^-4) at most, which fp16 has room for.
constexpr float kHuge = 1048576.0f;

// Eight codes as bf16 / fp16 (exact).
__device__ __forceinline__ bf16x8 codes_bf16(uint32_t lo, uint32_t hi) {
    union {
        bf16x2 p[4];
        bf16x8 v;
    } u;
    u.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    u.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    u.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    u.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    return u.v;
}

__device__ __forceinline__ halfx8 codes_f16(uint32_t lo, uint32_t hi) {
    union {
        halfx2 p[4];
        halfx8 v;
    } u;
    u.p[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
    u.p[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
    u.p[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
    u.p[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
    return u.v;
}

__device__ __forceinline__ halfx8 weights_f16(const float (&w)[8]) {
    union {
        halfx2 p[4];
        halfx8 v;
    } u;
#pragma unroll
    for (int i = 0; i < 4; ++i) u.p[i] = __builtin_convertvector((floatx2){w[2 * i], w[2 * i + 1]}, halfx2);
    return u.v;
}

// Bytes of a word of 4 consecutive tokens, the first `first`, that lie in
// [lo, hi): 0xFF each.
__device__ __forceinline__ uint32_t bytes_in(int first, int lo, int hi) {
    const int skip = lo - first < 0 ? 0 : lo - first > 4 ? 4 : lo - first;
    const int count = hi - first < 0 ? 0 : hi - first > 4 ? 4 : hi - first;
    return static_cast<uint32_t>(((1ull << (8 * count)) - 1) & ~((1ull << (8 * skip)) - 1));
}

// 0x80 in each byte that is not a number.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// Largest over the four lanes that hold one row (lane % 16).
__device__ __forceinline__ float row_max(float v) {
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float row_sum(float v) {
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// What a block's exponents (eK in bits 0-7, eV in 8-15, the same for all
// lanes) make of the softmax scale, worked out on the bits of the powers of two.
struct BlockScales {
    float c, ev, inv_ev;   // |scale_log2| 2^eK, eV, 2^-eV
};

__device__ __forceinline__ BlockScales block_scales(const AttentionArgs &a, int e2) {
    BlockScales s;
    const int ek = static_cast<int8_t>(e2 & 0xFF), ev = static_cast<int8_t>(e2 >> 8);
    s.c = fabsf(a.scale_log2) * __uint_as_float(static_cast<uint32_t>(ek + 127) << 23);
    s.ev = static_cast<float>(ev);
    s.inv_ev = __uint_as_float(static_cast<uint32_t>(127 - ev) << 23);
    return s;
}

// One 16-row tile's running state in a wave: lane (r, g4) holds, for row r, the
// reference m, the largest score that leaves it (none where m is huge: see
// block_weights), its share of the sum l, and dimensions 16 i + 4 g4 + j of O.
template <int D>
struct Tile {
    float m, limit, l;
    floatx4 o[D / 16];

    __device__ __forceinline__ void clear() {
        m = limit = kLowest;
        l = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) o[i] = (floatx4){0, 0, 0, 0};
    }

    // The lane's largest score of a block.  st: q . k, -inf where the row does
    // not see the token; c > 0.
    __device__ __forceinline__ float top(const floatx4 (&st)[2], float c, float ev) const {
        float x = st[0][0];
#pragma unroll
        for (int i = 1; i < 8; ++i) x = fmaxf(x, st[i / 4][i % 4]);
        return fmaf(x, c, ev);
    }

    // m is raised to the rows' largest score, and the sums follow.  (A score
    // that is not a number raises nothing; its weight is not a number either.)
    __device__ __forceinline__ void raise(float top) {
        const float raised = fmaxf(m, row_max(top));
        const float f = __builtin_amdgcn_exp2f(m - raised);
        m = raised;
        limit = fabsf(m) > kHuge && m != kLowest ? -__builtin_inff() : m + kSlack;
        l *= f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) o[i] = o[i] * f;
    }

    __device__ __forceinline__ halfx8 weights(const floatx4 (&st)[2], float c, float shift, float inv_ev) {
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __builtin_amdgcn_exp2f(fmaf(st[i / 4][i % 4], c, shift));
        l = fmaf(((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7])), inv_ev, l);
        return weights_f16(w);
    }

    // A value that is not a number reaches the rows that see its token and no
    // others (0 * NaN is NaN): such tokens are counted for each output, and
    // the product gets 0 for them.  n0, n1: 1 in such bytes of operand d.
    __device__ __forceinline__ void mark_nans(int d, uint32_t n0, uint32_t n1, halfx8 seen) {
        floatx4 hits = {0, 0, 0, 0};
        // 0x38 is 1.0
        hits = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes_f16(n0 * 0x38u, n1 * 0x38u), seen, hits, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (hits[j] > 0.0f) o[d][j] = __builtin_nanf("");
    }
};

// The lane's tokens of a block are first + i and first + 16 + i; a row sees
// `seen` tokens from lo on.
__device__ __forceinline__ void hide_unseen(floatx4 (&st)[2], int first, int lo, uint32_t seen) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        st[i / 4][i % 4] = static_cast<uint32_t>(first - lo + (i / 4 * 16 + i % 4)) < seen ? st[i / 4][i % 4] : -__builtin_inff();
}

__device__ __forceinline__ halfx8 seen_tokens(int first, int lo, uint32_t seen) {   // 1 for each that the row sees
    float one[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) one[i] = static_cast<uint32_t>(first - lo + (i / 4 * 16 + i % 4)) < seen ? 1.0f : 0.0f;
    return weights_f16(one);
}

// A block's weights for all of a wave's tiles; m is raised where some score
// passes it by kSlack.  As a rule a weight's exponent is one fma of the score
// with eV - m + kUp, whose rounding is that of m.  Where m is raised, or so large
// that this would matter, the scores are rounded as m was before m is taken from
// them: the largest is m itself then.
template <int D, int NR>
__device__ __forceinline__ void block_weights(Tile<D> (&tile)[NR], floatx4 (&st)[NR][2], const BlockScales &e,
                                              halfx8 (&wf)[NR]) {
    float top[NR], shift[NR], c = e.c;
    bool over = false;
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        top[n] = tile[n].top(st[n], e.c, e.ev);
        over |= top[n] > tile[n].limit;
        shift[n] = e.ev - tile[n].m + kUp;
    }
    if (__any(over)) {
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            tile[n].raise(top[n]);
#pragma unroll
            for (int i = 0; i < 8; ++i) st[n][i / 4][i % 4] = fmaf(st[n][i / 4][i % 4], c, e.ev) - tile[n].m;
            shift[n] = kUp;
        }
        c = 1.0f;
    }
#pragma unroll
    for (int n = 0; n < NR; ++n) wf[n] = tile[n].weights(st[n], c, shift[n], e.inv_ev);
}

// Which row of q a lane has, and what it sees.
struct LaneRow {
    bool live;
    int t, pos, lo;    // row of the sequence, its position, the first token that it sees (or a place before them)
    uint32_t seen;     // how many from lo on
    int64_t at;        // its first element in q and out
};

// Rows times heads of a group are at most 2^20 * 64: 32 bits hold them.
__device__ __forceinline__ int row_of(const AttentionArgs &a, int i) {   // i / group
    return a.group == 1 ? i : static_cast<int>(__umulhi(static_cast<uint32_t>(i), a.group_inverse));
}

__device__ __forceinline__ LaneRow lane_row(const AttentionArgs &a, const KvSequence &s, int head, int rr, int all_rows, int D) {
    LaneRow x;
    x.live = rr < all_rows;
    const int last = x.live ? rr : all_rows - 1;
    x.t = row_of(a, last);
    x.pos = s.pos0 + x.t;
    x.lo = a.window ? x.pos - a.window + 1 : 0;
    x.seen = a.window ? a.window : x.pos < 0 ? 0 : x.pos + 1;
    x.at = (static_cast<int64_t>(s.row0 + x.t) * a.q_heads + head * a.group + last - x.t * a.group) * D;
    return x;
}

// The lane's operand slices of its row of q.
template <int D>
__device__ __forceinline__ void load_q(const AttentionArgs &a, int64_t at, int g4, bf16x8 (&q)[D / 32]) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
        q[i] = reinterpret_cast<const bf16x8 *>(a.q + at + 64 * (i / 2) + 16 * g4 + 8 * (i % 2))[0];
    if (a.scale_log2 < 0.0f) {   // its sign is taken in here (and only then is q waited for)
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            u32x4 w = __builtin_bit_cast(u32x4, q[i]);
            w.x ^= 0x80008000u;
            w.y ^= 0x80008000u;
            w.z ^= 0x80008000u;
            w.w ^= 0x80008000u;
            q[i] = __builtin_bit_cast(bf16x8, w);
        }
    }
}

// The blocks that a group of rows reads, and their division over the splits
// of the launch: split i has blocks [first + i * chunk, first + (i + 1) * chunk).
struct Span {
    int first, last, chunk, splits;   // blocks [first, last), splits that have some
};

// p_first, p_last: positions of the group's first and last row (p_last < 0:
// nothing is seen).  Tokens past the block table are not read: the rows that
// would see them give what is not a number (`past` below).
__device__ __forceinline__ Span span_of(const KvView &kv, int p_first, int p_last, int window, int chunk, int grid_splits) {
    Span s;
    int lo = window ? p_first - window + 1 : 0;
    if (lo < 0) lo = 0;
    s.first = lo / kKvBlock;
    s.last = p_last < 0 ? 0 : p_last / kKvBlock + 1;
    if (s.last > kv.table_width) s.last = kv.table_width;
    if (s.last <= s.first) {
        s.last = s.first;
        s.chunk = 1;
        s.splits = 0;
        return s;
    }
    const int n = s.last - s.first;
    if (grid_splits == 1) {
        s.chunk = n;
        s.splits = 1;
        return s;
    }
    s.chunk = chunk;
    if (static_cast<int64_t>(chunk) * grid_splits < n) s.chunk = (n + grid_splits - 1) / grid_splits;
    s.splits = (n + s.chunk - 1) / s.chunk;
    return s;
}

__device__ __forceinline__ bool past(const KvView &kv, int pos) { return pos >= 0 && pos / kKvBlock >= kv.table_width; }

// How a launch is shaped: groups of `group_rows` rows of a sequence and kv
// head, and the split of their blocks.
struct Plan {
    int group_rows;      // 16 or 32
    int waves;           // of a workgroup
    int groups;          // of the sequence with most rows
    int rows_held;       // rows of a group that the workspace has room for
    int chunk, splits;
};

// Whether a group's blocks are split: groups and rows past those that the
// launch was shaped for have no place in the workspace.
__device__ __forceinline__ bool is_split(const Plan &p, int group, int rows) {
    return p.splits > 1 && group < p.groups && rows <= p.rows_held;
}

// Where a split's partial results of a row are in the workspace: first
// {m, l} [row][split], then O [row][split][D], rows counted over batch, kv
// head, group and row of the group.  A split without blocks has {kLowest,
// kNoBlocks} and no O.  (The O of one that has blocks counts also where its l
// or its factor is 0: what is not a number stays it.)
constexpr float kNoBlocks = -1.0f;   // no sum of weights

struct Partials {
    floatx2 *ml;
    float *o;
};

__device__ __forceinline__ int64_t partial_row(const KvView &kv, const Plan &p, int b, int head, int group) {
    return ((static_cast<int64_t>(b) * kv.kv_heads + head) * p.groups + group) * p.rows_held;
}

__device__ __forceinline__ Partials partials(const AttentionArgs &a, const Plan &p) {
    Partials w;
    w.ml = reinterpret_cast<floatx2 *>(a.workspace);
    const int64_t rows = static_cast<int64_t>(a.kv.batch) * a.kv.kv_heads * p.groups * p.rows_held;
    w.o = a.workspace + (rows * p.splits * 2 + 3) / 4 * 4;   // 16-byte aligned
    return w;
}

// A split without blocks says so.
__device__ __forceinline__ void write_empty(const AttentionArgs &a, const Plan &p, int b, int head, int group, int rows, int split) {
    const Partials ws = partials(a, p);
    const int64_t row = partial_row(a.kv, p, b, head, group);
    for (int i = threadIdx.x; i < rows; i += blockDim.x) ws.ml[(row + i) * p.splits + split] = (floatx2){kLowest, kNoBlocks};
}

// What a row's sums are multiplied by: a row without a position sees nothing
// and gives 0.  Every other one sees its own token, so a total of 0 means
// scores of -inf alone, whose softmax is not a number (0 times infinity).
__device__ __forceinline__ float inverse(const KvView &kv, int pos, float total) {
    return pos < 0 ? 0.0f : past(kv, pos) ? kNan : 1.0f / total;
}

// A workgroup has NR tiles of 16 rows (of rows x heads of the group) of one
// sequence and kv head, and one chunk of its blocks; its W waves take the
// blocks in turn with all the rows, so a block's codes go from memory to the
// registers of one wave, as its operand slices, and nowhere else, and no wave
// waits for another before the end.  Groups with the most tokens start first.
//
// What bounds it for single tokens is reading the cache: two sequences of
// 131072 tokens of 8 heads of 128 (537 MB) take 85 us, 6.3 TB/s; 32 sequences
// of 2048 to 8191 (332 MB) 59 us, 5.7 TB/s.  The loads are nontemporal, as
// nothing is read twice (99 -> 91 us for the former, 80 -> 74 for the latter
// when measured).  Short caches are bound by what follows from each other:
// length and block ids together, codes, a block's products, the join of the
// waves: one token over 64 takes 4.3 us, over 512 5.9 and over 1505, in 12
// splits, 7.5, of which the join of the splits is 2.5.
//
// For many rows it is the issue of instructions: a wave's 32 rows and a block of
// heads of 128 are 32 MFMAs of 16 cycles and about 170 other instructions of 2
// to 8 (64 conversions of codes, 16 exponentials), and little of the two runs at
// once: 1080 cycles.  A prompt of 2048 with 32 heads of 128 takes 49 us, 700
// TFLOP/s, one of 8192 585 us, 940.  Two tiles share what a wave converts (one
// tile: 75 us for the former), and fill the registers.  Workgroups of two waves
// start and join less often for what they compute.  Blocks that pass through
// LDS to eight waves with 64 or 128 rows, converted there or not, took 57 to 65
// us: their waves wait for each other.
constexpr int kWaves = 4;   // but for many rows, see plan_of

template <int D, int NR, int W>
__global__ __launch_bounds__(64 * W, 2) void attention_kernel(AttentionArgs a, Plan plan) {
    constexpr int kRows = 16 * NR;
    constexpr int KQ = D / 32;   // k slices of the first product
    constexpr int DT = D / 16;   // 16-dimension tiles of the output
    // Codes of the next block: in registers of their own while this one is
    // worked on, or, with two tiles, in this one's as soon as a product has read
    // them (with 20 spilled values otherwise; one tile, which reads more than it
    // computes, takes 61.6 instead of 59.5 us so for 32 sequences up to 8191)
    constexpr int BUFS = NR == 1 ? 2 : 1;
    __shared__ float part_m[W][16], part_l[W][16];
    __shared__ floatx4 part_o[W][DT][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g4 = lane >> 4;
    const int b = blockIdx.z, head = blockIdx.x;
    const int split = plan.splits == 1 ? 0 : blockIdx.y % plan.splits;
    // the ids of the blocks that the wave has where there is no window, read
    // before the length is known
    const int guessed = split * plan.chunk + wave;
    const int guess = kv_block_id(a.kv, b, guessed + lane * W);
    const KvSequence s = kv_sequence(a.kv, b);
    const int grid_groups = plan.splits == 1 ? gridDim.y : gridDim.y / plan.splits;
    const int all_rows = s.rows * a.group;
    const int groups = (all_rows + kRows - 1) / kRows;
    for (int back = plan.splits == 1 ? blockIdx.y : blockIdx.y / plan.splits; back < groups; back += grid_groups) {
        const int group = groups - 1 - back;
        const int rr0 = group * kRows, rr1 = rr0 + kRows < all_rows ? rr0 + kRows : all_rows;
        const int p_first = s.pos0 + row_of(a, rr0), p_last = s.pos0 + row_of(a, rr1 - 1);
        const bool whole = !is_split(plan, group, rr1 - rr0);
        const Span sp = span_of(a.kv, p_first, p_last, a.window, plan.chunk, whole ? 1 : plan.splits);
        if (whole ? split > 0 : split >= sp.splits) {   // uniform
            if (!whole) write_empty(a, plan, b, head, group, rr1 - rr0, split);
            continue;
        }
        const int blk0 = sp.first + split * sp.chunk;
        const int blk1 = blk0 + sp.chunk < sp.last ? blk0 + sp.chunk : sp.last;
        // the first tokens that all rows and that any row of the group see
        const int all_lo = a.window ? p_last - a.window + 1 : 0, any_lo = a.window ? p_first - a.window + 1 : 0;

        LaneRow row[NR];
        bf16x8 q[NR][KQ];
        Tile<D> tile[NR];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            row[n] = lane_row(a, s, head, rr0 + 16 * n + r, all_rows, D);
            load_q<D>(a, row[n].at, g4, q[n]);
            tile[n].clear();
        }
        // a block's ids and exponents are read 64 blocks at a time, one a lane
        for (int first = blk0 + wave; first < blk1; first += 64 * W) {
            const int count = (blk1 - first + W - 1) / W, blocks = count < 64 ? count : 64;
            int my_id = guess;
            if (first != guessed) my_id = kv_block_id(a.kv, b, first + lane * W);
            const int my_exps =
                reinterpret_cast<const uint16_t *>(a.kv.exps)[static_cast<int64_t>(my_id < 0 ? 0 : my_id) * a.kv.kv_heads + head];
            u32x4 codes[BUFS][2 * KQ];
            // (past the end the last block is read again)
            auto fetch = [&](int i, int from, int end, u32x4(&to)[2 * KQ]) {   // K's slices are [0, KQ), V's follow
                const int id = __builtin_amdgcn_readlane(my_id, i < blocks ? i : blocks - 1);
                const int64_t plane = (static_cast<int64_t>(id < 0 ? 0 : id) * a.kv.kv_heads + head) * 2;
                // a base that is the same for all lanes and a lane's offset,
                // which is hidden so that the compiler keeps them apart: the
                // loads then need no address registers of their own
                const uint8_t *src = a.kv.data + plane * (kKvBlock * D);
                uint32_t at = lane * 16;
                asm volatile("" : "+v"(at));
#pragma unroll
                for (int j = from; j < end; ++j) {
                    const u32x4 *p = reinterpret_cast<const u32x4 *>(src + 1024 * j + at);
                    // many rows read a block again (2048 over 8192 tokens: 257 against 268 us)
                    to[j] = NR == 1 ? __builtin_nontemporal_load(p) : *p;
                }
            };
            fetch(0, 0, 2 * KQ, codes[0]);
            asm volatile("" ::"v"(my_exps));   // has arrived before the loop, whose waits are for codes alone
            for (int i0 = 0; i0 < blocks; i0 += BUFS) {
#pragma unroll
                for (int u = 0; u < BUFS; ++u) {
                    const int i = i0 + u;
                    if (i >= blocks) break;
                    if constexpr (BUFS == 2) fetch(i + 1, 0, 2 * KQ, codes[u ^ 1]);
                    u32x4(&kc)[2 * KQ] = codes[u];
                    const BlockScales scales = block_scales(a, __builtin_amdgcn_readlane(my_exps, i));
                    const bool known = __builtin_amdgcn_readlane(my_id, i) >= 0;
                    floatx4 st[NR][2];
#pragma unroll
                    for (int tt = 0; tt < 2; ++tt) {
#pragma unroll
                        for (int n = 0; n < NR; ++n) st[n][tt] = (floatx4){0, 0, 0, 0};
#pragma unroll
                        for (int k = 0; k < KQ; ++k) {
                            const u32x4 w = kc[tt * (KQ / 2) + k / 2];
                            const bf16x8 kf = k % 2 ? codes_bf16(w.z, w.w) : codes_bf16(w.x, w.y);
#pragma unroll
                            for (int n = 0; n < NR; ++n)
                                st[n][tt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, q[n][k], st[n][tt], 0, 0, 0);
                        }
                        if (!known)
#pragma unroll
                            for (int n = 0; n < NR; ++n) st[n][tt] = (floatx4){kNan, kNan, kNan, kNan};
                    }
                    if constexpr (BUFS == 1) fetch(i + 1, 0, KQ, kc);
                    const int start = (first + i * W) * kKvBlock;
                    if (start < all_lo || start + kKvBlock - 1 > p_first) {   // some row does not see some token
                        const int tok = start + 4 * g4;
#pragma unroll
                        for (int n = 0; n < NR; ++n) hide_unseen(st[n], tok, row[n].lo, row[n].seen);
                        // bytes that no row of the group sees may hold anything
                        const uint32_t in0 = bytes_in(tok, any_lo, p_last + 1), in1 = bytes_in(tok + 16, any_lo, p_last + 1);
                        // and what is not a number must not meet a weight of 0:
                        // such bytes are noted, a bit each, and cleared
                        uint32_t bad[2] = {0, 0};
#pragma unroll
                        for (int j = 0; j < 4 * KQ; ++j) {
                            const uint32_t v = kc[KQ + j / 4][j % 4] & (j % 2 ? in1 : in0), n = nan_bytes(v) >> 7;
                            bad[j / 8] |= n << (j % 8);
                            kc[KQ + j / 4][j % 4] = v & ~(n * 0xFFu);
                        }
                        if (__any((bad[0] | bad[1]) != 0)) {
#pragma unroll
                            for (int n = 0; n < NR; ++n) {
                                const halfx8 seen = seen_tokens(tok, row[n].lo, row[n].seen);
#pragma unroll
                                for (int d = 0; d < DT; ++d) {
                                    const uint32_t n0 = bad[d / 4] >> (d % 4 * 2), n1 = n0 >> 1;
                                    tile[n].mark_nans(d, n0 & 0x01010101u, n1 & 0x01010101u, seen);
                                }
                            }
                        }
                    }
                    halfx8 wf[NR];
                    block_weights<D, NR>(tile, st, scales, wf);
#pragma unroll
                    for (int d = 0; d < DT; ++d) {
                        const u32x4 v = kc[KQ + d / 2];
                        const halfx8 vf = d % 2 ? codes_f16(v.z, v.w) : codes_f16(v.x, v.y);
#pragma unroll
                        for (int n = 0; n < NR; ++n)
                            tile[n].o[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, wf[n], tile[n].o[d], 0, 0, 0);
                    }
                    if constexpr (BUFS == 1) fetch(i + 1, KQ, 2 * KQ, kc);
                }
            }
        }
        // join the waves.  (The lane is hidden from the loop over the
        // groups, out of which the compiler would take the addresses below and
        // hold them all.)
        int re = r, ge = g4;
        asm volatile("" : "+v"(re), "+v"(ge));
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const float sum = row_sum(tile[n].l);
            __syncthreads();   // the tile before has been read
            if (ge == 0) {
                part_m[wave][re] = tile[n].m;
                part_l[wave][re] = sum;
            }
#pragma unroll
            for (int i = 0; i < DT; ++i) part_o[wave][i][16 * ge + re] = tile[n].o[i];
            __syncthreads();
            float top = part_m[0][re];
#pragma unroll
            for (int w = 1; w < W; ++w) top = fmaxf(top, part_m[w][re]);
            float f[W], total = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                f[w] = __builtin_amdgcn_exp2f(part_m[w][re] - top);
                total += f[w] * part_l[w][re];
            }
            if (!row[n].live) continue;
            // every wave sums some of the 16-dimension tiles
            const Partials ws = partials(a, plan);
            const int64_t at = (partial_row(a.kv, plan, b, head, group) + 16 * n + re) * plan.splits + split;
            const float inv = inverse(a.kv, row[n].pos, total);
#pragma unroll
            for (int i = 0; i < DT / W; ++i) {
                const int tile_i = wave * (DT / W) + i, d = 16 * tile_i + 4 * ge;
                floatx4 acc = part_o[0][tile_i][16 * ge + re] * f[0];
#pragma unroll
                for (int w = 1; w < W; ++w) acc = acc + part_o[w][tile_i][16 * ge + re] * f[w];
                if (!whole) *reinterpret_cast<floatx4 *>(ws.o + at * D + d) = acc;
                else if (a.out_bf16)
                    *reinterpret_cast<bf16x4 *>(static_cast<__bf16 *>(a.out) + row[n].at + d) = __builtin_convertvector(acc * inv, bf16x4);
                else *reinterpret_cast<floatx4 *>(static_cast<float *>(a.out) + row[n].at + d) = acc * inv;
            }
            if (!whole && wave == 0 && ge == 0) ws.ml[at] = (floatx2){top, total};
        }
    }
}

// Joins the splits of a row, a workgroup a row: D / 4 threads have four
// dimensions each, and 1024 / D of such sets sum splits side by side.  Every
// wave has all splits' m and l, 64 at a time, one a lane.  What is read does
// not depend on the sequence's length, so that all loads, for up to kAhead
// splits a thread, are on their way together.
template <int D>
__global__ __launch_bounds__(256) void attention_join_kernel(AttentionArgs a, Plan plan) {
    constexpr int LANES = D / 4, PARTS = 256 / LANES, kAhead = 4;
    __shared__ floatx4 part[PARTS][LANES];
    const int b = blockIdx.z, head = blockIdx.y % a.kv.kv_heads, group = blockIdx.y / a.kv.kv_heads;
    const int tid = threadIdx.x, lane = tid & 63, x = tid % LANES, y = tid / LANES;
    const int in_group = blockIdx.x;
    const Partials ws = partials(a, plan);
    const int64_t at0 = (partial_row(a.kv, plan, b, head, group) + in_group) * plan.splits;
    const floatx2 none = {kLowest, kNoBlocks};
    floatx2 ml = lane < plan.splits ? ws.ml[at0 + lane] : none;
    const floatx4 *src = reinterpret_cast<const floatx4 *>(ws.o + at0 * D) + x;
    floatx4 ahead[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
        if (y + PARTS * k < plan.splits) ahead[k] = src[(y + PARTS * k) * LANES];
    const KvSequence s = kv_sequence(a.kv, b);
    const int all_rows = s.rows * a.group, rr0 = group * plan.group_rows;
    const int rows = rr0 + plan.group_rows < all_rows ? plan.group_rows : all_rows - rr0;
    if (in_group >= rows || !is_split(plan, group, rows)) return;
    floatx4 acc = {0, 0, 0, 0};
    float top = ml.x, total = 0.0f;
    for (int i = 64 + lane; i < plan.splits; i += 64) top = fmaxf(top, ws.ml[at0 + i].x);
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) top = fmaxf(top, __shfl_xor(top, m));
    for (int i0 = 0; i0 < plan.splits; i0 += 64) {
        const int n = plan.splits - i0 < 64 ? plan.splits - i0 : 64;
        if (i0 > 0) ml = lane < n ? ws.ml[at0 + i0 + lane] : none;
        // (a split without blocks has no O: what was read for it is not used)
        const float f = ml.y == kNoBlocks ? kNoBlocks : __builtin_amdgcn_exp2f(ml.x - top);
        if (f != kNoBlocks) total += f * ml.y;
#pragma unroll
        for (int k = 0; k < 64 / PARTS; ++k) {
            const int i = y + PARTS * k;
            if (PARTS * k >= n) break;   // the same for the workgroup
            const float fi = __shfl(f, i);
            if (i < n && fi != kNoBlocks) acc = acc + (k < kAhead && i0 == 0 ? ahead[k % kAhead] : src[static_cast<int64_t>(i0 + i) * LANES]) * fi;
        }
    }
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) total += __shfl_xor(total, m);
    part[y][x] = acc;
    __syncthreads();
    if (y != 0) return;
#pragma unroll
    for (int i = 1; i < PARTS; ++i) acc = acc + part[i][x];
    const LaneRow row = lane_row(a, s, head, rr0 + in_group, all_rows, D);
    acc = acc * inverse(a.kv, row.pos, total);
    if (a.out_bf16)
        reinterpret_cast<bf16x4 *>(static_cast<__bf16 *>(a.out) + row.at)[x] = __builtin_convertvector(acc, bf16x4);
    else
        reinterpret_cast<floatx4 *>(static_cast<float *>(a.out) + row.at)[x] = acc;
}

// ------------------------------------------------------------------ launch
// Two tiles a wave where there are more tiles than fit on
// the chip at once with one (two workgroups a compute unit for heads of 128,
// four for heads of 64; us with one / two):
//   D = 128: 512 tiles, 5 blocks 6.6 / 7.3, 28 blocks 11.3 each; 1024 tiles, 3
//     blocks 10.6 / 8.9, 9 blocks 12.6 / 10.4; 2048 tiles, 17 blocks 29 / 23
//   D = 64: 640 tiles, 9 blocks 6.0 / 7.3; 1280 tiles, 5 blocks 8.7 / 8.9, 15
//     blocks 15.1 / 12.9, 17 blocks 11.2 / 11.9, 30 blocks 20.7 / 16.8, 78 blocks
//     34 / 29; 1536 tiles, 5 blocks 9.2 / 8.4
// or, of at least kManyTiles, where these have many blocks:
//   D = 128: 128 tiles, 256 blocks 26 / 23, 512 blocks 42 / 32; 256 tiles, 126
//     blocks 19 / 25, 254 blocks 35.5 / 35.4, 510 blocks 74 / 56; 512 tiles, 60
//     blocks 16.6 / 16.4, 250 blocks 56 / 47
//   D = 64: 640 tiles, 375 blocks on average 81 / 70; 960 tiles, 245 blocks 82 / 55
// For D = 64 with fewer, how the workgroups divide over the compute units decides:
// 500 tiles, 88 blocks 16.8 / 22.8, 151 blocks 27 / 34; 600, 151 blocks 31 / 33; 768,
// 62 blocks 17.7 / 19.2; but 160, 249 blocks 31 / 22; 320, 253 blocks 41 / 37; 640, 63
// blocks (16 sequences) 30 / 19.5; 960, 82 blocks 27 / 23.  They keep one tile.
constexpr int64_t tiles_at_once(int D) { return D == 64 ? 1024 : 512; }
constexpr int64_t many_blocks(int D) { return D == 64 ? 200000 : 40000; }
constexpr int64_t kManyTiles = 64;

// Two waves a workgroup instead of four where there are more workgroups than fit
// on the chip at once with four, and many for the blocks that each reads, so that
// they still even out (workgroups, blocks: us with four / two):
//   D = 128: 512, 9: 10.4 / 11.8; 520, 9: 14.4 / 13.0; 600, 10: 16.8 / 14.2; 640,
//     2: 13.0 / 8.2; 640, 31: 22.8 / 25.1; 744, 12: 18.8 / 16.8; 768, 82: 44 / 53;
//     1024, 17: 22.9 / 22.6; 1024, 30: 29.9 / 26.4; 1400, 22: 34.5 / 31.1; 1313, 95:
//     77 / 90; 2048, 9: 35 / 27; 2048, 33: 55 / 49; 2048, 121: 142 / 160; 4096, 65:
//     162 / 152; 8192, 129: 581 / 556
//   D = 64: 640, 3: 8.1 / 7.4; 768, 3: 7.7 / 7.0; 800, 5: 11.0 / 9.7; 880, 22: 16.3 /
//     19.9; 1280, 33: 24 / 29; 1920, 16: 25.3 / 23.9; 2048, 33: 36 / 40; 2560, 65: 68 /
//     70; 2560, 9: 25 / 22; 6144, 17: 65 / 57
// and sooner where a window makes them equal:
//   D = 128: 520, 24: 22.2 / 20.5; 520, 94: 47.9 / 55.3; 744, 24: 23.7 / 21.9; 744,
//     94: 50 / 57; 1000, 24: 29.0 / 23.5; 1024, 65: 48 / 45; 1024, 129: 82 / 81;
//     1104, 24: 35 / 33; 1400, 94: 90 / 107; 1512, 24: 41.0 / 42.5; 2048, 33: 59 / 57;
//     2504, 24: 63 / 56; 3000, 33: 84 / 75
//   D = 64: 760, 24: 15.2 / 17.5; 820, 24: 19.5 / 17.7; 820, 79: 38.3 / 38.1; 960, 24:
//     19.8 / 18.1; 960, 63: 33.0 / 32.6; 1260, 24: 23.1 / 23.2; 1260, 79: 45 / 52;
//     1880, 79: 67 / 78; 2380, 24: 40 / 35; 2380, 79: 82.2 / 80.5
bool two_waves(int64_t groups, int64_t each, bool equal, int D) {
    if (groups <= (D == 64 ? 767 : 512)) return false;
    if (equal) return each * 25 < groups * (D == 64 ? 1 : 2);
    return each * (D == 64 ? 100 : 25) < groups;
}

// Blocks of a workgroup of attention_kernel at most, where the workspace has room,
// for a sequence much longer than the others of its batch: 8192 tokens, which a
// workgroup reads in 30 to 85 us, as the others leave it room.
constexpr int64_t kMaxChunk = 256;

// A wave takes 0.43 us a block where it does not wait for memory (the products,
// conversions and exponentials of a block follow from each other), and a split's
// join 2.5 us and 1 more a thousand rows: blocks are split where that leaves a
// workgroup kSaved fewer of them, and one more for every 128 rows.  (One row:
// 700 tokens 7.1 us either way, 1200 7.4 against 8.8, 1505 7.7 against 10; 128
// rows of 20 heads over 1000 tokens 12.0 against 6.7.)  The smallest chunk has one
// block for each wave (3000 tokens 7.5 us; 8.8 with four blocks for each).
constexpr int64_t kSaved = 22;
constexpr int64_t kMinChunk = kWaves;

// Rows of partial results that a launch may write, which is what splits cost
// beside the join: at most 34 MB of workspace for heads of 128.  (32 heads on 8,
// D = 128, us and MB with 32768 / 65536 / 131072 rows / no limit:
//   512 rows over 131072 tokens 1280, 17 / 1204, 34 / 1225, 68 / 1355, 136
//   2048 rows over them 4640, 0 / 4520, 0 / 4640, 68 / 5340, 545
//   2048 rows of a prompt in a table for 131072 tokens 62, 0 / 61, 0 / 179, 68 / 364, 545
//   one sequence of 131072 among 255 of 500 211, 17 / 185, 34 / 230, 68 / 231, 68
//   one among 511 of 300 361, 17 / 244, 34 / 298, 68; unsplit 613
//   one among 99 of 500, 5 rows each 414, 17 / 235, 33 / 153, 67 / 154, 213
//   700 rows over 32768 449, 0 / 454, 23 / 419, 47 / 426, 47
//   600 sequences of 5000 to 20000 2260, 0 / 2360, 30 / 2360, 30; unsplit 2260)
constexpr int64_t kMaxPartialRows = 65536;

// Into how many parts attention_kernel's `work` groups of `held` rows have their
// blocks split: no more than a workgroup for every compute unit (32 sequences up
// to 8191 tokens 60 us in 256, 62 in 512; 20 sequences of 4000 28 us in 160, 36
// in 320), or else no chunk over kMaxChunk as far as kMaxPartialRows allows it.
int64_t splits_wanted(int64_t work, int64_t held, int64_t blocks) {
    if (blocks <= kSaved) return 1;
    const int64_t fill = work < 256 ? 256 / work : 1, least = (blocks + kMaxChunk - 1) / kMaxChunk;
    const int64_t room = kMaxPartialRows / (work * held), parts = least < room ? least : room;
    return parts < fill ? fill : parts;
}

Plan plan_of(const AttentionArgs &a, int D) {
    const int64_t rows = static_cast<int64_t>(a.max_rows) * a.group, sets = static_cast<int64_t>(a.kv.kv_heads) * a.kv.batch;
    // blocks that a row reads
    int64_t seen = a.max_length - (a.max_rows < a.max_length ? a.max_rows : a.max_length) / 2;
    if (a.window && a.window < seen) seen = a.window;
    const int64_t each = seen / kKvBlock + 1;
    Plan p;
    const int64_t tiles = (rows + 15) / 16 * sets;
    const bool two = tiles > tiles_at_once(D) || (tiles >= kManyTiles && tiles * each >= many_blocks(D));
    p.group_rows = rows > 16 && two ? 32 : 16;
    p.rows_held = rows < p.group_rows ? static_cast<int>(rows) : p.group_rows;
    p.groups = static_cast<int>((rows + p.group_rows - 1) / p.group_rows);
    p.waves = p.group_rows == 32 && two_waves(p.groups * sets, each, a.window && seen == a.window, D) ? 2 : kWaves;
    int64_t blocks = (static_cast<int64_t>(a.max_length) + kKvBlock - 1) / kKvBlock;
    if (a.window) {   // no group reads more than its rows and their window
        const int64_t reach = (static_cast<int64_t>(a.window) + p.group_rows / a.group + kKvBlock) / kKvBlock + 1;
        if (reach < blocks) blocks = reach;
    }
    const int64_t splits = splits_wanted(p.groups * sets, p.rows_held, blocks);
    int64_t chunk = (blocks + splits - 1) / splits;
    if (chunk < kMinChunk) chunk = kMinChunk;
    if (blocks - chunk < kSaved + p.rows_held * p.groups * sets / 128) chunk = blocks < 1 ? 1 : blocks;
    p.chunk = static_cast<int>(chunk);
    p.splits = static_cast<int>((blocks + chunk - 1) / chunk);
    return p;
}

template <int D>
hipError_t launch(const AttentionArgs &a, hipStream_t s) {
    const Plan p = plan_of(a, D);
    int grid_groups = p.groups;   // the kernels loop where a launch cannot hold them all
    if (static_cast<int64_t>(grid_groups) * p.splits > 65535) grid_groups = 65535 / p.splits;
    const dim3 grid(a.kv.kv_heads, grid_groups * p.splits, a.kv.batch);
    if (p.group_rows == 16)
        hipLaunchKernelGGL((attention_kernel<D, 1, kWaves>), grid, dim3(64 * kWaves), 0, s, a, p);
    else if (p.waves == kWaves)
        hipLaunchKernelGGL((attention_kernel<D, 2, kWaves>), grid, dim3(64 * kWaves), 0, s, a, p);
    else
        hipLaunchKernelGGL((attention_kernel<D, 2, 2>), grid, dim3(64 * 2), 0, s, a, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    hipLaunchKernelGGL((attention_join_kernel<D>), dim3(p.rows_held, p.groups * a.kv.kv_heads, a.kv.batch), dim3(256), 0, s, a, p);
    return hipGetLastError();
}

}  // namespace

// How many tiles a group has and in how many parts its blocks are depends on the
// window, which may be any: the most that some window takes.  Fewer blocks may
// be split into more parts, but never into more than there are for all of them
// with the smallest chunk, nor than splits_wanted gives for all of them.
size_t attention_workspace(const AttentionArgs &a, int head_dim) {
    const int64_t rows = static_cast<int64_t>(a.max_rows) * a.group, sets = static_cast<int64_t>(a.kv.kv_heads) * a.kv.batch;
    const int64_t blocks = (static_cast<int64_t>(a.max_length) + kKvBlock - 1) / kKvBlock;
    size_t most = 0;
    for (int64_t tile = 16; tile <= 32; tile += 16) {
        const int64_t held = rows < tile ? rows : tile, groups = (rows + tile - 1) / tile;
        int64_t splits = splits_wanted(groups * sets, held, blocks);
        if (splits > (blocks + kMinChunk - 1) / kMinChunk) splits = (blocks + kMinChunk - 1) / kMinChunk;
        if (splits <= 1) continue;
        const size_t parts = static_cast<size_t>(groups) * held * sets * splits;   // as in partials()
        const size_t bytes = ((parts * 2 + 3) / 4 * 4 + parts * head_dim) * sizeof(float);
        if (bytes > most) most = bytes;
    }
    return most;
}

void attention_plan(const AttentionArgs &a, int head_dim, int32_t *rows, int32_t *waves, int32_t *parts) {
    const Plan p = plan_of(a, head_dim);
    *rows = p.group_rows;
    *waves = p.waves;
    *parts = p.splits;
}

hipError_t launch_kv_attention(const AttentionArgs &a, int head_dim, hipStream_t s) {
    return head_dim == 128 ? launch<128>(a, s) : launch<64>(a, s);
}

}  // namespace q4
