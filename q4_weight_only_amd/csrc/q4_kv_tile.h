// What the attention kernels over the paged 8-bit cache share: codes as operands
// of the matrix products, and the running state of a tile of 16 rows.  The
// mathematics is beside the kernels (q4_kv_attention.hip).
#pragma once

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

}  // namespace
}  // namespace q4
