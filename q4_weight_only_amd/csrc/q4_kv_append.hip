// Rotation of q and k, quantization of k and v to 8 bits, and the append to
// the paged cache (include/q4_decoder.h).
//
// A workgroup of 2 * D threads has one of two tasks.  The first: one block of
// one sequence, one kv head, K or V.  Each thread holds 16 values of the
// block's 32 tokens; the largest finite value of the new tokens gives the
// block's exponent, the codes of tokens that were there before are rescaled
// where the exponent rises, and the codes pass through LDS, where they take the
// block's order, as words of four.  The second: pieces of the rotated q, of two
// heads a thread.
//
// What bounds it is memory: 4515 rows of 32 + 2 * 8 heads of 128 in fp32
// (157 MB) take 32 us, 4.9 TB/s; 8192 rows of 20 + 2 * 20 heads of 64 37 us,
// 4.5 TB/s.  Lanes run along a row's dimensions four at a time, so that a
// wave's loads are whole lines (16 dimensions a lane: 52 and 66 us), and both
// halves of the turned pairs are in one thread, which reads each of them once.
// One token for each of 32 sequences takes 4.8 us: bounds and block ids, rows
// and old codes, the largest value, the codes, one after the other.
//
// The rotated q is stored with the nontemporal hint for few rows of a sequence,
// and without it for a prompt's, which the attention after it reads many times
// (append and attention, us with / without: one token for each of 64 sequences of
// 1000 33.0 / 33.6, for each of 32 of 411 13.6 / 13.7; 512 rows over 2048 36.5 /
// 35.9; 3 prompts of 1505 117.0 / 114.7, with neighbours as pairs 118.5 / 115.5; 8 of
// 256 37.8 / 36.9; append alone 30.7 / 32.4 for these 3, 14.0 / 14.1 for the 8, 15.0 /
// 14.0 for one prompt of 2048 with neighbours as pairs).  Stores through to the
// device's scope write such pairs twice (18.2 for the last).
//
// The rotation's products are rounded before they are added, so that a value
// on the edge between two exponents does not depend on how the compiler pairs
// them.

#include <hip/hip_bf16.h>

#include "q4_decoder_internal.h"

namespace q4 {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef float floatx2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ floatx4 load4(const float *p) { return *reinterpret_cast<const floatx4 *>(p); }
__device__ __forceinline__ floatx4 load4(const uint16_t *p) {
    const u32x2 v = *reinterpret_cast<const u32x2 *>(p);
    return (floatx4){__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                     __uint_as_float(v.y & 0xFFFF0000u)};
}

// Piece c of a head's dimensions, c in [0, D / 8): four pairs that are turned
// together, as four dimensions from lo and four from hi (the halves of the
// pairs, or pairs side by side), or eight that are not turned.
struct Piece {
    bool turned, split;
    int lo, hi;
};

__device__ __forceinline__ Piece piece_of(const AppendArgs &a, int c) {
    Piece p;
    p.turned = 8 * c < a.rot;
    p.split = p.turned && !a.interleaved;
    p.lo = p.split ? 4 * c : 8 * c;
    p.hi = p.split ? p.lo + a.rot / 2 : p.lo + 4;
    return p;
}

// Cosines and sines of the piece's pairs: not numbers past the table.
struct Angles {
    floatx4 cs[2];
};

__device__ __forceinline__ Angles angles(const AppendArgs &a, const Piece &p, int c, int pos) {
    Angles x;
    if (p.turned && pos >= 0 && pos < a.positions) {
        const floatx4 *row = reinterpret_cast<const floatx4 *>(a.rope + (static_cast<int64_t>(pos) * (a.rot / 2) + 4 * c) * 2);
        x.cs[0] = row[0];
        x.cs[1] = row[1];
    } else {
        const float nan = __builtin_nanf("");
        x.cs[0] = x.cs[1] = (floatx4){nan, nan, nan, nan};
    }
    return x;
}

__device__ __forceinline__ void turn_pair(float &xa, float &xb, float c, float s) {
#pragma clang fp contract(off)
    const float ya = xa * c - xb * s, yb = xb * c + xa * s;
    xa = ya;
    xb = yb;
}

__device__ __forceinline__ void turn(const Piece &p, const Angles &w, floatx4 &lo, floatx4 &hi) {
    if (!p.turned) return;
    float x[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    if (p.split) {
#pragma unroll
        for (int j = 0; j < 4; ++j) turn_pair(x[j], x[4 + j], w.cs[j / 2][j % 2 * 2], w.cs[j / 2][j % 2 * 2 + 1]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) turn_pair(x[2 * j], x[2 * j + 1], w.cs[j / 2][j % 2 * 2], w.cs[j / 2][j % 2 * 2 + 1]);
    }
    lo = (floatx4){x[0], x[1], x[2], x[3]};
    hi = (floatx4){x[4], x[5], x[6], x[7]};
}

__device__ __forceinline__ float finite_abs(float x) {
    const float m = fabsf(x);
    return m <= 3.402823466e38f ? m : 0.0f;
}

// The smallest e with amax <= 448 * 2^e, held to the stored range.
__device__ __forceinline__ int exponent_of(float amax) {
    if (amax == 0.0f) return kExpMin;
    int x;
    const float m = frexpf(amax, &x);   // amax = m * 2^x, 0.5 <= m < 1; 448 = 0.875 * 2^9
    const int e = m <= 0.875f ? x - 9 : x - 8;
    return e < kExpMin ? kExpMin : e > kExpMax ? kExpMax : e;
}

__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// A value already divided by the block's scale, ready for the conversion to
// e4m3 (which rounds to nearest even): finite ones held to the largest code,
// others not a number.
__device__ __forceinline__ float for_code(float x) {
    return fabsf(x) <= 3.402823466e38f ? fminf(fmaxf(x, -kE4m3Max), kE4m3Max) : __builtin_nanf("");
}

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    uint32_t w = __builtin_amdgcn_cvt_pk_fp8_f32(for_code(a), for_code(b), 0, false);
    return __builtin_amdgcn_cvt_pk_fp8_f32(for_code(c), for_code(d), w, true);
}

// Four codes times 2^-shift (shift > 0).
__device__ __forceinline__ uint32_t rescaled4(uint32_t w, float factor) {
    const floatx2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
    return codes4(lo.x * factor, lo.y * factor, hi.x * factor, hi.y * factor);
}

// One block of one sequence, kv head `head`, K (which = 0) or V (1).  A thread
// has 16 values: of K a piece of two tokens, of V four dimensions of four
// tokens, so that four of its codes are a word of the block's layout.
template <int D, typename T>
__device__ __forceinline__ void append_block(const AppendArgs &a, const KvSequence &s, int b, int blk, int head,
                                             int which, u32x4 *block, float *wave_max) {
    const int tid = threadIdx.x;
    // the tokens of this block that the call writes: slots [s0, s1)
    const int p0 = s.pos0 > 0 ? s.pos0 : 0, start = blk * kKvBlock;
    const int s0 = p0 > start ? p0 - start : 0;
    const int s1 = s.length - start < kKvBlock ? s.length - start : kKvBlock;
    const int id = kv_block_id(a.kv, b, blk);
    if (id < 0) return;   // uniform over the workgroup
    const int64_t plane = (static_cast<int64_t>(id) * a.kv.kv_heads + head) * 2 + which;
    u32x4 *dst = reinterpret_cast<u32x4 *>(a.kv.data + plane * (kKvBlock * D)) + tid;
    const bool whole = s1 - s0 == kKvBlock;
    u32x4 old = {0, 0, 0, 0};
    int before = kExpMin;
    if (!whole) old = *dst;
    if (s0 > 0) before = a.kv.exps[plane];
    auto row_of = [&](int slot) { return s.row0 + (start + slot - s.pos0); };
    auto mine = [&](int slot) { return slot >= s0 && slot < s1; };
    // K: x[2 t], x[2 t + 1] of token slot0 + t; V: x[t]
    const int slot0 = which == 0 ? tid / (D / 8) * 2 : tid / (D / 4) * 4;
    const int c = which == 0 ? tid % (D / 8) : tid % (D / 4);
    const Piece piece = piece_of(a, c);
    floatx4 x[4];
    float amax = 0.0f;
    if (which == 0) {
        Angles w[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            x[2 * t] = x[2 * t + 1] = (floatx4){0, 0, 0, 0};
            if (!mine(slot0 + t)) continue;
            const T *src = static_cast<const T *>(a.k) + row_of(slot0 + t) * a.k_stride + head * D;
            x[2 * t] = load4(src + piece.lo);
            x[2 * t + 1] = load4(src + piece.hi);
            w[t] = angles(a, piece, c, start + slot0 + t);
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
            if (mine(slot0 + t)) turn(piece, w[t], x[2 * t], x[2 * t + 1]);
    } else {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            x[t] = (floatx4){0, 0, 0, 0};
            if (mine(slot0 + t)) x[t] = load4(static_cast<const T *>(a.v) + row_of(slot0 + t) * a.v_stride + head * D + 4 * c);
        }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = fmaxf(amax, finite_abs(x[i / 4][i % 4]));
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) amax = fmaxf(amax, __shfl_xor(amax, m));
    if ((tid & 63) == 0) wave_max[tid >> 6] = amax;
    if (!whole) block[tid] = old;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < D / 32; ++w) amax = fmaxf(amax, wave_max[w]);
    int e = exponent_of(amax);
    if (before > e) e = before;
    if (s0 > 0 && before < e) {   // the codes that are there follow (uniform)
        const float factor = pow2(before - e < -126 ? -126 : before - e);
#pragma unroll
        for (int i = 0; i < 4; ++i) old[i] = rescaled4(old[i], factor);
        block[tid] = old;
        __syncthreads();
    }
    const float inv = pow2(-e);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = x[i] * inv;
    uint32_t *words = reinterpret_cast<uint32_t *>(block);
    if (which == 0) {
        // K: token / 16, d / 64, d / 16 % 4, token % 16, d % 16
        auto put = [&](int slot, int d, floatx4 v) {
            words[((slot / 16 * (D / 64) + d / 64) * 4 + d / 16 % 4) * 64 + slot % 16 * 4 + d % 16 / 4] = codes4(v.x, v.y, v.z, v.w);
        };
#pragma unroll
        for (int t = 0; t < 2; ++t)
            if (mine(slot0 + t)) {
                put(slot0 + t, piece.lo, x[2 * t]);
                put(slot0 + t, piece.hi, x[2 * t + 1]);
            }
    } else {
        // V: d / 32, token / 4 % 4, d % 16, d / 16 % 2, token / 16, token % 4
        uint32_t keep = 0;   // bytes of tokens that were there
#pragma unroll
        for (int t = 0; t < 4; ++t)
            if (!mine(slot0 + t)) keep |= 0xFFu << (8 * t);
        if (keep != 0xFFFFFFFFu) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int d = 4 * c + j;
                uint32_t &word = words[(d / 32 * 4 + slot0 / 4 % 4) * 64 + d % 16 * 4 + d / 16 % 2 * 2 + slot0 / 16];
                const uint32_t now = codes4(x[0][j], x[1][j], x[2][j], x[3][j]);
                word = keep ? (word & keep) | (now & ~keep) : now;
            }
        }
    }
    __syncthreads();
    *dst = block[tid];
    if (tid == 0) a.kv.exps[plane] = static_cast<int8_t>(e);   // all have read it
    __syncthreads();   // the block has been read
}

constexpr int kManyRows = 32;   // from here on the rotated q is read many times

// A piece of kHeads heads' rotated q, for which the angles are read once.
constexpr int kHeads = 2;

template <int D, typename T, bool STREAM>
__device__ __forceinline__ void rotate_q(const AppendArgs &a, int64_t row, int pos, int head0, int c) {
    const int heads = a.q_heads - head0 < kHeads ? a.q_heads - head0 : kHeads;
    const Piece piece = piece_of(a, c);
    const T *src = static_cast<const T *>(a.q) + row * a.q_stride + head0 * D;
    const Angles w = angles(a, piece, c, pos);
    floatx4 x[kHeads][2];
#pragma unroll
    for (int h = 0; h < kHeads; ++h)
        if (h < heads) {
            x[h][0] = load4(src + h * D + piece.lo);
            x[h][1] = load4(src + h * D + piece.hi);
        }
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
        if (h >= heads) break;
        turn(piece, w, x[h][0], x[h][1]);
        uint16_t *dst = a.q_out + (row * a.q_heads + head0 + h) * D;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const bf16x4 y = pos >= 0 ? __builtin_convertvector(x[h][i], bf16x4) : (bf16x4){};
            bf16x4 *to = reinterpret_cast<bf16x4 *>(dst + (i ? piece.hi : piece.lo));
            if constexpr (STREAM) __builtin_nontemporal_store(y, to);
            else *to = y;
        }
    }
}

// STREAM: with the nontemporal hint on the rotated q (a branch in the kernel would
// not do: the compiler joins two stores that differ by the hint alone).
template <int D, typename T, bool STREAM>
__global__ __launch_bounds__(2 * D) void kv_append_kernel(AppendArgs a, int block_units, int q_units) {
    __shared__ u32x4 block[2 * D];
    __shared__ float wave_max[D / 32];
    const int b = blockIdx.y;
    const KvSequence s = kv_sequence(a.kv, b);
    if (s.rows == 0) return;
    const int heads2 = a.kv.kv_heads * 2;
    int unit = blockIdx.x;
    if (unit < block_units) {
        if (s.length == 0) return;
        const int j0 = (s.pos0 > 0 ? s.pos0 : 0) / kKvBlock, j1 = (s.length - 1) / kKvBlock;
        const int step = block_units / heads2;
        for (int blk = j0 + unit / heads2; blk <= j1; blk += step)
            append_block<D, T>(a, s, b, blk, unit % heads2 / 2, unit % 2, block, wave_max);
        return;
    }
    unit -= block_units;
    const int per_row = (a.q_heads + kHeads - 1) / kHeads * (D / 8);
    const int64_t total = static_cast<int64_t>(s.rows) * per_row;
    for (int64_t u = static_cast<int64_t>(unit) * (2 * D) + threadIdx.x; u < total;
         u += static_cast<int64_t>(q_units) * (2 * D)) {
        const int t = static_cast<int>(u / per_row), in_row = static_cast<int>(u % per_row);
        rotate_q<D, T, STREAM>(a, s.row0 + t, s.pos0 + t, in_row / (D / 8) * kHeads, in_row % (D / 8));
    }
}

template <int D, typename T>
hipError_t launch(const AppendArgs &a, hipStream_t s) {
    // a sequence of n rows touches at most (n + 30) / 32 + 1 blocks; the kernel
    // loops where a launch has fewer units than that
    int64_t blocks = (static_cast<int64_t>(a.max_rows) + kKvBlock - 2) / kKvBlock + 1;
    if (blocks > 4096) blocks = 4096;
    const int64_t block_units = blocks * a.kv.kv_heads * 2;
    const int64_t per_row = (a.q_heads + kHeads - 1) / kHeads * (D / 8);
    int64_t q_units = (a.max_rows * per_row + 2 * D - 1) / (2 * D);
    if (q_units > (1 << 20)) q_units = 1 << 20;
    const dim3 grid(static_cast<uint32_t>(block_units + q_units), static_cast<uint32_t>(a.kv.batch));
    if (a.max_rows < kManyRows)
        hipLaunchKernelGGL((kv_append_kernel<D, T, true>), grid, dim3(2 * D), 0, s, a, static_cast<int>(block_units),
                           static_cast<int>(q_units));
    else
        hipLaunchKernelGGL((kv_append_kernel<D, T, false>), grid, dim3(2 * D), 0, s, a, static_cast<int>(block_units),
                           static_cast<int>(q_units));
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs &a, int head_dim, int dtype, hipStream_t s) {
    if (head_dim == 128)
        return dtype == Q4_BF16 ? launch<128, uint16_t>(a, s) : launch<128, float>(a, s);
    return dtype == Q4_BF16 ? launch<64, uint16_t>(a, s) : launch<64, float>(a, s);
}

}  // namespace q4
