// Rotation of q and k, quantization of k and v to 8 bits, and the append to
// the paged cache (include/q4_decoder.h).
//
// A workgroup of 2 * D threads has one of two tasks.  The first: one block of
// one sequence, one kv head, K or V.  Each thread holds 16 dimensions of one
// of the block's 32 tokens; the largest finite value of the new tokens gives
// the block's exponent, the codes of tokens that were there before are
// rescaled where the exponent rises, and the codes go out as 16-byte pieces
// of the block's layout (V, whose bytes run along the tokens, turns through
// LDS).  The second: 16 dimensions a thread of the rotated q.
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
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ void load16(const float *p, float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const floatx4 v = reinterpret_cast<const floatx4 *>(p)[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[4 * i + j] = v[j];
    }
}

__device__ __forceinline__ void load16(const uint16_t *p, float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const u32x4 v = reinterpret_cast<const u32x4 *>(p)[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[8 * i + 2 * j] = __uint_as_float(v[j] << 16);
            x[8 * i + 2 * j + 1] = __uint_as_float(v[j] & 0xFFFF0000u);
        }
    }
}

// The 16 values at dimension d0 of a head's row, rotated by position pos.
template <typename T>
__device__ __forceinline__ void rotated16(const T *head, int d0, int pos, const AppendArgs &a, float (&x)[16]) {
#pragma clang fp contract(off)
    load16(head + d0, x);
    if (d0 >= a.rot) return;
    if (pos >= a.positions) {
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = __builtin_nanf("");
        return;
    }
    const int half = a.rot / 2;
    const floatx2 *row = reinterpret_cast<const floatx2 *>(a.rope) + static_cast<int64_t>(pos) * half;
    if (a.interleaved) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const floatx2 cs = row[d0 / 2 + j];
            const float xa = x[2 * j], xb = x[2 * j + 1];
            x[2 * j] = xa * cs.x - xb * cs.y;
            x[2 * j + 1] = xb * cs.x + xa * cs.y;
        }
    } else {
        const bool first = d0 < half;
        float m[16];   // the other value of each pair
        load16(head + (first ? d0 + half : d0 - half), m);
        const floatx2 *cs16 = row + (first ? d0 : d0 - half);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const floatx2 cs = cs16[j];
            const float turn = m[j] * cs.y;
            x[j] = first ? x[j] * cs.x - turn : x[j] * cs.x + turn;
        }
    }
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

// One block of one sequence, kv head `head`, K (which = 0) or V (1).
template <int D, typename T>
__device__ __forceinline__ void append_block(const AppendArgs &a, const KvSequence &s, int b, int blk, int head,
                                             int which, uint8_t *turn, float *wave_max) {
    const int tid = threadIdx.x;
    // the tokens of this block that the call writes: slots [s0, s1)
    const int p0 = s.pos0 > 0 ? s.pos0 : 0, start = blk * kKvBlock;
    const int s0 = p0 > start ? p0 - start : 0;
    const int s1 = s.length - start < kKvBlock ? s.length - start : kKvBlock;
    const int id = kv_block_id(a.kv, b, blk);
    if (id < 0) return;   // uniform over the workgroup
    // K: the thread's 16 bytes of the block are 16 dimensions of one token;
    // V: threads run along a token's dimensions
    int slot, d0;
    if (which == 0) {
        slot = tid / (64 * (D / 64)) * 16 + tid % 16;
        d0 = tid / 64 % (D / 64) * 64 + tid / 16 % 4 * 16;
    } else {
        slot = tid / (D / 16);
        d0 = tid % (D / 16) * 16;
    }
    const bool mine = slot >= s0 && slot < s1;
    float x[16];
    float amax = 0.0f;
    if (mine) {
        const int pos = start + slot;
        const int64_t row = s.row0 + (pos - s.pos0);
        if (which == 0)
            rotated16(static_cast<const T *>(a.k) + row * a.k_stride + head * D, d0, pos, a, x);
        else
            load16(static_cast<const T *>(a.v) + row * a.v_stride + head * D + d0, x);
#pragma unroll
        for (int j = 0; j < 16; ++j) amax = fmaxf(amax, finite_abs(x[j]));
    }
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) amax = fmaxf(amax, __shfl_xor(amax, m));
    if ((tid & 63) == 0) wave_max[tid >> 6] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < D / 32; ++w) amax = fmaxf(amax, wave_max[w]);
    const int64_t plane = (static_cast<int64_t>(id) * a.kv.kv_heads + head) * 2 + which;
    int e = exponent_of(amax);
    float factor = 1.0f;   // of the codes that are there
    if (s0 > 0) {
        const int before = a.kv.exps[plane];
        if (before > e) e = before;
        factor = pow2(before - e < -126 ? -126 : before - e);
    }
    const float inv = pow2(-e);
    u32x4 *dst = reinterpret_cast<u32x4 *>(a.kv.data + plane * (kKvBlock * D)) + tid;
    u32x4 w = {0, 0, 0, 0};
    if (mine)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = codes4(x[4 * i] * inv, x[4 * i + 1] * inv, x[4 * i + 2] * inv, x[4 * i + 3] * inv);
    if (which == 0) {
        if (mine) {
            *dst = w;
        } else if (factor != 1.0f) {
            u32x4 old = *dst;
#pragma unroll
            for (int i = 0; i < 4; ++i) old[i] = rescaled4(old[i], factor);
            *dst = old;
        }
    } else {
        if (s1 - s0 < kKvBlock) {
            u32x4 old = *dst;
            if (factor != 1.0f)
#pragma unroll
                for (int i = 0; i < 4; ++i) old[i] = rescaled4(old[i], factor);
            reinterpret_cast<u32x4 *>(turn)[tid] = old;
            __syncthreads();
        }
        if (mine) {
            const int piece = d0 / 16;
            uint8_t *to = turn + (piece / 2 * 4 + slot / 4 % 4) * 256 + piece % 2 * 8 + slot / 16 * 4 + slot % 4;
#pragma unroll
            for (int j = 0; j < 16; ++j) to[16 * j] = static_cast<uint8_t>(w[j / 4] >> (8 * (j % 4)));
        }
        __syncthreads();
        *dst = reinterpret_cast<const u32x4 *>(turn)[tid];
    }
    // read above by every thread, before its data-dependent stores; the
    // exponent changes only after all have it
    __syncthreads();
    if (tid == 0) a.kv.exps[plane] = static_cast<int8_t>(e);
}

template <int D, typename T>
__global__ __launch_bounds__(2 * D) void kv_append_kernel(AppendArgs a, int block_units, int q_units) {
    __shared__ __align__(16) uint8_t turn[kKvBlock * D];
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
            append_block<D, T>(a, s, b, blk, unit % heads2 / 2, unit % 2, turn, wave_max);
        return;
    }
    unit -= block_units;
    const int per_row = a.q_heads * (D / 16);
    const int64_t total = static_cast<int64_t>(s.rows) * per_row;
    for (int64_t u = static_cast<int64_t>(unit) * (2 * D) + threadIdx.x; u < total;
         u += static_cast<int64_t>(q_units) * (2 * D)) {
        const int t = static_cast<int>(u / per_row), piece = static_cast<int>(u % per_row);
        const int64_t row = s.row0 + t;
        const int pos = s.pos0 + t, head = piece / (D / 16), d0 = piece % (D / 16) * 16;
        u32x4 o[2] = {};
        if (pos >= 0) {
            float x[16];
            rotated16(static_cast<const T *>(a.q) + row * a.q_stride + head * D, d0, pos, a, x);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                o[i / 4][i % 4] =
                    __builtin_bit_cast(uint32_t, __builtin_convertvector((floatx2){x[2 * i], x[2 * i + 1]}, bf16x2));
        }
        u32x4 *dst = reinterpret_cast<u32x4 *>(a.q_out + (row * a.q_heads + head) * D + d0);
        dst[0] = o[0];
        dst[1] = o[1];
    }
}

template <int D, typename T>
hipError_t launch(const AppendArgs &a, hipStream_t s) {
    // a sequence of n rows touches at most (n + 30) / 32 + 1 blocks; the kernel
    // loops where a launch has fewer units than that
    int64_t blocks = (static_cast<int64_t>(a.max_rows) + kKvBlock - 2) / kKvBlock + 1;
    if (blocks > 4096) blocks = 4096;
    const int64_t block_units = blocks * a.kv.kv_heads * 2;
    int64_t q_units = (static_cast<int64_t>(a.max_rows) * a.q_heads * (D / 16) + 2 * D - 1) / (2 * D);
    if (q_units > (1 << 20)) q_units = 1 << 20;
    hipLaunchKernelGGL((kv_append_kernel<D, T>),
                       dim3(static_cast<uint32_t>(block_units + q_units), static_cast<uint32_t>(a.kv.batch)),
                       dim3(2 * D), 0, s, a, static_cast<int>(block_units), static_cast<int>(q_units));
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs &a, int head_dim, int dtype, hipStream_t s) {
    if (head_dim == 128)
        return dtype == Q4_BF16 ? launch<128, uint16_t>(a, s) : launch<128, float>(a, s);
    return dtype == Q4_BF16 ? launch<64, uint16_t>(a, s) : launch<64, float>(a, s);
}

}  // namespace q4
