// Penalties for repeated tokens, biases and the grammar mask on logits
// (include/q4_decoder.h).
//
// A workgroup has CH consecutive tokens of one row, eight to a thread, and
// loads them, the row's bounds and the first ids of its lists together.  It
// counts in LDS how often each of its tokens occurs in the history, applies
// the penalties in registers, adds up the biases in the same LDS and writes
// its tokens: one pass over the logits, no counts in memory.  The counts are
// whole numbers, so the order of the LDS atomics does not matter; biases of
// one token are added one by one in the order of the list.

#include "q4_decoder_internal.h"

namespace q4 {
namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kAtOnce = 16;  // ids of a thread in flight

struct RowParams {
    float rho, inv_rho, frequency, presence;
};

// Without branches: among 64 tokens some are nearly always seen.  z / rho is
// z * (1 / rho), within 2 roundings of it, as a division of every token takes
// longer than the rest of the kernel.
__device__ __forceinline__ float penalized(float z, uint32_t in_prompt, uint32_t n, const RowParams &p) {
    const float scale = z > 0.0f ? p.inv_rho : p.rho;
    z *= in_prompt | n ? scale : 1.0f;
    z -= n ? p.frequency * static_cast<float>(n) : 0.0f;
    return z - (n ? p.presence : 0.0f);
}

// p[i], or, where p is null, `none`: a load either way (of other memory that
// is there), so that a row's parameters are all on their way at once.
template <typename T>
__device__ __forceinline__ T value_or(const T *p, int64_t i, const void *there, T none) {
    const T v = *(p ? p + i : static_cast<const T *>(there));
    return p ? v : none;
}

template <int CH, int VEC>
__global__ __launch_bounds__(CH / 8) void logits_adjust_kernel(LogitsArgs a) {
    constexpr int kThreads = CH / 8;
    __shared__ __align__(16) uint32_t slot[CH];    // a token's count in the answer, later its bias
    __shared__ __align__(16) uint32_t other[CH];   // its count in the prompt, later of pending biases
    const int m = blockIdx.y, base = blockIdx.x * CH;
    const int tid = threadIdx.x;
    const int n = a.V - base < CH ? a.V - base : CH;
    const float *src = a.logits + static_cast<int64_t>(m) * a.V + base;
    float *dst = a.out + static_cast<int64_t>(m) * a.V + base;
    const uint32_t *mask = a.mask ? a.mask + static_cast<int64_t>(m) * ((a.V + 31) / 32) + base / 32 : nullptr;
    int32_t h0 = value_or(a.cu_history, m, src, 0), h1 = value_or(a.cu_history, m + 1, src, 0);
    int32_t b0 = value_or(a.cu_bias, m, src, 0), b1 = value_or(a.cu_bias, m + 1, src, 0);
    const int32_t prompt = value_or(a.prompt_lengths, m, src, 0);
    RowParams p;
    p.rho = value_or(a.repetition, m, src, 1.0f);
    p.frequency = value_or(a.frequency, m, src, 0.0f);
    p.presence = value_or(a.presence, m, src, 0.0f);
    p.inv_rho = 1.0f / p.rho;
    auto hold = [](int32_t &lo, int32_t &hi, int32_t size) {   // bounds within their list
        lo = lo < 0 ? 0 : lo > size ? size : lo;
        hi = hi < lo ? lo : hi > size ? size : hi;
    };
    hold(h0, h1, a.history_size);
    hold(b0, b1, a.bias_size);
    // entries count from the row's first
    const int nh = h1 - h0, nb = b1 - b0;
    const int32_t *history = a.history + h0, *bias_ids = a.bias_ids + b0;
    const float *biases = a.bias + b0;

    // token of the thread's j-th value of half u
    auto token = [&](int u, int j) { return VEC ? 4 * (tid + kThreads * u) + j : tid + kThreads * (4 * u + j); };
    floatx4 z[2];
    uint32_t bits[2] = {15u, 15u};   // which values the mask allows
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        if constexpr (VEC) {
            const int i = tid + kThreads * u;
            if (4 * i < n) {
                z[u] = reinterpret_cast<const floatx4 *>(src)[i];
                if (mask) bits[u] = mask[i / 8] >> (i % 8 * 4);
            }
        } else {
            if (mask) bits[u] = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = token(u, j);
                if (i < n) z[u][j] = src[i];
                if (mask && i < n) bits[u] |= ((mask[i / 32] >> (i % 32)) & 1u) << j;
            }
        }
    }
    auto load_ids = [&](uint32_t i0, int32_t(&to)[kAtOnce]) {
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const uint32_t i = i0 + tid + kThreads * k;
            to[k] = -1;
            if (i0 + kThreads * k < static_cast<uint32_t>(nh) && i < static_cast<uint32_t>(nh)) to[k] = history[i];
        }
    };
    int32_t bias_id;
    float bias;
    auto load_bias = [&](uint32_t i) {
        bias_id = i < static_cast<uint32_t>(nb) ? bias_ids[i] : -1;
        bias = i < static_cast<uint32_t>(nb) ? biases[i] : 0.0f;
    };
    int32_t id[kAtOnce];
    load_ids(0, id);
    load_bias(tid);
    auto clear = [&] {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int j = 0; j < 4; ++j) slot[token(u, j)] = other[token(u, j)] = 0;
    };
    if (nh > 0) {
        clear();
        __syncthreads();
        for (uint32_t i0 = 0; i0 < static_cast<uint32_t>(nh); i0 += kThreads * kAtOnce) {
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                if (i0 + kThreads * k >= static_cast<uint32_t>(nh)) break;
                const uint32_t t = static_cast<uint32_t>(id[k] - base);
                const bool answer = static_cast<int64_t>(i0 + tid + kThreads * k) >= prompt;
                if (id[k] >= base && t < CH) atomicAdd(&(answer ? slot : other)[t], 1u);
            }
            load_ids(i0 + kThreads * kAtOnce, id);
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int j = 0; j < 4; ++j) z[u][j] = penalized(z[u][j], other[token(u, j)], slot[token(u, j)], p);
    }
    if (nb > 0) {
        clear();   // each thread its own slots, which it has read
        __syncthreads();
        for (uint32_t i0 = 0; i0 < static_cast<uint32_t>(nb); i0 += kThreads) {
            const uint32_t t = static_cast<uint32_t>(bias_id - base);
            bool pending = bias_id >= base && t < CH;
            const float value = bias;
            const bool repeated = pending && atomicAdd(&other[t], 1u) > 0;
            if (__syncthreads_or(repeated)) {
                // the first pending entry of a token adds its bias, then the next
                while (__syncthreads_or(pending)) {
                    if (pending) other[t] = 0xFFFFFFFFu;
                    __syncthreads();
                    if (pending) atomicMin(&other[t], static_cast<uint32_t>(tid));
                    __syncthreads();
                    if (pending && other[t] == static_cast<uint32_t>(tid)) {
                        slot[t] = __float_as_uint(__uint_as_float(slot[t]) + value);
                        pending = false;
                    }
                }
                if (bias_id >= base && t < CH) other[t] = 0;
            } else if (pending) {
                slot[t] = __float_as_uint(__uint_as_float(slot[t]) + value);
                other[t] = 0;
            }
            __syncthreads();
            load_bias(i0 + kThreads + tid);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int j = 0; j < 4; ++j) z[u][j] += __uint_as_float(slot[token(u, j)]);
    }
    const float ninf = -__builtin_inff();
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int j = 0; j < 4; ++j) z[u][j] = (bits[u] >> j) & 1u ? z[u][j] : ninf;
        if constexpr (VEC) {
            const int i = tid + kThreads * u;
            if (4 * i < n) reinterpret_cast<floatx4 *>(dst)[i] = z[u];
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (token(u, j) < n) dst[token(u, j)] = z[u][j];
        }
    }
}

template <int CH>
hipError_t launch(const LogitsArgs &a, hipStream_t s) {
    const dim3 grid(static_cast<uint32_t>((a.V + CH - 1) / CH), static_cast<uint32_t>(a.M));
    // rows start on 16 bytes only where V is a multiple of four
    if (a.V % 4 == 0)
        hipLaunchKernelGGL((logits_adjust_kernel<CH, 1>), grid, dim3(CH / 8), 0, s, a);
    else
        hipLaunchKernelGGL((logits_adjust_kernel<CH, 0>), grid, dim3(CH / 8), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_logits_adjust(const LogitsArgs &a, hipStream_t s) {
    // Every workgroup reads its row's history, so long runs of tokens read it
    // less often; short ones spread few rows over the chip.
    return static_cast<int64_t>(a.M) * a.V >= int64_t(4096) * 256 ? launch<4096>(a, s) : launch<1024>(a, s);
}

}  // namespace q4
