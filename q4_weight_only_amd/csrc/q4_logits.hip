// Penalties for repeated tokens, biases and the grammar mask on logits
// (include/q4_decoder.h).
//
// A workgroup has CH consecutive tokens of one row, eight to a thread, and
// loads them, the row's bounds and the first entries of its lists together.
// It counts in LDS how often each of its tokens occurs in the history, notes
// there the token's bias, and applies both in registers, where some lane's
// four tokens have any: one pass over the logits, no counts in memory.  The
// counts are whole numbers, so the order of the LDS atomics does not matter;
// biases of one token are added one by one in the order of the list.
//
// 32 rows of 131072 tokens with the mask alone take 6.6 us (34 MB: 5.1 TB/s),
// with 4099 ids and 300 biases each 8.9, of which the chain from the bounds to
// the ids to the counts is the most; one row with 200 ids 3.6.  What cost time
// here: instructions for every token (a second array of counts took 0.9 us),
// the length of the code, which short calls fetch as they go (0.5 us for ids
// read one by one), stores that stay in the writer's L2 (1.6 us).
//
// The stores go through to the device's scope.  What takes the logits next reads
// all of them at once, and such stores leave them where it finds them, while the
// nontemporal hint, as fast here, does not, and plain stores are slower here (32
// rows with the mask alone, plain / nontemporal / these: 7.2 / 7.0 / 7.0 us, with
// an arg max behind it 47.0 / 59.8 / 46.8, with a softmax 51.6 / 64.9 / 51.4; with
// 4099 ids and 300 biases 10.7 / 8.9 / 8.8).

#include "q4_decoder_internal.h"

namespace q4 {
namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));
// rows start on 4 bytes only, which such loads and stores allow
typedef float floatx4_row __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kQuads = 4;     // of ids of a thread in flight
constexpr int kBiases = 4;    // entries of the bias list that a thread has at first
constexpr int kDeviceScope = 16;   // of a buffer store's cache policy: the bit sc1

struct RowParams {
    float rho, inv_rho, frequency, presence;
};

// Without branches; z / rho is z * (1 / rho), within 2 roundings of it.  n: how
// often the token is in the answer.
__device__ __forceinline__ float penalized(float z, bool seen, uint32_t n, const RowParams &p) {
    const float scale = z > 0.0f ? p.inv_rho : p.rho;
    const float off = fmaf(p.frequency, static_cast<float>(n), p.presence);
    return z * (seen ? scale : 1.0f) - (n ? off : 0.0f);
}

// p[i], or, where p is null, `none`: a load either way (of other memory that
// is there), so that a row's parameters are all on their way at once.
template <typename T>
__device__ __forceinline__ T value_or(const T *p, int64_t i, const void *there, T none) {
    const T v = *(p ? p + i : static_cast<const T *>(there));
    return p ? v : none;
}

template <int CH>
__global__ __launch_bounds__(CH / 8) void logits_adjust_kernel(LogitsArgs a) {
    constexpr int kThreads = CH / 8;
    __shared__ __align__(16) uint32_t count[CH];   // how often a token is in the answer
    __shared__ __align__(4) uint8_t seen[CH];      // 1 where it is in the history at all
    __shared__ __align__(16) float noted[CH];      // its bias, where `biased` has its bit
    __shared__ uint32_t biased[CH / 32];           // a bit for each token of the bias list
    const int m = blockIdx.y, base = blockIdx.x * CH;
    const int tid = threadIdx.x;
    const int n = a.V - base < CH ? a.V - base : CH;
    const float *src = a.logits + static_cast<int64_t>(m) * a.V + base;
    float *dst = a.out + static_cast<int64_t>(m) * a.V + base;
    const uint32_t *mask = a.mask ? a.mask + static_cast<int64_t>(m) * ((a.V + 31) / 32) + base / 32 : nullptr;
    int32_t h0 = value_or(a.cu_history, m, src, 0), h1 = value_or(a.cu_history, m + 1, src, 0);
    int32_t b0 = value_or(a.cu_bias, m, src, 0), b1 = value_or(a.cu_bias, m + 1, src, 0);
    const int32_t prompt_length = value_or(a.prompt_lengths, m, src, 0);
    const int32_t prompt = prompt_length > 0 ? prompt_length : 0;
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
    auto token = [&](int u, int j) { return 4 * (tid + kThreads * u) + j; };
    floatx4 z[2];
    uint32_t bits[2] = {15u, 15u};   // which values the mask allows
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int t = token(u, 0);
        if (t < n && mask) bits[u] = mask[t / 32] >> t % 32;
        if (t + 4 <= n) {
            z[u] = *reinterpret_cast<const floatx4_row *>(src + t);
        } else {
#pragma unroll
            for (int j = 0; j < 3; ++j)
                if (t + j < n) z[u][j] = src[t + j];
        }
    }
    int32_t id[4 * kQuads], bias_id[kBiases];
    float bias[kBiases];
    // the thread's entries i0 + 4 * (tid + kThreads * k) + j of the history
    // (what lies past its end reads as 0 and is not counted)
    auto load_ids = [&](int32_t i0) {
        const int32_t left = nh - i0 < 4 * kQuads * kThreads ? nh - i0 : 4 * kQuads * kThreads;
        const __amdgpu_buffer_rsrc_t list =
            __builtin_amdgcn_make_buffer_rsrc(const_cast<int32_t *>(history + i0), 0, 4 * left, 0x00020000);
#pragma unroll
        for (int k = 0; k < kQuads; ++k) {
            if (4 * kThreads * k >= left) break;
            const u32x4 v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(list, 16 * (tid + kThreads * k), 0, 0));
#pragma unroll
            for (int j = 0; j < 4; ++j) id[4 * k + j] = static_cast<int32_t>(v[j]);
        }
    };
    if (nh > 0) load_ids(0);
#pragma unroll
    for (int k = 0; k < kBiases; ++k) {
        const uint32_t i = tid + kThreads * k;
        bias_id[k] = -1;
        if (kThreads * k < nb && i < static_cast<uint32_t>(nb)) {
            bias_id[k] = bias_ids[i];
            bias[k] = biases[i];
        }
    }
    if (nh > 0 || nb > 0) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int j = 0; j < 4; ++j) count[token(u, j)] = seen[token(u, j)] = 0;
        if (tid < CH / 32) biased[tid] = 0;
        __syncthreads();
        for (int32_t i0 = 0;;) {
#pragma unroll
            for (int k = 0; k < kQuads; ++k) {
                const int32_t first = 4 * kThreads * k;
                if (first >= nh - i0) break;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int32_t i = first + 4 * tid + j;
                    const uint32_t t = static_cast<uint32_t>(id[4 * k + j] - base);
                    if (t < CH && i < nh - i0) {   // not for ids below base or 0 either
                        atomicAdd(&count[t], i >= prompt - i0 ? 1u : 0u);
                        seen[t] = 1;
                    }
                }
            }
            if (nh - i0 <= 4 * kQuads * kThreads) break;
            i0 += 4 * kQuads * kThreads;
            load_ids(i0);
        }
        // whether some token has more than one bias, or some thread more than kBiases
        bool again = nb > kThreads * kBiases;
#pragma unroll
        for (int k = 0; k < kBiases; ++k) {
            const uint32_t t = static_cast<uint32_t>(bias_id[k] - base);
            if (t < CH) {
                noted[t] = bias[k];
                again |= (atomicOr(&biased[t / 32], 1u << t % 32) >> t % 32) & 1;
            }
        }
        again = __syncthreads_or(again);
        if (nh > 0)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                bool any = false, is_seen[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) any |= is_seen[j] = seen[token(u, j)] != 0;
                if (any)
#pragma unroll
                    for (int j = 0; j < 4; ++j) z[u][j] = penalized(z[u][j], is_seen[j], count[token(u, j)], p);
            }
        if (nb > 0 && !again)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int t = token(u, 0);
                const uint32_t has = biased[t / 32] >> t % 32 & 15u;
                if (has)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (has >> j & 1u) z[u][j] += noted[token(u, j)];
            }
        if (again) {   // noted: the sum of a token's biases; count: its pending entries
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    count[token(u, j)] = 0;
                    noted[token(u, j)] = 0.0f;
                }
            __syncthreads();
            for (uint32_t i0 = 0; i0 < static_cast<uint32_t>(nb); i0 += kThreads) {
                const uint32_t i = i0 + tid;
                const uint32_t t = static_cast<uint32_t>((i < static_cast<uint32_t>(nb) ? bias_ids[i] : -1) - base);
                const float add = i < static_cast<uint32_t>(nb) ? biases[i] : 0.0f;
                bool pending = t < CH;
                const bool repeated = pending && atomicAdd(&count[t], 1u) > 0;
                if (__syncthreads_or(repeated)) {
                    // the first pending entry of a token adds its bias, then the next
                    while (__syncthreads_or(pending)) {
                        if (pending) count[t] = 0xFFFFFFFFu;
                        __syncthreads();
                        if (pending) atomicMin(&count[t], static_cast<uint32_t>(tid));
                        __syncthreads();
                        if (pending && count[t] == static_cast<uint32_t>(tid)) {
                            noted[t] += add;
                            pending = false;
                        }
                    }
                } else if (pending) {
                    noted[t] += add;
                }
                if (t < CH) count[t] = 0;
                __syncthreads();
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int j = 0; j < 4; ++j) z[u][j] += noted[token(u, j)];
        }
    }
    const float ninf = -__builtin_inff();
    const __amdgpu_buffer_rsrc_t row = __builtin_amdgcn_make_buffer_rsrc(dst, 0, 4 * n, 0x00020000);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int j = 0; j < 4; ++j) z[u][j] = (bits[u] >> j) & 1u ? z[u][j] : ninf;
        const int t = token(u, 0);
        if (t + 4 <= n) {
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, z[u]), row, 4 * t, 0, kDeviceScope);
        } else {
#pragma unroll
            for (int j = 0; j < 3; ++j)
                if (t + j < n) dst[t + j] = z[u][j];
        }
    }
}

template <int CH>
hipError_t launch(const LogitsArgs &a, hipStream_t s) {
    const dim3 grid(static_cast<uint32_t>((a.V + CH - 1) / CH), static_cast<uint32_t>(a.M));
    hipLaunchKernelGGL((logits_adjust_kernel<CH>), grid, dim3(CH / 8), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_logits_adjust(const LogitsArgs &a, hipStream_t s) {
    // Every workgroup reads its row's history, so where that is long, long runs
    // of tokens take less time (4099 ids and 300 biases a row of 131072: 4.7
    // against 5.4 us for one row, 8.9 against 11.3 for 32), and where it is
    // short, short ones do, which spread few rows over the chip (200 and 16: 3.6
    // against 4.0 us for one row, 7.3 against 7.4 for 32).
    return a.history_size > int64_t(1000) * a.M ? launch<4096>(a, s) : launch<1024>(a, s);
}

}  // namespace q4
