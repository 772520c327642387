// Penalties for repeated tokens, biases and the grammar mask on logits
// (include/q4_decoder.h).
//
// A workgroup has CH consecutive tokens of one row.  It walks the row's
// history once and counts, in LDS, how often each of its tokens occurs (bit 0:
// seen in the prompt, the rest: occurrences after it), then its biases, then
// writes its tokens: one pass over the logits, no counts in memory.  The
// counts are whole numbers, so the order of the LDS atomics does not matter;
// biases of one token are added one by one in the order of the list.

#include "q4_decoder_internal.h"

namespace q4 {
namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;

struct RowParams {
    float rho, frequency, presence;
};

__device__ __forceinline__ float adjusted(float z, uint32_t seen, float bias, const RowParams &p) {
#pragma clang fp contract(off)
    if (seen) z = z > 0.0f ? z / p.rho : z * p.rho;
    const uint32_t n = seen >> 1;
    if (n) {
        z = z - p.frequency * static_cast<float>(n);
        z = z - p.presence;
    }
    return z + bias;
}

// the bounds of row m in a list of `size` entries
__device__ __forceinline__ void bounds(const int32_t *cu, int m, int32_t size, int32_t &lo, int32_t &hi) {
    lo = cu[m];
    hi = cu[m + 1];
    lo = lo < 0 ? 0 : lo > size ? size : lo;
    hi = hi < lo ? lo : hi > size ? size : hi;
}

template <int CH, int VEC>
__global__ __launch_bounds__(kThreads) void logits_adjust_kernel(LogitsArgs a) {
    __shared__ uint32_t count[CH];
    __shared__ float bias[CH];
    __shared__ int32_t owner[CH];
    const int m = blockIdx.y, base = blockIdx.x * CH;
    const int tid = threadIdx.x;
    for (int i = tid; i < CH; i += kThreads) {
        count[i] = 0;
        bias[i] = 0.0f;
        owner[i] = 0x7FFFFFFF;
    }
    __syncthreads();
    if (a.history_size) {
        int32_t lo, hi;
        bounds(a.cu_history, m, a.history_size, lo, hi);
        const int64_t answer = lo + (a.prompt_lengths ? static_cast<int64_t>(a.prompt_lengths[m]) : 0);
        for (int64_t i = lo + tid; i < hi; i += kThreads) {
            const int64_t t = static_cast<int64_t>(a.history[i]) - base;
            if (t >= 0 && t < CH) {
                if (i >= answer) atomicAdd(&count[t], 2u);
                else atomicOr(&count[t], 1u);
            }
        }
    }
    if (a.bias_size) {
        int32_t lo, hi;
        bounds(a.cu_bias, m, a.bias_size, lo, hi);
        for (int64_t i0 = lo; i0 < hi; i0 += kThreads) {
            const int64_t i = i0 + tid;
            const int64_t t = i < hi ? static_cast<int64_t>(a.bias_ids[i]) - base : -1;
            bool pending = t >= 0 && t < CH;
            // the first pending entry of a token adds its bias, then the next
            while (__syncthreads_or(pending)) {
                if (pending) atomicMin(&owner[t], tid);
                __syncthreads();
                const bool wins = pending && owner[t] == tid;
                if (wins) {
                    bias[t] += a.bias[i];
                    pending = false;
                }
                __syncthreads();
                if (wins) owner[t] = 0x7FFFFFFF;
            }
        }
    }
    __syncthreads();
    RowParams p;
    p.rho = a.repetition ? a.repetition[m] : 1.0f;
    p.frequency = a.frequency ? a.frequency[m] : 0.0f;
    p.presence = a.presence ? a.presence[m] : 0.0f;
    const int n = a.V - base < CH ? a.V - base : CH;
    const float *src = a.logits + static_cast<int64_t>(m) * a.V + base;
    float *dst = a.out + static_cast<int64_t>(m) * a.V + base;
    const uint32_t *mask = a.mask ? a.mask + static_cast<int64_t>(m) * ((a.V + 31) / 32) + base / 32 : nullptr;
    const float ninf = -__builtin_inff();
    if constexpr (VEC) {
        for (int i = tid; i < n / 4; i += kThreads) {
            floatx4 z = reinterpret_cast<const floatx4 *>(src)[i];
            const uint32_t bits = mask ? mask[i / 8] >> (i % 8 * 4) : 15u;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                z[j] = (bits >> j) & 1u ? adjusted(z[j], count[4 * i + j], bias[4 * i + j], p) : ninf;
            reinterpret_cast<floatx4 *>(dst)[i] = z;
        }
    } else {
        for (int i = tid; i < n; i += kThreads)
            dst[i] = !mask || ((mask[i / 32] >> (i % 32)) & 1u) ? adjusted(src[i], count[i], bias[i], p) : ninf;
    }
}

template <int CH>
hipError_t launch(const LogitsArgs &a, hipStream_t s) {
    const dim3 grid(static_cast<uint32_t>((a.V + CH - 1) / CH), static_cast<uint32_t>(a.M));
    // rows start on 16 bytes only where V is a multiple of four
    if (a.V % 4 == 0)
        hipLaunchKernelGGL((logits_adjust_kernel<CH, 1>), grid, dim3(kThreads), 0, s, a);
    else
        hipLaunchKernelGGL((logits_adjust_kernel<CH, 0>), grid, dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_logits_adjust(const LogitsArgs &a, hipStream_t s) { return launch<2048>(a, s); }

}  // namespace q4
