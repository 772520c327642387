// The residual step between two blocks (include/q4_decoder.h): norm of the
// block's output, gate, residual scale, residual add, norm for the next block
// and its modulation, in one pass over the rows.
//
// T threads have one row, and a thread holds NV groups of four consecutive
// elements of it in registers from the first sum to the last store, so that y
// and the residual are read once.  Rows longer than 16384 are read again for
// each sum instead.
//
// What bounds it is memory: 2048 rows of 3072 (fp32 in, bf16 x out) take
// 15.5 us, 5.7 TB/s, with a post norm 15.8; 6020 rows of 1280 18.0, 6.0 TB/s.
// Two rows of 3072 take 2.5 us: a launch, a load and a sum.
//
// The new residual, which is read only after the block, is stored with the
// nontemporal hint (without it 15.6, 18.3 and 22.4).  x is not: the linear after
// it reads it at once, and pays more than the hint saves here (norm, linear up
// and linear down, us with / without it on x: 128 rows of 3072 81.4 / 77.1, 256
// 83.5 / 78.2, 512 92.9 / 90.1, 2048 189 / 187, 4096 363.3 / 362.9, 6020 of 1280
// 206.6 / 206.0; the norm alone 17.5 / 18.0 for these, 24.2 / 29.1 for 2048 of
// 5120).

#include "q4_decoder_internal.h"

namespace q4 {
namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

template <int BF16>
__device__ __forceinline__ floatx4 load4(const void *p, int64_t i) {   // i: group of four elements
    if constexpr (BF16)
        return __builtin_convertvector(reinterpret_cast<const bf16x4 *>(p)[i], floatx4);
    else
        return reinterpret_cast<const floatx4 *>(p)[i];
}

// STREAM: with the nontemporal hint, for what no kernel reads soon.
template <int BF16, bool STREAM>
__device__ __forceinline__ void store4(void *p, int64_t i, floatx4 v) {
    if constexpr (BF16) {
        const bf16x4 h = __builtin_convertvector(v, bf16x4);
        if constexpr (STREAM) __builtin_nontemporal_store(h, reinterpret_cast<bf16x4 *>(p) + i);
        else reinterpret_cast<bf16x4 *>(p)[i] = h;
    } else {
        if constexpr (STREAM) __builtin_nontemporal_store(v, reinterpret_cast<floatx4 *>(p) + i);
        else reinterpret_cast<floatx4 *>(p)[i] = v;
    }
}

__device__ __forceinline__ float sum_sq(floatx4 v) { return v.x * v.x + v.y * v.y + v.z * v.z + v.w * v.w; }

template <int T>
__device__ __forceinline__ float row_sum(float v, float *part) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m);
    if constexpr (T == 64) return v;
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    float sum = part[0];
#pragma unroll
    for (int i = 1; i < T / 64; ++i) sum += part[i];
    return sum;
}

// y's group i, normed (where post_weight is given) and gated
template <int YB>
__device__ __forceinline__ floatx4 update(const NormArgs &a, floatx4 y, float inv, const float *gate, int i) {
    if (a.post_weight) y = y * inv * load4<0>(a.post_weight, i);
    if (gate) y = y * load4<0>(gate, i);
    return y * a.scale;
}

template <int T>
constexpr int kBlock = T < 256 ? 256 : T;   // threads of a workgroup

template <int RB, int YB, int XB, int T, int NV>
__global__ __launch_bounds__(kBlock<T>) void add_rmsnorm_kernel(NormArgs a) {
    __shared__ float part[2][kBlock<T> / 64];
    constexpr int kRows = kBlock<T> / T;
    const int64_t m = kRows == 1 ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / T;
    if (m >= a.M) return;   // rows that share a workgroup have a wave each, and no barrier
    const int tid = threadIdx.x % T;
    const int groups = a.C / 4;
    const int64_t base = m * groups;
    const float *gate = a.gate ? a.gate + m / a.gate_run * a.C : nullptr;
    const float *mod = a.modulation ? a.modulation + m / a.modulation_run * a.C : nullptr;
    const float inv_c = 1.0f / static_cast<float>(a.C);
    if constexpr (NV > 0) {
        floatx4 r[NV], y[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int i = tid + T * v;
            r[v] = y[v] = (floatx4){0, 0, 0, 0};
            if (i < groups) {
                r[v] = load4<RB>(a.residual, base + i);
                if (a.y) y[v] = load4<YB>(a.y, base + i);
            }
        }
        float inv = 1.0f;
        if (a.post_weight) {
            float ss = 0.0f;
#pragma unroll
            for (int v = 0; v < NV; ++v) ss += sum_sq(y[v]);
            inv = 1.0f / sqrtf(row_sum<T>(ss, part[0]) * inv_c + a.eps);
        }
        float ss = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int i = tid + T * v;
            if (a.y && i < groups) {
                r[v] = r[v] + update<YB>(a, y[v], inv, gate, i);
                store4<RB, true>(a.residual_out, base + i, r[v]);
            }
            ss += sum_sq(r[v]);
        }
        inv = 1.0f / sqrtf(row_sum<T>(ss, part[1]) * inv_c + a.eps);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int i = tid + T * v;
            if (i < groups) {
                floatx4 x = r[v] * inv * load4<0>(a.weight, i);
                if (mod) x = x * (1.0f + load4<0>(mod, i));
                store4<XB, false>(a.x, base + i, x);
            }
        }
    } else {
        float inv = 1.0f, ss = 0.0f;
        if (a.post_weight) {
            for (int i = tid; i < groups; i += T) ss += sum_sq(load4<YB>(a.y, base + i));
            inv = 1.0f / sqrtf(row_sum<T>(ss, part[0]) * inv_c + a.eps);
        }
        auto value = [&](int i) {
            floatx4 r = load4<RB>(a.residual, base + i);
            if (a.y) r = r + update<YB>(a, load4<YB>(a.y, base + i), inv, gate, i);
            return r;
        };
        ss = 0.0f;
        for (int i = tid; i < groups; i += T) ss += sum_sq(value(i));
        const float inv_r = 1.0f / sqrtf(row_sum<T>(ss, part[1]) * inv_c + a.eps);
        for (int i = tid; i < groups; i += T) {
            const floatx4 r = value(i);   // before residual_out, which may be the residual itself, gets it
            if (a.y) store4<RB, true>(a.residual_out, base + i, r);
            floatx4 x = r * inv_r * load4<0>(a.weight, i);
            if (mod) x = x * (1.0f + load4<0>(mod, i));
            store4<XB, false>(a.x, base + i, x);
        }
    }
}

template <int RB, int YB, int XB>
hipError_t launch(const NormArgs &a, hipStream_t s) {
#define Q4_NORM(T, NV)                                                                                       \
    hipLaunchKernelGGL((add_rmsnorm_kernel<RB, YB, XB, T, NV>),                                              \
                       dim3(static_cast<uint32_t>((a.M * T + kBlock<T> - 1) / kBlock<T>)), dim3(kBlock<T>), 0, s, a)
    // While all rows can be on the chip together (2048 threads a compute unit),
    // as many threads a row as have four elements each: two rows of 3072 take
    // 2.5 against 3.6 us with 256 threads, 512 rows 5.1 against 5.6, but 1024
    // rows 9.1 against 7.9; 2048 rows of 512 3.4 against 3.8 with a wave.
    // Past that, a wave a row as long as that holds it in few registers (6020
    // rows of 256 5.7 against 7.1, of 512 9.1 against 10.0, but of 1024 17.8
    // against 16.1), then 256 threads, and above 4096 elements 1024 of them
    // (2048 rows of 5120 32 us, 75 with 256 threads).
    auto fit = [&](int64_t threads) { return a.M * threads <= 2048 * 256; };
    if (a.C <= 256) Q4_NORM(64, 1);
    else if (a.C <= 512 && !fit(256)) Q4_NORM(64, 2);
    else if (a.C <= 1024) Q4_NORM(256, 1);
    else if (a.C <= 4096 && fit(1024)) Q4_NORM(1024, 1);
    else if (a.C <= 2048) Q4_NORM(256, 2);
    else if (a.C <= 3072) Q4_NORM(256, 3);
    else if (a.C <= 4096) Q4_NORM(256, 4);
    else if (a.C <= 8192) Q4_NORM(1024, 2);
    else if (a.C <= 12288) Q4_NORM(1024, 3);
    else if (a.C <= 16384) Q4_NORM(1024, 4);
    else Q4_NORM(1024, 0);
#undef Q4_NORM
    return hipGetLastError();
}

}  // namespace

hipError_t launch_add_rmsnorm(const NormArgs &a, int residual_dtype, int y_dtype, int x_dtype, hipStream_t s) {
    switch (residual_dtype * 4 + y_dtype * 2 + x_dtype) {
        case 0: return launch<0, 0, 0>(a, s);
        case 1: return launch<0, 0, 1>(a, s);
        case 2: return launch<0, 1, 0>(a, s);
        case 3: return launch<0, 1, 1>(a, s);
        case 4: return launch<1, 0, 0>(a, s);
        case 5: return launch<1, 0, 1>(a, s);
        case 6: return launch<1, 1, 0>(a, s);
        default: return launch<1, 1, 1>(a, s);
    }
}

}  // namespace q4
