// The residual step between two blocks (include/q4_decoder.h): norm of the
// block's output, gate, residual scale, residual add, norm for the next block
// and its modulation, in one pass over the rows.
//
// A workgroup of 256 threads has one row; a thread holds NV groups of four
// consecutive elements of it in registers from the first sum to the last
// store, so that y and the residual are read once.  Rows longer than
// 256 * 4 * kMaxGroups are read again for each sum instead.

#include "q4_decoder_internal.h"

namespace q4 {
namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;

template <int BF16>
__device__ __forceinline__ floatx4 load4(const void *p, int64_t i) {   // i: group of four elements
    if constexpr (BF16)
        return __builtin_convertvector(reinterpret_cast<const bf16x4 *>(p)[i], floatx4);
    else
        return reinterpret_cast<const floatx4 *>(p)[i];
}

template <int BF16>
__device__ __forceinline__ void store4(void *p, int64_t i, floatx4 v) {
    if constexpr (BF16)
        reinterpret_cast<bf16x4 *>(p)[i] = __builtin_convertvector(v, bf16x4);
    else
        reinterpret_cast<floatx4 *>(p)[i] = v;
}

__device__ __forceinline__ float sum_sq(floatx4 v) { return v.x * v.x + v.y * v.y + v.z * v.z + v.w * v.w; }

__device__ __forceinline__ float block_sum(float v, float *part) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    return part[0] + part[1] + part[2] + part[3];
}

// y's group i, normed (where post_weight is given) and gated
template <int YB>
__device__ __forceinline__ floatx4 update(const NormArgs &a, floatx4 y, float inv, const float *gate, int i) {
    if (a.post_weight) y = y * inv * load4<0>(a.post_weight, i);
    if (gate) y = y * load4<0>(gate, i);
    return y * a.scale;
}

template <int RB, int YB, int XB, int NV>
__global__ __launch_bounds__(kThreads) void add_rmsnorm_kernel(NormArgs a) {
    __shared__ float part[2][4];
    const int64_t m = blockIdx.x;
    const int groups = a.C / 4;
    const int64_t base = m * groups;
    const float *gate = a.gate ? a.gate + m / a.gate_run * a.C : nullptr;
    const float *mod = a.modulation ? a.modulation + m / a.modulation_run * a.C : nullptr;
    const float inv_c = 1.0f / static_cast<float>(a.C);
    if constexpr (NV > 0) {
        floatx4 r[NV], y[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int i = threadIdx.x + kThreads * v;
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
            inv = 1.0f / sqrtf(block_sum(ss, part[0]) * inv_c + a.eps);
        }
        float ss = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int i = threadIdx.x + kThreads * v;
            if (a.y && i < groups) {
                r[v] = r[v] + update<YB>(a, y[v], inv, gate, i);
                store4<RB>(a.residual_out, base + i, r[v]);
            }
            ss += sum_sq(r[v]);
        }
        inv = 1.0f / sqrtf(block_sum(ss, part[1]) * inv_c + a.eps);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int i = threadIdx.x + kThreads * v;
            if (i < groups) {
                floatx4 x = r[v] * inv * load4<0>(a.weight, i);
                if (mod) x = x * (1.0f + load4<0>(mod, i));
                store4<XB>(a.x, base + i, x);
            }
        }
    } else {
        float inv = 1.0f, ss = 0.0f;
        if (a.post_weight) {
            for (int i = threadIdx.x; i < groups; i += kThreads) ss += sum_sq(load4<YB>(a.y, base + i));
            inv = 1.0f / sqrtf(block_sum(ss, part[0]) * inv_c + a.eps);
        }
        auto value = [&](int i) {
            floatx4 r = load4<RB>(a.residual, base + i);
            if (a.y) r = r + update<YB>(a, load4<YB>(a.y, base + i), inv, gate, i);
            return r;
        };
        ss = 0.0f;
        for (int i = threadIdx.x; i < groups; i += kThreads) ss += sum_sq(value(i));
        const float inv_r = 1.0f / sqrtf(block_sum(ss, part[1]) * inv_c + a.eps);
        for (int i = threadIdx.x; i < groups; i += kThreads) {
            const floatx4 r = value(i);   // before residual_out, which may be the residual itself, gets it
            if (a.y) store4<RB>(a.residual_out, base + i, r);
            floatx4 x = r * inv_r * load4<0>(a.weight, i);
            if (mod) x = x * (1.0f + load4<0>(mod, i));
            store4<XB>(a.x, base + i, x);
        }
    }
}

template <int RB, int YB, int XB>
hipError_t launch(const NormArgs &a, hipStream_t s) {
    const dim3 grid(static_cast<uint32_t>(a.M));
    const int nv = (a.C / 4 + kThreads - 1) / kThreads;
#define Q4_NORM(NV) hipLaunchKernelGGL((add_rmsnorm_kernel<RB, YB, XB, NV>), grid, dim3(kThreads), 0, s, a)
    if (nv <= 1) Q4_NORM(1);
    else if (nv <= 2) Q4_NORM(2);
    else if (nv <= 3) Q4_NORM(3);
    else if (nv <= 4) Q4_NORM(4);
    else if (nv <= 8) Q4_NORM(8);
    else Q4_NORM(0);
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
