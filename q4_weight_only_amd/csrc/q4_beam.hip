// Beam search: the best continuations of a group's beams, and the tokens of
// those that were kept (include/q4_search.h).
//
// The mathematics.  A candidate's score is s = score + (z - lse), and of equal
// ones the lower (beam, token) precedes: a total order.  Cut each row into
// segments of 32 consecutive tokens.  The n first candidates lie in the n
// segments whose own first candidates precede the others', since each such
// candidate stands in front of everything in the segments after its own.  So one
// pass over the logits leaves the largest of each segment, and what it takes for
// lse, and the rest works on a 32nd of the data.
//
// lse in 64 bits: a sum over 131072 tokens in 32 bits is off by some 1e-7, and
// scores of two beams that are nearer than that are met in practice.

#include "q4_search_internal.h"

namespace q4 {
namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef float floatx4_row __attribute__((ext_vector_type(4), aligned(4)));   // rows start on 4 bytes only
typedef int32_t i32x4_row __attribute__((ext_vector_type(4), aligned(4)));

constexpr float kNone = -__builtin_inff();

// What beam_scan_kernel leaves in the workspace for beam_pick_kernel: for each
// wave's part of a row its largest logit m and sum e^(z - m), and the segments'
// largest logits.
struct Scan {
    double *sum;      // [rows][parts]
    float *top;       // [rows][parts]
    float *segment;   // [rows][segments]
    int32_t parts, segments, loads;
};

// Loads of four tokens that a lane has: more of them mean fewer parts to join,
// fewer more waves to read with.
int loads_of(int64_t rows, int64_t V) {
    const int64_t waves = rows * ((V + 255) / 256);
    return waves >= 32768 ? 8 : waves >= 8192 ? 4 : waves >= 4096 ? 2 : 1;
}

Scan scan_of(void *workspace, int64_t rows, int64_t V) {
    Scan s;
    s.loads = loads_of(rows, V);
    s.parts = static_cast<int32_t>((V + 256 * s.loads - 1) / (256 * s.loads));
    s.segments = static_cast<int32_t>((V + kBeamSegment - 1) / kBeamSegment);
    s.sum = static_cast<double *>(workspace);
    s.top = reinterpret_cast<float *>(s.sum + rows * s.parts);
    s.segment = s.top + rows * s.parts;
    return s;
}

// The larger of the lane's and another lane's.
template <int CTRL>
__device__ __forceinline__ float max_dpp(float v) {
    const int w = __float_as_int(v);
    return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(w, w, CTRL, 0xF, 0xF, false)));
}

// Largest of each 8 lanes, in all of them.
__device__ __forceinline__ float max_of_8(float v) {
    v = max_dpp<0xB1>(v);    // lane ^ 1
    v = max_dpp<0x4E>(v);    // lane ^ 2
    return max_dpp<0x141>(v);   // 7 - lane, within 8
}

// e^x for x <= 0 (a difference of two fp32 values), within 3e-10 of itself:
// 2^n times a Taylor sum of degree 8 on [-1/2, 1/2] ln 2.  Below -80 it is 0, which no
// sum of 2^24 terms with a largest one of 1 notices; what is not a number stays it.
__device__ __forceinline__ double exp64(double x) {
    const double y = x * 1.4426950408889634074;
    const double n = __builtin_rint(y);
    const double f = (y - n) * 0.69314718055994530942;
    double p = 1.0 / 40320;
    p = fma(p, f, 1.0 / 5040);
    p = fma(p, f, 1.0 / 720);
    p = fma(p, f, 1.0 / 120);
    p = fma(p, f, 1.0 / 24);
    p = fma(p, f, 1.0 / 6);
    p = fma(p, f, 0.5);
    p = fma(p, f, 1.0);
    p = fma(p, f, 1.0);
    return x < -80.0 ? 0.0 : __builtin_ldexp(p, x >= -80.0 ? static_cast<int>(n) : 0);
}

// A wave has 256 * J consecutive tokens of a row, loads all of them, and waits
// for nobody.
template <int J>
__global__ __launch_bounds__(256) void beam_scan_kernel(BeamArgs a, Scan out) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t row = blockIdx.y;
    const int part = blockIdx.x * 4 + wave;
    if (part >= out.parts) return;
    if (a.finished && a.finished[row]) return;   // nothing of it is read
    const int base = part * 256 * J;
    const float *src = a.logits + row * a.V;
    floatx4 z[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int t = base + 256 * j + 4 * lane;
        if (t + 4 <= a.V) {
            z[j] = *reinterpret_cast<const floatx4_row *>(src + t);
        } else {
            z[j] = (floatx4){kNone, kNone, kNone, kNone};
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (t + i < a.V) z[j][i] = src[t + i];
        }
    }
    float top = kNone, seg[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        seg[j] = max_of_8(fmaxf(fmaxf(z[j][0], z[j][1]), fmaxf(z[j][2], z[j][3])));
        top = fmaxf(top, seg[j]);
    }
    top = fmaxf(top, __shfl_xor(top, 8));
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    const double m = top == kNone ? 0.0 : top;   // all -inf: the sum is 0
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < J; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) sum += exp64(z[j][i] - m);
    }
#pragma unroll
    for (int i = 1; i < 64; i *= 2) sum += __shfl_xor(sum, i);
    if (lane == 0) {
        out.sum[row * out.parts + part] = sum;
        out.top[row * out.parts + part] = top;
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int s = (base + 256 * j) / kBeamSegment + lane / 8;
        if (lane % 8 == 0 && s < out.segments) out.segment[row * out.segments + s] = seg[j];
    }
}

// A place in the order: s, then id.  What is no candidate has kNone.
struct Place {
    double s;
    int32_t id;
};
__device__ __forceinline__ bool precedes(const Place &x, const Place &y) { return x.s > y.s || (x.s == y.s && x.id < y.id); }

// Doubles in the order of unsigned numbers.
__device__ __forceinline__ uint64_t ordered(double s) {
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(s));
    return b >> 63 ? ~b : b | (uint64_t(1) << 63);
}

constexpr int kPickThreads = 1024;
constexpr int kSlots = 256;       // the items of four threads are a slot
constexpr int kListed = 512;     // segments that may be listed before they are cut down to `keep`

// A workgroup has one group.  The n-th of the first items of its 256 slots is a
// bound that at least n items do not stand behind, and hardly more where they are spread
// evenly; those are listed and the n first of them found by counting, for each, the
// ones in front.  Where too many are in front of the bound (they lie together,
// or are equal), the n-th item itself is found, bit by bit.
__global__ __launch_bounds__(kPickThreads) void beam_pick_kernel(BeamArgs a, Scan in) {
    __shared__ double base[kMaxBeams], lse[kMaxBeams];
    __shared__ int32_t ended[kMaxBeams];
    __shared__ double slot_s[kSlots];
    __shared__ int32_t slot_id[kSlots];
    __shared__ double list_s[kListed];
    __shared__ int32_t list_id[kListed];
    __shared__ int32_t segment_id[kMaxKeep];
    __shared__ double bound_s;
    __shared__ int32_t bound_id, listed, counted[2];
    extern __shared__ __align__(16) uint8_t dynamic[];   // keep * 32 elements: s, then ids
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int n = a.keep, group = blockIdx.x;
    const int segments = in.segments, items = a.beams * segments;
    double *element_s = reinterpret_cast<double *>(dynamic);
    int32_t *element_id = reinterpret_cast<int32_t *>(element_s + n * kBeamSegment);

    for (int b = wave; b < a.beams; b += kPickThreads / 64) {
        const int64_t row = static_cast<int64_t>(group) * a.beams + b;
        const bool done = a.finished && a.finished[row];
        double l = 0.0;
        if (!done) {
            const float *tops = in.top + row * in.parts;
            const double *sums = in.sum + row * in.parts;
            float top = kNone;
            for (int i = lane; i < in.parts; i += 64) top = fmaxf(top, tops[i]);
#pragma unroll
            for (int i = 1; i < 64; i *= 2) top = fmaxf(top, __shfl_xor(top, i));
            double sum = 0.0;
            for (int i = lane; i < in.parts; i += 64)   // a part without a logit has 0, or what is not a number
                sum += tops[i] == kNone ? sums[i] : sums[i] * exp64(static_cast<double>(tops[i]) - top);
#pragma unroll
            for (int i = 1; i < 64; i *= 2) sum += __shfl_xor(sum, i);
            l = top + log(sum);
        }
        if (lane == 0) {
            base[b] = a.scores[row] + 0.0;
            lse[b] = l;
            ended[b] = done;
        }
    }
    if (tid == 0) listed = 0;
    __syncthreads();

    const auto score = [&](int b, float z) {
        const double s = base[b] + (z - lse[b]) + 0.0;   // no -0, which would be equal to 0 and ordered before it
        return __builtin_isfinite(s) ? s : static_cast<double>(kNone);
    };
    // every item of the thread: its place.  An ended beam has one candidate, in its first item.
    const float *segment = in.segment + static_cast<int64_t>(group) * items;
    const auto each_item = [&](auto f) {
        int b = 0, at = tid;
        for (int id = tid; id < items; id += kPickThreads, at += kPickThreads) {
            while (at >= segments) {
                at -= segments;
                ++b;
            }
            Place p;
            p.id = id;
            if (ended[b]) p.s = at == 0 && __builtin_isfinite(base[b]) ? base[b] : static_cast<double>(kNone);
            else p.s = score(b, segment[id]);
            f(p);
        }
    };
    Place best = {kNone, 0x7fffffff};
    each_item([&](const Place &p) {
        if (precedes(p, best)) best = p;
    });
#pragma unroll
    for (int i = 1; i < 4; i *= 2) {
        const Place other = {__shfl_xor(best.s, i), __shfl_xor(best.id, i)};
        if (precedes(other, best)) best = other;
    }
    if (tid % 4 == 0) {
        slot_s[tid / 4] = best.s;
        slot_id[tid / 4] = best.id;
    }
    __syncthreads();
    {   // the n-th slot (n <= 128): each of its four threads compares with a quarter
        const int mine = tid / 4;
        int front = 0;
#pragma unroll 8
        for (int i = 0; i < kSlots / 4; ++i) {
            const int other = i * 4 + tid % 4;
            const Place p = {slot_s[other], slot_id[other]};
            front += precedes(p, best) || (p.s == best.s && p.id == best.id && other < mine);   // empty slots are alike
        }
        front += __shfl_xor(front, 1);
        front += __shfl_xor(front, 2);
        if (tid % 4 == 0 && front == n - 1) {
            bound_s = best.s;
            bound_id = best.id;
        }
    }
    __syncthreads();
    Place bound = {bound_s, bound_id};
    const auto list_items = [&] {
        each_item([&](const Place &p) {
            if (p.s == kNone || precedes(bound, p)) return;
            const int at = atomicAdd(&listed, 1);   // their order does not matter: they are counted below
            if (at < kListed) {
                list_s[at] = p.s;
                list_id[at] = p.id;
            }
        });
    };
    list_items();
    __syncthreads();
    if (listed > kListed) {   // the same for the workgroup
        const auto count = [&](auto f) {   // of items; the counters take turns
            if (tid < 2) counted[tid] = 0;
            __syncthreads();
            int c = 0;
            each_item([&](const Place &p) { c += p.s != kNone && f(p); });
#pragma unroll
            for (int i = 1; i < 64; i *= 2) c += __shfl_xor(c, i);
            if (lane == 0) atomicAdd(&counted[0], c);
            __syncthreads();
            const int total = counted[0];
            __syncthreads();
            return total;
        };
        uint64_t key = 0;
        for (int bit = 63; bit >= 0; --bit) {
            const uint64_t higher = key | uint64_t(1) << bit;
            if (count([&](const Place &p) { return ordered(p.s) >= higher; }) >= n) key = higher;
        }
        // of those that are equal to it, the first ones
        const int want = n - count([&](const Place &p) { return ordered(p.s) > key; });
        int32_t last = 0;   // the largest id for which fewer than `want` lie below it
        for (int bit = 25; bit >= 0; --bit) {
            const int32_t higher = last | 1 << bit;
            if (count([&](const Place &p) { return ordered(p.s) == key && p.id < higher; }) < want) last = higher;
        }
        bound.s = __longlong_as_double(static_cast<long long>(key >> 63 ? key & ~(uint64_t(1) << 63) : ~key));
        bound.id = last;
        if (tid == 0) listed = 0;
        __syncthreads();
        list_items();
        __syncthreads();
    }
    const int found = listed;   // at most kListed now
    const int taken = found < n ? found : n;
    __syncthreads();
    if (tid < found) {
        const Place me = {list_s[tid], list_id[tid]};
        int front = 0;
        for (int i = 0; i < found; ++i) front += precedes(Place{list_s[i], list_id[i]}, me);
        if (front < n) segment_id[front] = me.id;
        if (front == taken - 1) bound_s = me.s;   // with n segments, n elements have at least this
    }
    if (tid == 0) listed = 0;
    __syncthreads();
    const double least = taken == n ? bound_s : static_cast<double>(kNone);
    for (int i = tid; i < taken * kBeamSegment; i += kPickThreads) {
        const int id = segment_id[i / kBeamSegment], b = id / segments, token = (id - b * segments) * kBeamSegment + i % kBeamSegment;
        double s = kNone;
        int32_t at = token;
        if (ended[b]) {
            if (i % kBeamSegment == 0) s = base[b];
            at = 0;
        } else if (token < a.V) {
            s = score(b, a.logits[(static_cast<int64_t>(group) * a.beams + b) * a.V + token]);
        }
        if (s == kNone || s < least) continue;
        const int place = atomicAdd(&listed, 1);
        element_s[place] = s;
        element_id[place] = b << 24 | at;
    }
    __syncthreads();
    const int elements = listed;
    const int64_t out = static_cast<int64_t>(group) * n;
    for (int j = tid; j < elements; j += kPickThreads) {
        const Place me = {element_s[j], element_id[j]};
        int front = 0;
        for (int i = 0; i < elements; ++i) front += precedes(Place{element_s[i], element_id[i]}, me);
        if (front >= n) continue;
        const int b = me.id >> 24;
        a.parents[out + front] = group * a.beams + b;
        a.tokens[out + front] = ended[b] ? a.pad : me.id & 0xFFFFFF;
        a.out_scores[out + front] = static_cast<float>(me.s);
    }
    for (int j = elements + tid; j < n; j += kPickThreads) {
        a.parents[out + j] = -1;
        a.tokens[out + j] = -1;
        a.out_scores[out + j] = kNone;
    }
}

// A workgroup has 1024 tokens of one new sequence.
constexpr int kAdvanceTokens = 1024;

__global__ __launch_bounds__(256) void beam_advance_kernel(AdvanceArgs a) {
    const int64_t row = blockIdx.y + static_cast<int64_t>(blockIdx.z) * 65535;
    if (row >= a.n_out) return;
    const int32_t parent = a.parents[row], token = a.tokens[row];
    const bool live = parent >= 0 && parent < a.rows;
    int32_t was = live ? a.lengths[parent] : 0;
    was = was < 0 ? 0 : was > a.width ? a.width : was;
    const bool done = !live || (a.finished && a.finished[parent]);
    const bool adds = !done && was < a.width;
    const int32_t *src = a.sequences + (live ? parent : 0) * static_cast<int64_t>(a.width);
    int32_t *dst = a.out_sequences + row * a.width;
    const int t = blockIdx.x * kAdvanceTokens + 4 * threadIdx.x;
    const auto value = [&](int i, int32_t copied) { return i < was ? copied : adds && i == was ? token : a.pad; };
    if (t + 4 <= a.width) {
        i32x4_row v = {a.pad, a.pad, a.pad, a.pad};
        if (t < was) v = *reinterpret_cast<const i32x4_row *>(src + t);   // (past `was` the row may hold anything)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = value(t + i, v[i]);
        *reinterpret_cast<i32x4_row *>(dst + t) = v;
    } else {
        for (int i = t; i < a.width && i < t + 4; ++i) dst[i] = value(i, i < was ? src[i] : 0);
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        a.out_lengths[row] = was + adds;
        a.out_finished[row] = done || !adds || (a.eos >= 0 && token == a.eos);
    }
}

}  // namespace

size_t beam_workspace(int64_t rows, int64_t V) {
    const Scan s = scan_of(nullptr, rows, V);
    return (static_cast<size_t>(rows) * (static_cast<size_t>(s.parts) * 12 + static_cast<size_t>(s.segments) * 4) + 15) / 16 * 16;
}

hipError_t launch_beam_select(const BeamArgs &a, hipStream_t s) {
    const int64_t rows = static_cast<int64_t>(a.groups) * a.beams;
    const Scan scan = scan_of(a.workspace, rows, a.V);
    const dim3 grid((scan.parts + 3) / 4, static_cast<uint32_t>(rows));
    switch (scan.loads) {
        case 1: hipLaunchKernelGGL((beam_scan_kernel<1>), grid, dim3(256), 0, s, a, scan); break;
        case 2: hipLaunchKernelGGL((beam_scan_kernel<2>), grid, dim3(256), 0, s, a, scan); break;
        case 4: hipLaunchKernelGGL((beam_scan_kernel<4>), grid, dim3(256), 0, s, a, scan); break;
        default: hipLaunchKernelGGL((beam_scan_kernel<8>), grid, dim3(256), 0, s, a, scan); break;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const uint32_t lds = static_cast<uint32_t>(a.keep) * kBeamSegment * 12;   // at most 48 KB
    hipLaunchKernelGGL(beam_pick_kernel, dim3(a.groups), dim3(kPickThreads), lds, s, a, scan);
    return hipGetLastError();
}

hipError_t launch_beam_advance(const AdvanceArgs &a, hipStream_t s) {
    const uint32_t y = a.n_out < 65535 ? a.n_out : 65535, z = (static_cast<uint32_t>(a.n_out) + 65534) / 65535;
    hipLaunchKernelGGL(beam_advance_kernel, dim3((a.width + kAdvanceTokens - 1) / kAdvanceTokens, y, z), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace q4
