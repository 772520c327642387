// Attention over the paged 8-bit cache (include/q4_decoder.h).
//
// The mathematics.  For a query row r and the tokens j it sees,
//     s_j = c * 2^eK * (q . k_j),   o = sum_j 2^s_j 2^eV v_j / sum_j 2^s_j
// with c = scale * log2(e), k_j and v_j the codes and eK, eV the exponents of
// token j's block.  The kernels work with t_j = s_j + eV, the exponent of
// token j's weight on its codes: with m at least about max_j t_j,
//     w_j = 2^(t_j - m),   o = sum_j w_j v_j / sum_j w_j 2^-eV,
// so the codes go into the matrix products as they are, and w, held to fp16,
// is exact to 2^-11 wherever it matters for the result, also where the blocks'
// scales differ widely.  m and the sums are fp32 and are carried over the
// tokens in one pass.  m is only raised when some t_j passes it by 8: w stays
// at most 2^8, within fp16, and most blocks need no rescaling.
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

constexpr float kLowest = -3.402823466e38f;
constexpr float kSlack = 8.0f;   // how far a score may pass m before m is raised

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
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (first + j >= lo && first + j < hi) m |= 0xFFu << (8 * j);
    return m;
}

// 0x80 in each byte that is not a number, and the word with those bytes zero.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ uint32_t without(uint32_t w, uint32_t nan) { return w & ~((nan >> 7) * 0xFFu); }

// Largest over the four lanes that hold one row (lane % 16).
__device__ __forceinline__ float row_max(float v) {
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float row_sum(float v) {
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// The blocks that a tile of rows reads, and their division over the splits of
// the launch: split i has blocks [first + i * chunk, first + (i + 1) * chunk).
struct Span {
    int first, last, chunk, splits;   // blocks [first, last), splits that have some
};

// p_first, p_last: positions of the tile's first and last row (p_last < 0:
// nothing is seen).  Tokens past the block table are not read: the rows that
// would see them give what is not a number (`past` below).
__device__ __forceinline__ Span span_of(const KvView &kv, int p_first, int p_last, int window, int chunk,
                                        int grid_splits) {
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
    s.chunk = chunk;
    if (grid_splits == 1 || static_cast<int64_t>(chunk) * grid_splits < n) s.chunk = (n + grid_splits - 1) / grid_splits;
    s.splits = (n + s.chunk - 1) / s.chunk;
    return s;
}

__device__ __forceinline__ bool past(const KvView &kv, int pos) { return pos >= 0 && pos / kKvBlock >= kv.table_width; }

// ------------------------------------------------------- few rows: decode
// A workgroup has 16 rows (of rows x heads of the group) of one sequence and
// kv head, and one chunk of its blocks; its four waves take every fourth block.
// Each lane's loads are its operand slices, so the cache goes from memory to
// registers and nowhere else.
constexpr int kWaves = 4;

template <int D>
struct Partial {
    static constexpr int kFloats = 16 * (D + 2);   // one tile's m[16], l[16], O[16][D]
};

template <int D>
__global__ __launch_bounds__(64 * kWaves) void attention_rows_kernel(AttentionArgs a, int chunk, int tiles) {
    constexpr int KQ = D / 32;   // k slices of the first product
    constexpr int DT = D / 16;   // 16-dimension tiles of the output
    __shared__ float part_m[kWaves][16], part_l[kWaves][16];
    __shared__ float part_o[kWaves][D * 16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 15, g4 = lane >> 4;
    const int b = blockIdx.z, head = blockIdx.y % a.kv.kv_heads;
    const KvSequence s = kv_sequence(a.kv, b);
    const int grid_tiles = gridDim.y / a.kv.kv_heads;
    const int64_t all_rows = static_cast<int64_t>(s.rows) * a.group;
    for (int64_t tile = blockIdx.y / a.kv.kv_heads; tile * 16 < all_rows; tile += grid_tiles) {
        const int64_t rr = tile * 16 + r;
        const bool live = rr < all_rows;
        const int t = static_cast<int>((live ? rr : all_rows - 1) / a.group);
        const int g = static_cast<int>((live ? rr : all_rows - 1) % a.group);
        const int pos = s.pos0 + t;
        const int t_first = static_cast<int>(tile * 16 / a.group);
        const int64_t r_last = tile * 16 + 15 < all_rows ? tile * 16 + 15 : all_rows - 1;
        const int p_first = s.pos0 + t_first, p_last = s.pos0 + static_cast<int>(r_last / a.group);
        // tiles past those that the launch was shaped for are not split: they
        // have no place in the workspace
        const Span sp = span_of(a.kv, p_first, p_last, a.window, chunk, tile < tiles ? gridDim.x : 1);
        const int split = blockIdx.x;
        if (split >= (sp.splits ? sp.splits : 1)) continue;   // uniform
        const int blk0 = sp.first + split * sp.chunk;
        const int blk1 = blk0 + sp.chunk < sp.last ? blk0 + sp.chunk : sp.last;
        // the tokens that all rows and that any row of the tile see
        const int lo = a.window ? pos - a.window + 1 : 0;
        const int all_lo = a.window ? p_last - a.window + 1 : 0, any_lo = a.window ? p_first - a.window + 1 : 0;
        const int64_t out_row = s.row0 + t;
        const int64_t out_at = (out_row * a.q_heads + head * a.group + g) * D;

        bf16x8 q[KQ];
#pragma unroll
        for (int i = 0; i < KQ; ++i)
            q[i] = reinterpret_cast<const bf16x8 *>(a.q + out_at + 64 * (i / 2) + 16 * g4 + 8 * (i % 2))[0];

        float m = kLowest, l = 0.0f;
        floatx4 o[DT];
#pragma unroll
        for (int i = 0; i < DT; ++i) o[i] = (floatx4){0, 0, 0, 0};

        for (int blk = blk0 + wave; blk < blk1; blk += kWaves) {
            const int id = __builtin_amdgcn_readfirstlane(kv_block_id(a.kv, b, blk));
            const int64_t plane = (static_cast<int64_t>(id < 0 ? 0 : id) * a.kv.kv_heads + head) * 2;
            const u32x4 *src = reinterpret_cast<const u32x4 *>(a.kv.data + plane * (kKvBlock * D)) + lane;
            u32x4 kc[KQ], vc[KQ];
#pragma unroll
            for (int i = 0; i < KQ; ++i) kc[i] = src[64 * i];
#pragma unroll
            for (int i = 0; i < KQ; ++i) vc[i] = src[64 * (KQ + i)];
            const float ek = static_cast<float>(a.kv.exps[plane]), ev = static_cast<float>(a.kv.exps[plane + 1]);
            const float c = id < 0 ? __builtin_nanf("") : a.scale_log2 * __builtin_amdgcn_exp2f(ek);
            floatx4 st[2];
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
                st[tt] = (floatx4){0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < KQ; ++i) {
                    const u32x4 w = kc[tt * (KQ / 2) + i / 2];
                    const bf16x8 kf = i % 2 ? codes_bf16(w.z, w.w) : codes_bf16(w.x, w.y);
                    st[tt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, q[i], st[tt], 0, 0, 0);
                }
            }
            float w[8];   // scores, then weights, of tokens 4 g4 + i and 16 + 4 g4 + i
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = fmaf(st[i / 4][i % 4], c, ev);
            const int start = blk * kKvBlock;
            const bool whole = start >= all_lo && start + kKvBlock - 1 <= p_first;   // all rows see all tokens
            uint32_t seen = 0xFF;
            if (!whole) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int j = start + i / 4 * 16 + 4 * g4 + i % 4;
                    if (j < lo || j > pos) {
                        w[i] = -__builtin_inff();
                        seen &= ~(1u << i);
                    }
                }
            }
            float top = w[0];
#pragma unroll
            for (int i = 1; i < 8; ++i) top = fmaxf(top, w[i]);
            if (__any(top > m + kSlack)) {
                const float raised = fmaxf(m, row_max(top));
                const float f = __builtin_amdgcn_exp2f(m - raised);
                m = raised;
                l *= f;
#pragma unroll
                for (int i = 0; i < DT; ++i) o[i] = o[i] * f;
            }
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                w[i] = __builtin_amdgcn_exp2f(w[i] - m);
                sum += w[i];
            }
            l = fmaf(sum, __builtin_amdgcn_exp2f(-ev), l);
            const halfx8 wf = weights_f16(w);
            if (!whole) {
                // bytes that no row of the tile sees may hold anything
                const uint32_t in0 = bytes_in(start + 4 * g4, any_lo, p_last + 1);
                const uint32_t in1 = bytes_in(start + 16 + 4 * g4, any_lo, p_last + 1);
                uint32_t bad = 0;
#pragma unroll
                for (int i = 0; i < KQ; ++i) {
                    vc[i].x &= in0;
                    vc[i].y &= in1;
                    vc[i].z &= in0;
                    vc[i].w &= in1;
                    bad |= nan_bytes(vc[i].x) | nan_bytes(vc[i].y) | nan_bytes(vc[i].z) | nan_bytes(vc[i].w);
                }
                if (__any(bad != 0)) {
                    // a value that is not a number reaches the rows that see
                    // its token, and no others (0 * NaN is NaN): count such
                    // tokens for each output and leave them out of the product
                    float one[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) one[i] = (seen >> i) & 1u ? 1.0f : 0.0f;
                    const halfx8 sf = weights_f16(one);
#pragma unroll
                    for (int i = 0; i < DT; ++i) {
                        const int at = i % 2 * 2;
                        const uint32_t n0 = nan_bytes(vc[i / 2][at]), n1 = nan_bytes(vc[i / 2][at + 1]);
                        floatx4 hits = {0, 0, 0, 0};
                        // 0x38 is 1.0
                        hits = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes_f16((n0 >> 7) * 0x38u, (n1 >> 7) * 0x38u),
                                                                      sf, hits, 0, 0, 0);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (hits[j] > 0.0f) o[i][j] = __builtin_nanf("");
                        vc[i / 2][at] = without(vc[i / 2][at], n0);
                        vc[i / 2][at + 1] = without(vc[i / 2][at + 1], n1);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < DT; ++i) {
                const u32x4 v = vc[i / 2];
                const halfx8 vf = i % 2 ? codes_f16(v.z, v.w) : codes_f16(v.x, v.y);
                o[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, wf, o[i], 0, 0, 0);
            }
        }
        l = row_sum(l);
        // join the four waves
        __syncthreads();   // the previous tile's sums have been read
        if (g4 == 0) {
            part_m[wave][r] = m;
            part_l[wave][r] = l;
        }
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) part_o[wave][(16 * i + 4 * g4 + j) * 16 + r] = o[i][j];
        __syncthreads();
        float top = part_m[0][r];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) top = fmaxf(top, part_m[w][r]);
        float f[kWaves], total = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            f[w] = __builtin_amdgcn_exp2f(part_m[w][r] - top);
            total += f[w] * part_l[w][r];
        }
        // thread: row r, dimensions tid / 16 + 16 i
        const int d0 = threadIdx.x >> 4;
        const bool final_out = sp.splits <= 1;
        float *ws = a.workspace +
                    (((static_cast<int64_t>(b) * a.kv.kv_heads + head) * tiles + tile) * gridDim.x + split) * Partial<D>::kFloats;
        const float inv = past(a.kv, pos) ? __builtin_nanf("") : total == 0.0f ? 0.0f : 1.0f / total;
#pragma unroll
        for (int i = 0; i < DT; ++i) {
            const int d = d0 + 16 * i;
            float acc = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) acc += f[w] * part_o[w][d * 16 + r];
            if (!final_out)
                ws[32 + r * D + d] = acc;
            else if (live) {
                acc *= inv;
                if (a.out_bf16) static_cast<__bf16 *>(a.out)[out_at + d] = static_cast<__bf16>(acc);
                else static_cast<float *>(a.out)[out_at + d] = acc;
            }
        }
        if (!final_out && threadIdx.x < 16) {
            ws[r] = top;
            ws[16 + r] = total;
        }
    }
}

// Joins the splits of a tile: one workgroup a row.
template <int D>
__global__ __launch_bounds__(256) void attention_join_kernel(AttentionArgs a, int chunk, int tiles, int splits) {
    constexpr int LANES = D / 4;            // threads with four dimensions each
    constexpr int PARTS = 256 / LANES;      // splits summed side by side
    __shared__ floatx4 part[PARTS][LANES];
    __shared__ float part_l[PARTS];
    const int b = blockIdx.z, head = blockIdx.y % a.kv.kv_heads;
    const KvSequence s = kv_sequence(a.kv, b);
    const int64_t all_rows = static_cast<int64_t>(s.rows) * a.group;
    const int64_t tile = blockIdx.y / a.kv.kv_heads;
    const int r = blockIdx.x;
    const int64_t rr = tile * 16 + r;
    if (rr >= all_rows) return;
    const int64_t r_last = tile * 16 + 15 < all_rows ? tile * 16 + 15 : all_rows - 1;
    const Span sp = span_of(a.kv, s.pos0 + static_cast<int>(tile * 16 / a.group), s.pos0 + static_cast<int>(r_last / a.group),
                            a.window, chunk, splits);
    if (sp.splits <= 1) return;
    const float *ws = a.workspace +
                      ((static_cast<int64_t>(b) * a.kv.kv_heads + head) * tiles + tile) * splits * Partial<D>::kFloats;
    float top = kLowest;
    for (int i = 0; i < sp.splits; ++i) top = fmaxf(top, ws[static_cast<int64_t>(i) * Partial<D>::kFloats + r]);
    const int x = threadIdx.x % LANES, y = threadIdx.x / LANES;
    floatx4 acc = {0, 0, 0, 0};
    float total = 0.0f;
    for (int i = y; i < sp.splits; i += PARTS) {
        const float *p = ws + static_cast<int64_t>(i) * Partial<D>::kFloats;
        const float f = __builtin_amdgcn_exp2f(p[r] - top);
        total += f * p[16 + r];
        acc = acc + reinterpret_cast<const floatx4 *>(p + 32 + r * D)[x] * f;
    }
    part[y][x] = acc;
    if (x == 0) part_l[y] = total;
    __syncthreads();
    if (y != 0) return;
#pragma unroll
    for (int i = 1; i < PARTS; ++i) {
        acc = acc + part[i][x];
        total += part_l[i];
    }
    const int t = static_cast<int>(rr / a.group), g = static_cast<int>(rr % a.group);
    acc = acc * (past(a.kv, s.pos0 + t) ? __builtin_nanf("") : total == 0.0f ? 0.0f : 1.0f / total);
    const int64_t at = ((static_cast<int64_t>(s.row0 + t)) * a.q_heads + head * a.group + g) * D / 4 + x;
    if (a.out_bf16)
        reinterpret_cast<bf16x4 *>(a.out)[at] = __builtin_convertvector(acc, bf16x4);
    else
        reinterpret_cast<floatx4 *>(a.out)[at] = acc;
}

// The launch of the row kernel: 16-row tiles of a sequence, and how its
// blocks are split.
struct RowsPlan {
    int tiles;          // tiles of the longest sequence
    int chunk, splits;
};

RowsPlan rows_plan(const AttentionArgs &a) {
    RowsPlan p;
    p.tiles = static_cast<int>((static_cast<int64_t>(a.max_rows) * a.group + 15) / 16);
    const int64_t blocks = (static_cast<int64_t>(a.max_length) + kKvBlock - 1) / kKvBlock;
    const int64_t work = static_cast<int64_t>(p.tiles) * a.kv.kv_heads * a.kv.batch;
    // about four workgroups a compute unit, each with a block for every wave
    int64_t splits = (1024 + work - 1) / work;
    int64_t chunk = (blocks + splits - 1) / splits;
    if (chunk < kWaves) chunk = kWaves;
    p.chunk = static_cast<int>(chunk);
    p.splits = static_cast<int>((blocks + chunk - 1) / chunk);
    return p;
}

template <int D>
hipError_t launch_rows(const AttentionArgs &a, hipStream_t s) {
    const RowsPlan p = rows_plan(a);
    int grid_tiles = p.tiles;
    if (static_cast<int64_t>(grid_tiles) * a.kv.kv_heads > 65535) grid_tiles = 65535 / a.kv.kv_heads;
    // the tiles of a launch with splits fit its workspace: such a launch has
    // fewer than 1024 tiles
    const dim3 grid(p.splits, grid_tiles * a.kv.kv_heads, a.kv.batch);
    hipLaunchKernelGGL((attention_rows_kernel<D>), grid, dim3(64 * kWaves), 0, s, a, p.chunk, p.tiles);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    hipLaunchKernelGGL((attention_join_kernel<D>), dim3(16, p.tiles * a.kv.kv_heads, a.kv.batch), dim3(256), 0, s, a,
                       p.chunk, p.tiles, p.splits);
    return hipGetLastError();
}

}  // namespace

size_t attention_workspace(const AttentionArgs &a, int head_dim) {
    const RowsPlan p = rows_plan(a);
    if (p.splits == 1) return 0;
    return static_cast<size_t>(p.tiles) * a.kv.kv_heads * a.kv.batch * p.splits * 16 * (head_dim + 2) * sizeof(float);
}

hipError_t launch_kv_attention(const AttentionArgs &a, int head_dim, hipStream_t s) {
    return head_dim == 128 ? launch_rows<128>(a, s) : launch_rows<64>(a, s);
}

}  // namespace q4
