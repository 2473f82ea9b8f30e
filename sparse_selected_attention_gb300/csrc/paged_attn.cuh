// What the two kernels of qsa_paged_attn share: paged_attn.cu takes rows one by
// one, paged_group.cu rows of q that read one sequence together.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include "check.cuh"
#include "qsa_internal.h"
#include "tc_common.cuh"

namespace qsa {
namespace {

constexpr float LN2 = 0.6931471805599453f;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float SLACK = 8.0f;   // weights stay below 2^8 of the running maximum's

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ __half2 u2h(uint32_t u) { return *reinterpret_cast<__half2 *>(&u); }

// Two scales with an infinite or NaN one replaced by 0.
__device__ __forceinline__ uint32_t finite2(uint32_t x) { return x & ~__vcmpgeu2(x & 0x7FFF7FFFu, 0x7C007C00u); }

// floor(log2) of the largest finite |scale| of a cell; of a cell whose scales are
// 0, below any other's, so that what adds nothing to the values never is their
// maximum.
constexpr int NO_SCALE = -25;
__device__ __forceinline__ int scale_exponent(uint2 sc) {
    auto largest = [](uint32_t x, uint32_t y) {
        const uint32_t m = __vmaxu2(x & 0x7FFF7FFFu, y & 0x7FFF7FFFu);
        return max(m & 0xFFFFu, m >> 16);
    };
    uint32_t m = largest(sc.x, sc.y);
    if (m >= 0x7C00u) m = largest(finite2(sc.x), finite2(sc.y));
    return max((int)(__float_as_uint(__half2float(__ushort_as_half((unsigned short)m))) >> 23) - 127, NO_SCALE);
}

// The row of q (or, of a group, its first and the number of them) that starts in
// a CTA's share and spans n CTAs of its KV head; row -1: none.
struct Part {
    int row, n, tokens, pad;
};

// Workspace of one kernel: partials of up to `ctas` CTAs, two each (of the row
// that ends in the share and of the one that starts there), `rows` heads each.
struct Work {
    Part *part;  // [ctas]
    float *ml;   // [ctas][2][rows][2]
    float *o;    // [ctas][2][rows][head_dim]
    __host__ __device__ Work(void *ws, int ctas, int rows) {
        uint8_t *b = static_cast<uint8_t *>(ws);
        part = reinterpret_cast<Part *>(b);
        b += ((size_t)ctas * sizeof(Part) + 255) / 256 * 256;
        ml = reinterpret_cast<float *>(b);
        b += ((size_t)ctas * 2 * rows * 2 * sizeof(float) + 255) / 256 * 256;
        o = reinterpret_cast<float *>(b);
    }
    static size_t bytes(int ctas, int rows, int head_dim) {
        const Work w(nullptr, ctas, rows);
        return reinterpret_cast<uintptr_t>(w.o) + (size_t)ctas * 2 * rows * head_dim * sizeof(float);
    }
};

// Groups: every `block` rows, counted from its start, of a run of rows of q with
// one table row (within aligned spans of group_span rows, which bound the search
// for the start).  Either paged_group.cu takes all rows of a call, by groups, or
// paged_attn.cu, one by one: one of them alone, as a few rows of a kind would
// still cost its whole latency (14 groups of four rows and three rows more, 2 K
// cells, 8/2 heads of 256: 59 us by both, 44 us one by one).  Both decide it from
// the lengths.
constexpr int WHOLE = 16;  // rows of up to this many units are not shared out
template <int S>
__device__ __forceinline__ int units_of(int len) {  // one at least, so that an empty row's output is written
    constexpr int UNIT = 32 / S;
    return max((len + UNIT - 1) / UNIT, 1);
}
// alone: units of all rows; together: of the longest row of each group; longer:
// some row has more than WHOLE.  A group costs what 3 to 3.5 rows of 256 dims or
// 4 of 128 cost, and some microseconds more for a few long tiles than for many
// small units: groups where they save 4096 units of a KV head (33 MB of codes).
// One by one and by groups, us:
//   48/4 heads of 256, 12 sequences: 3 rows of 6 K cells 102, 103; 4 131, 104; 8 238, 114
//                                    5 rows of 1 K cells 48, 51; 8 65, 58
//                      1 sequence:   8 rows of 1 K cells 19, 26; of 6 K 38, 31
//   32/8 heads of 128, 12 sequences: 4 rows of 6 K cells 127, 128; 5 152, 129; 8 234, 129
//                                    5 rows of 1 K cells 42, 47; 8 58, 48
//                      1 sequence:   8 rows of 1 K cells 18, 21; of 6 K 33, 27
template <int S>
__device__ __forceinline__ bool take_groups(const qsa_paged_attn_args &a, long long alone, long long together, bool longer) {
    return longer && (2 * alone - (S == 1 ? 8 : 7) * together) * a.n_kv_heads > 2 * 4096;
}
// Whether rows of up to `units` units could be: if not, the groups' launch is left out (2 us).
template <int S>
inline bool may_take_groups(const qsa_paged_attn_args &a, long long units, int block) {
    const long long groups = a.n_tokens < block ? 1 : a.n_tokens / block;
    return a.rows && (2ll * a.n_tokens - (S == 1 ? 8 : 7) * groups) * units * a.n_kv_heads > 2 * 4096;
}
constexpr int GROUP_ROWS = 128;  // heads of a group, all its rows' (the M of its products)
__host__ __device__ inline int group_block(int per) {
    int b = 1;
    while (2 * b * per <= GROUP_ROWS) b *= 2;
    return b;
}
__device__ __forceinline__ int group_span(int block) { return block > 64 ? block : 64; }
// The first row of the group that row t would belong to.
__device__ __forceinline__ int group_start(const int32_t *rows, int t, int block) {
    const int row = __ldg(rows + t);
    int s = t;
    while ((s & (group_span(block) - 1)) && __ldg(rows + s - 1) == row) --s;
    return s + ((t - s) & -block);
}
// The row after the last one that the group of t, its first, could have.
__device__ __forceinline__ int group_end(const qsa_paged_attn_args &a, int t, int block) {
    return min(min(a.n_tokens, t + block), (t | (group_span(block) - 1)) + 1);
}

// Row t's length, cut to its range, and its table row (0 with length 0 if it
// is out of range).
__device__ __forceinline__ int row_len(const qsa_paged_attn_args &a, int t, int &row, bool &bad) {
    row = a.rows ? __ldg(a.rows + t) : t;
    const int len = __ldg(a.seq_lens + t), most = a.max_pages * a.page_size;
    if (row < 0 || row >= a.n_rows) {
        bad = true;
        row = 0;
        return 0;
    }
    bad |= len < 0 || len > most;
    return min(max(len, 0), most);
}
__device__ __forceinline__ void store_out(const qsa_paged_attn_args &a, size_t i, float2 y) {
    if (a.dtype == QSA_F16)
        *reinterpret_cast<__half2 *>(static_cast<__half *>(a.out) + i) = __floats2half2_rn(y.x, y.y);
    else
        *reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(a.out) + i) = __floats2bfloat162_rn(y.x, y.y);
}
// lse of a base-2 maximum and sum.  The sum's exponent goes to the maximum first,
// so that only the result's own size is rounded.  A row without cells has -inf
// and 0, which gives -inf; one whose scores are all NaN has -inf and NaN, which
// gives NaN.
__device__ __forceinline__ float lse_of(float m, float l) {
    const int e = (int)(__float_as_uint(l) >> 23) - 127;
    if (e <= -127 || e >= 128) return (m + log2f(l)) * LN2;  // 0, infinite or NaN
    return (m + (float)e + log2f(__uint_as_float((__float_as_uint(l) & 0x007FFFFFu) | 0x3F800000u))) * LN2;
}
// y / (1 + exp(-gate)); each step off by a few 2^-23, and a gate far below 0 gives 0.
__device__ __forceinline__ float gated(float y, float gate) { return __fdividef(y, 1.0f + ex2(-gate * LOG2E)); }

// Joins the partials of rows that span CTAs, of one kernel or of both.  Part p
// of the row that starts in CTA x is slot 1 of that CTA, then slot 0 of the
// next ones of its KV head.  A block lists the CTAs in which such rows start,
// and blocks go round over these and chunks of their heads.  A warp takes 32 V
// dims of one head and every G-th part; it works the weights out itself (a few
// loads per lane), so there is nothing to wait for but the last sum.  Many
// rows: HB heads and no split per block; few, whose parts are many: the block's
// warps split the parts of one head.
constexpr int JOIN_WARPS = 16;
constexpr int MAX_PARTS = 152 * 2;          // CTAs of paged_attn_kernel
constexpr int MAX_GROUP_PARTS = 152;        // CTAs of paged_group_kernel
struct Joined {  // a kernel's partials: where, room for how many CTAs and heads, CTAs launched
    void *ws;
    int cap, rows, ctas;
};
template <int S, int HB>
__global__ void __launch_bounds__(JOIN_WARPS * 32)
    paged_join_kernel(const qsa_paged_attn_args a, const Joined one, const Joined two) {
    // Dims of a lane.  Few rows of 256: 4, for more loads at once (one of 321 cells 11.4
    // us, 12.8 with 2; of 128 dims 10.6, 10.1).
    constexpr int V = HB == 1 && S == 2 ? 4 : 2;
    constexpr int D = 128 * S, DC = D / (32 * V), G = JOIN_WARPS / (HB * DC);
    constexpr int LOADS = (MAX_PARTS + 31) / 32;
    static_assert(MAX_PARTS + MAX_GROUP_PARTS <= JOIN_WARPS * 32, "a thread per CTA");
    __shared__ float2 so[G > 1 ? JOIN_WARPS : 1][V / 2][32];
    __shared__ int at[JOIN_WARPS * 32], found[2][JOIN_WARPS];
    wait_for_previous_grid();
    allow_dependent_launch();
    const int per = a.n_q_heads / a.n_kv_heads, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Work w1(one.ws, one.cap, one.rows), w2(two.ws, two.cap, two.rows);
    const bool first = tid < one.ctas && w1.part[tid].row >= 0;
    const bool second = tid >= one.ctas && tid - one.ctas < two.ctas && w2.part[tid - one.ctas].row >= 0;
    const unsigned m1 = __ballot_sync(0xffffffffu, first), m2 = __ballot_sync(0xffffffffu, second);
    if (lane == 0) {
        found[0][warp] = __popc(m1);
        found[1][warp] = __popc(m2);
    }
    __syncthreads();
    int before1 = 0, before2 = 0, n1 = 0, n2 = 0;
#pragma unroll
    for (int w = 0; w < JOIN_WARPS; ++w) {
        before1 += w < warp ? found[0][w] : 0;
        before2 += w < warp ? found[1][w] : 0;
        n1 += found[0][w];
        n2 += found[1][w];
    }
    if (first) at[before1 + __popc(m1 & ((1u << lane) - 1))] = tid;
    if (second) at[n1 + before2 + __popc(m2 & ((1u << lane) - 1))] = tid - one.ctas;
    __syncthreads();
    const int chunks1 = (one.rows + HB - 1) / HB, chunks2 = (two.rows + HB - 1) / HB;
    for (int it = blockIdx.x; it < n1 * chunks1 + n2 * chunks2; it += gridDim.x) {
        const bool group = it >= n1 * chunks1;
        const int in = group ? it - n1 * chunks1 : it, chunks = group ? chunks2 : chunks1, rows = group ? two.rows : one.rows;
        const Work &work = group ? w2 : w1;
        const int x = at[(group ? n1 : 0) + in / chunks], h0 = in % chunks * HB;
        const int h = h0 + warp / (DC * G), dc = warp / G % DC, grp = warp % G;
        const Part part = work.part[x];
        if (h0 >= part.tokens * per) continue;  // the same in all warps
        auto slot = [&](int p) { return (size_t)(x + p * a.n_kv_heads) * 2 + (p == 0 ? 1 : 0); };
        const int n = h < part.tokens * per ? part.n : 0;
        float w[LOADS], l[LOADS], M = -CUDART_INF_F, L = 0.0f;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int p = i * 32 + lane;
            float2 v = make_float2(-CUDART_INF_F, 0.0f);
            if (p < n) v = *reinterpret_cast<const float2 *>(work.ml + (slot(p) * rows + h) * 2);
            w[i] = v.x;
            l[i] = v.y;
            M = fmaxf(M, v.x);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            w[i] = w[i] == -CUDART_INF_F ? 0.0f : exp2f(w[i] - M);
            L += w[i] * l[i];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
        const int d = (dc * 32 + lane) * V;
        float2 o[V / 2];
#pragma unroll
        for (int e = 0; e < V / 2; ++e) o[e] = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            if (i * 32 >= n) break;
            const int top = min(n - i * 32, 32);
#pragma unroll 8
            for (int k = grp; k < top; k += G) {  // G divides 32
                const float f = __shfl_sync(0xffffffffu, w[i], k);
                const float *src = work.o + (slot(i * 32 + k) * rows + h) * D + d;
                float2 v[V / 2];
                if constexpr (V == 4) {
                    const float4 x = *reinterpret_cast<const float4 *>(src);
                    v[0] = make_float2(x.x, x.y);
                    v[1] = make_float2(x.z, x.w);
                } else {
                    v[0] = *reinterpret_cast<const float2 *>(src);
                }
#pragma unroll
                for (int e = 0; e < V / 2; ++e) o[e] = __ffma2_rn(make_float2(f, f), v[e], o[e]);
            }
        }
        if constexpr (G > 1) {
#pragma unroll
            for (int e = 0; e < V / 2; ++e) so[warp][e][lane] = o[e];
            __syncthreads();
            if (grp == 0) {
#pragma unroll
                for (int i = 1; i < G; ++i)
#pragma unroll
                    for (int e = 0; e < V / 2; ++e) o[e] = __fadd2_rn(o[e], so[warp + i][e][lane]);
            }
            __syncthreads();
        }
        if (grp || h >= part.tokens * per) continue;
        const float inv = M == -CUDART_INF_F ? 0.0f : 1.0f / L;
        const size_t row = (size_t)(part.row + h / per) * a.n_q_heads + (size_t)(x % a.n_kv_heads) * per + h % per;
        if (dc == 0 && lane == 0 && a.lse) a.lse[row] = lse_of(M, L);
        if (!QSA_IN(row * D + d + V - 1, (size_t)a.n_tokens * a.n_q_heads * D)) continue;
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
            float2 y = make_float2(o[e].x * inv, o[e].y * inv);
            if (a.gate) {
                const float2 gate = __ldg(reinterpret_cast<const float2 *>(a.gate + row * D + d + 2 * e));
                y = make_float2(gated(y.x, gate.x), gated(y.y, gate.y));
            }
            store_out(a, row * D + d + 2 * e, y);
        }
    }
}

// Fewer pairs of a row and a KV head than half the SMs: their parts are many (a
// row of 30 K cells alone: 118), and a block's warps share them.
template <int S>
cudaError_t launch_join(const qsa_paged_attn_args &a, const Joined &one, const Joined &two, cudaStream_t s) {
    constexpr int HB = S == 1 ? 8 : 4;
    const dim3 block(JOIN_WARPS * 32);
    const long long most = (long long)a.n_tokens * a.n_kv_heads;
    const bool few = most < 76;
    // Rows that span CTAs: no more than there are, nor than one per CTA.
    const int heads = one.rows > two.rows ? one.rows : two.rows;
    const long long items = (most < one.ctas + two.ctas ? most : one.ctas + two.ctas) * (few ? heads : (heads + HB - 1) / HB);
    const dim3 grid((unsigned)(items < 152 * 4 ? items : 152 * 4));
    return few ? launch_dependent(paged_join_kernel<S, 1>, grid, block, 0, s, a, one, two)
               : launch_dependent(paged_join_kernel<S, HB>, grid, block, 0, s, a, one, two);
}

}  // namespace

size_t paged_group_workspace_bytes(int head_dim);
// paged_group.cu: the groups, where a.rows is given.  ws as Work of GROUP_ROWS
// rows; `ctas` receives how many leave partials there, to be joined.
cudaError_t launch_paged_group(const qsa_paged_attn_args &a, void *ws, int &ctas, cudaStream_t s);

}  // namespace qsa
