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

// Groups: a maximal run of rows of q with one table row, within an aligned block
// of `block` rows, is taken by paged_group.cu if it has GROUP_MIN rows or more.
constexpr int GROUP_MIN = 3;
constexpr int GROUP_ROWS = 128;  // heads of a group, all its rows' (the M of its products)
__host__ __device__ inline int group_block(int per) {
    int b = 1;
    while (2 * b * per <= GROUP_ROWS) b *= 2;
    return b;
}
// Whether row t belongs to a group.
__device__ __forceinline__ bool grouped(const qsa_paged_attn_args &a, int t, int block) {
    const int row = __ldg(a.rows + t);
    int n = 1;
    for (int u = t; n < GROUP_MIN && (u & (block - 1)) && __ldg(a.rows + u - 1) == row; --u) ++n;
    for (int u = t + 1; n < GROUP_MIN && u < a.n_tokens && (u & (block - 1)) && __ldg(a.rows + u) == row; ++u) ++n;
    return n >= GROUP_MIN;
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
// y / (1 + exp(-gate)); each step off by a few 2^-23, and a gate far below 0 gives 0.
__device__ __forceinline__ float gated(float y, float gate) { return __fdividef(y, 1.0f + ex2(-gate * LOG2E)); }

// Joins the partials of rows that span CTAs.  Block x looks after the row that
// starts in CTA x and continues in others, if there is one: part p is slot 1 of
// that CTA, then slot 0 of the next ones of its KV head.  A warp takes 64 dims
// of one query head and every G-th part; it works the weights out itself (a
// few loads per lane), so there is nothing to wait for but the last sum.  Many
// rows: HB heads and no split per block; few, whose parts are many: the block's
// warps split the parts of one head.
constexpr int JOIN_WARPS = 16;
constexpr int MAX_PARTS = 152 * 2;  // CTAs of either kernel
template <int S, int HB>
__global__ void __launch_bounds__(JOIN_WARPS * 32)
    paged_join_kernel(const qsa_paged_attn_args a, void *ws, int ctas, int rows) {
    constexpr int D = 128 * S, DC = D / 64, G = JOIN_WARPS / (HB * DC);
    constexpr int LOADS = (MAX_PARTS + 31) / 32;
    __shared__ float2 so[G > 1 ? JOIN_WARPS : 1][32];
    wait_for_previous_grid();
    allow_dependent_launch();
    const int per = a.n_q_heads / a.n_kv_heads, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int h = blockIdx.y * HB + warp / (DC * G), dc = warp / G % DC, grp = warp % G;
    const Work work(ws, ctas, rows);
    const Part part = work.part[blockIdx.x];
    if (part.row < 0) return;
    auto slot = [&](int p) { return (size_t)(blockIdx.x + p * a.n_kv_heads) * 2 + (p == 0 ? 1 : 0); };
    const int n = h < part.tokens * per ? part.n : 0;
    float w[LOADS], l[LOADS], M = -CUDART_INF_F, L = 0.0f;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int p = i * 32 + lane;
        w[i] = -CUDART_INF_F;
        l[i] = 0.0f;
        if (p < n) {
            const float2 v = *reinterpret_cast<const float2 *>(work.ml + (slot(p) * rows + h) * 2);
            w[i] = v.x;
            l[i] = v.y;
        }
        M = fmaxf(M, w[i]);
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
    const int d = dc * 64 + lane * 2;
    float2 o = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        if (i * 32 >= n) break;
        const int top = min(n - i * 32, 32);
#pragma unroll 4
        for (int k = (grp - i * 32 % G + G) % G; k < top; k += G) {
            const float f = __shfl_sync(0xffffffffu, w[i], k);
            const float2 v = *reinterpret_cast<const float2 *>(work.o + (slot(i * 32 + k) * rows + h) * D + d);
            o.x = fmaf(f, v.x, o.x);
            o.y = fmaf(f, v.y, o.y);
        }
    }
    if constexpr (G > 1) {
        so[warp][lane] = o;
        __syncthreads();
        if (grp) return;
#pragma unroll
        for (int i = 1; i < G; ++i) {
            o.x += so[warp + i][lane].x;
            o.y += so[warp + i][lane].y;
        }
    }
    if (h >= part.tokens * per) return;
    const float inv = M == -CUDART_INF_F ? 0.0f : 1.0f / L;
    const size_t row = (size_t)(part.row + h / per) * a.n_q_heads + (size_t)(blockIdx.x % a.n_kv_heads) * per + h % per;
    if (dc == 0 && lane == 0 && a.lse) a.lse[row] = M == -CUDART_INF_F ? M : (M + log2f(L)) * LN2;
    if (!QSA_IN(row * D + d + 1, (size_t)a.n_tokens * a.n_q_heads * D)) return;
    o = make_float2(o.x * inv, o.y * inv);
    if (a.gate) {
        const float2 gate = __ldg(reinterpret_cast<const float2 *>(a.gate + row * D + d));
        o = make_float2(gated(o.x, gate.x), gated(o.y, gate.y));
    }
    store_out(a, row * D + d, o);
}

// `ctas` launched CTAs whose partials lie in ws (room for `cap` of them, `rows`
// heads each).  Fewer pairs of a row and a KV head than half the SMs: their
// parts are many (a row of 30 K cells alone: 118), and a block's warps share
// them.
template <int S>
cudaError_t launch_join(const qsa_paged_attn_args &a, void *ws, int cap, int rows, int ctas, cudaStream_t s) {
    constexpr int HB = S == 1 ? 8 : 4;
    const dim3 block(JOIN_WARPS * 32);
    if ((long long)a.n_tokens * a.n_kv_heads < 76)
        return launch_dependent(paged_join_kernel<S, 1>, dim3(ctas, rows), block, 0, s, a, ws, cap, rows);
    return launch_dependent(paged_join_kernel<S, HB>, dim3(ctas, (rows + HB - 1) / HB), block, 0, s, a, ws, cap, rows);
}

// paged_group.cu: the groups, where a.rows is given; ws as Work of GROUP_ROWS rows.
}  // namespace

size_t paged_group_workspace_bytes(int head_dim);
cudaError_t launch_paged_group(const qsa_paged_attn_args &a, void *ws, cudaStream_t s);

}  // namespace qsa
