// qsa_paged_attn: attention of one new token per row over a paged sequence.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include "check.cuh"
#include "qsa_internal.h"

namespace qsa {
namespace {

constexpr int WARPS = 4;
constexpr int MAX_PER = 16;  // query heads per KV head

__device__ __forceinline__ float load_q(const void *q, int dtype, size_t i) {
    return dtype == QSA_F16 ? __half2float(static_cast<const __half *>(q)[i])
                            : __bfloat162float(static_cast<const __nv_bfloat16 *>(q)[i]);
}

// One block per (row, KV head); a warp takes every fourth cell, a lane
// head_dim/32 dims of it, with one running maximum, sum and value row per
// query head; the warps' states are joined at the end.
template <int D>
__global__ void __launch_bounds__(WARPS * 32) paged_attn_kernel(const qsa_paged_attn_args a) {
    constexpr int N = D / 32;
    __shared__ float so[WARPS][D], sm[WARPS], sl[WARPS];
    wait_for_previous_grid();
    allow_dependent_launch();
    const int t = blockIdx.x / a.n_kv_heads, kvh = blockIdx.x % a.n_kv_heads;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, per = a.n_q_heads / a.n_kv_heads;
    const int row = a.rows ? a.rows[t] : t;
    int len = a.seq_lens[t];
    bool bad = false;
    if (row < 0 || row >= a.n_rows) {
        bad = true;
        len = 0;
    }
    const int most = a.max_pages * a.page_size;
    if (len < 0 || len > most) {
        bad = true;
        len = len < 0 ? 0 : most;
    }
    for (int g = 0; g < per; ++g) {
        const size_t qi = ((size_t)t * a.n_q_heads + kvh * per + g) * D + lane * N;
        float q[N], o[N], m = -CUDART_INF_F, l = 0.0f;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            q[e] = load_q(a.q, a.dtype, qi + e) * a.softmax_scale;
            o[e] = 0.0f;
        }
        for (int c = warp; c < len; c += WARPS) {
            const int page = a.page_table[(size_t)row * a.max_pages + c / a.page_size];
            if (page < 0 || page >= a.n_pages) {
                bad = true;
                continue;
            }
            const size_t cell = ((size_t)page * a.page_size + c % a.page_size) * a.n_kv_heads + kvh;
            if (!QSA_IN(cell, (size_t)a.n_pages * a.page_size * a.n_kv_heads)) continue;
            const float ks = __half2float(__ushort_as_half(a.ksc[cell * 4 + lane / 8]));
            const float vs = __half2float(__ushort_as_half(a.vsc[cell * 4 + lane / 8]));
            float s = 0.0f;
#pragma unroll
            for (int e = 0; e < N; ++e) s = fmaf(q[e], (float)a.kq[cell * D + lane * N + e], s);
            s *= ks;
#pragma unroll
            for (int i = 16; i > 0; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
            const float mn = fmaxf(m, s), al = expf(m - mn), p = expf(s - mn);
            m = mn;
            l = l * al + p;
#pragma unroll
            for (int e = 0; e < N; ++e) o[e] = o[e] * al + p * vs * (float)a.vq[cell * D + lane * N + e];
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < N; ++e) so[warp][lane * N + e] = o[e];
        if (lane == 0) {
            sm[warp] = m;
            sl[warp] = l;
        }
        __syncthreads();
        float M = -CUDART_INF_F, L = 0.0f;
        for (int w = 0; w < WARPS; ++w) M = fmaxf(M, sm[w]);
        for (int w = 0; w < WARPS; ++w) L += M == -CUDART_INF_F ? 0.0f : sl[w] * expf(sm[w] - M);
        for (int d = threadIdx.x; d < D; d += WARPS * 32) {
            float r = 0.0f;
            for (int w = 0; w < WARPS; ++w)
                if (sm[w] != -CUDART_INF_F) r += expf(sm[w] - M) * so[w][d];
            if (M != -CUDART_INF_F) r /= L;
            const size_t i = ((size_t)t * a.n_q_heads + kvh * per + g) * D + d;
            if (a.gate) r = r / (1.0f + expf(-a.gate[i]));
            if (a.dtype == QSA_F16)
                static_cast<__half *>(a.out)[i] = __float2half_rn(r);
            else
                static_cast<__nv_bfloat16 *>(a.out)[i] = __float2bfloat16_rn(r);
        }
        if (threadIdx.x == 0 && a.lse)
            a.lse[(size_t)t * a.n_q_heads + kvh * per + g] = M == -CUDART_INF_F ? M : M + logf(L);
    }
    if (bad && lane == 0 && a.err) atomicOr(a.err, QSA_DEVERR_BAD_ID);
}

}  // namespace

size_t paged_attn_workspace_bytes(int, int, int) { return 256; }

cudaError_t launch_paged_attn(const qsa_paged_attn_args &a, cudaStream_t s) {
    const dim3 grid(a.n_tokens * a.n_kv_heads), block(WARPS * 32);
    return a.head_dim == 128 ? launch_dependent(paged_attn_kernel<128>, grid, block, 0, s, a)
                             : launch_dependent(paged_attn_kernel<256>, grid, block, 0, s, a);
}

}  // namespace qsa

QSA_DEFINE_CHECK_READER(take_check_word_paged_attn)
