// qsa_paged_prep and qsa_paged_gather: rows into and out of the paged cache.
//
// Prep: for each token, the query and key heads' RMS norm and rotation and the
// K/V rows' int8 codes, written to the token's slot.  One block of four warps
// per token and 16 of its head rows (query heads, then key, then value heads);
// a warp takes four rows side by side, so that their loads and their sums of
// squares are in flight together, and a lane holds head_dim/32 consecutive
// elements.  The token's angles are computed once per block, one per thread,
// while the rows are on their way.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "check.cuh"
#include "qsa_internal.h"

namespace qsa {
namespace {

constexpr int ROWS_PER_WARP = 4;
constexpr int PREP_WARPS = 4;
constexpr int ROWS_PER_BLOCK = ROWS_PER_WARP * PREP_WARPS;

template <int BYTES>
struct Words {
    static_assert(BYTES % 8 == 0, "rows move in 8- or 16-byte words");
};
template <>
struct Words<8> {
    uint2 w[1];
};
template <>
struct Words<16> {
    uint4 w[1];
};
template <>
struct Words<32> {
    uint4 w[2];
};

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_float(float v, float &o) { o = v; }
__device__ __forceinline__ void from_float(float v, __half &o) { o = __float2half_rn(v); }
__device__ __forceinline__ void from_float(float v, __nv_bfloat16 &o) { o = __float2bfloat16_rn(v); }

template <int N, class T>
__device__ __forceinline__ void load_elems(const T *p, float (&x)[N]) {
    union {
        Words<N * (int)sizeof(T)> w;
        T e[N];
    } u;
    const auto *src = reinterpret_cast<const decltype(u.w) *>(p);
#pragma unroll
    for (int i = 0; i < (int)(sizeof(u.w.w) / sizeof(u.w.w[0])); ++i) u.w.w[i] = __ldg(&src->w[i]);
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = to_float(u.e[e]);
}

template <int N, class T>
__device__ __forceinline__ void store_elems(T *p, const float (&x)[N]) {
    union U {
        Words<N * (int)sizeof(T)> w;
        T e[N];
        __device__ U() {}
    } u;
#pragma unroll
    for (int e = 0; e < N; ++e) from_float(x[e], u.e[e]);
    *reinterpret_cast<decltype(u.w) *>(p) = u.w;
}

// cos and sin of p * f, times m.  f = mant * 2^(ex - 150), so |p| * mant is an
// exact integer below 2^55, and its product with 1/(2 pi) in 66 fractional
// bits is the angle in turns times 2^(216 - ex); the 32 bits below the point
// are the fraction of a turn to 2^-32.  All in integers: an fp32 product is
// off by 2e-3 rad at p ~ 32k, and a double-precision one costs eight times as
// much on this chip.  (f at or above 2^57, where a step of p is no angle any
// more, is cut off there.)
__device__ __forceinline__ float2 cos_sin_of(int p, float f, float m) {
    constexpr unsigned long long INV_2PI_Q66 = 0xA2F9836E4E44152Aull;
    const uint32_t bits = __float_as_uint(f);
    const int ex = min(max((int)((bits >> 23) & 0xFFu), 1), 184);
    const uint32_t mant = (bits & 0x7FFFFFu) | ((bits & 0x7F800000u) ? 0x800000u : 0u);
    const unsigned long long pm = (unsigned long long)(p < 0 ? 0u - (uint32_t)p : (uint32_t)p) * mant;
    const unsigned long long lo = pm * INV_2PI_Q66, hi = __umul64hi(pm, INV_2PI_Q66);
    const int sh = 216 - ex - 32;  // 0 .. 183
    unsigned long long v;
    if (sh >= 128)
        v = 0ull;
    else if (sh >= 64)
        v = hi >> (sh - 64);
    else
        v = sh == 0 ? lo : (lo >> sh) | (hi << (64 - sh));
    float s, c;
    sincospif((float)(int32_t)(uint32_t)v * 4.656612873077393e-10f, &s, &c);  // 2^-31 half turns
    return make_float2(c * m, p < 0 ? -s * m : s * m);
}

template <int D, class TI, class TO>
__global__ void __launch_bounds__(PREP_WARPS * 32) paged_prep_kernel(const qsa_paged_prep_args a) {
    constexpr int N = D / 32;  // elements per lane
    __shared__ float2 cs[D / 2];
    wait_for_previous_grid();
    allow_dependent_launch();
    const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int slot = __ldg(a.slots + t);
    if (slot < 0 || slot >= a.cache_cells) {
        if (slot != -1 && threadIdx.x == 0 && blockIdx.y == 0 && a.err) atomicOr(a.err, QSA_DEVERR_BAD_ID);
        return;
    }
    const int hq = a.n_q_heads, hkv = a.n_kv_heads, nrows = hq + 2 * hkv;
    const int row0 = blockIdx.y * ROWS_PER_BLOCK + warp * ROWS_PER_WARP;
    float x[ROWS_PER_WARP][N];
#pragma unroll
    for (int j = 0; j < ROWS_PER_WARP; ++j) {
        const int row = row0 + j;
#pragma unroll
        for (int e = 0; e < N; ++e) x[j][e] = 0.0f;
        if (row < nrows) {
            const TI *src = row < hq         ? static_cast<const TI *>(a.q_in) + t * a.q_stride + row * D
                            : row < hq + hkv ? static_cast<const TI *>(a.k_in) + t * a.k_stride + (row - hq) * D
                                             : static_cast<const TI *>(a.v_in) + t * a.v_stride + (row - hq - hkv) * D;
            load_elems<N>(src + lane * N, x[j]);
        }
    }
    const int half = a.rope_dims >> 1;
    if ((int)threadIdx.x < half)
        cs[threadIdx.x] = cos_sin_of(__ldg(a.positions + t), __ldg(a.inv_freq + threadIdx.x), a.rope_mscale);

    float ss[ROWS_PER_WARP];
#pragma unroll
    for (int j = 0; j < ROWS_PER_WARP; ++j) {
        ss[j] = 0.0f;
#pragma unroll
        for (int e = 0; e < N; ++e) ss[j] = fmaf(x[j][e], x[j][e], ss[j]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int j = 0; j < ROWS_PER_WARP; ++j) ss[j] += __shfl_xor_sync(0xffffffffu, ss[j], o);
    __syncthreads();  // cs

#pragma unroll
    for (int j = 0; j < ROWS_PER_WARP; ++j) {
        const int row = row0 + j;
        if (row >= nrows) break;
        const bool is_q = row < hq, is_v = row >= hq + hkv;
        const float *w = is_q ? a.q_norm_w : is_v ? nullptr : a.k_norm_w;
        if (w) {
            float wv[N];
            load_elems<N>(w + lane * N, wv);
            const float rs = __frsqrt_rn(ss[j] * (1.0f / D) + a.eps);
#pragma unroll
            for (int e = 0; e < N; ++e) x[j][e] = (rs * x[j][e]) * wv[e];
        }
        const int i0 = lane * N;
        if (!is_v && half > 0) {
            if (a.interleaved) {
                if (i0 < 2 * half) {
#pragma unroll
                    for (int e = 0; e < N; e += 2) {
                        const float2 c = cs[(i0 + e) >> 1];
                        const float u = x[j][e], v = x[j][e + 1];
                        x[j][e] = u * c.x - v * c.y;
                        x[j][e + 1] = v * c.x + u * c.y;
                    }
                }
            } else {
                const int sh = half / N;  // lanes between partners
                const bool first = i0 < half;
                const int from = first ? lane + sh : lane - sh;
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const float o = __shfl_sync(0xffffffffu, x[j][e], from & 31);
                    if (i0 < 2 * half) {
                        const float2 c = cs[first ? i0 + e : i0 - half + e];
                        x[j][e] = first ? x[j][e] * c.x - o * c.y : x[j][e] * c.x + o * c.y;
                    }
                }
            }
        }
        if (is_q) {
            const size_t at = ((size_t)t * hq + row) * D;
            if (QSA_IN(at + D - 1, (size_t)a.ntok * hq * D)) store_elems<N>(static_cast<TO *>(a.q_out) + at + i0, x[j]);
            continue;
        }
        // The largest magnitude as an integer, so that a NaN is the largest.
        uint32_t top = 0u;
#pragma unroll
        for (int e = 0; e < N; ++e) top = max(top, __float_as_uint(x[j][e]) & 0x7FFFFFFFu);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const __half sch = __float2half_rn(__fdiv_rn(__uint_as_float(top), 127.0f));
        const float sc = __half2float(sch);
        const size_t cell = (size_t)slot * hkv + (row - hq - (is_v ? hkv : 0));
        if (!QSA_IN(cell, (size_t)a.cache_cells * hkv)) continue;
        uint32_t code[N / 4];
#pragma unroll
        for (int e = 0; e < N; ++e) {
            float c = 0.0f;
            if (sc != 0.0f) c = fminf(fmaxf(rintf(__fdiv_rn(x[j][e], sc)), -127.0f), 127.0f);
            const uint32_t b = (uint32_t)(uint8_t)(int8_t)(int)c << (8 * (e & 3));
            code[e / 4] = (e & 3) ? code[e / 4] | b : b;
        }
        int8_t *dst = (is_v ? a.vq : a.kq) + cell * D + i0;
        if constexpr (N == 4)
            *reinterpret_cast<uint32_t *>(dst) = code[0];
        else
            *reinterpret_cast<uint2 *>(dst) = make_uint2(code[0], code[1]);
        if ((lane & 7) == 0) (is_v ? a.vsc : a.ksc)[cell * 4 + (lane >> 3)] = __half_as_ushort(sch);
    }
}

// Gather: a thread takes eight dims of one (cell, KV head), of both K and V,
// so that neighbouring threads read 8-byte and write 16-byte words of one row.
constexpr int GATHER_THREADS = 256;

template <class T>
__global__ void __launch_bounds__(GATHER_THREADS) paged_gather_kernel(const qsa_paged_gather_args a) {
    wait_for_previous_grid();
    allow_dependent_launch();
    const int per_row = a.head_dim / 8, per_id = a.n_kv_heads * per_row;
    const long long i = (long long)blockIdx.x * GATHER_THREADS + threadIdx.x;
    const long long id_i = i / per_id;
    if (id_i >= a.n_ids) return;
    const int in_id = (int)(i - id_i * per_id), h = in_id / per_row, d = (in_id - h * per_row) * 8;
    long long cell = __ldg(a.ids + id_i);
    bool bad = cell < -1;
    if (cell >= 0 && a.page_table) {
        const int row = __ldg(a.rows + id_i);
        const long long page = cell / a.page_size;
        if (row < 0 || row >= a.n_rows || page >= a.max_pages) {
            bad = true;
            cell = -1;
        } else {
            const int e = __ldg(a.page_table + (size_t)row * a.max_pages + page);
            cell = e < 0 ? -2 : (long long)e * a.page_size + cell % a.page_size;
            bad = e < 0;
        }
    }
    bad |= cell >= a.cache_cells;
    if (bad && in_id == 0 && a.err) atomicOr(a.err, QSA_DEVERR_BAD_ID);
    float k[8], v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) k[e] = v[e] = 0.0f;
    if (cell >= 0 && cell < a.cache_cells) {
        const size_t row = (size_t)cell * a.n_kv_heads + h;
        const uint2 kw = __ldg(reinterpret_cast<const uint2 *>(a.kq + row * a.head_dim + d));
        const uint2 vw = __ldg(reinterpret_cast<const uint2 *>(a.vq + row * a.head_dim + d));
        const float ks = __half2float(__ushort_as_half(__ldg(a.ksc + row * 4 + d / a.group)));
        const float vs = __half2float(__ushort_as_half(__ldg(a.vsc + row * 4 + d / a.group)));
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            k[e] = (float)(int8_t)((e < 4 ? kw.x : kw.y) >> (8 * (e & 3))) * ks;
            v[e] = (float)(int8_t)((e < 4 ? vw.x : vw.y) >> (8 * (e & 3))) * vs;
        }
    }
    const size_t at = ((size_t)id_i * a.n_kv_heads + h) * a.head_dim + d;
    if (!QSA_IN(at + 7, (size_t)a.n_ids * a.n_kv_heads * a.head_dim)) return;
    store_elems<8>(static_cast<T *>(a.k_out) + at, k);
    store_elems<8>(static_cast<T *>(a.v_out) + at, v);
}

template <int D, class TI>
cudaError_t prep_to(const qsa_paged_prep_args &a, cudaStream_t s) {
    const int nrows = a.n_q_heads + 2 * a.n_kv_heads;
    const dim3 grid(a.ntok, (nrows + ROWS_PER_BLOCK - 1) / ROWS_PER_BLOCK);
    if (a.q_out_dtype == QSA_F16)
        return launch_dependent(paged_prep_kernel<D, TI, __half>, grid, dim3(PREP_WARPS * 32), 0, s, a);
    return launch_dependent(paged_prep_kernel<D, TI, __nv_bfloat16>, grid, dim3(PREP_WARPS * 32), 0, s, a);
}

template <int D>
cudaError_t prep_from(const qsa_paged_prep_args &a, cudaStream_t s) {
    return a.in_dtype == QSA_F32   ? prep_to<D, float>(a, s)
           : a.in_dtype == QSA_F16 ? prep_to<D, __half>(a, s)
                                   : prep_to<D, __nv_bfloat16>(a, s);
}

}  // namespace

cudaError_t launch_paged_prep(const qsa_paged_prep_args &a, cudaStream_t s) {
    return a.head_dim == 128 ? prep_from<128>(a, s) : prep_from<256>(a, s);
}

cudaError_t launch_paged_gather(const qsa_paged_gather_args &a, cudaStream_t s) {
    const long long n = (long long)a.n_ids * a.n_kv_heads * (a.head_dim / 8);
    const dim3 grid((unsigned)((n + GATHER_THREADS - 1) / GATHER_THREADS)), block(GATHER_THREADS);
    return a.out_dtype == QSA_F32   ? launch_dependent(paged_gather_kernel<float>, grid, block, 0, s, a)
           : a.out_dtype == QSA_F16 ? launch_dependent(paged_gather_kernel<__half>, grid, block, 0, s, a)
                                    : launch_dependent(paged_gather_kernel<__nv_bfloat16>, grid, block, 0, s, a);
}

}  // namespace qsa

QSA_DEFINE_CHECK_READER(take_check_word_paged_prep)
