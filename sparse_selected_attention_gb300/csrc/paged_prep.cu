// qsa_paged_prep and qsa_paged_gather: rows into and out of the paged cache.
//
// Prep: for each token, the query and key heads' RMS norm and rotation and the
// K/V rows' int8 codes, written to the token's slot.  Its traffic is small
// beside its arithmetic and latency (some 100 instructions per row of 256 to 512
// bytes), so a warp works alone, without shared memory or barriers: it takes a
// run of one token's rows (query heads, then key, then value heads), two at a
// time with the next two on their way, and keeps the token's cosines and sines
// in registers.  Few tokens are split over more warps, down to two rows each.
// 1984 tokens of 12/1 heads of 128, with their gather: 7.0 us; 8191 of 24/2 heads of
// 256, 230 MB with their gather: 50 us, 4.6 TB/s, with 57% of the issue slots
// used.  (Rows fetched into L2 ahead, or fewer warps with more registers: 52 and
// 53 us.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "check.cuh"
#include "qsa_internal.h"

namespace qsa {
namespace {

constexpr int PREP_WARPS = 4;
constexpr int BATCH = 2;  // rows worked on together, with as many on their way

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
union Raw {
    Words<N * (int)sizeof(T)> w;
    T e[N];
    __device__ Raw() {}
};

template <int N, class T>
__device__ __forceinline__ void load_raw(Raw<N, T> &u, const T *p) {
    const auto *src = reinterpret_cast<const decltype(u.w) *>(p);
#pragma unroll
    for (int i = 0; i < (int)(sizeof(u.w.w) / sizeof(u.w.w[0])); ++i) u.w.w[i] = __ldg(&src->w[i]);
}

template <int N, class T>
__device__ __forceinline__ void store_elems(T *p, const float (&x)[N]) {
    Raw<N, T> u;
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
    // The special-function unit's sine and cosine are off by 2^-21 in this range
    // (as much as the angle's own rounding), a fraction of a query's fp16 or a
    // key's int8 step; the accurate ones cost as much as a row.
    float s, c;
    __sincosf((float)(int32_t)(uint32_t)v * 1.4629180792671596e-09f, &s, &c);  // pi 2^-31
    return make_float2(c * m, p < 0 ? -s * m : s * m);
}

// The code of x under scale s (normal or subnormal fp16, inv = 1/s correctly
// rounded), in the low byte: clamp(rint(x / s), -127, 127).  The quotient is
// the correctly rounded one by P. Markstein's theorem ("Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990): one
// correction of x * inv by its exact remainder.  Adding 1.5 * 2^23 rounds it to
// the nearest even integer, in the low mantissa bits.
__device__ __forceinline__ uint32_t code_of(float x, float s, float inv) {
    const float q = x * inv;
    const float c = fminf(fmaxf(fmaf(fmaf(-q, s, x), inv, q), -127.0f), 127.0f);
    return __float_as_uint(c + 12582912.0f);
}

struct PrepPlan {
    int chunks, rows;  // runs per token, rows of a run (even)
};

// Seven blocks an SM: 72 registers.  Two-byte rows fit but for some 50 bytes of
// halves of 256 dims; fp32 rows of 256 dims spill (halves 288 bytes stored and 576
// loaded a thread, interleaved 104 and 172: 4096 tokens of 24/2 heads, 27 us for
// their bytes, take 47 and 36 us).
template <int D, bool INTER, class TI, class TO>
__global__ void __launch_bounds__(PREP_WARPS * 32, 7) paged_prep_kernel(const qsa_paged_prep_args a, const PrepPlan plan) {
    constexpr int N = D / 32;  // elements per lane
    wait_for_previous_grid();
    allow_dependent_launch();
    const int lane = threadIdx.x & 31, i0 = lane * N, half = a.rope_dims >> 1;
    const long long task = (long long)blockIdx.x * PREP_WARPS + (threadIdx.x >> 5);
    const int t = (int)(task / plan.chunks), chunk = (int)(task - (long long)t * plan.chunks);
    if (t >= a.ntok) return;
    const int hq = a.n_q_heads, hkv = a.n_kv_heads, nrows = hq + 2 * hkv;
    const int r0 = chunk * plan.rows, r1 = min(r0 + plan.rows, nrows);
    // The rows do not wait for the slot: a padding token's first ones are read
    // too, and dropped.
    const int slot = __ldg(a.slots + t);
    const int pos = __ldg(a.positions + t);
    const TI *q = static_cast<const TI *>(a.q_in) + t * a.q_stride + i0;
    const TI *k = static_cast<const TI *>(a.k_in) + t * a.k_stride + i0;
    const TI *v = static_cast<const TI *>(a.v_in) + t * a.v_stride + i0;
    Raw<N, TI> raw[BATCH];  // the next batch's rows, on their way
    auto fetch = [&](int r) {
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            const int row = min(r + j, nrows - 1);
            load_raw(raw[j], row < hq ? q + row * D : row < hq + hkv ? k + (row - hq) * D : v + (row - hq - hkv) * D);
        }
    };
    fetch(r0);
    if (slot < 0 || slot >= a.cache_cells) {
        if (slot != -1 && lane == 0 && chunk == 0 && a.err) atomicOr(a.err, QSA_DEVERR_BAD_ID);
        return;
    }

    // cos and sin of this lane's dims.  Interleaved: a pair's two dims are in
    // one lane.  Halves: the partner dims are `sh` lanes away and turn by the
    // same angles, so each of the two lanes works out half of them.
    constexpr int NA = INTER ? N / 2 : N;
    const bool turns = i0 < 2 * half, first = INTER || i0 < half;
    const int sh = half / N, from = (first ? lane + sh : lane - sh) & 31;
    float2 cs[NA];
    if (half > 0 && r0 < hq + hkv) {
        const int a0 = INTER ? i0 >> 1 : first ? i0 : i0 - half + N / 2;
        float2 mine[N / 2];
#pragma unroll
        for (int e = 0; e < N / 2; ++e)
            mine[e] = cos_sin_of(pos, turns ? __ldg(a.inv_freq + a0 + e) : 0.0f, a.rope_mscale);
        if constexpr (INTER) {
#pragma unroll
            for (int e = 0; e < NA; ++e) cs[e] = mine[e];
        } else {
#pragma unroll
            for (int e = 0; e < N / 2; ++e) {
                const float2 o = make_float2(__shfl_sync(0xffffffffu, mine[e].x, from), __shfl_sync(0xffffffffu, mine[e].y, from));
                cs[e] = first ? mine[e] : o;
                cs[e + N / 2] = first ? o : mine[e];
            }
        }
    }

    const float *w = nullptr;
    float wv[N];
    auto weights = [&](const float *wr) {  // once for a run's rows of one kind
        if (w == wr) return;
        Raw<N, float> u;
        load_raw(u, wr + i0);
#pragma unroll
        for (int e = 0; e < N; ++e) wv[e] = u.e[e];
        w = wr;
    };
    float x[BATCH][N], ss[BATCH];
    auto squares = [&] {
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int e = 0; e < N; e += 2) s2 = __ffma2_rn(make_float2(x[j][e], x[j][e + 1]), make_float2(x[j][e], x[j][e + 1]), s2);
            ss[j] = s2.x + s2.y;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int j = 0; j < BATCH; ++j) ss[j] += __shfl_xor_sync(0xffffffffu, ss[j], o);
    };
    auto norm = [&](int j) {
        const float rs = rsqrtf(ss[j] * (1.0f / D) + a.eps);  // off by at most 2^-22
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            float2 y = __fmul2_rn(make_float2(x[j][e], x[j][e + 1]), make_float2(rs, rs));
            y = __fmul2_rn(y, make_float2(wv[e], wv[e + 1]));
            x[j][e] = y.x;
            x[j][e + 1] = y.y;
        }
    };
    auto turn = [&](int j) {
        if constexpr (INTER) {
            if (turns) {
#pragma unroll
                for (int e = 0; e < N; e += 2) {
                    const float y0 = x[j][e], y1 = x[j][e + 1];
                    x[j][e] = y0 * cs[e / 2].x - y1 * cs[e / 2].y;
                    x[j][e + 1] = y1 * cs[e / 2].x + y0 * cs[e / 2].y;
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float o = __shfl_sync(0xffffffffu, x[j][e], from);
                if (turns) x[j][e] = fmaf(x[j][e], cs[e].x, first ? -o * cs[e].y : o * cs[e].y);
            }
        }
    };
    auto take = [&](int r) {  // batch r's rows; the next one's loads start
#pragma unroll
        for (int j = 0; j < BATCH; ++j)
#pragma unroll
            for (int e = 0; e < N; ++e) x[j][e] = to_float(raw[j].e[e]);
        if (r + BATCH < r1) fetch(r + BATCH);
    };

    // Query rows by whole batches, without the branches of the mixed ones below.
    int r = r0;
    TO *out = static_cast<TO *>(a.q_out) + (size_t)t * hq * D + i0;
    if (a.q_norm_w && r + BATCH <= min(r1, hq)) weights(a.q_norm_w);
    for (; r + BATCH <= min(r1, hq); r += BATCH) {
        take(r);
        if (a.q_norm_w) {
            squares();
#pragma unroll
            for (int j = 0; j < BATCH; ++j) norm(j);
        }
        if (half > 0) {
#pragma unroll
            for (int j = 0; j < BATCH; ++j) turn(j);
        }
#pragma unroll
        for (int j = 0; j < BATCH; ++j)
            if (QSA_IN(((size_t)t * hq + r + j) * D + D - 1, (size_t)a.ntok * hq * D)) store_elems<N>(out + (r + j) * D, x[j]);
    }
    for (; r < r1; r += BATCH) {
        take(r);
        if (r < hq + hkv) squares();
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            const int row = r + j;
            if (row >= r1) break;
            const bool is_q = row < hq, is_v = row >= hq + hkv;
            if (!is_v) {
                const float *wr = is_q ? a.q_norm_w : a.k_norm_w;
                if (wr) {
                    weights(wr);
                    norm(j);
                }
                if (half > 0) turn(j);
            }
            if (is_q) {
                if (QSA_IN(((size_t)t * hq + row) * D + D - 1, (size_t)a.ntok * hq * D)) store_elems<N>(out + row * D, x[j]);
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
            const bool fine = sc > 0.0f && sc <= 65504.0f;
            const float inv = fine ? __frcp_rn(sc) : 0.0f;
#pragma unroll
            for (int e = 0; e < N; e += 4) {
                uint32_t b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) b[i] = fine ? code_of(x[j][e + i], sc, inv) : 0u;
                code[e / 4] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
            }
            int8_t *dst = (is_v ? a.vq : a.kq) + cell * D + i0;
            if constexpr (N == 4)
                *reinterpret_cast<uint32_t *>(dst) = code[0];
            else
                *reinterpret_cast<uint2 *>(dst) = make_uint2(code[0], code[1]);
            if ((lane & 7) == 0) (is_v ? a.vsc : a.ksc)[cell * 4 + (lane >> 3)] = __half_as_ushort(sch);
        }
    }
}

// Gather: bound by its traffic, 2 (D + 8) bytes read and 2 D elements written
// per (cell, KV head).  A thread takes sixteen dims of one (cell, KV head), of
// both K and V, so that a warp reads and writes whole rows.  A block takes
// ids_per_block whole ids, so that an item's id and place need 32-bit
// arithmetic only.  240 K cells of 2 heads of 256 to bf16, 744 MB: 119 us, 6.3 TB/s
// (256 threads a block 125 us, 64 119 us).
constexpr int GATHER_THREADS = 128;

struct GatherPlan {
    int per_id, ids_per_block;
    uint32_t magic;  // ceil(2^32 / per_id): item * magic >> 32 is item / per_id for the at most 1024 items; 0 for one id
};

template <class T>
__global__ void __launch_bounds__(GATHER_THREADS) paged_gather_kernel(const qsa_paged_gather_args a, const GatherPlan g) {
    wait_for_previous_grid();
    allow_dependent_launch();
    const int per_row = a.head_dim / 16, shift = a.head_dim == 128 ? 3 : 4, page_shift = 31 - __clz(a.page_size | 1);
    const long long id0 = (long long)blockIdx.x * g.ids_per_block;
    const int items = (int)(a.n_ids - id0 < g.ids_per_block ? a.n_ids - id0 : g.ids_per_block) * g.per_id;
    for (int it = threadIdx.x; it < items; it += GATHER_THREADS) {
        const int id = (int)__umulhi((uint32_t)it, g.magic), in_id = it - id * g.per_id;
        int cell = __ldg(a.ids + id0 + id);
        bool bad = cell < -1;
        if (cell >= 0 && a.page_table) {
            const int row = __ldg(a.rows + id0 + id), page = cell >> page_shift, in_page = cell & (a.page_size - 1);
            bad = row < 0 || row >= a.n_rows || page >= a.max_pages;
            const int e = bad ? -1 : __ldg(a.page_table + (size_t)row * a.max_pages + page);
            bad |= e < 0 || e > ((a.cache_cells - 1) >> page_shift);
            cell = bad ? -1 : (e << page_shift) + in_page;
        }
        if (cell >= a.cache_cells) {
            bad = true;
            cell = -1;
        }
        if (bad && in_id == 0 && a.err) atomicOr(a.err, QSA_DEVERR_BAD_ID);
        uint4 k = make_uint4(0u, 0u, 0u, 0u), v = k;
        uint16_t ks = 0, vs = 0;
        if (cell >= 0) {
            const int h = in_id >> shift, c = in_id & (per_row - 1);
            const size_t row = (size_t)cell * a.n_kv_heads + h;
            k = __ldg(reinterpret_cast<const uint4 *>(a.kq + row * a.head_dim) + c);
            v = __ldg(reinterpret_cast<const uint4 *>(a.vq + row * a.head_dim) + c);
            ks = __ldg(a.ksc + row * 4 + (c >> (shift - 2)));
            vs = __ldg(a.vsc + row * 4 + (c >> (shift - 2)));
        }
        const size_t at = (size_t)(id0 + id) * a.n_kv_heads * a.head_dim + in_id * 16;
        if (!QSA_IN(at + 15, (size_t)a.n_ids * a.n_kv_heads * a.head_dim)) continue;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float f = __half2float(__ushort_as_half(i ? vs : ks));
            const uint32_t w[4] = {i ? v.x : k.x, i ? v.y : k.y, i ? v.z : k.z, i ? v.w : k.w};
            T *dst = static_cast<T *>(i ? a.v_out : a.k_out) + at;
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = (float)(int8_t)(w[2 * p + (e >> 2)] >> (8 * (e & 3))) * f;
                store_elems<8>(dst + 8 * p, y);
            }
        }
    }
}

template <int D, class TI, class TO>
cudaError_t prep_run(const qsa_paged_prep_args &a, cudaStream_t s) {
    // One run per token, or more while there are fewer runs than 24 warps per SM.
    const int nrows = a.n_q_heads + 2 * a.n_kv_heads;
    const long long want = (152 * 24 + a.ntok - 1) / a.ntok;
    PrepPlan p;
    p.rows = (int)((nrows + want - 1) / want);
    p.rows += p.rows & 1;
    p.chunks = (nrows + p.rows - 1) / p.rows;
    const long long tasks = (long long)a.ntok * p.chunks;
    const dim3 grid((unsigned)((tasks + PREP_WARPS - 1) / PREP_WARPS)), block(PREP_WARPS * 32);
    return a.interleaved ? launch_dependent(paged_prep_kernel<D, true, TI, TO>, grid, block, 0, s, a, p)
                         : launch_dependent(paged_prep_kernel<D, false, TI, TO>, grid, block, 0, s, a, p);
}

template <int D, class TI>
cudaError_t prep_to(const qsa_paged_prep_args &a, cudaStream_t s) {
    return a.q_out_dtype == QSA_F16 ? prep_run<D, TI, __half>(a, s) : prep_run<D, TI, __nv_bfloat16>(a, s);
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
    GatherPlan g;
    g.per_id = a.n_kv_heads * (a.head_dim / 16);
    // Up to four rounds of a block's threads (two 120 us, eight 128 us), fewer
    // while that leaves blocks out (321 cells: 5.3 us with three blocks, 1.9 us
    // with one per id); a power of two (14.5 K cells of 4 heads of 128: 9.3 us with
    // 16 ids, 12.5 us with 12).
    const int most = 4 * GATHER_THREADS / g.per_id;
    g.ids_per_block = 1;
    while (2 * g.ids_per_block <= most && (long long)g.ids_per_block * 1216 < a.n_ids) g.ids_per_block *= 2;
    g.magic = g.ids_per_block == 1 ? 0u : (uint32_t)(((1ull << 32) + g.per_id - 1) / g.per_id);
    const dim3 grid((unsigned)(((long long)a.n_ids + g.ids_per_block - 1) / g.ids_per_block)), block(GATHER_THREADS);
    return a.out_dtype == QSA_F32   ? launch_dependent(paged_gather_kernel<float>, grid, block, 0, s, a, g)
           : a.out_dtype == QSA_F16 ? launch_dependent(paged_gather_kernel<__half>, grid, block, 0, s, a, g)
                                    : launch_dependent(paged_gather_kernel<__nv_bfloat16>, grid, block, 0, s, a, g);
}

}  // namespace qsa

QSA_DEFINE_CHECK_READER(take_check_word_paged_prep)
