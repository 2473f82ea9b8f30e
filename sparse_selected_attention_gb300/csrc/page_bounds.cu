// qsa_page_bounds: the largest and smallest key per dim of the pages that new
// tokens are in, as codes and scales rounded outwards.
//
//   hi_d = max_c s_c k_cd,  scale = roundup16(max_d |hi_d| / 127),  code = ceil(hi_d / scale)
//
// A key s_c k_cd has 19 bits and is exact in fp32; a division rounded up to fp32
// and then to fp16 gives the value rounded up once, as the coarser numbers are fp32
// numbers too.  So the results are exact by definition.
//
// It is bound by reading the keys.  A warp takes a page of one KV head: 16 codes a
// lane, four cells (of 128 dims) or two at a time, maxima and minima in registers,
// exchanged across the lanes of other cells by halves.  The pages that the rows' new
// tokens are in are shared out evenly.  8 prompts of 29 to 30 K cells, 2 heads of 256, 125
// MB of keys: 42.9 us, 2.9 TB/s, at 56 % of the issue slots (a code's conversion, product
// and two comparisons; 81 us before loads went two batches ahead).  One new token of each
// of 61 rows, 4 heads of 128: 3 us of latency.
#include <math_constants.h>

#include "check.cuh"
#include "page_share.cuh"
#include "qsa_internal.h"
#include "tc_common.cuh"

namespace qsa {
namespace {

constexpr int WARPS = 4, THREADS = 32 * WARPS, CTAS_PER_SM = 5;
constexpr int BATCH = 4;  // loads of a lane on their way, twice

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
    float d;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// The pages of row r that are to be written: n from `first` on.
struct Span {
    int first, n, len;
};
__device__ __forceinline__ Span span_of(const qsa_page_bounds_args &a, int r, bool &bad) {
    const int len = __ldg(a.seq_lens + r), most = a.max_pages * a.page_size;
    Span s{0, 0, min(max(len, 0), most)};
    int fresh = s.len;
    if (a.n_new) {
        const int n = __ldg(a.n_new + r);
        fresh = min(max(n, 0), s.len);
        bad |= n != fresh;
    }
    bad |= len != s.len;
    const int shift = 31 - __clz(a.page_size);
    if (fresh > 0) {
        s.first = (s.len - fresh) >> shift;
        s.n = ((s.len - 1) >> shift) + 1 - s.first;
    }
    return s;
}

// Codes 0, 1 (or 2, 3) of w as floats.
__device__ __forceinline__ float2 codes2(uint32_t w, bool high) {
    const uint32_t x = w ^ 0x80808080u;  // code + 128, in the mantissa of 2^23
    const float2 f = make_float2(__uint_as_float(tc::prmt(x, 0x4B000000u, high ? 0x7542 : 0x7540)),
                                 __uint_as_float(tc::prmt(x, 0x4B000000u, high ? 0x7543 : 0x7541)));
    return __fadd2_rn(f, make_float2(-8388736.0f, -8388736.0f));
}

// One bound of a page and head: v [K dims of a lane], top the largest |v| of their
// quarter.  x / s rounded upwards to a whole number c is where c s >= x > (c - 1) s;
// both products have 18 bits, so the reciprocal's rounding is put right exactly.
template <int K>
__device__ __forceinline__ void write_bound(const float (&v)[K], float top, bool nan, bool up, int8_t *q, uint16_t *sc, bool one) {
    const __half scale = nan ? __ushort_as_half(0x7E00) : __float2half_ru(__fdiv_ru(top, 127.0f));
    const float s = __half2float(scale), inv = __frcp_rn(s);
    uint32_t w[K / 4];
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const float x = up ? v[i] : -v[i];  // floor(x / s) = -ceil(-x / s)
        float c = ceilf(x * inv);
        c += c * s < x ? 1.0f : (c - 1.0f) * s >= x ? -1.0f : 0.0f;
        const uint32_t code = s > 0.0f ? (uint32_t)(int)(up ? c : -c) & 0xFFu : 0u;
        w[i / 4] = i % 4 ? w[i / 4] | code << (8 * (i % 4)) : code;
    }
    if constexpr (K == 4)
        *reinterpret_cast<uint32_t *>(q) = w[0];
    else
        *reinterpret_cast<uint2 *>(q) = make_uint2(w[0], w[1]);
    if (one) *sc = __half_as_ushort(scale);
}

template <int S>
__global__ void __launch_bounds__(THREADS, CTAS_PER_SM) page_bounds_kernel(const qsa_page_bounds_args a) {
    constexpr int D = 128 * S, LANES = 8 * S, CELLS = 32 / LANES;  // lanes of a cell's row, cells at a time
    const int lane = threadIdx.x & 31, c16 = lane % LANES, sub = lane / LANES;
    const int quarter = c16 / (2 * S), page_shift = 31 - __clz(a.page_size), hkv = a.n_kv_heads;
    __shared__ ShareSmem<WARPS> found;
    wait_for_previous_grid();
    allow_dependent_launch();
    bool bad = false;
    // This block's pages, of all heads; its warps take the (page, head) pairs in turn.
    int r, at, pages;
    find_share(found, a.n_rows, blockIdx.x, gridDim.x, 1, [&](int i) { return span_of(a, i, bad).n; }, r, at, pages);
    long long left = (long long)pages * hkv - (threadIdx.x >> 5);  // pairs from this warp's first on
    if (left > 0) {
        Span s = span_of(a, r, bad);
        int j = at, head = threadIdx.x >> 5;
        auto settle = [&] {
            while (head >= hkv) {
                head -= hkv;
                for (++j; j == s.n; j = 0) s = span_of(a, ++r, bad);  // there is a next row with pages
            }
        };
        settle();
        for (;;) {
            const int lp = s.first + j, page = __ldg(a.page_table + (size_t)r * a.max_pages + lp);
            const int filled = min(a.page_size, s.len - (lp << page_shift));
            const bool there = page >= 0 && page < a.n_pages;
            bad |= !there;
            if (there) {
                const size_t row0 = ((size_t)page << page_shift) * hkv + head;  // of the first cell, in rows of D
                float hi[16], lo[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    hi[i] = -CUDART_INF_F;
                    lo[i] = CUDART_INF_F;
                }
                bool nan = false;
                uint4 w[2][BATCH] = {};
                uint16_t sc[2][BATCH] = {};
                auto load = [&](int buf, int c0) {
#pragma unroll
                    for (int i = 0; i < BATCH; ++i) {
                        // Cells behind the last stand for it: twice counts once.
                        const size_t row = row0 + (size_t)min(c0 + i * CELLS + sub, filled - 1) * hkv;
                        if (QSA_IN(row, (size_t)a.n_pages * a.page_size * hkv)) {
                            w[buf][i] = __ldg(reinterpret_cast<const uint4 *>(a.kq + row * D) + c16);
                            sc[buf][i] = __ldg(a.ksc + row * 4 + quarter);
                        }
                    }
                };
                auto fold = [&](int buf) {  // two cells' values of a dim at a time
#pragma unroll
                    for (int i = 0; i < BATCH; i += 2) {
                        nan |= (sc[buf][i] & 0x7C00u) == 0x7C00u || (sc[buf][i + 1] & 0x7C00u) == 0x7C00u;
                        const float f0 = __half2float(__ushort_as_half(sc[buf][i])), f1 = __half2float(__ushort_as_half(sc[buf][i + 1]));
                        const uint32_t x0[4] = {w[buf][i].x, w[buf][i].y, w[buf][i].z, w[buf][i].w};
                        const uint32_t x1[4] = {w[buf][i + 1].x, w[buf][i + 1].y, w[buf][i + 1].z, w[buf][i + 1].w};
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float2 v0 = __fmul2_rn(codes2(x0[e / 2], e & 1), make_float2(f0, f0));
                            const float2 v1 = __fmul2_rn(codes2(x1[e / 2], e & 1), make_float2(f1, f1));
                            hi[2 * e] = max3(hi[2 * e], v0.x, v1.x);
                            hi[2 * e + 1] = max3(hi[2 * e + 1], v0.y, v1.y);
                            lo[2 * e] = min3(lo[2 * e], v0.x, v1.x);
                            lo[2 * e + 1] = min3(lo[2 * e + 1], v0.y, v1.y);
                        }
                    }
                };
                load(0, 0);
                for (int c0 = 0; c0 < filled; c0 += 2 * CELLS * BATCH) {
                    if (c0 + CELLS * BATCH < filled) load(1, c0 + CELLS * BATCH);
                    fold(0);
                    if (c0 + CELLS * BATCH >= filled) break;
                    if (c0 + 2 * CELLS * BATCH < filled) load(0, c0 + 2 * CELLS * BATCH);
                    fold(1);
                }
                // Across the lanes of other cells: each step a lane keeps half of its dims.
                constexpr int K = 4 * S;
                float h[8], l[8];
                const bool up16 = lane & 16;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float oh = __shfl_xor_sync(0xffffffffu, up16 ? hi[i] : hi[i + 8], 16);
                    const float ol = __shfl_xor_sync(0xffffffffu, up16 ? lo[i] : lo[i + 8], 16);
                    h[i] = fmaxf(up16 ? hi[i + 8] : hi[i], oh);
                    l[i] = fminf(up16 ? lo[i + 8] : lo[i], ol);
                }
                float vh[K], vl[K];
                int d0 = 16 * c16 + (up16 ? 8 : 0);
                if constexpr (S == 1) {
                    const bool up8 = lane & 8;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float oh = __shfl_xor_sync(0xffffffffu, up8 ? h[i] : h[i + 4], 8);
                        const float ol = __shfl_xor_sync(0xffffffffu, up8 ? l[i] : l[i + 4], 8);
                        vh[i] = fmaxf(up8 ? h[i + 4] : h[i], oh);
                        vl[i] = fminf(up8 ? l[i + 4] : l[i], ol);
                    }
                    d0 += up8 ? 4 : 0;
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        vh[i] = h[i];
                        vl[i] = l[i];
                    }
                }
                // The quarter's lanes: 2 S neighbours, and those of other cells.
                float th = 0.0f, tl = 0.0f;
#pragma unroll
                for (int i = 0; i < K; ++i) {
                    th = fmaxf(th, fabsf(vh[i]));
                    tl = fmaxf(tl, fabsf(vl[i]));
                }
                int n = nan;
#pragma unroll
                for (int o = 1; o < 32; o = o == S ? LANES : 2 * o) {
                    th = fmaxf(th, __shfl_xor_sync(0xffffffffu, th, o));
                    tl = fmaxf(tl, __shfl_xor_sync(0xffffffffu, tl, o));
                    n |= __shfl_xor_sync(0xffffffffu, n, o);
                }
                const size_t out = (size_t)page * hkv + head;
                const bool one = sub == 0 && c16 % (2 * S) == 0;
                if (QSA_IN(out, (size_t)a.n_pages * hkv)) {
                    write_bound<K>(vh, th, n, true, a.hi_q + out * D + d0, a.hi_sc + out * 4 + quarter, one);
                    write_bound<K>(vl, tl, n, false, a.lo_q + out * D + d0, a.lo_sc + out * 4 + quarter, one);
                }
            }
            if ((left -= WARPS) <= 0) break;
            head += WARPS;
            settle();
        }
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0 && a.err) atomicOr(a.err, QSA_DEVERR_BAD_ID);
}

template <int S>
cudaError_t launch(const qsa_page_bounds_args &a, cudaStream_t s) {
    const long long most = (long long)a.n_rows * a.max_pages;
    const int grid = (int)(most < 152 * CTAS_PER_SM ? most : 152 * CTAS_PER_SM);
    return launch_dependent(page_bounds_kernel<S>, dim3(grid), dim3(THREADS), 0, s, a);
}

}  // namespace

cudaError_t launch_page_bounds(const qsa_page_bounds_args &a, cudaStream_t s) {
    return a.head_dim == 128 ? launch<1>(a, s) : launch<2>(a, s);
}

}  // namespace qsa

QSA_DEFINE_CHECK_READER(take_check_word_page_bounds)
