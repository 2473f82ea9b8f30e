// qsa_paged_attn, rows that read one sequence together: the consecutive tokens
// of a draft window, each with its own length.
//
// Their heads, up to 128, are the M side of tcgen05 products over one pass of
// the cache, so a cell's codes are read and converted once for all of them.
// (Eight tokens x 12 heads over 30 K cells of 2 x 256 dims: row by row the
// cache would be read, and its 2 x 15 M codes converted, eight times.)
//
// A CTA takes tiles of 64 cells.  Warps 4-7 load a tile's codes (the next
// tile's loads are in flight meanwhile), convert them to fp16 and write them
// to shared memory, K as [64 cells][D] and V transposed as [D][64 cells], both
// K-major with the 128-byte swizzle; one of their threads issues
// S = Q K^T (128 x 64) and O += P V (128 x D).  Warps 0-3, a thread per head
// row, take S from tensor memory, do the softmax and write P as fp16 to shared
// memory.  S has two buffers, so the softmax of tile i runs beside the
// conversion of K i + 1 and V i.  Tiles are shared out over the chip and joined
// as in paged_attn.cu.  A tile is bound by the two halves' latency, some 1500
// cycles each, not by its 2 x 128 x 64 x 256 products.
//
// Scales.  K's are multiplied into the codes under a power of two per cell,
// 2^ek, that the softmax undoes (codes x scales then use fp16's range whatever
// the scales are); V's under 2^ev, so that a cell's largest scale is in [1, 2).
// The softmax works on s - ev: P = 2^(s - ev - m) is the weight of the scaled
// values, its running maximum m is one of weight x value, and the denominator
// adds P 2^ev.
#include "paged_attn.cuh"

namespace qsa {
namespace {

using namespace tc;

constexpr int M = GROUP_ROWS, N = 64;  // heads and cells of a tile
constexpr int THREADS = 256;

template <int S>
struct GroupShape {
    static constexpr int D = 128 * S, CTAS_PER_SM = S == 1 ? 2 : 1, MAX_CTAS = 152 * CTAS_PER_SM;
    static constexpr uint32_t TMEM_COLS = S == 1 ? 256 : 512, O_COL = 2 * N;  // S at 0 and N
    static constexpr uint32_t IDESC_S = idesc_f16(M, N, false, false), IDESC_O = idesc_f16(M, D, false, false);
};

// Everything of shared memory; tiles of 64 halves (128 bytes) a row, 16-byte
// unit u of row r at u ^ (r % 8).
template <int S>
struct GroupSmem {
    uint8_t q[2 * S][M * 128];  // per 64 dims
    uint8_t k[2 * S][N * 128];
    uint8_t v[128 * S * 128];   // a row per dim
    uint8_t p[M * 128];
    float kf[2][N], vb[2][N], vw[2][N];  // a cell's 2^-ek, -ev (-inf: not there), 2^ev
    float qinv[M];                       // 2^-e of a head's scaled query
    uint64_t s_full[2], p_full, pv_full, drain;
    long long scan[THREADS / 32];
    long long total, before;
    int t, tokens, tiles;  // the group in which the CTA's share starts
    int abort;
    uint32_t tmem;
};

__device__ __forceinline__ uint32_t unit_off(int r, int u) { return r * 128 + ((u ^ (r & 7)) << 4); }

// -floor(log2) of the largest |scale| of a cell, 0 where it is 0, infinite or NaN.
__device__ __forceinline__ int scale_exponent(uint2 sc) {
    const uint32_t m2 = __vmaxu2(sc.x & 0x7FFF7FFFu, sc.y & 0x7FFF7FFFu), m = max(m2 & 0xFFFFu, m2 >> 16);
    if (m == 0u || m >= 0x7C00u) return 0;
    return 127 - (int)(__float_as_uint(__half2float(__ushort_as_half((unsigned short)m))) >> 23);
}
// Scale `i` of a cell times 2^e, in both halves.
__device__ __forceinline__ __half2 scaled(uint2 sc, int i, int e) {
    const uint32_t w = i >> 1 ? sc.y : sc.x;
    const float f = __half2float(__ushort_as_half((unsigned short)(i & 1 ? w >> 16 : w & 0xFFFFu)));
    return __float2half2_rn(f * exp2i(e));
}
__device__ __forceinline__ uint32_t prod(uint32_t codes, __half2 f) {  // (1152 + code) pairs to code * f
    const uint32_t off = 0x64806480u;
    return h2u(__hmul2(__hsub2(u2h(codes), u2h(off)), f));
}
// Barrier of warps 4-7; whether all of them are fine.
__device__ __forceinline__ bool converters_agree(bool ok) {
    int r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.s32 p, %1, 0;\n barrier.cta.red.and.pred q, 1, 128, p;\n selp.s32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"((int)ok)
        : "memory");
    return r != 0;
}

// The group that starts at row t: its rows (0: none starts), and the tiles of
// its longest row.
__device__ __forceinline__ int group_at(const qsa_paged_attn_args &a, int t, int block, int &tiles, bool &bad) {
    const int row = __ldg(a.rows + t);
    tiles = 0;
    if ((t & (block - 1)) && __ldg(a.rows + t - 1) == row) return 0;
    int n = 1;
    while (t + n < a.n_tokens && ((t + n) & (block - 1)) && __ldg(a.rows + t + n) == row) ++n;
    if (n < GROUP_MIN) return 0;
    int most = 0, trow;
    for (int i = 0; i < n; ++i) most = max(most, row_len(a, t + i, trow, bad));
    tiles = max((most + N - 1) / N, 1);
    return n;
}

template <int S>
__global__ void __launch_bounds__(THREADS, GroupShape<S>::CTAS_PER_SM)
    paged_group_kernel(const qsa_paged_attn_args a, void *ws, int block) {
    using G = GroupShape<S>;
    constexpr int D = G::D;
    extern __shared__ __align__(1024) uint8_t raw[];
    GroupSmem<S> &sh = *reinterpret_cast<GroupSmem<S> *>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = a.n_q_heads / a.n_kv_heads, page_shift = 31 - __clz(a.page_size);
    const int kvh = blockIdx.x % a.n_kv_heads, range = blockIdx.x / a.n_kv_heads, ranges = gridDim.x / a.n_kv_heads;
    volatile int *abort = &sh.abort;
    if (tid == 0) {
        mbar_init(smem_u32(&sh.s_full[0]), 1);
        mbar_init(smem_u32(&sh.s_full[1]), 1);
        mbar_init(smem_u32(&sh.p_full), 128);
        mbar_init(smem_u32(&sh.pv_full), 1);
        mbar_init(smem_u32(&sh.drain), 1);
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    wait_for_previous_grid();
    allow_dependent_launch();
    const Work work(ws, G::MAX_CTAS, M);
    bool bad = false;

    // The groups' tiles, and where this CTA's share of them starts.
    int share, left;
    {
        const int run = (a.n_tokens + THREADS - 1) / THREADS;
        const int t0 = min(tid * run, a.n_tokens), t1 = min(t0 + run, a.n_tokens);
        long long mine = 0;
        for (int t = t0; t < t1; ++t) {
            int tiles;
            group_at(a, t, block, tiles, bad);
            mine += tiles;
        }
        long long s = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += u;
        }
        if (lane == 31) sh.scan[warp] = s;
        __syncthreads();
        long long total = 0, before = s - mine;
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < warp) before += sh.scan[w];
            total += sh.scan[w];
        }
        share = (int)max((total + ranges - 1) / ranges, 1ll);
        const long long x = (long long)share * range;
        if (x >= before && x < before + mine) {
            for (int t = t0;; ++t) {
                int tiles;
                const int n = group_at(a, t, block, tiles, bad);
                if (x < before + tiles) {
                    sh.t = t;
                    sh.tokens = n;
                    sh.tiles = tiles;
                    sh.before = before;
                    break;
                }
                before += tiles;
            }
        }
        left = (int)max(min((long long)share, total - x), 0ll);
        if (left == 0) {  // the same in all threads
            if (tid == 0) work.part[blockIdx.x] = Part{-1, 0, 0, 0};
            if (bad && blockIdx.x == 0 && a.err) atomicOr(a.err, QSA_DEVERR_BAD_ID);
            return;
        }
    }
    if (warp == 4) tmem_alloc(smem_u32(&sh.tmem), G::TMEM_COLS);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = sh.tmem;
    int t = sh.t, tokens = sh.tokens, tiles = sh.tiles;
    int i0 = (int)((long long)share * range - sh.before);
    Part part{-1, 0, 0, 0};
    int k = 0;  // tiles done: the barriers' phases
    bool ok = true, issued = false;

    for (bool first = true;; first = false) {
        // Segment: tiles i0 .. i1-1 of the group of `tokens` rows at t.
        const int i1 = min(tiles, i0 + left), rows = tokens * per;
        int trow, least = 0x7fffffff, most = 0;
        for (int i = 0; i < tokens; ++i) {
            const int len = row_len(a, t + i, trow, bad);
            least = min(least, len);
            most = max(most, len);
        }

        // The queries: a warp takes every eighth head row, four in flight.
        constexpr int E = 4 * S;  // elements per lane
        for (int m0 = warp; m0 < M; m0 += 32) {
            uint32_t x[4][E / 2];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int m = m0 + 8 * b;
                const size_t at = ((size_t)(t + m / per) * a.n_q_heads + (size_t)kvh * per + m % per) * D + lane * E;
#pragma unroll
                for (int e = 0; e < E / 2; ++e) x[b][e] = 0u;
                if (m < rows && QSA_IN(at + E - 1, (size_t)a.n_tokens * a.n_q_heads * D)) {
                    const uint16_t *src = static_cast<const uint16_t *>(a.q) + at;
                    if constexpr (S == 1)
                        *reinterpret_cast<uint2 *>(x[b]) = __ldg(reinterpret_cast<const uint2 *>(src));
                    else
                        *reinterpret_cast<uint4 *>(x[b]) = __ldg(reinterpret_cast<const uint4 *>(src));
                }
            }
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int m = m0 + 8 * b;
                int ex = 0;
                if (a.dtype != QSA_F16) {  // bf16 under a power of two that keeps it in the fp16 range
                    uint32_t top = 0u;
#pragma unroll
                    for (int e = 0; e < E / 2; ++e) top = __vmaxu2(top, x[b][e] & 0x7FFF7FFFu);
                    top = __reduce_max_sync(0xffffffffu, max(top & 0xFFFFu, top >> 16));
                    ex = head_sum_exponent(__uint_as_float(top << 16));
                    const float f = exp2i(ex);
#pragma unroll
                    for (int e = 0; e < E / 2; ++e)
                        x[b][e] = h2u(__floats2half2_rn(__uint_as_float(x[b][e] << 16) * f,
                                                        __uint_as_float(x[b][e] & 0xFFFF0000u) * f));
                }
                if (lane == 0) sh.qinv[m] = exp2i(-ex);
                const int d = lane * E;
                uint8_t *dst = sh.q[d >> 6] + unit_off(m, (d & 63) >> 3) + 2 * (d & 7);
                if constexpr (S == 1)
                    *reinterpret_cast<uint2 *>(dst) = *reinterpret_cast<const uint2 *>(x[b]);
                else
                    *reinterpret_cast<uint4 *>(dst) = *reinterpret_cast<const uint4 *>(x[b]);
            }
        }
        fence_async_smem();
        __syncthreads();

        if (warp >= 4) {
            // ---- loads, conversion, products ----
            const int ct = tid - 128, kc = ct & 63, kh = ct >> 6, vq = ct & 15, vd = ct >> 4;
            const int32_t *tab = a.page_table + (size_t)trow * a.max_pages;
            uint4 kw[4 * S], vw[4 * S];  // K: dims kh D/2 .. of cell kc; V: dims vd D/8 .. of cells 4 vq .. + 3
            uint2 ksc, kvs, vsc[4];
            int kpage, vpage;
            auto pages = [&](int i) {
                const int kj = (i * N + kc) >> page_shift, vj = (i * N + 4 * vq) >> page_shift;
                kpage = i < i1 && kj < a.max_pages ? __ldg(tab + kj) : -1;
                vpage = i < i1 && vj < a.max_pages ? __ldg(tab + vj) : -1;
            };
            auto cell_of = [&](int c, int page) -> long long {  // its (cell, KV head) row, or -1
                if (c >= most) return -1;
                if (page < 0 || page >= a.n_pages) {
                    bad = true;
                    return -1;
                }
                return ((((long long)page << page_shift) + (c & (a.page_size - 1))) * a.n_kv_heads) + kvh;
            };
            bool there;
            auto load_k = [&](int i) {
                const long long row = i < i1 ? cell_of(i * N + kc, kpage) : -1;
                there = row >= 0 && QSA_IN(row, (long long)a.n_pages * a.page_size * a.n_kv_heads);
                const uint4 *src = reinterpret_cast<const uint4 *>(a.kq + (there ? row * D + kh * (D / 2) : 0));
#pragma unroll
                for (int j = 0; j < 4 * S; ++j) kw[j] = there ? __ldg(src + j) : make_uint4(0u, 0u, 0u, 0u);
                ksc = there ? __ldg(reinterpret_cast<const uint2 *>(a.ksc + row * 4)) : make_uint2(0u, 0u);
                kvs = there ? __ldg(reinterpret_cast<const uint2 *>(a.vsc + row * 4)) : make_uint2(0u, 0u);
            };
            auto load_v = [&](int i) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const long long row = i < i1 ? cell_of(i * N + 4 * vq + c, vpage) : -1;
                    const bool in = row >= 0 && QSA_IN(row, (long long)a.n_pages * a.page_size * a.n_kv_heads);
                    const uint4 *src = reinterpret_cast<const uint4 *>(a.vq + (in ? row * D + vd * (D / 8) : 0));
#pragma unroll
                    for (int j = 0; j < S; ++j) vw[c * S + j] = in ? __ldg(src + j) : make_uint4(0u, 0u, 0u, 0u);
                    vsc[c] = in ? __ldg(reinterpret_cast<const uint2 *>(a.vsc + row * 4)) : make_uint2(0u, 0u);
                }
            };
            auto store_k = [&](int buf) {
                const int ek = scale_exponent(ksc);
                const __half2 f0 = scaled(ksc, 2 * kh, ek), f1 = scaled(ksc, 2 * kh + 1, ek);
#pragma unroll
                for (int j = 0; j < 4 * S; ++j) {
                    const uint32_t w[4] = {kw[j].x ^ 0x80808080u, kw[j].y ^ 0x80808080u, kw[j].z ^ 0x80808080u, kw[j].w ^ 0x80808080u};
                    const __half2 f = j >= 2 * S ? f1 : f0;
                    const int d = kh * (D / 2) + 16 * j;
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        uint4 o;
                        o.x = prod(prmt(w[2 * u], 0x64646464u, 0x4140), f);
                        o.y = prod(prmt(w[2 * u], 0x64646464u, 0x4342), f);
                        o.z = prod(prmt(w[2 * u + 1], 0x64646464u, 0x4140), f);
                        o.w = prod(prmt(w[2 * u + 1], 0x64646464u, 0x4342), f);
                        *reinterpret_cast<uint4 *>(sh.k[d >> 6] + unit_off(kc, ((d & 63) >> 3) + u)) = o;
                    }
                }
                if (kh == 0) {
                    const int ev = scale_exponent(kvs);
                    sh.kf[buf][kc] = exp2i(-ek);
                    sh.vb[buf][kc] = there ? -(float)ev : -CUDART_INF_F;
                    sh.vw[buf][kc] = exp2i(ev);
                }
            };
            auto store_v = [&] {
                __half2 f01, f23;
                {
                    float f[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) f[c] = __low2float(scaled(vsc[c], vd >> 1, scale_exponent(vsc[c])));
                    f01 = __floats2half2_rn(f[0], f[1]);
                    f23 = __floats2half2_rn(f[2], f[3]);
                }
#pragma unroll
                for (int j = 0; j < 4 * S; ++j) {  // four dims of the four cells
                    uint32_t w[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint4 &q4 = vw[c * S + j / 4];
                        w[c] = (j % 4 == 0 ? q4.x : j % 4 == 1 ? q4.y : j % 4 == 2 ? q4.z : q4.w) ^ 0x80808080u;
                    }
                    const uint32_t a01 = prmt(w[0], w[1], 0x5140), b01 = prmt(w[0], w[1], 0x7362);  // dims 0 1, 2 3
                    const uint32_t a23 = prmt(w[2], w[3], 0x5140), b23 = prmt(w[2], w[3], 0x7362);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t sel = e & 1 ? 0x4342u : 0x4140u;
                        const int d = vd * (D / 8) + 4 * j + e;
                        uint2 o;
                        o.x = prod(prmt(e < 2 ? a01 : b01, 0x64646464u, sel), f01);
                        o.y = prod(prmt(e < 2 ? a23 : b23, 0x64646464u, sel), f23);
                        *reinterpret_cast<uint2 *>(sh.v + unit_off(d, vq >> 1) + 8 * (vq & 1)) = o;
                    }
                }
            };
            auto issue_s = [&](int kk) {  // one thread
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint32_t off = (ks & 3) * 32;
                    mma_f16(tmem + (kk & 1) * N, sw128_kmajor(smem_u32(sh.q[ks >> 2]) + off),
                            sw128_kmajor(smem_u32(sh.k[ks >> 2]) + off), G::IDESC_S, ks ? 1u : 0u);
                }
                mma_commit(smem_u32(&sh.s_full[kk & 1]));
            };
            pages(i0);
            load_k(i0);
            load_v(i0);
            pages(i0 + 1);
            bool good = ok;
            store_k(k & 1);
            load_k(i0 + 1);
            fence_async_smem();
            good = converters_agree(good);
            if (good && ct == 0) {
                fence_after();
                issue_s(k);
                issued = true;
            }
            for (int i = i0; i < i1 && good; ++i, ++k) {
                // K of the next tile, once S of this one has been computed.
                if (i + 1 < i1) {
                    bool fine = mbar_wait_or_abort(smem_u32(&sh.s_full[k & 1]), (k >> 1) & 1, abort);
                    if (fine) store_k((k + 1) & 1);
                    fence_async_smem();
                    good = converters_agree(fine);
                    if (!good) break;
                    if (ct == 0) {
                        fence_after();
                        issue_s(k + 1);
                    }
                }
                // V of this tile, once the values of the one before are added.
                bool fine = k == 0 || mbar_wait_or_abort(smem_u32(&sh.pv_full), (k - 1) & 1, abort);
                if (fine) store_v();
                load_v(i + 1);  // vpage is the next tile's
                pages(i + 2);
                load_k(i + 2);
                fence_async_smem();
                good = converters_agree(fine);
                if (!good) break;
                fine = mbar_wait_or_abort(smem_u32(&sh.p_full), k & 1, abort);
                if (fine && ct == 0) {
                    fence_after();
#pragma unroll
                    for (int ks = 0; ks < N / 16; ++ks)
                        mma_f16(tmem + G::O_COL, sw128_kmajor(smem_u32(sh.p) + ks * 32), sw128_kmajor(smem_u32(sh.v) + ks * 32),
                                G::IDESC_O, i > i0 || ks ? 1u : 0u);
                    mma_commit(smem_u32(&sh.pv_full));
                }
                // The cells' factors are written two tiles on: not before all
                // know that the softmax of this one is done.
                good = converters_agree(fine);
            }
            ok = good;
        } else {
            // ---- softmax, a thread per head row ----
            const int m = tid;
            const bool mine = m < rows;
            const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
            const float sl2 = a.softmax_scale * LOG2E * sh.qinv[m];
            int len = 0, tr;
            if (mine) len = row_len(a, t + m / per, tr, bad);
            float ref = -CUDART_INF_F, l = 0.0f;
            bool good = ok;
            for (int i = i0; i < i1 && good; ++i, ++k) {
                good = __all_sync(0xffffffffu, mbar_wait_or_abort(smem_u32(&sh.s_full[k & 1]), (k >> 1) & 1, abort));
                if (!good) break;
                fence_after();
                float y[N];
#pragma unroll
                for (int c = 0; c < N / 16; ++c) {
                    uint32_t v[16];
                    tmem_ld16(lane_base + (k & 1) * N + 16 * c, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        asm volatile("" : "+r"(v[j]));  // not before the wait
                        y[16 * c + j] = __uint_as_float(v[j]);
                    }
                }
                const float *kf = sh.kf[k & 1], *vb = sh.vb[k & 1], *vw = sh.vw[k & 1];
                float top = -CUDART_INF_F;
#pragma unroll
                for (int j = 0; j < N; j += 2) {
                    const float2 f = *reinterpret_cast<const float2 *>(kf + j), b = *reinterpret_cast<const float2 *>(vb + j);
                    float2 s = __fmul2_rn(make_float2(y[j], y[j + 1]), f);
                    s = __ffma2_rn(s, make_float2(sl2, sl2), b);
                    y[j] = s.x;
                    y[j + 1] = s.y;
                }
                if ((i + 1) * N > least) {  // some row ends in this tile
#pragma unroll
                    for (int j = 0; j < N; ++j)
                        if (i * N + j >= len) y[j] = -CUDART_INF_F;
                }
#pragma unroll
                for (int j = 0; j < N; j += 2) top = max3(top, y[j], y[j + 1]);
                // The reference moves only when a tile exceeds it by 2^SLACK.
                const bool up = top > ref + SLACK;
                const float alpha = up ? ex2(ref - top) : 1.0f;
                ref = up ? top : ref;
                l *= alpha;
                // P's buffer and the values: the tile before must be done with them.
                if (k > 0) good = __all_sync(0xffffffffu, mbar_wait_or_abort(smem_u32(&sh.pv_full), (k - 1) & 1, abort));
                if (!good) break;
                if (i > i0 && __any_sync(0xffffffffu, up)) {
                    fence_after();
                    for (int c = 0; c < D / 16; ++c) {
                        uint32_t v[16];
                        tmem_ld16(lane_base + G::O_COL + 16 * c, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            asm volatile("" : "+r"(v[j]));
                            v[j] = __float_as_uint(__uint_as_float(v[j]) * alpha);
                        }
                        tmem_st16(lane_base + G::O_COL + 16 * c, v);
                    }
                    tmem_wait_st();
                }
                const float base = ref == -CUDART_INF_F ? 0.0f : -ref;
                float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int u = 0; u < N / 8; ++u) {
                    uint32_t h[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int c = 8 * u + 2 * j;
                        float2 p = __fadd2_rn(make_float2(y[c], y[c + 1]), make_float2(base, base));
                        p = make_float2(ex2(p.x), ex2(p.y));
                        sum = __ffma2_rn(p, *reinterpret_cast<const float2 *>(vw + c), sum);
                        h[j] = h2u(__floats2half2_rn(p.x, p.y));
                    }
                    *reinterpret_cast<uint4 *>(sh.p + unit_off(m, u)) = make_uint4(h[0], h[1], h[2], h[3]);
                }
                l += sum.x + sum.y;
                fence_async_smem();
                fence_before();
                mbar_arrive(smem_u32(&sh.p_full));
            }
            if (good && k > 0) good = __all_sync(0xffffffffu, mbar_wait_or_abort(smem_u32(&sh.pv_full), (k - 1) & 1, abort));
            if (good) {
                fence_after();
                const bool whole = i1 - i0 == tiles, none = ref == -CUDART_INF_F;
                const size_t at = (size_t)blockIdx.x * 2 + (first && i0 > 0 ? 0 : 1);
                const float w = whole ? (none ? 0.0f : 1.0f / l) : 1.0f;
                const size_t row = (size_t)(t + (mine ? m / per : 0)) * a.n_q_heads + (size_t)kvh * per + m % per;
                const bool put = mine && QSA_IN(row * D + D - 1, (size_t)a.n_tokens * a.n_q_heads * D);
                for (int c = 0; c < D / 16; ++c) {
                    uint32_t v[16];
                    tmem_ld16(lane_base + G::O_COL + 16 * c, v);
                    tmem_wait_ld();
                    float o[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        asm volatile("" : "+r"(v[j]));
                        o[j] = __uint_as_float(v[j]) * w;
                    }
                    if (!put) continue;
                    if (!whole) {
                        float4 *dst = reinterpret_cast<float4 *>(work.o + (at * M + m) * D + 16 * c);
#pragma unroll
                        for (int j = 0; j < 4; ++j) dst[j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                        continue;
                    }
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        const size_t oi = row * D + 16 * c + j;
                        float2 y2 = make_float2(o[j], o[j + 1]);
                        if (a.gate) {
                            const float2 gate = __ldg(reinterpret_cast<const float2 *>(a.gate + oi));
                            y2 = make_float2(gated(y2.x, gate.x), gated(y2.y, gate.y));
                        }
                        store_out(a, oi, y2);
                    }
                }
                if (mine) {
                    if (!whole)
                        *reinterpret_cast<float2 *>(work.ml + (at * M + m) * 2) = make_float2(ref, l);
                    else if (a.lse)
                        a.lse[row] = none ? ref : (ref + log2f(l)) * LN2;
                }
                fence_before();  // O is overwritten by the next segment
            }
            ok = good;
        }
        if (i1 - i0 < tiles && i0 == 0) part = Part{t, 1 + (tiles - i1 + share - 1) / share, tokens, 0};
        left -= i1 - i0;
        if (!__syncthreads_and(ok)) {
            ok = false;
            break;
        }
        if (left <= 0) break;
        i0 = 0;
        do {
            t += tokens;
            tokens = 1;
            const int n = group_at(a, t, block, tiles, bad);
            if (n) tokens = n;
        } while (tiles == 0);
    }

    // Products issued before a time-out are complete before tensor memory is freed.
    if (issued) {
        mma_commit(smem_u32(&sh.drain));
        if (!mbar_wait_bounded(smem_u32(&sh.drain), 0, DRAIN_LIMIT)) ok = false;
    }
    fence_before();
    __syncthreads();
    if (__any_sync(0xffffffffu, bad) && lane == 0 && a.err) atomicOr(a.err, QSA_DEVERR_BAD_ID);
    if (tid == 0) {
        if (!ok && a.err) atomicOr(a.err, QSA_DEVERR_TIMEOUT);
        work.part[blockIdx.x] = ok ? part : Part{-1, 0, 0, 0};
    }
    if (warp == 4) {
        fence_after();
        tmem_dealloc(tmem, G::TMEM_COLS);
    }
}

template <int S>
cudaError_t launch(const qsa_paged_attn_args &a, void *ws, cudaStream_t s) {
    using G = GroupShape<S>;
    const int per = a.n_q_heads / a.n_kv_heads, ranges = G::MAX_CTAS / a.n_kv_heads > 1 ? G::MAX_CTAS / a.n_kv_heads : 1;
    const int smem = (int)sizeof(GroupSmem<S>), grid = ranges * a.n_kv_heads;
    cudaError_t e = cudaFuncSetAttribute(paged_group_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess)
        e = launch_dependent(paged_group_kernel<S>, dim3(grid), dim3(THREADS), smem, s, a, ws, group_block(per));
    return e == cudaSuccess ? launch_join<S>(a, ws, G::MAX_CTAS, M, grid, s) : e;
}

}  // namespace

size_t paged_group_workspace_bytes(int head_dim) {
    return head_dim == 128 ? Work::bytes(GroupShape<1>::MAX_CTAS, M, 128) : Work::bytes(GroupShape<2>::MAX_CTAS, M, 256);
}

cudaError_t launch_paged_group(const qsa_paged_attn_args &a, void *ws, cudaStream_t s) {
    return a.head_dim == 128 ? launch<1>(a, ws, s) : launch<2>(a, ws, s);
}

}  // namespace qsa

QSA_DEFINE_CHECK_READER(take_check_word_paged_group)
