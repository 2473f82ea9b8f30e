// qsa_paged_attn, rows that read one sequence together: the consecutive tokens
// of a draft window, each with its own length.
//
// Their heads, up to 128, are the M side of tcgen05 products over one pass of
// the cache, so a cell's codes are read and converted once for all of them.
// (Eight tokens x 12 heads over 30 K cells of 2 x 256 dims: row by row the
// cache would be read, and its 2 x 15 M codes converted, eight times.)
//
// A CTA takes tiles of 64 cells.  Warps 4-7 load a tile's K and warps 8-11 its
// V (the next tile's loads are in flight meanwhile), convert the codes to fp16
// and write them to shared memory as [64 cells][D], 64 dims to a 128-byte row
// with the swizzle: K-major for S = Q K^T (128 x 64), and read transposed
// (N-major) for O += P V (128 x D).  One thread of warp 12 issues the products.
// Warps 0-3, a thread per head row, take S from tensor memory, do the softmax
// and write P as fp16 to shared memory.  The roles hand tiles over by
// mbarriers (warp 13 provides the cells' factors): S has two buffers, so the softmax of tile i runs beside the
// conversions of K i + 1 and V i.  Tiles are shared out over the chip and joined
// as in paged_attn.cu.  A tile is bound by the roles' latency, not by its
// 2 x 128 x 64 x 256 products.
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
constexpr int CONVERTERS = 128;  // threads each for K and V
constexpr int THREADS = 128 + 2 * CONVERTERS + 64;
constexpr int MIN_TILES = 6;     // of a share: a partial of 128 rows costs as much as some tiles

template <int S>
struct GroupShape {
    static constexpr int D = 128 * S;
    static constexpr uint32_t TMEM_COLS = S == 1 ? 256 : 512, O_COL = 2 * N;  // S at 0 and N
    static constexpr uint32_t IDESC_S = idesc_f16(M, N, false, false), IDESC_O = idesc_f16(M, D, false, true);
};

// Everything of shared memory; tiles of 64 halves (128 bytes) a row, 16-byte
// unit u of row r at u ^ (r % 8).
template <int S>
struct GroupSmem {
    uint8_t q[2 * S][M * 128];  // per 64 dims; from here on also the values at the end of a segment, fp32 [M][D]
    uint8_t k[2 * S][N * 128];
    uint8_t v[2 * S][N * 128];
    uint8_t p[M * 128];
    alignas(16) float kf[3][N], vb[3][N], vw[3][N];  // a cell's 2^-ek, -ev (-inf: not there), 2^ev
    float qinv[M];                       // 2^-e of a head's scaled query
    uint64_t k_full, v_full, s_full[2], p_full, pv_full, drain;
    long long scan[THREADS / 32];
    long long before;  // tiles before the group at t, in which the CTA's share starts
    int t;
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
// Scale i of a cell times 2^e, in both halves.
__device__ __forceinline__ __half2 scaled(uint2 sc, int i, int e) {
    const uint32_t w = i >> 1 ? sc.y : sc.x;
    const float f = __half2float(__ushort_as_half((unsigned short)(i & 1 ? w >> 16 : w & 0xFFFFu)));
    return __float2half2_rn(f * exp2i(e));
}
__device__ __forceinline__ uint32_t prod(uint32_t codes, __half2 f) {  // (1152 + code) pairs to code * f
    const uint32_t off = 0x64806480u;
    return h2u(__hmul2(__hsub2(u2h(codes), u2h(off)), f));
}
// The group that starts at row t, looked up by a warp: its rows (0: none
// starts), and the shortest and longest length.
struct Group {
    int rows, least, most, trow;
    __device__ __forceinline__ int tiles() const { return rows ? max((most + N - 1) / N, 1) : 0; }
};
__device__ __forceinline__ Group group_at(const qsa_paged_attn_args &a, int t, int block, bool &bad) {
    const int lane = threadIdx.x & 31, row = __ldg(a.rows + t);
    Group g{0, 0x7fffffff, 0, 0};
    if ((t & (block - 1)) && __ldg(a.rows + t - 1) == row) return g;
    const int end = min(a.n_tokens, (t | (block - 1)) + 1);
    int n = 0, least = 0x7fffffff, most = 0;
    for (bool more = true; more && t + n < end;) {
        const int u = t + n + lane;
        int trow, len = 0;
        const bool same = u < end && __ldg(a.rows + u) == row;
        if (u < end) len = row_len(a, u, trow, bad);
        const unsigned m = __ballot_sync(0xffffffffu, same);
        const int k = m == 0xffffffffu ? 32 : __ffs(~m) - 1;  // rows that go on with the run
        if (lane < k) {
            least = min(least, len);
            most = max(most, len);
        }
        n += k;
        more = k == 32;
    }
    if (n < GROUP_MIN) return g;
    g.rows = n;
    g.least = __reduce_min_sync(0xffffffffu, least);
    g.most = __reduce_max_sync(0xffffffffu, most);
    g.trow = row >= 0 && row < a.n_rows ? row : 0;
    return g;
}

template <int S>
__global__ void __launch_bounds__(THREADS, 1)
    paged_group_kernel(const qsa_paged_attn_args a, void *ws, int block) {
    using G = GroupShape<S>;
    constexpr int D = G::D;
    extern __shared__ __align__(1024) uint8_t raw[];
    GroupSmem<S> &sh = *reinterpret_cast<GroupSmem<S> *>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = a.n_q_heads / a.n_kv_heads, page_shift = 31 - __clz(a.page_size);
    const uint32_t per_inv = 65536u / per + 1;
    const int kvh = blockIdx.x % a.n_kv_heads, range = blockIdx.x / a.n_kv_heads, ranges = gridDim.x / a.n_kv_heads;
    volatile int *abort = &sh.abort;
    if (tid == 0) {
        mbar_init(smem_u32(&sh.s_full[0]), 1);
        mbar_init(smem_u32(&sh.s_full[1]), 1);
        mbar_init(smem_u32(&sh.k_full), CONVERTERS + 32);
        mbar_init(smem_u32(&sh.v_full), CONVERTERS);
        mbar_init(smem_u32(&sh.p_full), 128);
        mbar_init(smem_u32(&sh.pv_full), 1);
        mbar_init(smem_u32(&sh.drain), 1);
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    wait_for_previous_grid();
    allow_dependent_launch();
    const Work work(ws, MAX_GROUP_PARTS, M);
    bool bad = false;

    // The groups' tiles, and where this CTA's share of them starts: rows and
    // lengths go to shared memory a chunk of whole blocks at a time, and the
    // thread of a row in which a group starts adds it up there.
    int share, left;
    {
        constexpr int CHUNK = 384;  // a multiple of any block
        static_assert(CHUNK <= THREADS && CHUNK % M == 0, "a thread per row");
        int *srow = reinterpret_cast<int *>(sh.q), *slen = srow + CHUNK;
        auto tiles_from = [&](int base, int &n) -> int {  // of the group in which row base + tid starts
            const int t = base + tid;
            __syncthreads();
            if (tid < CHUNK && t < a.n_tokens) {
                int trow;
                srow[tid] = __ldg(a.rows + t);
                slen[tid] = row_len(a, t, trow, bad);
            }
            __syncthreads();
            n = 0;
            if (tid >= CHUNK || t >= a.n_tokens || ((t & (block - 1)) && srow[tid - 1] == srow[tid])) return 0;
            const int end = min(min(a.n_tokens - base, CHUNK), (tid | (block - 1)) + 1);
            int most = 0, u = tid;
            for (; u < end && srow[u] == srow[tid]; ++u) most = max(most, slen[u]);
            if (u - tid < GROUP_MIN) return 0;
            n = u - tid;
            return max((most + N - 1) / N, 1);
        };
        auto block_sum = [&](int v, long long &before) -> long long {  // of THREADS values, and of those before
            long long sum = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long u = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += u;
            }
            if (lane == 31) sh.scan[warp] = sum;
            __syncthreads();
            long long total = 0;
            before = sum - v;
            for (int w = 0; w < THREADS / 32; ++w) {
                if (w < warp) before += sh.scan[w];
                total += sh.scan[w];
            }
            __syncthreads();
            return total;
        };
        long long total = 0, before;
        int n, tiles = 0;
        for (int base = 0; base < a.n_tokens; base += CHUNK) {
            tiles = tiles_from(base, n);
            total += block_sum(tiles, before);
        }
        share = (int)max((total + ranges - 1) / ranges, (long long)MIN_TILES);
        const long long x = (long long)share * range;
        left = (int)max(min((long long)share, total - x), 0ll);
        if (left == 0) {  // the same in all threads
            if (tid == 0) work.part[blockIdx.x] = Part{-1, 0, 0, 0};
            if (bad && blockIdx.x == 0 && a.err) atomicOr(a.err, QSA_DEVERR_BAD_ID);
            return;
        }
        long long done = 0;
        for (int base = 0; base < a.n_tokens; base += CHUNK) {
            if (a.n_tokens > CHUNK) tiles = tiles_from(base, n);
            const long long sum = block_sum(tiles, before);
            if (x >= done + before && x < done + before + tiles) {
                sh.t = base + tid;
                sh.before = done + before;
            }
            done += sum;
            if (x < done) break;
        }
    }
    if (warp == 12) tmem_alloc(smem_u32(&sh.tmem), G::TMEM_COLS);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = sh.tmem;
    int t = sh.t;
    Group grp = group_at(a, t, block, bad);
    int tokens = grp.rows, tiles = grp.tiles();
    int i0 = (int)((long long)share * range - sh.before);
    Part part{-1, 0, 0, 0};
    int k = 0;  // tiles done: the barriers' phases
    bool ok = true, issued = false;

    for (bool first = true;; first = false) {
        // Segment: tiles i0 .. i1-1 of the group of `tokens` rows at t.
        const int i1 = min(tiles, i0 + left), rows = tokens * per;
        const bool whole = i1 - i0 == tiles;
        const size_t at = (size_t)blockIdx.x * 2 + (first && i0 > 0 ? 0 : 1);
        float *values = reinterpret_cast<float *>(sh.q);
        auto head_row = [&](int m) -> size_t {  // of q: token t + m / per, head kvh per + m % per
            const int i = (int)((uint32_t)m * per_inv >> 16);  // m / per, m < 128
            return (size_t)(t + i) * a.n_q_heads + (size_t)kvh * per + (m - i * per);
        };
        const int trow = grp.trow, least = grp.least, most = grp.most;

        // The queries: a warp takes every fourteenth head row, five in flight.
        auto stage_q = [&] {
            constexpr int E = 4 * S, QW = THREADS / 32, QB = 5;  // elements per lane; warps; rows in flight
            for (int m0 = warp; m0 < M; m0 += QB * QW) {
                uint32_t x[QB][E / 2];
#pragma unroll
                for (int b = 0; b < QB; ++b) {
                    const int m = m0 + QW * b;
                    const size_t at = head_row(m) * D + lane * E;
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
                for (int b = 0; b < QB; ++b) {
                    const int m = m0 + QW * b;
                    if (m >= M) break;
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
            asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");  // of all roles, each at its place
        };

        if (warp >= 4 && warp < 12) {
            // ---- loads and conversion: K (warps 4-7) or V ----
            // Sixteen codes an item: CH lanes take a cell's row, so that a load
            // reads whole rows, ITEMS cells per thread.
            constexpr int CH = D / 16, ITEMS = N * CH / CONVERTERS, STEP = N / ITEMS;
            const bool is_v = warp >= 8;
            const int ct = (tid - 128) % CONVERTERS, ch = ct % CH, c0 = ct / CH;
            const int8_t *codes = (is_v ? a.vq : a.kq) + 16 * ch;
            const uint16_t *scales = is_v ? a.vsc : a.ksc;
            uint8_t *dst = is_v ? sh.v[ch >> 2] : sh.k[ch >> 2];
            const int32_t *tab = a.page_table + (size_t)trow * a.max_pages;
            uint4 w[ITEMS];
            uint2 sc[ITEMS];
            auto page_of = [&](int i) {  // of cells 2 lane and 2 lane + 1 of tile i
                const int j = (i * N + 2 * lane) >> page_shift;
                return i < i1 && j < a.max_pages ? __ldg(tab + j) : -1;
            };
            auto load = [&](int i, int pages) {
#pragma unroll
                for (int j = 0; j < ITEMS; ++j) {
                    const int in = c0 + j * STEP, c = i * N + in, page = __shfl_sync(0xffffffffu, pages, in >> 1);
                    const bool wanted = i < i1 && c < most;
                    bool have = wanted && page >= 0 && page < a.n_pages;
                    bad |= wanted && !have;
                    const long long row = ((((long long)page << page_shift) + (c & (a.page_size - 1))) * a.n_kv_heads) + kvh;
                    have = have && QSA_IN(row, (long long)a.n_pages * a.page_size * a.n_kv_heads);
                    w[j] = have ? __ldg(reinterpret_cast<const uint4 *>(codes + row * D)) : make_uint4(0u, 0u, 0u, 0u);
                    sc[j] = have ? __ldg(reinterpret_cast<const uint2 *>(scales + row * 4)) : make_uint2(0u, 0u);
                }
            };
            int pages = page_of(i0);
            load(i0, pages);
            pages = page_of(i0 + 1);
            stage_q();
            bool good = ok;
            for (int i = i0; i < i1 && good; ++i, ++k) {
                // Until the products with the tile before are done.
                if (k > 0)
                    good = is_v ? mbar_wait_or_abort(smem_u32(&sh.pv_full), (k - 1) & 1, abort)
                                : mbar_wait_or_abort(smem_u32(&sh.s_full[(k - 1) & 1]), ((k - 1) >> 1) & 1, abort);
                good = __all_sync(0xffffffffu, good);
                if (!good) break;
#pragma unroll
                for (int j = 0; j < ITEMS; ++j) {
                    const int in = c0 + j * STEP, e = scale_exponent(sc[j]);
                    const __half2 f = scaled(sc[j], ch / (CH / 4), e);
                    const uint32_t x[4] = {w[j].x ^ 0x80808080u, w[j].y ^ 0x80808080u, w[j].z ^ 0x80808080u, w[j].w ^ 0x80808080u};
#pragma unroll
                    for (int u = 0; u < 2; ++u)
                        *reinterpret_cast<uint4 *>(dst + unit_off(in, 2 * (ch & 3) + u)) =
                            make_uint4(prod(prmt(x[2 * u], 0x64646464u, 0x4140), f), prod(prmt(x[2 * u], 0x64646464u, 0x4342), f),
                                       prod(prmt(x[2 * u + 1], 0x64646464u, 0x4140), f),
                                       prod(prmt(x[2 * u + 1], 0x64646464u, 0x4342), f));
                }
                fence_async_smem();
                mbar_arrive(smem_u32(is_v ? &sh.v_full : &sh.k_full));
                load(i + 1, pages);
                pages = page_of(i + 2);
            }
            ok = good;
        } else if (warp == 13) {
            // ---- the cells' factors, two cells a lane ----
            const int32_t *tab = a.page_table + (size_t)trow * a.max_pages;
            uint2 ks[2], vs[2];
            bool there[2];
            auto load = [&](int i) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int c = i * N + 2 * lane + e, j = c >> page_shift;
                    const int page = i < i1 && c < most && j < a.max_pages ? __ldg(tab + j) : -1;
                    there[e] = page >= 0 && page < a.n_pages;
                    const long long row = ((((long long)page << page_shift) + (c & (a.page_size - 1))) * a.n_kv_heads) + kvh;
                    there[e] = there[e] && QSA_IN(row, (long long)a.n_pages * a.page_size * a.n_kv_heads);
                    ks[e] = there[e] ? __ldg(reinterpret_cast<const uint2 *>(a.ksc + row * 4)) : make_uint2(0u, 0u);
                    vs[e] = there[e] ? __ldg(reinterpret_cast<const uint2 *>(a.vsc + row * 4)) : make_uint2(0u, 0u);
                }
            };
            load(i0);
            stage_q();
            bool good = ok;
            for (int i = i0; i < i1 && good; ++i, ++k) {
                // Three buffers: with S k - 1, issued after P k - 3 came, the softmax of tile k - 3 is done.
                if (k > 0) good = mbar_wait_or_abort(smem_u32(&sh.s_full[(k - 1) & 1]), ((k - 1) >> 1) & 1, abort);
                good = __all_sync(0xffffffffu, good);
                if (!good) break;
                const int b = k % 3;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int ev = scale_exponent(vs[e]);
                    sh.kf[b][2 * lane + e] = exp2i(-scale_exponent(ks[e]));
                    sh.vb[b][2 * lane + e] = there[e] ? -(float)ev : -CUDART_INF_F;
                    sh.vw[b][2 * lane + e] = exp2i(ev);
                }
                mbar_arrive(smem_u32(&sh.k_full));
                load(i + 1);
            }
            ok = good;
        } else if (warp == 12) {
            // ---- products ----
            stage_q();
            bool good = ok;
            if (lane == 0) {
                auto issue_s = [&](int kk) {
                    good = mbar_wait_or_abort(smem_u32(&sh.k_full), kk & 1, abort);
                    if (!good) return;
                    fence_after();
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        mma_f16(tmem + (kk & 1) * N, sw128_kmajor(smem_u32(sh.q[ks >> 2]) + (ks & 3) * 32),
                                sw128_kmajor(smem_u32(sh.k[ks >> 2]) + (ks & 3) * 32), G::IDESC_S, ks ? 1u : 0u);
                    mma_commit(smem_u32(&sh.s_full[kk & 1]));
                    issued = true;
                };
                issue_s(k);
                for (int i = i0; i < i1 && good; ++i, ++k) {
                    // The buffer of S k + 1 was S k - 1's, whose P has come.
                    if (i + 1 < i1) issue_s(k + 1);
                    good = good && mbar_wait_or_abort(smem_u32(&sh.v_full), k & 1, abort) &&
                           mbar_wait_or_abort(smem_u32(&sh.p_full), k & 1, abort);
                    if (!good) break;
                    fence_after();
                    // V transposed: 64 dims apart N * 128 bytes, eight cells 1024.
#pragma unroll
                    for (int ks = 0; ks < N / 16; ++ks)
                        mma_f16(tmem + G::O_COL, sw128_kmajor(smem_u32(sh.p) + ks * 32),
                                smem_desc(smem_u32(sh.v[0]) + ks * 16 * 128, N * 128, 1024, 2), G::IDESC_O, i > i0 || ks ? 1u : 0u);
                    mma_commit(smem_u32(&sh.pv_full));
                }
            }
            k = __shfl_sync(0xffffffffu, k, 0);
            ok = __shfl_sync(0xffffffffu, (int)good, 0);
        } else {
            // ---- softmax, a thread per head row ----
            stage_q();
            const int m = tid;
            const bool mine = m < rows;
            const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
            const float sl2 = a.softmax_scale * LOG2E * sh.qinv[m];
            int len = 0, tr;
            if (mine) len = row_len(a, t + (int)((uint32_t)m * per_inv >> 16), tr, bad);
            float ref = -CUDART_INF_F, l = 0.0f;
            bool good = ok;
            for (int i = i0; i < i1 && good; ++i, ++k) {
                good = __all_sync(0xffffffffu, mbar_wait_or_abort(smem_u32(&sh.s_full[k & 1]), (k >> 1) & 1, abort));
                if (!good) break;
                fence_after();
                float y[N];
                {
                    uint32_t v[N / 16][16];
#pragma unroll
                    for (int c = 0; c < N / 16; ++c) tmem_ld16(lane_base + (k & 1) * N + 16 * c, v[c]);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        asm volatile("" : "+r"(v[j / 16][j % 16]));  // not before the wait
                        y[j] = __uint_as_float(v[j / 16][j % 16]);
                    }
                }
                const float *kf = sh.kf[k % 3], *vb = sh.vb[k % 3], *vw = sh.vw[k % 3];
                float top = -CUDART_INF_F;
#pragma unroll
                for (int j = 0; j < N; j += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(kf + j), b = *reinterpret_cast<const float4 *>(vb + j);
                    float2 s0 = __fmul2_rn(make_float2(y[j], y[j + 1]), make_float2(f.x, f.y));
                    float2 s1 = __fmul2_rn(make_float2(y[j + 2], y[j + 3]), make_float2(f.z, f.w));
                    s0 = __ffma2_rn(s0, make_float2(sl2, sl2), make_float2(b.x, b.y));
                    s1 = __ffma2_rn(s1, make_float2(sl2, sl2), make_float2(b.z, b.w));
                    y[j] = s0.x;
                    y[j + 1] = s0.y;
                    y[j + 2] = s1.x;
                    y[j + 3] = s1.y;
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
                    for (int j = 0; j < 4; j += 2) {
                        const int c = 8 * u + 2 * j;
                        const float4 f = *reinterpret_cast<const float4 *>(vw + c);
                        float2 p0 = __fadd2_rn(make_float2(y[c], y[c + 1]), make_float2(base, base));
                        float2 p1 = __fadd2_rn(make_float2(y[c + 2], y[c + 3]), make_float2(base, base));
                        p0 = make_float2(ex2(p0.x), ex2(p0.y));
                        p1 = make_float2(ex2(p1.x), ex2(p1.y));
                        sum = __ffma2_rn(p0, make_float2(f.x, f.y), sum);
                        sum = __ffma2_rn(p1, make_float2(f.z, f.w), sum);
                        h[j] = h2u(__floats2half2_rn(p0.x, p0.y));
                        h[j + 1] = h2u(__floats2half2_rn(p1.x, p1.y));
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
                // The values to shared memory, in place of the tiles (whose
                // products are done): 16-byte unit c of row m at c ^ (m % 8).
                fence_after();
                const bool none = ref == -CUDART_INF_F;
                const float w = whole ? (none ? 0.0f : 1.0f / l) : 1.0f;
                for (int c = 0; c < D / 16; c += 4) {
                    uint32_t v[4][16];
#pragma unroll
                    for (int i = 0; i < 4; ++i) tmem_ld16(lane_base + G::O_COL + 16 * (c + i), v[i]);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) asm volatile("" : "+r"(v[i][4 * j + e]));
                            float *dst = values + m * D + 4 * ((4 * (c + i) + j) ^ (m & 7));
                            *reinterpret_cast<float4 *>(dst) =
                                make_float4(__uint_as_float(v[i][4 * j]) * w, __uint_as_float(v[i][4 * j + 1]) * w,
                                            __uint_as_float(v[i][4 * j + 2]) * w, __uint_as_float(v[i][4 * j + 3]) * w);
                        }
                }
                if (mine) {
                    if (!whole)
                        *reinterpret_cast<float2 *>(work.ml + (at * M + m) * 2) = make_float2(ref, l);
                    else if (a.lse)
                        a.lse[head_row(m)] = none ? ref : (ref + log2f(l)) * LN2;
                }
                fence_before();  // O is overwritten by the next segment
            }
            ok = good;
        }
        if (!__syncthreads_and(ok)) {
            ok = false;
            break;
        }
        // All threads write the values out, whole rows at a time.
        for (int u = tid; u < rows * (D / 4); u += THREADS) {
            const int m = u / (D / 4), c = u % (D / 4);
            const float4 y = *reinterpret_cast<const float4 *>(values + m * D + 4 * (c ^ (m & 7)));
            if (!whole) {
                *reinterpret_cast<float4 *>(work.o + (at * M + m) * D + 4 * c) = y;
                continue;
            }
            const size_t oi = head_row(m) * D + 4 * c;
            if (!QSA_IN(oi + 3, (size_t)a.n_tokens * a.n_q_heads * D)) continue;
            float2 y0 = make_float2(y.x, y.y), y1 = make_float2(y.z, y.w);
            if (a.gate) {
                const float2 g0 = __ldg(reinterpret_cast<const float2 *>(a.gate + oi));
                const float2 g1 = __ldg(reinterpret_cast<const float2 *>(a.gate + oi + 2));
                y0 = make_float2(gated(y0.x, g0.x), gated(y0.y, g0.y));
                y1 = make_float2(gated(y1.x, g1.x), gated(y1.y, g1.y));
            }
            store_out(a, oi, y0);
            store_out(a, oi + 2, y1);
        }
        if (i1 - i0 < tiles && i0 == 0) part = Part{t, 1 + (tiles - i1 + share - 1) / share, tokens, 0};
        left -= i1 - i0;
        if (left <= 0) break;
        i0 = 0;
        __syncthreads();  // the values have been read; the tiles take their place again
        do {  // the next group: there is one
            t += max(tokens, 1);
            grp = group_at(a, t, block, bad);
            tokens = grp.rows;
            tiles = grp.tiles();
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
    if (warp == 12) {
        fence_after();
        tmem_dealloc(tmem, G::TMEM_COLS);
    }
}

template <int S>
cudaError_t launch(const qsa_paged_attn_args &a, void *ws, int &ctas, cudaStream_t s) {
    const int per = a.n_q_heads / a.n_kv_heads, smem = (int)sizeof(GroupSmem<S>);
    ctas = (MAX_GROUP_PARTS / a.n_kv_heads > 1 ? MAX_GROUP_PARTS / a.n_kv_heads : 1) * a.n_kv_heads;
    const cudaError_t e = cudaFuncSetAttribute(paged_group_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    return e != cudaSuccess ? e : launch_dependent(paged_group_kernel<S>, dim3(ctas), dim3(THREADS), smem, s, a, ws, group_block(per));
}

}  // namespace

size_t paged_group_workspace_bytes(int head_dim) { return Work::bytes(MAX_GROUP_PARTS, M, head_dim); }

cudaError_t launch_paged_group(const qsa_paged_attn_args &a, void *ws, int &ctas, cudaStream_t s) {
    return a.head_dim == 128 ? launch<1>(a, ws, ctas, s) : launch<2>(a, ws, ctas, s);
}

}  // namespace qsa

QSA_DEFINE_CHECK_READER(take_check_word_paged_group)
