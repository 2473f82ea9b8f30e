// qsa_paged_attn, rows that read one sequence together: the consecutive tokens
// of a draft window or of a chunk, each with its own length.
//
// Their heads, up to 128, are the M side of tcgen05 products over one pass of
// the cache, so a cell's codes are read and converted once for all of them.
// (Eight tokens x 12 heads over 30 K cells of 2 x 256 dims, with the join:
// 38 us; row by row, where the cache comes eight times from L2 and its 2 x 15 M
// codes are converted eight times, 61 us.)
//
// A CTA takes tiles of 64 cells; its warps have roles, which hand tiles over by
// mbarriers:
//   softmax (8 warps, two threads per head row, 32 cells each): the queries to
//   tensor memory, then of each tile S from there, and the weights P back in
//   its place, fp16, as the A operand of the next product;
//   converters (8): codes to fp16 in shared memory, [64 cells][D], 64 dims to a
//   128-byte row with the swizzle: K-major for S = Q K^T (128 x 64), read
//   transposed (N-major) for O += P V (128 x D).  K is a tile ahead of V;
//   products (1 warp, one thread issues);
//   loads (1 warp each for K and V, up to two tiles ahead).
// Tiles are shared out over the chip and joined as in paged_attn.cu.  A tile
// takes 3.8 K cycles of the chain K converted - S - K converted, of which the
// 32 products of S are 1.7 K; issue slots are used to a third and the tensor
// pipe to a fifth, so the rest is the roles' latency.  The seven tiles a CTA of
// the rows above are 14 us so; what does not shrink with the tiles (the launch
// of the kernel that takes rows one by one, the share, queries and first loads,
// partials of up to 98 KB a CTA and the join of them) is as much again and more:
// two tiles a CTA take 21 to 26 us.  (Dropped, each without
// gain: K converted by halves of the dims beside the other half's products; TMA
// boxes in place of cp.async; two warps each for the loads.  A bulk copy per
// cell, 256 bytes each, took 70 cycles a copy: 53 us where cp.async took 35.)
//
// Scales.  K's are multiplied into the codes under a power of two per cell,
// 2^ek, that the softmax undoes (codes x scales then use fp16's range whatever
// the scales are), in two fp16 parts that hold the 19-bit product exactly (one
// part alone, each product off by up to 2^-11 of itself: 36 us).  V's are multiplied in under 2^ev, so that a cell's largest
// scale is in [1, 2), and rounded to fp16.  The softmax works on s - ev: P =
// 2^(s - ev - m) is the weight of the scaled values, its running maximum m is
// one of weight x value, and the denominator adds P 2^ev, in fp32.
#include "paged_attn.cuh"

namespace qsa {
namespace {

using namespace tc;

constexpr int M = GROUP_ROWS, N = 64;  // heads and cells of a tile
constexpr int SOFTMAX = 256;     // threads of the softmax, two for a head row
constexpr int CONVERTERS = 256;  // threads that turn codes to halves
constexpr int PRODUCTS = (SOFTMAX + CONVERTERS) / 32, LOADER = PRODUCTS + 1, WARPS = LOADER + 2;  // roles by warp, in this order
constexpr int THREADS = 32 * WARPS;
constexpr int STAGES = 2;        // tiles on their way
// Of a share.  Eight rows of 2 K cells, 8/2 heads of 256: 20.5 us; shares of four
// 23.1, of six 26.3.
constexpr int MIN_TILES = 2;

template <int S>
struct GroupShape {
    static constexpr int D = 128 * S;
    static constexpr uint32_t TMEM_COLS = 512, Q_COL = 2 * N, O_COL = Q_COL + D / 2;  // S at 0 and N, P in its place
    static_assert(O_COL + D <= TMEM_COLS, "tensor memory");
    static constexpr uint32_t IDESC_S = idesc_f16(M, N, false, false), IDESC_O = idesc_f16(M, D, false, true);
};

// Zeros where not `have`.
template <int BYTES>
__device__ __forceinline__ void cp_async(void *dst, const void *src, bool have) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(smem_u32(dst)), "l"(src), "r"(have ? 16 : 0) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;\n" ::"r"(smem_u32(dst)), "l"(src), "n"(BYTES), "r"(have ? BYTES : 0)
                     : "memory");
}
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0u;
}
// The group that starts at a row t: its rows (0: none starts), and the shortest
// and longest length.
struct Group {
    int rows, least, most, trow;
    __device__ __forceinline__ int tiles() const { return rows ? max((most + N - 1) / N, 1) : 0; }
};

// Everything of shared memory; tiles of 64 halves (128 bytes) a row, 16-byte
// unit u of row r at u ^ (r % 8).
template <int S>
struct GroupSmem {
    uint8_t k[2][2 * S][N * 128];  // high and low part, per 64 dims; from here on also the values at the end of a segment, fp32 [M][D]
    uint8_t v[2][2 * S][N * 128];
    alignas(16) int8_t codes[STAGES][2][N * 128 * S];  // K's and V's as they come
    uint2 scales[STAGES][2][N];
    bool there[STAGES][N];
    alignas(16) uint32_t poison[3][CONVERTERS / 32];  // by converter warp: its lanes whose V scale is infinite or NaN
    alignas(16) float kf[3][N], vb[3][N], vw[3][N];  // a cell's 2^-ek, -ev (-inf: not there), 2^ev
    float top[2][2][M], l[2][M];         // the two halves' maxima (two buffers) and sums of a head row
    uint64_t full[2][STAGES], empty[2][STAGES];  // K's and V's codes
    uint64_t q_full, k_full, v_full[2], s_full[2], p_full[2], pv_full[2], drain;
    long long scan[3][WARPS];
    long long before;  // tiles before the group at t, in which the CTA's share starts
    int t;
    Group grp;
    int abort;
    uint32_t tmem;
};

__device__ __forceinline__ uint32_t unit_off(int r, int u) { return r * 128 + ((u ^ (r & 7)) << 4); }

// Scale i of a cell times 2^e, in both halves.
__device__ __forceinline__ __half2 scaled(uint2 sc, int i, int e) {
    const uint32_t w = i >> 1 ? sc.y : sc.x;
    const float f = __half2float(__ushort_as_half((unsigned short)(i & 1 ? w >> 16 : w & 0xFFFFu)));
    return __float2half2_rn(f * exp2i(e));
}
// Looked up by a warp.
__device__ __forceinline__ Group group_at(const qsa_paged_attn_args &a, int t, int block, bool &bad) {
    const int lane = threadIdx.x & 31, row = __ldg(a.rows + t);
    Group g{0, 0x7fffffff, 0, 0};
    if (group_start(a.rows, t, block) != t) return g;
    const int end = group_end(a, t, block);
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
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&sh.s_full[b]), 1);
            mbar_init(smem_u32(&sh.v_full[b]), CONVERTERS);
            mbar_init(smem_u32(&sh.p_full[b]), SOFTMAX);
            mbar_init(smem_u32(&sh.pv_full[b]), 1);
        }
        mbar_init(smem_u32(&sh.q_full), SOFTMAX);
        for (int b = 0; b < 2 * STAGES; ++b) {
            mbar_init(smem_u32(&sh.full[0][0] + b), b < STAGES ? 64 : 32);
            mbar_init(smem_u32(&sh.empty[0][0] + b), CONVERTERS / 32);
        }
        mbar_init(smem_u32(&sh.k_full), CONVERTERS);
        mbar_init(smem_u32(&sh.drain), 1);
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    wait_for_previous_grid();
    allow_dependent_launch();
    const Work work(ws, MAX_GROUP_PARTS, M);
    // Results in fp16 take weights in two parts (22 bits); bf16's own rounding,
    // up to 2^-8, hides one of 11 bits.
    const bool fine = a.dtype == QSA_F16;
    bool bad = false;

    // The groups' tiles, and the group in which this CTA's share of them starts.
    int share = 0, left = 0, t = 0;
    long long tiles_before = 0;
    Group grp{0, 0, 0, 0};
    auto take_share = [&](long long total) {  // false: nothing to do, the same in all threads
        const long long each = total < 0x7fffffffll - MAX_GROUP_PARTS ? ((int)total + ranges - 1) / ranges : (total + ranges - 1) / ranges;
        share = (int)max(each, (long long)MIN_TILES);
        const long long x = (long long)share * range;
        left = (int)max(min((long long)share, total - x), 0ll);
        return left > 0;
    };
    bool any;
    if (a.n_tokens <= 32) {
        // Few rows: each warp works it out for itself, a lane per row (2 us
        // less than by the block).
        const bool in = lane < a.n_tokens;
        int row = -1, len = 0, trow = 0;
        if (in) {
            row = __ldg(a.rows + lane);
            len = row_len(a, lane, trow, bad);
        }
        const int prev = __shfl_up_sync(0xffffffffu, row, 1);
        const unsigned upto = 0xffffffffu >> (31 - lane), runs = __ballot_sync(0xffffffffu, in && (lane == 0 || prev != row));
        const int run = 31 - __clz(runs & upto);  // where the lane's starts
        const bool starts = in && ((lane - run) & (block - 1)) == 0;
        const unsigned groups = __ballot_sync(0xffffffffu, starts), after = groups & ~upto;
        const int id = __popc(groups & upto);
        Group g{(after ? __ffs(after) - 1 : a.n_tokens) - lane, len, len, trow};
        struct {
            long long tiles, alone, together;
        } v{0, in ? units_of<S>(len) : 0, 0};
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {  // over the rest of the lane's group
            const int least = __shfl_down_sync(0xffffffffu, g.least, o), most = __shfl_down_sync(0xffffffffu, g.most, o);
            const int other = __shfl_down_sync(0xffffffffu, id, o);
            if (lane + o < a.n_tokens && other == id) {
                g.least = min(g.least, least);
                g.most = max(g.most, most);
            }
        }
        if (starts) {
            v.tiles = g.tiles();
            v.together = units_of<S>(g.most);
        }
        const bool longer = __any_sync(0xffffffffu, v.alone > WHOLE);
        long long sum = v.tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += u;
            v.alone += __shfl_xor_sync(0xffffffffu, v.alone, o);
            v.together += __shfl_xor_sync(0xffffffffu, v.together, o);
        }
        any = take_groups<S>(a, v.alone, v.together, longer) && take_share(__shfl_sync(0xffffffffu, sum, 31));
        const long long x = (long long)share * range;
        const unsigned here = __ballot_sync(0xffffffffu, any && starts && x >= sum - v.tiles && x < sum);
        t = here ? __ffs(here) - 1 : 0;
        tiles_before = __shfl_sync(0xffffffffu, sum - v.tiles, t);
        grp = Group{__shfl_sync(0xffffffffu, g.rows, t), __shfl_sync(0xffffffffu, g.least, t), __shfl_sync(0xffffffffu, g.most, t),
                    __shfl_sync(0xffffffffu, g.trow, t)};
    } else {
        // Rows and lengths go to shared memory a chunk of whole spans at a
        // time, and the thread of a row in which a group starts adds it up there.
        constexpr int CHUNK = 512;  // a multiple of any block
        static_assert(CHUNK <= THREADS && CHUNK % M == 0, "a thread per row");
        int *srow = reinterpret_cast<int *>(sh.k), *slen = srow + CHUNK;
        auto group_from = [&](int base) -> Group {  // that starts in row base + tid
            const int t = base + tid;
            __syncthreads();
            if (tid < CHUNK && t < a.n_tokens) {
                int trow;
                srow[tid] = __ldg(a.rows + t);
                slen[tid] = row_len(a, t, trow, bad);
            }
            __syncthreads();
            Group g{0, 0x7fffffff, 0, 0};
            if (tid >= CHUNK || t >= a.n_tokens) return g;
            const int row = srow[tid], span = group_span(block);
            int u = tid;
            while ((u & (span - 1)) && srow[u - 1] == row) --u;
            if ((tid - u) & (block - 1)) return g;
            const int end = min(group_end(a, t, block) - base, CHUNK);
            u = tid;
            for (; u < end && srow[u] == row; ++u) {
                g.least = min(g.least, slen[u]);
                g.most = max(g.most, slen[u]);
            }
            g.rows = u - tid;
            g.trow = row >= 0 && row < a.n_rows ? row : 0;
            return g;
        };
        // Sums over the block: of tiles, with those before the thread's, and of
        // the rows' and the groups' units.
        struct Sums {
            long long tiles, alone, together;
        };
        auto block_sum = [&](Sums v, long long &before) -> Sums {
            long long sum = v.tiles;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long u = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += u;
                v.alone += __shfl_xor_sync(0xffffffffu, v.alone, o);
                v.together += __shfl_xor_sync(0xffffffffu, v.together, o);
            }
            if (lane == 31) {
                sh.scan[0][warp] = sum;
                sh.scan[1][warp] = v.alone;
                sh.scan[2][warp] = v.together;
            }
            __syncthreads();
            Sums total{0, 0, 0};
            before = sum - v.tiles;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                if (w < warp) before += sh.scan[0][w];
                total.tiles += sh.scan[0][w];
                total.alone += sh.scan[1][w];
                total.together += sh.scan[2][w];
            }
            __syncthreads();
            return total;
        };
        long long total = 0, before = 0, alone = 0, together = 0;
        int longer = 0;
        Group g;
        for (int base = 0; base < a.n_tokens; base += CHUNK) {
            g = group_from(base);
            const int u = tid < CHUNK && base + tid < a.n_tokens ? units_of<S>(slen[tid]) : 0;
            longer |= u > WHOLE;
            const Sums sums = block_sum(Sums{g.tiles(), u, g.rows ? units_of<S>(g.most) : 0}, before);
            total += sums.tiles;
            alone += sums.alone;
            together += sums.together;
        }
        any = take_groups<S>(a, alone, together, __syncthreads_or(longer)) && take_share(total);
        const long long x = (long long)share * range;
        long long done = 0;
        for (int base = 0; any && base < a.n_tokens; base += CHUNK) {
            long long sum = total;  // of one chunk, g and before are still at hand
            if (a.n_tokens > CHUNK) {
                g = group_from(base);
                sum = block_sum(Sums{g.tiles(), 0, 0}, before).tiles;
            }
            if (x >= done + before && x < done + before + g.tiles()) {
                sh.t = base + tid;
                sh.before = done + before;
                sh.grp = g;
            }
            done += sum;
            if (x < done) break;
        }
    }
    if (!any) {  // the same in all threads; also where paged_attn.cu takes the rows
        if (tid == 0) work.part[blockIdx.x] = Part{-1, 0, 0, 0};
        if (bad && blockIdx.x == 0 && a.err) atomicOr(a.err, QSA_DEVERR_BAD_ID);
        return;
    }
    if (warp == PRODUCTS) tmem_alloc(smem_u32(&sh.tmem), G::TMEM_COLS);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = sh.tmem;
    if (a.n_tokens > 32) {
        t = sh.t;
        tiles_before = sh.before;
        grp = sh.grp;
    }
    int tokens = grp.rows, tiles = grp.tiles();
    int i0 = (int)((long long)share * range - tiles_before);
    Part part{-1, 0, 0, 0};
    int k = 0;  // tiles done: the barriers' phases
    bool ok = true, issued = false;  // issued: products, by this thread
    uint32_t segment = 0;

    for (bool first = true;; first = false, ++segment) {
        // Segment: tiles i0 .. i1-1 of the group of `tokens` rows at t.
        const int i1 = min(tiles, i0 + left), rows = tokens * per;
        const bool whole = i1 - i0 == tiles;
        const size_t at = (size_t)blockIdx.x * 2 + (first && i0 > 0 ? 0 : 1);
        float *values = reinterpret_cast<float *>(sh.k);
        auto head_row = [&](int m) -> size_t {  // of q: token t + m / per, head kvh per + m % per
            const int i = (int)((uint32_t)m * per_inv >> 16);  // m / per, m < 128
            return (size_t)(t + i) * a.n_q_heads + (size_t)kvh * per + (m - i * per);
        };
        const int trow = grp.trow, least = grp.least, most = grp.most;

        constexpr int CH = D / 16;  // items of sixteen codes of a cell
        // A converter warp takes CELLS cells at a time and ITEMS times that of a
        // tile: eight cells, so a lane makes the factor of one scale of K and
        // one of V (scale lane % 4 of the warp's cell lane / 4).
        constexpr int CELLS = 32 / CH, ITEMS = N * CH / CONVERTERS, STEP = N / ITEMS;
        static_assert(CELLS * ITEMS * 4 == 32, "a factor per lane");
        auto factor_cell = [](int converter, int lane) { return converter * CELLS + (lane >> 2) % CELLS + (lane >> 2) / CELLS * STEP; };
        if (warp >= LOADER) {
            // ---- loads, a warp each for K (with the scales of both) and V ----
            // A lane finds two neighbouring cells, which are of one page; all
            // then copy, CH lanes to a cell's row.
            constexpr int AT_ONCE = 32 / CH;
            const int kind = warp - LOADER;
            const int32_t *tab = a.page_table + (size_t)trow * a.max_pages;
            auto page_of = [&](int i) {
                const int j = (i * N + 2 * lane) >> page_shift;
                return i < i1 && j < a.max_pages ? __ldg(tab + j) : -1;
            };
            // The lane's part of a copy: its cell of the pair, its codes.
            const int8_t *codes = (kind ? a.vq : a.kq) + (size_t)(lane / CH & 1) * a.n_kv_heads * D + lane % CH * 16;
            int page = page_of(i0);
            bool good = ok;
            for (int i = i0; i < i1; ++i, ++k) {
                const int st = k % STAGES, c = i * N + 2 * lane;
                // The pool's (cell, KV head) row of the first, and which are there.
                const bool known = page >= 0 && page < a.n_pages;
                bool have[2] = {known && c < most, known && c + 1 < most};
                bad |= !known && c < most;
                const long long row = ((((long long)page << page_shift) + (c & (a.page_size - 1))) * a.n_kv_heads) + kvh;
                have[0] = have[0] && QSA_IN(row, (long long)a.n_pages * a.page_size * a.n_kv_heads);
                have[1] = have[1] && QSA_IN(row + a.n_kv_heads, (long long)a.n_pages * a.page_size * a.n_kv_heads);
                const unsigned m0 = __ballot_sync(0xffffffffu, have[0]), m1 = __ballot_sync(0xffffffffu, have[1]);
                const unsigned mine = lane / CH & 1 ? m1 : m0;
                page = page_of(i + 1);
                if (k >= STAGES) good = mbar_wait_or_abort(smem_u32(&sh.empty[kind][st]), (k / STAGES - 1) & 1, abort);
                good = __all_sync(0xffffffffu, good);
                if (!good) break;
                const long long off = row * D;
#pragma unroll 8
                for (int j = 0; j < N / AT_ONCE; ++j) {
                    const int pair = j * AT_ONCE / 2 + lane / (2 * CH);
                    const long long o = __shfl_sync(0xffffffffu, off, pair);
                    const bool in = mine >> pair & 1u;
                    cp_async<16>(sh.codes[st][kind] + j * 512 + 16 * lane, codes + (in ? o : 0), in);
                }
                const uint32_t bar = smem_u32(&sh.full[kind][st]);
                if (kind == 0) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const size_t r = have[e] ? (row + e * a.n_kv_heads) * 4 : 0;
                        cp_async<8>(&sh.scales[st][0][2 * lane + e], a.ksc + r, have[e]);
                        cp_async<8>(&sh.scales[st][1][2 * lane + e], a.vsc + r, have[e]);
                        sh.there[st][2 * lane + e] = have[e];
                    }
                    mbar_arrive(bar);
                }
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(bar) : "memory");
            }
            ok = good;
        } else if (warp >= SOFTMAX / 32 && warp < PRODUCTS) {
            // ---- conversion ----
            const int ct = tid % CONVERTERS, ch = ct % CH, c0 = ct / CH;
            const int fcell = factor_cell(ct >> 5, lane);
            auto convert = [&](int kind, int k, uint32_t mine) {  // of the k-th tile; mine: the lane's factor
                const int st = k % STAGES;
                uint8_t *dst = kind ? sh.v[k & 1][ch >> 2] : sh.k[0][ch >> 2];
#pragma unroll
                for (int j = 0; j < ITEMS; ++j) {
                    const int in = c0 + j * STEP, odd = ch >> 2 & 1;  // 64 dims apart, lanes write units of other banks
                    const uint4 w = *reinterpret_cast<const uint4 *>(sh.codes[st][kind] + in * D + 16 * ch);
                    const __half2 f = u2h(__shfl_sync(0xffffffffu, mine, (j * CELLS + lane / CH) * 4 + ch / (CH / 4)));
                    const uint32_t x[4] = {(odd ? w.z : w.x) ^ 0x80808080u, (odd ? w.w : w.y) ^ 0x80808080u,
                                           (odd ? w.x : w.z) ^ 0x80808080u, (odd ? w.y : w.w) ^ 0x80808080u};
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int at = unit_off(in, 2 * (ch & 3) + (u ^ odd));
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const __half2 c = __hsub2(u2h(prmt(x[2 * u + e / 2], 0x64646464u, e & 1 ? 0x4342 : 0x4140)), u2h(0x64806480u));
                            const __half2 h = __hmul2(c, f);
                            hi[e] = h2u(h);
                            lo[e] = h2u(__hfma2(c, f, __hneg2(h)));
                        }
                        *reinterpret_cast<uint4 *>(dst + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        if (kind == 0) *reinterpret_cast<uint4 *>(dst + at + (sh.k[1][0] - sh.k[0][0])) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh.empty[kind][st]));
            };
            uint32_t vnext = 0u, vmine;  // V's factors of the tile whose K was converted, and of this
            auto convert_k = [&](int k) {  // of the k-th tile
                const int st = k % STAGES, b = k % 3;
                bool good = mbar_wait_or_abort(smem_u32(&sh.full[0][st]), (k / STAGES) & 1, abort);
                // Until the products with the tile before are done.  Then also
                // the softmax of tile k - 3, as S k - 1 was issued after P k - 3 came.
                if (k > 0) good = good && mbar_wait_or_abort(smem_u32(&sh.s_full[(k - 1) & 1]), ((k - 1) >> 1) & 1, abort);
                if (!__all_sync(0xffffffffu, good)) return false;
                const uint2 ks = sh.scales[st][0][fcell], vs = sh.scales[st][1][fcell];
                const int ek = -scale_exponent(ks), ev = -scale_exponent(vs);
                // A V scale that is infinite or NaN counts as 0 here: times a
                // weight of 0 it would reach rows that end before its cell.
                vnext = h2u(scaled(make_uint2(finite2(vs.x), finite2(vs.y)), lane & 3, ev));
                const uint32_t mine = lane & 2 ? vs.y : vs.x;
                const unsigned poison = __ballot_sync(0xffffffffu, (mine >> (lane & 1 ? 16 : 0) & 0x7C00u) == 0x7C00u);
                if (lane == 0) sh.poison[b][ct >> 5] = poison;
                if ((lane & 3) == 0) {
                    sh.kf[b][fcell] = exp2i(-ek);
                    sh.vb[b][fcell] = sh.there[st][fcell] ? -(float)ev : -CUDART_INF_F;
                    sh.vw[b][fcell] = exp2i(ev);
                }
                // An infinite or NaN K scale: the low parts are NaN, and the cell's scores.
                convert(0, k, h2u(scaled(ks, lane & 3, ek)));
                mbar_arrive(smem_u32(&sh.k_full));
                return true;
            };
            // K is a tile ahead of V.
            bool good = ok;
            for (int i = i0 - 1; i < i1; ++i) {
                vmine = vnext;
                if (i + 1 < i1) good = good && convert_k(k + (i >= i0));
                if (i < i0) continue;
                if (!good) break;
                good = mbar_wait_or_abort(smem_u32(&sh.full[1][k % STAGES]), (k / STAGES) & 1, abort);
                if (k > 1) good = good && mbar_wait_or_abort(smem_u32(&sh.pv_full[k & 1]), ((k - 2) >> 1) & 1, abort);
                good = __all_sync(0xffffffffu, good);
                if (!good) break;
                convert(1, k, vmine);
                mbar_arrive(smem_u32(&sh.v_full[k & 1]));
                ++k;
            }
            ok = good;
        } else if (warp == PRODUCTS) {
            // ---- products ----
            // The whole warp goes through the loop, so that what the products
            // need is the same in all lanes; one lane issues them.
            const bool one = elect_one();
            bool good = ok;
            auto wait = [&](uint64_t &bar, int phase) {
                good = good && __all_sync(0xffffffffu, mbar_wait_or_abort(smem_u32(&bar), phase & 1, abort));
            };
            // Descriptors differ in their address field (16-byte units) only.
            const uint64_t dk = sw128_kmajor(smem_u32(sh.k[0][0]));
            // V transposed: 64 dims apart N * 128 bytes, eight cells 1024.
            const uint64_t dv = smem_desc(smem_u32(sh.v[0][0]), N * 128, 1024, 2);
            auto issue_s = [&](int kk) {
                wait(sh.k_full, kk);
                // The buffer holds P kk - 2.
                if (kk > 1) wait(sh.pv_full[kk & 1], (kk - 2) >> 1);
                if (!good) return;
                fence_after();
                if (one) {
#pragma unroll
                    for (int ks = 0; ks < D / 8; ++ks)  // high parts, then low parts
                        mma_f16_ts(tmem + (kk & 1) * N, tmem + G::Q_COL + ks % (D / 16) * 8, dk + (ks >> 2) * (N * 8) + (ks & 3) * 2,
                                   G::IDESC_S, ks ? 1u : 0u);
                    mma_commit(smem_u32(&sh.s_full[kk & 1]));
                }
                issued |= one;
                __syncwarp();
            };
            wait(sh.q_full, segment);
            if (good) issue_s(k);
            for (int i = i0; i < i1 && good; ++i, ++k) {
                if (i + 1 < i1) issue_s(k + 1);
                wait(sh.v_full[k & 1], k >> 1);
                wait(sh.p_full[k & 1], k >> 1);
                if (!good) break;
                fence_after();
                if (one) {
#pragma unroll
                    for (int ks = 0; ks < N / 8; ++ks) {  // high parts, then low parts
                        if (ks == N / 16 && !fine) break;
                        mma_f16_ts(tmem + G::O_COL, tmem + (k & 1) * N + ks * 8, dv + (k & 1) * (2 * S * N * 8) + ks % (N / 16) * 16 * 8,
                                   G::IDESC_O, i > i0 || ks ? 1u : 0u);
                    }
                    mma_commit(smem_u32(&sh.pv_full[k & 1]));
                }
                __syncwarp();
            }
            ok = good;
        } else {
            // ---- softmax: a head row is two threads', NH of a tile's cells each ----
            constexpr int NH = N / 2, DH = D / 2;
            const int m = tid & (M - 1), half = tid / M, j0 = half * NH;
            const bool mine = m < rows;
            const uint32_t lane_base = tmem + ((uint32_t)(warp % 4 * 32) << 16);
            int len = 0, tr;
            if (mine) len = row_len(a, t + (int)((uint32_t)m * per_inv >> 16), tr, bad);
            // Of the two warps that share their head rows.  Both come here once a
            // tile whatever they waited for, and go on or stop together.
            auto both = [&](bool good) {
                int r;
                asm volatile("{\n.reg .pred p, q;\nsetp.ne.s32 p, %1, 0;\nbar.red.and.pred q, %2, 64, p;\nselp.s32 %0, 1, 0, q;\n}\n"
                             : "=r"(r)
                             : "r"((int)good), "r"(1 + warp % 4)
                             : "memory");
                return r != 0;
            };
            bool good = ok;
            // The queries to tensor memory; bf16 ones under a power of two per
            // head row that keeps them in the fp16 range.
            float sl2 = a.softmax_scale * LOG2E;
            {
                uint32_t x[DH / 32][16];
                const size_t at = head_row(mine ? m : 0) * D + half * DH;
                const bool in = mine && QSA_IN(at + DH - 1, (size_t)a.n_tokens * a.n_q_heads * D);
                const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) + (in ? at : 0));
#pragma unroll
                for (int j = 0; j < DH / 8; ++j)
                    *reinterpret_cast<uint4 *>(&x[j / 4][j % 4 * 4]) = in ? __ldg(src + j) : make_uint4(0u, 0u, 0u, 0u);
                if (a.dtype != QSA_F16) {
                    uint32_t top = 0u;
#pragma unroll
                    for (int j = 0; j < DH / 2; ++j) top = __vmaxu2(top, x[j / 16][j % 16] & 0x7FFF7FFFu);
                    top = max(top & 0xFFFFu, top >> 16);
                    sh.l[half][m] = __uint_as_float(top);
                    good = both(good);
                    top = max(top, __float_as_uint(sh.l[half ^ 1][m]));
                    const int ex = head_sum_exponent(__uint_as_float(top << 16));
                    const float f = exp2i(ex);
                    sl2 *= exp2i(-ex);
#pragma unroll
                    for (int j = 0; j < DH / 2; ++j) {
                        const uint32_t v = x[j / 16][j % 16];
                        x[j / 16][j % 16] = h2u(__floats2half2_rn(__uint_as_float(v << 16) * f, __uint_as_float(v & 0xFFFF0000u) * f));
                    }
                }
#pragma unroll
                for (int c = 0; c < DH / 32; ++c) tmem_st16(lane_base + G::Q_COL + half * (DH / 2) + 16 * c, x[c]);
                tmem_wait_st();
                fence_before();
                mbar_arrive(smem_u32(&sh.q_full));
            }
            float ref = -CUDART_INF_F, l = 0.0f;
            uint32_t poison = 0u;  // quarters of the dims whose value is NaN: an infinite or NaN V scale was attended to
            for (int i = i0; i < i1; ++i, ++k) {
                good = __all_sync(0xffffffffu, good && mbar_wait_or_abort(smem_u32(&sh.s_full[k & 1]), (k >> 1) & 1, abort));
                fence_after();
                float y[NH];
                {
                    uint32_t v[NH / 16][16];
#pragma unroll
                    for (int c = 0; c < NH / 16; ++c) tmem_ld16(lane_base + (k & 1) * N + j0 + 16 * c, v[c]);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < NH; ++j) {
                        asm volatile("" : "+r"(v[j / 16][j % 16]));  // not before the wait
                        y[j] = __uint_as_float(v[j / 16][j % 16]);
                    }
                }
                const float *kf = sh.kf[k % 3] + j0, *vb = sh.vb[k % 3] + j0, *vw = sh.vw[k % 3] + j0;
#pragma unroll
                for (int j = 0; j < NH; j += 4) {
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
                const uint4 bad0 = *reinterpret_cast<const uint4 *>(sh.poison[k % 3]), bad1 = *reinterpret_cast<const uint4 *>(sh.poison[k % 3] + 4);
                if (bad0.x | bad0.y | bad0.z | bad0.w | bad1.x | bad1.y | bad1.z | bad1.w) {
                    for (int w = 0; w < CONVERTERS / 32; ++w)
                        for (uint32_t bits = sh.poison[k % 3][w]; bits; bits &= bits - 1) {
                            const int b = __ffs(bits) - 1;
                            if (i * N + factor_cell(w, b) < len) poison |= 1u << (b & 3);
                        }
                }
                if (i * N > least - N) {  // some row ends in this tile
#pragma unroll
                    for (int j = 0; j < NH; ++j)
                        if (i * N + j0 + j >= len) y[j] = -CUDART_INF_F;
                }
                float top = -CUDART_INF_F;
#pragma unroll
                for (int j = 0; j < NH; j += 2) top = max3(top, y[j], y[j + 1]);
                sh.top[k & 1][half][m] = top;
                good = both(good);
                if (!good) break;
                top = fmaxf(top, sh.top[k & 1][half ^ 1][m]);
                // The reference moves only when a tile exceeds it by 2^SLACK.
                const bool up = top > ref + SLACK;
                const float alpha = up ? ex2(ref - top) : 1.0f;
                ref = up ? top : ref;
                l *= alpha;
                if (i > i0 && __any_sync(0xffffffffu, up)) {
                    // The values so far: each of the two scales half of them.
                    good = __all_sync(0xffffffffu, mbar_wait_or_abort(smem_u32(&sh.pv_full[(k - 1) & 1]), ((k - 1) >> 1) & 1, abort));
                    fence_after();
#pragma unroll 1
                    for (int c = 0; c < DH / 16 && good; ++c) {
                        uint32_t v[16];
                        tmem_ld16(lane_base + G::O_COL + half * DH + 16 * c, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            asm volatile("" : "+r"(v[j]));
                            v[j] = __float_as_uint(__uint_as_float(v[j]) * alpha);
                        }
                        tmem_st16(lane_base + G::O_COL + half * DH + 16 * c, v);
                    }
                    tmem_wait_st();
                }
                const float base = ref == -CUDART_INF_F ? 0.0f : -ref;
                float2 sum = make_float2(0.0f, 0.0f);
                uint32_t h[NH / 2], low[NH / 2];
#pragma unroll
                for (int c = 0; c < NH; c += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(vw + c);
                    float2 p0 = __fadd2_rn(make_float2(y[c], y[c + 1]), make_float2(base, base));
                    float2 p1 = __fadd2_rn(make_float2(y[c + 2], y[c + 3]), make_float2(base, base));
                    p0 = make_float2(ex2(p0.x), ex2(p0.y));
                    p1 = make_float2(ex2(p1.x), ex2(p1.y));
                    sum = __ffma2_rn(p0, make_float2(f.x, f.y), sum);
                    sum = __ffma2_rn(p1, make_float2(f.z, f.w), sum);
                    const __half2 h0 = __floats2half2_rn(p0.x, p0.y), h1 = __floats2half2_rn(p1.x, p1.y);
                    h[c / 2] = h2u(h0);
                    h[c / 2 + 1] = h2u(h1);
                    if (fine) {
                        low[c / 2] = h2u(__floats2half2_rn(p0.x - __low2float(h0), p0.y - __high2float(h0)));
                        low[c / 2 + 1] = h2u(__floats2half2_rn(p1.x - __low2float(h1), p1.y - __high2float(h1)));
                    }
                }
                l += sum.x + sum.y;
                // P in the place of S: both halves of its cells have been read.
                tmem_st16(lane_base + (k & 1) * N + half * (NH / 2), h);
                if (fine) tmem_st16(lane_base + (k & 1) * N + N / 2 + half * (NH / 2), low);
                tmem_wait_st();
                fence_before();
                if (good) mbar_arrive(smem_u32(&sh.p_full[k & 1]));
            }
            if (good && k > 0)
                good = mbar_wait_or_abort(smem_u32(&sh.pv_full[(k - 1) & 1]), ((k - 1) >> 1) & 1, abort);
            good = __all_sync(0xffffffffu, good);
            sh.l[half][m] = l;
            good = both(good);
            if (good) {
                // The values to shared memory, in place of the tiles (whose
                // products are done): 16-byte unit c of row m at c ^ (m % 8).
                fence_after();
                l += sh.l[half ^ 1][m];
                const bool none = ref == -CUDART_INF_F;
                const float scale = whole ? (none ? 0.0f : 1.0f / l) : 1.0f;
#pragma unroll 1
                for (int c = 0; c < DH / 16; c += 2) {
                    uint32_t v[2][16];
#pragma unroll
                    for (int i = 0; i < 2; ++i) tmem_ld16(lane_base + G::O_COL + half * DH + 16 * (c + i), v[i]);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) asm volatile("" : "+r"(v[i][4 * j + e]));
                            const float w = poison >> ((half * DH + 16 * (c + i)) / (D / 4)) & 1u ? CUDART_NAN_F : scale;
                            float *dst = values + m * D + 4 * ((half * (DH / 4) + 4 * (c + i) + j) ^ (m & 7));
                            *reinterpret_cast<float4 *>(dst) =
                                make_float4(__uint_as_float(v[i][4 * j]) * w, __uint_as_float(v[i][4 * j + 1]) * w,
                                            __uint_as_float(v[i][4 * j + 2]) * w, __uint_as_float(v[i][4 * j + 3]) * w);
                        }
                }
                if (mine && half == 0) {
                    if (!whole)
                        *reinterpret_cast<float2 *>(work.ml + (at * M + m) * 2) = make_float2(ref, l);
                    else if (a.lse)
                        a.lse[head_row(m)] = lse_of(ref, l);
                }
                fence_before();  // O is overwritten by the next segment
            }
            ok = good;
        }
        asm volatile("cp.async.wait_all;\n" ::: "memory");
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

    // After a time-out: copies on their way land before the block ends, and
    // products issued are complete before tensor memory is freed.
    if (warp >= LOADER && !ok) {
        for (int j = max(k - STAGES, 0); j < k; ++j)
            mbar_wait_bounded(smem_u32(&sh.full[warp - LOADER][j % STAGES]), (j / STAGES) & 1, DRAIN_LIMIT);
    }
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
    if (warp == PRODUCTS) {
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
