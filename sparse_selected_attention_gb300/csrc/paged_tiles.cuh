// Rows of q that read the same cells, together: attention over the paged cache on
// tcgen05, for drafted tokens (qsa_paged_tree_attn) and for tokens whose lists of
// pages are alike (qsa_paged_sparse_attn).
//
// The heads of such rows, up to 128, are the M side of products over one pass of the
// cells, so that a cell's codes are read and converted once for all of them.  A
// tree's rows go through their sequence, and see its end by bits; listed rows go
// through the pages that any of them lists (Union), and see a page by a bit.
//
// A CTA takes tiles of 128 cells (of 128 dims; 64 of 256); its warps have roles,
// which hand things over by mbarriers:
//   loads (1 warp): TMA boxes of codes, two tiles of K and of V ahead;
//   scales (2 warps): the factors of a tile's cells, and their powers of two;
//   converters (8 warps K, 4 V): codes to fp16 in shared memory, K by halves of the
//   dims, so that a half is converted again as soon as its products are done;
//   products (1 thread): S = Q K^T (Q in tensor memory), two buffers, and O += P V,
//   with S of the next tile issued before P V of this;
//   softmax (2 x 8 warps): two threads to a head row, half of a tile's cells each.  The
//   two sets take turns at the tiles: a row's reference maximum goes from one to
//   the other, and each keeps its own sums.
//
// Scales.  K's are multiplied into the codes, in two fp16 parts that hold the
// 19-bit product, V's likewise in one, each under a power of two that puts the
// tile's largest |scale| into [2^7, 2^8).  So a score needs one product and one sum,
// p = 2^(c S + d) with c and d of the row and tile, and nothing per cell.  Weights
// are 2^6 times those of the reference maximum, a whole number: a cell's product
// of weight and V scale then has as many bits above fp16's least step as if its own
// scale had set the maximum, where the tile's V scales lie within 2^SPREAD of one
// another.  Tiles whose scales do not (or K's not within 2^16: rare, by a few odd
// cells) are marked, and take a power of two per cell.
//
// What bounds it.  24 trees of 16 to 32 tokens over up to 8 K cells, 32/8 heads of 128: 132 us,
// 355 TFLOP/s; 63 tokens over 30 K cells, 24/2 of 256: 100 us, 465 TFLOP/s; 1984 tokens
// over 2 K listed cells each, 12/1 of 128: 138 us.  Tensor pipe 39 to 42 % busy, issue
// slots 67 %: a tile of 128 cells takes 4.1 K cycles, of which its products take 2.1 K, the
// conversion of K 3 K, the softmax of one set 5 K of 8.2 K.  Each role is near its own
// latency, so that more of one thing brings little.  In the cases' order: 64-cell tiles by
// four sets 192, 114 and 213 us where two sets took 129, 114 and 149; two warps for the two
// products 140, 140 and 148; roles that go on to the next segment by themselves 133, 116 and
// 149; all softmax warps on one tile 125, 117 and 140 where this took 128, 112 and 139 then;
// unrolled conversion 131, 114 and 145 (129, 112 and 143).  Beginning and end of a share
// cost 12 us of 100, mostly first fetches of instructions.
#pragma once

#include "paged_rows.cuh"

namespace qsa {
namespace {

using namespace tc;

constexpr int M = GROUP_ROWS;
constexpr int SOFTMAX = 512, K_WARPS = 8, V_WARPS = 4, SCALERS = 2;
constexpr int V_FIRST = SOFTMAX / 32 + K_WARPS, PRODUCTS = V_FIRST + V_WARPS, LOADER = PRODUCTS + 1, SCALER = LOADER + 1, WARPS = SCALER + SCALERS;
constexpr int THREADS = 32 * WARPS;
constexpr int STAGES = 2;  // tiles of codes on their way
constexpr int INFOS = 4;   // tiles of factors
constexpr int SPREAD = 6, K_SPREAD = 16;
constexpr int LIFT = 6;    // weights are 2^LIFT times those of the reference maximum
constexpr uint32_t SAW = 1u << 31;  // beside the quarters that are NaN
constexpr int CHUNK = 1024;  // tokens that are looked up at once, one a thread; groups end where one ends
static_assert(CHUNK == THREADS, "a thread per token");

template <int S>
struct TileShape {
    static constexpr int D = 128 * S, BLOCKS = D / 64;     // of 64 dims
    static constexpr int N = 128 / S, PARTS = N / 32;      // cells of a tile; 32 of them have a power of two of their own
    static constexpr uint32_t TMEM_COLS = 512, Q_COL = 2 * N, O_COL = Q_COL + D / 2;  // S at 0 and N, P in its place
    static_assert(O_COL + D <= TMEM_COLS, "tensor memory");
    static constexpr uint32_t IDESC_S = idesc_f16(M, N, false, false), IDESC_O = idesc_f16(M, D, false, true);
};
// The group that starts at a token: its head rows (0: none starts), from head `head` of
// the token on, the fewest cells that a token of it sees for certain and the most that
// one goes through.  A tree's head rows fill groups one after the other, whatever tokens
// they are of (63 tokens of 12 heads: six groups; seven of ten whole tokens); a group of
// listed rows has whole tokens.
template <int S>
struct TileGroup {
    int rows, least, most, trow, head;
    __device__ __forceinline__ int tiles() const {
        constexpr int N = TileShape<S>::N;
        return rows ? max((most + N - 1) / N, 1) : 0;
    }
};

template <int N>
struct alignas(16) Info {  // of a tile's cells
    float kf[N], vb[N], vw[N];      // by cell, of a marked tile: 2^-ek, -ev, 2^ev
    uint2 fk[N], fv[N];             // the four factors of K and V
    float ck[N / 32], cb[N / 32], cw[N / 32];  // of all of 32 cells, of the others
    uint32_t there[N / 32];
    uint8_t poison[N];              // quarters whose V scale is infinite or NaN
    uint2 unit[N / 16];             // of listed pages, by 16 cells: the first one's place in the sequence, and the tokens that list it
    int flags[N / 32];
};
constexpr int MARKED = 1, POISONED = 2, GAPS = 4, WILD = 8;  // GAPS: some cell is not there; WILD: a K scale is infinite or NaN

// Tiles of rows of 64 halves (128 bytes), 16-byte unit u of row r at u ^ (r % 8).
template <int S>
struct TileSmem {
    using G = TileShape<S>;
    static constexpr int N = G::N;
    uint8_t k[2][2][S][N * 128];         // halves of the dims, high and low part
    uint8_t v[2][G::BLOCKS][N * 128];
    uint8_t codes[2][STAGES][S][N * 128];  // K's and V's as they come, by 128 dims
    Info<N> info[INFOS];
    uint2 scales[3][2][N], unit[3][N / 16];
    float top[2][2][M], ref[2][M], l[4][M], lref[4][M];
    uint32_t poison[4][M];
    uint64_t full[2][STAGES], empty[2][STAGES];  // codes
    uint64_t info_full[INFOS], info_empty[INFOS];
    uint64_t k_full[2], k_empty[2], v_full[2], s_full[2], p_full[2], pv_full[2], ref_full[2];
    uint64_t q_full, drain;
    long long scan[WARPS], saved[WARPS];
    unsigned starts[CHUNK / 32];
    TileGroup<S> next;
    long long before;
    int t;
    TileGroup<S> grp;
    int abort;
    uint32_t tmem;
};

__device__ __forceinline__ uint32_t tile_unit(int r, int u) { return r * 128 + ((u ^ (r & 7)) << 4); }
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0u;
}
// 32 columns, there when this returns.
__device__ __forceinline__ void tmem_read32(uint32_t taddr, uint32_t (&v)[2][16]) {
    tmem_ld16(taddr, v[0]);
    tmem_ld16(taddr + 16, v[1]);
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0][0]), "+r"(v[0][1]), "+r"(v[0][2]), "+r"(v[0][3]), "+r"(v[0][4]), "+r"(v[0][5]), "+r"(v[0][6]), "+r"(v[0][7]),
                   "+r"(v[0][8]), "+r"(v[0][9]), "+r"(v[0][10]), "+r"(v[0][11]), "+r"(v[0][12]), "+r"(v[0][13]), "+r"(v[0][14]), "+r"(v[0][15]));
    asm volatile(""
                 : "+r"(v[1][0]), "+r"(v[1][1]), "+r"(v[1][2]), "+r"(v[1][3]), "+r"(v[1][4]), "+r"(v[1][5]), "+r"(v[1][6]), "+r"(v[1][7]),
                   "+r"(v[1][8]), "+r"(v[1][9]), "+r"(v[1][10]), "+r"(v[1][11]), "+r"(v[1][12]), "+r"(v[1][13]), "+r"(v[1][14]), "+r"(v[1][15]));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
// The rest of a wait whose first look did not see the phase completed; in one
// place, since every line of the roles' loops counts in the instruction cache.
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int *abort) { return mbar_wait_or_abort(bar, parity, abort); }
// Two values of the output, gated, as they are stored.
template <bool FINE>
__device__ __forceinline__ uint32_t tile_value(const qsa_paged_attn_args &a, size_t at, float2 y) {
    if (a.gate) {
        const float2 g = __ldg(reinterpret_cast<const float2 *>(a.gate + at));
        y = make_float2(gated(y.x, g.x), gated(y.y, g.y));
    }
    if constexpr (FINE) return h2u(__floats2half2_rn(y.x, y.y));
    const __nv_bfloat162 b = __floats2bfloat162_rn(y.x, y.y);
    return *reinterpret_cast<const uint32_t *>(&b);
}
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 512;" ::: "memory"); }

// The group that starts at head `head` of t, looked up by a warp.
template <int S, class A>
__device__ __forceinline__ TileGroup<S> group_at(const A &a, int kvh, int t, int head, int per, bool &bad) {
    if constexpr (LISTED<A>) {
        const int size = __ldcg(a.shared.size + (size_t)kvh * a.n_tokens + t);
        return TileGroup<S>{(size >> SIZE_BITS) * per, 0, (size & SIZE_MASK) * a.page_size, 0, 0};
    }
    const int lane = threadIdx.x & 31, row = __ldg(a.rows + t);
    const int end = min(min(a.n_tokens, t + (head + M + per - 1) / per), (t | (CHUNK - 1)) + 1);
    TileGroup<S> g{0, 0x7fffffff, 0, row >= 0 && row < a.n_rows ? row : 0, head};
    int tokens = 0;
    for (bool more = true; more && t + tokens < end;) {
        const int u = t + tokens + lane;
        int trow, len = 0, sure = 0;
        const bool same = u < end && __ldg(a.rows + u) == row;
        if (same) len = row_len(a, u, 0, trow, sure, bad);
        const unsigned m = __ballot_sync(0xffffffffu, same);
        const int k = m == 0xffffffffu ? 32 : __ffs(~m) - 1;
        if (lane < k) {
            g.least = min(g.least, sure);
            g.most = max(g.most, len);
        }
        tokens += k;
        more = k == 32;
    }
    g.rows = min(tokens * per - head, M);
    g.least = __reduce_min_sync(0xffffffffu, g.least);
    g.most = __reduce_max_sync(0xffffffffu, g.most);
    return g;
}

// Scale i of a cell times 2^e.
__device__ __forceinline__ uint2 scales_by(uint2 sc, int e) {
    const float f = exp2i(e);
    const __half2 a = u2h(sc.x), b = u2h(sc.y);
    return make_uint2(h2u(__floats2half2_rn(__low2float(a) * f, __high2float(a) * f)),
                      h2u(__floats2half2_rn(__low2float(b) * f, __high2float(b) * f)));
}

// FINE: weights in two parts, for results in fp16.
template <int S, bool FINE, class A>
__global__ void __launch_bounds__(THREADS, 1)
    paged_tiles_kernel(const A a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, void *ws) {
    using G = TileShape<S>;
    constexpr int D = G::D, N = G::N, BLOCKS = G::BLOCKS, PARTS = G::PARTS;
    extern __shared__ __align__(1024) uint8_t raw[];
    TileSmem<S> &sh = *reinterpret_cast<TileSmem<S> *>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = a.n_q_heads / a.n_kv_heads, page_shift = 31 - __clz(a.page_size);
    const uint32_t per_inv = 65536u / per + 1;
    const int kvh = blockIdx.x % a.n_kv_heads, range = blockIdx.x / a.n_kv_heads, ranges = gridDim.x / a.n_kv_heads;
    volatile int *abort = &sh.abort;
    if (tid == 0) {
        for (int b = 0; b < 2; ++b) {
            for (int i = 0; i < STAGES; ++i) {
                mbar_init(smem_u32(&sh.full[b][i]), 1);
                mbar_init(smem_u32(&sh.empty[b][i]), b ? V_WARPS : K_WARPS);
            }
            mbar_init(smem_u32(&sh.k_full[b]), K_WARPS);
            mbar_init(smem_u32(&sh.k_empty[b]), 1);
            mbar_init(smem_u32(&sh.v_full[b]), V_WARPS);
            mbar_init(smem_u32(&sh.s_full[b]), 1);
            mbar_init(smem_u32(&sh.p_full[b]), 2 * M);
            mbar_init(smem_u32(&sh.pv_full[b]), 1);
            mbar_init(smem_u32(&sh.ref_full[b]), 2 * M / 32);
        }
        for (int i = 0; i < INFOS; ++i) {
            mbar_init(smem_u32(&sh.info_full[i]), 32 * SCALERS);
            mbar_init(smem_u32(&sh.info_empty[i]), 2 * M / 32 + V_WARPS);
        }
        mbar_init(smem_u32(&sh.q_full), SOFTMAX);
        mbar_init(smem_u32(&sh.drain), 1);
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == PRODUCTS) tmem_alloc(smem_u32(&sh.tmem), G::TMEM_COLS);
    wait_for_previous_grid();
    allow_dependent_launch();
    const Work work(ws, MAX_GROUP_PARTS, M);
    bool bad = false;

    // The groups' tiles, and the group in which this CTA's share of them starts.
    // Loops, as all of this kernel that runs once or rarely: an instruction's first
    // fetch costs more than its execution (unrolled, this took 9 us of 63 tokens').
    int share = 0, left = 0, t = 0;
    TileGroup<S> grp;
    if constexpr (LISTED<A>) {
        // The groups are there already; whether they are taken is the same for all of a
        // KV head's CTAs, and for the kernel of rows one by one, which reads it.
        const int run = (a.n_tokens + THREADS - 1) / THREADS, t0 = min(tid * run, a.n_tokens), t1 = min(t0 + run, a.n_tokens);
        long long tiles = 0, saved = 0;
        int trow, most = 0;
#pragma unroll 1
        for (int u = t0; u < t1; ++u) {
            const TileGroup<S> g = group_at<S>(a, kvh, u, 0, per, bad);
            const int units = units_of<S>(row_len(a, u, kvh, trow, bad));
            most = max(most, units);
            tiles += g.tiles();
            saved += saved_by(units, g.tiles());
            if (g.most == SIZE_MASK * a.page_size) saved -= 1ll << 40;
        }
        long long sum = tiles;
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, sum, o), w = __shfl_xor_sync(0xffffffffu, saved, o);
            if (lane >= o) sum += v;
            saved += w;
        }
        if (lane == 31) {
            sh.scan[warp] = sum;
            sh.saved[warp] = saved;
        }
        const bool longer = __syncthreads_or(most > WHOLE);
        long long before = lane < warp ? sh.scan[lane] : 0, total = sh.scan[lane];
        saved = sh.saved[lane];
#pragma unroll 1
        for (int o = 16; o > 0; o >>= 1) {
            before += __shfl_xor_sync(0xffffffffu, before, o);
            total += __shfl_xor_sync(0xffffffffu, total, o);
            saved += __shfl_xor_sync(0xffffffffu, saved, o);
        }
        const bool taken = longer && saves_enough(a, saved);
        if (range == 0 && tid == 0) a.taken[kvh] = taken;
        if (taken) {
            share = (int)max((total + ranges - 1) / ranges, 1ll);
            const long long x = (long long)share * range;
            left = (int)max(min((long long)share, total - x), 0ll);
            before += sum - tiles;
            if (x >= before && x < before + tiles) {
#pragma unroll 1
                for (int u = t0; u < t1; ++u) {
                    const TileGroup<S> g = group_at<S>(a, kvh, u, 0, per, bad);
                    if (x < before + g.tiles()) {
                        sh.t = u;
                        sh.before = before;
                        sh.grp = g;
                        break;
                    }
                    before += g.tiles();
                }
            }
        }
    } else {
        int *srow = reinterpret_cast<int *>(sh.k), *most = srow + CHUNK, *least = most + CHUNK, *size = least + CHUNK;
        long long total = 0, x = 0, done = 0, saved = 0;
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {  // the tiles; then where the share starts
#pragma unroll 1
            for (int base = 0; base < a.n_tokens; base += CHUNK) {
                if (pass && a.n_tokens <= CHUNK) break;  // found already
                const int u = base + tid;
                const bool in = u < a.n_tokens;
                int row = 0, trow = 0, len = 0, sure = 0;
                if (in) {
                    row = __ldg(a.rows + u);
                    len = row_len(a, u, 0, trow, sure, bad);
                }
                __syncthreads();  // of the chunk before
                srow[tid] = row;
                most[tid] = 0;
                least[tid] = 0x7fffffff;
                size[tid] = 0;
                __syncthreads();
                // Where the token's run of one sequence starts: in its warp, or before.
                const unsigned starts = __ballot_sync(0xffffffffu, in && (tid == 0 || srow[tid - 1] != row));
                if (lane == 0) sh.starts[warp] = starts;
                __syncthreads();
                unsigned mine = starts & (0xffffffffu >> (31 - lane));
                int w = warp;
                while (!mine && w > 0) mine = sh.starts[--w];
                // The groups of its head rows, one or two, and the tokens that those start at.
                const int start = w * 32 + 31 - __clz(mine), from = (tid - start) * per, to = from + per;
                for (int i = from / M; in && i * M < to; ++i) {
                    const int lead = start + i * M / per;
                    atomicMax(most + lead, len);
                    atomicMin(least + lead, sure);
                    atomicAdd(size + lead, min(to, i * M + M) - max(from, i * M));
                }
                __syncthreads();
                const int own = (from + M - 1) / M * M;  // where a group starts, if before `to`
                const TileGroup<S> g{in && own < to ? size[tid] : 0, least[tid], most[tid], trow, own - from};
                const int tiles = g.tiles();
                if (!pass && in) saved += saved_by(units_of<S>(len), tiles);
                long long sum = tiles;
#pragma unroll 1
                for (int o = 1; o < 32; o <<= 1) {
                    const long long v = __shfl_up_sync(0xffffffffu, sum, o);
                    if (lane >= o) sum += v;
                }
                if (lane == 31) sh.scan[warp] = sum;
                __syncthreads();
                long long before = done + sum - tiles, all = sh.scan[lane];
                if (lane >= warp) all = 0;  // of the warps before
#pragma unroll 1
                for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
                before += all;
                const long long chunk = sh.scan[lane];
                all = chunk;
#pragma unroll 1
                for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
                if (!pass) total += all;
                done += all;
                if (pass || a.n_tokens <= CHUNK) {
                    if (!pass) {
                        share = (int)max((total + ranges - 1) / ranges, (long long)S);
                        x = (long long)share * range;
                    }
                    if (tiles && x >= before && x < before + tiles) {
                        sh.t = u;
                        sh.before = before;
                        sh.grp = g;
                    }
                }
            }
            if (!pass) {
                share = (int)max((total + ranges - 1) / ranges, (long long)S);
                x = (long long)share * range;
                done = 0;
            }
        }
        left = (int)max(min((long long)share, total - x), 0ll);
        if constexpr (TREE<A>) {
            if (a.taken) {  // else they are taken whatever it saves
#pragma unroll 1
                for (int o = 16; o > 0; o >>= 1) saved += __shfl_xor_sync(0xffffffffu, saved, o);
                if (lane == 0) sh.saved[warp] = saved;
                __syncthreads();
                saved = sh.saved[lane];
#pragma unroll 1
                for (int o = 16; o > 0; o >>= 1) saved += __shfl_xor_sync(0xffffffffu, saved, o);
                const bool taken = saves_enough(a, saved);
                if (range == 0 && tid == 0) a.taken[kvh] = taken;
                if (!taken) left = 0;
            }
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    constexpr uint32_t tmem = 0u;  // all columns are this block's
    Part part{-1, 0, 0, 0};
    bool ok = true, issued = false;  // issued: products, by this thread
    int k = 0;  // tiles done: the barriers' phases
    int i0 = 0;
    if (left > 0) {
        t = sh.t;
        grp = sh.grp;
        i0 = (int)((long long)share * range - sh.before);
    }
    uint32_t segment = 0;
    int sent[2] = {0, 0};  // tiles of K's and V's codes asked for, by the loader

    for (bool first = true; left > 0; first = false, ++segment) {
        // Segment: tiles i0 .. i1-1 of the group at t.
        const int tiles = grp.tiles(), i1 = min(tiles, i0 + left), n = i1 - i0, rows = grp.rows;
        const bool whole = n == tiles;
        const size_t at = (size_t)blockIdx.x * 2 + (first && i0 > 0 ? 0 : 1);
        const int head = LISTED<A> ? 0 : grp.head;
        auto token_of = [&](int m) { return t + (int)((uint32_t)(head + m) * per_inv >> 16); };  // (head + m) / per, below 144
        auto head_row = [&](int m) -> size_t {  // of q
            const int u = token_of(m);
            return (size_t)u * a.n_q_heads + (size_t)kvh * per + (head + m - (u - t) * per);
        };
        const int32_t *tab = a.page_table + (size_t)grp.trow * a.max_pages;
        const int *pages = nullptr;  // of a union, and what tokens see of them
        const uint2 *units = nullptr;
        if constexpr (LISTED<A>) {
            pages = a.shared.page + ((size_t)kvh * a.n_tokens + t) * a.width;
            units = a.shared.unit + ((size_t)kvh * a.n_tokens + t) * a.width;
        }
        bool good = true;
        auto wait = [&](uint64_t &bar, int phase) {
            if (WAIT_LIMIT == 0 || !mbar_try_wait(smem_u32(&bar), phase & 1)) good = good && wait_on(smem_u32(&bar), phase & 1, abort);
            good = __all_sync(0xffffffffu, good);
            return good;
        };

        if (warp == LOADER) {
            // ---- codes: a lane takes a box of a page's cells ----
            const int box = min(a.page_size, N), boxes = N / box;
            for (int i = 0; i < n; ++i) {
                const int kk = k + i, st = kk % STAGES, c = (i0 + i) * N + lane * box, j = c >> page_shift;
                const bool want = lane < boxes && c < grp.most;
                int page = -1;
                if constexpr (LISTED<A>)
                    page = want ? __ldcg(pages + j) : -1;
                else if (want && j < a.max_pages)
                    page = __ldg(tab + j);
                const bool there = page >= 0 && page < a.n_pages;
                const int cell = (page << page_shift) + (c & (a.page_size - 1));
                const unsigned m = __ballot_sync(0xffffffffu, there);
#pragma unroll
                for (int kind = 0; kind < 2; ++kind) {
                    if (kk >= STAGES && !wait(sh.empty[kind][st], kk / STAGES - 1)) break;
                    const uint32_t bar = smem_u32(&sh.full[kind][st]);
                    sent[kind] = kk + 1;
                    if (lane == 0) expect_tx(bar, __popc(m) * box * D);
                    __syncwarp();
                    if (there) {
#pragma unroll
                        for (int x = 0; x < S; ++x)
                            tma_box(smem_u32(sh.codes[kind][st][x]) + lane * box * 128, kind ? &vmap : &kmap, 128 * x, kvh, cell, bar);
                    }
                }
                if (!good) break;
            }
            if (left > n) {  // the next group, for all
                const int end = head + rows;
                const TileGroup<S> g = group_at<S>(a, kvh, t + end / per, end % per, per, bad);
                if (lane == 0) sh.next = g;
            }
        } else if (warp >= SCALER) {
            // ---- factors: 32 cells of each tile ----
            // A lane copies its cells' scales two tiles ahead and reads no others; their
            // pages are looked up a tile before that.
            constexpr int MINE = PARTS / SCALERS;
            const int part0 = warp - SCALER;
            int page[MINE];
            uint2 unit[MINE];
            auto look = [&](int i) {  // up the pages of tile i
#pragma unroll
                for (int p = 0; p < MINE; ++p) {
                    const int c = (i0 + i) * N + (part0 + p * SCALERS) * 32 + lane, j = c >> page_shift;
                    if constexpr (LISTED<A>) {
                        const bool want = i < n && c < grp.most;
                        page[p] = want ? __ldcg(pages + j) : -1;
                        unit[p] = want && !(lane & 15) ? __ldcg(units + j) : make_uint2(0u, 0u);
                    } else {
                        page[p] = i < n && c < grp.most && j < a.max_pages ? __ldg(tab + j) : -1;
                    }
                }
            };
            uint32_t held = 0u;  // whether the cells are there: MINE bits a tile, the latest lowest
            auto copy = [&](int i) {
#pragma unroll
                for (int p = 0; p < MINE; ++p) {
                    const int cell = (part0 + p * SCALERS) * 32 + lane, c = (i0 + i) * N + cell;
                    bool there = page[p] >= 0 && page[p] < a.n_pages;
                    const size_t r = (((size_t)(there ? page[p] : 0) << page_shift) + (c & (a.page_size - 1))) * a.n_kv_heads + kvh;
                    there = there && QSA_IN(r, (size_t)a.n_pages * a.page_size * a.n_kv_heads);
                    cp_async8(smem_u32(&sh.scales[i % 3][0][cell]), a.ksc + (there ? r * 4 : 0), there);
                    cp_async8(smem_u32(&sh.scales[i % 3][1][cell]), a.vsc + (there ? r * 4 : 0), there);
                    held = held << 1 | (there ? 1u : 0u);
                    if constexpr (LISTED<A>) {
                        if (!(lane & 15)) sh.unit[i % 3][cell / 16] = make_uint2((unit[p].x << page_shift) + (c & (a.page_size - 1)), unit[p].y);
                    }
                }
                asm volatile("cp.async.commit_group;\n" ::);
                look(i + 1);
            };
            look(0);
            copy(0);
            copy(1);
#pragma unroll 1
            for (int i = 0; i < n; ++i) {
                const int kk = k + i, slot = kk % INFOS;
                if (kk >= INFOS && !wait(sh.info_empty[slot], kk / INFOS - 1)) break;
                copy(i + 2);
                asm volatile("cp.async.wait_group 2;\n" ::: "memory");
                Info<N> &f = sh.info[slot];
#pragma unroll 1
                for (int p = 0; p < MINE; ++p) {
                    const int part = part0 + p * SCALERS, cell = part * 32 + lane;
                    const uint2 ks = sh.scales[i % 3][0][cell], vs = sh.scales[i % 3][1][cell];
                    // The exponents of the largest scales; cells whose scales are 0 have none.
                    int ke = scale_exponent(ks), ve = scale_exponent(vs);
                    const int kmost = __reduce_max_sync(0xffffffffu, ke), vmost = __reduce_max_sync(0xffffffffu, ve);
                    const int kleast = __reduce_min_sync(0xffffffffu, ke > NO_SCALE ? ke : 127);
                    const int vleast = __reduce_min_sync(0xffffffffu, ve > NO_SCALE ? ve : 127);
                    const unsigned here = __ballot_sync(0xffffffffu, held >> (3 * MINE - 1 - p) & 1u);
                    const bool marked = kmost - kleast > K_SPREAD || vmost - vleast > SPREAD;
                    if (!marked) {
                        ke = kmost;
                        ve = vmost;
                    }
                    // A V scale that is infinite or NaN counts as 0 here: times a
                    // weight of 0 it would reach rows that do not see its cell.
                    const uint2 fin = make_uint2(finite2(vs.x), finite2(vs.y));
                    f.fk[cell] = scales_by(ks, 7 - ke);
                    f.fv[cell] = scales_by(fin, 7 - ve);
                    const uint32_t x = vs.x ^ fin.x, y = vs.y ^ fin.y;
                    const bool any = __any_sync(0xffffffffu, (x | y) != 0u);
                    bool wild = false;
                    if constexpr (LISTED<A>) {
                        wild = __any_sync(0xffffffffu, finite2(ks.x) != ks.x || finite2(ks.y) != ks.y);
                        if (!(lane & 15)) f.unit[cell / 16] = sh.unit[i % 3][cell / 16];
                    }
                    // What the softmax asks for of each cell, where it does.
                    f.kf[cell] = exp2i(ke - 7);
                    f.vb[cell] = (float)(ve - 7);
                    f.vw[cell] = exp2i(7 - ve);
                    if (any)
                        f.poison[cell] = (uint8_t)(((x & 0x7C00u) ? 1u : 0u) | ((x >> 16 & 0x7C00u) ? 2u : 0u) | ((y & 0x7C00u) ? 4u : 0u) |
                                                   ((y >> 16 & 0x7C00u) ? 8u : 0u));
                    if (lane == 0) {
                        f.ck[part] = exp2i(kmost - 7);
                        f.cb[part] = (float)(vmost - 7);
                        f.cw[part] = exp2i(7 - vmost);
                        f.there[part] = here;
                        f.flags[part] = (marked ? MARKED : 0) | (any ? POISONED : 0) | (here == 0xffffffffu ? 0 : GAPS) | (wild ? WILD : 0);
                    }
                }
                mbar_arrive(smem_u32(&sh.info_full[slot]));
            }
            asm volatile("cp.async.wait_group 0;\n" ::: "memory");
        } else if (warp >= SOFTMAX / 32 && warp < PRODUCTS) {
            // ---- conversion: sixteen codes of a cell at a time, eight cells a warp ----
            // Two cells' lanes, four to each, read and write together; the cells'
            // numbers differ in bits 0 and 2, so that they meet a bank once.
            const int u4 = lane & 3, in8 = (lane >> 3) ^ (lane >> 2 & 1) * 5;
            // Dims 64 c .. of a cell; factors: its four.
            auto convert = [&](auto part, const uint8_t *codes, const uint2 *factors, int cell, int c, uint8_t *hi, uint8_t *lo) {
                constexpr bool TWO = decltype(part)::value;
                const uint4 w = *reinterpret_cast<const uint4 *>(codes + tile_unit(cell, 4 * (c & 1) + u4));
                const int q = S == 2 ? c : 2 * c + (u4 >> 1);  // the quarter: 64 dims of 256, or 32 of 128
                const __half2 s = __half2half2(reinterpret_cast<const __half *>(factors + cell)[q]);
                const uint32_t x[4] = {w.x ^ 0x80808080u, w.y ^ 0x80808080u, w.z ^ 0x80808080u, w.w ^ 0x80808080u};
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint32_t to = tile_unit(cell, 2 * u4 + u);
                    uint32_t h[4], l[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const __half2 v = __hsub2(u2h(prmt(x[2 * u + e / 2], 0x64646464u, e & 1 ? 0x4342 : 0x4140)), u2h(0x64806480u));
                        const __half2 p = __hmul2(v, s);
                        h[e] = h2u(p);
                        if constexpr (TWO) l[e] = h2u(__hfma2(v, s, __hneg2(p)));
                    }
                    *reinterpret_cast<uint4 *>(hi + to) = make_uint4(h[0], h[1], h[2], h[3]);
                    if constexpr (TWO) *reinterpret_cast<uint4 *>(lo + to) = make_uint4(l[0], l[1], l[2], l[3]);
                }
            };
            auto arrive = [&](uint64_t &bar) {
                if (lane == 0) mbar_arrive(smem_u32(&bar));
            };
            if (warp < V_FIRST) {
                constexpr int ITEMS = N / (8 * K_WARPS);  // of 64 dims
                const int cell0 = (warp - SOFTMAX / 32) * 8 + in8;
                for (int i = 0; i < n; ++i) {
                    const int kk = k + i, st = kk % STAGES;
                    wait(sh.full[0][st], kk / STAGES);
                    if (!wait(sh.info_full[kk % INFOS], kk / INFOS)) break;
                    // Loops are kept short: the roles' code shares the instruction caches.
#pragma unroll 1
                    for (int b = 0; b < 2; ++b) {
                        if (kk > 0 && !wait(sh.k_empty[b], kk - 1)) break;
#pragma unroll 1
                        for (int j = 0; j < ITEMS * S; ++j) {
                            const int c = b * S + j % S;
                            convert(std::true_type{}, sh.codes[0][st][c >> 1], sh.info[kk % INFOS].fk, cell0 + j / S * 8 * K_WARPS, c, sh.k[b][0][j % S],
                                    sh.k[b][1][j % S]);
                        }
                        fence_async_smem();
                        __syncwarp();
                        arrive(sh.k_full[b]);
                    }
                    if (!good) break;
                    arrive(sh.empty[0][st]);
                }
            } else {
                constexpr int ITEMS = N / (8 * V_WARPS);
                const int cell0 = (warp - V_FIRST) * 8 + in8;
                for (int i = 0; i < n; ++i) {
                    const int kk = k + i, st = kk % STAGES, b = kk & 1;
                    wait(sh.full[1][st], kk / STAGES);
                    wait(sh.info_full[kk % INFOS], kk / INFOS);
                    if (kk > 1) wait(sh.pv_full[b], (kk - 2) >> 1);
                    if (!good) break;
#pragma unroll 1
                    for (int j = 0; j < ITEMS * BLOCKS; ++j)
                        convert(std::false_type{}, sh.codes[1][st][j % BLOCKS >> 1], sh.info[kk % INFOS].fv, cell0 + j / BLOCKS * 8 * V_WARPS,
                                j % BLOCKS, sh.v[b][j % BLOCKS], nullptr);
                    fence_async_smem();
                    __syncwarp();
                    arrive(sh.v_full[b]);
                    arrive(sh.empty[1][st]);
                    arrive(sh.info_empty[kk % INFOS]);
                }
            }
        } else if (warp == PRODUCTS) {
            // ---- products ----
            // The whole warp goes through the loop; one lane issues.  Addresses are
            // constants or the same in all lanes (each buffer has its code): a product
            // takes 64 cycles or fewer, so what its issue takes counts.
            const bool one = elect_one();
            const uint64_t dk = sw128_kmajor(smem_u32(sh.k[0][0][0]));
            // V transposed: 64 dims apart N * 128 bytes, eight cells 1024.
            const uint64_t dv = smem_desc(smem_u32(sh.v[0][0]), N * 128, 1024, 2);
            auto issue_s = [&](auto buffer, int kk) {
                constexpr int B = decltype(buffer)::value;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (!wait(sh.k_full[half], kk)) return;
                    fence_after();
                    if (one) {
#pragma unroll
                        for (int x = 0; x < 2 * S; ++x)  // 64 dims: high parts, then low parts
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                mma_f16_ts(B * N, G::Q_COL + half * (S * 32) + x % S * 32 + ks * 8,
                                           dk + (uint64_t)((half * 2 * S + x) * (N * 8) + ks * 2), G::IDESC_S, half | x | ks ? 1u : 0u);
                        mma_commit(smem_u32(&sh.k_empty[half]));
                        if (half) mma_commit(smem_u32(&sh.s_full[B]));
                    }
                    __syncwarp();
                }
                issued |= one;
            };
            auto issue_o = [&](auto buffer, int kk, bool more) {
                constexpr int B = decltype(buffer)::value;
                wait(sh.v_full[B], kk >> 1);
                if (!wait(sh.p_full[B], kk >> 1)) return;
                fence_after();
                if (one) {
#pragma unroll
                    for (int ks = 0; ks < N / 16; ++ks) {  // sixteen columns for sixteen cells: high parts, low parts
                        const uint64_t d = dv + (uint64_t)(B * (BLOCKS * N * 8) + ks * 16 * 8);
                        mma_f16_ts(G::O_COL, B * N + ks * 16, d, G::IDESC_O, ks ? 1u : (uint32_t)more);
                        if (FINE) mma_f16_ts(G::O_COL, B * N + ks * 16 + 8, d, G::IDESC_O, 1u);
                    }
                    mma_commit(smem_u32(&sh.pv_full[B]));
                }
                __syncwarp();
            };
            auto of_buffer = [&](int b, auto &&f) {
                if (b)
                    f(std::integral_constant<int, 1>{});
                else
                    f(std::integral_constant<int, 0>{});
            };
            wait(sh.q_full, segment);
#pragma unroll 1
            for (int i = -1; i < n && good; ++i) {
                if (i + 1 < n) {  // S of the next tile
                    const int kk = k + i + 1;
                    if (kk > 1) wait(sh.pv_full[kk & 1], (kk - 2) >> 1);  // the buffer holds P kk - 2
                    if (!good) break;
                    of_buffer(kk & 1, [&](auto c) { issue_s(c, kk); });
                }
                if (i < 0 || !good) continue;
                const int kk = k + i;
                of_buffer(kk & 1, [&](auto c) { issue_o(c, kk, i > 0); });
            }
        } else {
            // ---- softmax: tiles k + i of one parity, half of the cells, of a head row ----
            // Tensor memory and barriers want the warp's threads together: a __syncwarp
            // stands where rows may have gone different ways before.
            constexpr int DQ = D / 4, H = N / 2;
            const int m = tid & (M - 1), wg = tid / M, set = wg >> 1, half = wg & 1;
            const bool mine = m < rows;
            const uint32_t lane_base = tmem + ((uint32_t)(warp % 4 * 32) << 16);
            const int token = token_of(m);
            int len = 0, sure = 0, tr;
            if (mine) {
                if constexpr (LISTED<A>)
                    sure = row_cells(a, token, tr, bad);
                else
                    len = row_len(a, token, 0, tr, sure, bad);
            }
            // Of the two warps that share their head rows and tiles.  Both come here once
            // a tile whatever they waited for, and go on or stop together.
            auto both = [&](bool fine) {
                int r;
                asm volatile("{\n.reg .pred p, q;\nsetp.ne.s32 p, %1, 0;\nbar.red.and.pred q, %2, 64, p;\nselp.s32 %0, 1, 0, q;\n}\n"
                             : "=r"(r)
                             : "r"((int)fine), "r"(2 + set * 4 + warp % 4)
                             : "memory");
                return r != 0;
            };
            // The queries to tensor memory, a quarter of the dims by each; bf16 ones
            // under a power of two per head row that keeps them in the fp16 range.  A
            // negative softmax scale flips their sign.
            const bool flip = a.softmax_scale < 0.0f;
            float sl2 = fabsf(a.softmax_scale) * LOG2E;
            {
                const size_t from = head_row(mine ? m : 0) * D + wg * DQ;
                const bool in = mine && QSA_IN(from + DQ - 1, (size_t)a.n_tokens * a.n_q_heads * D);
                const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) + (in ? from : 0));
                uint32_t x[DQ / 32][16];
#pragma unroll
                for (int j = 0; j < DQ / 8; ++j) *reinterpret_cast<uint4 *>(&x[j / 4][j % 4 * 4]) = in ? __ldg(src + j) : make_uint4(0u, 0u, 0u, 0u);
                if constexpr (!FINE) {  // bf16
                    uint32_t top = 0u;
#pragma unroll
                    for (int j = 0; j < DQ / 2; ++j) top = __vmaxu2(top, x[j / 16][j % 16] & 0x7FFF7FFFu);
                    sh.poison[wg][m] = max(top & 0xFFFFu, top >> 16);
                    softmax_sync();
                    top = max(max(sh.poison[0][m], sh.poison[1][m]), max(sh.poison[2][m], sh.poison[3][m]));
                    const int ex = head_sum_exponent(__uint_as_float(top << 16));
                    const float f = flip ? -exp2i(ex) : exp2i(ex);
                    sl2 *= exp2i(-ex);
#pragma unroll
                    for (int j = 0; j < DQ / 2; ++j) {
                        const uint32_t v = x[j / 16][j % 16];
                        x[j / 16][j % 16] = h2u(__floats2half2_rn(__uint_as_float(v << 16) * f, __uint_as_float(v & 0xFFFF0000u) * f));
                    }
                } else if (flip) {
#pragma unroll
                    for (int j = 0; j < DQ / 2; ++j) x[j / 16][j % 16] ^= 0x80008000u;
                }
                __syncwarp();
#pragma unroll
                for (int c = 0; c < DQ / 32; ++c) tmem_st16(lane_base + G::Q_COL + wg * (DQ / 2) + 16 * c, x[c]);
                tmem_wait_st();
                fence_before();
                mbar_arrive(smem_u32(&sh.q_full));
            }
            float l = 0.0f, lref = -CUDART_INF_F;  // the sum, in units of 2^lref
            uint32_t poison = 0u;  // quarters of the dims whose value is NaN: an infinite or NaN V scale was attended to
            for (int i = (k & 1) == set ? 0 : 1; i < n; i += 2) {
                const int kk = k + i, c0 = (i0 + i) * N + half * H;
                const uint32_t s_col = lane_base + set * N + half * H;
                wait(sh.info_full[kk % INFOS], kk / INFOS);
                const Info<N> &f = sh.info[kk % INFOS];
                constexpr int MY = H / 32;  // parts of the half
                int flags = 0;
#pragma unroll
                for (int x = 0; x < MY; ++x) flags |= f.flags[half * MY + x];
                // What the row sees of 32 cells, where some row ends in this tile, or
                // sees by its bits, or cells are not there.
                // Of listed pages, 16 cells are mostly seen or not as one; the score's offset
                // says that below.
                bool edge;
                uint32_t sees[MY];
                if constexpr (LISTED<A>) {
                    bool partly = flags & WILD;
#pragma unroll
                    for (int x = 0; x < 2 * MY; ++x) {
                        const uint2 u = f.unit[half * 2 * MY + x];
                        const int k = (u.y >> (token - t) & 1u) ? min(max(sure - (int)u.x, 0), 16) : 0;
                        const uint32_t bits = ((1u << k) - 1) & f.there[half * MY + x / 2] >> (16 * (x & 1));
                        partly |= bits && bits != 0xFFFFu;
                        sees[x / 2] = x & 1 ? sees[x / 2] | bits << 16 : bits;
                    }
                    edge = __any_sync(0xffffffffu, partly);
                } else {
                    edge = c0 > grp.least - H || (flags & GAPS);
                }
                auto seen = [&](int c) -> uint32_t {
                    if constexpr (LISTED<A>) return c ? sees[MY - 1] : sees[0];
                    const int from = c0 + 32 * c;
                    if (from >= len) return 0u;
                    uint32_t bits = 0xffffffffu;
                    if constexpr (TREE<A>) bits = tree_bits(a, token, from, sure);
                    if (len - from < 32) bits &= (1u << (len - from)) - 1;
                    const uint32_t there = f.there[half * MY + c];
                    bad |= good && (bits & ~there);  // a page that no row attends to may be missing
                    return bits & there;
                };
                wait(sh.s_full[set], kk >> 1);
                fence_after();
                // There, -inf takes the place of the scores that it does not see, and
                // of a marked tile's the scores with their cells' powers of two.
                if (edge || (flags & MARKED)) {
#pragma unroll 1
                    for (int c = 0; c < H / 16; ++c) {
                        const uint32_t bits = edge || LISTED<A> ? seen(c >> 1) >> (16 * (c & 1)) : 0xffffffffu;
                        uint32_t v[16];
                        __syncwarp();
                        tmem_ld16(s_col + 16 * c, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            asm volatile("" : "+r"(v[j]));  // not before the wait
                            if (flags & MARKED) v[j] = __float_as_uint(fmaf(__uint_as_float(v[j]) * f.kf[half * H + 16 * c + j], sl2, f.vb[half * H + 16 * c + j]));
                            if (!(bits >> j & 1u)) v[j] = 0xFF800000u;
                        }
                        tmem_st16(s_col + 16 * c, v);
                    }
                    tmem_wait_st();
                }
                // In base 2: p = 2^(c S + d - reference), c and d of 32 cells.  With scale 0
                // the weights are uniform, and a masked -inf stays -inf.
                auto factor = [&](int c) { return flags & MARKED ? 1.0f : fmaxf(sl2 * f.ck[half * MY + c], 1.17549435e-38f); };
                auto offset = [&](int c) { return flags & MARKED ? 0.0f : f.cb[half * MY + c]; };
                float top = -CUDART_INF_F;
#pragma unroll 1
                for (int c = 0; c < MY; ++c) {
                    uint32_t v[2][16];
                    tmem_read32(s_col + 32 * c, v);
                    float x[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {  // of 16 cells x[0] and x[1], of the others x[2] and x[3]
                        float &y = x[j / 16 * 2 + j / 2 % 2];
                        y = max3(y, __uint_as_float(v[j / 16][j % 16]), __uint_as_float(v[j / 16][j % 16 + 1]));
                    }
                    if constexpr (LISTED<A>) {
                        const float lo = seen(c) & 0xFFFFu ? fmaf(fmaxf(x[0], x[1]), factor(c), offset(c)) : -CUDART_INF_F;
                        const float hi = seen(c) >> 16 ? fmaf(fmaxf(x[2], x[3]), factor(c), offset(c)) : -CUDART_INF_F;
                        top = max3(top, lo, hi);
                    } else {
                        top = fmaxf(top, fmaf(max3(x[0], x[1], fmaxf(x[2], x[3])), factor(c), offset(c)));
                    }
                }
                sh.top[set][half][m] = top;
                __syncwarp();
                good = both(good);
                if (!good) break;  // and no break from here to there
                top = ceilf(fmaxf(top, sh.top[set][half ^ 1][m]));
                if (flags & POISONED) {
                    for (int c = 0; c < H; ++c)
                        if ((f.flags[half * MY + (c >> 5)] & POISONED) && f.poison[half * H + c] && (seen(c >> 5) >> (c & 31) & 1u))
                            poison |= f.poison[half * H + c];
                    __syncwarp();
                }
                if constexpr (LISTED<A>) poison |= seen(0) | seen(1) ? SAW : 0u;
                // The reference moves only when a tile exceeds it by 2^SLACK.
                float ref = -CUDART_INF_F;
                if (i > 0) {
                    wait(sh.ref_full[set ^ 1], (kk - 1) >> 1);
                    ref = sh.ref[set ^ 1][m];
                }
                const bool up = top > ref + SLACK;
                const float alpha = up ? ex2(ref - top) : 1.0f;
                ref = up ? top : ref;
                // Both halves say so: the other set writes over the one before only then.
                if (half == 0) sh.ref[set][m] = ref;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh.ref_full[set]));
                if (i > 0 && __any_sync(0xffffffffu, up)) {
                    // The values so far, half of them by each.
                    wait(sh.pv_full[set ^ 1], (kk - 1) >> 1);
                    fence_after();
#pragma unroll 1
                    for (int c = 0; c < D / 32 && good; ++c) {
                        uint32_t v[16];
                        tmem_ld16(lane_base + G::O_COL + half * (D / 2) + 16 * c, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            asm volatile("" : "+r"(v[j]));
                            v[j] = __float_as_uint(__uint_as_float(v[j]) * alpha);
                        }
                        tmem_st16(lane_base + G::O_COL + half * (D / 2) + 16 * c, v);
                    }
                    tmem_wait_st();
                }
                const float base = ref == -CUDART_INF_F ? 0.0f : (float)LIFT - ref;
                float total = 0.0f;
                if (flags & MARKED) {
#pragma unroll 1
                    for (int c = 0; c < H / 16; ++c) {
                        uint32_t v[16];
                        tmem_ld16(s_col + 16 * c, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            asm volatile("" : "+r"(v[j]));
                            total = fmaf(ex2(__uint_as_float(v[j]) + base), f.vw[half * H + 16 * c + j], total);
                        }
                    }
                }
#pragma unroll 1
                for (int c = 0; c < MY; ++c) {
                    const float cs = factor(c), d = offset(c) + base;
                    const float2 c2 = make_float2(cs, cs), less = make_float2(-1.0f, -1.0f);
                    float2 sum = make_float2(0.0f, 0.0f);
                    uint32_t v[2][16];
                    tmem_read32(s_col + 32 * c, v);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t w[16];
                        const float de = !LISTED<A> || (seen(c) >> (16 * e) & 0xFFFFu) ? d : -CUDART_INF_F;
                        const float2 d2 = make_float2(de, de);
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            float2 p = __ffma2_rn(make_float2(__uint_as_float(v[e][j]), __uint_as_float(v[e][j + 1])), c2, d2);
                            p = make_float2(ex2(p.x), ex2(p.y));
                            sum = __fadd2_rn(p, sum);
                            if constexpr (FINE) {
                                // The high part by cutting, so that the rest is exact.
                                const float2 h = make_float2(__uint_as_float(__float_as_uint(p.x) & 0xFFFFE000u),
                                                             __uint_as_float(__float_as_uint(p.y) & 0xFFFFE000u));
                                const float2 r = __ffma2_rn(h, less, p);
                                w[j / 2] = h2u(__floats2half2_rn(h.x, h.y));
                                w[8 + j / 2] = h2u(__floats2half2_rn(r.x, r.y));
                            } else {
                                w[j / 2] = h2u(__floats2half2_rn(p.x, p.y));
                            }
                        }
                        // In the place of their scores.
                        if constexpr (FINE)
                            tmem_st16(s_col + 32 * c + 16 * e, w);
                        else
                            tmem_st8(s_col + 32 * c + 16 * e, w);
                    }
                    if (!(flags & MARKED)) total = fmaf(sum.x + sum.y, f.cw[half * MY + c], total);
                }
                l = l * (lref == ref ? 1.0f : ex2(lref - ref)) + total;
                lref = ref;
                tmem_wait_st();
                fence_before();
                if (good) mbar_arrive(smem_u32(&sh.p_full[set]));
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh.info_empty[kk % INFOS]));
            }
            if (good) wait(sh.pv_full[(k + n - 1) & 1], (k + n - 1) >> 1);
            if (good) {
                sh.l[wg][m] = l;
                sh.lref[wg][m] = lref;
                sh.poison[wg][m] = poison;
            }
            softmax_sync();
            if (good) {
                fence_after();
                float ref = -CUDART_INF_F;
                l = 0.0f;
                poison = 0u;
#pragma unroll 1
                for (int w = 0; w < 4; ++w) ref = fmaxf(ref, sh.lref[w][m]);
#pragma unroll 1
                for (int w = 0; w < 4; ++w) {
                    l += sh.l[w][m] * (sh.lref[w][m] == ref ? 1.0f : ex2(sh.lref[w][m] - ref));
                    poison |= sh.poison[w][m];
                }
                float scale = whole ? (ref == -CUDART_INF_F ? 0.0f : 1.0f / l) : 1.0f;
                const bool saw = !LISTED<A> || (poison & SAW);  // or nothing, whatever its query is
                if (!saw) {
                    l = 0.0f;
                    ref = -CUDART_INF_F;
                }
                if (poison >> wg & 1u) scale = CUDART_NAN_F;  // a quarter of the dims has a V scale of its own
                const size_t row = head_row(mine ? m : 0), d0 = row * D + wg * DQ;
                float *part_o = work.o + at * M * D + (size_t)(wg * DQ) * M + m;  // [D][M]: a warp's lanes next to one another
                const bool in = mine && QSA_IN(d0 + DQ - 1, (size_t)a.n_tokens * a.n_q_heads * D);
#pragma unroll 1
                for (int c = 0; c < DQ; c += 16) {
                    uint32_t v[16];
                    __syncwarp();
                    tmem_ld16(lane_base + G::O_COL + wg * DQ + c, v);
                    tmem_wait_ld();
                    if (!whole) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            asm volatile("" : "+r"(v[j]));
                            part_o[(size_t)(c + j) * M] = saw ? __uint_as_float(v[j]) * scale : 0.0f;
                        }
                    } else if (in) {
                        uint32_t w[8];
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            asm volatile("" : "+r"(v[j]), "+r"(v[j + 1]));
                            if (!saw) v[j] = v[j + 1] = 0u;
                            w[j / 2] = tile_value<FINE>(a, d0 + c + j, make_float2(__uint_as_float(v[j]) * scale, __uint_as_float(v[j + 1]) * scale));
                        }
                        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + d0 + c);
                        dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
                        dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
                    }
                }
                if (mine && wg == 0) {
                    if (!whole)
                        *reinterpret_cast<float2 *>(work.ml + (at * M + m) * 2) = make_float2(ref - LIFT, l);
                    else if (a.lse)
                        a.lse[row] = lse_of(ref - LIFT, l);
                }
                fence_before();  // O is overwritten by the next segment
            }
        }
        k += n;
        if (!__syncthreads_and(good)) {
            ok = false;
            break;
        }
        if (!whole && i0 == 0) part = Part{t, 1 + (tiles - i1 + share - 1) / share, rows, head};
        left -= n;
        if (left <= 0) break;
        i0 = 0;
        t += (head + rows) / per;
        grp = sh.next;
        __syncthreads();  // the next is written over
    }

    // After a time-out: copies on their way land before the block ends, and
    // products issued are complete before tensor memory is freed.
    if (warp == LOADER && !ok) {
        for (int kind = 0; kind < 2; ++kind)
            for (int j = max(sent[kind] - STAGES, 0); j < sent[kind]; ++j)
                mbar_wait_bounded(smem_u32(&sh.full[kind][j % STAGES]), (j / STAGES) & 1, DRAIN_LIMIT);
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
        if (gridDim.x <= MAX_GROUP_PARTS) work.part[blockIdx.x] = ok ? part : Part{-1, 0, 0, 0};
    }
    if (warp == PRODUCTS) {
        fence_after();
        tmem_dealloc(sh.tmem, G::TMEM_COLS);
    }
}

// Joins the partials of a group that spans CTAs: part p of the one that starts in
// CTA x is slot 1 of that CTA, then slot 0 of the next ones of its KV head, values as
// [D][M].  A block takes COLS dims of all head rows, a thread each
// (four of 256: 128 head rows' partials by 64 blocks; by 32, a row of 30 K cells took 5
// us more).
// SETS: sets of threads that share the parts of a group, where these are many; else a
// block takes as many slices of the dims.
template <int S>
constexpr int COLS = 8 / S;
constexpr int SLICES = JOIN_THREADS / M;
template <int S, bool FINE, int SETS>
__device__ __forceinline__ void tiles_join(const qsa_paged_attn_args &a, void *ws, int x, int block) {
    constexpr int D = 128 * S, COLS = qsa::COLS<S>;
    __shared__ float2 so[SETS > 1 ? SETS : 1][COLS / 2][SETS > 1 ? M : 1];
    __shared__ float sl[SETS > 1 ? SETS : 1][SETS > 1 ? M : 1];
    const Work work(ws, MAX_GROUP_PARTS, M);
    const int m = threadIdx.x % M, k = threadIdx.x / M, set = SETS > 1 ? k : 0, d0 = (SETS > 1 ? block : block * SLICES + k) * COLS;
    const int per = a.n_q_heads / a.n_kv_heads;
    const Part part = work.part[x];
    if (part.row < 0) return;
    const int n = m < part.tokens ? part.n : 0;
    auto slot = [&](int p) { return ((size_t)(x + p * a.n_kv_heads) * 2 + (p == 0 ? 1 : 0)) * M; };
    float top = -CUDART_INF_F, l = 0.0f;
    float2 o[COLS / 2];
#pragma unroll
    for (int j = 0; j < COLS / 2; ++j) o[j] = make_float2(0.0f, 0.0f);
#pragma unroll 4
    for (int p = 0; p < n; ++p) top = fmaxf(top, work.ml[(slot(p) + m) * 2]);
#pragma unroll 1
    for (int p = set; p < n; p += SETS) {
        const float2 ml = reinterpret_cast<const float2 *>(work.ml)[slot(p) + m];
        const float w = ml.x == -CUDART_INF_F ? 0.0f : exp2f(ml.x - top), *src = work.o + slot(p) * D + (size_t)d0 * M + m;
        l = fmaf(w, ml.y, l);
#pragma unroll
        for (int j = 0; j < COLS / 2; ++j) o[j] = __ffma2_rn(make_float2(w, w), make_float2(src[2 * j * M], src[(2 * j + 1) * M]), o[j]);
    }
    if constexpr (SETS > 1) {
#pragma unroll
        for (int j = 0; j < COLS / 2; ++j) so[set][j][m] = o[j];
        sl[set][m] = l;
        __syncthreads();
        if (set) return;
#pragma unroll 1
        for (int i = 1; i < SETS; ++i) {
#pragma unroll
            for (int j = 0; j < COLS / 2; ++j) o[j] = __fadd2_rn(o[j], so[i][j][m]);
            l += sl[i][m];
        }
    }
    if (!n) return;
    const float inv = top == -CUDART_INF_F ? 0.0f : 1.0f / l;
    const int i = (part.head + m) / per;
    const size_t row = (size_t)(part.row + i) * a.n_q_heads + (size_t)(x % a.n_kv_heads) * per + (part.head + m - i * per);
    if (d0 == 0 && a.lse) a.lse[row] = lse_of(top, l);
    if (!QSA_IN(row * D + d0 + COLS - 1, (size_t)a.n_tokens * a.n_q_heads * D)) return;
    uint32_t y[COLS / 2];
#pragma unroll
    for (int j = 0; j < COLS / 2; ++j) y[j] = tile_value<FINE>(a, row * D + d0 + 2 * j, make_float2(o[j].x * inv, o[j].y * inv));
    uint16_t *dst = static_cast<uint16_t *>(a.out) + row * D + d0;
    if constexpr (S == 1)
        *reinterpret_cast<uint4 *>(dst) = make_uint4(y[0], y[1], y[2], y[3]);
    else
        *reinterpret_cast<uint2 *>(dst) = make_uint2(y[0], y[1]);
}
// The groups' partials, then those of rows one by one (none: no CTAs).  Blocks list the
// CTAs in which a group or a row that spans CTAs starts, and go round over these.
template <int S, bool FINE>
__global__ void __launch_bounds__(JOIN_THREADS) paged_tiles_join_kernel(const qsa_paged_attn_args a, void *ws, int ctas, const Joined rows) {
    __shared__ int at[JOIN_THREADS], found[32];
    static_assert(MAX_CTAS <= JOIN_THREADS / 2 && MAX_GROUP_PARTS <= JOIN_THREADS / 2, "a thread per CTA");
    wait_for_previous_grid();
    allow_dependent_launch();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, x = tid % (JOIN_THREADS / 2);
    const bool group = tid < JOIN_THREADS / 2;
    const bool starts = group ? x < ctas && Work(ws, MAX_GROUP_PARTS, M).part[x].row >= 0
                              : x < rows.ctas && Work(rows.ws, rows.cap, rows.rows).part[x].row >= 0;
    const unsigned m = __ballot_sync(0xffffffffu, starts);
    if (lane == 0) found[warp] = __popc(m);
    __syncthreads();
    const int mine = found[lane];
    const int groups = __reduce_add_sync(0xffffffffu, lane < 16 ? mine : 0), others = __reduce_add_sync(0xffffffffu, lane < 16 ? 0 : mine);
    const int before = __reduce_add_sync(0xffffffffu, lane < warp ? mine : 0);
    if (starts) at[before + __popc(m & ((1u << lane) - 1))] = x;
    __syncthreads();
    // Few of a kind have many parts each, which sets of threads share: where blocks need
    // not go round for it.
    const bool few_groups = groups * (128 * S / COLS<S>) <= gridDim.x;
    const bool few_rows = others * ((rows.rows + JOIN_HEADS<S, 4> - 1) / JOIN_HEADS<S, 4>) <= gridDim.x;
    const int slices = 128 * S / COLS<S> / (few_groups ? 1 : SLICES), heads = few_rows ? JOIN_HEADS<S, 4> : JOIN_HEADS<S, 1>;
    const int chunks = (rows.rows + heads - 1) / heads;
    for (int it = blockIdx.x; it < groups * slices + others * chunks; it += gridDim.x) {
        const int k = it - groups * slices;
        if (k < 0) {
            if (few_groups)
                tiles_join<S, FINE, SLICES>(a, ws, at[it / slices], it % slices);
            else
                tiles_join<S, FINE, 1>(a, ws, at[it / slices], it % slices);
        } else {
            if (few_rows)
                rows_join<S, 4>(a, rows, at[groups + k / chunks], k % chunks * heads);
            else
                rows_join<S, 1>(a, rows, at[groups + k / chunks], k % chunks * heads);
        }
        __syncthreads();  // what they share is written over
    }
}
// The same where most CTAs of 128 dims have a part that starts there: a block for each
// (1984 listed tokens 139 us in all, 143 by the list; of 256 dims, fewer blocks are more).
template <int S, bool FINE>
__global__ void __launch_bounds__(JOIN_THREADS) paged_tiles_join_all_kernel(const qsa_paged_attn_args a, void *ws, int ctas, const Joined rows) {
    constexpr int BLOCKS = 128 * S / (COLS<S> * SLICES);
    wait_for_previous_grid();
    allow_dependent_launch();
    const int x = blockIdx.x, y = x - ctas * BLOCKS;
    if (y < 0)
        tiles_join<S, FINE, 1>(a, ws, x / BLOCKS, x % BLOCKS);
    else
        rows_join<S, 1>(a, rows, y % rows.ctas, y / rows.ctas * JOIN_HEADS<S, 1>);
}
inline int tiles_ctas(int n_kv_heads) { return std::max(MAX_GROUP_PARTS / n_kv_heads, 1) * n_kv_heads; }

// Codes [cells, heads, D] in boxes of a tile's cells (or a page's, if fewer) x one
// head x 128 dims.
template <int S>
cudaError_t encode_tiles(CUtensorMap &map, const qsa_paged_attn_args &a, const int8_t *codes) {
    return encode_boxes(map, a, codes, std::min(a.page_size, TileShape<S>::N));
}

// ws: where the partials go, Work of M rows.
template <int S, class A>
cudaError_t launch_tiles(const A &a, void *ws, cudaStream_t s) {
    CUtensorMap kmap, vmap;
    cudaError_t e = encode_tiles<S>(kmap, a, a.kq);
    if (e == cudaSuccess) e = encode_tiles<S>(vmap, a, a.vq);
    if (e != cudaSuccess) return e;
    const int ctas = tiles_ctas(a.n_kv_heads);
    const auto kernel = a.dtype == QSA_F16 ? paged_tiles_kernel<S, true, A> : paged_tiles_kernel<S, false, A>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(TileSmem<S>));
    return e == cudaSuccess ? launch_dependent(kernel, dim3(ctas), dim3(THREADS), sizeof(TileSmem<S>), s, a, kmap, vmap, ws) : e;
}
// Joins what both kinds of kernels left, one of which has had the rows.
template <int S, class A>
cudaError_t launch_tiles_join(const A &a, void *ws, cudaStream_t s) {
    // The rows' kernel has all the CTAs that fit: there is more than enough for them.
    const Joined rows{a.workspace, MAX_CTAS, a.n_q_heads / a.n_kv_heads, MAX_CTAS / a.n_kv_heads * a.n_kv_heads};
    const int ctas = tiles_ctas(a.n_kv_heads);
    const bool fine = a.dtype == QSA_F16, all = S == 1 && ((long long)a.n_tokens * rows.rows / M + 1) * a.n_kv_heads > MAX_GROUP_PARTS / 2;
    const auto kernel = all ? (fine ? paged_tiles_join_all_kernel<S, true> : paged_tiles_join_all_kernel<S, false>)
                            : (fine ? paged_tiles_join_kernel<S, true> : paged_tiles_join_kernel<S, false>);
    const int grid = all ? ctas * (128 * S / (COLS<S> * SLICES)) + rows.ctas * ((rows.rows + JOIN_HEADS<S, 1> - 1) / JOIN_HEADS<S, 1>) : MAX_CTAS;
    return launch_dependent(kernel, dim3(grid), dim3(JOIN_THREADS), 0, s, static_cast<const qsa_paged_attn_args &>(a), ws, ctas, rows);
}

}  // namespace
}  // namespace qsa
