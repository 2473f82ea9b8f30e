// qsa_page_update and qsa_page_compact: the paged cache's bookkeeping and the
// page copies that it calls for.
//
// Each call is two launches.  The first works out the new table: it counts how
// often each page is held, ranks the free (or moved) pages by prefix sums,
// deals them out and leaves a list of copies in the workspace.  It is bound by
// the latency of its phases, a few dependent loads each, so it is one block
// with the counts in shared memory while pool and table are small (SMALL_*),
// and one cluster of eight blocks with the counts in the refs output above
// that; the phases are separated by the block's or the cluster's hardware
// barrier, where a grid-wide form would need one launch per phase.  The second
// launch runs over the whole chip and copies the listed pages; sources and
// targets are disjoint, so no order among them matters.
//
// A compaction that moves 1.04 GB takes 164 us (6.3 TB/s), a fork of 64 rows into
// 256 with its page copies of 16 layers, 227 MB, 36 us, a decode step 8 us.
//
// All results are whole numbers and do not depend on the order of the atomic
// counts.
#include <cuda_runtime.h>

#include "check.cuh"
#include "qsa_internal.h"

namespace qsa {
namespace {

constexpr int CLUSTER = 8;
constexpr int THREADS = 1024;
constexpr int SEG = 128;  // table columns a warp takes at a time

// One block up to this many pages (32 KB of counts) and table entries.  One block
// and a cluster, us, of an update by a token a row and of a compaction:
//   table 64 x 27, pool of 1700 pages: 8.0, 11.5; 9.4, 13.0
//   table 64 x 64, pool of 4096:       8.8, 12.3; 11.5, 15.5
//   table 256 x 64, pool of 16384:     14.2, 14.3; 32.2, 24.7
//   table 1024 x 64, pool of 32768:    33.2, 19.8; 68.1, 29.7
constexpr int SMALL_PAGES = 8192;
constexpr long long SMALL_ENTRIES = 16384;

// One page copy: the first `cells` cells of page src go to page dst.
struct Copy {
    int src, dst, cells;
};

// Workspace: counters, per-row records, the free (or hole) list, the moved
// list, the copies.
struct RowPlan {
    long long off, upto;  // packed place of the row's first new token; pages asked for up to and with this row
    int keep, need;       // length before growing; pages asked for (-1: does not fit)
};
struct Header {
    int n_copies, n_live;
    long long asked, tokens;       // pages asked for; tokens of the packed batch
    int count[CLUSTER * THREADS / 32];  // a warp's count of its slice of the pool
};
constexpr size_t HEADER_BYTES = 2048;
static_assert(sizeof(Header) <= HEADER_BYTES, "workspace header");

struct Ws {
    Header *h;
    RowPlan *rows;
    int *list, *moved;
    Copy *copies;
};
__host__ __device__ inline size_t align16(size_t n) { return (n + 15) & ~(size_t)15; }
__host__ __device__ inline Ws carve(void *p, int n_rows, int n_pages) {
    uint8_t *b = static_cast<uint8_t *>(p);
    Ws w;
    w.h = reinterpret_cast<Header *>(b);
    b += HEADER_BYTES;
    w.rows = reinterpret_cast<RowPlan *>(b);
    b += align16((size_t)n_rows * sizeof(RowPlan));
    w.list = reinterpret_cast<int *>(b);
    b += align16((size_t)n_pages * sizeof(int));
    w.moved = reinterpret_cast<int *>(b);
    b += align16((size_t)n_pages * sizeof(int));
    w.copies = reinterpret_cast<Copy *>(b);
    return w;
}
size_t ws_bytes(int n_rows, int n_pages) {
    // A row copies at most one page (update); a move has a page of its own (compact).
    const size_t copies = (size_t)(n_rows > n_pages ? n_rows : n_pages);
    return HEADER_BYTES + align16((size_t)n_rows * sizeof(RowPlan)) + 2 * align16((size_t)n_pages * sizeof(int)) +
           align16(copies * sizeof(Copy));
}

// The blocks that work on one table: CTAS of them, with counts in shared
// memory (one) or in the refs output (a cluster).
template <int CTAS>
struct Team {
    static constexpr int ALL = CTAS * THREADS, WARPS = ALL / 32;

    static __device__ __forceinline__ int rank() {
        if constexpr (CTAS == 1) return 0;
        unsigned r;
        asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
        return (int)r;
    }
    static __device__ __forceinline__ void sync() {
        if constexpr (CTAS == 1)
            __syncthreads();
        else
            asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    // A value that another block may have written in an earlier phase.
    template <class T>
    static __device__ __forceinline__ T peek(const T *p) {
        if constexpr (CTAS == 1)
            return *p;
        else
            return __ldcg(p);
    }
    // Slice of the pool that warp w counts and ranks: whole groups of 32 pages.
    static __device__ __forceinline__ void slice(int w, int n_pages, int &p0, int &p1) {
        const int per = ((n_pages + 31) / 32 + WARPS - 1) / WARPS * 32;
        p0 = (int)min((long long)w * per, (long long)n_pages);
        p1 = min(p0 + per, n_pages);
    }
    // Sum of the warps' counts, and of those before warp w.
    static __device__ __forceinline__ void totals(const int *count, int w, int &before, int &total) {
        const int lane = threadIdx.x & 31;
        before = total = 0;
#pragma unroll
        for (int i = 0; i < WARPS / 32; ++i) {
            const int v = peek(count + i * 32 + lane);
            total += v;
            before += i * 32 + lane < w ? v : 0;
        }
        before = __reduce_add_sync(0xffffffffu, before);
        total = __reduce_add_sync(0xffffffffu, total);
    }
};

// Exclusive prefix of v over the block (in thread order); total to all.
__device__ __forceinline__ long long block_scan(long long v, long long &total, long long *tmp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
    }
    __syncthreads();  // tmp may still be read from the scan before
    if (lane == 31) tmp[warp] = s;
    __syncthreads();
    long long w = tmp[lane];  // every warp adds up the warps before it
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += u;
    }
    total = __shfl_sync(0xffffffffu, w, 31);
    const long long before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    return s - v + (warp ? before : 0);
}

__device__ __forceinline__ void flag(unsigned int *err, unsigned bit) {
    if (err) atomicOr(err, bit);
}

struct TableArgs {
    int n_rows_in, n_rows, max_pages, n_pages, page_size;
    const int32_t *table, *lens, *src;
    int32_t *table_out, *refs;
    unsigned int *err;
};

// The length that row r starts from (its source row's, cut to what a table
// row can hold) and the source row (-1: none).
__device__ __forceinline__ int row_keep(const TableArgs &a, int r, int &from) {
    from = a.src ? a.src[r] : r;
    if (from < 0 || from >= a.n_rows_in) {
        if (from != -1) flag(a.err, QSA_DEVERR_BAD_ID);
        from = -1;
        return 0;
    }
    const int len = a.lens[from];
    const long long most = (long long)a.max_pages * a.page_size;
    if (len >= 0 && len <= most) return len;
    flag(a.err, QSA_DEVERR_BAD_ID);
    return len < 0 ? 0 : (int)most;
}

__device__ __forceinline__ int pages_of(long long cells, int page_size) {
    return (int)((cells + page_size - 1) / page_size);
}

// Copies the kept entries to the new table (-1 behind them and for an entry
// outside the pool) and counts them in refs, which is zero before.  A warp
// takes SEG columns of a row at a time, and BATCH of these items at once, so
// that the chains of loads (source row, length, entries) of several rows are in
// flight together.  With WRITE the rows' lengths go to their plans.
template <int CTAS, bool WRITE>
__device__ __forceinline__ void gather_and_count(const TableArgs &a, int *refs, RowPlan *rows, int warp) {
    constexpr int BATCH = 4, E = SEG / 32, W = Team<CTAS>::WARPS;
    const int lane = threadIdx.x & 31;
    const int segs = (a.max_pages + SEG - 1) / SEG;
    const long long items = (long long)a.n_rows * segs;
    for (long long it0 = warp; it0 < items; it0 += W * BATCH) {
        int row = 0, from = -1, had = 0;  // lane b's: item it0 + b W
        if (lane < BATCH && it0 + lane * W < items) {
            row = (int)(segs == 1 ? it0 + lane * W : (it0 + lane * W) / segs);
            const int keep = row_keep(a, row, from);
            had = pages_of(keep, a.page_size);
            if (WRITE) rows[row].keep = keep;  // the same from each of a row's items
        }
        int e[BATCH][E];
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const int f = __shfl_sync(0xffffffffu, from, b), n = __shfl_sync(0xffffffffu, had, b);
            const int j0 = segs == 1 ? lane : (int)((it0 + b * W) % segs) * SEG + lane;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int j = j0 + i * 32;
                e[b][i] = j < n && QSA_IN((size_t)f * a.max_pages + j, (size_t)a.n_rows_in * a.max_pages)
                              ? a.table[(size_t)f * a.max_pages + j]
                              : -1;
                if (j < n && (e[b][i] < 0 || e[b][i] >= a.n_pages)) {
                    flag(a.err, QSA_DEVERR_BAD_ID);
                    e[b][i] = -1;
                }
            }
        }
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            if (it0 + b * W >= items) break;
            const int r = __shfl_sync(0xffffffffu, row, b);
            const int j0 = segs == 1 ? lane : (int)((it0 + b * W) % segs) * SEG + lane;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int j = j0 + i * 32;
                if (e[b][i] >= 0) atomicAdd(refs + e[b][i], 1);
                if (WRITE && j < a.max_pages && QSA_IN((size_t)r * a.max_pages + j, (size_t)a.n_rows * a.max_pages))
                    a.table_out[(size_t)r * a.max_pages + j] = e[b][i];
            }
        }
    }
}

struct UpdateLaunch {
    TableArgs t;
    const int32_t *n_new;
    int32_t *lens_out, *slots, *positions;
    int n_slots;
    void *ws;
};

template <int CTAS>
__global__ void __launch_bounds__(THREADS) page_update_kernel(const UpdateLaunch a) {
    using T = Team<CTAS>;
    extern __shared__ int counts[];
    __shared__ long long tmp[32];
    __shared__ Header local;
    const TableArgs &t = a.t;
    const int rank = T::rank(), tid = threadIdx.x, gtid = rank * THREADS + tid, lane = tid & 31, warp = gtid >> 5;
    const Ws ws = carve(a.ws, t.n_rows, t.n_pages);
    int *refs = CTAS == 1 ? counts : t.refs;
    Header *h = CTAS == 1 ? &local : ws.h;
    for (int p = gtid; CTAS == 1 && p < t.n_pages; p += T::ALL) refs[p] = 0;
    wait_for_previous_grid();
    allow_dependent_launch();
    for (int p = gtid; CTAS > 1 && p < t.n_pages; p += T::ALL) refs[p] = 0;
    if (gtid == 0) ws.h->n_copies = 0;
    T::sync();
    gather_and_count<CTAS, true>(t, refs, ws.rows, warp);
    T::sync();

    // Each warp counts the free pages of its slice, and block 0 plans the rows
    // in order.
    int p0, p1;
    T::slice(warp, t.n_pages, p0, p1);
    int n_mine = 0;
    for (int p = p0 + lane; p - lane < p1; p += 32)
        n_mine += __popc(__ballot_sync(0xffffffffu, p < p1 && T::peek(refs + p) == 0));
    if (lane == 0) h->count[warp] = n_mine;
    if (rank == 0) {
        long long off0 = 0, need0 = 0;
        for (int base = 0; base < t.n_rows; base += THREADS) {
            const int r = base + tid;
            int n = 0, keep = 0, need = 0, held = -1;
            if (r < t.n_rows) {
                keep = T::peek(&ws.rows[r].keep);
                n = a.n_new[r];
                if (n < 0) {
                    flag(t.err, QSA_DEVERR_BAD_ID);
                    n = 0;
                }
                if (n > 0 && keep % t.page_size) held = T::peek(t.table_out + (size_t)r * t.max_pages + keep / t.page_size);
            }
            long long total;
            const long long off = off0 + block_scan(n, total, tmp);
            off0 += total;
            if (n > 0) {
                const long long want = ((long long)keep + n + t.page_size - 1) / t.page_size;
                if (want > t.max_pages || off + n > a.n_slots)
                    need = -1;
                else
                    need = (int)want - pages_of(keep, t.page_size) + (held >= 0 && T::peek(refs + held) > 1);
            }
            const long long upto = need0 + block_scan(max(need, 0), total, tmp) + max(need, 0);
            need0 += total;
            if (r < t.n_rows) {
                ws.rows[r].off = off;
                ws.rows[r].upto = upto;
                ws.rows[r].need = need;
            }
        }
        if (tid == 0) {
            h->tokens = off0;
            h->asked = need0;
        }
    }
    T::sync();

    // The free pages by rank, as far as they are asked for.
    const long long asked = T::peek(&h->asked);
    int before, n_free;
    T::totals(h->count, warp, before, n_free);
    for (int p = p0 + lane; p - lane < p1 && before < asked; p += 32) {
        const bool is_free = p < p1 && T::peek(refs + p) == 0;
        const unsigned m = __ballot_sync(0xffffffffu, is_free);
        const int at = before + __popc(m & ((1u << lane) - 1));
        if (is_free && at < asked) ws.list[at] = p;
        before += __popc(m);
    }
    T::sync();

    // Deal the pages out: a lane per row works out what the row gets, and
    // writes it where that is a few tokens; the warp writes the long ones.
    for (int base = warp * 32; base < t.n_rows; base += T::WARPS * 32) {
        const int r = base + lane;
        int n = 0, keep = 0, had = 0, want = 0, copied = 0, last = -1;
        long long off = 0, first = 0;
        bool ok = false;
        if (r < t.n_rows) {
            n = max(a.n_new[r], 0);
            keep = T::peek(&ws.rows[r].keep);
            const int need = T::peek(&ws.rows[r].need);
            off = T::peek(&ws.rows[r].off);
            const long long upto = T::peek(&ws.rows[r].upto);
            ok = n > 0 && need >= 0 && (need == 0 || upto <= n_free);
            had = pages_of(keep, t.page_size);
            if (n > 0 && !ok) flag(t.err, QSA_DEVERR_NO_PAGES);
            a.lens_out[r] = keep + (ok ? n : 0);
            if (ok) {
                want = pages_of((long long)keep + n, t.page_size);
                copied = need - (want - had);  // 1: the last page is copied first
                first = upto - need;
                int32_t *const slot = t.table_out + (size_t)r * t.max_pages + had - 1;
                if (keep % t.page_size) last = T::peek(slot);
                if (copied) {
                    const int to = T::peek(ws.list + first);
                    ws.copies[atomicAdd(&ws.h->n_copies, 1)] = Copy{last, to, keep % t.page_size};
                    atomicSub(refs + last, 1);
                    refs[to] = 1;
                    *slot = last = to;
                }
                first += copied;
            }
        }
        // Row rr's pages from index j0 and tokens from i0 on, every `step`-th.
        auto write = [&](int rr, int n, int keep, int had, int want, int last, long long off, long long first, bool ok, int i0,
                         int step) {
            for (int j = had + i0; ok && j < want; j += step) {
                const int p = T::peek(ws.list + first + (j - had));
                t.table_out[(size_t)rr * t.max_pages + j] = p;
                refs[p] = 1;
            }
            for (int i = i0; i < n && off + i < a.n_slots; i += step) {  // token i sits at position keep + i
                const int pos = keep + i, j = pos / t.page_size;
                const int p = !ok ? -1 : j < had ? last : T::peek(ws.list + first + (j - had));
                a.slots[off + i] = p < 0 ? -1 : p * t.page_size + pos % t.page_size;
                a.positions[off + i] = ok ? pos : -1;
            }
        };
        if (n <= 8) write(r, n, keep, had, want, last, off, first, ok, 0, 1);
        for (unsigned m = __ballot_sync(0xffffffffu, n > 8); m; m &= m - 1) {
            const int b = __ffs(m) - 1;
            write(base + b, __shfl_sync(0xffffffffu, n, b), __shfl_sync(0xffffffffu, keep, b), __shfl_sync(0xffffffffu, had, b),
                  __shfl_sync(0xffffffffu, want, b), __shfl_sync(0xffffffffu, last, b), __shfl_sync(0xffffffffu, off, b),
                  __shfl_sync(0xffffffffu, first, b), __shfl_sync(0xffffffffu, (int)ok, b), lane, 32);
        }
    }
    for (long long i = T::peek(&h->tokens) + gtid; i < a.n_slots; i += T::ALL) a.slots[i] = a.positions[i] = -1;
    if constexpr (CTAS == 1) {
        __syncthreads();
        for (int p = tid; p < t.n_pages; p += THREADS) t.refs[p] = refs[p];
    }
}

struct CompactLaunch {
    TableArgs t;
    int32_t *page_map, *n_live;
    void *ws;
};

template <int CTAS>
__global__ void __launch_bounds__(THREADS) page_compact_kernel(const CompactLaunch a) {
    using T = Team<CTAS>;
    extern __shared__ int counts[];
    __shared__ Header local;
    const TableArgs &t = a.t;
    const int rank = T::rank(), tid = threadIdx.x, gtid = rank * THREADS + tid, lane = tid & 31, warp = gtid >> 5;
    const Ws ws = carve(a.ws, t.n_rows, t.n_pages);
    int *refs = CTAS == 1 ? counts : t.refs;
    Header *h = CTAS == 1 ? &local : ws.h;
    for (int p = gtid; CTAS == 1 && p < t.n_pages; p += T::ALL) refs[p] = 0;
    wait_for_previous_grid();
    allow_dependent_launch();
    for (int p = gtid; CTAS > 1 && p < t.n_pages; p += T::ALL) refs[p] = 0;
    T::sync();
    gather_and_count<CTAS, false>(t, refs, nullptr, warp);
    T::sync();

    // L, the number of held pages.
    int p0, p1;
    T::slice(warp, t.n_pages, p0, p1);
    int n_mine = 0;
    for (int p = p0 + lane; p - lane < p1; p += 32)
        n_mine += __popc(__ballot_sync(0xffffffffu, p < p1 && T::peek(refs + p) > 0));
    if (lane == 0) h->count[warp] = n_mine;
    T::sync();
    int before, live;
    T::totals(h->count, warp, before, live);

    // Rank of each free page below L among the free, and of each held page at
    // or above L among the held: with b held pages before p, a hole p < L has
    // rank p - b, and a mover p >= L has L - 1 - b held pages after it, its
    // rank from the end.  So one pass ranks both, and the movers are listed
    // from the last one; there are as many of them as holes, L less the held
    // pages before L.
    for (int p = p0 + lane; p - lane < p1; p += 32) {
        const bool held = p < p1 && T::peek(refs + p) > 0;
        const unsigned m = __ballot_sync(0xffffffffu, held);
        const int b = before + __popc(m & ((1u << lane) - 1));
        if (p < p1) {
            if (p < live && !held) ws.list[p - b] = p;
            if (p >= live && held) ws.moved[live - 1 - b] = p;
            a.page_map[p] = held && p < live ? p : -1;
            if (p == live) h->n_live = p - b;
            if (p + 1 == t.n_pages && live == t.n_pages) h->n_live = 0;
        }
        before += __popc(m);
    }
    T::sync();

    const int moves = T::peek(&h->n_live);
    for (int i = gtid; i < moves; i += T::ALL) {
        const int to = T::peek(ws.list + i), from = T::peek(ws.moved + (moves - 1 - i));
        a.page_map[from] = to;
        ws.copies[i] = Copy{from, to, t.page_size};
        refs[to] = T::peek(refs + from);
        refs[from] = 0;
    }
    if (gtid == 0) {
        ws.h->n_copies = moves;
        *a.n_live = live;
    }
    T::sync();

    const int segs = (t.max_pages + SEG - 1) / SEG;
    const long long items = (long long)t.n_rows * segs;
    for (long long it = warp; it < items; it += T::WARPS) {
        const int r = (int)(segs == 1 ? it : it / segs), j0 = segs == 1 ? 0 : (int)(it % segs) * SEG;
        int from;
        const int had = pages_of(row_keep(t, r, from), t.page_size);
        int e[SEG / 32];
#pragma unroll
        for (int i = 0; i < SEG / 32; ++i) {
            const int j = j0 + i * 32 + lane;
            e[i] = j < min(had, t.max_pages) ? t.table[(size_t)r * t.max_pages + j] : -1;
        }
#pragma unroll
        for (int i = 0; i < SEG / 32; ++i) {
            const int j = j0 + i * 32 + lane;
            if (j < t.max_pages)
                t.table_out[(size_t)r * t.max_pages + j] = e[i] < 0 || e[i] >= t.n_pages ? -1 : T::peek(a.page_map + e[i]);
        }
    }
    if constexpr (CTAS == 1)
        for (int p = tid; p < t.n_pages; p += THREADS) t.refs[p] = refs[p];
}

// The listed copies, all layers, codes and scales: bound by reading and writing
// them.  A block takes a run of cells of one layer's copy, of K or of V, at a
// time: up to PIECE bytes of codes in 16-byte words, four per thread in flight,
// and the same cells' scales in 8-byte words.  Blocks: 32 per SM (8: 174 us, 16: 167
// us, 32: 164 us for 1.04 GB), pieces of 32 KB (of 16: 36.6 us, of 32: 35.7 us for
// half-filled pages).
constexpr int COPY_THREADS = 256;
constexpr int PIECE = COPY_THREADS * 8 * 16;

struct CopyLaunch {
    int n_layers, n_pages, page_size, code_row, scale_row, n_copies_max;  // bytes per cell
    int piece_cells, pieces;                                            // cells of a piece, pieces of a page
    uint8_t *kq, *vq, *ksc, *vsc;
    void *ws;
    int n_rows;
};

__global__ void __launch_bounds__(COPY_THREADS) page_copy_kernel(const CopyLaunch a) {
    wait_for_previous_grid();
    allow_dependent_launch();
    const Ws ws = carve(a.ws, a.n_rows, a.n_pages);
    const int n = min(__ldcg(&ws.h->n_copies), a.n_copies_max), tid = threadIdx.x;
    const size_t code_page = (size_t)a.page_size * a.code_row, scale_page = (size_t)a.page_size * a.scale_row;
    const int per_copy = 2 * a.pieces * a.n_layers;
    const long long items = (long long)n * per_copy;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        const Copy c = ws.copies[it / per_copy];
        const int in = (int)(it % per_copy), layer = in / (2 * a.pieces), part = in % (2 * a.pieces);
        const bool is_v = part >= a.pieces;
        const int c0 = (part - (is_v ? a.pieces : 0)) * a.piece_cells, cells = min(c.cells - c0, a.piece_cells);
        if (cells <= 0 || !QSA_IN(c.src, a.n_pages) || !QSA_IN(c.dst, a.n_pages) || !QSA_IN(c.cells, a.page_size + 1)) continue;
        const size_t from = (size_t)layer * a.n_pages + c.src, to = (size_t)layer * a.n_pages + c.dst;
        uint8_t *codes = (is_v ? a.vq : a.kq) + (size_t)c0 * a.code_row, *scales = (is_v ? a.vsc : a.ksc) + (size_t)c0 * a.scale_row;
        const uint4 *src = reinterpret_cast<const uint4 *>(codes + from * code_page);
        uint4 *dst = reinterpret_cast<uint4 *>(codes + to * code_page);
        const int n16 = cells * (a.code_row / 16), n8 = cells * (a.scale_row / 8);
        const uint2 *ssrc = reinterpret_cast<const uint2 *>(scales + from * scale_page);
        uint2 *sdst = reinterpret_cast<uint2 *>(scales + to * scale_page);
        uint2 s = make_uint2(0u, 0u);
        if (tid < n8) s = ssrc[tid];
        for (int i = tid; i < n16; i += COPY_THREADS * 4) {
            uint4 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (i + k * COPY_THREADS < n16) v[k] = src[i + k * COPY_THREADS];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (i + k * COPY_THREADS < n16) dst[i + k * COPY_THREADS] = v[k];
        }
        if (tid < n8) sdst[tid] = s;
        for (int i = tid + COPY_THREADS; i < n8; i += COPY_THREADS) sdst[i] = ssrc[i];
    }
}

template <class A>
cudaError_t launch_copies(const A &a, int n_copies_max, cudaStream_t s) {
    const int code_row = a.n_kv_heads * a.head_dim;
    int piece_cells = PIECE / code_row;
    piece_cells = piece_cells < 1 ? 1 : piece_cells > a.page_size ? a.page_size : piece_cells;
    const int pieces = (a.page_size + piece_cells - 1) / piece_cells;
    const CopyLaunch c{a.n_layers, a.n_pages, a.page_size, code_row, a.n_kv_heads * 8, n_copies_max, piece_cells, pieces,
                       reinterpret_cast<uint8_t *>(a.kq), reinterpret_cast<uint8_t *>(a.vq),
                       reinterpret_cast<uint8_t *>(a.ksc), reinterpret_cast<uint8_t *>(a.vsc), a.workspace, a.n_rows};
    const long long items = (long long)n_copies_max * 2 * pieces * a.n_layers;
    const int blocks = (int)(items < 152 * 32 ? (items < 1 ? 1 : items) : 152 * 32);
    return launch_dependent(page_copy_kernel, dim3(blocks), dim3(COPY_THREADS), 0, s, c);
}

// The table's launch: one block, or one cluster of eight.
template <class L>
cudaError_t launch_team(void (*one)(L), void (*cluster)(L), const L &l, cudaStream_t s) {
    const bool small = l.t.n_pages <= SMALL_PAGES && (long long)l.t.n_rows * l.t.max_pages <= SMALL_ENTRIES;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(small ? 1 : CLUSTER);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = small ? (size_t)l.t.n_pages * sizeof(int) : 0;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CLUSTER;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = small ? 1 : 2;
    static_assert(SMALL_PAGES * sizeof(int) <= 40 * 1024, "below the default limit, with the kernels' own");
    return cudaLaunchKernelEx(&cfg, small ? one : cluster, l);
}

}  // namespace

size_t pages_workspace_bytes(int n_rows, int n_pages) { return ws_bytes(n_rows, n_pages); }

cudaError_t launch_page_update(const qsa_page_update_args &a, cudaStream_t s) {
    const UpdateLaunch u{{a.n_rows_in, a.n_rows, a.max_pages, a.n_pages, a.page_size, a.page_table, a.seq_lens, a.src,
                          a.page_table_out, a.refs, a.err},
                         a.n_new, a.seq_lens_out, a.slots, a.positions, a.n_slots, a.workspace};
    const cudaError_t e = launch_team(page_update_kernel<1>, page_update_kernel<CLUSTER>, u, s);
    return e != cudaSuccess ? e : launch_copies(a, a.n_rows, s);  // a row copies at most one page
}

cudaError_t launch_page_compact(const qsa_page_compact_args &a, cudaStream_t s) {
    const CompactLaunch c{{a.n_rows, a.n_rows, a.max_pages, a.n_pages, a.page_size, a.page_table, a.seq_lens, nullptr,
                           a.page_table_out, a.refs, a.err},
                          a.page_map, a.n_live, a.workspace};
    const cudaError_t e = launch_team(page_compact_kernel<1>, page_compact_kernel<CLUSTER>, c, s);
    return e != cudaSuccess ? e : launch_copies(a, a.n_pages / 2, s);  // as many movers as holes
}

}  // namespace qsa

QSA_DEFINE_CHECK_READER(take_check_word_pages)
