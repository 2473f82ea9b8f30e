// qsa_page_update and qsa_page_compact: the paged cache's bookkeeping and the
// page copies that it calls for.
//
// Each call is two launches.  The first, one cluster of eight blocks, works
// out the new table: it counts how often each page is held, ranks the free
// (or moved) pages by prefix sums, deals them out and leaves a list of copies
// in the workspace.  Its phases are separated by the cluster's hardware
// barrier, which also orders their global-memory traffic; a grid-wide form
// would need one launch per phase, and the tables are small (a phase is a few
// loads per thread).  The second launch runs over the whole chip and copies
// the listed pages in 16-byte words; sources and targets are disjoint, so no
// order among them matters.
//
// All results are whole numbers and do not depend on the order of the atomic
// counts.
#include <cuda_runtime.h>

#include "check.cuh"
#include "qsa_internal.h"

namespace qsa {
namespace {

constexpr int CTAS = 8;
constexpr int THREADS = 1024;
constexpr int ALL = CTAS * THREADS;
constexpr int SEG = 256;  // table columns a warp takes at a time

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
    int n_copies, pad[3];
    long long n_free_or_live, tokens;
    long long part[CTAS][2];
};
constexpr size_t HEADER_BYTES = 256;
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

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ unsigned cluster_rank() {
    unsigned r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

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
    if (warp == 0) {
        long long w = tmp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += u;
        }
        tmp[lane] = w;
    }
    __syncthreads();
    total = tmp[31];
    return s - v + (warp ? tmp[warp - 1] : 0);
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
// takes SEG columns of a row at a time.
template <bool WRITE>
__device__ __forceinline__ void gather_and_count(const TableArgs &a, int rank) {
    const int lane = threadIdx.x & 31;
    const int segs = (a.max_pages + SEG - 1) / SEG;
    const long long items = (long long)a.n_rows * segs;
    for (long long it = rank * (THREADS / 32) + (threadIdx.x >> 5); it < items; it += ALL / 32) {
        const int r = (int)(it / segs), j0 = (int)(it % segs) * SEG;
        int from;
        const int had = pages_of(row_keep(a, r, from), a.page_size);
        int e[SEG / 32];
#pragma unroll
        for (int i = 0; i < SEG / 32; ++i) {
            const int j = j0 + i * 32 + lane;
            e[i] = -1;
            if (j < had && QSA_IN((size_t)from * a.max_pages + j, (size_t)a.n_rows_in * a.max_pages)) {
                e[i] = a.table[(size_t)from * a.max_pages + j];
                if (e[i] < 0 || e[i] >= a.n_pages) {
                    flag(a.err, QSA_DEVERR_BAD_ID);
                    e[i] = -1;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < SEG / 32; ++i) {
            const int j = j0 + i * 32 + lane;
            if (e[i] >= 0) atomicAdd(a.refs + e[i], 1);
            if (WRITE && j < a.max_pages && QSA_IN((size_t)r * a.max_pages + j, (size_t)a.n_rows * a.max_pages))
                a.table_out[(size_t)r * a.max_pages + j] = e[i];
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

__global__ void __cluster_dims__(CTAS, 1, 1) __launch_bounds__(THREADS) page_update_kernel(const UpdateLaunch a) {
    __shared__ long long tmp[32];
    const TableArgs &t = a.t;
    const int rank = (int)cluster_rank(), tid = threadIdx.x, gtid = rank * THREADS + tid;
    const Ws ws = carve(a.ws, t.n_rows, t.n_pages);
    wait_for_previous_grid();
    allow_dependent_launch();
    for (int p = gtid; p < t.n_pages; p += ALL) t.refs[p] = 0;
    if (gtid == 0) ws.h->n_copies = 0;
    cluster_sync();
    gather_and_count<true>(t, rank);
    cluster_sync();

    // Block 0 plans the rows in order; the others count the free pages of
    // their slices of the pool.
    constexpr int SCAN = CTAS - 1;
    const int per = (t.n_pages + SCAN - 1) / SCAN;
    const int p0 = min((rank - 1) * per, t.n_pages), p1 = min(p0 + per, t.n_pages);
    if (rank == 0) {
        long long off0 = 0, need0 = 0;
        for (int base = 0; base < t.n_rows; base += THREADS) {
            const int r = base + tid;
            int n = 0, keep = 0, need = 0;
            if (r < t.n_rows) {
                int from;
                keep = row_keep(t, r, from);
                n = a.n_new[r];
                if (n < 0) {
                    flag(t.err, QSA_DEVERR_BAD_ID);
                    n = 0;
                }
            }
            long long total;
            const long long off = off0 + block_scan(n, total, tmp);
            off0 += total;
            if (n > 0) {
                const long long want = ((long long)keep + n + t.page_size - 1) / t.page_size;
                if (want > t.max_pages || off + n > a.n_slots) {
                    need = -1;
                } else {
                    need = (int)want - pages_of(keep, t.page_size);
                    if (keep % t.page_size) {
                        const int held = __ldcg(t.table_out + (size_t)r * t.max_pages + keep / t.page_size);
                        need += held >= 0 && __ldcg(t.refs + held) > 1;
                    }
                }
            }
            const long long upto = need0 + block_scan(need > 0 ? need : 0, total, tmp) + (need > 0 ? need : 0);
            need0 += total;
            if (r < t.n_rows) ws.rows[r] = RowPlan{off, upto, keep, need};
        }
        if (tid == 0) {
            ws.h->tokens = off0;
            ws.h->part[0][0] = need0;
        }
    } else {
        long long mine = 0, total;
        for (int p = p0 + tid; p < p1; p += THREADS) mine += __ldcg(t.refs + p) == 0;
        block_scan(mine, total, tmp);
        if (tid == 0) ws.h->part[rank][0] = total;
    }
    cluster_sync();

    // The free pages by rank, as far as they are asked for.
    const long long asked = __ldcg(&ws.h->part[0][0]);
    long long free_before = 0, n_free = 0;
    for (int c = 1; c < CTAS; ++c) {
        const long long v = __ldcg(&ws.h->part[c][0]);
        n_free += v;
        if (c < rank) free_before += v;
    }
    if (rank > 0) {
        for (int base = p0; base < p1 && free_before < asked; base += THREADS) {
            const int p = base + tid;
            const int is_free = p < p1 && __ldcg(t.refs + p) == 0;
            long long total;
            const long long at = free_before + block_scan(is_free, total, tmp);
            if (is_free && at < asked) ws.list[at] = p;
            free_before += total;
        }
    }
    cluster_sync();

    // Deal the pages out, a warp per row.
    const int lane = tid & 31;
    for (int r = gtid >> 5; r < t.n_rows; r += ALL / 32) {
        const RowPlan pl{__ldcg(&ws.rows[r].off), __ldcg(&ws.rows[r].upto), __ldcg(&ws.rows[r].keep), __ldcg(&ws.rows[r].need)};
        const int n = max(a.n_new[r], 0);
        const bool ok = n > 0 && pl.need >= 0 && (pl.need == 0 || pl.upto <= n_free);
        int32_t *row = t.table_out + (size_t)r * t.max_pages;
        const int had = pages_of(pl.keep, t.page_size), tail = pl.keep % t.page_size;
        if (n > 0 && !ok && lane == 0) flag(t.err, QSA_DEVERR_NO_PAGES);
        if (ok) {
            const int want = pages_of((long long)pl.keep + n, t.page_size);
            const int copied = pl.need - (want - had);  // 1: the last page is copied first
            const long long first = pl.upto - pl.need;
            int last = tail ? __ldcg(row + had - 1) : -1;
            if (copied) {
                const int to = __ldcg(ws.list + first);
                if (lane == 0) {
                    ws.copies[atomicAdd(&ws.h->n_copies, 1)] = Copy{last, to, tail};
                    atomicSub(t.refs + last, 1);
                    t.refs[to] = 1;
                    row[had - 1] = to;
                }
                last = to;
            }
            for (int j = had + lane; j < want; j += 32) {
                const int p = __ldcg(ws.list + first + copied + (j - had));
                row[j] = p;
                t.refs[p] = 1;
            }
            // Token i of the row sits at position keep + i.
            for (int i = lane; i < n; i += 32) {
                const int pos = pl.keep + i, j = pos / t.page_size;
                const int p = j < had ? last : __ldcg(ws.list + first + copied + (j - had));
                if (!QSA_IN(pl.off + i, a.n_slots)) continue;
                a.slots[pl.off + i] = p < 0 ? -1 : p * t.page_size + pos % t.page_size;
                a.positions[pl.off + i] = pos;
            }
        } else {
            for (long long i = pl.off + lane; i < pl.off + n && i < a.n_slots; i += 32) a.slots[i] = a.positions[i] = -1;
        }
        __syncwarp();
        if (lane == 0) a.lens_out[r] = pl.keep + (ok ? n : 0);
    }
    for (long long i = __ldcg(&ws.h->tokens) + gtid; i < a.n_slots; i += ALL) a.slots[i] = a.positions[i] = -1;
}

struct CompactLaunch {
    TableArgs t;
    int32_t *page_map, *n_live;
    void *ws;
};

__global__ void __cluster_dims__(CTAS, 1, 1) __launch_bounds__(THREADS) page_compact_kernel(const CompactLaunch a) {
    __shared__ long long tmp[32];
    const TableArgs &t = a.t;
    const int rank = (int)cluster_rank(), tid = threadIdx.x, gtid = rank * THREADS + tid;
    const Ws ws = carve(a.ws, t.n_rows, t.n_pages);
    wait_for_previous_grid();
    allow_dependent_launch();
    for (int p = gtid; p < t.n_pages; p += ALL) t.refs[p] = 0;
    cluster_sync();
    gather_and_count<false>(t, rank);
    cluster_sync();

    // L, the number of held pages.
    const int per = (t.n_pages + CTAS - 1) / CTAS;
    const int p0 = min(rank * per, t.n_pages), p1 = min(p0 + per, t.n_pages);
    long long mine = 0, total;
    for (int p = p0 + tid; p < p1; p += THREADS) mine += __ldcg(t.refs + p) > 0;
    block_scan(mine, total, tmp);
    if (tid == 0) ws.h->part[rank][0] = total;
    cluster_sync();
    int live = 0, live_before = 0;
    for (int c = 0; c < CTAS; ++c) {
        const int v = (int)__ldcg(&ws.h->part[c][0]);
        live += v;
        if (c < rank) live_before += v;
    }

    // Rank of each free page below L among the free, and of each held page at
    // or above L among the held: with b held pages before p, a hole p < L has
    // rank p - b, a mover p >= L has rank b - (held pages below L).  The last
    // is L less the number of holes, so a mover's rank from the end is
    // (held pages from p on), and it needs no second count: movers are ranked
    // from the last one, and the number of holes is known after this pass.
    for (int base = p0; base < p1; base += THREADS) {
        const int p = base + tid;
        const int held = p < p1 && __ldcg(t.refs + p) > 0;
        const int before = live_before + (int)block_scan(held, total, tmp);
        if (p < p1) {
            if (p < live && !held) ws.list[p - before] = p;
            if (p >= live && held) ws.moved[live - 1 - before] = p;  // the last mover is entry 0
            a.page_map[p] = held && p < live ? p : -1;
            if (p == live) ws.h->n_free_or_live = p - before;  // holes below L = movers
            if (p + 1 == t.n_pages && live == t.n_pages) ws.h->n_free_or_live = 0;
        }
        live_before += (int)total;
    }
    cluster_sync();

    const int moves = (int)__ldcg(&ws.h->n_free_or_live);
    for (int i = gtid; i < moves; i += ALL) {
        const int to = __ldcg(ws.list + i), from = __ldcg(ws.moved + (moves - 1 - i));
        a.page_map[from] = to;
        ws.copies[i] = Copy{from, to, t.page_size};
        t.refs[to] = __ldcg(t.refs + from);
        t.refs[from] = 0;
    }
    if (gtid == 0) {
        ws.h->n_copies = moves;
        *a.n_live = live;
    }
    cluster_sync();

    const int lane = tid & 31;
    const int segs = (t.max_pages + SEG - 1) / SEG;
    const long long items = (long long)t.n_rows * segs;
    for (long long it = gtid >> 5; it < items; it += ALL / 32) {
        const int r = (int)(it / segs), j0 = (int)(it % segs) * SEG;
        int from;
        const int had = pages_of(row_keep(t, r, from), t.page_size);
#pragma unroll
        for (int i = 0; i < SEG / 32; ++i) {
            const int j = j0 + i * 32 + lane;
            if (j >= t.max_pages) continue;
            int e = j < had ? t.table[(size_t)r * t.max_pages + j] : -1;
            if (e >= t.n_pages) e = -1;
            t.table_out[(size_t)r * t.max_pages + j] = e < 0 ? -1 : __ldcg(a.page_map + e);
        }
    }
}

// The listed copies, all layers, codes and scales.  A block takes one piece
// of PIECE bytes of one layer's copy at a time, in the order codes of K, codes
// of V, scales of K, scales of V.
constexpr int COPY_THREADS = 256;
constexpr int PIECE = COPY_THREADS * 2 * 16;

struct CopyLaunch {
    int n_layers, n_pages, page_size, code_row, scale_row, n_copies_max;  // bytes per cell
    uint8_t *kq, *vq, *ksc, *vsc;
    void *ws;
    int n_rows;
};

__global__ void __launch_bounds__(COPY_THREADS) page_copy_kernel(const CopyLaunch a) {
    wait_for_previous_grid();
    allow_dependent_launch();
    const Ws ws = carve(a.ws, a.n_rows, a.n_pages);
    const int n = min(__ldcg(&ws.h->n_copies), a.n_copies_max);
    const size_t code_page = (size_t)a.page_size * a.code_row, scale_page = (size_t)a.page_size * a.scale_row;
    const int code_pieces = (int)((code_page + PIECE - 1) / PIECE), scale_pieces = (int)((scale_page + PIECE - 1) / PIECE);
    const int pieces = 2 * (code_pieces + scale_pieces);
    const long long items = (long long)n * a.n_layers * pieces;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        const int piece = (int)(it % pieces);
        const long long cl = it / pieces;
        const int layer = (int)(cl % a.n_layers);
        const Copy c = ws.copies[cl / a.n_layers];
        if (!QSA_IN(c.src, a.n_pages) || !QSA_IN(c.dst, a.n_pages) || !QSA_IN(c.cells, a.page_size + 1)) continue;
        const bool code = piece < 2 * code_pieces;
        const int local = code ? piece : piece - 2 * code_pieces, each = code ? code_pieces : scale_pieces;
        const bool is_v = local >= each;
        const size_t start = (size_t)(local - (is_v ? each : 0)) * PIECE;
        const size_t page = code ? code_page : scale_page;
        const size_t bytes = (size_t)c.cells * (code ? a.code_row : a.scale_row);
        if (start >= bytes) continue;
        uint8_t *base = (code ? (is_v ? a.vq : a.kq) : (is_v ? a.vsc : a.ksc)) + (size_t)layer * a.n_pages * page;
        const uint8_t *src = base + (size_t)c.src * page + start;
        uint8_t *dst = base + (size_t)c.dst * page + start;
        const int len = (int)(bytes - start < PIECE ? bytes - start : PIECE);
        uint4 v[PIECE / (COPY_THREADS * 16)];
#pragma unroll
        for (int k = 0; k < PIECE / (COPY_THREADS * 16); ++k) {
            const int at = (k * COPY_THREADS + (int)threadIdx.x) * 16;
            if (at + 16 <= len) v[k] = *reinterpret_cast<const uint4 *>(src + at);
        }
#pragma unroll
        for (int k = 0; k < PIECE / (COPY_THREADS * 16); ++k) {
            const int at = (k * COPY_THREADS + (int)threadIdx.x) * 16;
            if (at + 16 <= len) *reinterpret_cast<uint4 *>(dst + at) = v[k];
        }
        // An odd number of cells of one KV head leaves eight bytes of scales.
        if ((len & 15) && threadIdx.x == 0)
            *reinterpret_cast<uint2 *>(dst + (len & ~15)) = *reinterpret_cast<const uint2 *>(src + (len & ~15));
    }
}

template <class A>
cudaError_t launch_copies(const A &a, cudaStream_t s) {
    const CopyLaunch c{a.n_layers, a.n_pages, a.page_size, a.n_kv_heads * a.head_dim, a.n_kv_heads * 8,
                       a.n_rows > a.n_pages ? a.n_rows : a.n_pages,
                       reinterpret_cast<uint8_t *>(a.kq), reinterpret_cast<uint8_t *>(a.vq),
                       reinterpret_cast<uint8_t *>(a.ksc), reinterpret_cast<uint8_t *>(a.vsc), a.workspace, a.n_rows};
    return launch_dependent(page_copy_kernel, dim3(152 * 8), dim3(COPY_THREADS), 0, s, c);
}

}  // namespace

size_t pages_workspace_bytes(int n_rows, int n_pages) { return ws_bytes(n_rows, n_pages); }

cudaError_t launch_page_update(const qsa_page_update_args &a, cudaStream_t s) {
    const UpdateLaunch u{{a.n_rows_in, a.n_rows, a.max_pages, a.n_pages, a.page_size, a.page_table, a.seq_lens, a.src,
                          a.page_table_out, a.refs, a.err},
                         a.n_new, a.seq_lens_out, a.slots, a.positions, a.n_slots, a.workspace};
    const cudaError_t e = launch_dependent(page_update_kernel, dim3(CTAS), dim3(THREADS), 0, s, u);
    return e != cudaSuccess ? e : launch_copies(a, s);
}

cudaError_t launch_page_compact(const qsa_page_compact_args &a, cudaStream_t s) {
    const CompactLaunch c{{a.n_rows, a.n_rows, a.max_pages, a.n_pages, a.page_size, a.page_table, a.seq_lens, nullptr,
                           a.page_table_out, a.refs, a.err},
                          a.page_map, a.n_live, a.workspace};
    const cudaError_t e = launch_dependent(page_compact_kernel, dim3(CTAS), dim3(THREADS), 0, s, c);
    return e != cudaSuccess ? e : launch_copies(a, s);
}

}  // namespace qsa

QSA_DEFINE_CHECK_READER(take_check_word_pages)
