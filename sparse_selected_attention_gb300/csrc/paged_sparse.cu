// qsa_paged_sparse_attn: rows of q over listed pages, a list per KV head.
//
// Neighbours in a sequence mostly list the same pages (1984 tokens of 2048 cells each:
// ten of them list a fifth of what they count).  Where that saves enough, rows are
// taken by groups over the pages that any of a group's rows lists (paged_tiles.cuh),
// else one by one (paged_rows.cuh).  What the groups go through is found by a kernel
// before; both kinds then start, and one of them finds that it has nothing to do.  Those
// tokens, 12/1 heads of 128: 138 us by groups (cold: union 10, groups 132, join 12), 229
// one by one.  Lists that turn out not to be alike pay 11 to 14 us for the attempt.
//
// Rows one by one: 61 rows of 2 K cells, 48/4 heads of 128, 146 MB: 47.8 us, 3.1 TB/s,
// thirteen units a warp between some 20 us of launch, first loads and ends of rows.
#include "paged_tiles.cuh"

namespace qsa {
namespace {

// Entries of all unions, and groups' first rows, that the workspace has room for; and
// the rows' bits of pages that a block holds.
constexpr long long ENTRIES = 1 << 20;
constexpr int UNION_WARPS = 32, UNION_BYTES = 96 * 1024, BATCH = 4;  // warps at most; BATCH: loads of a lane on their way

// The unions of the groups among `tokens` rows: a bit for each row and page, and the
// pages of 32 at once from these.  A row without neighbours of its sequence is a group
// by itself, which costs what its own tiles cost and leaves the others theirs.
__global__ void __launch_bounds__(32 * UNION_WARPS) listed_union_kernel(const ListedArgs a, int tokens, int words) {
    extern __shared__ unsigned bits[];  // [tokens][words | 1]
    __shared__ int row[32], sure[32], count[32], sums[32][UNION_WARPS];
    __shared__ unsigned starts, twice;
    wait_for_previous_grid();
    allow_dependent_launch();
    const int tid = threadIdx.x, warps = blockDim.x >> 5, lane = tid & 31, warp = tid >> 5, kvh = blockIdx.y, page_shift = 31 - __clz(a.page_size);
    const int t0 = blockIdx.x * tokens, n = min(tokens, a.n_tokens - t0), pitch = words | 1;
    bool bad = false;
    if (warp == 0) {
        int trow = 0, known = 0, raw = 0;
        if (lane < n) {
            count[lane] = row_len(a, t0 + lane, kvh, trow, known, bad) >> page_shift;
            row[lane] = trow;
            sure[lane] = known;
            raw = __ldg(a.rows + t0 + lane);
        }
        const int before = __shfl_up_sync(0xffffffffu, raw, 1);
        const unsigned m = __ballot_sync(0xffffffffu, lane < n && (lane == 0 || raw != before));
        if (lane == 0) {
            starts = m;
            twice = 0u;
        }
    }
    for (int i = tid; i < n * pitch; i += 32 * warps) bits[i] = 0u;
    __syncthreads();
    const unsigned single = starts & (starts >> 1 | 1u << (n - 1));  // rows that are a group by themselves
    for (int i = warp; i < n; i += warps) {
        const int32_t *list = a.lists + ((size_t)(t0 + i) * a.n_kv_heads + kvh) * a.width;
        const bool alone = single >> i & 1u;  // then its list is the union, whatever its order
        const size_t base = ((size_t)kvh * a.n_tokens + t0 + i) * a.width;
        int total = 0;
        for (int x0 = 0; x0 < count[i]; x0 += 32 * BATCH) {
            int j[BATCH], page[BATCH];
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const int x = x0 + 32 * k + lane;
                j[k] = x < count[i] ? __ldg(list + x) : -1;
            }
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                bad |= j[k] < -1 || j[k] >= a.max_pages;
                if (j[k] >= a.max_pages || (j[k] >= 0 && j[k] << page_shift >= sure[i])) j[k] = -1;
                page[k] = alone && j[k] >= 0 ? __ldg(a.page_table + (size_t)row[i] * a.max_pages + j[k]) : -1;
            }
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                if (alone) {
                    const unsigned in = __ballot_sync(0xffffffffu, j[k] >= 0);
                    if (j[k] >= 0) {
                        const size_t to = base + total + __popc(in & ((1u << lane) - 1));
                        const bool held = page[k] >= 0 && page[k] < a.n_pages;
                        bad |= !held;
                        a.shared.unit[to] = make_uint2(j[k], 1u);
                        a.shared.page[to] = held ? page[k] : -1;
                    }
                    total += __popc(in);
                } else if (j[k] >= 0) {
                    const unsigned bit = 1u << (j[k] & 31);
                    if (atomicOr(&bits[i * pitch + (j[k] >> 5)], bit) & bit) atomicOr(&twice, 1u << i);
                }
            }
        }
        if (alone && lane == 0) a.shared.size[(size_t)kvh * a.n_tokens + t0 + i] = 1 << SIZE_BITS | total;
    }
    if (single == starts) {  // the same in all threads
        if (__any_sync(0xffffffffu, bad) && lane == 0 && a.err) atomicOr(a.err, QSA_DEVERR_BAD_ID);
        return;
    }
    __syncthreads();
    // The other groups: rows s .. e - 1.  Of each, a warp takes a run of the words: it counts its
    // pages, and writes them behind those of the warps before.
    const int run = (words + warps - 1) / warps, w0 = min(warp * run, words), w1 = min(w0 + run, words);
    auto each_group = [&](auto &&f) {
        for (unsigned left = starts & ~single; left; left &= left - 1) {
            const int s = __ffs(left) - 1;
            const unsigned later = starts & (0xfffffffeu << s);
            f(s, later ? __ffs(later) - 1 : n);
        }
    };
    auto any_of = [&](int s, int e, int w) {
        unsigned any = 0u;
        for (int i = s; i < e; ++i) any |= w < w1 ? bits[i * pitch + w] : 0u;
        return any;
    };
    each_group([&](int s, int e) {
        int pages = 0;
        for (int w = w0; w < w1; w += 32) pages += __popc(any_of(s, e, w + lane));
        pages = __reduce_add_sync(0xffffffffu, pages);
        if (lane == 0) sums[s][warp] = pages;
    });
    __syncthreads();
    each_group([&](int s, int e) {
        size_t to = ((size_t)kvh * a.n_tokens + t0 + s) * a.width;
        for (int w = 0; w < warp; ++w) to += sums[s][w];
        for (int base = w0; base < w1; base += 32) {
            const unsigned any = any_of(s, e, base + lane);
            for (unsigned left = __ballot_sync(0xffffffffu, any != 0u); left; left &= left - 1) {
                const int in = __ffs(left) - 1;
                const unsigned all = __shfl_sync(0xffffffffu, any, in), mine = lane < e - s ? bits[(s + lane) * pitch + base + in] : 0u;
                unsigned who = 0u;
                for (int i = 0; i < e - s; ++i) who |= (__shfl_sync(0xffffffffu, mine, i) >> lane & 1u) << i;
                if (who) a.shared.unit[to + __popc(all & ((1u << lane) - 1))] = make_uint2(32 * (base + in) + lane, who);
                to += __popc(all);
            }
        }
    });
    __syncthreads();
    // Their places in the pool, 32 at a time by the warps in turn.
    int turn = 0;
    each_group([&](int s, int e) {
        int total = 0;
        for (int w = 0; w < warps; ++w) total += sums[s][w];
        const size_t to = ((size_t)kvh * a.n_tokens + t0 + s) * a.width;
        for (int x = lane; x - lane < total; x += 32, ++turn) {
            if (turn % warps != warp || x >= total) continue;
            const int page = __ldg(a.page_table + (size_t)row[s] * a.max_pages + a.shared.unit[to + x].x);
            const bool held = page >= 0 && page < a.n_pages;
            bad |= !held;
            a.shared.page[to + x] = held ? page : -1;
        }
        if (tid >= s && tid < e) {
            const unsigned own = (e - s == 32 ? 0xffffffffu : (1u << (e - s)) - 1) << s;
            a.shared.size[(size_t)kvh * a.n_tokens + t0 + tid] = tid > s ? 0 : (e - s) << SIZE_BITS | (twice & own ? SIZE_MASK : total);
        }
    });
    if (__any_sync(0xffffffffu, bad) && lane == 0 && a.err) atomicOr(a.err, QSA_DEVERR_BAD_ID);
}

size_t rows_bytes(int per, int head_dim) { return (Work::bytes(MAX_CTAS, per, head_dim) + 255) / 256 * 256; }
size_t tiles_bytes(int head_dim) { return (Work::bytes(MAX_GROUP_PARTS, GROUP_ROWS, head_dim) + 255) / 256 * 256; }

// Words of a row's bits of pages.
int bit_words(const ListedArgs &a) { return (a.max_pages + 31) / 32; }

// a: rows that groups may be taken of, with no more list entries than ENTRIES.
template <int S>
cudaError_t launch_slice(ListedArgs a, cudaStream_t s) {
    const long long cells = (long long)a.width * a.page_size, heads = (long long)a.n_tokens * a.n_kv_heads;
    const int per = a.n_q_heads / a.n_kv_heads, tokens = group_tokens(per), words = bit_words(a);
    // Groups, where like lists would save enough: a tile then does for four units of each
    // of a group's rows.
    const bool may = a.n_tokens >= 4 && heads * (cells / Shape<S>::UNIT) * (tokens - 2) * 10 > (long long)CALL_COST * tokens;
    if (!may) return launch_rows<S>(a, cells, s);
    uint8_t *ws = static_cast<uint8_t *>(a.workspace) + rows_bytes(per, a.head_dim), *u = ws + tiles_bytes(a.head_dim);
    int *const ints = reinterpret_cast<int *>(u + ENTRIES * sizeof(uint2));
    a.shared = Union{reinterpret_cast<uint2 *>(u), ints, ints + ENTRIES};
    a.taken = ints + 2 * ENTRIES;
    cudaError_t e = cudaFuncSetAttribute(listed_union_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, UNION_BYTES);
    // Blocks of eight warps go round sooner, few blocks end sooner with all the warps that
    // fit: 1984 tokens of 12/1 heads (199 blocks) 139 us in all, 143; 61 rows of 32/8 (16) 86, 81.
    const dim3 grid((a.n_tokens + tokens - 1) / tokens, a.n_kv_heads);
    const int warps = grid.x * grid.y > 152 ? 8 : UNION_WARPS;
    if (e == cudaSuccess)
        e = launch_dependent(listed_union_kernel, grid, dim3(32 * warps), sizeof(unsigned) * tokens * (size_t)(words | 1), s, a, tokens, words);
    if (e == cudaSuccess) e = launch_tiles<S>(a, ws, s);
    if (e == cudaSuccess) e = launch_rows<S>(a, cells, s);
    return e == cudaSuccess ? launch_tiles_join<S>(a, ws, s) : e;
}

// A call, in slices of tokens whose lists the workspace has room for, one after the other
// in the same workspace; they end where groups do.  1984 tokens of 32/8 heads, 128 pages of
// 16: 480 us in two slices, one by one 1805; in lists of 1024, 872 in sixteen.  Slices of not
// even MIN_SLICE tokens could cost more in launches than their groups save (256 rows
// without neighbours, 32 pages in lists of 1024: 123 us in two slices, one by one 85).
constexpr long long MIN_SLICE = 128;
template <int S>
cudaError_t launch(const ListedArgs &a, cudaStream_t s) {
    const int tokens = group_tokens(a.n_q_heads / a.n_kv_heads);
    const long long cells = (long long)a.width * a.page_size, fit = ENTRIES / ((long long)a.n_kv_heads * a.width), most = fit / tokens * tokens;
    const bool all = (long long)a.n_tokens * a.n_kv_heads * a.width <= ENTRIES;
    const bool groups = a.rows && shared_out<S>(a, cells) && a.n_kv_heads <= MAX_GROUP_PARTS / 2 &&
                        sizeof(unsigned) * tokens * (size_t)(bit_words(a) | 1) <= UNION_BYTES;
    if (!groups || (!all && fit < MIN_SLICE)) return launch_rows<S>(a, cells, s);
    if (all) return launch_slice<S>(a, s);
    const long long slices = (a.n_tokens + most - 1) / most, each = ((a.n_tokens + slices - 1) / slices + tokens - 1) / tokens * tokens;
    cudaError_t e = cudaSuccess;
    for (long long t = 0; t < a.n_tokens && e == cudaSuccess; t += each) {
        const size_t head = (size_t)t * a.n_q_heads, list = (size_t)t * a.n_kv_heads, at = head * a.head_dim;
        ListedArgs x = a;
        x.n_tokens = (int)std::min(each, a.n_tokens - t);
        x.q = static_cast<const uint16_t *>(a.q) + at;
        x.out = static_cast<uint16_t *>(a.out) + at;
        x.gate = a.gate ? a.gate + at : nullptr;
        x.lse = a.lse ? a.lse + head : nullptr;
        x.seq_lens = a.seq_lens + t;
        x.rows = a.rows + t;
        x.lists = a.lists + list * a.width;
        x.counts = a.counts + list;
        e = launch_slice<S>(x, s);
    }
    return e;
}

}  // namespace

size_t paged_sparse_attn_workspace_bytes(int n_q_heads, int n_kv_heads, int head_dim) {
    return rows_bytes(n_q_heads / n_kv_heads, head_dim) + tiles_bytes(head_dim) + ENTRIES * (sizeof(uint2) + 2 * sizeof(int)) +
           sizeof(int) * MAX_GROUP_PARTS;
}

cudaError_t launch_paged_sparse_attn(const qsa_paged_sparse_attn_args &x, cudaStream_t s) {
    ListedArgs a{};
    static_cast<qsa_paged_attn_args &>(a) =
        qsa_paged_attn_args{x.n_tokens,  x.n_q_heads, x.n_kv_heads, x.head_dim,   x.group,    x.page_size,     x.n_pages, x.n_rows,
                            x.max_pages, x.dtype,     x.q,          x.kq,         x.vq,       x.ksc,           x.vsc,     x.page_table,
                            x.seq_lens,  x.rows,      x.softmax_scale, x.gate,    x.out,      x.lse,           x.workspace,
                            x.workspace_bytes, x.err};
    a.lists = x.pages;
    a.counts = x.counts;
    a.width = x.width;
    return x.head_dim == 128 ? launch<1>(a, s) : launch<2>(a, s);
}

}  // namespace qsa

QSA_DEFINE_CHECK_READER(take_check_word_paged_sparse)
