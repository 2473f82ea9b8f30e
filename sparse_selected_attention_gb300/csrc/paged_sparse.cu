// qsa_paged_sparse_attn: rows of q over listed pages, a list per KV head.
//
// Neighbours in a sequence mostly list the same pages (1984 tokens of 2048 cells each:
// ten of them list a fifth of what they count).  Where that saves enough, rows are
// taken by groups over the pages that any of a group's rows lists (paged_tiles.cuh),
// else one by one (paged_rows.cuh).  What the groups go through is found by a kernel
// before; both kinds then start, and one of them finds that it has nothing to do.  Those
// tokens, 12/1 heads of 128: 138 us by groups (cold: union 8, groups 132, join 12), 229
// one by one.  Lists that turn out not to be alike pay 12 us for the attempt.
//
// Rows one by one: 61 rows of 2 K cells, 48/4 heads of 128, 146 MB: 46.4 us, 3.1 TB/s,
// thirteen units a warp between some 20 us of launch, first loads and ends of rows.
#include "paged_tiles.cuh"

namespace qsa {
namespace {

// Entries of all unions, and groups' first rows, that the workspace has room for; and
// the rows' bits of pages that a block holds.
constexpr long long ENTRIES = 1 << 20;
constexpr int UNION_WARPS = 8, UNION_BYTES = 96 * 1024;
// Sequences that a block's rows may belong to; with more, there is little to share.
constexpr int MOST_RUNS = 4;

// The unions of the groups among `tokens` rows: a bit for each row and page, and the
// pages of 32 at once from these.
__global__ void __launch_bounds__(32 * UNION_WARPS) listed_union_kernel(const ListedArgs a, int tokens, int words) {
    extern __shared__ unsigned bits[];  // [tokens][words | 1]
    __shared__ int row[32], sure[32], count[32], sums[UNION_WARPS], twice;
    __shared__ unsigned starts;
    wait_for_previous_grid();
    allow_dependent_launch();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, kvh = blockIdx.y, page_shift = 31 - __clz(a.page_size);
    const int t0 = blockIdx.x * tokens, n = min(tokens, a.n_tokens - t0), pitch = words | 1;
    int *size = a.shared.size + (size_t)kvh * a.n_tokens + t0;
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
        if (lane == 0) starts = m;
    }
    __syncthreads();
    const unsigned m = starts;
    if (__popc(m) > MOST_RUNS) {
        if (tid < n) size[tid] = tid ? 0 : n << SIZE_BITS | SIZE_MASK;
        return;
    }
    for (int s = 0; s < n;) {
        const unsigned later = m & (0xfffffffeu << s);
        const int e = later ? __ffs(later) - 1 : n;
        for (int i = tid; i < (e - s) * pitch; i += 32 * UNION_WARPS) bits[i] = 0u;
        if (tid == 0) twice = 0;
        __syncthreads();
        for (int i = s + warp; i < e; i += UNION_WARPS) {
            const int32_t *list = a.lists + ((size_t)(t0 + i) * a.n_kv_heads + kvh) * a.width;
            for (int x = lane; x < count[i]; x += 32) {
                const int j = __ldg(list + x);
                bad |= j < -1 || j >= a.max_pages;
                if (j < 0 || j >= a.max_pages || j << page_shift >= sure[i]) continue;
                const unsigned bit = 1u << (j & 31);
                if (atomicOr(&bits[(i - s) * pitch + (j >> 5)], bit) & bit) twice = 1;
            }
        }
        __syncthreads();
        // A warp takes a run of the words.
        const int run = (words + UNION_WARPS - 1) / UNION_WARPS, w0 = min(warp * run, words), w1 = min(w0 + run, words);
        int at = 0;
        for (int w = w0; w < w1; ++w) at += __popc(__reduce_or_sync(0xffffffffu, lane < e - s ? bits[lane * pitch + w] : 0u));
        if (lane == 0) sums[warp] = at;
        __syncthreads();
        int total = 0;
        at = 0;
        for (int w = 0; w < UNION_WARPS; ++w) {
            at += w < warp ? sums[w] : 0;
            total += sums[w];
        }
        const size_t base = ((size_t)kvh * a.n_tokens + t0 + s) * a.width;
        for (int w = w0; w < w1; ++w) {
            const unsigned mine = lane < e - s ? bits[lane * pitch + w] : 0u, any = __reduce_or_sync(0xffffffffu, mine);
            if (!any) continue;
            unsigned who = 0u;
            for (int i = 0; i < e - s; ++i) who |= (__shfl_sync(0xffffffffu, mine, i) >> lane & 1u) << i;
            if (who) {
                const size_t to = base + at + __popc(any & ((1u << lane) - 1));
                const int j = 32 * w + lane, page = __ldg(a.page_table + (size_t)row[s] * a.max_pages + j);
                const bool held = page >= 0 && page < a.n_pages;
                bad |= !held;
                a.shared.unit[to] = make_uint2(j, who);
                a.shared.page[to] = held ? page : -1;
            }
            at += __popc(any);
        }
        for (int i = s + tid; i < e; i += 32 * UNION_WARPS) size[i] = i > s ? 0 : (e - s) << SIZE_BITS | (twice ? SIZE_MASK : total);
        __syncthreads();  // before the words and `twice` are written again
        s = e;
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0 && a.err) atomicOr(a.err, QSA_DEVERR_BAD_ID);
}

size_t rows_bytes(int per, int head_dim) { return (Work::bytes(MAX_CTAS, per, head_dim) + 255) / 256 * 256; }
size_t tiles_bytes(int head_dim) { return (Work::bytes(MAX_GROUP_PARTS, GROUP_ROWS, head_dim) + 255) / 256 * 256; }

template <int S>
cudaError_t launch(ListedArgs a, cudaStream_t s) {
    const long long cells = (long long)a.width * a.page_size, heads = (long long)a.n_tokens * a.n_kv_heads;
    const int per = a.n_q_heads / a.n_kv_heads, tokens = group_tokens(per), words = (a.max_pages + 31) / 32;
    const size_t bytes = sizeof(unsigned) * tokens * (size_t)(words | 1);
    // Groups, where they can be had and like lists would save enough: a tile then does
    // for four units of each of a group's rows.
    const bool may = a.rows && a.n_tokens >= 4 && tokens >= 4 && shared_out<S>(a, cells) && a.n_kv_heads <= MAX_GROUP_PARTS / 2 &&
                     heads * a.width <= ENTRIES && bytes <= UNION_BYTES && heads * (cells / Shape<S>::UNIT) * (tokens - 2) * 10 > (long long)CALL_COST * tokens;
    if (!may) return launch_rows<S>(a, cells, s);
    uint8_t *ws = static_cast<uint8_t *>(a.workspace) + rows_bytes(per, a.head_dim), *u = ws + tiles_bytes(a.head_dim);
    int *const ints = reinterpret_cast<int *>(u + ENTRIES * sizeof(uint2));
    a.shared = Union{reinterpret_cast<uint2 *>(u), ints, ints + ENTRIES};
    a.taken = ints + 2 * ENTRIES;
    cudaError_t e = cudaFuncSetAttribute(listed_union_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, UNION_BYTES);
    if (e == cudaSuccess)
        e = launch_dependent(listed_union_kernel, dim3((a.n_tokens + tokens - 1) / tokens, a.n_kv_heads), dim3(32 * UNION_WARPS), bytes, s, a, tokens, words);
    if (e == cudaSuccess) e = launch_tiles<S>(a, ws, s);
    if (e == cudaSuccess) e = launch_rows<S>(a, cells, s);
    return e == cudaSuccess ? launch_tiles_join<S>(a, ws, s) : e;
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
