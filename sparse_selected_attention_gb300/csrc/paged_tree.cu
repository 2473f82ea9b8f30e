// qsa_paged_tree_attn: drafted tokens over a prefix and, by bits, each other.
//
// Tokens of one sequence (rows of q that follow one another) read it together
// (paged_tiles.cuh), where that saves enough; else, and where tables are short, they go
// one by one (paged_rows.cuh).  As with listed rows, both kinds start, and one of them
// finds that it has nothing to do.
#include "paged_tiles.cuh"

namespace qsa {
namespace {

// The rows' partials, the groups', and a word for each KV head.
size_t rows_and_tiles_bytes(int per, int head_dim) {
    return (Work::bytes(MAX_CTAS, per, head_dim) + 255) / 256 * 256 + (Work::bytes(MAX_GROUP_PARTS, M, head_dim) + 255) / 256 * 256;
}

template <int S>
cudaError_t launch(TreeArgs a, cudaStream_t s) {
    const long long cells = (long long)a.max_pages * a.page_size;
    const int per = a.n_q_heads / a.n_kv_heads;
    // Tenths of a unit, if all rows are as long as the table is wide.
    const long long most = (long long)a.n_tokens * a.n_kv_heads * (cells / Shape<S>::UNIT) * 10;
    // The lengths and the order of the tokens say which kind is taken, and those only the
    // device knows.  (Together unseen, 24 trees of 16 to 32 tokens, 32/8 heads, would take
    // 127 us, not 132, but given level by level, rows 0, 1, 2, .., 0, 1, 2, .., 2600, where
    // one by one they take 1150.)  With more KV heads than there are places for partials,
    // no kind has more than one CTA for a head, and all go together.
    const bool both = a.n_kv_heads <= MAX_GROUP_PARTS;
    if (!a.rows || a.n_tokens < 2 || cells <= WHOLE * Shape<S>::UNIT || (both && most <= CALL_COST)) return launch_rows<S>(a, cells, s);
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    if (both) a.taken = reinterpret_cast<int *>(ws + rows_and_tiles_bytes(per, a.head_dim));
    ws += (Work::bytes(MAX_CTAS, per, a.head_dim) + 255) / 256 * 256;
    cudaError_t e = launch_tiles<S>(a, ws, s);
    if (e == cudaSuccess && both) e = launch_rows<S>(a, cells, s);
    return e == cudaSuccess && both ? launch_tiles_join<S>(a, ws, s) : e;
}

}  // namespace

size_t paged_tree_attn_workspace_bytes(int n_q_heads, int n_kv_heads, int head_dim) {
    return rows_and_tiles_bytes(n_q_heads / n_kv_heads, head_dim) + sizeof(int) * MAX_GROUP_PARTS;
}

cudaError_t launch_paged_tree_attn(const qsa_paged_tree_attn_args &x, cudaStream_t s) {
    TreeArgs a{};
    static_cast<qsa_paged_attn_args &>(a) =
        qsa_paged_attn_args{x.n_tokens,  x.n_q_heads, x.n_kv_heads, x.head_dim,   x.group,    x.page_size,     x.n_pages, x.n_rows,
                            x.max_pages, x.dtype,     x.q,          x.kq,         x.vq,       x.ksc,           x.vsc,     x.page_table,
                            x.prefix_lens, x.rows,    x.softmax_scale, x.gate,    x.out,      x.lse,           x.workspace,
                            x.workspace_bytes, x.err};
    a.mask = reinterpret_cast<const uint32_t *>(x.mask);
    a.words = x.words;
    return x.head_dim == 128 ? launch<1>(a, s) : launch<2>(a, s);
}

}  // namespace qsa

QSA_DEFINE_CHECK_READER(take_check_word_paged_tree)
