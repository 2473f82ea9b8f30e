// qsa_paged_tree_attn: drafted tokens over a prefix and, by bits, each other.
//
// Tokens of one sequence (rows of q that follow one another) read it together
// (paged_tiles.cuh); rows without such company, and short tables, go row by row
// (paged_rows.cuh).
#include "paged_tiles.cuh"

namespace qsa {
namespace {

template <int S>
cudaError_t launch(const TreeArgs &a, cudaStream_t s) {
    const long long cells = (long long)a.max_pages * a.page_size;
    if (!a.rows || a.n_tokens < 2 || cells <= WHOLE * Shape<S>::UNIT) return launch_rows<S>(a, cells, s);
    return launch_tiles<S>(a, static_cast<uint8_t *>(a.workspace) + Work::bytes(MAX_CTAS, a.n_q_heads / a.n_kv_heads, a.head_dim), s);
}

}  // namespace

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
