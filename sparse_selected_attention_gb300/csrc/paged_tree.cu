// qsa_paged_tree_attn: drafted tokens over a prefix and, by bits, each other.
#include "paged_rows.cuh"

namespace qsa {

cudaError_t launch_paged_tree_attn(const qsa_paged_tree_attn_args &x, cudaStream_t s) {
    TreeArgs a{};
    static_cast<qsa_paged_attn_args &>(a) =
        qsa_paged_attn_args{x.n_tokens,  x.n_q_heads, x.n_kv_heads, x.head_dim,   x.group,    x.page_size,     x.n_pages, x.n_rows,
                            x.max_pages, x.dtype,     x.q,          x.kq,         x.vq,       x.ksc,           x.vsc,     x.page_table,
                            x.prefix_lens, x.rows,    x.softmax_scale, x.gate,    x.out,      x.lse,           x.workspace,
                            x.workspace_bytes, x.err};
    a.mask = reinterpret_cast<const uint32_t *>(x.mask);
    a.words = x.words;
    const long long cells = (long long)x.max_pages * x.page_size;
    return x.head_dim == 128 ? launch_rows<1>(a, cells, s) : launch_rows<2>(a, cells, s);
}

}  // namespace qsa

QSA_DEFINE_CHECK_READER(take_check_word_paged_tree)
