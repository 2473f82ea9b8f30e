// qsa_paged_sparse_attn: rows of q over listed pages, a list per KV head.
#include "paged_rows.cuh"

namespace qsa {

size_t paged_sparse_attn_workspace_bytes(int n_q_heads, int n_kv_heads, int head_dim) {
    return Work::bytes(MAX_CTAS, n_q_heads / n_kv_heads, head_dim);
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
    const long long cells = (long long)x.width * x.page_size;
    return x.head_dim == 128 ? launch_rows<1>(a, cells, s) : launch_rows<2>(a, cells, s);
}

}  // namespace qsa

QSA_DEFINE_CHECK_READER(take_check_word_paged_sparse)
