// qsa_paged_attn: rows of q over whole sequences.
#include "paged_rows.cuh"

namespace qsa {

size_t paged_attn_workspace_bytes(int n_q_heads, int n_kv_heads, int head_dim) {
    return Work::bytes(MAX_CTAS, n_q_heads / n_kv_heads, head_dim) + paged_group_workspace_bytes(head_dim);
}

cudaError_t launch_paged_attn(const qsa_paged_attn_args &a, cudaStream_t s) {
    const long long cells = (long long)a.max_pages * a.page_size;
    return a.head_dim == 128 ? launch_rows<1>(a, cells, s) : launch_rows<2>(a, cells, s);
}

}  // namespace qsa

QSA_DEFINE_CHECK_READER(take_check_word_paged_attn)
