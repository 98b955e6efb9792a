// sparse_attention.hip -- attention over the paged cache where the queries do not see
// all that came before them: the nodes of a tree, and a window with sinks.  The
// sparse form of attention.h, and for many rows that of wide_attention.hip.

#include "attention.h"

extern "C" {

int xpress_tree_attention(const xpress_paged_attention_args* args, const int32_t* tree,
                          int64_t stride_tree_n, int64_t stride_tree_i, int64_t sinks, hipStream_t stream)
{
    if (!tree && args && args->cache.seqs > 0 && args->Q > 0) return XPRESS_EINVAL;
    return call_attention<true>(args, Sparse{tree, stride_tree_n, stride_tree_i, sinks}, stream);
}

int xpress_sink_attention(const xpress_paged_attention_args* args, int64_t sinks, hipStream_t stream)
{
    return call_attention<true>(args, Sparse{nullptr, 0, 0, sinks}, stream);
}

int xpress_sparse_attention_reserve(int64_t N, int64_t Q, int64_t Hq, int64_t heads, int64_t dim,
                                    int64_t max_len, int64_t window, int64_t sinks, int tree,
                                    hipStream_t stream)
{
    const Shape s = {N, Q, Hq, heads, dim, max_len, window, sinks, tree != 0, true};
    if (!shape_ok(s)) return XPRESS_EINVAL;
    if (N == 0 || Q == 0) return XPRESS_OK;
    const Plan p = plan_of(s);
    if (!plan_ok(s, p)) return XPRESS_EINVAL;
    if (p.splits == 1) return XPRESS_OK;
    uint64_t* table = nullptr;
    return workspace_table(stream, plan_words(s, p), &table);
}

}  // extern "C"
