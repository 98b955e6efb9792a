// paged_attention.hip -- attention of the newest tokens over the paged cache: the
// dense form of attention.h.

#include "attention.h"

extern "C" {

int xpress_paged_attention(const xpress_paged_attention_args* args, hipStream_t stream)
{
    return call_attention<false>(args, Sparse{nullptr, 0, 0, 0}, stream);
}

int xpress_paged_attention_reserve(int64_t N, int64_t Q, int64_t Hq, int64_t heads, int64_t dim,
                                   int64_t max_len, int64_t window, hipStream_t stream)
{
    const Shape s = {N, Q, Hq, heads, dim, max_len, window};
    if (!shape_ok(s)) return XPRESS_EINVAL;
    if (N == 0 || Q == 0) return XPRESS_OK;
    const Plan p = plan_of(s);
    if (!plan_ok(s, p)) return XPRESS_EINVAL;
    if (p.splits == 1) return XPRESS_OK;
    uint64_t* table = nullptr;
    return workspace_table(stream, plan_words(s, p), &table);
}

int xpress_paged_attention_plan(int64_t N, int64_t Q, int64_t Hq, int64_t heads, int64_t dim,
                                int64_t max_len, int64_t window, int* chunk, int* splits, int* rows,
                                int* launches)
{
    const Shape s = {N, Q, Hq, heads, dim, max_len, window};
    if (!shape_ok(s)) return XPRESS_EINVAL;
    Plan p = {1, 0, 0, 0, 0, 0};
    if (N > 0 && Q > 0) {
        p = plan_of(s);
        if (!plan_ok(s, p)) return XPRESS_EINVAL;
    }
    if (chunk) *chunk = (int)p.chunk;
    if (splits) *splits = (int)p.splits;
    if (rows) *rows = 16 * p.rw;
    if (launches) *launches = p.splits > 1 ? 2 : (int)p.splits;
    return XPRESS_OK;
}

}  // extern "C"
