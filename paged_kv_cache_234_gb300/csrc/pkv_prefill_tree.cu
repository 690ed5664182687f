// pkv_prefill_tree.cu -- attention of trees of drafted tokens with many rows per kv
// head: the prefill kernel, whose products have rows as their long side, with the
// masks and positions of trees.
#define PKV_PREFILL_TREES
#include "pkv_prefill.cu"

#include "pkv_tree_call.h"

namespace pkv {
namespace {

PrefillCall rows_call(const TreeCall &c)
{
    return {c.out, c.query, c.kpool, c.vpool, c.k_scales, c.v_scales, c.num_blocks,
            c.block_tables, c.max_blocks_per_seq, c.query_starts, c.context_lens,
            c.max_context_len, c.num_tokens, c.num_seqs, c.num_heads, c.num_kv_heads, c.head_dim,
            c.block_size, c.softmax_scale, c.logit_cap, c.window, c.slopes, c.prefix_lens,
            c.workspace, c.workspace_bytes, c.dev_status, c.stream, c.parents, c.max_tree_len};
}

}  // namespace

pkv_status tree_rows_workspace(int num_tokens, int num_seqs, int num_heads, int num_kv_heads,
                               int head_dim, int max_context_len, int max_tree_len,
                               size_t *bytes)
{
    Plan plan;
    const pkv_status st = plan_of(num_tokens, num_seqs, num_heads, num_kv_heads, head_dim,
                                  max_context_len, &plan, max_tree_len);
    *bytes = plan.bytes;
    return st;
}

pkv_status launch_tree_rows(const TreeCall &c, TreeKind kind)
{
    return prefill_entry(rows_call(c), kind == kTreeFp8   ? kKvF8
                                       : kind == kTreeInt8 ? kKvI8
                                                           : kKvF16);
}

#ifdef PKV_DEBUG
int set_tree_waits_rows(int give_role, int give_at, int slow_role, int slow_ns, int slow_warp)
{
    const WaitDebug d = {give_role < 0 ? -2 : give_role, give_at, slow_role < 0 ? -2 : slow_role,
                         slow_ns, slow_warp};
    return cudaMemcpyToSymbol(g_wait_debug, &d, sizeof(d)) == cudaSuccess ? 0 : -1;
}
#endif

}  // namespace pkv
