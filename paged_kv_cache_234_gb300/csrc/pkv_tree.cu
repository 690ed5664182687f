// pkv_tree.cu -- entry points of the tree attention (pkv_tree.cuh): checks, and the
// plan of a call from its sizes.
#include <cuda_runtime.h>
#include <math.h>

#include "pkv_host.cuh"
#include "pkv_score.cuh"
#include "pkv_tree_call.h"

namespace pkv {
namespace {

constexpr int kPage = 16, kTile = 128;   // tokens of a page, keys of a step

// From the sizes alone.  Up to 64 rows per kv head (tokens times heads) are the short
// side of both products, keys the long one; with more the rows are.  The two ways, in us,
// back to back (32 / 8 heads, head_dim 128; a tree of 8 tokens has 32 rows, of 16 tokens 64):
//                          fp16            INT8            FP8
//   64 trees of 8, 2048    96.1 | 102.2    81.1 | 114.8    78.1 | 113.5
//   64 trees of 16, 2048  102.3 | 104.3    95.0 | 117.1    90.8 | 116.3
//   one of 8, 131072       92.6 |  93.0    70.6 |  94.6    67.3 |  99.2
//   8 trees of 16, 512     14.1 |  12.6    15.3 |  14.0    15.1 |  14.1
// Beyond 64 the short side no longer fits the score warps' registers; short contexts of
// more than 32 rows lose up to a seventh here.
pkv_status tree_plan(int num_tokens, int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                     int max_context_len, int max_tree_len, TreePlan *plan)
{
    if (num_tokens < 0 || num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
        max_context_len < 0 || max_tree_len < 0 || num_heads % num_kv_heads != 0)
        return PKV_ERR_INVALID_ARG;
    if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
    // (a token at least, also where the bound allows none: an item has room for its heads)
    const int most = max_tree_len < num_tokens ? max_tree_len : num_tokens;
    const int64_t rows = static_cast<int64_t>(most > 0 ? most : 1) * (num_heads / num_kv_heads);
    plan->rows = rows <= 32 ? 32 : rows <= 64 ? 64 : 0;
    if (num_heads / num_kv_heads > 64) plan->rows = 0;
    if (plan->rows == 0)
        return tree_rows_workspace(num_tokens, num_seqs, num_heads, num_kv_heads, head_dim,
                                   max_context_len, max_tree_len, &plan->bytes);
    plan->bytes =
        kTreePieces * (2 * plan->rows * (head_dim + 2) * sizeof(float) + kTreeMetaBytes);
    return PKV_OK;
}

pkv_status tree_entry(const TreeCall &c, TreeKind kind)
{
    const bool codes = kind != kTreeFp16;
    if (!c.kpool || !c.vpool || !c.query_starts) return PKV_ERR_INVALID_ARG;
    // (arrays without elements may be null)
    if (c.num_tokens != 0 && (!c.out || !c.query || !c.parents)) return PKV_ERR_INVALID_ARG;
    if (c.num_seqs != 0 && (!c.context_lens || (!c.block_tables && c.max_blocks_per_seq != 0)))
        return PKV_ERR_INVALID_ARG;
    if (codes && (!c.k_scales || !c.v_scales)) return PKV_ERR_INVALID_ARG;
    if (c.num_blocks <= 0 || c.block_size <= 0 || c.max_blocks_per_seq < 0 || c.window < 0)
        return PKV_ERR_INVALID_ARG;
    if (!(fabsf(c.softmax_scale) <= 2.0e38f) || !valid_cap(c.logit_cap)) return PKV_ERR_INVALID_ARG;
    TreePlan plan;
    const pkv_status st = tree_plan(c.num_tokens, c.num_seqs, c.num_heads, c.num_kv_heads,
                                    c.head_dim, c.max_context_len, c.max_tree_len, &plan);
    if (st != PKV_OK) return st;
    if (c.block_size != kPage) return PKV_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(c.num_blocks) * c.num_kv_heads * kPage > 0x7fffffffLL ||
        c.max_context_len > INT32_MAX - 4 * kTile)
        return PKV_ERR_UNSUPPORTED;
    if (!aligned(c.out, 16) || !aligned(c.query, 16) || !aligned(c.kpool, 16) ||
        !aligned(c.vpool, 16) || !aligned(c.block_tables, 4) || !aligned(c.query_starts, 4) ||
        !aligned(c.context_lens, 4) || !aligned(c.parents, 4) || !aligned(c.dev_status, 4) ||
        !aligned(c.k_scales, 4) || !aligned(c.v_scales, 4) || !aligned(c.slopes, 4) ||
        !aligned(c.prefix_lens, 4))
        return PKV_ERR_MISALIGNED;
    if (c.num_tokens == 0 || c.num_seqs == 0) return PKV_OK;
    if (plan.rows == 0) return launch_tree_rows(c, kind);
    // the line of tiles is counted in 32 bits
    const int64_t cap = static_cast<int64_t>(c.max_blocks_per_seq) * kPage;
    const int64_t most = (c.max_context_len < cap ? c.max_context_len : cap) / kTile + 2;
    const int64_t line = static_cast<int64_t>(c.num_seqs) * c.num_kv_heads;
    if (line > INT32_MAX || line * most > INT32_MAX) return PKV_ERR_UNSUPPORTED;
    if (plan.bytes > 0 && (!c.workspace || c.workspace_bytes < plan.bytes)) return PKV_ERR_WORKSPACE;
    if (!aligned(c.workspace, 16)) return PKV_ERR_MISALIGNED;
    return kind == kTreeFp8    ? launch_tree_fp8(c, plan)
           : kind == kTreeInt8 ? launch_tree_int8(c, plan)
                               : launch_tree_fp16(c, plan);
}

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_paged_tree_fp16(
    void *out, const void *query, const void *k_cache, const void *v_cache, int num_blocks,
    const int32_t *block_tables, int max_blocks_per_seq, const int32_t *query_starts,
    const int32_t *context_lens, const int32_t *parents, int max_context_len, int max_tree_len,
    int num_tokens, int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
    float softmax_scale, float logit_cap, int window, const float *slopes,
    const int32_t *prefix_lens, void *workspace, size_t workspace_bytes, int32_t *dev_status,
    void *stream)
{
    const pkv::TreeCall c{out, query, k_cache, v_cache, nullptr, nullptr, num_blocks, block_tables,
                          max_blocks_per_seq, query_starts, context_lens, parents,
                          max_context_len, max_tree_len, num_tokens, num_seqs, num_heads,
                          num_kv_heads, head_dim, block_size, softmax_scale, logit_cap, window,
                          slopes, prefix_lens, workspace, workspace_bytes, dev_status, stream};
    return pkv::tree_entry(c, pkv::kTreeFp16);
}

extern "C" pkv_status pkv_paged_tree_int8(
    void *out, const void *query, const int8_t *k_codes, const int8_t *v_codes,
    const float *k_scales, const float *v_scales, int num_blocks, const int32_t *block_tables,
    int max_blocks_per_seq, const int32_t *query_starts, const int32_t *context_lens,
    const int32_t *parents, int max_context_len, int max_tree_len, int num_tokens, int num_seqs,
    int num_heads, int num_kv_heads, int head_dim, int block_size, float softmax_scale,
    float logit_cap, int window, const float *slopes, const int32_t *prefix_lens, void *workspace,
    size_t workspace_bytes, int32_t *dev_status, void *stream)
{
    const pkv::TreeCall c{out, query, k_codes, v_codes, k_scales, v_scales, num_blocks,
                          block_tables, max_blocks_per_seq, query_starts, context_lens, parents,
                          max_context_len, max_tree_len, num_tokens, num_seqs, num_heads,
                          num_kv_heads, head_dim, block_size, softmax_scale, logit_cap, window,
                          slopes, prefix_lens, workspace, workspace_bytes, dev_status, stream};
    return pkv::tree_entry(c, pkv::kTreeInt8);
}

extern "C" pkv_status pkv_paged_tree_fp8(
    void *out, const void *query, const uint8_t *k_codes, const uint8_t *v_codes,
    const float *k_scales, const float *v_scales, int num_blocks, const int32_t *block_tables,
    int max_blocks_per_seq, const int32_t *query_starts, const int32_t *context_lens,
    const int32_t *parents, int max_context_len, int max_tree_len, int num_tokens, int num_seqs,
    int num_heads, int num_kv_heads, int head_dim, int block_size, float softmax_scale,
    float logit_cap, int window, const float *slopes, const int32_t *prefix_lens, void *workspace,
    size_t workspace_bytes, int32_t *dev_status, void *stream)
{
    const pkv::TreeCall c{out, query, k_codes, v_codes, k_scales, v_scales, num_blocks,
                          block_tables, max_blocks_per_seq, query_starts, context_lens, parents,
                          max_context_len, max_tree_len, num_tokens, num_seqs, num_heads,
                          num_kv_heads, head_dim, block_size, softmax_scale, logit_cap, window,
                          slopes, prefix_lens, workspace, workspace_bytes, dev_status, stream};
    return pkv::tree_entry(c, pkv::kTreeFp8);
}

extern "C" size_t pkv_tree_workspace_size(int num_tokens, int num_seqs, int num_heads,
                                          int num_kv_heads, int head_dim, int max_context_len,
                                          int max_tree_len)
{
    pkv::TreePlan plan;
    if (pkv::tree_plan(num_tokens, num_seqs, num_heads, num_kv_heads, head_dim, max_context_len,
                       max_tree_len, &plan) != PKV_OK)
        return 0;
    return plan.bytes;
}

#ifdef PKV_DEBUG
// Debug builds only: see WaitDebug (roles 0 rows, 1 products, 2 K and query loads, 3
// V loads, 4 items, 5 widening of codes).  A negative role resets its setting.
// Synchronises with the device; returns 0, or -1 if the CUDA runtime fails or an
// argument is out of range.
static int set_tree(int give_role, int give_at, int slow_role, int slow_ns, int slow_warp)
{
    if (give_role > 5 || slow_role > 5 || slow_ns < 0 || slow_ns > 1000000 ||
        cudaDeviceSynchronize() != cudaSuccess)
        return -1;
    return pkv::set_tree_waits_rows(give_role, give_at, slow_role, slow_ns, slow_warp) |
           pkv::set_tree_waits_fp16(give_role, give_at, slow_role, slow_ns, slow_warp) |
           pkv::set_tree_waits_int8(give_role, give_at, slow_role, slow_ns, slow_warp) |
           pkv::set_tree_waits_fp8(give_role, give_at, slow_role, slow_ns, slow_warp);
}

extern "C" __attribute__((visibility("default"))) int pkv_debug_set_tree(int give_role, int give_at,
                                                                         int slow_role, int slow_ns)
{
    return set_tree(give_role, give_at, slow_role, slow_ns, 0);
}

// Warp `warp` (0 to 3) of every group of score warps alone begins its waits slow_ns
// later; a negative one resets the setting.
extern "C" __attribute__((visibility("default"))) int pkv_debug_set_tree_warp(int warp, int slow_ns)
{
    if (warp > 3) return -1;
    return set_tree(-1, 0, warp < 0 ? -1 : 0, slow_ns, warp < 0 ? 0 : warp + 1);
}
#endif
