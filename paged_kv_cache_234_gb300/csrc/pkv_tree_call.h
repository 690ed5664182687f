// pkv_tree_call.h -- a call of the tree attention between its translation units: one
// for each kind of cache, so that they compile side by side.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/pkv.h"

namespace pkv {

struct TreeCall {
    void *out;
    const void *query, *kpool, *vpool;
    const float *k_scales, *v_scales;
    int num_blocks;
    const int32_t *block_tables;
    int max_blocks_per_seq;
    const int32_t *query_starts, *context_lens, *parents;
    int max_context_len, max_tree_len, num_tokens, num_seqs, num_heads, num_kv_heads, head_dim,
        block_size;
    float softmax_scale, logit_cap;
    int window;
    const float *slopes;
    const int32_t *prefix_lens;
    void *workspace;
    size_t workspace_bytes;
    int32_t *dev_status;
    void *stream;
};

constexpr int kTreeMetaBytes = 16;   // of a CTA in the workspace: see TreeMeta

constexpr int kTreePieces = 152;     // GB300: one for every SM

struct TreePlan {
    int rows = 0;      // of a work item: 32 or 64 (pkv_tree.cuh); 0: pkv_prefill_tree.cu
    size_t bytes = 0;  // of workspace
};

enum TreeKind { kTreeFp16, kTreeInt8, kTreeFp8 };

// Many rows per kv head.
pkv_status launch_tree_rows(const TreeCall &c, TreeKind kind);
pkv_status tree_rows_workspace(int num_tokens, int num_seqs, int num_heads, int num_kv_heads,
                               int head_dim, int max_context_len, int max_tree_len,
                               size_t *bytes);

// Few of them.

pkv_status launch_tree_fp16(const TreeCall &c, const TreePlan &plan);
pkv_status launch_tree_int8(const TreeCall &c, const TreePlan &plan);
pkv_status launch_tree_fp8(const TreeCall &c, const TreePlan &plan);

#ifdef PKV_DEBUG
// Sets a unit's WaitDebug; 0, or -1 if the CUDA runtime fails.
int set_tree_waits_rows(int give_role, int give_at, int slow_role, int slow_ns, int slow_warp);
int set_tree_waits_fp16(int give_role, int give_at, int slow_role, int slow_ns, int slow_warp);
int set_tree_waits_int8(int give_role, int give_at, int slow_role, int slow_ns, int slow_warp);
int set_tree_waits_fp8(int give_role, int give_at, int slow_role, int slow_ns, int slow_warp);
#endif

}  // namespace pkv
