// pkv_decode_scored.cu -- decode-step attention whose scores are capped by a
// tanh, get a bias that depends on the distance, or are masked to a window and
// a visible prefix: the kernels of pkv_decode.cuh with kScored.
//
// With the query at position i = ctx - 1, key t and z = softmax_scale <q, K_t>:
//   z' = cap tanh(z / cap)  (cap > 0),   z'' = z' - slope[h] (i - t),
//   t is seen if i - t < window (window > 0) or t < prefix_len.
// Bound by memory like the plain decode, over the pages that hold a seen key:
// the page stream leaves out the pages between the prefix and the window, so a
// worker's share is of bytes that are read.  The cap, the bias and the masks
// work on the scores in registers, base-2 units; the masked keys' V rows are
// zeroed in the fragments, so they may hold anything.  The output is fp16, the
// type of the query and of the projection that reads it, rounded once from the
// fp32 quotient; partial results stay fp32.  Measured on GB300, 32 / 8 heads,
// head_dim 128: 64 x 2048, fp16, capped 86 us (6.2 TB/s, 0.92 of the copy
// rate); 256 sequences up to 4096, INT8, window 1024 with 16 prefix tokens 101
// us (4.8 TB/s); 1 x 131072, FP8, biased 58 us (4.6 TB/s).
#include "pkv_decode.cuh"

extern "C" pkv_status pkv_paged_decode_scored_fp16(
    void *out, const void *query, const void *k_cache, const void *v_cache, int num_blocks,
    const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
    int max_context_len, int num_seqs, int num_heads, int num_kv_heads, int head_dim,
    int block_size, float softmax_scale, float logit_cap, int window, const float *slopes,
    const int32_t *prefix_lens, void *workspace, size_t workspace_bytes, int32_t *dev_status,
    void *stream)
{
    const pkv::DecodeCall call{out, query, k_cache, v_cache, nullptr, nullptr, num_blocks,
                               block_tables, max_blocks_per_seq, context_lens, max_context_len,
                               num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                               softmax_scale, workspace, workspace_bytes, dev_status, stream,
                               logit_cap, window, slopes, prefix_lens};
    return pkv::decode_entry<true>(call, pkv::kKvF16);
}

extern "C" pkv_status pkv_paged_decode_scored_int8(
    void *out, const void *query, const int8_t *k_codes, const int8_t *v_codes,
    const float *k_scales, const float *v_scales, int num_blocks,
    const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
    int max_context_len, int num_seqs, int num_heads, int num_kv_heads, int head_dim,
    int block_size, float softmax_scale, float logit_cap, int window, const float *slopes,
    const int32_t *prefix_lens, void *workspace, size_t workspace_bytes, int32_t *dev_status,
    void *stream)
{
    const pkv::DecodeCall call{out, query, k_codes, v_codes, k_scales, v_scales, num_blocks,
                               block_tables, max_blocks_per_seq, context_lens, max_context_len,
                               num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                               softmax_scale, workspace, workspace_bytes, dev_status, stream,
                               logit_cap, window, slopes, prefix_lens};
    return pkv::decode_entry<true>(call, pkv::kKvI8);
}

extern "C" pkv_status pkv_paged_decode_scored_fp8(
    void *out, const void *query, const uint8_t *k_codes, const uint8_t *v_codes,
    const float *k_scales, const float *v_scales, int num_blocks,
    const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
    int max_context_len, int num_seqs, int num_heads, int num_kv_heads, int head_dim,
    int block_size, float softmax_scale, float logit_cap, int window, const float *slopes,
    const int32_t *prefix_lens, void *workspace, size_t workspace_bytes, int32_t *dev_status,
    void *stream)
{
    const pkv::DecodeCall call{out, query, k_codes, v_codes, k_scales, v_scales, num_blocks,
                               block_tables, max_blocks_per_seq, context_lens, max_context_len,
                               num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                               softmax_scale, workspace, workspace_bytes, dev_status, stream,
                               logit_cap, window, slopes, prefix_lens};
    return pkv::decode_entry<true>(call, pkv::kKvF8);
}

#ifdef PKV_DEBUG
// pkv_debug_flags for the kernels of this file.
extern "C" __attribute__((visibility("default"))) unsigned int pkv_debug_scored_flags(int reset)
{
    unsigned int v = 0;
    if (cudaDeviceSynchronize() != cudaSuccess ||
        cudaMemcpyFromSymbol(&v, pkv::g_debug_flags, sizeof(v)) != cudaSuccess)
        return 0xffffffffu;
    if (reset) {
        const unsigned int z = 0;
        if (cudaMemcpyToSymbol(pkv::g_debug_flags, &z, sizeof(z)) != cudaSuccess) return 0xffffffffu;
    }
    return v;
}

// pkv_debug_set_stage_wait_ns for the kernels of this file.
extern "C" __attribute__((visibility("default"))) int pkv_debug_set_scored_stage_wait_ns(
    long long ns)
{
    const unsigned long long v =
        ns < 0 ? pkv::kWaitLimitNs : static_cast<unsigned long long>(ns);
    if (cudaDeviceSynchronize() != cudaSuccess ||
        cudaMemcpyToSymbol(pkv::g_debug_stage_wait_ns, &v, sizeof(v)) != cudaSuccess)
        return -1;
    return 0;
}
#endif
