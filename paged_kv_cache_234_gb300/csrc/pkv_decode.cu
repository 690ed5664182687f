// pkv_decode.cu -- the decode entry points (pkv_decode.cuh holds the kernels),
// the workspace size and the worker cap, and the decode without allocation.
#include "pkv_decode.cuh"

extern "C" pkv_status pkv_paged_decode_fp16(float *out, const void *query, const void *k_cache,
                                            const void *v_cache, int num_blocks,
                                            const int32_t *block_tables, int max_blocks_per_seq,
                                            const int32_t *context_lens, int max_context_len,
                                            int num_seqs, int num_heads, int num_kv_heads,
                                            int head_dim, int block_size, float softmax_scale,
                                            void *workspace, size_t workspace_bytes,
                                            int32_t *dev_status, void *stream)
{
    const pkv::DecodeCall call{out, query, k_cache, v_cache, nullptr, nullptr, num_blocks,
                               block_tables, max_blocks_per_seq, context_lens, max_context_len,
                               num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                               softmax_scale, workspace, workspace_bytes, dev_status, stream};
    return pkv::decode_entry<false>(call, pkv::kKvF16);
}

extern "C" pkv_status pkv_paged_decode_int8(float *out, const void *query, const int8_t *k_codes,
                                            const int8_t *v_codes, const float *k_scales,
                                            const float *v_scales, int num_blocks,
                                            const int32_t *block_tables, int max_blocks_per_seq,
                                            const int32_t *context_lens, int max_context_len,
                                            int num_seqs, int num_heads, int num_kv_heads,
                                            int head_dim, int block_size, float softmax_scale,
                                            void *workspace, size_t workspace_bytes,
                                            int32_t *dev_status, void *stream)
{
    const pkv::DecodeCall call{out, query, k_codes, v_codes, k_scales, v_scales, num_blocks,
                               block_tables, max_blocks_per_seq, context_lens, max_context_len,
                               num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                               softmax_scale, workspace, workspace_bytes, dev_status, stream};
    return pkv::decode_entry<false>(call, pkv::kKvI8);
}

extern "C" pkv_status pkv_paged_decode_fp8(float *out, const void *query, const uint8_t *k_codes,
                                           const uint8_t *v_codes, const float *k_scales,
                                           const float *v_scales, int num_blocks,
                                           const int32_t *block_tables, int max_blocks_per_seq,
                                           const int32_t *context_lens, int max_context_len,
                                           int num_seqs, int num_heads, int num_kv_heads,
                                           int head_dim, int block_size, float softmax_scale,
                                           void *workspace, size_t workspace_bytes,
                                           int32_t *dev_status, void *stream)
{
    const pkv::DecodeCall call{out, query, k_codes, v_codes, k_scales, v_scales, num_blocks,
                               block_tables, max_blocks_per_seq, context_lens, max_context_len,
                               num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                               softmax_scale, workspace, workspace_bytes, dev_status, stream};
    return pkv::decode_entry<false>(call, pkv::kKvF8);
}

extern "C" size_t pkv_decode_workspace_size(int num_seqs, int num_heads, int num_kv_heads,
                                            int head_dim, int max_context_len)
{
    pkv::Shape sh;
    // the block table can hold any context up to max_context_len here
    const int mbps = (max_context_len + 15) / 16;
    if (pkv::check_shape(num_seqs, num_heads, num_kv_heads, head_dim, max_context_len, mbps,
                         &sh) != PKV_OK)
        return 0;
    return pkv::workspace_bytes_for(sh, head_dim);
}

extern "C" pkv_status pkv_set_decode_workers(int max_workers)
{
    if (max_workers < 0) return PKV_ERR_INVALID_ARG;
    std::lock_guard<std::mutex> lock(pkv::g_cfg_mu);
    pkv::g_worker_cap = max_workers;
    return PKV_OK;
}

// ------------------------------------------------- decode without allocation
// Scratch for pkv_paged_decode_int8_static_workspace: a fixed device array
// that every GPU loading this library holds until the process exits.  Only
// the partial records and split descriptors of the decode live here; they are
// fully rewritten by every call before they are read, so nothing needs to
// start at zero.  Host code must not pass `g_static_ws` itself to a kernel:
// on the host that name is a stand-in, not a device address.
static __device__ __align__(256) unsigned char g_static_ws[PKV_STATIC_WORKSPACE_BYTES];

namespace pkv {
namespace {
std::mutex g_static_mu;
void *g_static_ptr[64] = {};  // device address of g_static_ws, per device
}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_paged_decode_int8_static_workspace(
    float *out, const void *query, const int8_t *k_codes, const int8_t *v_codes,
    const float *k_scales, const float *v_scales, int num_blocks, const int32_t *block_tables,
    int max_blocks_per_seq, const int32_t *context_lens, int max_context_len, int num_seqs,
    int num_heads, int num_kv_heads, int head_dim, int block_size, float softmax_scale,
    int32_t *dev_status, void *stream)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PKV_ERR_CUDA;
    void *ws = nullptr;
    {
        // set-up, once per device, with that device current
        std::lock_guard<std::mutex> lock(pkv::g_static_mu);
        if (!pkv::g_static_ptr[dev]) {
            void *ptr = nullptr;
            if (cudaGetSymbolAddress(&ptr, g_static_ws) != cudaSuccess || !ptr) {
                cudaGetLastError();
                return PKV_ERR_CUDA;
            }
            pkv::g_static_ptr[dev] = ptr;
        }
        ws = pkv::g_static_ptr[dev];
    }
    const pkv::DecodeCall call{out, query, k_codes, v_codes, k_scales, v_scales, num_blocks,
                               block_tables, max_blocks_per_seq, context_lens, max_context_len,
                               num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                               softmax_scale, ws, PKV_STATIC_WORKSPACE_BYTES, dev_status, stream};
    // a call needing more than PKV_STATIC_WORKSPACE_BYTES of scratch is
    // rejected with PKV_ERR_WORKSPACE before anything is launched
    return pkv::decode_entry<false>(call, pkv::kKvI8);
}

#ifdef PKV_DEBUG
// Debug builds only (not part of the C ABI header): the OR of the check bits
// set since the last reset (1: a shared-memory address outside the dynamic
// shared memory, 2: a misaligned one, 4: a table index out of range); reset
// nonzero clears them.  Synchronises with the device.
extern "C" __attribute__((visibility("default"))) unsigned int pkv_debug_flags(int reset)
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

// Debug builds only: the limit of the decode kernel's waits for a stage, in
// ns, on the current device (0: a wait gives up at once, as if its limit had
// run out, while its copies are still in flight; the drain that follows a
// timeout keeps its 1 s limit).  Negative restores the default of 1 s.  Synchronises with the
// device; returns 0, or -1 if the CUDA runtime fails.
extern "C" __attribute__((visibility("default"))) int pkv_debug_set_stage_wait_ns(long long ns)
{
    const unsigned long long v =
        ns < 0 ? pkv::kWaitLimitNs : static_cast<unsigned long long>(ns);
    if (cudaDeviceSynchronize() != cudaSuccess ||
        cudaMemcpyToSymbol(pkv::g_debug_stage_wait_ns, &v, sizeof(v)) != cudaSuccess)
        return -1;
    return 0;
}
#endif
