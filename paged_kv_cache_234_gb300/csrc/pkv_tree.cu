// pkv_tree.cu -- attention of trees of drafted tokens over the paged cache: a
// token sees its sequence's context (window, visible prefix), its ancestors in
// the tree and itself, with the scores of the scored decode (tanh cap, bias by
// distance).
//
// A CTA per (token, query head), a warp per key, running maximum and sum.
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "pkv_host.cuh"
#include "pkv_ptx.cuh"
#include "pkv_ragged.cuh"
#include "pkv_score.cuh"

namespace pkv {
namespace {

constexpr int kPage = 16;
constexpr int kKvF16 = 0, kKvI8 = 1, kKvF8 = 2;
constexpr int kTreeWarps = 8;

struct TreeArgs {
    __half *out;
    const __half *query;
    const void *k_pool, *v_pool;
    const int32_t *block_tables, *query_starts, *context_lens, *parents;
    const float *k_scales, *v_scales;
    const float *slopes;
    const int32_t *prefix_lens;
    int32_t *dev_status;
    int num_tokens, num_seqs, num_heads, num_kv_heads, group;
    int max_blocks_per_seq, num_blocks, ctx_cap, max_tree_len, window;
    float scale_log2, cap, cap_inv;
};

template <int kKv, int kD>
__device__ __forceinline__ void read_row(const void *pool, int64_t row, int lane, float (&x)[kD / 32])
{
#pragma unroll
    for (int c = 0; c < kD / 32; ++c) {
        const int64_t at = row * kD + 32 * c + lane;
        if constexpr (kKv == kKvF16)
            x[c] = __half2float(static_cast<const __half *>(pool)[at]);
        else if constexpr (kKv == kKvI8)
            x[c] = static_cast<float>(static_cast<const int8_t *>(pool)[at]);
        else
            x[c] = static_cast<float>(static_cast<const __nv_fp8_e4m3 *>(pool)[at]);
    }
}

template <int kKv, int kD>
__global__ void __launch_bounds__(32 * kTreeWarps) tree_kernel(const __grid_constant__ TreeArgs p)
{
    constexpr int kC = kD / 32;
    __shared__ float part[kTreeWarps][kD + 2];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int tok = blockIdx.x, head = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (tok == 0 && head == 0 && p.dev_status)
        report_bad_sequences(p.query_starts, p.context_lens, p.num_seqs, p.num_tokens, p.ctx_cap,
                             p.dev_status, threadIdx.x, 32 * kTreeWarps);
    const int seq = warp_search(p.num_seqs, tok, [&](int s) { return __ldg(p.query_starts + s); });
    if (seq < 0) return;
    SeqRows sr;
    sr.load(p.query_starts, p.context_lens, seq, p.num_tokens, p.ctx_cap);
    const int row = tok - sr.start, n = sr.len;
    if (row >= n) return;
    unsigned wrong = sr.ok && n <= p.max_tree_len ? 0u : PKV_DEV_BAD_CTX;
    const int32_t *parents = p.parents + sr.start;
    if (!wrong) {
        int bad = 0;
        for (int j = threadIdx.x; j < n; j += 32 * kTreeWarps) {
            const int q = __ldg(parents + j);
            bad |= q < -1 || q >= j;
        }
        if (__syncthreads_or(bad)) wrong = PKV_DEV_BAD_TREE;
    }
    const int base = sr.ctx - n;
    const int kvh = head / p.group;
    const int64_t at = static_cast<int64_t>(tok) * p.num_heads + head;
    float acc[kC] = {}, m = -INFINITY, l = 0.f;
    if (!wrong) {
        int depth = 0;
        for (int j = __ldg(parents + row); j >= 0; j = __ldg(parents + j)) ++depth;
        const int pos = base + depth;
        const int pre = p.prefix_lens ? min(max(__ldg(p.prefix_lens + seq), 0), base) : 0;
        const float slope = p.slopes ? __ldg(p.slopes + head) * 1.4426950408889634f : 0.f;
        float q[kC];
#pragma unroll
        for (int c = 0; c < kC; ++c) q[c] = __half2float(p.query[at * kD + 32 * c + lane]);
        const int32_t *table = p.block_tables + static_cast<int64_t>(seq) * p.max_blocks_per_seq;
        for (int t = warp; t <= base + row; t += kTreeWarps) {
            int gap = pos - t;
            bool seen = p.window <= 0 || gap < p.window || t < pre;
            if (t >= base) {
                int j = row, up = 0;
                for (; j > t - base; ++up) j = __ldg(parents + j);
                gap = up;
                seen = j == t - base && (p.window <= 0 || gap < p.window);
            }
            if (!seen) continue;
            const int64_t blk = __ldg(table + t / kPage);
            if (blk < 0 || blk >= p.num_blocks) {
                wrong = PKV_DEV_BAD_BLOCK;
                continue;
            }
            const int64_t tile = blk * p.num_kv_heads + kvh;
            float x[kC], z = 0.f;
            read_row<kKv, kD>(p.k_pool, tile * kPage + t % kPage, lane, x);
#pragma unroll
            for (int c = 0; c < kC; ++c) z += q[c] * x[c];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
            z *= p.scale_log2;
            if constexpr (kKv != kKvF16) z *= __ldg(p.k_scales + tile);
            if (p.cap > 0.f) z = cap_score(z, p.cap, p.cap_inv);
            z -= slope * static_cast<float>(gap);
            const float mn = fmaxf(m, z), f = ptx::ex2(m - mn), w = ptx::ex2(z - mn);
            m = mn;
            l = l * f + w;
            read_row<kKv, kD>(p.v_pool, tile * kPage + t % kPage, lane, x);
            float vs = kKv != kKvF16 ? __ldg(p.v_scales + tile) : 1.f;
            if (!(vs >= 0.f && vs < INFINITY)) vs = NAN;
#pragma unroll
            for (int c = 0; c < kC; ++c) acc[c] = acc[c] * f + w * vs * x[c];
        }
    }
#pragma unroll
    for (int c = 0; c < kC; ++c) part[warp][32 * c + lane] = acc[c];
    if (lane == 0) {
        part[warp][kD] = m;
        part[warp][kD + 1] = l;
        if (wrong && p.dev_status) atomicOr(p.dev_status, static_cast<int32_t>(wrong));
    }
    const bool zero = __syncthreads_or(wrong != 0);
    if (threadIdx.x < kD) {
        float top = -INFINITY, sum = 0.f, o = 0.f;
        for (int w = 0; w < kTreeWarps; ++w) top = fmaxf(top, part[w][kD]);
        for (int w = 0; w < kTreeWarps; ++w) {
            const float f = part[w][kD + 1] == 0.f ? 0.f : ptx::ex2(part[w][kD] - top);
            sum += f * part[w][kD + 1];
            o += f * part[w][threadIdx.x];
        }
        p.out[at * kD + threadIdx.x] = __float2half_rn(zero || sum == 0.f ? 0.f : o / sum);
    }
}

// -------------------------------------------------------------------- host
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

struct TreePlan {
    size_t bytes = 0;
};

pkv_status tree_plan(int num_tokens, int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                     int max_context_len, int max_tree_len, TreePlan *plan)
{
    if (num_tokens < 0 || num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
        max_context_len < 0 || max_tree_len < 0 || num_heads % num_kv_heads != 0)
        return PKV_ERR_INVALID_ARG;
    if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
    plan->bytes = 0;
    return PKV_OK;
}

template <int kKv, int kD>
pkv_status launch_tree(const TreeCall &c)
{
    TreeArgs a;
    a.out = static_cast<__half *>(c.out);
    a.query = static_cast<const __half *>(c.query);
    a.k_pool = c.kpool;
    a.v_pool = c.vpool;
    a.block_tables = c.block_tables;
    a.query_starts = c.query_starts;
    a.context_lens = c.context_lens;
    a.parents = c.parents;
    a.k_scales = c.k_scales;
    a.v_scales = c.v_scales;
    a.slopes = c.slopes;
    a.prefix_lens = c.prefix_lens;
    a.dev_status = c.dev_status;
    a.num_tokens = c.num_tokens;
    a.num_seqs = c.num_seqs;
    a.num_heads = c.num_heads;
    a.num_kv_heads = c.num_kv_heads;
    a.group = c.num_heads / c.num_kv_heads;
    a.max_blocks_per_seq = c.max_blocks_per_seq;
    a.num_blocks = c.num_blocks;
    const int64_t cap_tab = static_cast<int64_t>(c.max_blocks_per_seq) * kPage;
    a.ctx_cap = static_cast<int>(c.max_context_len < cap_tab ? c.max_context_len : cap_tab);
    a.max_tree_len = c.max_tree_len;
    a.window = c.window;
    a.scale_log2 = c.softmax_scale * 1.4426950408889634f;
    a.cap = c.logit_cap * 1.4426950408889634f;
    a.cap_inv = c.logit_cap > 0.f ? 1.f / a.cap : 0.f;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(c.num_tokens), static_cast<unsigned>(c.num_heads));
    cfg.blockDim = dim3(32 * kTreeWarps);
    cfg.stream = static_cast<cudaStream_t>(c.stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, tree_kernel<kKv, kD>, a) != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    return PKV_OK;
}

pkv_status tree_entry(const TreeCall &c, int kv)
{
    const bool codes = kv != kKvF16;
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
        c.max_context_len > INT32_MAX - 512 || c.num_heads > 65535)
        return PKV_ERR_UNSUPPORTED;
    if (!aligned(c.out, 16) || !aligned(c.query, 16) || !aligned(c.kpool, 16) ||
        !aligned(c.vpool, 16) || !aligned(c.block_tables, 4) || !aligned(c.query_starts, 4) ||
        !aligned(c.context_lens, 4) || !aligned(c.parents, 4) || !aligned(c.dev_status, 4) ||
        !aligned(c.k_scales, 4) || !aligned(c.v_scales, 4) || !aligned(c.slopes, 4) ||
        !aligned(c.prefix_lens, 4))
        return PKV_ERR_MISALIGNED;
    if (c.num_tokens == 0 || c.num_seqs == 0) return PKV_OK;
    if (plan.bytes > 0 && (!c.workspace || c.workspace_bytes < plan.bytes)) return PKV_ERR_WORKSPACE;
    if (!aligned(c.workspace, 16)) return PKV_ERR_MISALIGNED;
    auto pick = [&](auto kind) -> pkv_status {
        constexpr int kKv = decltype(kind)::value;
        return c.head_dim == 128 ? launch_tree<kKv, 128>(c) : launch_tree<kKv, 64>(c);
    };
    if (kv == kKvF8) return pick(std::integral_constant<int, kKvF8>());
    if (kv == kKvI8) return pick(std::integral_constant<int, kKvI8>());
    return pick(std::integral_constant<int, kKvF16>());
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
    return pkv::tree_entry(c, pkv::kKvF16);
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
    return pkv::tree_entry(c, pkv::kKvI8);
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
    return pkv::tree_entry(c, pkv::kKvF8);
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
