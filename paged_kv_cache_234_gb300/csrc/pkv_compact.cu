// pkv_compact.cu -- the cached rows that stay, moved together in place: position
// base + j of a sequence gets the row of position base + kept[j], where kept
// rises (the accepted path of a tree of drafted tokens, or what is left of a
// whole context).  For INT8 / FP8 caches every tile that got a row is quantized
// again, as the quantizer does (pkv_quant.cuh).
//
// In place: kept[j] >= j, so a row moves towards the front, and target page p
// takes its rows from pages >= p.  A page may be written as soon as every row
// that lies in it has been read, and those go to pages <= p.  The pages of one
// (sequence, kv head, K | V) are therefore taken in rounds by a team -- a warp, a
// CTA or a cluster of CTAs -- one page to a warp: a round's rows are read into
// registers, the team meets at a barrier, the round's pages are written.  Reading
// ahead is always safe, so the next round's rows are on their way before this
// one's are written.  No row is read twice and nothing is kept in memory.
//
// Bound by memory: a moved row is read once and written once; code caches write
// the codes too.  A page's 16 rows of head_dim 128 are 4 KB, eight 16-byte loads
// of a lane in flight, and a quantized tile's largest magnitude is found by
// shuffles alone, since a tile is a warp's.
#include <cuda_fp16.h>
#include <stdint.h>

#include "pkv_host.cuh"
#include "pkv_ptx.cuh"
#include "pkv_quant.cuh"
#include "pkv_ragged.cuh"

namespace pkv {
namespace {

enum { kMoveF16 = 0, kMoveI8 = 1, kMoveF8 = 2 };
constexpr int kMoveWarps = 8;

struct CompactArgs {
    __half *k_pool, *v_pool;
    uint8_t *k_codes, *v_codes;
    float *k_scales, *v_scales;
    const int32_t *kept, *kept_lens, *query_starts, *context_lens, *block_tables;
    int32_t *new_context_lens;
    int32_t *dev_status;
    int max_blocks_per_seq, num_tokens, num_seqs, num_kv_heads, num_blocks;
    int64_t chains;   // num_seqs * num_kv_heads * 2
};

// Barriers of a team.  arrive() is behind the reads of a round, wait() ahead of
// its writes.
template <bool kWarp>
__device__ __forceinline__ void team_arrive()
{
    if constexpr (kWarp)
        __syncwarp();
    else
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}

template <bool kWarp>
__device__ __forceinline__ void team_wait()
{
    if constexpr (!kWarp) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int kD, int kKind, bool kWarp>
__global__ void __launch_bounds__(32 * kMoveWarps)
    compact_kernel(const __grid_constant__ CompactArgs p)
{
    constexpr bool kCodes = kKind != kMoveF16;
    constexpr int kChunks = kD / 8;           // 16-byte chunks of a row
    constexpr int kStep = 32 / kChunks;       // rows of one load of the warp
    constexpr int kLoads = 16 / kStep;        // loads of a page
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int team = 1, rank = 0;                   // warps of the team, this one's number
    int64_t chain;
    if constexpr (kWarp) {
        chain = static_cast<int64_t>(blockIdx.x) * kMoveWarps + warp;
        if (chain >= p.chains) return;
    } else {
        const int ctas = static_cast<int>(ptx::cluster_nctarank());
        team = ctas * kMoveWarps;
        rank = static_cast<int>(ptx::cluster_ctarank()) * kMoveWarps + warp;
        chain = blockIdx.x / ctas;
    }
    const bool is_v = chain & 1;
    const int64_t sh = chain >> 1;
    const int seq = static_cast<int>(sh / p.num_kv_heads);
    const int h = static_cast<int>(sh - static_cast<int64_t>(seq) * p.num_kv_heads);
    const bool first = rank == 0 && lane == 0 && h == 0 && !is_v;
    const int row0 = __ldg(p.query_starts + seq), row1 = __ldg(p.query_starts + seq + 1);
    const int m = __ldg(p.kept_lens + seq);
    SeqRows sr;
    sr.set(row0, row1, __ldg(p.context_lens + seq), p.num_tokens, p.max_blocks_per_seq * 16);
    unsigned wrong = 0;
    if (!sr.ok && row0 != row1) wrong = PKV_DEV_BAD_CTX;
    if (!wrong && (m < 0 || m > sr.len)) wrong = PKV_DEV_BAD_KEEP;
    if (first) {
        if (p.new_context_lens)
            p.new_context_lens[seq] = wrong || sr.len == 0 ? sr.ctx : sr.ctx - sr.len + m;
        if (wrong && p.dev_status) atomicOr(p.dev_status, static_cast<int32_t>(wrong));
    }
    if (wrong || m == 0) return;              // (the same for the whole team)
    const int base = sr.ctx - sr.len;
    const int32_t *table = p.block_tables + static_cast<int64_t>(seq) * p.max_blocks_per_seq;
    const int32_t *kept = p.kept + sr.start;
    uint4 *pool = reinterpret_cast<uint4 *>(is_v ? p.v_pool : p.k_pool);
    const int page0 = base >> 4, pages = ((base + m - 1) >> 4) - page0 + 1;
    auto report = [&](unsigned bit) {
        if (p.dev_status) atomicOr(p.dev_status, static_cast<int32_t>(bit));
    };

    // A page's rows, found: for lane < 16 the row of the pool that slot `lane`
    // gets (-1: none), whether some row moves and which, and the page's tile.
    struct Found {
        int64_t row, tile;
        unsigned moved;
    };
    auto find = [&](int g) -> Found {
        Found f{-1, -1, 0};
        if (g >= pages) return f;
        const int page = page0 + g, pos = page * 16 + (lane & 15), j = pos - base;
        int from = pos;
        bool moves = false;
        if (j >= 0 && j < m) {
            const int i = __ldg(kept + j), before = j > 0 ? __ldg(kept + j - 1) : -1;
            if (i >= j && i > before && i < sr.len) {
                from = base + i;
                moves = i != j;
            } else if (lane < 16) {
                report(PKV_DEV_BAD_KEEP);
            }
        }
        const int to_blk = __ldg(table + page);
        const int of_blk = moves ? __ldg(table + (from >> 4)) : to_blk;
        const bool to_ok = to_blk >= 0 && to_blk < p.num_blocks;
        const bool of_ok = of_blk >= 0 && of_blk < p.num_blocks;
        if (moves && !(to_ok && of_ok)) {
            if (lane < 16) report(PKV_DEV_BAD_BLOCK);
            moves = false;
            from = pos;
        }
        f.moved = __ballot_sync(0xffffffffu, moves) & 0xffffu;
        if (!to_ok) return f;
        f.tile = static_cast<int64_t>(to_blk) * p.num_kv_heads + h;
        f.row = moves ? (static_cast<int64_t>(of_blk) * p.num_kv_heads + h) * 16 + (from & 15)
                      : f.tile * 16 + (pos & 15);
        return f;
    };
    const int c = lane % kChunks, r0 = lane / kChunks;
    auto load = [&](const Found &f, uint4 (&x)[kLoads]) {
        if (!f.moved) return;
#pragma unroll
        for (int e = 0; e < kLoads; ++e) {
            const int r = r0 + kStep * e;
            const int64_t row = __shfl_sync(0xffffffffu, f.row, r);
            // (a code tile's other rows are quantized with the moved ones)
            if (kCodes || (f.moved >> r & 1u)) x[e] = pool[row * kChunks + c];
        }
    };
    auto store = [&](const Found &f, const uint4 (&x)[kLoads]) {
        if (!f.moved) return;
        uint4 *dst = pool + f.tile * (16 * kChunks);
#pragma unroll
        for (int e = 0; e < kLoads; ++e)
            if (f.moved >> (r0 + kStep * e) & 1u) dst[lane + 32 * e] = x[e];
        if constexpr (kCodes) {
            float amax = chunks_absmax(x);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            const float scale = __fdiv_rn(amax, kKind == kMoveF8 ? 448.0f : 127.0f);
            const float rcp = __frcp_rn(scale);
            uint2 *codes = reinterpret_cast<uint2 *>(is_v ? p.v_codes : p.k_codes) +
                           f.tile * (16 * kChunks);
#pragma unroll
            for (int e = 0; e < kLoads; ++e)
                codes[lane + 32 * e] = kKind == kMoveF8 ? chunk_codes_fp8(x[e], scale)
                                                        : chunk_codes(x[e], scale, rcp);
            if (lane == 0) (is_v ? p.v_scales : p.k_scales)[f.tile] = scale;
        }
    };

    uint4 x[kLoads], y[kLoads];
    Found f = find(rank);
    load(f, x);
    for (int g = rank; g - rank < pages; g += team) {
        const Found next = find(g + team);
        team_arrive<kWarp>();
        load(next, y);
        team_wait<kWarp>();
        store(f, x);
        f = next;
#pragma unroll
        for (int e = 0; e < kLoads; ++e) x[e] = y[e];
    }
}

struct CompactCall {
    void *k_cache, *v_cache, *k_codes, *v_codes;
    float *k_scales, *v_scales;
    int num_blocks;
    const int32_t *kept, *kept_lens;
    int32_t *new_context_lens;
    const int32_t *query_starts, *context_lens, *block_tables;
    int max_blocks_per_seq, num_tokens, num_seqs, num_kv_heads, head_dim, block_size;
    int32_t *dev_status;
    void *stream;
};

template <int kD, int kKind>
pkv_status launch_compact(const CompactCall &c, const CompactArgs &a)
{
    // pages of a sequence's rows on average, and one more for the rounding
    const int64_t pages = c.num_tokens / c.num_seqs / 16 + 2;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(32 * kMoveWarps);
    cfg.stream = static_cast<cudaStream_t>(c.stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cudaError_t e;
    if (pages <= 4) {
        const int64_t grid = (a.chains + kMoveWarps - 1) / kMoveWarps;
        if (grid > INT32_MAX) return PKV_ERR_UNSUPPORTED;
        cfg.gridDim = dim3(static_cast<unsigned>(grid));
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, compact_kernel<kD, kKind, true>, a);
    } else {
        int ctas = 1;
        while (ctas < 8 && ctas * kMoveWarps < pages && a.chains * ctas < 2 * 152) ctas *= 2;
        if (a.chains * ctas > INT32_MAX) return PKV_ERR_UNSUPPORTED;
        cfg.gridDim = dim3(static_cast<unsigned>(a.chains * ctas));
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = static_cast<unsigned>(ctas);
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
        e = cudaLaunchKernelEx(&cfg, compact_kernel<kD, kKind, false>, a);
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    return PKV_OK;
}

pkv_status compact_entry(const CompactCall &c, int kind)
{
    if (!c.k_cache || !c.v_cache || !c.query_starts) return PKV_ERR_INVALID_ARG;
    // (arrays without elements may be null)
    if (c.num_tokens != 0 && !c.kept) return PKV_ERR_INVALID_ARG;
    if (c.num_seqs != 0 && (!c.kept_lens || !c.context_lens)) return PKV_ERR_INVALID_ARG;
    if (kind != kMoveF16 && (!c.k_codes || !c.v_codes || !c.k_scales || !c.v_scales))
        return PKV_ERR_INVALID_ARG;
    if (c.num_blocks <= 0 || c.max_blocks_per_seq < 0 || c.num_tokens < 0 || c.num_seqs < 0 ||
        c.num_kv_heads <= 0 || c.head_dim <= 0 || c.block_size <= 0)
        return PKV_ERR_INVALID_ARG;
    if (!c.block_tables && c.max_blocks_per_seq > 0 && c.num_seqs > 0) return PKV_ERR_INVALID_ARG;
    if (c.new_context_lens && c.new_context_lens == c.context_lens) return PKV_ERR_INVALID_ARG;
    if (c.block_size != 16 || (c.head_dim != 64 && c.head_dim != 128)) return PKV_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(c.max_blocks_per_seq) * 16 > INT32_MAX) return PKV_ERR_UNSUPPORTED;
    if (!aligned(c.k_cache, 16) || !aligned(c.v_cache, 16) || !aligned(c.k_codes, 16) ||
        !aligned(c.v_codes, 16) || !aligned(c.k_scales, 4) || !aligned(c.v_scales, 4) ||
        !aligned(c.kept, 4) || !aligned(c.kept_lens, 4) || !aligned(c.new_context_lens, 4) ||
        !aligned(c.query_starts, 4) || !aligned(c.context_lens, 4) ||
        !aligned(c.block_tables, 4) || !aligned(c.dev_status, 4))
        return PKV_ERR_MISALIGNED;
    if (c.num_seqs == 0) return PKV_OK;
    CompactArgs a;
    a.k_pool = static_cast<__half *>(c.k_cache);
    a.v_pool = static_cast<__half *>(c.v_cache);
    a.k_codes = static_cast<uint8_t *>(c.k_codes);
    a.v_codes = static_cast<uint8_t *>(c.v_codes);
    a.k_scales = c.k_scales;
    a.v_scales = c.v_scales;
    a.kept = c.kept;
    a.kept_lens = c.kept_lens;
    a.query_starts = c.query_starts;
    a.context_lens = c.context_lens;
    a.block_tables = c.block_tables;
    a.new_context_lens = c.new_context_lens;
    a.dev_status = c.dev_status;
    a.max_blocks_per_seq = c.max_blocks_per_seq;
    a.num_tokens = c.num_tokens;
    a.num_seqs = c.num_seqs;
    a.num_kv_heads = c.num_kv_heads;
    a.num_blocks = c.num_blocks;
    a.chains = static_cast<int64_t>(c.num_seqs) * c.num_kv_heads * 2;
    if (c.head_dim == 128)
        return kind == kMoveF8   ? launch_compact<128, kMoveF8>(c, a)
               : kind == kMoveI8 ? launch_compact<128, kMoveI8>(c, a)
                                 : launch_compact<128, kMoveF16>(c, a);
    return kind == kMoveF8   ? launch_compact<64, kMoveF8>(c, a)
           : kind == kMoveI8 ? launch_compact<64, kMoveI8>(c, a)
                             : launch_compact<64, kMoveF16>(c, a);
}

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_compact_fp16(void *k_cache, void *v_cache, int num_blocks,
                                       const int32_t *kept, const int32_t *kept_lens,
                                       int32_t *new_context_lens, const int32_t *query_starts,
                                       const int32_t *context_lens, const int32_t *block_tables,
                                       int max_blocks_per_seq, int num_tokens, int num_seqs,
                                       int num_kv_heads, int head_dim, int block_size,
                                       int32_t *dev_status, void *stream)
{
    const pkv::CompactCall c{k_cache, v_cache, nullptr, nullptr, nullptr, nullptr, num_blocks, kept,
                             kept_lens, new_context_lens, query_starts, context_lens,
                             block_tables, max_blocks_per_seq, num_tokens, num_seqs,
                             num_kv_heads, head_dim, block_size, dev_status, stream};
    return pkv::compact_entry(c, pkv::kMoveF16);
}

extern "C" pkv_status pkv_compact_int8(void *k_cache, void *v_cache, int8_t *k_codes,
                                       int8_t *v_codes, float *k_scales, float *v_scales,
                                       int num_blocks, const int32_t *kept,
                                       const int32_t *kept_lens, int32_t *new_context_lens,
                                       const int32_t *query_starts, const int32_t *context_lens,
                                       const int32_t *block_tables, int max_blocks_per_seq,
                                       int num_tokens, int num_seqs, int num_kv_heads,
                                       int head_dim, int block_size, int32_t *dev_status,
                                       void *stream)
{
    const pkv::CompactCall c{k_cache, v_cache, k_codes, v_codes, k_scales, v_scales, num_blocks,
                             kept, kept_lens, new_context_lens, query_starts, context_lens,
                             block_tables, max_blocks_per_seq, num_tokens, num_seqs,
                             num_kv_heads, head_dim, block_size, dev_status, stream};
    return pkv::compact_entry(c, pkv::kMoveI8);
}

extern "C" pkv_status pkv_compact_fp8(void *k_cache, void *v_cache, uint8_t *k_codes,
                                      uint8_t *v_codes, float *k_scales, float *v_scales,
                                      int num_blocks, const int32_t *kept,
                                      const int32_t *kept_lens, int32_t *new_context_lens,
                                      const int32_t *query_starts, const int32_t *context_lens,
                                      const int32_t *block_tables, int max_blocks_per_seq,
                                      int num_tokens, int num_seqs, int num_kv_heads,
                                      int head_dim, int block_size, int32_t *dev_status,
                                      void *stream)
{
    const pkv::CompactCall c{k_cache, v_cache, k_codes, v_codes, k_scales, v_scales, num_blocks,
                             kept, kept_lens, new_context_lens, query_starts, context_lens,
                             block_tables, max_blocks_per_seq, num_tokens, num_seqs,
                             num_kv_heads, head_dim, block_size, dev_status, stream};
    return pkv::compact_entry(c, pkv::kMoveF8);
}
