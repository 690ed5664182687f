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
// CTA or a cluster of CTAs -- one page to a warp: a round's rows are fetched into
// shared memory, the team meets at a barrier, the round's pages are written.
// Reading ahead is always safe, so the rows of two rounds are on their way, their
// places found two rounds ahead of that, and a page is written a round after its
// rows came, which leaves the barrier a round to complete in.  No row is read twice.
//
// A moved row is read once and written once; code caches write the codes too.  A
// page's 16 rows of head_dim 128 are 4 KB; a quantized tile's largest magnitude is
// found by shuffles alone, since a tile is a warp's.
//
// Measured: 8 contexts of 16384 tokens to their halves, fp16, 8 kv heads: 93 us, 85 %
// of the copy's rate; one FP8 context of 131072 tokens to three quarters: 300 us, half of it:
// 16 chains keep 128 CTAs of 8 warps busy (16 warps: 348 us, 4: 478), and a page's
// codes take a warp longer than its rows.  Paths of 16 tokens in 64 trees, which
// is a warp's work each: 4.0 us (a launch), INT8 7.8.
#include <cuda_fp16.h>
#include <stdint.h>

#include <mutex>

#include "pkv_host.cuh"
#include "pkv_ptx.cuh"
#include "pkv_quant.cuh"
#include "pkv_ragged.cuh"

namespace pkv {
namespace {

enum { kMoveF16 = 0, kMoveI8 = 1, kMoveF8 = 2 };
constexpr int kMoveWarps = 8;
// Pages of a warp: the last round's, this one's, the next one's.  (Four leave an SM one
// CTA, and 16 clusters of 8 are not all placed at once: 479 against 299 us.)
constexpr int kBufs = 3;

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

// The codes of eight values by y = x * fl(1 / scale), which is within 2 ulp of the
// quotient q = fl(x / scale) that the quantizer rounds.  Returns a bit for every value
// whose y lies so close to the middle M of two codes that q may be M or beyond, or is
// NaN.  INT8: see quant_code.
__device__ __forceinline__ uint32_t near_codes_i8(const uint4 &raw, float rcp, uint2 &codes)
{
    const __half2 *h = reinterpret_cast<const __half2 *>(&raw);
    const uint64_t by = ptx::f32x2(rcp, rcp), magic = ptx::f32x2(kRoundMagic, kRoundMagic);
    const uint64_t back = ptx::f32x2(-kRoundMagic, -kRoundMagic), neg = ptx::f32x2(-1.f, -1.f);
    const float sure = 0.5f - 0.00006103515625f;   // 0.5 - 2^-14
    uint32_t c[4], doubt = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const float2 f = __half22float2(h[w]);
        const uint64_t y = ptx::mul2(ptx::f32x2(f.x, f.y), by);
        const uint64_t t = ptx::add2(y, magic);
        const float2 d = ptx::f32x2_parts(ptx::fma2(ptx::add2(t, back), neg, y));
        if (!(fabsf(d.x) < sure)) doubt |= 1u << 2 * w;
        if (!(fabsf(d.y) < sure)) doubt |= 2u << 2 * w;
        const float2 i = ptx::f32x2_parts(t);
        c[w] = ptx::prmt(__float_as_uint(i.x), __float_as_uint(i.y), 0x0040);
    }
    codes = make_uint2(ptx::prmt(c[0], c[1], 0x5410), ptx::prmt(c[2], c[3], 0x5410));
    return doubt;
}

// FP8: rounding is monotonic, so where the values a little below and above y (1 -+
// 2^-21: more than the 2 ulp) have the same code, q has it.
__device__ __forceinline__ uint32_t near_codes_f8(const uint4 &raw, float rcp, uint2 &codes)
{
    const __half2 *h = reinterpret_cast<const __half2 *>(&raw);
    const float down = 1.f - 0x1p-21f, up = 1.f + 0x1p-21f;
    const uint64_t by = ptx::f32x2(rcp, rcp);
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const float2 f = __half22float2(h[w]);
        const uint64_t y = ptx::mul2(ptx::f32x2(f.x, f.y), by);
        const float2 a = ptx::f32x2_parts(ptx::mul2(y, ptx::f32x2(down, down)));
        const float2 b = ptx::f32x2_parts(ptx::mul2(y, ptx::f32x2(up, up)));
        lo[w] = __nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3);
        hi[w] = __nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3);
    }
    codes = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
    // the bytes that differ, and NaN (0x7f, 0xff): their top bits
    auto tops = [](uint32_t a, uint32_t b) {
        const uint32_t d = a ^ b;
        return (((d & 0x7f7f7f7fu) + 0x7f7f7f7fu) | d | ((a & 0x7f7f7f7fu) + 0x01010101u)) &
               0x80808080u;
    };
    // (bits 7, 15, 23 and 31 to 0 - 3)
    auto four = [](uint32_t t) { return (t >> 7) * 0x00204081u >> 21 & 0xfu; };
    return four(tops(codes.x, hi[0] | hi[1] << 16)) |
           four(tops(codes.y, hi[2] | hi[3] << 16)) << 4;
}

// The codes of the values in doubt (fp16 normal ones hit ties exactly: one of 2000 for
// FP8), without the quotient: with a = |x| and the code L below M, e = a - M scale is
// exact (a multiple of the lowest bit of M scale, and less than 2^12 of them), and q
// is M -- which goes to the even code -- if e is not above half an ulp of M times the
// scale; the ulp below a power of two is half of that above.
// (One after the other: by divisions of all eight values a warp took a microsecond and
// more for every doubt.)
template <int kKind>
__device__ __forceinline__ void settle(const uint4 &raw, float scale, float rcp, uint32_t doubt,
                                       uint2 &codes)
{
#pragma unroll 1
    for (; doubt; doubt &= doubt - 1) {
        const int i = __ffs(doubt) - 1;
        const uint32_t two = i & 4 ? (i & 2 ? raw.w : raw.z) : (i & 2 ? raw.y : raw.x);
        const float x = __half2float(
            __ushort_as_half(static_cast<unsigned short>(i & 1 ? two >> 16 : two & 0xffffu)));
        const float a = fabsf(x), y = a * rcp;
        uint32_t code = 0;
        if (!isnan(y)) {
            uint32_t low;
            float mid;
            if constexpr (kKind == kMoveI8) {
                low = static_cast<uint32_t>(y);
                mid = static_cast<float>(low) + 0.5f;
            } else {
                low = __nv_cvt_float_to_fp8(y * (1.f - 0x1p-21f), __NV_SATFINITE, __NV_E4M3);
                const uint32_t both = ptx::e4m3x2_to_f16x2(low | (low + 1) << 8);
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&both));
                mid = 0.5f * (f.x + f.y);
            }
            const uint32_t bits = __float_as_uint(mid);
            const float e = fmaf(-mid, scale, a);
            const float half = scale * __uint_as_float((bits & 0x7f800000u) - (24u << 23));
            const bool tie = e >= 0.f ? e <= half : -e <= (bits & 0x7fffffu ? half : 0.5f * half);
            code = low + (tie ? low & 1u : e > 0.f);
            if (x < 0.f) code = kKind == kMoveI8 ? -code & 0xffu : code | 0x80u;
        }
        const int at = (i & 3) * 8;
        uint32_t &w = i & 4 ? codes.y : codes.x;
        w = (w & ~(0xffu << at)) | code << at;
    }
}

template <int kD, int kKind, bool kWarp>
__global__ void __launch_bounds__(32 * kMoveWarps)
    compact_kernel(const __grid_constant__ CompactArgs p)
{
    constexpr bool kCodes = kKind != kMoveF16;
    constexpr int kChunks = kD / 8;           // 16-byte chunks of a row
    constexpr int kStep = 32 / kChunks;       // rows of one load of the warp
    constexpr int kLoads = 16 / kStep;        // loads of a page
    constexpr int kPageBytes = 32 * kD;
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

    // A page's rows are found in three steps, a round apart each, so that nobody waits
    // for an index: the kept rows of its 16 slots and its own block; the blocks of the
    // rows; where all that is.  (Every lane its slot, lanes 16 - 31 as 0 - 15.)
    struct Kept {
        int g, i, before, to_blk;
    };
    auto ask = [&](int g) -> Kept {
        Kept a{g, -1, -1, -1};
        if (g >= pages) return a;
        const int j = (page0 + g) * 16 + (lane & 15) - base;
        if (j >= 0 && j < m) {
            a.i = __ldg(kept + j);
            if (j > 0) a.before = __ldg(kept + j - 1);
        }
        a.to_blk = __ldg(table + page0 + g);
        return a;
    };
    struct From {
        int g, from, to_blk, of_blk;
        bool moves;
    };
    auto follow = [&](const Kept &a) -> From {
        From b{a.g, -1, a.to_blk, a.to_blk, false};
        if (a.g >= pages) return b;
        b.from = (page0 + a.g) * 16 + (lane & 15);
        const int j = b.from - base;
        if (j >= 0 && j < m) {
            if (a.i >= j && a.i > a.before && a.i < sr.len) {
                b.from = base + a.i;
                b.moves = a.i != j;
            } else if (lane < 16) {
                report(PKV_DEV_BAD_KEEP);
            }
        }
        if (b.moves) b.of_blk = __ldg(table + (b.from >> 4));
        return b;
    };
    // For lane < 16 the row of the pool that slot `lane` gets (-1: none), which rows
    // move, and the page's tile.
    struct Found {
        int64_t row, tile;
        unsigned moved;
    };
    auto find = [&](const From &b) -> Found {
        Found f{-1, -1, 0};
        if (b.g >= pages) return f;
        const bool to_ok = b.to_blk >= 0 && b.to_blk < p.num_blocks;
        const bool of_ok = b.of_blk >= 0 && b.of_blk < p.num_blocks;
        bool moves = b.moves;
        if (moves && !(to_ok && of_ok)) {
            if (lane < 16) report(PKV_DEV_BAD_BLOCK);
            moves = false;
        }
        f.moved = __ballot_sync(0xffffffffu, moves) & 0xffffu;
        if (!to_ok) return f;
        f.tile = static_cast<int64_t>(b.to_blk) * p.num_kv_heads + h;
        f.row = moves ? (static_cast<int64_t>(b.of_blk) * p.num_kv_heads + h) * 16 + (b.from & 15)
                      : f.tile * 16 + (lane & 15);
        return f;
    };
    const int c = lane % kChunks, r0 = lane / kChunks;
    // Rows on their way to the warp's buffers: chunk lane + 32 e of a page by this lane,
    // which is the one that reads it again.
    extern __shared__ __align__(16) uint8_t smem[];
    const uint32_t buffers = ptx::smem_addr(smem) + warp * (kBufs * kPageBytes) + lane * 16;
    auto load = [&](const Found &f, int buf) {
        if (f.moved) {
            const uint32_t to = buffers + buf * kPageBytes;
#pragma unroll
            for (int e = 0; e < kLoads; ++e) {
                const int r = r0 + kStep * e;
                const int64_t row = __shfl_sync(0xffffffffu, f.row, r);
                // (a code tile's other rows are quantized with the moved ones)
                if (kCodes || (f.moved >> r & 1u))
                    ptx::cp_async_16(to + 512 * e, pool + row * kChunks + c);
            }
        }
        ptx::cp_async_commit();
    };
    // Codes and scale of a page.  Nobody reads them here: they need not wait for the team.
    auto quantize = [&](const Found &f, uint32_t from) {
        __half2 top = __float2half2_rn(0.f);   // (NaN left out, as the quantizer does)
#pragma unroll
        for (int e = 0; e < kLoads; ++e) {
            const uint4 v = ptx::lds128(from + 512 * e);
            const __half2 *x = reinterpret_cast<const __half2 *>(&v);
#pragma unroll
            for (int w = 0; w < 4; ++w) top = __hmax2(top, __habs2(x[w]));
        }
        float amax = fmaxf(__low2float(top), __high2float(top));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const float scale = __fdiv_rn(amax, kKind == kMoveF8 ? 448.0f : 127.0f);
        const float rcp = __frcp_rn(scale);
        uint2 *codes =
            reinterpret_cast<uint2 *>(is_v ? p.v_codes : p.k_codes) + f.tile * (16 * kChunks) + lane;
        // (paths of 64 trees over INT8: 7.8 us, 8.2 rolled, 10 and more with the tile in
        // registers and all unrolled, when the warps waited for instructions)
#pragma unroll 2
        for (int e = 0; e < kLoads; ++e) {
            const uint4 v = ptx::lds128(from + 512 * e);
            uint2 w;
            const uint32_t doubt =
                kKind == kMoveF8 ? near_codes_f8(v, rcp, w) : near_codes_i8(v, rcp, w);
            if (doubt) settle<kKind>(v, scale, rcp, doubt, w);
            codes[32 * e] = w;
        }
        if (lane == 0) (is_v ? p.v_scales : p.k_scales)[f.tile] = scale;
    };
    auto store = [&](const Found &f, uint32_t from) {
        uint4 *dst = pool + f.tile * (16 * kChunks) + lane;
#pragma unroll
        for (int e = 0; e < kLoads; ++e)
            if (f.moved >> (r0 + kStep * e) & 1u) dst[32 * e] = ptx::lds128(from + 512 * e);
    };

    // f[0]: this round's page, then those whose rows are on their way
    constexpr int kAhead = kBufs - 1;
    Found f[kAhead];
    {
        Kept a[kAhead];
        From b[kAhead];
#pragma unroll
        for (int q = 0; q < kAhead; ++q) a[q] = ask(rank + q * team);
#pragma unroll
        for (int q = 0; q < kAhead; ++q) b[q] = follow(a[q]);
#pragma unroll
        for (int q = 0; q < kAhead; ++q) load(f[q] = find(b[q]), q);
    }
    From from = follow(ask(rank + kAhead * team));
    Kept asked = ask(rank + (kAhead + 1) * team);
    // Round k: its rows are there; the rows of round k - 1 are written, for which the
    // team has met; its codes, which need not wait.  So a meeting has a round's work to
    // hide behind, and so have the writes that it makes visible.
    Found before{-1, -1, 0};
    int buf = 0;
    for (int g = rank; g - rank < pages; g += team) {
        const int free = buf == 0 ? kBufs - 1 : buf - 1;
        ptx::cp_async_wait<kAhead - 1>();
        team_arrive<kWarp>();
        if (before.moved) store(before, buffers + free * kPageBytes);
        const Found later = find(from);
        load(later, free);
        from = follow(asked);
        asked = ask(g + (kAhead + 2) * team);
        if (kCodes && f[0].moved) quantize(f[0], buffers + buf * kPageBytes);
        team_wait<kWarp>();
        before = f[0];
#pragma unroll
        for (int q = 0; q + 1 < kAhead; ++q) f[q] = f[q + 1];
        f[kAhead - 1] = later;
        buf = buf == kBufs - 1 ? 0 : buf + 1;
    }
    if (before.moved) store(before, buffers + (buf == 0 ? kBufs - 1 : buf - 1) * kPageBytes);
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
    cfg.dynamicSmemBytes = kMoveWarps * kBufs * 32 * kD;
    cfg.stream = static_cast<cudaStream_t>(c.stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    const auto kern = pages <= 4 ? compact_kernel<kD, kKind, true> : compact_kernel<kD, kKind, false>;
    DeviceInfo di;
    if (!current_device_info(&di)) return PKV_ERR_CUDA;
    {
        static bool ready[2][64] = {};
        std::lock_guard<std::mutex> lock(g_cfg_mu);
        bool &r = ready[pages <= 4][di.device & 63];
        if (!r) {
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     static_cast<int>(cfg.dynamicSmemBytes)) != cudaSuccess) {
                cudaGetLastError();
                return PKV_ERR_CUDA;
            }
            r = true;
        }
    }
    cudaError_t e;
    if (pages <= 4) {
        const int64_t grid = (a.chains + kMoveWarps - 1) / kMoveWarps;
        if (grid > INT32_MAX) return PKV_ERR_UNSUPPORTED;
        cfg.gridDim = dim3(static_cast<unsigned>(grid));
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, kern, a);
    } else {
        // CTAs until there is one for every SM (until there are two: the halves of 8
        // contexts of 16384 in 94.8 against 93.0 us)
        int ctas = 1;
        while (ctas < 8 && ctas * kMoveWarps < pages && a.chains * ctas < 152) ctas *= 2;
        if (a.chains * ctas > INT32_MAX) return PKV_ERR_UNSUPPORTED;
        cfg.gridDim = dim3(static_cast<unsigned>(a.chains * ctas));
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = static_cast<unsigned>(ctas);
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
        e = cudaLaunchKernelEx(&cfg, kern, a);
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    return PKV_OK;
}

// Whether two arrays of so many int32 have one in common.
bool overlap(const void *a, int64_t na, const void *b, int64_t nb)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && na > 0 && nb > 0 && x < y + 4 * static_cast<uintptr_t>(nb) &&
           y < x + 4 * static_cast<uintptr_t>(na);
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
    if (c.block_size != 16 || (c.head_dim != 64 && c.head_dim != 128)) return PKV_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(c.max_blocks_per_seq) * 16 > INT32_MAX) return PKV_ERR_UNSUPPORTED;
    if (!aligned(c.k_cache, 16) || !aligned(c.v_cache, 16) || !aligned(c.k_codes, 16) ||
        !aligned(c.v_codes, 16) || !aligned(c.k_scales, 4) || !aligned(c.v_scales, 4) ||
        !aligned(c.kept, 4) || !aligned(c.kept_lens, 4) || !aligned(c.new_context_lens, 4) ||
        !aligned(c.query_starts, 4) || !aligned(c.context_lens, 4) ||
        !aligned(c.block_tables, 4) || !aligned(c.dev_status, 4))
        return PKV_ERR_MISALIGNED;
    // The lengths are written while other warps read the call's arrays: with a sequence
    // that changes under them the warps of a cluster would not meet equally often.
    const int64_t n = c.num_seqs;
    if (overlap(c.new_context_lens, n, c.context_lens, n) ||
        overlap(c.new_context_lens, n, c.kept_lens, n) ||
        overlap(c.new_context_lens, n, c.query_starts, n + 1) ||
        overlap(c.new_context_lens, n, c.kept, c.num_tokens) ||
        overlap(c.new_context_lens, n, c.block_tables, n * c.max_blocks_per_seq))
        return PKV_ERR_INVALID_ARG;
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
