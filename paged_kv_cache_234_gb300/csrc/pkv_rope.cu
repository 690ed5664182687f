// pkv_rope.cu -- rotary positions applied to a ragged batch of new tokens on
// the way into the paged cache: the queries are rotated into q_out, the keys
// are rotated and written to their slots together with the values, and for
// INT8 / FP8 caches every tile that received a row is quantized again.
//
// With pair i of a head (values a = x[lo(i)], b = x[hi(i)]; lo, hi = i, i +
// rot/2, or 2i, 2i + 1 where neighbours are paired) and the table row of the
// position p that the pair's axis gives the token:
//   a' = a cos(p, i) - b sin(p, i),   b' = b cos(p, i) + a sin(p, i)
// in fp32, each product and each sum rounded, then once to fp16.  No fused
// multiply-add: the result does not depend on how a compiler contracts the
// expression, so the codes of a quantized cache can be reproduced bit for bit
// from elementary array operations.  For the same reason a tile's scale is
// amax times the fp32 reciprocal of the largest code: that is what an array
// library's division by a constant computes on a GPU.  (The other quantizers
// of this library divide; the two differ by 2^-23 at most.)
//
// Bound by memory: (Hq + 2 Hkv) d fp16 values in and out per token, next to
// which the table row (4 rot bytes, read once per token and head row from L1)
// and the fp32 arithmetic are small.  A thread owns one slot of a row, the 16
// values whose partners lie in the same two 16-byte chunks, so every load and
// store is 16 bytes wide and the cosines of its eight pairs are loaded once
// per token and serve every head.  Measured on GB300, 32 / 8 heads, head_dim
// 128: 65536 tokens, fp16 cache 238 us (1.02 of the floor by the copy rate); an
// INT8 chunk 50 us (0.73).
#include <cuda_fp16.h>
#include <stdint.h>

#include "pkv_host.cuh"
#include "pkv_ptx.cuh"
#include "pkv_quant.cuh"
#include "pkv_ragged.cuh"

namespace pkv {
namespace {

constexpr int kMaxPairs = 64;   // head_dim / 2
constexpr int kRowThreads = 128;

struct RopeArgs {
    __half *q_out, *k_pool, *v_pool;
    uint8_t *k_codes, *v_codes;
    float *k_scales, *v_scales;
    const __half *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;  // values from one token to the next
    const float *cos_sin;                  // [max_position][rot]: cosines, sines
    const int32_t *rope_positions;         // [axes][num_tokens] or null
    const int32_t *query_starts, *context_lens, *block_tables;
    int32_t *dev_status;
    int max_position, rot, interleaved, axes;
    int max_blocks_per_seq, num_tokens, num_seqs, num_heads, num_kv_heads, num_blocks;
    int units;                             // page units of the batch (code caches)
    int tokens_per_cta;                    // of rope_tokens
    unsigned check_from;                   // first CTA of check_sequences
    uint8_t axis_of_pair[kMaxPairs];
};

__device__ __forceinline__ void report(const RopeArgs &p, bool mine, unsigned bit)
{
    if (mine && p.dev_status) atomicOr(p.dev_status, static_cast<int32_t>(bit));
}

// The two 16-byte chunks of a row that slot c covers.
__device__ __forceinline__ void slot_chunks(const RopeArgs &p, int c, int &c0, int &c1)
{
    const int turned = p.rot >> 4;
    const bool half_split = c < turned && !p.interleaved;
    c0 = half_split ? c : 2 * c;
    c1 = half_split ? c + turned : 2 * c + 1;
}

struct Pair8 {
    float cs[8], sn[8];
};

// Cosines and sines of the pairs of slot c (c < rot / 16) for token tok, whose
// cache position is pos.  Every position was checked by positions_ok.
__device__ __forceinline__ void load_pairs(const RopeArgs &p, int c, int tok, int pos, Pair8 &t)
{
    const int half = p.rot >> 1;
    if (p.axes == 1) {
        const int at = p.rope_positions ? __ldg(p.rope_positions + tok) : pos;
        const float4 *row =
            reinterpret_cast<const float4 *>(p.cos_sin + static_cast<int64_t>(at) * p.rot + 8 * c);
        const float4 *rows = row + (half >> 2);
        const float4 a = __ldg(row), b = __ldg(row + 1), d = __ldg(rows), e = __ldg(rows + 1);
        t.cs[0] = a.x; t.cs[1] = a.y; t.cs[2] = a.z; t.cs[3] = a.w;
        t.cs[4] = b.x; t.cs[5] = b.y; t.cs[6] = b.z; t.cs[7] = b.w;
        t.sn[0] = d.x; t.sn[1] = d.y; t.sn[2] = d.z; t.sn[3] = d.w;
        t.sn[4] = e.x; t.sn[5] = e.y; t.sn[6] = e.z; t.sn[7] = e.w;
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int i = 8 * c + j;
        const int at =
            __ldg(p.rope_positions + static_cast<int64_t>(p.axis_of_pair[i]) * p.num_tokens + tok);
        const float *row = p.cos_sin + static_cast<int64_t>(at) * p.rot + i;
        t.cs[j] = __ldg(row);
        t.sn[j] = __ldg(row + half);
    }
}

// Whether the table holds every position of the token.
__device__ __forceinline__ bool positions_ok(const RopeArgs &p, int tok, int pos)
{
    if (!p.rope_positions) return pos < p.max_position;
    bool ok = true;
    for (int a = 0; a < p.axes; ++a) {
        const int at = __ldg(p.rope_positions + static_cast<int64_t>(a) * p.num_tokens + tok);
        ok &= at >= 0 && at < p.max_position;
    }
    return ok;
}

__device__ __forceinline__ float2 half2_at(const uint4 &x, int j)
{
    return __half22float2(reinterpret_cast<const __half2 *>(&x)[j]);
}

__device__ __forceinline__ float turn_a(float a, float b, float c, float s)
{
    return __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
}

__device__ __forceinline__ float turn_b(float a, float b, float c, float s)
{
    return __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}

// Rotates the eight pairs of a slot in its two chunks.
__device__ __forceinline__ void rotate(const RopeArgs &p, const Pair8 &t, uint4 &x0, uint4 &x1)
{
    uint4 y0, y1;
    __half2 *h0 = reinterpret_cast<__half2 *>(&y0), *h1 = reinterpret_cast<__half2 *>(&y1);
    if (p.interleaved) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = half2_at(x0, j), g = half2_at(x1, j);
            h0[j] = __floats2half2_rn(turn_a(f.x, f.y, t.cs[j], t.sn[j]),
                                      turn_b(f.x, f.y, t.cs[j], t.sn[j]));
            h1[j] = __floats2half2_rn(turn_a(g.x, g.y, t.cs[j + 4], t.sn[j + 4]),
                                      turn_b(g.x, g.y, t.cs[j + 4], t.sn[j + 4]));
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = half2_at(x0, j), g = half2_at(x1, j);
            h0[j] = __floats2half2_rn(turn_a(f.x, g.x, t.cs[2 * j], t.sn[2 * j]),
                                      turn_a(f.y, g.y, t.cs[2 * j + 1], t.sn[2 * j + 1]));
            h1[j] = __floats2half2_rn(turn_b(f.x, g.x, t.cs[2 * j], t.sn[2 * j]),
                                      turn_b(f.y, g.y, t.cs[2 * j + 1], t.sn[2 * j + 1]));
        }
    }
    x0 = y0;
    x1 = y1;
}

// One token's rows by a team of kTeam threads: the queries, and with kCache
// the keys and values too (into the fp16 pools).  The first rows are on their
// way while the token's sequence, block and table row are looked up.
template <int kD, int kTeam, bool kCache>
__device__ __forceinline__ void rope_token(const RopeArgs &p, int tok)
{
    const int tid = threadIdx.x % kTeam;
    constexpr int kSlots = kD / 16;              // slots per row
    constexpr int kRows = kTeam / kSlots;        // rows per pass of the team
    constexpr int kBatch = 4;                    // rows in flight per thread
    const int c = tid % kSlots, r0 = tid / kSlots;
    const int heads = p.num_heads, kv = p.num_kv_heads;
    const int rows = kCache ? heads + 2 * kv : heads;
    int c0, c1;
    slot_chunks(p, c, c0, c1);
    auto source = [&](int r) -> const uint4 * {
        const __half *s;
        if (r < heads)
            s = p.q + tok * p.q_stride + static_cast<int64_t>(r) * kD;
        else if (r < heads + kv)
            s = p.k + tok * p.k_stride + static_cast<int64_t>(r - heads) * kD;
        else
            s = p.v + tok * p.v_stride + static_cast<int64_t>(r - heads - kv) * kD;
        return reinterpret_cast<const uint4 *>(s);
    };
    uint4 x[kBatch][2];
    auto load = [&](int base) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int r = base + b * kRows;
            if (r < rows) {
                const uint4 *s = source(r);
                x[b][0] = s[c0];
                x[b][1] = s[c1];
            }
        }
    };
    load(r0);

    const int seq = warp_search(p.num_seqs, tok, [&](int s) { return __ldg(p.query_starts + s); });
    if (seq < 0) return;
    SeqRows sr;
    sr.load(p.query_starts, p.context_lens, seq, p.num_tokens, p.max_blocks_per_seq * 16);
    if (tok - sr.start >= sr.len) return;  // behind the last sequence: left as it was
    const int pos = sr.ctx - sr.len + (tok - sr.start);
    bool live = sr.ok;  // (see check_sequences)
    if (live && !positions_ok(p, tok, pos)) {
        live = false;
        report(p, tid == 0, PKV_DEV_BAD_POS);
    }
    int64_t blk = -1;
    if (kCache && live) {
        blk = __ldg(p.block_tables + static_cast<int64_t>(seq) * p.max_blocks_per_seq + (pos >> 4));
        if (blk < 0 || blk >= p.num_blocks) {
            blk = -1;
            report(p, tid == 0, PKV_DEV_BAD_BLOCK);
        }
    }
    Pair8 t;
    const bool turns = c < (p.rot >> 4);
    if (live && turns) load_pairs(p, c, tok, pos, t);

    for (int base = r0; base < rows; base += kBatch * kRows) {
        if (base != r0) load(base);
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int r = base + b * kRows;
            if (r >= rows) continue;
            if (live && turns && r < heads + kv) rotate(p, t, x[b][0], x[b][1]);
            uint4 *dst;
            if (r < heads) {
                dst = reinterpret_cast<uint4 *>(
                    p.q_out + (static_cast<int64_t>(tok) * heads + r) * kD);
                if (!live) x[b][0] = x[b][1] = make_uint4(0, 0, 0, 0);
            } else {
                if (blk < 0) continue;
                const bool is_v = r >= heads + kv;
                const int h = r - heads - (is_v ? kv : 0);
                dst = reinterpret_cast<uint4 *>(
                    (is_v ? p.v_pool : p.k_pool) + ((blk * kv + h) * 16 + (pos & 15)) * kD);
            }
            dst[c0] = x[b][0];
            dst[c1] = x[b][1];
        }
    }
}

// The tokens of a CTA: a warp each where a token has few rows (a CTA to itself
// would leave most of its threads without any: 64206 tokens of 8 heads of 64
// took 88 us so, against 52), else one.
template <int kD, bool kCache>
__device__ __forceinline__ void rope_tokens(const RopeArgs &p, int group)
{
    if (p.tokens_per_cta == 1) {
        rope_token<kD, kRowThreads, kCache>(p, group);
    } else {
        const int tok = group * p.tokens_per_cta + static_cast<int>(threadIdx.x >> 5);
        if (tok < p.num_tokens) rope_token<kD, 32, kCache>(p, tok);
    }
}

// The last CTAs of a call with a status word look at every sequence: one that
// does not fit need not have a token that a CTA works on.
__device__ __forceinline__ bool check_sequences(const RopeArgs &p)
{
    if (blockIdx.x < p.check_from) return false;
    report_bad_sequences(p.query_starts, p.context_lens, p.num_seqs, p.num_tokens,
                         p.max_blocks_per_seq * 16, p.dev_status,
                         static_cast<int>(blockIdx.x - p.check_from) * kRowThreads +
                             static_cast<int>(threadIdx.x),
                         static_cast<int>(gridDim.x - p.check_from) * kRowThreads);
    return true;
}

template <int kD>
__global__ void __launch_bounds__(kRowThreads) rope_fp16_kernel(const __grid_constant__ RopeArgs p)
{
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    if (check_sequences(p)) return;
    rope_tokens<kD, true>(p, blockIdx.x);
}

// Code caches.  The first CTAs own one (page, kv head, K | V) tile each, at
// head_dim 64 the K and the V tile of a (page, kv head): a tile's new rows come
// rotated from the input and go to the fp16 pool, its other rows come from the
// pool, and all 16 rows are quantized.  The CTAs behind them rotate a few
// tokens' queries each.
template <int kD, bool kFp8>
__global__ void __launch_bounds__(kRowThreads) rope_codes_kernel(const __grid_constant__ RopeArgs p)
{
    constexpr int kTileThreads = kD;                     // 16 rows of kD / 16 slots
    constexpr int kTiles = kRowThreads / kTileThreads;   // per CTA
    constexpr int kSlots = kD / 16, kRowChunks = kD / 8;
    __shared__ float warp_max[kRowThreads / 32];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    if (check_sequences(p)) return;
    const int kv = p.num_kv_heads;
    const int per_unit = kv * 2 / kTiles;                // CTAs of a page
    const int64_t tiles = static_cast<int64_t>(p.units) * per_unit;
    if (blockIdx.x >= tiles) {
        rope_tokens<kD, false>(p, static_cast<int>(blockIdx.x - tiles));
        return;
    }
    const int unit = static_cast<int>(blockIdx.x / per_unit);
    const int sub = static_cast<int>(blockIdx.x - static_cast<int64_t>(unit) * per_unit);
    const int tid = threadIdx.x % kTileThreads;
    const bool is_v = kTiles == 2 ? threadIdx.x >= kTileThreads : sub >= kv;
    const int h = kTiles == 2 || sub < kv ? sub : sub - kv;
    const bool first = threadIdx.x == 0 && sub == 0;

    // pages of sequence s: units from floor(starts[s] / 16) + 2 s on (a run
    // of 16 m + r tokens touches at most m + 2 pages)
    auto base_of = [&](int s) -> int64_t {
        return static_cast<int64_t>(__ldg(p.query_starts + s) >> 4) + 2 * s;
    };
    const int seq = warp_search(p.num_seqs, unit, base_of);
    if (seq < 0) return;
    SeqRows sr;
    sr.load(p.query_starts, p.context_lens, seq, p.num_tokens, p.max_blocks_per_seq * 16);
    if (sr.len == 0 || !sr.ok) return;
    const int old = sr.ctx - sr.len;
    const int64_t page = (old >> 4) + (unit - base_of(seq));
    if (page > (sr.ctx - 1) >> 4) return;
    const int64_t blk = __ldg(p.block_tables + static_cast<int64_t>(seq) * p.max_blocks_per_seq + page);
    if (blk < 0 || blk >= p.num_blocks) {
        report(p, first, PKV_DEV_BAD_BLOCK);
        return;
    }
    const int c = tid % kSlots, row = tid / kSlots;
    int c0 = 2 * c, c1 = 2 * c + 1;
    if (!is_v) slot_chunks(p, c, c0, c1);
    const int64_t tile = blk * kv + h;
    uint4 *pool = reinterpret_cast<uint4 *>(is_v ? p.v_pool : p.k_pool) +
                  (tile * 16 + row) * kRowChunks;
    const int pos = static_cast<int>(page) * 16 + row;
    const int tok = sr.start + (pos - old);
    uint4 raw[2];
    bool fresh = pos >= old && pos < sr.ctx;
    if (fresh) fresh = positions_ok(p, tok, pos);  // reported by the query CTAs
    if (fresh) {
        const uint4 *src = reinterpret_cast<const uint4 *>(
            (is_v ? p.v + tok * p.v_stride : p.k + tok * p.k_stride) + static_cast<int64_t>(h) * kD);
        raw[0] = src[c0];
        raw[1] = src[c1];
        if (!is_v && c < (p.rot >> 4)) {
            Pair8 t;
            load_pairs(p, c, tok, pos, t);
            rotate(p, t, raw[0], raw[1]);
        }
        pool[c0] = raw[0];
        pool[c1] = raw[1];
    } else {
        raw[0] = pool[c0];
        raw[1] = pool[c1];
    }
    // the largest magnitude of the tile's threads
    float amax = chunks_absmax(raw);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kTileThreads / 32; ++w)
        amax = fmaxf(amax, warp_max[threadIdx.x / kTileThreads * (kTileThreads / 32) + w]);
    const float scale = __fmul_rn(amax, kFp8 ? 1.0f / 448.0f : 1.0f / 127.0f);
    const float rcp = __frcp_rn(scale);
    uint2 *dst = reinterpret_cast<uint2 *>(is_v ? p.v_codes : p.k_codes) +
                 (tile * 16 + row) * kRowChunks;
    dst[c0] = kFp8 ? chunk_codes_fp8(raw[0], scale) : chunk_codes(raw[0], scale, rcp);
    dst[c1] = kFp8 ? chunk_codes_fp8(raw[1], scale) : chunk_codes(raw[1], scale, rcp);
    if (tid == 0) (is_v ? p.v_scales : p.k_scales)[tile] = scale;
}

struct RopeCall {
    void *q_out, *k_cache, *v_cache;
    void *k_codes, *v_codes;
    float *k_scales, *v_scales;
    int num_blocks;
    const void *q;
    int64_t q_stride;
    const void *k;
    int64_t k_stride;
    const void *v;
    int64_t v_stride;
    const float *cos_sin;
    int max_position, rot_dim, interleaved;
    const int32_t *rope_positions;
    int num_axes;
    const uint8_t *axis_of_pair;
    const int32_t *query_starts, *context_lens, *block_tables;
    int max_blocks_per_seq, num_tokens, num_seqs, num_heads, num_kv_heads, head_dim, block_size;
    int32_t *dev_status;
    void *stream;
};

template <typename Kernel>
pkv_status launch_rope(Kernel kernel, int64_t grid, const RopeCall &c, RopeArgs &a)
{
    a.check_from = static_cast<unsigned>(grid);
    if (c.dev_status)  // a sequence a thread, up to 256 CTAs
        grid += c.num_seqs < 256 * kRowThreads ? (c.num_seqs + kRowThreads - 1) / kRowThreads : 256;
    if (grid > INT32_MAX) return PKV_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kRowThreads);
    cfg.stream = static_cast<cudaStream_t>(c.stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    return PKV_OK;
}

enum { kRopeF16 = 0, kRopeI8 = 1, kRopeF8 = 2 };

pkv_status rope_entry(const RopeCall &c, int kind)
{
    if (!c.k_cache || !c.v_cache || !c.cos_sin || !c.query_starts) return PKV_ERR_INVALID_ARG;
    // (arrays without elements may be null)
    if (c.num_tokens != 0 && (!c.q_out || !c.q || !c.k || !c.v)) return PKV_ERR_INVALID_ARG;
    if (c.num_seqs != 0 && !c.context_lens) return PKV_ERR_INVALID_ARG;
    if (kind != kRopeF16 && (!c.k_codes || !c.v_codes || !c.k_scales || !c.v_scales))
        return PKV_ERR_INVALID_ARG;
    if (c.num_blocks <= 0 || c.max_position <= 0 || c.rot_dim <= 0 || c.num_axes <= 0 ||
        c.max_blocks_per_seq < 0 || c.num_tokens < 0 || c.num_seqs < 0 || c.num_heads <= 0 ||
        c.num_kv_heads <= 0 || c.head_dim <= 0 || c.block_size <= 0 || c.rot_dim > c.head_dim)
        return PKV_ERR_INVALID_ARG;
    if (!c.block_tables && c.max_blocks_per_seq > 0 && c.num_seqs > 0) return PKV_ERR_INVALID_ARG;
    // several axes: a position for each, and an axis for each pair
    if (c.num_axes > 1 && ((c.num_tokens != 0 && !c.rope_positions) || !c.axis_of_pair))
        return PKV_ERR_INVALID_ARG;
    if (c.block_size != 16 || (c.head_dim != 64 && c.head_dim != 128) || c.rot_dim % 16 != 0 ||
        c.num_axes > 255)
        return PKV_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(c.max_blocks_per_seq) * 16 > INT32_MAX) return PKV_ERR_UNSUPPORTED;
    if (c.q_stride < static_cast<int64_t>(c.num_heads) * c.head_dim ||
        c.k_stride < static_cast<int64_t>(c.num_kv_heads) * c.head_dim ||
        c.v_stride < static_cast<int64_t>(c.num_kv_heads) * c.head_dim)
        return PKV_ERR_INVALID_ARG;
    if (!aligned(c.q_out, 16) || !aligned(c.k_cache, 16) || !aligned(c.v_cache, 16) ||
        !aligned(c.q, 16) || !aligned(c.k, 16) || !aligned(c.v, 16) || c.q_stride % 8 ||
        c.k_stride % 8 || c.v_stride % 8 || !aligned(c.cos_sin, 16) ||
        !aligned(c.rope_positions, 4) || !aligned(c.query_starts, 4) ||
        !aligned(c.context_lens, 4) || !aligned(c.block_tables, 4) || !aligned(c.dev_status, 4) ||
        !aligned(c.k_codes, 16) || !aligned(c.v_codes, 16) || !aligned(c.k_scales, 4) ||
        !aligned(c.v_scales, 4))
        return PKV_ERR_MISALIGNED;
    RopeArgs a;
    for (int i = 0; i < kMaxPairs; ++i) a.axis_of_pair[i] = 0;
    if (c.axis_of_pair)
        for (int i = 0; i < c.rot_dim / 2; ++i) {
            if (c.axis_of_pair[i] >= c.num_axes) return PKV_ERR_INVALID_ARG;
            a.axis_of_pair[i] = c.axis_of_pair[i];
        }
    if (c.num_tokens == 0 || c.num_seqs == 0) return PKV_OK;
    a.q_out = static_cast<__half *>(c.q_out);
    a.k_pool = static_cast<__half *>(c.k_cache);
    a.v_pool = static_cast<__half *>(c.v_cache);
    a.k_codes = static_cast<uint8_t *>(c.k_codes);
    a.v_codes = static_cast<uint8_t *>(c.v_codes);
    a.k_scales = c.k_scales;
    a.v_scales = c.v_scales;
    a.q = static_cast<const __half *>(c.q);
    a.k = static_cast<const __half *>(c.k);
    a.v = static_cast<const __half *>(c.v);
    a.q_stride = c.q_stride;
    a.k_stride = c.k_stride;
    a.v_stride = c.v_stride;
    a.cos_sin = c.cos_sin;
    a.rope_positions = c.rope_positions;
    a.query_starts = c.query_starts;
    a.context_lens = c.context_lens;
    a.block_tables = c.block_tables;
    a.dev_status = c.dev_status;
    a.max_position = c.max_position;
    a.rot = c.rot_dim;
    a.interleaved = c.interleaved;
    a.axes = c.num_axes;
    a.max_blocks_per_seq = c.max_blocks_per_seq;
    a.num_tokens = c.num_tokens;
    a.num_seqs = c.num_seqs;
    a.num_heads = c.num_heads;
    a.num_kv_heads = c.num_kv_heads;
    a.num_blocks = c.num_blocks;
    a.units = 0;
    const int slots = (kind == kRopeF16 ? c.num_heads + 2 * c.num_kv_heads : c.num_heads) *
                      (c.head_dim / 16);
    a.tokens_per_cta = slots <= kRowThreads ? kRowThreads / 32 : 1;
    const int64_t groups = (c.num_tokens + a.tokens_per_cta - 1) / a.tokens_per_cta;
    if (kind == kRopeF16)
        return c.head_dim == 128 ? launch_rope(rope_fp16_kernel<128>, groups, c, a)
                                 : launch_rope(rope_fp16_kernel<64>, groups, c, a);
    const int64_t units = static_cast<int64_t>(c.num_tokens) / 16 + 2 * static_cast<int64_t>(c.num_seqs);
    if (units > INT32_MAX) return PKV_ERR_UNSUPPORTED;
    a.units = static_cast<int>(units);
    const int64_t grid = units * c.num_kv_heads * (c.head_dim == 128 ? 2 : 1) + groups;
    if (c.head_dim == 128)
        return kind == kRopeF8 ? launch_rope(rope_codes_kernel<128, true>, grid, c, a)
                               : launch_rope(rope_codes_kernel<128, false>, grid, c, a);
    return kind == kRopeF8 ? launch_rope(rope_codes_kernel<64, true>, grid, c, a)
                           : launch_rope(rope_codes_kernel<64, false>, grid, c, a);
}

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_rope_append_fp16(
    void *q_out, void *k_cache, void *v_cache, int num_blocks, const void *q, int64_t q_stride,
    const void *k, int64_t k_stride, const void *v, int64_t v_stride, const float *cos_sin,
    int max_position, int rot_dim, int interleaved, const int32_t *rope_positions, int num_axes,
    const uint8_t *axis_of_pair, const int32_t *query_starts, const int32_t *context_lens,
    const int32_t *block_tables, int max_blocks_per_seq, int num_tokens, int num_seqs,
    int num_heads, int num_kv_heads, int head_dim, int block_size, int32_t *dev_status,
    void *stream)
{
    const pkv::RopeCall c{q_out, k_cache, v_cache, nullptr, nullptr, nullptr, nullptr, num_blocks,
                          q, q_stride, k, k_stride, v, v_stride, cos_sin, max_position, rot_dim,
                          interleaved, rope_positions, num_axes, axis_of_pair, query_starts,
                          context_lens, block_tables, max_blocks_per_seq, num_tokens, num_seqs,
                          num_heads, num_kv_heads, head_dim, block_size, dev_status, stream};
    return pkv::rope_entry(c, pkv::kRopeF16);
}

extern "C" pkv_status pkv_rope_append_int8(
    void *q_out, void *k_cache, void *v_cache, int8_t *k_codes, int8_t *v_codes, float *k_scales,
    float *v_scales, int num_blocks, const void *q, int64_t q_stride, const void *k,
    int64_t k_stride, const void *v, int64_t v_stride, const float *cos_sin, int max_position,
    int rot_dim, int interleaved, const int32_t *rope_positions, int num_axes,
    const uint8_t *axis_of_pair, const int32_t *query_starts, const int32_t *context_lens,
    const int32_t *block_tables, int max_blocks_per_seq, int num_tokens, int num_seqs,
    int num_heads, int num_kv_heads, int head_dim, int block_size, int32_t *dev_status,
    void *stream)
{
    const pkv::RopeCall c{q_out, k_cache, v_cache, k_codes, v_codes, k_scales, v_scales, num_blocks,
                          q, q_stride, k, k_stride, v, v_stride, cos_sin, max_position, rot_dim,
                          interleaved, rope_positions, num_axes, axis_of_pair, query_starts,
                          context_lens, block_tables, max_blocks_per_seq, num_tokens, num_seqs,
                          num_heads, num_kv_heads, head_dim, block_size, dev_status, stream};
    return pkv::rope_entry(c, pkv::kRopeI8);
}

extern "C" pkv_status pkv_rope_append_fp8(
    void *q_out, void *k_cache, void *v_cache, uint8_t *k_codes, uint8_t *v_codes, float *k_scales,
    float *v_scales, int num_blocks, const void *q, int64_t q_stride, const void *k,
    int64_t k_stride, const void *v, int64_t v_stride, const float *cos_sin, int max_position,
    int rot_dim, int interleaved, const int32_t *rope_positions, int num_axes,
    const uint8_t *axis_of_pair, const int32_t *query_starts, const int32_t *context_lens,
    const int32_t *block_tables, int max_blocks_per_seq, int num_tokens, int num_seqs,
    int num_heads, int num_kv_heads, int head_dim, int block_size, int32_t *dev_status,
    void *stream)
{
    const pkv::RopeCall c{q_out, k_cache, v_cache, k_codes, v_codes, k_scales, v_scales, num_blocks,
                          q, q_stride, k, k_stride, v, v_stride, cos_sin, max_position, rot_dim,
                          interleaved, rope_positions, num_axes, axis_of_pair, query_starts,
                          context_lens, block_tables, max_blocks_per_seq, num_tokens, num_seqs,
                          num_heads, num_kv_heads, head_dim, block_size, dev_status, stream};
    return pkv::rope_entry(c, pkv::kRopeF8);
}
