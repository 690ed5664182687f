// pkv_prefill.cu -- attention of a ragged batch of new tokens over the paged
// cache, causal at their positions, with the scores of the scored decode
// (tanh cap, bias by distance, window, visible prefix).
//
// For the token at position i, key t and z = softmax_scale <q, K_t>:
//   z' = cap tanh(z / cap)  (cap > 0),   z'' = z' - slope[h] |i - t|,
//   t is seen if (t <= i and i - t < window) or t < prefix_len,
//   out = sum over seen t of softmax(z'')_t V_t.
//
// Bound by the tensor cores: 4 d products per pair of a query row and a seen
// key, against one exponential per pair.  A work item is 256 query rows of one
// kv head -- (token, head) pairs, token by token, so a kv head's whole group
// shares every key and value that is read -- as two tiles of 128 rows, the M of
// one tcgen05.mma.  Per 128 keys (eight pages) a tile does
//   S = Q K^T   (128 x 128 fp32 in TMEM; Q, K in shared memory)
//   P = 2^(S' - m)  (registers: one thread per row, so maxima and sums need no
//                    exchange between threads; back to TMEM as fp16)
//   O += P V    (128 x d fp32 in TMEM; P from TMEM, V in shared memory as it
//                lies in the page, rows of keys)
// and the two tiles take turns: while one is in its softmax, the tensor core
// works for the other.  The accumulators are rescaled only when a row's
// maximum has grown by more than 2^6; the probabilities enter the product with
// a factor 2^6, so up to that much smaller ones are normal fp16 numbers.  They
// are rounded to fp16 (2^-11 of each, in both directions): that error averages
// out over the keys and stays below the rounding of the fp16 output.  Sums,
// maxima and accumulators are fp32.
//
// Roles of the warps: 0-3 and 4-7 the rows of the two tiles, 8 issues the
// products, 9 the TMA loads of the pages (a ring of tiles of 128 keys, K and V
// in turn).  INT8 / FP8 pages land in a second ring, and warps 12-15 widen
// them exactly to fp16; the K scales multiply the scores, the V scales enter
// the probabilities as a ratio to the largest one so far.
//
// Items are numbered by bounds that the host knows (pkv_ragged.cuh), the ones
// with the most keys first.  When they are fewer than the SMs fill, each is
// split over its keys and a second kernel joins the parts.
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include <mutex>

#include "pkv_host.cuh"
#include "pkv_ptx.cuh"
#include "pkv_ragged.cuh"
#include "pkv_score.cuh"
#include "pkv_umma.cuh"

namespace pkv {
namespace {

constexpr int kRows = 256;      // query rows per item: two tiles
constexpr int kTile = 128;      // rows per tile, keys per step
constexpr int kPage = 16;
constexpr int kPagesPerTile = kTile / kPage;
constexpr int kSms = 152;       // GB300: what the split over the keys aims to fill
constexpr int kMaxSplits = 64;
constexpr uint64_t kWaitLimitNs = 1000000000ull;  // bounded waits: 1 s
constexpr float kLazy = 6.f;    // log2 growth of a maximum that is left in the sums
constexpr float kLift = 6.f;    // log2 factor of the probabilities
constexpr float kVLazy = 8.f;   // growth of a V scale that is left in the ratio

constexpr int kKvF16 = 0, kKvI8 = 1, kKvF8 = 2;

struct PrefillArgs {
    __half *out;
    const __half *query;
    const int32_t *block_tables, *query_starts, *context_lens;
    const float *k_scales, *v_scales;
    const float *slopes;
    const int32_t *prefix_lens;
    float *part_acc;    // [splits][num_tokens * num_heads][head_dim]
    float2 *part_ml;    // [splits][num_tokens * num_heads]: maximum, sum
    int32_t *dev_status;
    int num_tokens, num_seqs, num_heads, num_kv_heads, group;
    int max_blocks_per_seq, num_blocks, ctx_cap, window, splits, units;
    float scale_log2, cap, cap_inv;
};

// ------------------------------------------------------------ shared memory
template <int kKv, int kD>
struct Smem {
    static constexpr bool kCodes = kKv != kKvF16;
    static constexpr int kHalves = kD / 64;
    static constexpr int kHalfBytes = kTile * 128;             // 64 values of 128 rows
    static constexpr int kTileBytes = kHalves * kHalfBytes;    // 128 rows of Q, K or V
    static constexpr int kCodeBytes = kTile * kD;
    static constexpr int kStages = kCodes ? (kD == 128 ? 3 : 6) : (kD == 128 ? 5 : 10);
    static constexpr int kCodeStages = kCodes ? 4 : 0;
    static constexpr int kRing = 2 * kTileBytes;
    static constexpr int kCodeRing = kRing + kStages * kTileBytes;
    static constexpr int kCtl = kCodeRing + kCodeStages * kCodeBytes;
    static constexpr int kBars = 2 * kStages + 2 * kCodeStages + 8;
    // scales [kScaleTiles][K, V][8 pages]: the loads run at most five tiles
    // ahead of the softmax (the code ring, the ring and the tile at work)
    static constexpr int kScaleTiles = 8;
    static constexpr int kScales = kCtl + 8 * kBars;
    static constexpr int kFlags =
        kScales + (kCodes ? kScaleTiles * 2 * kPagesPerTile * 4 : 0);
    static constexpr int kBytes = kFlags + 16;
    // a second CTA on the SM would wait for TMEM: ask for more than half
    static constexpr int kAsk = 1024 + (kBytes > 120 * 1024 ? kBytes : 120 * 1024);
};

struct Waiter {
    volatile int *abort;
    int32_t *dev_status;
    // Bounded wait of a whole warp; false once any wait of the CTA ran out.
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const
    {
        bool ok = ptx::mbar_try_wait(bar, parity);
        if (!__all_sync(0xffffffffu, ok)) {
            const uint64_t t0 = ptx::globaltimer_ns();
            while (!ok) {
                for (int i = 0; i < 64 && !ok; ++i) ok = ptx::mbar_try_wait(bar, parity);
                if (ok || *abort) break;
                if (ptx::globaltimer_ns() - t0 > kWaitLimitNs) {
                    *abort = 1;
                    if (dev_status) atomicOr(dev_status, PKV_DEV_TIMEOUT);
                }
            }
            ok = __all_sync(0xffffffffu, ok);
        }
        return ok;
    }
};

// ------------------------------------------------------------------- items
struct Item {
    int seq, kvh, row0, rows;   // first row of the item among the sequence's, rows
    int start;                  // first token of the sequence
    int pos0;                   // position of the sequence's first new token
    int lo, hi, pre;            // keys of the item: lo .. hi and below pre
    int np1, gap, visited;      // pages: np1, a gap, the rest (see the decode)
    int ta, tb;                 // tiles of this split
    bool ok;

    __device__ __forceinline__ int real(int v) const { return v + (v >= np1 ? gap : 0); }

    // bits of a page's tokens (its first is t0) that some row may see
    __device__ __forceinline__ uint32_t live(int t0) const
    {
        return (below(hi + 1 - t0) & ~below(lo - t0)) | below(pre - t0);
    }
};

// The item of unit u; false if the unit names none.
__device__ __forceinline__ bool find_item(const PrefillArgs &p, int u, int kvh, int z, Item &it)
{
    auto base_of = [&](int s) -> int64_t {
        return static_cast<int64_t>(__ldg(p.query_starts + s)) * p.group / kRows + s;
    };
    const int seq = warp_search(p.num_seqs, u, base_of);
    if (seq < 0) return false;
    SeqRows sr;
    sr.load(p.query_starts, p.context_lens, seq, p.num_tokens, p.ctx_cap);
    const int64_t row0 = (u - base_of(seq)) * kRows;
    const int64_t rows = static_cast<int64_t>(sr.len) * p.group - row0;
    if (rows <= 0) return false;
    it.seq = seq;
    it.kvh = kvh;
    it.row0 = static_cast<int>(row0);
    it.rows = static_cast<int>(rows < kRows ? rows : kRows);
    it.start = sr.start;
    it.ok = sr.ok;
    it.pos0 = sr.ctx - sr.len;
    if (!sr.ok) return true;
    const int first = it.pos0 + it.row0 / p.group;
    const int last = it.pos0 + (it.row0 + it.rows - 1) / p.group;
    it.lo = p.window > 0 && first >= p.window ? first - p.window + 1 : 0;
    it.hi = last;
    it.pre = p.prefix_lens ? min(max(__ldg(p.prefix_lens + seq), 0), sr.ctx) : 0;
    const int fp = it.lo / kPage;
    it.np1 = min((it.pre + kPage - 1) / kPage, fp);
    it.gap = fp - it.np1;
    it.visited = max(last, it.pre - 1) / kPage + 1 - it.gap;
    const int tiles = (it.visited + kPagesPerTile - 1) / kPagesPerTile;
    it.ta = static_cast<int>(static_cast<int64_t>(tiles) * z / p.splits);
    it.tb = static_cast<int>(static_cast<int64_t>(tiles) * (z + 1) / p.splits);
    return true;
}

// Row r of the item: its index among all (token, head) rows of the batch.
__device__ __forceinline__ int64_t row_at(const PrefillArgs &p, const Item &it, int r)
{
    const int q = it.row0 + r, j = q / p.group;
    return (static_cast<int64_t>(it.start) + j) * p.num_heads + it.kvh * p.group + (q - j * p.group);
}

// ------------------------------------------------------------------ kernel
template <int kKv>
__host__ __device__ constexpr int prefill_threads()
{
    return kKv == kKvF16 ? 384 : 512;
}

// Registers: launched with 168 (128 with the widening warps) per thread; the
// softmax warpgroups take what the others give back.
template <int kKv>
__device__ __forceinline__ void more_registers()
{
    if constexpr (kKv == kKvF16)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    else
        asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
}

template <int kKv>
__device__ __forceinline__ void fewer_registers()
{
    if constexpr (kKv == kKvF16)
        asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    else
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ void st_shared16(uint32_t addr, uint4 v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w)
                 : "memory");
}

// kMod: any of cap, bias or scales, or a scale that is not positive -- the scores are
// worked out before their maximum is taken.  Without it the scale is folded
// into the exponent.
template <int kKv, int kD, bool kMod>
__global__ void __launch_bounds__(prefill_threads<kKv>(), 1)
    prefill_kernel(const __grid_constant__ PrefillArgs p, const __grid_constant__ CUtensorMap tmk,
                   const __grid_constant__ CUtensorMap tmv)
{
    using M = Smem<kKv, kD>;
    constexpr bool kCodes = M::kCodes;
    constexpr int S = M::kStages;
    constexpr int kRowChunks = kD / 8;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t base = ptx::smem_addr(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // barriers: ring full / empty, code ring full / empty, then single ones
    auto full = [&](int s) { return base + M::kCtl + 8 * s; };
    auto empty = [&](int s) { return base + M::kCtl + 8 * (S + s); };
    [[maybe_unused]] auto cfull = [&](int s) { return base + M::kCtl + 8 * (2 * S + s); };
    [[maybe_unused]] auto cempty = [&](int s) {
        return base + M::kCtl + 8 * (2 * S + M::kCodeStages + s);
    };
    const uint32_t one = base + M::kCtl + 8 * (2 * S + 2 * M::kCodeStages);
    const uint32_t q_full = one, drain = one + 8;
    auto s_full = [&](int i) { return one + 16 + 8 * i; };
    auto p_full = [&](int i) { return one + 32 + 8 * i; };
    auto o_full = [&](int i) { return one + 48 + 8 * i; };
    volatile int *flags = reinterpret_cast<volatile int *>(smem + M::kFlags);  // abort, bad, tmem
    const Waiter wait{flags, p.dev_status};

    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    // the units with the most keys (the last ones of a sequence) first; the
    // kv heads and key splits of a unit side by side
    const int per_unit = p.num_kv_heads * p.splits;
    const int u = p.units - 1 - static_cast<int>(blockIdx.x / per_unit);
    const int sub = static_cast<int>(blockIdx.x % per_unit);
    const int z = sub % p.splits;
    Item it;
    if (!find_item(p, u, sub / p.splits, z, it)) return;
    const int nt = it.ok ? it.tb - it.ta : 0;
    if (nt == 0) {
        // a sequence that does not fit (zeros), or a split without keys
        if (!it.ok && it.row0 == 0 && sub == 0 && threadIdx.x == 0 && p.dev_status)
            atomicOr(p.dev_status, PKV_DEV_BAD_CTX);
        for (int i = threadIdx.x; i < it.rows * kRowChunks; i += blockDim.x) {
            const int64_t row = row_at(p, it, i / kRowChunks);
            if (row < 0 || row >= static_cast<int64_t>(p.num_tokens) * p.num_heads) continue;
            if (p.splits == 1)
                reinterpret_cast<uint4 *>(p.out + row * kD)[i % kRowChunks] = make_uint4(0, 0, 0, 0);
            else if (i % kRowChunks == 0)
                p.part_ml[static_cast<int64_t>(z) * p.num_tokens * p.num_heads + row] =
                    make_float2(-INFINITY, 0.f);
        }
        return;
    }
    const bool two = it.rows > kTile;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            ptx::mbar_init(full(s), kCodes ? 128 : 1);
            ptx::mbar_init(empty(s), 1);
        }
        for (int s = 0; s < M::kCodeStages; ++s) {
            ptx::mbar_init(cfull(s), 1);
            ptx::mbar_init(cempty(s), 128);
        }
        ptx::mbar_init(q_full, kRows);
        ptx::mbar_init(drain, 1);
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(s_full(i), 1);
            ptx::mbar_init(p_full(i), kTile);
            ptx::mbar_init(o_full(i), 1);
        }
        ptx::fence_mbar_init();
        flags[0] = flags[1] = 0;
    }
    if (warp == 8) umma::alloc(base + M::kFlags + 8, 512);
    umma::fence_before();
    __syncthreads();
    umma::fence_after();
    const uint32_t tmem = static_cast<uint32_t>(flags[2]);
    auto t_s = [&](int i) { return tmem + kTile * i; };            // S, then P, of tile i
    auto t_o = [&](int i) { return tmem + 2 * kTile + kD * i; };   // O of tile i

    if (warp < 8) {
        // ------------------------------------------------ rows of the tiles
        more_registers<kKv>();
        const int i = warp >> 2;                        // tile
        const int tid = threadIdx.x & (kTile - 1);
        const int r = kTile * i + tid;                  // row of the item
        {
            // the tile's queries, K-major with the 128-byte swizzle; 16 bytes
            // a thread, neighbouring threads along a row
            const uint32_t dst = base + i * M::kTileBytes;
#pragma unroll 4
            for (int e = tid; e < kTile * kRowChunks; e += kTile) {
                const int row = e / kRowChunks, ch = e % kRowChunks;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (kTile * i + row < it.rows)
                    v = __ldg(reinterpret_cast<const uint4 *>(
                                  p.query + row_at(p, it, kTile * i + row) * kD) + ch);
                st_shared16(dst + (ch >> 3) * M::kHalfBytes + row * 128 +
                                (((ch & 7) ^ (row & 7)) << 4), v);
            }
            ptx::fence_proxy_async_smem();
            ptx::mbar_arrive(q_full);
        }
        if (i == 0 || two) {
            const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // TMEM lane 32 (w mod 4)
            const int rr = min(r, it.rows - 1);
            const int q = it.row0 + rr;
            const int pos = it.pos0 + q / p.group;
            const int lo = p.window > 0 ? pos - p.window + 1 : 0;
            // positions of the tile's first and last row: which tiles of keys
            // all of its rows see
            const int pos_a = it.pos0 + (it.row0 + kTile * i) / p.group;
            const int pos_b = it.pos0 + (it.row0 + min(kTile * i + kTile, it.rows) - 1) / p.group;
            float slope = 0.f;
            if (kMod && p.slopes)
                slope = __ldg(p.slopes + it.kvh * p.group + q % p.group) * 1.4426950408889634f;
            float m = -INFINITY, l = 0.f;
            float vref = 0.f, vinv = 0.f;
            bool ok = true;
            for (int j = 0; j < nt && ok; ++j) {
                int t0[kPagesPerTile];
#pragma unroll
                for (int g = 0; g < kPagesPerTile; ++g)
                    t0[g] = it.real((it.ta + j) * kPagesPerTile + g) * kPage;
                ok = wait(s_full(i), j & 1);
                if (!ok) break;
                umma::fence_after();
                float x[kTile];
#pragma unroll
                for (int c = 0; c < kTile; c += 32) umma::ld32(t_s(i) + lanes + c, x + c);
                [[maybe_unused]] float vr[kPagesPerTile];
                float ov = 1.f;  // change of the V reference
                if constexpr (kCodes) {
                    const float *ks = reinterpret_cast<const float *>(smem + M::kScales) +
                                      ((it.ta + j) & (M::kScaleTiles - 1)) * 2 * kPagesPerTile;
                    const float *vs = ks + kPagesPerTile;
                    umma::wait_ld();
                    float most = 0.f;
#pragma unroll
                    for (int g = 0; g < kPagesPerTile; ++g) {
                        const float f = ks[g] * p.scale_log2;
                        vr[g] = vs[g];
                        most = fmaxf(most, vr[g]);
#pragma unroll
                        for (int c = 0; c < kPage; ++c) x[kPage * g + c] *= f;
                    }
                    if (most > kVLazy * vref) {
                        vinv = __frcp_rn(most);
                        ov = vref * vinv;
                        vref = most;
                    }
#pragma unroll
                    for (int g = 0; g < kPagesPerTile; ++g) vr[g] *= vinv;
                } else {
                    umma::wait_ld();
                    if constexpr (kMod) {
#pragma unroll
                        for (int c = 0; c < kTile; ++c) x[c] *= p.scale_log2;
                    }
                }
                if constexpr (kMod) {
                    if (p.cap > 0.f) {
#pragma unroll
                        for (int c = 0; c < kTile; ++c) x[c] = cap_score(x[c], p.cap, p.cap_inv);
                    }
                    if (p.slopes) {
#pragma unroll
                        for (int g = 0; g < kPagesPerTile; ++g) {
                            const float f = static_cast<float>(pos - t0[g]);
#pragma unroll
                            for (int c = 0; c < kPage; ++c)
                                x[kPage * g + c] = fmaf(-slope, fabsf(f - c), x[kPage * g + c]);
                        }
                    }
                }
                const int tmin = t0[0], tmax = t0[kPagesPerTile - 1] + kPage - 1;
                if (!((tmax <= pos_a && (p.window <= 0 || tmin > pos_b - p.window)) ||
                      tmax < it.pre)) {
#pragma unroll
                    for (int g = 0; g < kPagesPerTile; ++g)
#pragma unroll
                        for (int c = 0; c < kPage; ++c) {
                            const int t = t0[g] + c;
                            const bool seen = (t <= pos && t >= lo) || t < it.pre;
                            if (!seen) x[kPage * g + c] = -INFINITY;
                        }
                }
                float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                for (int c = 4; c < kTile; c += 4) {
                    mx[0] = fmaxf(mx[0], x[c]);
                    mx[1] = fmaxf(mx[1], x[c + 1]);
                    mx[2] = fmaxf(mx[2], x[c + 2]);
                    mx[3] = fmaxf(mx[3], x[c + 3]);
                }
                float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                const float sl = kMod ? 1.f : p.scale_log2;
                top *= sl;
                if (__any_sync(0xffffffffu, top > m + kLazy || ov != 1.f)) {
                    const float mn = fmaxf(m, top);
                    const float f = m == -INFINITY ? 0.f : ptx::ex2(m - mn);
                    l *= f;
                    m = mn;
                    if (j > 0) {
                        const float fo = f * ov;
#pragma unroll
                        for (int c = 0; c < kD; c += 32) {
                            float o[32];
                            umma::ld32(t_o(i) + lanes + c, o);
                            umma::wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] *= fo;
                            umma::st32(t_o(i) + lanes + c, reinterpret_cast<const uint32_t *>(o));
                        }
                    }
                }
                // a row that has seen nothing yet: every exponent is -inf
                const float off = kLift - (m == -INFINITY ? 0.f : m);
                float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t pk[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const int c = 64 * h + 2 * e;
                        float a = ptx::ex2(fmaf(x[c], sl, off));
                        float b = ptx::ex2(fmaf(x[c + 1], sl, off));
                        ls[(2 * e) & 3] += a;
                        ls[(2 * e + 1) & 3] += b;
                        if constexpr (kCodes) {
                            a *= vr[c / kPage];
                            b *= vr[c / kPage];
                        }
                        pk[e] = pack2(a, b);
                    }
                    umma::st32(t_s(i) + lanes + 32 * h, pk);
                }
                l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
                umma::wait_st();
                umma::fence_before();
                ptx::mbar_arrive(p_full(i));
            }
            if (ok && wait(o_full(i), 0)) {
                umma::fence_after();
                const bool bad = flags[1] != 0;
                const bool mine = r < it.rows;
                const int64_t row = row_at(p, it, rr);
                const int64_t all = static_cast<int64_t>(p.num_tokens) * p.num_heads;
                const float vs = kCodes ? vref : 1.f;
                if (p.splits == 1) {
                    const float f = l > 0.f ? vs / l : l;  // an empty row: zeros; NaN stays
                    uint4 *dst = reinterpret_cast<uint4 *>(p.out + row * kD);
#pragma unroll
                    for (int c = 0; c < kD; c += 32) {
                        float o[32];
                        umma::ld32(t_o(i) + lanes + c, o);
                        umma::wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = bad ? 0.f : o[e] * f;
                        if (mine) {
#pragma unroll
                            for (int e = 0; e < 32; e += 8)
                                dst[(c + e) / 8] = make_uint4(
                                    pack2(o[e], o[e + 1]), pack2(o[e + 2], o[e + 3]),
                                    pack2(o[e + 4], o[e + 5]), pack2(o[e + 6], o[e + 7]));
                        }
                    }
                } else {
                    float4 *dst = reinterpret_cast<float4 *>(p.part_acc + (z * all + row) * kD);
                    if (mine) p.part_ml[z * all + row] = make_float2(m, bad ? -1.f : l);
#pragma unroll
                    for (int c = 0; c < kD; c += 32) {
                        float o[32];
                        umma::ld32(t_o(i) + lanes + c, o);
                        umma::wait_ld();
                        if (mine) {
#pragma unroll
                            for (int e = 0; e < 32; e += 4)
                                dst[(c + e) / 4] = make_float4(o[e] * vs, o[e + 1] * vs,
                                                               o[e + 2] * vs, o[e + 3] * vs);
                        }
                    }
                }
                umma::fence_before();
            }
        }
    } else if (warp < 12) {
        fewer_registers<kKv>();
        if (warp == 8) {
            // ------------------------------------------------ products
            constexpr uint32_t kQk = umma::f16_idesc(kTile, kTile, false);
            constexpr uint32_t kPv = umma::f16_idesc(kTile, kD, true);
            auto stage = [&](int n) { return base + M::kRing + (n % S) * M::kTileBytes; };
            auto qk = [&](int i, int n) {  // S_i = Q_i K^T
                if (lane == 0) {
#pragma unroll
                    for (int k = 0; k < kD / 16; ++k) {
                        const uint32_t at = (k >> 2) * M::kHalfBytes + (k & 3) * 32;
                        umma::mma_ss(t_s(i), umma::smem_desc(base + i * M::kTileBytes + at, 16),
                                     umma::smem_desc(stage(n) + at, 16), kQk, k > 0);
                    }
                    umma::commit(s_full(i));
                }
                __syncwarp();
            };
            auto pv = [&](int i, int n, bool more) {  // O_i += P_i V
                if (lane == 0) {
#pragma unroll
                    for (int k = 0; k < kTile / 16; ++k)
                        umma::mma_ts(t_o(i), t_s(i) + 8 * k,
                                     umma::smem_desc(stage(n) + k * 2048, M::kHalfBytes), kPv,
                                     more || k > 0);
                }
                __syncwarp();
            };
            auto free_stage = [&](int n) {
                if (lane == 0) umma::commit(empty(n % S));
                __syncwarp();
            };
            const int last = two ? 1 : 0;
            bool ok = wait(q_full, 0) && wait(full(0), 0);
            if (ok) {
                umma::fence_after();
                for (int i = 0; i <= last; ++i) qk(i, 0);
                free_stage(0);
            }
            for (int j = 0; j < nt && ok; ++j) {
                const int nv = 2 * j + 1, nk = 2 * j + 2;
                ok = wait(full(nv % S), (nv / S) & 1);
                if (!ok) break;
                if constexpr (!kCodes) {
                    // rows of V that no row of the item sees (they may hold
                    // anything, NaN included, and are not loaded for pages
                    // past the last) become zeros
                    const int v = (it.ta + j) * kPagesPerTile + lane;
                    uint32_t lv = 0xffffu;
                    if (lane < kPagesPerTile)
                        lv = v < it.visited ? it.live(it.real(v) * kPage) : 0u;
                    unsigned todo = __ballot_sync(0xffffffffu, lv != 0xffffu);
                    if (todo) {
                        while (todo) {
                            const int g = __ffs(todo) - 1;
                            todo &= todo - 1;
                            const uint32_t keep = __shfl_sync(0xffffffffu, lv, g);
                            for (int e = lane; e < kPage * kRowChunks; e += 32) {
                                const int row = e / kRowChunks, ch = e % kRowChunks;
                                if (!(keep >> row & 1u))
                                    st_shared16(stage(nv) + (ch >> 3) * M::kHalfBytes +
                                                    (g * kPage + row) * 128 + ((ch & 7) << 4),
                                                make_uint4(0, 0, 0, 0));
                            }
                        }
                        ptx::fence_proxy_async_smem();
                        __syncwarp();
                    }
                }
                for (int i = 0; i <= last && ok; ++i) {
                    ok = wait(p_full(i), j & 1);
                    if (!ok) break;
                    umma::fence_after();
                    pv(i, nv, j > 0);
                    if (i == last) free_stage(nv);
                    if (j + 1 < nt) {
                        if (i == 0) {
                            ok = wait(full(nk % S), (nk / S) & 1);
                            if (!ok) break;
                            umma::fence_after();
                        }
                        qk(i, nk);
                        if (i == last) free_stage(nk);
                    } else {
                        if (lane == 0) umma::commit(o_full(i));
                        __syncwarp();
                    }
                }
            }
            // nothing of this thread's is in flight after this
            if (lane == 0) umma::commit(drain);
            __syncwarp();
            ptx::mbar_wait_bounded(drain, 0, kWaitLimitNs);
        } else if (warp == 9) {
            // ------------------------------------------------ loads of the pages
            constexpr int R = kCodes ? M::kCodeStages : S;
            constexpr int kBox = kCodes ? kD : 64;                       // values per box
            constexpr int kBoxes = kCodes ? 1 : M::kHalves;
            constexpr int kPageBytes = kPage * kD * (kCodes ? 1 : 2);
            const uint32_t ring = base + (kCodes ? M::kCodeRing : M::kRing);
            constexpr int kStageBytes = kCodes ? M::kCodeBytes : M::kTileBytes;
            const int32_t *table =
                p.block_tables + static_cast<int64_t>(it.seq) * p.max_blocks_per_seq;
            int issued = 0;
            int32_t blk = -1;
            bool want = false, have = false;
            for (int n = 0; n < 2 * nt; ++n) {
                const int s = n % R;
                if ((n & 1) == 0) {
                    const int v = (it.ta + n / 2) * kPagesPerTile + lane;
                    want = lane < kPagesPerTile && v < it.visited;
                    blk = want ? __ldg(table + it.real(v)) : -1;
                    have = want && blk >= 0 && blk < p.num_blocks;
                    if (want && !have) {
                        flags[1] = 1;
                        if (p.dev_status) atomicOr(p.dev_status, PKV_DEV_BAD_BLOCK);
                    }
                }
                const uint32_t fb = kCodes ? cfull(s) : full(s);
                const uint32_t eb = kCodes ? cempty(s) : empty(s);
                [[maybe_unused]] float ks = 0.f, vs = 0.f;
                if constexpr (kCodes) {
                    if ((n & 1) == 0 && have) {
                        const int64_t at = static_cast<int64_t>(blk) * p.num_kv_heads + it.kvh;
                        ks = __ldg(p.k_scales + at);
                        vs = __ldg(p.v_scales + at);
                    }
                }
                if (!wait(eb, ((n / R) & 1) ^ 1)) break;
                if constexpr (kCodes) {
                    if ((n & 1) == 0 && lane < kPagesPerTile) {
                        float *sc = reinterpret_cast<float *>(smem + M::kScales) +
                                    ((it.ta + n / 2) & (M::kScaleTiles - 1)) * 2 * kPagesPerTile;
                        sc[lane] = ks;
                        sc[kPagesPerTile + lane] = vs;
                    }
                    __syncwarp();
                }
                const int pages = __popc(__ballot_sync(0xffffffffu, have));
                if (lane == 0) ptx::mbar_arrive_expect_tx(fb, pages * kPageBytes);
                __syncwarp();
                if (have) {
                    const int row = (blk * p.num_kv_heads + it.kvh) * kPage;
                    const void *tm = n & 1 ? static_cast<const void *>(&tmv) : &tmk;
#pragma unroll
                    for (int b = 0; b < kBoxes; ++b)
                        ptx::tma_load_2d(ring + s * kStageBytes + b * M::kHalfBytes +
                                             lane * (kPage * kBox * (kCodes ? 1 : 2)),
                                         tm, b * kBox, row, fb);
                }
                __syncwarp();
                issued = n + 1;
            }
            // leave no copy in flight: every stage that was issued has landed
            for (int n = max(0, issued - R); n < issued; ++n)
                ptx::mbar_wait_bounded(kCodes ? cfull(n % R) : full(n % R), (n / R) & 1,
                                       kWaitLimitNs);
        }
    } else {
        if constexpr (kCodes) {
            // ------------------------------------------------ codes to fp16
            fewer_registers<kKv>();
            constexpr int R = M::kCodeStages;
            constexpr int kCh = kD / 16;  // 16-byte chunks of codes per row
            const int tid = threadIdx.x - 384;
            for (int n = 0; n < 2 * nt; ++n) {
                if (!wait(cfull(n % R), (n / R) & 1) || !wait(empty(n % S), ((n / S) & 1) ^ 1))
                    break;
                const uint32_t src = base + M::kCodeRing + (n % R) * M::kCodeBytes;
                const uint32_t dst = base + M::kRing + (n % S) * M::kTileBytes;
                const int v0 = (it.ta + n / 2) * kPagesPerTile;
#pragma unroll
                for (int e = tid; e < kTile * kCh; e += kTile) {
                    const int row = e / kCh, ch = e % kCh;
                    const uint32_t sw = kD == 128 ? (ch ^ (row & 7)) : (ch ^ ((row >> 1) & 3));
                    uint4 w = ptx::lds128(src + row * kD + (sw << 4));
                    uint4 a, b;
                    if constexpr (kKv == kKvI8) {
                        w.x ^= 0x80808080u;
                        w.y ^= 0x80808080u;
                        w.z ^= 0x80808080u;
                        w.w ^= 0x80808080u;
                        a = make_uint4(ptx::i8pair_exact(w.x, 0x4140u), ptx::i8pair_exact(w.x, 0x4342u),
                                       ptx::i8pair_exact(w.y, 0x4140u), ptx::i8pair_exact(w.y, 0x4342u));
                        b = make_uint4(ptx::i8pair_exact(w.z, 0x4140u), ptx::i8pair_exact(w.z, 0x4342u),
                                       ptx::i8pair_exact(w.w, 0x4140u), ptx::i8pair_exact(w.w, 0x4342u));
                    } else {
                        a = make_uint4(ptx::e4m3x2_to_f16x2(w.x), ptx::e4m3x2_to_f16x2(w.x >> 16),
                                       ptx::e4m3x2_to_f16x2(w.y), ptx::e4m3x2_to_f16x2(w.y >> 16));
                        b = make_uint4(ptx::e4m3x2_to_f16x2(w.z), ptx::e4m3x2_to_f16x2(w.z >> 16),
                                       ptx::e4m3x2_to_f16x2(w.w), ptx::e4m3x2_to_f16x2(w.w >> 16));
                        if (n & 1) {
                            // rows of V that no row of the item sees
                            const int v = v0 + (row >> 4);
                            const uint32_t lv = v < it.visited ? it.live(it.real(v) * kPage) : 0u;
                            if (!(lv >> (row & 15) & 1u)) a = b = make_uint4(0, 0, 0, 0);
                        }
                    }
                    const uint32_t to = dst + (ch >> 2) * M::kHalfBytes + row * 128;
                    const int c0 = (2 * ch) & 7;
                    st_shared16(to + ((c0 ^ (row & 7)) << 4), a);
                    st_shared16(to + (((c0 + 1) ^ (row & 7)) << 4), b);
                }
                ptx::fence_proxy_async_smem();
                ptx::mbar_arrive(full(n % S));
                ptx::mbar_arrive(cempty(n % R));
            }
        }
    }
    __syncthreads();
    if (warp == 8) umma::dealloc(tmem, 512);
}

// Joins the key splits of every row: a warp per row, lanes along head_dim, the
// parts in their order.
//   out = sum_z 2^(m_z - M) acc_z / sum_z 2^(m_z - M) l_z,  M = max_z m_z
// A part with l < 0 (a bad block) makes the row zeros.  Rows that no sequence
// owns have no parts and are left alone.
constexpr int kJoinThreads = 256;

template <int kD>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ PrefillArgs p)
{
    constexpr int kC = kD / 32;
    const int lane = threadIdx.x & 31;
    const int64_t all = static_cast<int64_t>(p.num_tokens) * p.num_heads;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kJoinThreads / 32) + (threadIdx.x >> 5);
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    if (row >= all) return;
    const int tok = static_cast<int>(row / p.num_heads);
    const int seq = warp_search(p.num_seqs, tok, [&](int s) { return __ldg(p.query_starts + s); });
    if (seq < 0) return;
    SeqRows sr;
    sr.load(p.query_starts, p.context_lens, seq, p.num_tokens, p.ctx_cap);
    if (tok - sr.start >= sr.len) return;
    float m = -INFINITY;
    for (int z = lane; z < p.splits; z += 32) m = fmaxf(m, __ldcg(p.part_ml + z * all + row).x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float l = 0.f, acc[kC];
    bool bad = false;
#pragma unroll
    for (int c = 0; c < kC; ++c) acc[c] = 0.f;
    for (int z = 0; z < p.splits; ++z) {
        const float2 ml = __ldcg(p.part_ml + z * all + row);
        bad |= ml.y < 0.f;
        if (ml.y == 0.f) continue;  // no key seen (or no part: no accumulators)
        const float f = ptx::ex2(ml.x - m);
        l += f * ml.y;
        const float *a = p.part_acc + (z * all + row) * kD + lane * kC;
#pragma unroll
        for (int c = 0; c < kC; ++c) acc[c] += f * __ldcg(a + c);
    }
    const float f = bad || l == 0.f ? 0.f : 1.f / l;
    __half *dst = p.out + row * kD + lane * kC;
#pragma unroll
    for (int c = 0; c < kC; c += 2)
        *reinterpret_cast<__half2 *>(dst + c) =
            __floats2half2_rn(bad || l == 0.f ? 0.f : acc[c] * f,
                              bad || l == 0.f ? 0.f : acc[c + 1] * f);
}

// -------------------------------------------------------------------- host
struct PrefillCall {
    void *out;
    const void *query, *kpool, *vpool;
    const float *k_scales, *v_scales;
    int num_blocks;
    const int32_t *block_tables;
    int max_blocks_per_seq;
    const int32_t *query_starts, *context_lens;
    int max_context_len, num_tokens, num_seqs, num_heads, num_kv_heads, head_dim, block_size;
    float softmax_scale, logit_cap;
    int window;
    const float *slopes;
    const int32_t *prefix_lens;
    void *workspace;
    size_t workspace_bytes;
    int32_t *dev_status;
    void *stream;
};

struct Plan {
    int64_t units = 0;
    int splits = 1;
    size_t bytes = 0;
};

// Units of the batch and the number of key splits, from the sizes alone.  An
// SM works on one item at a time; a split costs it about three tiles' time
// (start, queries, epilogue) and the join about two.  The number of splits is
// the one with the smallest sum of waves * (tiles of a split + 3).
pkv_status plan_of(int num_tokens, int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                   int max_context_len, Plan *plan)
{
    if (num_tokens < 0 || num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
        max_context_len < 0 || num_heads % num_kv_heads != 0)
        return PKV_ERR_INVALID_ARG;
    if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
    const int64_t group = num_heads / num_kv_heads;
    plan->units = num_tokens * group / kRows + num_seqs;
    const int64_t items = plan->units * num_kv_heads;
    const int64_t tiles = (static_cast<int64_t>(max_context_len) + kTile - 1) / kTile + 1;
    if (plan->units > INT32_MAX || num_tokens * group + kRows > INT32_MAX ||
        items * kMaxSplits > INT32_MAX)
        return PKV_ERR_UNSUPPORTED;
    int64_t best = 0;
    plan->splits = 1;
    for (int z = 1; z <= kMaxSplits && z <= tiles; ++z) {
        const int64_t cost = (items * z + kSms - 1) / kSms * ((tiles + z - 1) / z + 3) + (z > 1 ? 2 : 0);
        if (z == 1 || cost < best) {
            best = cost;
            plan->splits = z;
        }
    }
    plan->bytes = plan->splits == 1 ? 0
                                    : static_cast<size_t>(plan->splits) * num_tokens * num_heads *
                                          (head_dim + 2) * sizeof(float);
    return PKV_OK;
}

template <int kKv, int kD, bool kMod>
pkv_status launch_prefill(const PrefillCall &c, const Plan &plan)
{
    using M = Smem<kKv, kD>;
    DeviceInfo di;
    if (!current_device_info(&di)) return PKV_ERR_CUDA;
    if (M::kAsk > static_cast<int>(di.max_smem_optin)) return PKV_ERR_UNSUPPORTED;
    auto kern = prefill_kernel<kKv, kD, kMod>;
    {
        static bool ready[64] = {};
        std::lock_guard<std::mutex> lock(g_cfg_mu);
        bool &r = ready[di.device & 63];
        if (!r) {
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, M::kAsk) !=
                cudaSuccess) {
                cudaGetLastError();
                return PKV_ERR_CUDA;
            }
            r = true;
        }
    }
    CUtensorMap tmk, tmv;
    const uint64_t rows = static_cast<uint64_t>(c.num_blocks) * c.num_kv_heads * kPage;
    const int elem = M::kCodes ? 1 : 2, box = M::kCodes ? kD : 64;
    const int swizzle = box * elem;
    if (!encode_tmap_2d(&tmk, c.kpool, elem, kD, rows, box, kPage, swizzle) ||
        !encode_tmap_2d(&tmv, c.vpool, elem, kD, rows, box, kPage, swizzle))
        return PKV_ERR_CUDA;
    PrefillArgs a;
    a.out = static_cast<__half *>(c.out);
    a.query = static_cast<const __half *>(c.query);
    a.block_tables = c.block_tables;
    a.query_starts = c.query_starts;
    a.context_lens = c.context_lens;
    a.k_scales = c.k_scales;
    a.v_scales = c.v_scales;
    a.slopes = c.slopes;
    a.prefix_lens = c.prefix_lens;
    a.part_acc = static_cast<float *>(c.workspace);
    a.part_ml = reinterpret_cast<float2 *>(
        a.part_acc + static_cast<size_t>(plan.splits) * c.num_tokens * c.num_heads * kD);
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
    a.window = c.window;
    a.splits = plan.splits;
    a.units = static_cast<int>(plan.units);
    a.scale_log2 = c.softmax_scale * 1.4426950408889634f;
    a.cap = c.logit_cap * 1.4426950408889634f;
    a.cap_inv = c.logit_cap > 0.f ? 1.f / a.cap : 0.f;

    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(plan.units * c.num_kv_heads * plan.splits));
    cfg.blockDim = dim3(prefill_threads<kKv>());
    cfg.dynamicSmemBytes = M::kAsk;
    cfg.stream = static_cast<cudaStream_t>(c.stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a, tmk, tmv);
    if (e == cudaSuccess && plan.splits > 1) {
        const int64_t all = static_cast<int64_t>(c.num_tokens) * c.num_heads;
        cfg.gridDim = dim3(static_cast<unsigned>((all + kJoinThreads / 32 - 1) / (kJoinThreads / 32)));
        cfg.blockDim = dim3(kJoinThreads);
        cfg.dynamicSmemBytes = 0;
        e = cudaLaunchKernelEx(&cfg, join_kernel<kD>, a);
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    return PKV_OK;
}

pkv_status prefill_entry(const PrefillCall &c, int kv)
{
    const bool codes = kv != kKvF16;
    if (!c.out || !c.query || !c.kpool || !c.vpool || !c.block_tables || !c.query_starts ||
        !c.context_lens)
        return PKV_ERR_INVALID_ARG;
    if (codes && (!c.k_scales || !c.v_scales)) return PKV_ERR_INVALID_ARG;
    if (c.num_blocks <= 0 || c.block_size <= 0 || c.max_blocks_per_seq < 0 || c.window < 0)
        return PKV_ERR_INVALID_ARG;
    if (!(fabsf(c.softmax_scale) <= 3.0e38f) || !(c.logit_cap >= 0.f) || c.logit_cap > 3.0e38f)
        return PKV_ERR_INVALID_ARG;
    Plan plan;
    const pkv_status st = plan_of(c.num_tokens, c.num_seqs, c.num_heads, c.num_kv_heads, c.head_dim,
                                  c.max_context_len, &plan);
    if (st != PKV_OK) return st;
    if (c.block_size != kPage) return PKV_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(c.num_blocks) * c.num_kv_heads * kPage > 0x7fffffffLL ||
        c.max_context_len > INT32_MAX - 4 * kTile)
        return PKV_ERR_UNSUPPORTED;
    if (!aligned(c.out, 16) || !aligned(c.query, 16) || !aligned(c.kpool, 16) ||
        !aligned(c.vpool, 16) || !aligned(c.block_tables, 4) || !aligned(c.query_starts, 4) ||
        !aligned(c.context_lens, 4) || !aligned(c.dev_status, 4) || !aligned(c.k_scales, 4) ||
        !aligned(c.v_scales, 4) || !aligned(c.slopes, 4) || !aligned(c.prefix_lens, 4))
        return PKV_ERR_MISALIGNED;
    if (c.num_tokens == 0 || c.num_seqs == 0) return PKV_OK;
    if (plan.bytes > 0 && (!c.workspace || c.workspace_bytes < plan.bytes)) return PKV_ERR_WORKSPACE;
    if (!aligned(c.workspace, 16)) return PKV_ERR_MISALIGNED;
    const bool mod = codes || c.logit_cap > 0.f || c.slopes || !(c.softmax_scale > 0.f);
    if (kv == kKvF8)
        return c.head_dim == 128 ? launch_prefill<kKvF8, 128, true>(c, plan)
                                 : launch_prefill<kKvF8, 64, true>(c, plan);
    if (kv == kKvI8)
        return c.head_dim == 128 ? launch_prefill<kKvI8, 128, true>(c, plan)
                                 : launch_prefill<kKvI8, 64, true>(c, plan);
    if (mod)
        return c.head_dim == 128 ? launch_prefill<kKvF16, 128, true>(c, plan)
                                 : launch_prefill<kKvF16, 64, true>(c, plan);
    return c.head_dim == 128 ? launch_prefill<kKvF16, 128, false>(c, plan)
                             : launch_prefill<kKvF16, 64, false>(c, plan);
}

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_paged_prefill_fp16(
    void *out, const void *query, const void *k_cache, const void *v_cache, int num_blocks,
    const int32_t *block_tables, int max_blocks_per_seq, const int32_t *query_starts,
    const int32_t *context_lens, int max_context_len, int num_tokens, int num_seqs, int num_heads,
    int num_kv_heads, int head_dim, int block_size, float softmax_scale, float logit_cap,
    int window, const float *slopes, const int32_t *prefix_lens, void *workspace,
    size_t workspace_bytes, int32_t *dev_status, void *stream)
{
    const pkv::PrefillCall c{out, query, k_cache, v_cache, nullptr, nullptr, num_blocks,
                             block_tables, max_blocks_per_seq, query_starts, context_lens,
                             max_context_len, num_tokens, num_seqs, num_heads, num_kv_heads,
                             head_dim, block_size, softmax_scale, logit_cap, window, slopes,
                             prefix_lens, workspace, workspace_bytes, dev_status, stream};
    return pkv::prefill_entry(c, pkv::kKvF16);
}

extern "C" pkv_status pkv_paged_prefill_int8(
    void *out, const void *query, const int8_t *k_codes, const int8_t *v_codes,
    const float *k_scales, const float *v_scales, int num_blocks,
    const int32_t *block_tables, int max_blocks_per_seq, const int32_t *query_starts,
    const int32_t *context_lens, int max_context_len, int num_tokens, int num_seqs, int num_heads,
    int num_kv_heads, int head_dim, int block_size, float softmax_scale, float logit_cap,
    int window, const float *slopes, const int32_t *prefix_lens, void *workspace,
    size_t workspace_bytes, int32_t *dev_status, void *stream)
{
    const pkv::PrefillCall c{out, query, k_codes, v_codes, k_scales, v_scales, num_blocks,
                             block_tables, max_blocks_per_seq, query_starts, context_lens,
                             max_context_len, num_tokens, num_seqs, num_heads, num_kv_heads,
                             head_dim, block_size, softmax_scale, logit_cap, window, slopes,
                             prefix_lens, workspace, workspace_bytes, dev_status, stream};
    return pkv::prefill_entry(c, pkv::kKvI8);
}

extern "C" pkv_status pkv_paged_prefill_fp8(
    void *out, const void *query, const uint8_t *k_codes, const uint8_t *v_codes,
    const float *k_scales, const float *v_scales, int num_blocks,
    const int32_t *block_tables, int max_blocks_per_seq, const int32_t *query_starts,
    const int32_t *context_lens, int max_context_len, int num_tokens, int num_seqs, int num_heads,
    int num_kv_heads, int head_dim, int block_size, float softmax_scale, float logit_cap,
    int window, const float *slopes, const int32_t *prefix_lens, void *workspace,
    size_t workspace_bytes, int32_t *dev_status, void *stream)
{
    const pkv::PrefillCall c{out, query, k_codes, v_codes, k_scales, v_scales, num_blocks,
                             block_tables, max_blocks_per_seq, query_starts, context_lens,
                             max_context_len, num_tokens, num_seqs, num_heads, num_kv_heads,
                             head_dim, block_size, softmax_scale, logit_cap, window, slopes,
                             prefix_lens, workspace, workspace_bytes, dev_status, stream};
    return pkv::prefill_entry(c, pkv::kKvF8);
}

extern "C" size_t pkv_prefill_workspace_size(int num_tokens, int num_seqs, int num_heads,
                                             int num_kv_heads, int head_dim, int max_context_len)
{
    pkv::Plan plan;
    if (pkv::plan_of(num_tokens, num_seqs, num_heads, num_kv_heads, head_dim, max_context_len,
                     &plan) != PKV_OK)
        return 0;
    return plan.bytes;
}
