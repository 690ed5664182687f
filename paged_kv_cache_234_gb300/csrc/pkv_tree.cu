// pkv_tree.cu -- attention of trees of drafted tokens over the paged cache: a
// token sees its sequence's context (window, visible prefix), its ancestors in
// the tree and itself, with the scores of the scored decode (tanh cap, bias by
// distance).
//
// For the token at position i (the context's length plus its depth), a key t at
// position p(t) and z = softmax_scale <q, K_t>:
//   z' = cap tanh(z / cap)  (cap > 0),   z'' = z' - slope[h] (i - p(t)),
//   out = sum over seen t of softmax(z'')_t V_t.
//
// Bound by memory: a tree has few rows (tokens times the heads of a kv head), and
// every cached key and value is read once for all of them.  So the keys are the
// long side of both products: per tile of 128 keys (eight pages)
//   S^T = K Q^T     (128 keys x N rows, fp32 in TMEM; K as it lies in the page)
//   P^T = 2^(S' - m)  (a thread per key, half of the rows each; fp16, to shared
//                    memory in the layout of a product's operand)
//   O^T += V^T P^T  (head_dim x N, fp32 in TMEM; V as it lies in the page)
// With rows as the N of the products, 32 rows take a quarter of the time of 128,
// and the exponentials of all rows are spread over all threads.  Since a row's
// scores lie across threads, its maximum is not taken for every tile: the
// exponentials are relative to a reference per row, and a tile whose scores
// exceed it by more than 2^6 (every row's first, hardly any other) makes all
// threads take the maxima and rescale sums and accumulators.  The probabilities
// enter the product with a factor 2^6, so up to that much smaller ones are normal
// fp16 numbers.  Sums, maxima and accumulators are fp32.
//
// The tiles of all (sequence, kv head) pairs form one line, which is cut into as
// many equal pieces as there are SMs: a CTA walks its piece, whatever the lengths
// of the sequences.  Where a cut lies inside a pair, the parts are joined by a
// second kernel.  Trees with more than N rows take a CTA for every N of them, side
// by side on the same piece, so that they read the same pages at the same time.
//
// Roles of the warps: 0-7 scores and rows, 8 issues the products, 9 and 11 the TMA
// loads of K and Q, and of V (a ring of tiles, K and V in turn), 10 the items.
// INT8 / FP8 pages land in a second ring, and further warps widen them exactly to
// fp16.  The K scale of a page multiplies its keys' scores.  Its V scale enters
// the exponent, 2^(S' + log2 v - m), so that the reference is that of the largest
// contribution p V, and the sums take the probability times 1 / v.
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include <mutex>
#include <type_traits>

#include "pkv_host.cuh"
#include "pkv_ptx.cuh"
#include "pkv_ragged.cuh"
#include "pkv_score.cuh"
#include "pkv_umma.cuh"
#include "pkv_wait.cuh"

namespace pkv {
namespace {

constexpr int kPage = 16;
constexpr int kTile = 128;      // keys per step
constexpr int kPagesPerTile = kTile / kPage;
constexpr int kKvF16 = 0, kKvI8 = 1, kKvF8 = 2;
constexpr int kSoftWarps = 8, kSoftThreads = 32 * kSoftWarps;
constexpr int kWidenWarps = 4;
constexpr int kSms = 152;       // GB300: pieces of the line of tiles
constexpr int kPieceTiles = 2;  // tiles of a piece at least
constexpr float kLift = 6.f;    // log2 factor of the probabilities
constexpr float kLazy = 6.f;    // log2 excess over the reference that is let be
constexpr float kNone = -3.0e38f;        // reference of a row that has seen nothing
constexpr float kLeastV = 0x1p-60f;      // V scales below (zero) count as this
constexpr int kParents = 1024;  // parents of a sequence kept in shared memory

struct TreeMeta {               // the part of an item that a piece ends in
    int tok, toks, head, heads, parts;
    int unused[3];
};

struct TreeArgs {
    __half *out;
    const int32_t *block_tables, *query_starts, *context_lens, *parents;
    const float *k_scales, *v_scales;
    const float *slopes;
    const int32_t *prefix_lens;
    float *part_acc;    // [2 CTAs][kN][head_dim]: the part a piece begins with, ends in
    float2 *part_ml;    // [2 CTAs][kN]: reference, sum
    TreeMeta *meta;     // [CTAs]
    int32_t *dev_status;
    int num_tokens, num_seqs, num_heads, num_kv_heads, group;
    int chunk, chunks;  // heads of a kv head per item (the group, at most 128), chunks of them
    int tokens;         // tokens per item
    int sides;          // CTAs side by side on a piece
    int pieces;
    int max_blocks_per_seq, num_blocks, ctx_cap, max_tree_len, window;
    float scale_log2, cap, cap_inv;
};

// ------------------------------------------------------------ shared memory
template <int kKv, int kD, int kN>
struct TreeSmem {
    static constexpr bool kCodes = kKv != kKvF16;
    static constexpr int kHalves = kD / 64;
    static constexpr int kHalfBytes = kTile * 128;             // 64 values of 128 keys
    static constexpr int kTileBytes = kHalves * kHalfBytes;
    static constexpr int kQHalfBytes = kN * 128;               // 64 values of the rows
    static constexpr int kPBytes = kN * kTile * 2;
    static constexpr int kPBufs = kN <= 32 ? 2 : 1;
    static constexpr int kCodeBytes = kTile * kD;
    static constexpr int kMore = 128 / kD;
    static constexpr int kStages = kMore * (kCodes ? (kN <= 32 ? 3 : 2) : (kN <= 32 ? 6 : 4));
    static constexpr int kCodeStages = kCodes ? kMore * (kN <= 32 ? 6 : 5) : 0;
    static constexpr int kP = kHalves * kQHalfBytes;
    static constexpr int kRing = kP + kPBufs * kPBytes;
    static constexpr int kCodeRing = kRing + kStages * kTileBytes;
    static constexpr int kCtl = kCodeRing + kCodeStages * kCodeBytes;
    static constexpr int kBars = 2 * kStages + 2 * kCodeStages + 13;
    static constexpr int kItems = (kCtl + 8 * kBars + 15) & ~15;
    static constexpr int kFlags = kItems + 2 * 80;
    static constexpr int kIssued = kFlags + 16;   // see drain_copies
    // scales [kScaleTiles][K, V][8 pages], written by the K warp ahead of its
    // arrival for the tile's K codes; the scores of the tile are behind that.  The
    // warp runs ahead by the elements of both rings and one that it holds, and the
    // scores lag behind the products by two tiles.
    static constexpr int kScaleTiles = 16;
    static_assert((kStages + kCodeStages + 1) / 2 + 3 <= kScaleTiles, "scales overwritten");
    static constexpr int kScales = kIssued + 16;
    static constexpr int kOff = kScales + (kCodes ? kScaleTiles * 2 * kPagesPerTile * 4 : 0);
    static constexpr int kMax = kOff + 4 * kN;      // a row's reference
    static constexpr int kFac = kMax + 4 * kN;      // factor of its sums; 1 / sum at the end
    static constexpr int kSlope = kFac + 4 * kN;
    static constexpr int kPos = kSlope + 4 * kN;
    static constexpr int kAt = kPos + 4 * kN;       // the row's place in the output, or -1
    static constexpr int kSums = kAt + 8 * kN;      // [4 quarters of the keys][kN]
    static constexpr int kMask = kSums + 16 * kN;   // [kN]: bits of the tile's 128 keys
    static constexpr int kLive = kMask + 16 * kN;   // [4 warps]: of all their rows
    static constexpr int kScan = kLive + 64;        // sums of the warps, where the piece begins
    static constexpr int kUp = kScan + 8 * 32;      // parents
    static constexpr int kBytes = kUp + 4 * kParents;
    // a second CTA on the SM would wait for TMEM: ask for more than half
    static constexpr int kAsk = kBytes > 120 * 1024 ? kBytes : 120 * 1024;
    static_assert(kAsk <= 227 * 1024, "shared memory of one CTA");
    static_assert(kRing % 1024 == 0 && kCodeRing % 1024 == 0, "swizzled tiles");
};

enum Role { kRoleRows, kRoleProducts, kRoleLoadK, kRoleLoadV, kRoleItems, kRoleWiden, kRoles };

// ------------------------------------------------------------------- items
// Keys of a sequence that some row sees: lo .. and below pre, as pages np1, a gap,
// the rest; `tiles` of 8 pages.
struct SeqKeys {
    int base, lo, pre, np1, gap, tiles;

    __device__ __forceinline__ void set(const TreeArgs &p, int ctx, int n, int prefix)
    {
        base = ctx - n;
        lo = p.window > 0 && base >= p.window ? base - p.window + 1 : 0;
        pre = min(max(prefix, 0), base);
        const int fp = lo / kPage;
        np1 = min((pre + kPage - 1) / kPage, fp);
        gap = fp - np1;
        tiles = ((ctx + kPage - 1) / kPage - gap + kPagesPerTile - 1) / kPagesPerTile;
    }
};

struct __align__(16) TreeItem {
    int seq, kvh;
    int tok, toks;              // first token (of the batch) and tokens of the item
    int head, heads;            // first query head, heads
    int row;                    // row of the first token in its sequence
    int start, n;               // first token of the sequence, its tokens
    int base, lo, pre;          // see SeqKeys
    int np1, gap, visited;      // visited: pages up to the item's last token
    int ta, nt;                 // tiles of keys: the first, how many; 0: no further item
    int part;                   // -1: the whole item; else part 0 or 1 of the CTA
    int unused[2];

    __device__ __forceinline__ int real(int v) const { return v + (v >= np1 ? gap : 0); }
};
static_assert(sizeof(TreeItem) == 80, "an item is 80 bytes of shared memory");

// ------------------------------------------------------------------ kernel
template <int kKv>
__host__ __device__ constexpr int tree_threads()
{
    return 32 * (kSoftWarps + 4 + (kKv == kKvF16 ? 0 : kWidenWarps));
}

// Registers: all threads are launched with 65536 / threads, rounded down to a
// multiple of 8 (fp16: 168 for 384 threads; codes: 128 for 512).  With 128 rows a
// thread holds 64 scores and 64 sums, and takes what the others give back.
template <int kKv, int kN>
__device__ __forceinline__ void soft_registers()
{
    if constexpr (kKv == kKvF16 && kN > 32) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    if constexpr (kKv != kKvF16 && kN > 32) asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
}

template <int kN>
__device__ __forceinline__ void issue_registers()
{
    if constexpr (kN > 32) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
}

template <int kN>
__device__ __forceinline__ void widen_registers()
{
    if constexpr (kN > 32) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
}

// Barriers of the score warps alone.
__device__ __forceinline__ void soft_sync()
{
    asm volatile("bar.sync 1, 256;" ::: "memory");
}

__device__ __forceinline__ bool soft_any(bool x)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(x ? 1u : 0u)
        : "memory");
    return r != 0;
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

__device__ __forceinline__ float log2_of(float x)
{
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// fp32 values in an order of their own as integers, and back.
__device__ __forceinline__ int ordered(float x)
{
    const int b = __float_as_int(x);
    return b ^ (b >> 31 & 0x7fffffff);
}

__device__ __forceinline__ float from_ordered(int b)
{
    return __int_as_float(b ^ (b >> 31 & 0x7fffffff));
}

// Eight codes as fp16 values, exactly.
template <int kKv>
__device__ __forceinline__ uint4 widen(uint32_t a, uint32_t b)
{
    if constexpr (kKv == kKvI8) {
        a ^= 0x80808080u;
        b ^= 0x80808080u;
        return make_uint4(ptx::i8pair_exact(a, 0x4140u), ptx::i8pair_exact(a, 0x4342u),
                          ptx::i8pair_exact(b, 0x4140u), ptx::i8pair_exact(b, 0x4342u));
    } else {
        return make_uint4(ptx::e4m3x2_to_f16x2(a), ptx::e4m3x2_to_f16x2(a >> 16),
                          ptx::e4m3x2_to_f16x2(b), ptx::e4m3x2_to_f16x2(b >> 16));
    }
}

// x <- tanh(x): u P(u^2) (see tanh_coef) where all of the warp's |u| <= 1, the
// exponential for what lies beyond.
template <int kC>
__device__ __forceinline__ void tanh_all(float (&x)[kC])
{
    float most = 0.f;
#pragma unroll
    for (int c = 0; c < kC; ++c) most = fmaxf(most, fabsf(x[c]));
    const bool near = __all_sync(0xffffffffu, most <= 1.f);
#pragma unroll
    for (int c = 0; c < kC; c += 2) {
        const uint64_t u = ptx::f32x2(x[c], x[c + 1]), w = ptx::mul2(u, u);
        uint64_t q = ptx::f32x2(tanh_coef(6), tanh_coef(6));
#pragma unroll
        for (int k = 5; k >= 0; --k) q = ptx::fma2(q, w, ptx::f32x2(tanh_coef(k), tanh_coef(k)));
        const float2 y = ptx::f32x2_parts(ptx::mul2(u, q));
        if (near) {
            x[c] = y.x;
            x[c + 1] = y.y;
        } else {
            x[c] = fabsf(x[c]) <= 1.f ? y.x : cap_far(x[c], 1.f);
            x[c + 1] = fabsf(x[c + 1]) <= 1.f ? y.y : cap_far(x[c + 1], 1.f);
        }
    }
}

// Sums of kC <= 32 columns over the lanes of the warp: afterwards v[0] of a lane is
// column lane * kC / 32's.
template <int kC>
__device__ __forceinline__ void lane_sums(float *v, int lane)
{
    int n = kC;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        if (n > 1) {
            n >>= 1;
            const bool up = lane & o;
#pragma unroll
            for (int i = 0; i < kC / 2; ++i)
                if (i < n) {
                    const float send = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
                }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
        }
    }
}

template <int kKv, int kD, int kN>
__global__ void __launch_bounds__(tree_threads<kKv>(), 1)
    tree_kernel(const __grid_constant__ TreeArgs p, const __grid_constant__ CUtensorMap tmq,
                const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv)
{
    using M = TreeSmem<kKv, kD, kN>;
    constexpr bool kCodes = M::kCodes;
    constexpr int S = M::kStages;
    constexpr int kC = kN / 2;          // rows of a score thread
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = ptx::smem_addr(smem);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    auto full = [&](int s) { return base + M::kCtl + 8 * s; };
    auto empty = [&](int s) { return base + M::kCtl + 8 * (S + s); };
    [[maybe_unused]] auto cfull = [&](int s) { return base + M::kCtl + 8 * (2 * S + s); };
    [[maybe_unused]] auto cempty = [&](int s) {
        return base + M::kCtl + 8 * (2 * S + M::kCodeStages + s);
    };
    const uint32_t one = base + M::kCtl + 8 * (2 * S + 2 * M::kCodeStages);
    const uint32_t q_full = one, q_empty = one + 8, drain = one + 16;
    // of tile number g of the CTA: scores there, probabilities there, product done
    auto s_full = [&](uint32_t g) { return one + 24 + 8 * (g & 1); };
    auto p_full = [&](uint32_t g) { return one + 40 + 8 * (g & 1); };
    auto pv_done = [&](uint32_t g) { return one + 56 + 8 * (g & 1); };
    auto i_full = [&](int k) { return one + 72 + 8 * (k & 1); };
    auto i_empty = [&](int k) { return one + 88 + 8 * (k & 1); };
    volatile int *flags = reinterpret_cast<volatile int *>(smem + M::kFlags);
    // flags: abort, bad block in item slot 0, in slot 1, TMEM address
    const Waiter waiter{flags, p.dev_status};
    // what was issued: K tiles, V tiles, items' queries
    volatile int *issued = reinterpret_cast<volatile int *>(smem + M::kIssued);
    auto item = [&](int k) -> TreeItem & {
        return *reinterpret_cast<TreeItem *>(smem + M::kItems + sizeof(TreeItem) * (k & 1));
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            ptx::mbar_init(full(s), kCodes ? kWidenWarps : 1);
            ptx::mbar_init(empty(s), 1);
        }
        for (int s = 0; s < M::kCodeStages; ++s) {
            ptx::mbar_init(cfull(s), 1);
            ptx::mbar_init(cempty(s), kWidenWarps);
        }
        ptx::mbar_init(q_full, 1);
        ptx::mbar_init(q_empty, 1);
        ptx::mbar_init(drain, 1);
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(s_full(i), 1);
            ptx::mbar_init(p_full(i), kSoftWarps);
            ptx::mbar_init(pv_done(i), 1);
            ptx::mbar_init(i_full(i), 1);
            ptx::mbar_init(i_empty(i), kSoftWarps + 3 + (kCodes ? kWidenWarps : 0));
        }
        ptx::fence_mbar_init();
        flags[0] = flags[1] = flags[2] = 0;
        issued[0] = issued[1] = issued[2] = 0;
        ptx::prefetch_tmap(&tmq);
        ptx::prefetch_tmap(&tmk);
        ptx::prefetch_tmap(&tmv);
    }
    if (warp == kSoftWarps) umma::alloc(base + M::kFlags + 12, 512);
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    // ------------------------------------------------ this CTA's piece of the line
    const int side = blockIdx.x % p.sides, piece = blockIdx.x / p.sides;
    int64_t *scan = reinterpret_cast<int64_t *>(smem + M::kScan);
    // tiles of a sequence, or 1 where it only gets zeros, or 0
    auto tiles_of = [&](int s, bool &zeros) -> int {
        SeqRows sr;
        const int first = __ldg(p.query_starts + s), end = __ldg(p.query_starts + s + 1);
        sr.set(first, end, __ldg(p.context_lens + s), p.num_tokens, p.ctx_cap);
        zeros = first != end && (!sr.ok || sr.len > p.max_tree_len);
        if (zeros || sr.len == 0) return sr.len > 0;
        SeqKeys k;
        k.set(p, sr.ctx, sr.len, p.prefix_lens ? __ldg(p.prefix_lens + s) : 0);
        return k.tiles;
    };
    const int per_tile = p.num_kv_heads * p.chunks;   // items of a sequence
    constexpr int kWarps = tree_threads<kKv>() / 32;
    const int seg = (p.num_seqs + 32 * kWarps - 1) / (32 * kWarps);
    int64_t own = 0;
    {
        bool any = false;
        const int s1 = min((static_cast<int>(threadIdx.x) + 1) * seg, p.num_seqs);
        for (int s = threadIdx.x * seg; s < s1; ++s) {
            bool zeros;
            own += static_cast<int64_t>(tiles_of(s, zeros)) * per_tile;
            any |= zeros;
        }
        if (any && blockIdx.x == 0 && p.dev_status)
            atomicOr(p.dev_status, static_cast<int32_t>(PKV_DEV_BAD_CTX));
    }
    int64_t sum = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
    }
    if (lane == 31) scan[warp] = sum;
    umma::fence_before();
    __syncthreads();
    umma::fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, static_cast<uint32_t>(flags[3]), 0);
    int64_t total = 0, before = sum - own;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += scan[w];
        total += scan[w];
    }
    const int64_t pieces = max(int64_t(1), min(int64_t(p.pieces), total / kPieceTiles));
    auto cut = [&](int64_t i) { return i < pieces ? total * i / pieces : total; };
    const int64_t begin = cut(piece), end = piece < pieces ? cut(piece + 1) : begin;
    if (begin < end && before <= begin && begin < before + own) {
        int64_t at = before;
        for (int s = threadIdx.x * seg;; ++s) {
            bool zeros;
            const int64_t here = static_cast<int64_t>(tiles_of(s, zeros)) * per_tile;
            if (begin < at + here) {
                scan[kWarps] = s;
                scan[kWarps + 1] = begin - at;
                break;
            }
            at += here;
        }
    }
    __syncthreads();

    auto t_s = [&](uint32_t g) { return tmem + kN * (g & 1); };   // S^T of tile g
    const uint32_t t_o = tmem + 2 * kN;                           // O^T

    if (warp < kSoftWarps) {
        // ------------------------------------------------ scores and rows
        soft_registers<kKv, kN>();
        const Waiter wait = waiter.as(kRoleRows);
        const int quad = warp & 3, key = 32 * quad + lane;   // of the tile
        const int c0 = warp / 4 * kC;                        // the thread's rows
        const uint32_t lanes = static_cast<uint32_t>(quad) << 21;   // TMEM lane 32 quad
        const int t = threadIdx.x;                           // the row that threads < kN look after
        const int vkey = t & (kTile - 1);                    // and the key, half of whose V
        float *off = reinterpret_cast<float *>(smem + M::kOff);   // kLift - reference
        float *ref = reinterpret_cast<float *>(smem + M::kMax);
        float *fac = reinterpret_cast<float *>(smem + M::kFac);
        float *slp = reinterpret_cast<float *>(smem + M::kSlope);
        float *posf = reinterpret_cast<float *>(smem + M::kPos);
        int64_t *place = reinterpret_cast<int64_t *>(smem + M::kAt);
        float *sums = reinterpret_cast<float *>(smem + M::kSums);
        uint32_t *mask = reinterpret_cast<uint32_t *>(smem + M::kMask);
        uint32_t *live = reinterpret_cast<uint32_t *>(smem + M::kLive);
        int *up = reinterpret_cast<int *>(smem + M::kUp);
        uint32_t g = 0;        // tiles of keys of the CTA so far
        bool fail = false;     // of this warp's waits; the warps leave together, at a barrier
        for (int k = 0;; ++k) {
            fail |= !wait(i_full(k), k >> 1 & 1);
            if (soft_any(fail)) break;
            const TreeItem &it = item(k);
            const int nt = it.nt;
            if (nt == 0) break;
            // the tree: every parent an earlier row
            const int32_t *par = p.parents + it.start;
            bool wrong = false;
            for (int j = t; j < it.n; j += kSoftThreads) {
                const int q = __ldg(par + j);
                wrong |= q < -1 || q >= j;
                if (j < kParents) up[j] = q;
            }
            const int rj = t / p.chunk, rh = t - rj * p.chunk;   // token and head of row t
            const bool mine = t < kN && rj < it.toks && rh < it.heads;
            if (t < kN) {
                // rows that are not the item's: a reference that nothing exceeds
                off[t] = mine ? kLift - kNone : -INFINITY;
                ref[t] = kNone;
                place[t] = mine ? static_cast<int64_t>(it.tok + rj) * p.num_heads + it.head + rh
                                : int64_t(-1);
            }
            const bool bad_tree = soft_any(wrong);
            if (bad_tree && t == 0 && p.dev_status)
                atomicOr(p.dev_status, static_cast<int32_t>(PKV_DEV_BAD_TREE));
            auto parent = [&](int j) { return j < kParents ? up[j] : __ldg(par + j); };
            const int node = mine && !bad_tree ? it.row + rj : -1;
            int pos = it.base;
            if ((p.window > 0 || p.slopes) && node >= 0)
                for (int j = parent(node); j >= 0; j = parent(j)) ++pos;
            const int lo = p.window > 0 ? max(pos - p.window + 1, 0) : 0;
            if (p.slopes) {
                if (t < kN) {
                    slp[t] = mine ? __ldg(p.slopes + it.head + rh) * 1.4426950408889634f : 0.f;
                    posf[t] = static_cast<float>(pos);
                }
                soft_sync();
            }
            float l[kC];
#pragma unroll
            for (int c = 0; c < kC; ++c) l[c] = 0.f;
            bool left = false;
            for (int j = 0; j < nt; ++j, ++g) {
                const int v0 = (it.ta + j) * kPagesPerTile;
                const int t0 = it.real(v0) * kPage;
                const int t1 = it.real(v0 + kPagesPerTile - 1) * kPage + kPage - 1;
                // whether all rows see all keys
                const bool clean = (t1 < it.base && (p.window <= 0 ||
                                                     it.base + it.n - 1 - t0 < p.window)) ||
                                   t1 < it.pre;
                bool dead = false;   // no row sees the key whose V this thread looks after
                if (!clean) {
                    // bits of the keys that row t sees
                    uint32_t w[4] = {0, 0, 0, 0};
                    if (t < kN) {
                        if (mine) {
#pragma unroll
                            for (int q = 0; q < kPagesPerTile; ++q) {
                                const int k0 = it.real(v0 + q) * kPage;
                                const uint32_t seen = (below(it.base - k0) & ~below(lo - k0)) |
                                                      below(it.pre - k0);
                                w[q >> 1] |= seen << (q & 1) * 16;
                            }
                            if (t1 >= it.base)
                                for (int a = node, far = 0;
                                     a >= 0 && (p.window <= 0 || far < p.window);
                                     a = parent(a), ++far) {
                                    const int at = it.base + a;   // behind the gap
                                    const int e = ((at >> 4) - it.gap - v0) * kPage + (at & 15);
                                    if (e < 0) break;
                                    const uint32_t bit = 1u << (e & 31);
                                    if (e < 32) w[0] |= bit;
                                    else if (e < 64) w[1] |= bit;
                                    else if (e < 96) w[2] |= bit;
                                    else if (e < kTile) w[3] |= bit;
                                }
                        }
                        *reinterpret_cast<uint4 *>(mask + 4 * t) =
                            make_uint4(w[0], w[1], w[2], w[3]);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const uint32_t any = __reduce_or_sync(0xffffffffu, w[q]);
                            if (lane == 0) live[4 * warp + q] = any;
                        }
                    }
                    soft_sync();
                    uint32_t any = 0;
#pragma unroll
                    for (int e = 0; e < kN / 32; ++e) any |= live[4 * e + (vkey >> 5)];
                    dead = !(any >> (vkey & 31) & 1u);
                }
                fail |= !wait(s_full(g), g >> 1 & 1);
                umma::fence_after();
                float x[kC];
                if constexpr (kC == 16) {
                    umma::ld16(t_s(g) + lanes + c0, x);
                } else {
#pragma unroll
                    for (int c = 0; c < kC; c += 32) umma::ld32(t_s(g) + lanes + c0 + c, x + c);
                }
                // what a product is multiplied with, log2 of the page's V scale, and
                // the scale's reciprocal
                float f = p.scale_log2;
                [[maybe_unused]] float lv = 0.f, rv = 1.f;
                if constexpr (kCodes) {
                    const float *sc = reinterpret_cast<const float *>(smem + M::kScales) +
                                      (g & (M::kScaleTiles - 1)) * 2 * kPagesPerTile + (key >> 4);
                    const float vs = sc[kPagesPerTile], vc = fmaxf(vs, kLeastV);
                    f *= sc[0];
                    lv = vs >= 0.f && vs < INFINITY ? log2_of(vc) : NAN;
                    rv = __frcp_rn(vc);
                }
                umma::wait_ld();
                const uint32_t *words = mask + 4 * c0 + quad;
                if (p.cap > 0.f || p.slopes) {
                    const float by = p.cap > 0.f ? f * p.cap_inv : f;
#pragma unroll
                    for (int c = 0; c < kC; ++c) x[c] *= by;
                    if (p.cap > 0.f) {
                        // (unseen keys and other rows have no say in how it is
                        // evaluated)
#pragma unroll
                        for (int c = 0; c < kC; ++c)
                            if (off[c0 + c] == -INFINITY ||
                                (!clean && !(words[4 * c] >> lane & 1u)))
                                x[c] = 0.f;
                        tanh_all(x);
#pragma unroll
                        for (int c = 0; c < kC; ++c) x[c] *= p.cap;
                    }
                    if (p.slopes) {
                        int at = it.real(v0 + (key >> 4)) * kPage + (key & 15);
                        if (at >= it.base && !bad_tree) {
                            const int a = at - it.base;
                            at = it.base;
                            if (a < it.n)
                                for (int b = parent(a); b >= 0; b = parent(b)) ++at;
                        }
                        const float af = static_cast<float>(at);
#pragma unroll
                        for (int c = 0; c < kC; ++c)
                            x[c] = fmaf(-slp[c0 + c], posf[c0 + c] - af, x[c]);
                    }
                    f = 1.f;
                }
                if constexpr (kCodes) {
#pragma unroll
                    for (int c = 0; c < kC; ++c) x[c] = fmaf(x[c], f, lv);
                    f = 1.f;
                }
                if (!clean) {
#pragma unroll
                    for (int c = 0; c < kC; ++c)
                        x[c] = words[4 * c] >> lane & 1u ? x[c] * f : -INFINITY;
                    f = 1.f;
                }
                float top = -INFINITY;
#pragma unroll
                for (int c = 0; c < kC; c += 4) {
                    const float4 o = *reinterpret_cast<const float4 *>(off + c0 + c);
                    top = fmaxf(fmaxf(top, fmaf(x[c], f, o.x)), fmaf(x[c + 1], f, o.y));
                    top = fmaxf(fmaxf(top, fmaf(x[c + 2], f, o.z)), fmaf(x[c + 3], f, o.w));
                }
                if (soft_any(fail || top > kLift + kLazy)) {
                    if (soft_any(fail)) {
                        left = true;
                        break;
                    }
                    // the rows' maxima over the tile
#pragma unroll
                    for (int c = 0; c < kC; c += 32) {
                        int kept = 0;
#pragma unroll
                        for (int e = 0; e < (kC < 32 ? kC : 32); ++e) {
                            const int most =
                                __reduce_max_sync(0xffffffffu, ordered(x[c + e] * f));
                            if (lane == e) kept = most;
                        }
                        if (lane < kC) sums[quad * kN + c0 + c + lane] = from_ordered(kept);
                    }
                    soft_sync();
                    if (t < kN) {
                        float m = ref[t];
#pragma unroll
                        for (int q = 0; q < 4; ++q) m = fmaxf(m, sums[q * kN + t]);
                        fac[t] = ptx::ex2(ref[t] - m);
                        ref[t] = m;
                        if (mine) off[t] = kLift - m;
                    }
                    soft_sync();
#pragma unroll
                    for (int c = 0; c < kC; ++c) l[c] *= fac[c0 + c];
                    if (j > 0) {
                        fail |= !wait(pv_done(g - 1), (g - 1) >> 1 & 1);
                        umma::fence_after();
#pragma unroll 1
                        for (int c = c0; c < c0 + kC; c += 16) {
                            float o[16];
                            umma::ld16(t_o + lanes + c, o);
                            umma::wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] *= fac[c + e];
                            umma::st16(t_o + lanes + c, reinterpret_cast<const uint32_t *>(o));
                        }
                        umma::wait_st();
                    }
                }
                // the probabilities' buffer was read by the product before
                const uint32_t was = g - M::kPBufs;
                if (g >= M::kPBufs) fail |= !wait(pv_done(was), was >> 1 & 1);
                if (__any_sync(0xffffffffu, dead)) {
                    // V rows of keys that no row sees may hold anything, NaN included
                    // (and are not loaded for pages past the last): zeros.  The product
                    // waits for this.  (The stage's element before this one has landed:
                    // it is K of a tile before, or V of one whose product is done.)
                    static_assert(S % 2 ? S >= 3 : S / 2 >= M::kPBufs, "phase of the stage");
                    const uint32_t n = 2 * g + 1;
                    fail |= !wait(full(n % S), (n / S) & 1);
                    const uint32_t row = base + M::kRing + (n % S) * M::kTileBytes + vkey * 128 +
                                         (t >> 7) * (kD == 128 ? M::kHalfBytes : 64);
                    if (dead)
#pragma unroll
                        for (int e = 0; e < (kD == 128 ? 8 : 4); ++e)
                            st_shared16(row + 16 * e, make_uint4(0, 0, 0, 0));
                }
                const uint32_t to = base + M::kP + (g % M::kPBufs) * M::kPBytes +
                                    c0 / 8 * (16 * kTile) + key * 16;
#pragma unroll
                for (int c = 0; c < kC; c += 8) {
                    uint32_t pk[4];
#pragma unroll
                    for (int e = 0; e < 8; e += 4) {
                        const float4 o = *reinterpret_cast<const float4 *>(off + c0 + c + e);
                        const float y0 = ptx::ex2(fmaf(x[c + e], f, o.x));
                        const float y1 = ptx::ex2(fmaf(x[c + e + 1], f, o.y));
                        const float y2 = ptx::ex2(fmaf(x[c + e + 2], f, o.z));
                        const float y3 = ptx::ex2(fmaf(x[c + e + 3], f, o.w));
                        l[c + e] = kCodes ? fmaf(y0, rv, l[c + e]) : l[c + e] + y0;
                        l[c + e + 1] = kCodes ? fmaf(y1, rv, l[c + e + 1]) : l[c + e + 1] + y1;
                        l[c + e + 2] = kCodes ? fmaf(y2, rv, l[c + e + 2]) : l[c + e + 2] + y2;
                        l[c + e + 3] = kCodes ? fmaf(y3, rv, l[c + e + 3]) : l[c + e + 3] + y3;
                        pk[e / 2] = pack2(y0, y1);
                        pk[e / 2 + 1] = pack2(y2, y3);
                    }
                    st_shared16(to + c / 8 * (16 * kTile), make_uint4(pk[0], pk[1], pk[2], pk[3]));
                }
                ptx::fence_proxy_async_smem();
                umma::fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(p_full(g));
            }
            if (left) break;
            // the rows' sums, the quarters of the keys in their order
            fail |= !wait(pv_done(g - 1), (g - 1) >> 1 & 1);
            umma::fence_after();
            if constexpr (kC == 16) {
                lane_sums<16>(l, lane);
                if ((lane & 1) == 0) sums[quad * kN + c0 + (lane >> 1)] = l[0];
            } else {
#pragma unroll
                for (int c = 0; c < kC; c += 32) {
                    lane_sums<32>(l + c, lane);
                    sums[quad * kN + c0 + c + lane] = l[c];
                }
            }
            if (soft_any(fail)) break;
            const bool bad = bad_tree || flags[1 + (k & 1)] != 0;
            const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + max(it.part, 0);
            if (t < kN) {
                const float a = sums[t] + sums[kN + t] + sums[2 * kN + t] + sums[3 * kN + t];
                fac[t] = a > 0.f ? 1.f / a : a;   // a row that saw nothing: zeros; NaN stays
                if (it.part >= 0) p.part_ml[slot * kN + t] = make_float2(ref[t], bad ? -1.f : a);
            }
            soft_sync();
            const int dim = kD == 128 ? key : 16 * quad + lane;   // M = 64 has 16 of 32 lanes
            const bool has = kD == 128 || lane < 16;
#pragma unroll 1
            for (int c = c0; c < c0 + kC; c += 16) {
                float o[16];
                umma::ld16(t_o + lanes + c, o);
                umma::wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int64_t row = place[c + e];
                    if (row < 0 || !has) continue;
                    if (it.part < 0)
                        p.out[row * kD + dim] = __float2half_rn(bad ? 0.f : o[e] * fac[c + e]);
                    else
                        p.part_acc[(slot * kN + c + e) * kD + dim] = o[e];
                }
            }
            // (the next item's first product into O waits for its probabilities,
            // which come after this)
            umma::fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(i_empty(k));
        }
    } else if (warp < kSoftWarps + 4) {
        issue_registers<kN>();
        if (warp == kSoftWarps) {
            // ------------------------------------------------ products
            const Waiter wait = waiter.as(kRoleProducts);
            if (umma::elect_one()) {
                constexpr uint32_t kQk = umma::f16_idesc(kTile, kN, false);
                constexpr uint32_t kPv = umma::f16_idesc(kD, kN, true) | umma::kAMn;
                const uint32_t q_lo = umma::desc_lo(base, 16);
                const uint32_t k_lo = umma::desc_lo(base + M::kRing, 16);
                const uint32_t v_lo = umma::desc_lo(base + M::kRing, M::kHalfBytes);
                auto qk = [&](uint32_t g) -> bool {   // S^T = K Q^T
                    const uint32_t n = 2 * g, s = n % S;
                    if (!wait.one(full(s), (n / S) & 1)) return false;
                    umma::fence_after();
                    const uint32_t a = k_lo + s * (M::kTileBytes >> 4);
#pragma unroll
                    for (int k = 0; k < kD / 16; ++k)
                        umma::mma_ss(
                            t_s(g),
                            umma::desc(a + (((k >> 2) * M::kHalfBytes + (k & 3) * 32) >> 4)),
                            umma::desc(q_lo + (((k >> 2) * M::kQHalfBytes + (k & 3) * 32) >> 4)),
                            kQk, k > 0);
                    umma::commit(s_full(g));
                    umma::commit(empty(s));
                    return true;
                };
                uint32_t g = 0;
                bool ok = true;
                for (int k = 0; ok; ++k) {
                    ok = wait.one(i_full(k), k >> 1 & 1);
                    if (!ok) break;
                    const int nt = item(k).nt;
                    if (nt == 0) break;
                    ok = wait.one(q_full, k & 1) && qk(g);
                    if (!ok) break;
                    if (nt == 1) umma::commit(q_empty);
                    for (int j = 0; j < nt; ++j, ++g) {
                        if (j + 1 < nt) {
                            ok = qk(g + 1);
                            if (!ok) break;
                            if (j + 2 == nt) umma::commit(q_empty);
                        }
                        const uint32_t n = 2 * g + 1, s = n % S;
                        ok = wait.one(p_full(g), g >> 1 & 1) && wait.one(full(s), (n / S) & 1);
                        if (!ok) break;
                        umma::fence_after();
                        const uint32_t a = v_lo + s * (M::kTileBytes >> 4);
                        const uint32_t b = base + M::kP + (g % M::kPBufs) * M::kPBytes;
#pragma unroll
                        for (int k2 = 0; k2 < kTile / 16; ++k2)   // O^T += V^T P^T
                            umma::mma_ss(t_o, umma::desc(a + k2 * (2048 >> 4)),
                                         umma::desc_plain(b + k2 * 256, 16 * kTile), kPv,
                                         j > 0 || k2 > 0);
                        umma::commit(pv_done(g));
                        umma::commit(empty(s));
                    }
                    if (ok) ptx::mbar_arrive(i_empty(k));
                }
                // nothing of this thread's is in flight after this
                umma::commit(drain);
                ptx::mbar_wait_bounded(drain, 0, kWaitLimitNs);
            }
            __syncwarp();
        } else if (warp == kSoftWarps + 1 || warp == kSoftWarps + 3) {
            // ------------------------------------------------ loads of Q and the pages
            // A lane per page looks its block up; one thread issues the copies, 2 KB
            // of a page each.
            constexpr int R = kCodes ? M::kCodeStages : S;
            constexpr int kBox = kCodes ? kD : 64;                       // values per box
            constexpr int kBoxes = kCodes ? 1 : M::kHalves;
            constexpr int kBoxBytes = kPage * kBox * (kCodes ? 1 : 2);
            constexpr int kStageBytes = kCodes ? M::kCodeBytes : M::kTileBytes;
            const uint32_t ring = base + (kCodes ? M::kCodeRing : M::kRing);
            const bool is_v = warp == kSoftWarps + 3;
            const Waiter wait = waiter.as(is_v ? kRoleLoadV : kRoleLoadK);
            const void *tm = is_v ? static_cast<const void *>(&tmv) : &tmk;
            uint32_t tiles = 0;   // tiles of keys so far: ring elements 2 tiles (+ 1)
            int queries = 0;      // items whose queries were asked for
            bool ok = true;
            for (int k = 0; ok; ++k) {
                ok = wait(i_full(k), k >> 1 & 1);
                if (!ok) break;
                const TreeItem &it = item(k);
                const int nt = it.nt;
                if (nt == 0) break;
                const int32_t *table =
                    p.block_tables + static_cast<int64_t>(it.seq) * p.max_blocks_per_seq;
                auto lookup = [&](int j) -> int32_t {  // block of the lane's page, -2: none
                    const int v = (it.ta + j) * kPagesPerTile + lane;
                    if (lane >= kPagesPerTile || v >= it.visited) return -2;
                    const int32_t b = __ldg(table + it.real(v));
                    return b >= 0 && b < p.num_blocks ? b : -1;
                };
                if (!is_v) {
                    // the queries: tokens x heads x 64 values, which land as the item's
                    // rows in their order (rows of heads that are not the item's, or
                    // behind the batch, do not count)
                    ok = wait(q_empty, (k & 1) ^ 1);
                    if (!ok) break;
                    if (umma::elect_one()) {
                        ptx::mbar_arrive_expect_tx(q_full, p.tokens * p.chunk * M::kHalves * 128);
#pragma unroll
                        for (int b = 0; b < M::kHalves; ++b)
                            ptx::tma_load_3d(base + b * M::kQHalfBytes, &tmq, b * 64, it.head,
                                             it.tok, q_full);
                    }
                    __syncwarp();
                    ++queries;
                }
                int32_t blk = lookup(0);
                for (int j = 0; j < nt; ++j) {
                    const uint32_t n = 2 * tiles + (is_v ? 1 : 0);
                    const int s = n % R;
                    const bool have = blk >= 0;
                    if (blk == -1) {
                        flags[1 + (k & 1)] = 1;
                        if (p.dev_status)
                            atomicOr(p.dev_status, static_cast<int32_t>(PKV_DEV_BAD_BLOCK));
                    }
                    [[maybe_unused]] float k_scale = 0.f, v_scale = 0.f;
                    if constexpr (kCodes)
                        if (have && !is_v) {
                            const int64_t at = static_cast<int64_t>(blk) * p.num_kv_heads + it.kvh;
                            k_scale = __ldg(p.k_scales + at);
                            v_scale = __ldg(p.v_scales + at);
                        }
                    const int row = (blk * p.num_kv_heads + it.kvh) * kPage;
                    const unsigned pages = __ballot_sync(0xffffffffu, have);
                    const uint32_t fb = kCodes ? cfull(s) : full(s);
                    const uint32_t eb = kCodes ? cempty(s) : empty(s);
                    if (j + 1 < nt) blk = lookup(j + 1);
                    ok = wait(eb, ((n / R) & 1) ^ 1);
                    if (!ok) break;
                    if constexpr (kCodes)
                        if (!is_v && lane < kPagesPerTile) {
                            float *to = reinterpret_cast<float *>(smem + M::kScales) +
                                        (tiles & (M::kScaleTiles - 1)) * 2 * kPagesPerTile + lane;
                            to[0] = k_scale;
                            to[kPagesPerTile] = v_scale;
                        }
                    __syncwarp();  // (the arrival is behind the flag and the scales)
                    if (umma::elect_one())
                        ptx::mbar_arrive_expect_tx(fb, __popc(pages) * kBoxes * kBoxBytes);
                    __syncwarp();
                    const uint32_t dst = ring + s * kStageBytes;
#pragma unroll
                    for (int q = 0; q < kPagesPerTile; ++q) {
                        const int y = __shfl_sync(0xffffffffu, row, q);
                        if ((pages >> q & 1u) && umma::elect_one()) {
#pragma unroll
                            for (int b = 0; b < kBoxes; ++b)
                                ptx::tma_load_2d(dst + b * M::kHalfBytes + q * kBoxBytes, tm,
                                                 b * kBox, y, fb);
                        }
                    }
                    __syncwarp();
                    ++tiles;
                }
                __syncwarp();
                if (ok && lane == 0) ptx::mbar_arrive(i_empty(k));
            }
            // what was issued, for the drain behind a wait that ran out
            if (lane == 0) {
                issued[is_v] = static_cast<int>(tiles);
                if (!is_v) issued[2] = queries;
            }
        } else {
            // ------------------------------------------------ the items of the piece
            const Waiter wait = waiter.as(kRoleItems);
            TreeMeta tail = {};
            bool ok = true;
            int k = 0;
            int64_t at = begin;
            int seq = 0;
            int64_t rest = 0;   // tiles of the sequence before `at`
            if (begin < end) {
                seq = static_cast<int>(scan[kWarps]);
                rest = scan[kWarps + 1];
            }
            for (; at < end && ok; ++seq, rest = 0) {
                bool zeros;
                const int tiles = tiles_of(seq, zeros);
                if (tiles == 0) continue;
                SeqRows sr;
                sr.load(p.query_starts, p.context_lens, seq, p.num_tokens, p.ctx_cap);
                TreeItem it;
                it.seq = seq;
                it.start = sr.start;
                it.n = sr.len;
                it.row = side * p.tokens;
                it.tok = sr.start + it.row;
                it.toks = min(p.tokens, sr.len - it.row);
                SeqKeys sk = {};
                if (!zeros)
                    sk.set(p, sr.ctx, sr.len, p.prefix_lens ? __ldg(p.prefix_lens + seq) : 0);
                it.base = sk.base;
                it.lo = sk.lo;
                it.pre = sk.pre;
                it.np1 = sk.np1;
                it.gap = sk.gap;
                it.visited = (sk.base + it.row + it.toks - 1) / kPage + 1 - sk.gap;
                for (int i = static_cast<int>(rest / tiles); i < per_tile && at < end && ok; ++i) {
                    it.ta = static_cast<int>(rest - static_cast<int64_t>(i) * tiles);
                    it.nt = static_cast<int>(min(static_cast<int64_t>(tiles - it.ta), end - at));
                    const int64_t stop = at + (tiles - it.ta);   // the item's end on the line
                    it.part = it.ta > 0 ? 0 : it.nt < tiles ? 1 : -1;
                    it.kvh = i / p.chunks;
                    const int c = i - it.kvh * p.chunks;
                    it.head = it.kvh * p.group + c * p.chunk;
                    it.heads = min(p.chunk, p.group - c * p.chunk);
                    at += it.nt;
                    rest += it.nt;
                    if (zeros) {
                        // (all of the sequence's rows, also beyond those of the sides)
                        if (side == 0)
                            for (int64_t e = lane; e < static_cast<int64_t>(sr.len) * it.heads *
                                                           (kD / 8);
                                 e += 32) {
                                const int64_t q = e / (kD / 8);
                                const int64_t tk = sr.start + q / it.heads;
                                if (tk < 0 || tk >= p.num_tokens) continue;
                                const int64_t row = tk * p.num_heads + it.head + q % it.heads;
                                reinterpret_cast<uint4 *>(p.out + row * kD)[e % (kD / 8)] =
                                    make_uint4(0, 0, 0, 0);
                            }
                        continue;
                    }
                    if (it.toks <= 0) continue;
                    if (it.part == 1) {
                        // pieces that the rest of the item lies in
                        int last = piece + 1;
                        while (cut(last + 1) < stop) ++last;
                        tail.tok = it.tok;
                        tail.toks = it.toks;
                        tail.head = it.head;
                        tail.heads = it.heads;
                        tail.parts = last - piece + 1;
                    }
                    ok = wait(i_empty(k), (k >> 1 & 1) ^ 1);
                    if (ok && lane == 0) {
                        item(k) = it;
                        flags[1 + (k & 1)] = 0;
                        ptx::mbar_arrive(i_full(k));
                    }
                    __syncwarp();
                    ++k;
                }
            }
            if (lane == 0) p.meta[blockIdx.x] = tail;
            if (ok) ok = wait(i_empty(k), (k >> 1 & 1) ^ 1);
            if (ok && lane == 0) {
                item(k).nt = 0;
                ptx::mbar_arrive(i_full(k));
            }
            __syncwarp();
        }
    } else {
        if constexpr (kCodes) {
            // ------------------------------------------------ codes to fp16
            widen_registers<kN>();
            const Waiter wait = waiter.as(kRoleWiden);
            constexpr int R = M::kCodeStages;
            constexpr int kCh = kD / 16;  // 16-byte chunks of codes per key
            constexpr int kStep = 32 * kWidenWarps / kCh;
            constexpr int kLoads = kTile / kStep;
            const int tid = threadIdx.x - 32 * (kSoftWarps + 4);
            const int ch = tid % kCh, row0 = tid / kCh;
            uint32_t n = 0;
            bool ok = true;
            for (int k = 0; ok; ++k) {
                ok = wait(i_full(k), k >> 1 & 1);
                if (!ok) break;
                const int nt = item(k).nt;
                if (nt == 0) break;
                for (int j = 0; j < 2 * nt; ++j, ++n) {
                    ok = wait(cfull(n % R), (n / R) & 1) && wait(empty(n % S), ((n / S) & 1) ^ 1);
                    if (!ok) break;
                    const uint32_t src = base + M::kCodeRing + (n % R) * M::kCodeBytes;
                    const uint32_t dst = base + M::kRing + (n % S) * M::kTileBytes;
                    // all loads first
                    uint4 w[kLoads];
#pragma unroll
                    for (int e = 0; e < kLoads; ++e) {
                        const int row = row0 + e * kStep;
                        const uint32_t sx = kD == 128 ? (ch ^ (row & 7)) : (ch ^ ((row >> 1) & 3));
                        w[e] = ptx::lds128(src + row * kD + (sx << 4));
                    }
#pragma unroll
                    for (int e = 0; e < kLoads; ++e) {
                        const int row = row0 + e * kStep;
                        const uint4 a = widen<kKv>(w[e].x, w[e].y);
                        const uint4 b = widen<kKv>(w[e].z, w[e].w);
                        const uint32_t to = dst + (ch >> 2) * M::kHalfBytes + row * 128;
                        const int cc = (2 * ch) & 7;
                        st_shared16(to + ((cc ^ (row & 7)) << 4), a);
                        st_shared16(to + (((cc + 1) ^ (row & 7)) << 4), b);
                    }
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        ptx::mbar_arrive(full(n % S));
                        ptx::mbar_arrive(cempty(n % R));
                    }
                }
                __syncwarp();
                if (ok && lane == 0) ptx::mbar_arrive(i_empty(k));
            }
        }
    }
    __syncthreads();
    if (flags[0]) {  // a wait ran out (the same for all: nobody waits any more)
        if (warp == kSoftWarps + 1)
            drain_copies<kCodes ? M::kCodeStages : S>(kCodes ? cfull(0) : full(0), q_full,
                                                      issued[0], issued[1], issued[2]);
        __syncthreads();
    }
    if (warp == kSoftWarps) umma::dealloc(tmem, 512);
}

// Joins the parts of the items that the cuts went through, a warp a row.
//   out = sum_z 2^(m_z - M) acc_z / sum_z 2^(m_z - M) l_z,  M = max_z m_z
// A part with l < 0 (a bad block or tree) makes the row zeros.
constexpr int kJoinWarps = 8;

template <int kD, int kN>
__global__ void __launch_bounds__(32 * kJoinWarps) tree_join_kernel(const __grid_constant__ TreeArgs p)
{
    constexpr int kC = kD / 32, kPer = (kSms + 31) / 32;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int owner = blockIdx.x / (kN / kJoinWarps);
    const int r = blockIdx.x % (kN / kJoinWarps) * kJoinWarps + warp;
    const TreeMeta meta = p.meta[owner];
    const int rj = r / p.chunk, rh = r - rj * p.chunk;
    if (meta.parts <= 0 || rj >= meta.toks || rh >= meta.heads) return;
    // part 0 is the owner's last one, the others are the first of the pieces behind
    auto at = [&](int z) -> int64_t {
        return (2 * (static_cast<int64_t>(owner) + static_cast<int64_t>(z) * p.sides) + (z == 0)) *
                   kN + r;
    };
    float pm[kPer], pl[kPer], m = kNone;
    bool bad = false;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        const int z = lane + 32 * e;
        const float2 ml = z < meta.parts ? __ldcg(p.part_ml + at(z)) : make_float2(kNone, 0.f);
        pm[e] = ml.x;
        pl[e] = ml.y;
        m = fmaxf(m, ml.x);
        bad |= ml.y < 0.f;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    bad = __any_sync(0xffffffffu, bad);
    float l = 0.f, acc[kC];
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        pm[e] = ptx::ex2(pm[e] - m);
        l += pm[e] * pl[e];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
#pragma unroll
    for (int c = 0; c < kC; ++c) acc[c] = 0.f;
#pragma unroll
    for (int e = 0; e < kPer; ++e)
#pragma unroll 1
        for (int z0 = 32 * e; z0 < meta.parts && z0 < 32 * e + 32; z0 += 8) {
            float v[8][kC];
#pragma unroll
            for (int u = 0; u < 8; ++u)
#pragma unroll
                for (int c = 0; c < kC; ++c) {
                    const int z = z0 + u;
                    v[u][c] = z < meta.parts ? __ldcg(p.part_acc + at(z) * kD + 32 * c + lane) : 0.f;
                }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const float f = __shfl_sync(0xffffffffu, pm[e], (z0 + u) & 31);
#pragma unroll
                for (int c = 0; c < kC; ++c) acc[c] += f * v[u][c];
            }
        }
    const bool zero = bad || l == 0.f;
    const int64_t row = static_cast<int64_t>(meta.tok + rj) * p.num_heads + meta.head + rh;
#pragma unroll
    for (int c = 0; c < kC; ++c)
        p.out[row * kD + 32 * c + lane] = __float2half_rn(zero ? 0.f : acc[c] / l);
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
    int rows = 0;              // of an item: 32 or 128
    int chunk = 0, chunks = 0, tokens = 0, sides = 0, pieces = 0;
    size_t bytes = 0;
};

// From the sizes alone.  32 rows to an item where no tree has more.
pkv_status tree_plan(int num_tokens, int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                     int max_context_len, int max_tree_len, TreePlan *plan)
{
    if (num_tokens < 0 || num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
        max_context_len < 0 || max_tree_len < 0 || num_heads % num_kv_heads != 0)
        return PKV_ERR_INVALID_ARG;
    if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
    const int group = num_heads / num_kv_heads;
    int tree = max_tree_len < num_tokens ? max_tree_len : num_tokens;
    if (tree < 1) tree = 1;
    plan->chunk = group < kTile ? group : kTile;
    plan->chunks = (group + plan->chunk - 1) / plan->chunk;
    plan->rows = static_cast<int64_t>(tree) * plan->chunk <= 32 ? 32 : 128;
    plan->tokens = plan->rows / plan->chunk;
    plan->sides = (tree - 1) / plan->tokens + 1;
    plan->pieces = plan->sides < kSms ? kSms / plan->sides : 1;
    const size_t ctas = static_cast<size_t>(plan->sides) * plan->pieces;
    plan->bytes = ctas * (2 * plan->rows * (head_dim + 2) * sizeof(float) + sizeof(TreeMeta));
    return PKV_OK;
}

template <int kKv, int kD, int kN>
pkv_status launch_tree(const TreeCall &c, const TreePlan &plan)
{
    using M = TreeSmem<kKv, kD, kN>;
    DeviceInfo di;
    if (!current_device_info(&di)) return PKV_ERR_CUDA;
    if (M::kAsk > static_cast<int>(di.max_smem_optin)) return PKV_ERR_UNSUPPORTED;
    auto kern = tree_kernel<kKv, kD, kN>;
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
    CUtensorMap tmq, tmk, tmv;
    const uint64_t rows = static_cast<uint64_t>(c.num_blocks) * c.num_kv_heads * kPage;
    const int elem = M::kCodes ? 1 : 2, box = M::kCodes ? kD : 64;
    if (!encode_tmap_3d_f16(&tmq, c.query, kD, c.num_heads, c.num_tokens, 64, plan.chunk,
                            plan.tokens) ||
        !encode_tmap_2d(&tmk, c.kpool, elem, kD, rows, box, kPage, box * elem) ||
        !encode_tmap_2d(&tmv, c.vpool, elem, kD, rows, box, kPage, box * elem))
        return PKV_ERR_CUDA;
    const int64_t ctas = static_cast<int64_t>(plan.sides) * plan.pieces;
    TreeArgs a;
    a.out = static_cast<__half *>(c.out);
    a.block_tables = c.block_tables;
    a.query_starts = c.query_starts;
    a.context_lens = c.context_lens;
    a.parents = c.parents;
    a.k_scales = c.k_scales;
    a.v_scales = c.v_scales;
    a.slopes = c.slopes;
    a.prefix_lens = c.prefix_lens;
    a.part_acc = static_cast<float *>(c.workspace);
    a.part_ml = reinterpret_cast<float2 *>(a.part_acc + 2 * ctas * kN * kD);
    a.meta = reinterpret_cast<TreeMeta *>(a.part_ml + 2 * ctas * kN);
    a.dev_status = c.dev_status;
    a.num_tokens = c.num_tokens;
    a.num_seqs = c.num_seqs;
    a.num_heads = c.num_heads;
    a.num_kv_heads = c.num_kv_heads;
    a.group = c.num_heads / c.num_kv_heads;
    a.chunk = plan.chunk;
    a.chunks = plan.chunks;
    a.tokens = plan.tokens;
    a.sides = plan.sides;
    a.pieces = plan.pieces;
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
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(tree_threads<kKv>());
    cfg.dynamicSmemBytes = M::kAsk;
    cfg.stream = static_cast<cudaStream_t>(c.stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a, tmq, tmk, tmv);
    if (e == cudaSuccess) {
        cfg.gridDim = dim3(static_cast<unsigned>(ctas * (kN / kJoinWarps)));
        cfg.blockDim = dim3(32 * kJoinWarps);
        cfg.dynamicSmemBytes = 0;
        e = cudaLaunchKernelEx(&cfg, tree_join_kernel<kD, kN>, a);
    }
    if (e != cudaSuccess) {
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
        c.max_context_len > INT32_MAX - 4 * kTile)
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
        if (c.head_dim == 128)
            return plan.rows == 32 ? launch_tree<kKv, 128, 32>(c, plan)
                                   : launch_tree<kKv, 128, 128>(c, plan);
        return plan.rows == 32 ? launch_tree<kKv, 64, 32>(c, plan)
                               : launch_tree<kKv, 64, 128>(c, plan);
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

#ifdef PKV_DEBUG
// Debug builds only: see WaitDebug (roles 0 rows, 1 products, 2 K and query loads, 3
// V loads, 4 items, 5 widening of codes).  A negative role resets its setting.
// Synchronises with the device; returns 0, or -1 if the CUDA runtime fails or an
// argument is out of range.
extern "C" __attribute__((visibility("default"))) int pkv_debug_set_tree(int give_role, int give_at,
                                                                         int slow_role, int slow_ns)
{
    if (give_role >= pkv::kRoles || slow_role >= pkv::kRoles || slow_ns < 0 || slow_ns > 1000000)
        return -1;
    const pkv::WaitDebug d = {give_role < 0 ? -2 : give_role, give_at,
                              slow_role < 0 ? -2 : slow_role, slow_ns};
    if (cudaDeviceSynchronize() != cudaSuccess ||
        cudaMemcpyToSymbol(pkv::g_wait_debug, &d, sizeof(d)) != cudaSuccess)
        return -1;
    return 0;
}
#endif
