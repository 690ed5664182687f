// pkv_tree.cuh -- attention of trees of drafted tokens over the paged cache: a
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
//   P^T = 2^(S' - m)  (a thread per key, in a group of them for every 16 rows; fp16, to
//                    shared memory in the layout of a product's operand)
//   O^T += V^T P^T  (head_dim x N, fp32 in TMEM; V as it lies in the page)
// With rows as the N of the products, 32 rows take a quarter of the time of 128,
// and the exponentials of all rows are spread over all threads.  Since a row's
// scores lie across threads, its maximum is not taken for every tile: the
// exponentials are relative to a reference per row, and a tile whose scores
// exceed it by more than 2^9 makes the group take the maxima, rescale sums and
// accumulators and work the tile out once more.  That is every row's first tile and
// hardly any other -- but with a bias by distance, under which the scores rise from
// tile to tile, nearly every tile of a head whose slope is above 0.05 (9 / (128
// log2 e)): 64 trees of 8 tokens over 2048 with the usual slopes take 132 us in fp16
// and 174 in INT8, without them 99 and 79.  The probabilities enter the product with a
// factor 2^6, so up to that much smaller ones are normal fp16 numbers, and the
// largest are 2^15.  Sums, maxima and accumulators are fp32.
//
// The tiles of all (sequence, kv head) pairs form one line, which is cut into as
// many equal pieces as there are SMs: a CTA walks its piece, whatever the lengths
// of the sequences.  Where a cut lies inside a pair, the parts are joined by a
// second kernel.  (Up to 64 rows per kv head; with more the rows are the long side:
// pkv_prefill_tree.cu.)
//
// Roles of the warps: four for every 16 rows work on scores and rows; of the next four
// one issues the products, two the TMA loads of K and Q, and of V (a ring of tiles, K
// and V in turn), one finds the items.
// INT8 / FP8 pages land in a ring of codes, and two teams of four warps widen them
// exactly to fp16: K, a thread per key, into TMEM, from where it is the A operand of
// its product without passing shared memory again; V into shared memory, where it lies
// as the pages' fp16 would.  The K scale of a page multiplies its keys' scores.  Its V
// scale enters the exponent, 2^(S' + log2 v - m), so that the reference is that of the
// largest contribution p V, and the sums take the probability times 1 / v.
//
// Measured back to back, 64 trees of 8 tokens over 2048 keys, 32 / 8 heads, head_dim 128:
// fp16 96 to 99 us, 81 to 84 % of the copy's rate; INT8 79 to 81, FP8 76 to 78 (51 to 54 %):
// there the score warps' chain
// and the widening (40 instructions for 32 codes) share the schedulers, which issue in
// 44 % of the cycles, and wait for instructions more than for any pipe.  One tree of 8
// over 131072: fp16 93, INT8 71, FP8 67 us.  Eight trees of 8 over 512, one head to a kv
// head, INT8: 13.4, latencies from the launch to the join one after the other.
#pragma once

#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include <mutex>
#include <type_traits>

#include "pkv_host.cuh"
#include "pkv_ptx.cuh"
#include "pkv_ragged.cuh"
#include "pkv_score.cuh"
#include "pkv_tree_call.h"
#include "pkv_umma.cuh"
#include "pkv_wait.cuh"

namespace pkv {
namespace {

constexpr int kPage = 16;
constexpr int kTile = 128;      // keys per step
constexpr int kPagesPerTile = kTile / kPage;
constexpr int kKvF16 = 0, kKvI8 = 1, kKvF8 = 2;
constexpr int kGroup = 128;     // threads that share rows: one per key of a tile
constexpr int kPieceTiles = 2;  // tiles of a piece at least
constexpr float kLift = 6.f;    // log2 factor of the probabilities
constexpr float kLazy = 9.f;    // log2 excess over the reference that is let be
static_assert(kLift + kLazy < 16.f, "probabilities up to 2^(kLift + kLazy) are finite in fp16");
constexpr float kNone = -3.0e38f;        // reference of a row that has seen nothing
// V scales below (zero) count as this.  A code is 448 at most, so what such a page adds
// to an output stays below 2^-51, nothing beside fp16's smallest number, 2^-24.
constexpr float kLeastV = 0x1p-60f;
constexpr float kGone = 110.f;           // log2 share beyond which older sums are nothing

// Score warps: a group of four, a thread per key, for every 16 rows.  A tile's chain
// (scores, exponentials, reference, product) has more waits than work, which groups
// with rows of their own and nothing to tell each other fill.  (32 rows to a group: 8
// tokens of 4 heads over 131072 INT8 keys took 93.6 us, with 16 78.8.)
constexpr int kRows = 16;       // of a group, and the columns of one TMEM access

__host__ __device__ constexpr int soft_warps(int rows)
{
    return 4 * (rows / kRows);
}

// Warps that widen codes: a team for K, a team for V.
constexpr int kTeam = 4;
__host__ __device__ constexpr int widen_warps(int kv)
{
    return kv == kKvF16 ? 0 : 2 * kTeam;
}

__host__ __device__ constexpr int tree_threads(int kv, int rows)
{
    return 32 * (soft_warps(rows) + 4 + widen_warps(kv));
}

struct TreeMeta {               // the part of an item that a piece ends in
    int start, n, kvh, parts;
};
static_assert(sizeof(TreeMeta) == kTreeMetaBytes, "what the plan counts");

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
    int tokens;         // tokens that an item's rows have room for
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
    static constexpr int kPBufs = 2;
    static constexpr int kCodeBytes = kTile * kD;
    static constexpr int kMore = 128 / kD;
    // fp16: K and V tiles in turn; codes: widened V tiles (widened K lies in TMEM), and
    // the codes of K and V in turn
    static constexpr int kStages =
        kMore * (kCodes ? 2 : kN <= 32 ? 6 : 5);
    static constexpr int kCodeStages = kCodes ? kMore * (kN <= 32 ? 8 : 6) : 0;
    static constexpr int kKBufs = 2;                           // widened K tiles
    // A waiting warp must not be two phases of a barrier off.  K and V have a producer
    // each, which has seen the element S + 2 before its next one given back and takes
    // for granted that the one 2 S before it was.  With an even number of stages these
    // are both K or both V.  With an odd one, V's producer has seen a K, whose product
    // follows the one with V of two tiles before: 5 stages will do, 3 will not.
    static_assert(kCodes || kStages % 2 == 0 || kStages >= 5, "phases of the ring");
    static_assert(kCodeStages % 2 == 0, "K and V codes in slots of their own");
    static constexpr int kP = kHalves * kQHalfBytes;
    static constexpr int kRing = kP + kPBufs * kPBytes;
    static constexpr int kCodeRing = kRing + kStages * kTileBytes;
    static constexpr int kCtl = kCodeRing + kCodeStages * kCodeBytes;
    static constexpr int kBars = 2 * kStages + 2 * kCodeStages + 15 + 2 * kKBufs;
    static constexpr int kItems = (kCtl + 8 * kBars + 15) & ~15;
    static constexpr int kFlags = kItems + 2 * 64;
    static constexpr int kIssued = kFlags + 32;   // see drain_copies
    // scales [kScaleTiles][3][8 pages], written by the K warp ahead of its arrival for
    // the tile's K codes and worked out by K's widening team (scales_at); the scores of
    // the tile are behind that.  The K warp runs ahead by the K tiles of its ring, the widened ones and one that it
    // holds, and the scores lag behind the products by two tiles.
    static constexpr int kScaleTiles = 16;
    static_assert(kCodeStages / 2 + kKBufs + 4 <= kScaleTiles, "scales overwritten");
    static constexpr int kScales = kIssued + 16;
    static constexpr int kOff = kScales + (kCodes ? kScaleTiles * 3 * kPagesPerTile * 4 : 0);
    static constexpr int kMax = kOff + 4 * kN;      // a row's reference
    static constexpr int kFac = kMax + 4 * kN;      // factor of its sums; 1 / sum at the end
    static constexpr int kOld = kFac + 4 * kN;      // kOff before the last change
    static constexpr int kSlope = kOld + 4 * kN;
    static constexpr int kAt = kSlope + 4 * kN;     // the row's place in the output, or -1
    static constexpr int kSums = kAt + 8 * kN;      // [4 quarters of the keys][kN]
    static constexpr int kMask = kSums + 16 * kN;   // [4 quarters of the keys][kN]: bits
    static constexpr int kUp = kMask + 16 * kN;     // [2 item slots][kN]: parents
    static constexpr int kBytes = kUp + 8 * kN;
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
    int start, n;               // first token of the sequence, its tokens
    int base, lo, pre;          // see SeqKeys
    int np1, gap, visited;      // visited: pages
    int ta, nt;                 // tiles of keys: the first, how many; 0: no further item
    int part;                   // -1: the whole item; else part 0 or 1 of the CTA
    int unused[3];

    __device__ __forceinline__ int real(int v) const { return v + (v >= np1 ? gap : 0); }
};
static_assert(sizeof(TreeItem) == 64, "an item is 64 bytes of shared memory");

// ------------------------------------------------------------------ kernel
// Registers: all threads are launched with 65536 / threads, rounded down to a
// multiple of 8 (72 for the 896 threads of codes with 64 rows).  The 512 score threads,
// which hold 16 scores and 16 sums, take what the other 384 give back.
template <int kKv, int kN>
__device__ __forceinline__ void soft_registers()
{
    if constexpr (kKv != kKvF16 && kN == 64) asm volatile("setmaxnreg.inc.sync.aligned.u32 80;");
}

template <int kKv, int kN>
__device__ __forceinline__ void other_registers()
{
    if constexpr (kKv != kKvF16 && kN == 64) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
}

// Barriers of a group of score warps alone.
__device__ __forceinline__ void group_sync(int i)
{
    asm volatile("bar.sync %0, 128;" ::"r"(i + 1) : "memory");
}

__device__ __forceinline__ bool group_any(int i, bool x)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(x ? 1u : 0u), "r"(i + 1)
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

// The same for bytes that this thread does not read, so that loads may pass it.
__device__ __forceinline__ void put_shared16(uint32_t addr, uint4 v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w));
}

__device__ __forceinline__ float log2_of(float x)
{
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The largest of the warp's values (NaN aside).
__device__ __forceinline__ float warp_max(float x)
{
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
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

// tanh(u) of two values as u P(u^2), P of degree 4 for |u| <= 0.5 or of degree 6 for
// |u| <= 1 (tanh_close, tanh_coef).
template <int kDegree>
__device__ __forceinline__ uint64_t tanh2(uint64_t u)
{
    auto coef = [](int k) { return kDegree == 4 ? tanh_close(k) : tanh_coef(k); };
    const uint64_t w = ptx::mul2(u, u);
    uint64_t q = ptx::f32x2(coef(kDegree), coef(kDegree));
#pragma unroll
    for (int k = kDegree - 1; k >= 0; --k) q = ptx::fma2(q, w, ptx::f32x2(coef(k), coef(k)));
    return ptx::mul2(u, q);
}

// x <- tanh(x), by the largest |x| of the warp: the short polynomial (the usual case:
// scores inside half the cap), the longer one, or the exponential for what lies
// beyond the cap.
template <int kC>
__device__ __forceinline__ void tanh_all(float (&x)[kC])
{
    float top[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < kC; c += 2)
        top[c / 2 & 1] = fmaxf(fmaxf(top[c / 2 & 1], fabsf(x[c])), fabsf(x[c + 1]));
    const float most = fmaxf(top[0], top[1]);
    if (__all_sync(0xffffffffu, most <= 0.5f)) {
#pragma unroll
        for (int c = 0; c < kC; c += 2) {
            const float2 y = ptx::f32x2_parts(tanh2<4>(ptx::f32x2(x[c], x[c + 1])));
            x[c] = y.x;
            x[c + 1] = y.y;
        }
    } else if (__all_sync(0xffffffffu, most <= 1.f)) {
#pragma unroll
        for (int c = 0; c < kC; c += 2) {
            const float2 y = ptx::f32x2_parts(tanh2<6>(ptx::f32x2(x[c], x[c + 1])));
            x[c] = y.x;
            x[c + 1] = y.y;
        }
    } else {
#pragma unroll
        for (int c = 0; c < kC; ++c) x[c] = cap_score(x[c], 1.f, 1.f);
    }
}

// Sums of kC columns over the lanes of the warp: afterwards v[0] of a lane is the
// column of its number, modulo kC.
template <int kC>
__device__ __forceinline__ void lane_sums(float (&v)[kC], int lane)
{
#pragma unroll
    for (int o = kC / 2; o > 0; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float send = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
#pragma unroll
    for (int o = kC; o < 32; o <<= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
}

template <int kKv, int kD, int kN>
__global__ void __launch_bounds__(tree_threads(kKv, kN), 1)
    tree_kernel(const __grid_constant__ TreeArgs p, const __grid_constant__ CUtensorMap tmq,
                const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv)
{
    using M = TreeSmem<kKv, kD, kN>;
    constexpr bool kCodes = M::kCodes;
    constexpr int S = M::kStages;
    constexpr int kGroups = kN / kRows;
    constexpr int kSoftWarps = soft_warps(kN);
    constexpr int kWidenWarps = widen_warps(kKv);
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
    auto t_full = [&](int k) { return one + 104 + 8 * (k & 1); };   // the item's tree is there
    // codes: widened K of tile number g there, read
    [[maybe_unused]] auto k_full = [&](uint32_t g) { return one + 120 + 8 * (g % M::kKBufs); };
    [[maybe_unused]] auto k_empty = [&](uint32_t g) {
        return one + 120 + 8 * (M::kKBufs + g % M::kKBufs);
    };
    volatile int *flags = reinterpret_cast<volatile int *>(smem + M::kFlags);
    // flags: abort, bad block in item slot 0, in slot 1, TMEM address, bad tree in slots
    const Waiter waiter{flags, p.dev_status};
    // what was issued: K tiles, V tiles, items' queries
    volatile int *issued = reinterpret_cast<volatile int *>(smem + M::kIssued);
    auto item = [&](int k) -> TreeItem & {
        return *reinterpret_cast<TreeItem *>(smem + M::kItems + sizeof(TreeItem) * (k & 1));
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            ptx::mbar_init(full(s), kCodes ? kTeam : 1);
            ptx::mbar_init(empty(s), 1);
        }
        for (int s = 0; s < M::kCodeStages; ++s) {
            ptx::mbar_init(cfull(s), 1);
            ptx::mbar_init(cempty(s), kTeam);
        }
        for (int i = 0; kCodes && i < M::kKBufs; ++i) {
            ptx::mbar_init(k_full(i), kTeam);
            ptx::mbar_init(k_empty(i), 1);
        }
        ptx::mbar_init(q_full, 1);
        ptx::mbar_init(q_empty, 1);
        ptx::mbar_init(drain, 1);
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(s_full(i), 1);
            ptx::mbar_init(p_full(i), kSoftWarps);
            ptx::mbar_init(pv_done(i), 1);
            ptx::mbar_init(i_full(i), 1);
            ptx::mbar_init(t_full(i), 1);
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
    umma::fence_before();
    __syncthreads();
    umma::fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, static_cast<uint32_t>(flags[3]), 0);
    // (each role waits for the work before this launch where it touches its data)
    ptx::griddep_launch_dependents();

    auto t_s = [&](uint32_t g) { return tmem + kN * (g & 1); };   // S^T of tile g
    const uint32_t t_o = tmem + 2 * kN;                           // O^T
    [[maybe_unused]] auto t_k = [&](uint32_t g) {                 // widened K
        return tmem + 4 * kN + kD / 2 * (g % M::kKBufs);
    };
    static_assert(4 * kN + kD / 2 * M::kKBufs <= 512, "columns of TMEM");

    // codes: of tile number g, a page's K scale times the softmax's, its V scale's log2
    // and reciprocal
    [[maybe_unused]] auto scales_at = [&](uint32_t g) {
        return reinterpret_cast<float *>(smem + M::kScales) +
               (g & (M::kScaleTiles - 1)) * 3 * kPagesPerTile;
    };

    if (warp < kSoftWarps) {
        // ------------------------------------------------ scores and rows
        soft_registers<kKv, kN>();
        const Waiter wait = waiter.as(kRoleRows);
        const int i = warp >> 2, quad = warp & 3;       // the group; its quarter of the keys
        const int key = threadIdx.x & (kGroup - 1);     // the thread's key of a tile
        const int c0 = i * kRows;                       // the group's rows
        const uint32_t lanes = static_cast<uint32_t>(quad) << 21;   // TMEM lane 32 quad
        // the row that a thread looks after, if key < kRows
        const int t = c0 + key;
        float *off = reinterpret_cast<float *>(smem + M::kOff);   // kLift - reference
        float *ref = reinterpret_cast<float *>(smem + M::kMax);
        float *fac = reinterpret_cast<float *>(smem + M::kFac);
        float *old = reinterpret_cast<float *>(smem + M::kOld);
        float *slp = reinterpret_cast<float *>(smem + M::kSlope);
        int64_t *place = reinterpret_cast<int64_t *>(smem + M::kAt);
        float *sums = reinterpret_cast<float *>(smem + M::kSums);
        uint32_t *mask = reinterpret_cast<uint32_t *>(smem + M::kMask);
        auto four = [](const float *v, int c) { return *reinterpret_cast<const float4 *>(v + c); };
        uint32_t g = 0;        // tiles of keys of the CTA so far
        bool fail = false;     // of this warp's waits; a group leaves together, at a barrier
        ptx::griddep_wait();
        for (int k = 0;; ++k) {
            fail |= !wait(i_full(k), k >> 1 & 1);
            const TreeItem &it = item(k);
            const int nt = it.nt, n = it.n, ctx = it.base, pre = it.pre, np1 = it.np1, gap = it.gap;
            const int ta = it.ta, part = it.part;
            auto real = [&](int v) { return v + (v >= np1 ? gap : 0); };
            const int rj = t / p.group, rh = t - rj * p.group;   // token and head of row t
            const bool mine = key < kRows && rj < n;
            const int head = it.kvh * p.group + rh;
            if (key < kRows && nt > 0) {
                // rows that are not the item's: a reference that nothing exceeds
                off[t] = mine ? kLift - kNone : -INFINITY;
                ref[t] = kNone;
                place[t] = mine ? static_cast<int64_t>(it.start + rj) * p.num_heads + head
                                : int64_t(-1);
                if (p.slopes)
                    slp[t] = mine && !fail ? __ldg(p.slopes + head) * 1.4426950408889634f : 0.f;
            }
            fail |= !wait(t_full(k), k >> 1 & 1);
            if (group_any(i, fail)) break;
            if (nt == 0) break;
            const bool bad_tree = flags[4 + (k & 1)] != 0;
            const int *up = reinterpret_cast<const int *>(smem + M::kUp) + kN * (k & 1);
            const int node = mine && !bad_tree ? rj : -1;
            int lo = 0;
            if (p.window > 0) {
                int pos = ctx;
                if (node >= 0)
                    for (int j = up[node]; j >= 0; j = up[j]) ++pos;
                lo = max(pos - p.window + 1, 0);
            }
            // whether some rows of the group are not the item's
            const bool ragged = c0 + kRows > n * p.group;
            // all rows see all keys of the tiles (of 8 pages) clean_a <= t < clean_b, which
            // lie behind the gap, and t < clean_p, in the prefix
            const int late = ctx + n - 1 - p.window;   // the deepest row sees what is behind
            const int first = p.window > 0 && late >= 0 ? late / kPage + 1 - gap : 0;
            const int clean_a = (max(first, gap ? np1 : 0) + kPagesPerTile - 1) / kPagesPerTile;
            const int clean_b = max(ctx / kPage - gap, 0) / kPagesPerTile;
            const int clean_p = (gap ? min(pre / kPage, np1) : pre / kPage) / kPagesPerTile;
            const bool plain = !(p.cap > 0.f) && !p.slopes;
            bool left = false;
            float l[kRows];   // the thread's shares of the rows' sums
#pragma unroll
            for (int e = 0; e < kRows; ++e) l[e] = 0.f;
            for (int j = 0; j < nt; ++j) {
                const int v0 = (ta + j) * kPagesPerTile;
                const bool clean = (ta + j >= clean_a && ta + j < clean_b) || ta + j < clean_p;
                const int at = real(v0 + (key >> 4)) * kPage + (key & 15);   // the key's slot
                if (!clean) {
                    // bits of the keys that row t sees
                    if (key < kRows) {
                        uint32_t w[4] = {0, 0, 0, 0};
                        if (mine) {
#pragma unroll
                            for (int q = 0; q < kPagesPerTile; ++q) {
                                const int k0 = real(v0 + q) * kPage;
                                const uint32_t seen =
                                    (below(ctx - k0) & ~below(lo - k0)) | below(pre - k0);
                                w[q >> 1] |= seen << (q & 1) * 16;
                            }
                            if (real(v0 + kPagesPerTile) * kPage > ctx)
                                for (int a = node, far = 0;
                                     a >= 0 && (p.window <= 0 || far < p.window);
                                     a = up[a], ++far) {
                                    const int e = ((ctx + a) >> 4 << 4) - (gap + v0) * kPage +
                                                  ((ctx + a) & 15);   // (behind the gap)
                                    if (e < 0) break;
                                    const uint32_t bit = 1u << (e & 31);
                                    if (e < 32) w[0] |= bit;
                                    else if (e < 64) w[1] |= bit;
                                    else if (e < 96) w[2] |= bit;
                                    else if (e < kTile) w[3] |= bit;
                                }
                        }
#pragma unroll
                        for (int q = 0; q < 4; ++q) mask[q * kN + t] = w[q];
                    }
                    group_sync(i);
                }
                float far = 0.f;   // p(t) - ctx
                if (p.slopes) {
                    int d = at - ctx;
                    if (d >= 0 && !bad_tree) {
                        int b = d < n ? up[d] : -1;
                        for (d = 0; b >= 0; b = up[b]) ++d;
                    }
                    far = static_cast<float>(d);
                }
                fail |= !wait(s_full(g), g >> 1 & 1);
                umma::fence_after();
                // what a product is multiplied with, log2 of the page's V scale, and
                // the scale's reciprocal
                float f0 = p.scale_log2;
                [[maybe_unused]] float lv = 0.f, rv = 1.f;
                if constexpr (kCodes) {
                    const float *sc = scales_at(g) + (key >> 4);
                    f0 = sc[0];
                    lv = sc[kPagesPerTile];
                    rv = sc[2 * kPagesPerTile];
                }
                const uint64_t rv2 = ptx::f32x2(rv, rv);
                const uint32_t *words = mask + quad * kN;
                const uint32_t to = base + M::kP + (g % M::kPBufs) * M::kPBytes + key * 16;
                // The scores x of the tile, which times f are in log2 units.
                auto scores = [&](float (&x)[kRows], float &f, auto simple) {
                    constexpr bool kSimple = decltype(simple)::value;
                    umma::ld16(t_s(g) + lanes + c0, x);
                    umma::wait_ld();
                    f = f0;
                    auto scale_all = [&](float by, float add) {
                        const uint64_t b2 = ptx::f32x2(by, by), a2 = ptx::f32x2(add, add);
#pragma unroll
                        for (int e = 0; e < kRows; e += 2) {
                            const float2 y =
                                ptx::f32x2_parts(ptx::fma2(ptx::f32x2(x[e], x[e + 1]), b2, a2));
                            x[e] = y.x;
                            x[e + 1] = y.y;
                        }
                    };
                    // x of the keys that a row does not see
                    auto hide = [&](float value) {
#pragma unroll
                        for (int e = 0; e < kRows; e += 4) {
                            const uint4 w = *reinterpret_cast<const uint4 *>(words + c0 + e);
                            if (!(w.x >> lane & 1u)) x[e] = value;
                            if (!(w.y >> lane & 1u)) x[e + 1] = value;
                            if (!(w.z >> lane & 1u)) x[e + 2] = value;
                            if (!(w.w >> lane & 1u)) x[e + 3] = value;
                        }
                    };
                    if constexpr (!kSimple) {
                        if (p.cap > 0.f) {
                            scale_all(f * p.cap_inv, 0.f);
                            f = p.cap;
                            // (unseen keys and other rows have no say in how it is
                            // evaluated)
                            if (!clean) hide(0.f);
                            if (ragged) {
#pragma unroll
                                for (int e = 0; e < kRows; e += 4) {
                                    const float4 o = four(off, c0 + e);
                                    if (o.x == -INFINITY) x[e] = 0.f;
                                    if (o.y == -INFINITY) x[e + 1] = 0.f;
                                    if (o.z == -INFINITY) x[e + 2] = 0.f;
                                    if (o.w == -INFINITY) x[e + 3] = 0.f;
                                }
                            }
                            tanh_all(x);
                        }
                    }
                    if (kCodes || !kSimple) {
                        scale_all(f, lv);
                        f = 1.f;
                    }
                    if constexpr (!kSimple) {
                        if (p.slopes) {
                            // slope (p(t) - ctx): what a row's own position adds is the same
                            // for all of its keys, and the softmax does not see it
#pragma unroll
                            for (int e = 0; e < kRows; e += 4) {
                                const float4 s = four(slp, c0 + e);
                                x[e] = fmaf(s.x, far, x[e]);
                                x[e + 1] = fmaf(s.y, far, x[e + 1]);
                                x[e + 2] = fmaf(s.z, far, x[e + 2]);
                                x[e + 3] = fmaf(s.w, far, x[e + 3]);
                            }
                        }
                        if (!clean) hide(-INFINITY);
                    }
                };
                // x f - reference + kLift of two rows
                auto exponents = [](const float (&x)[kRows], float f, int e, float a, float b) {
                    return ptx::f32x2_parts(ptx::fma2(ptx::f32x2(x[e], x[e + 1]), ptx::f32x2(f, f),
                                                      ptx::f32x2(a, b)));
                };
                // The probabilities, by the references as they are: into shared memory, and
                // into the sums.  Returns the largest exponent.
                auto probabilities = [&](auto simple) -> float {
                    float top = -INFINITY, x[kRows], f;
                    uint32_t pk[kRows / 2];
                    scores(x, f, simple);
#pragma unroll
                    for (int e = 0; e < kRows; e += 4) {
                        const float4 o = four(off, c0 + e);
#pragma unroll
                        for (int q = 0; q < 4; q += 2) {
                            const float2 z = q == 0 ? exponents(x, f, e, o.x, o.y)
                                                    : exponents(x, f, e + 2, o.z, o.w);
                            top = max3(top, z.x, z.y);
                            const float2 y = make_float2(ptx::ex2(z.x), ptx::ex2(z.y));
                            const uint64_t y2 = ptx::f32x2(y.x, y.y);
                            const uint64_t l2 = ptx::f32x2(l[e + q], l[e + q + 1]);
                            const float2 s = ptx::f32x2_parts(kCodes ? ptx::fma2(y2, rv2, l2)
                                                                     : ptx::add2(l2, y2));
                            l[e + q] = s.x;
                            l[e + q + 1] = s.y;
                            pk[(e + q) / 2] = pack2(y.x, y.y);
                        }
                    }
                    // (the buffer was read by the product before)
                    const uint32_t was = g - M::kPBufs;
                    if (g >= M::kPBufs) fail |= !wait(pv_done(was), was >> 1 & 1);
#pragma unroll
                    for (int e = 0; e < kRows; e += 8)
                        put_shared16(to + (c0 + e) / 8 * (16 * kTile),
                                     make_uint4(pk[e / 2], pk[e / 2 + 1], pk[e / 2 + 2],
                                                pk[e / 2 + 3]));
                    return top;
                };
                // New references: the rows' maxima over the tile, where these are above.
                auto references = [&]() {
                    float x[kRows], f;
                    scores(x, f, std::false_type());
#pragma unroll
                    for (int e = 0; e < kRows; e += 4) {
                        const float4 m = make_float4(warp_max(x[e] * f), warp_max(x[e + 1] * f),
                                                     warp_max(x[e + 2] * f), warp_max(x[e + 3] * f));
                        if (lane == 0) *reinterpret_cast<float4 *>(sums + quad * kN + c0 + e) = m;
                    }
                    group_sync(i);
                    if (key < kRows) {
                        float m = ref[t];
#pragma unroll
                        for (int q = 0; q < 4; ++q) m = fmaxf(m, sums[q * kN + t]);
                        fac[t] = ptx::ex2(ref[t] - m);
                        ref[t] = m;
                        old[t] = off[t];
                        if (mine) off[t] = kLift - m;
                    }
                    group_sync(i);
                };
                // What the probabilities added to the sums is taken off again, and sums and
                // accumulators follow the new references.  What was added may be beyond fp32,
                // as y or as y / v: where either is above 2^kGone, the sum so far is nothing
                // beside it (2^(kLift + kLazy) / kLeastV a key at most: 2^75) and is dropped.
                // Else both are finite, the reference grows by 2^kLazy at least, and with it
                // the rounding of a sum that held too much goes below the sum's own.
                auto follow = [&]() {
                    float x[kRows], f;
                    scores(x, f, std::false_type());
#pragma unroll
                    for (int e = 0; e < kRows; e += 2) {
                        const float2 z = exponents(x, f, e, old[c0 + e], old[c0 + e + 1]);
                        const float a = fmaf(-ptx::ex2(z.x), rv, l[e]);
                        const float b = fmaf(-ptx::ex2(z.y), rv, l[e + 1]);
                        l[e] = fmaxf(z.x, z.x - lv) > kGone ? 0.f : a * fac[c0 + e];
                        l[e + 1] = fmaxf(z.y, z.y - lv) > kGone ? 0.f : b * fac[c0 + e + 1];
                    }
                    fail |= !wait(pv_done(g - 1), (g - 1) >> 1 & 1);
                    umma::fence_after();
                    float o[kRows];
                    umma::ld16(t_o + lanes + c0, o);
                    umma::wait_ld();
#pragma unroll
                    for (int e = 0; e < kRows; ++e) o[e] *= fac[c0 + e];
                    umma::st16(t_o + lanes + c0, reinterpret_cast<const uint32_t *>(o));
                    umma::wait_st();
                };
                // In an item's first tile the references come first, so that its
                // probabilities hold; later an exponent too far above its reference makes
                // the tile's be worked out once more.
                if (j == 0) references();
                const float top = clean && plain ? probabilities(std::true_type())
                                                 : probabilities(std::false_type());
                if (group_any(i, fail || (j > 0 && top > kLift + kLazy))) {
                    left = group_any(i, fail);
                    if (left) break;
                    references();
                    follow();
                    probabilities(std::false_type());
                    // (the next tile's masks are written ahead of any barrier: behind
                    // the other warps' use of this one's)
                    if (!clean) group_sync(i);
                }
                if (!clean) {
                    // V rows of keys that no row of the tree sees may hold anything, NaN
                    // included (and are not loaded for pages past the item's last):
                    // zeros.  The product waits for all groups, which take turns.
                    const bool dead = v0 + (key >> 4) >= it.visited || at >= ctx + n ||
                                      (at < it.lo && at >= pre);
                    if (__any_sync(0xffffffffu, dead)) {
                        // (the stage's element before this one must have landed: it is K
                        // of a tile before, or V of one whose product is done)
                            static_assert(kCodes ? S >= M::kPBufs
                                                 : S % 2 ? S >= 3 : S / 2 >= M::kPBufs,
                                          "phase of the stage");
                            const uint32_t e = kCodes ? g : 2 * g + 1;
                        fail |= !wait(full(e % S), (e / S) & 1);
                        const uint32_t row =
                            base + M::kRing + (e % S) * M::kTileBytes + key * 128;
                        if (dead)
#pragma unroll 1
                            for (int b = i; b < kD / 8; b += kGroups)
                                st_shared16(row + (b >> 3) * M::kHalfBytes + (b & 7) * 16,
                                            make_uint4(0, 0, 0, 0));
                    }
                }
                ptx::fence_proxy_async_smem();
                umma::fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(p_full(g));
                ++g;
            }
            if (left) break;
            // the rows' sums, the quarters of the keys in their order
            fail |= !wait(pv_done(g - 1), (g - 1) >> 1 & 1);
            umma::fence_after();
            lane_sums(l, lane);
            if (lane < kRows) sums[quad * kN + c0 + lane] = l[0];
            if (group_any(i, fail)) break;
            const bool bad = bad_tree || flags[1 + (k & 1)] != 0;
            const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + max(part, 0);
            if (key < kRows) {
                const float a = sums[t] + sums[kN + t] + sums[2 * kN + t] + sums[3 * kN + t];
                fac[t] = a > 0.f ? 1.f / a : a;   // a row that saw nothing: zeros; NaN stays
                if (part >= 0) p.part_ml[slot * kN + t] = make_float2(ref[t], bad ? -1.f : a);
            }
            group_sync(i);
            const int dim = kD == 128 ? key : 16 * quad + lane;   // M = 64 has 16 of 32 lanes
            const bool has = kD == 128 || lane < 16, odd = lane & 1;
            float o[kRows];
            umma::ld16(t_o + lanes + c0, o);
            umma::wait_ld();
            if (part < 0) {
                // two neighbouring values of a row to a lane: even lanes store row e, odd
                // ones row e + 1
#pragma unroll
                for (int e = 0; e < kRows; e += 2) {
                    const float a = bad ? 0.f : o[e] * fac[c0 + e];
                    const float b = bad ? 0.f : o[e + 1] * fac[c0 + e + 1];
                    const float y = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
                    const int64_t row = place[c0 + e + odd];
                    if (row >= 0 && has)
                        *reinterpret_cast<uint32_t *>(p.out + row * kD + (dim & ~1)) =
                            odd ? pack2(y, b) : pack2(a, y);
                }
            } else if (has) {
#pragma unroll
                for (int e = 0; e < kRows; ++e)
                    if (place[c0 + e] >= 0) p.part_acc[(slot * kN + c0 + e) * kD + dim] = o[e];
            }
            // (the next item's first product into O waits for its probabilities,
            // which come after this; its rows' places are written behind a barrier)
            umma::fence_before();
            group_sync(i);
            if (lane == 0) ptx::mbar_arrive(i_empty(k));
        }
    } else if (warp < kSoftWarps + 4) {
        other_registers<kKv, kN>();
        if (warp == kSoftWarps) {
            // ------------------------------------------------ products
            const Waiter wait = waiter.as(kRoleProducts);
            if (umma::elect_one()) {
                constexpr uint32_t kQk = umma::f16_idesc(kTile, kN, false);
                constexpr uint32_t kPv = umma::f16_idesc(kD, kN, true) | umma::kAMn;
                const uint32_t q_lo = umma::desc_lo(base, 16);
                const uint32_t k_lo = umma::desc_lo(base + M::kRing, 16);
                const uint32_t v_lo = umma::desc_lo(base + M::kRing, M::kHalfBytes);
                const uint64_t p_at = umma::desc_plain(base + M::kP, 16 * kTile);
                auto qk = [&](uint32_t g) -> bool {   // S^T = K Q^T
                    const uint32_t n = 2 * g, s = n % S;
                    if constexpr (kCodes) {
                        if (!wait.one(k_full(g), (g / M::kKBufs) & 1)) return false;
                    } else {
                        if (!wait.one(full(s), (n / S) & 1)) return false;
                    }
                    umma::fence_after();
                    [[maybe_unused]] const uint32_t a = k_lo + s * (M::kTileBytes >> 4);
#pragma unroll 1
                    for (int k = 0; k < kD / 16; ++k) {
                        const uint64_t b = umma::desc(
                            q_lo + (((k >> 2) * M::kQHalfBytes + (k & 3) * 32) >> 4));
                        if constexpr (kCodes)
                            umma::mma_ts(t_s(g), t_k(g) + 8 * k, b, kQk, k > 0);
                        else
                            umma::mma_ss(
                                t_s(g),
                                umma::desc(a + (((k >> 2) * M::kHalfBytes + (k & 3) * 32) >> 4)),
                                b, kQk, k > 0);
                    }
                    umma::commit(s_full(g));
                    umma::commit(kCodes ? k_empty(g) : empty(s));
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
                        const uint32_t n = kCodes ? g : 2 * g + 1, s = n % S;
                        ok = wait.one(p_full(g), g >> 1 & 1) && wait.one(full(s), (n / S) & 1);
                        if (!ok) break;
                        umma::fence_after();
                        const uint32_t a = v_lo + s * (M::kTileBytes >> 4);
                        const uint64_t b = p_at + (g % M::kPBufs * M::kPBytes >> 4);
#pragma unroll 1
                        for (int k2 = 0; k2 < kTile / 16; ++k2)   // O^T += V^T P^T
                            umma::mma_ss(t_o, umma::desc(a + k2 * (2048 >> 4)), b + k2 * (256 >> 4),
                                         kPv, j > 0 || k2 > 0);
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
            // A lane per page looks its block up and issues its copies, 2 KB of a page each.
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
            ptx::griddep_wait();
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
                // scales of the lane's page, both by the K warp: see TreeSmem::kScales
                auto scales_of = [&](int32_t b, float &ks, float &vs) {
                    ks = vs = 0.f;
                    if constexpr (kCodes)
                        if (b >= 0 && !is_v) {
                            const int64_t at = static_cast<int64_t>(b) * p.num_kv_heads + it.kvh;
                            ks = __ldg(p.k_scales + at);
                            vs = __ldg(p.v_scales + at);
                        }
                };
                int32_t blk = lookup(0), next = nt > 1 ? lookup(1) : -2;
                float k_scale, v_scale;
                scales_of(blk, k_scale, v_scale);
                for (int j = 0; j < nt; ++j) {
                    const uint32_t n = 2 * tiles + (is_v ? 1 : 0);
                    const int s = n % R;
                    const bool have = blk >= 0;
                    if (blk == -1) {
                        flags[1 + (k & 1)] = 1;
                        if (p.dev_status)
                            atomicOr(p.dev_status, static_cast<int32_t>(PKV_DEV_BAD_BLOCK));
                    }
                    const int row = (blk * p.num_kv_heads + it.kvh) * kPage;
                    const unsigned pages = __ballot_sync(0xffffffffu, have);
                    const uint32_t fb = kCodes ? cfull(s) : full(s);
                    const uint32_t eb = kCodes ? cempty(s) : empty(s);
                    // (ahead: the blocks of the tile after the next, the next one's scales)
                    const int32_t after = j + 2 < nt ? lookup(j + 2) : -2;
                    float k_next, v_next;
                    scales_of(next, k_next, v_next);
                    ok = wait(eb, ((n / R) & 1) ^ 1);
                    if (!ok) break;
                    if (umma::elect_one())
                        ptx::mbar_expect_tx(fb, __popc(pages) * kBoxes * kBoxBytes);
                    __syncwarp();
                    const uint32_t dst = ring + s * kStageBytes;
                    if (have) {
#pragma unroll
                        for (int b = 0; b < kBoxes; ++b)
                            ptx::tma_load_2d(dst + b * M::kHalfBytes + lane * kBoxBytes, tm,
                                             b * kBox, row, fb);
                    }
                    if constexpr (kCodes)
                        if (!is_v && lane < kPagesPerTile) {
                            float *to = scales_at(tiles) + lane;
                            to[0] = k_scale;
                            to[kPagesPerTile] = v_scale;
                        }
                    __syncwarp();  // (the arrival is behind the flag and the scales)
                    if (lane == 0) ptx::mbar_arrive(fb);
                    ++tiles;
                    blk = next;
                    next = after;
                    k_scale = k_next;
                    v_scale = v_next;
                    if (!is_v && j == 0) {
                        // the queries: tokens x heads x 64 values, which land as the item's
                        // rows in their order (rows of heads that are not the item's, or
                        // behind the batch, do not count)
                        ok = wait(q_empty, (k & 1) ^ 1);
                        if (!ok) break;
                        if (umma::elect_one()) {
                            ptx::mbar_arrive_expect_tx(q_full, p.tokens * p.group * M::kHalves * 128);
    #pragma unroll
                            for (int b = 0; b < M::kHalves; ++b)
                                ptx::tma_load_3d(base + b * M::kQHalfBytes, &tmq, b * 64,
                                                 it.kvh * p.group, it.start, q_full);
                        }
                        __syncwarp();
                        ++queries;
                    }
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
            const int piece = blockIdx.x;
            ptx::griddep_wait();
            struct Seq {
                SeqRows rows;
                SeqKeys keys;   // (one tile where the rows only get zeros)
                bool zeros;
            };
            auto sequence = [&](int s) -> Seq {
                Seq q;
                const int first = __ldg(p.query_starts + s), last = __ldg(p.query_starts + s + 1);
                const int len = __ldg(p.context_lens + s);
                const int pre = p.prefix_lens ? __ldg(p.prefix_lens + s) : 0;
                q.rows.set(first, last, len, p.num_tokens, p.ctx_cap);
                q.zeros = first != last && (!q.rows.ok || q.rows.len > p.max_tree_len);
                q.keys = SeqKeys{};
                if (q.zeros)
                    q.keys.tiles = q.rows.len > 0;
                else if (q.rows.len > 0)
                    q.keys.set(p, q.rows.ctx, q.rows.len, pre);
                return q;
            };
            // The whole line, then where the piece begins: twice over the sequences, 32
            // at a time.
            int total = 0, begin = 0, end = 0, quo = 0, rem = 0;
            auto cut = [&](int i) { return quo * i + min(i, rem); };
            int seq = 0, rest = 0;   // the present sequence, its tiles before `at`
            int before = 0;
            bool any = false;
#pragma unroll 1
            for (int s0 = 0, pass = 0;; s0 += 32) {
                if (s0 >= p.num_seqs) {
                    if (pass == 1 || total == 0) break;
                    // (cuts are whole tiles, pieces not below kPieceTiles where they can)
                    const int pieces = max(min(total / kPieceTiles, kTreePieces), 1);
                    quo = total / pieces;
                    rem = total - quo * pieces;
                    begin = piece < pieces ? cut(piece) : total;
                    end = piece < pieces ? cut(piece + 1) : total;
                    if (begin >= end) break;
                    pass = 1;
                    s0 = 0;
                }
                int t = 0;
                if (s0 + lane < p.num_seqs) {
                    const Seq q = sequence(s0 + lane);
                    t = q.keys.tiles * p.num_kv_heads;
                    any |= q.zeros;
                }
                int sum = t;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, sum, o);
                    if (lane >= o) sum += v;
                }
                const int all = __shfl_sync(0xffffffffu, sum, 31);
                if (pass == 0) {
                    total += all;
                } else if (begin < before + all) {
                    const unsigned m = __ballot_sync(0xffffffffu, begin < before + sum);
                    const int l0 = __ffs(m) - 1;
                    seq = s0 + l0;
                    rest = begin - before - __shfl_sync(0xffffffffu, sum - t, l0);
                    break;
                } else {
                    before += all;
                }
            }
            if (any && blockIdx.x == 0 && p.dev_status)
                atomicOr(p.dev_status, static_cast<int32_t>(PKV_DEV_BAD_CTX));
            TreeMeta tail = {};
            bool ok = true;
            int k = 0, at = begin;
            for (; at < end && ok; ++seq, rest = 0) {
                const Seq q = sequence(seq);
                const int tiles = q.keys.tiles;
                if (tiles == 0) continue;
                TreeItem it;
                it.seq = seq;
                it.start = q.rows.start;
                it.n = q.rows.len;
                it.base = q.keys.base;
                it.lo = q.keys.lo;
                it.pre = q.keys.pre;
                it.np1 = q.keys.np1;
                it.gap = q.keys.gap;
                it.visited = (it.base + it.n - 1) / kPage + 1 - it.gap;
                it.kvh = rest / tiles;
                it.ta = rest - it.kvh * tiles;
                for (; it.kvh < p.num_kv_heads && at < end && ok; ++it.kvh, it.ta = 0) {
                    it.nt = min(tiles - it.ta, end - at);
                    const int stop = at + (tiles - it.ta);   // the item's end on the line
                    it.part = it.ta > 0 ? 0 : it.nt < tiles ? 1 : -1;
                    at += it.nt;
                    if (q.zeros) {
                        // (all of the sequence's rows)
                        const int64_t all = static_cast<int64_t>(it.n) * p.group * (kD / 8);
                        for (int64_t e = lane; e < all; e += 32) {
                            const int64_t r = e / (kD / 8);
                            const int64_t tk = it.start + r / p.group;
                            if (tk < 0 || tk >= p.num_tokens) continue;
                            const int64_t row =
                                tk * p.num_heads + it.kvh * p.group + r % p.group;
                            reinterpret_cast<uint4 *>(p.out + row * kD)[e % (kD / 8)] =
                                make_uint4(0, 0, 0, 0);
                        }
                        continue;
                    }
                    if (it.part == 1) {
                        // pieces that the rest of the item lies in
                        int last = piece + 1;
                        while (cut(last + 1) < stop) ++last;
                        tail.start = it.start;
                        tail.n = it.n;
                        tail.kvh = it.kvh;
                        tail.parts = last - piece + 1;
                    }
                    ok = wait(i_empty(k), (k >> 1 & 1) ^ 1);
                    if (!ok) break;
                    if (lane == 0) {
                        item(k) = it;
                        flags[1 + (k & 1)] = 0;
                        ptx::mbar_arrive(i_full(k));
                    }
                    // its tree: every parent an earlier row
                    // (a token has a row at least: kN are enough)
                    int *up = reinterpret_cast<int *>(smem + M::kUp) + kN * (k & 1);
                    bool wrong = false;
                    for (int j = lane; j < it.n; j += 32) {
                        const int a = __ldg(p.parents + it.start + j);
                        wrong |= a < -1 || a >= j;
                        up[j] = a;
                    }
                    wrong = __any_sync(0xffffffffu, wrong);
                    if (lane == 0) {
                        flags[4 + (k & 1)] = wrong;
                        if (wrong && p.dev_status)
                            atomicOr(p.dev_status, static_cast<int32_t>(PKV_DEV_BAD_TREE));
                    }
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(t_full(k));
                    ++k;
                }
            }
            if (lane == 0) p.meta[blockIdx.x] = tail;
            if (ok) ok = wait(i_empty(k), (k >> 1 & 1) ^ 1);
            if (ok && lane == 0) {
                item(k).nt = 0;
                ptx::mbar_arrive(i_full(k));
                ptx::mbar_arrive(t_full(k));
            }
            __syncwarp();
        }
    } else {
        if constexpr (kCodes) {
            // ------------------------------------------------ codes to fp16
            other_registers<kKv, kN>();
            const Waiter wait = waiter.as(kRoleWiden);
            constexpr int R = M::kCodeStages;
            constexpr int kCh = kD / 16;  // 16-byte chunks of codes per key
            const bool is_v = warp >= kSoftWarps + 4 + kTeam;
            const int tid = threadIdx.x & (32 * kTeam - 1);
            // The loops here, of the products and of the loads are left rolled: 20 to 28
            // warps run seven programs on four schedulers, and what they wait for most is
            // instructions.  (INT8, 64 trees of 8 tokens over 2048, 4 heads to a kv head:
            // 111 us with all of them unrolled, 80 so.)
            // K: a thread per key, whose codes become the key's lane of TMEM.
            auto widen_k = [&](uint32_t g, uint32_t src) {
                const uint32_t from = src + tid * kD;
                const uint32_t to = t_k(g) + (static_cast<uint32_t>(tid >> 5) << 21);
                const int sw = kD == 128 ? tid & 7 : tid >> 1 & 3;
#pragma unroll 1
                for (int ch = 0; ch < kCh; ch += 2) {
                    uint4 w[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) w[e] = ptx::lds128(from + (((ch + e) ^ sw) << 4));
                    uint32_t r[16];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint4 &c = w[e / 2];
                        const uint4 x = e & 1 ? widen<kKv>(c.z, c.w) : widen<kKv>(c.x, c.y);
                        r[4 * e] = x.x;
                        r[4 * e + 1] = x.y;
                        r[4 * e + 2] = x.z;
                        r[4 * e + 3] = x.w;
                    }
                    umma::st16(to + 8 * ch, r);
                }
                umma::wait_st();
                umma::fence_before();
            };
            // V: eight lanes take four chunks of two rows: r and r ^ 5 of eight at head_dim
            // 128, r and r + 1 at 64, whose swizzles put the loads and both stores on
            // different banks.
            constexpr int kStep = 32 * kTeam / kCh;
            constexpr int kLoads = kTile / kStep;
            static_assert(kTile % kStep == 0 && kStep % 8 == 0, "whole groups of eight rows");
            int ch = tid % kCh, row0 = tid / kCh;
            if constexpr (kD == 128) {
                // bits of tid: chunk 0-1, row of the pair 2, half 3, pair 4-5, rows by eight
                ch = (tid & 3) | (tid >> 1 & 4);
                row0 = ((tid >> 4 & 3) ^ (tid & 4 ? 5 : 0)) | (tid >> 6) << 3;
            }
            // (rows advance by whole groups of eight, so the swizzles stay)
            const uint32_t sx = kD == 128 ? (ch ^ (row0 & 7)) : (ch ^ ((row0 >> 1) & 3));
            const int c_a = ((2 * ch) & 7) ^ (row0 & 7);
            auto widen_v = [&](uint32_t src, uint32_t dst) {
                const uint32_t from = src + row0 * kD + (sx << 4);
                const uint32_t to = dst + (ch >> 2) * M::kHalfBytes + row0 * 128;
#pragma unroll 1
                for (int e = 0; e < kLoads; ++e) {
                    const uint4 w = ptx::lds128(from + e * kStep * kD);
                    const uint32_t at = to + e * kStep * 128;
                    st_shared16(at + (c_a << 4), widen<kKv>(w.x, w.y));
                    st_shared16(at + ((c_a ^ 1) << 4), widen<kKv>(w.z, w.w));
                }
                ptx::fence_proxy_async_smem();
            };
            uint32_t g = 0;
            bool ok = true;
            for (int k = 0; ok; ++k) {
                ok = wait(i_full(k), k >> 1 & 1);
                if (!ok) break;
                const int nt = item(k).nt;
                if (nt == 0) break;
                for (int j = 0; j < nt; ++j, ++g) {
                    const uint32_t n = 2 * g + is_v, r = n % R;
                    const uint32_t src = base + M::kCodeRing + r * M::kCodeBytes;
                    const uint32_t s = g % S;
                    ok = wait(cfull(r), (n / R) & 1) &&
                         (is_v ? wait(empty(s), ((g / S) & 1) ^ 1)
                               : wait(k_empty(g), ((g / M::kKBufs) & 1) ^ 1));
                    if (!ok) break;
                    if (is_v) {
                        widen_v(src, base + M::kRing + s * M::kTileBytes);
                    } else {
                        if (tid < kPagesPerTile) {
                            float *sc = scales_at(g) + tid;
                            const float vs = sc[kPagesPerTile], vc = fmaxf(vs, kLeastV);
                            sc[0] *= p.scale_log2;
                            sc[kPagesPerTile] = vs >= 0.f && vs < INFINITY ? log2_of(vc) : NAN;
                            sc[2 * kPagesPerTile] = __frcp_rn(vc);
                        }
                        umma::fence_after();
                        widen_k(g, src);
                    }
                    __syncwarp();
                    if (lane == 0) {
                        ptx::mbar_arrive(is_v ? full(s) : k_full(g));
                        ptx::mbar_arrive(cempty(r));
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
// A part with l < 0 (a bad block or tree) makes the row zeros.  Most items have two
// parts, whose numbers are asked for at once with the question whether there are any.
constexpr int kJoinWarps = 8;

template <int kD, int kN>
__global__ void __launch_bounds__(32 * kJoinWarps) tree_join_kernel(const __grid_constant__ TreeArgs p)
{
    constexpr int kC = kD / 32;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int owner = blockIdx.x, r = blockIdx.y * kJoinWarps + warp;
    // part 0 is the owner's last one, the others are the first of the pieces behind
    auto at = [&](int z) -> int64_t {
        return (2 * static_cast<int64_t>(min(owner + z, kTreePieces - 1)) + (z == 0)) * kN + r;
    };
    constexpr int kAt = 4;      // parts at a time
    float2 ml[kAt];
    float v[kAt][kC];
    auto load = [&](int z0, int z1) {
#pragma unroll
        for (int u = 0; u < kAt; ++u)
            if (z0 + u < z1) {
                ml[u] = __ldcg(p.part_ml + at(z0 + u));
                const float *a = p.part_acc + at(z0 + u) * kD + lane * kC;
                if constexpr (kC == 4) {
                    const float4 w = __ldcg(reinterpret_cast<const float4 *>(a));
                    v[u][0] = w.x;
                    v[u][1] = w.y;
                    v[u][2] = w.z;
                    v[u][3] = w.w;
                } else {
                    const float2 w = __ldcg(reinterpret_cast<const float2 *>(a));
                    v[u][0] = w.x;
                    v[u][1] = w.y;
                }
            }
    };
    const int4 mw = __ldcg(reinterpret_cast<const int4 *>(p.meta) + owner);
    load(0, 2);
    const int parts = mw.w, rj = r / p.group, rh = r - rj * p.group;
    if (parts <= 0 || rj >= mw.y) return;
    float m = kNone, l = 0.f, acc[kC];
    bool bad = false;
#pragma unroll
    for (int c = 0; c < kC; ++c) acc[c] = 0.f;
    int have = 2;
    for (int z = 0;;) {
        float top = m;
#pragma unroll
        for (int u = 0; u < kAt; ++u)
            if (u < have) top = fmaxf(top, ml[u].x);
        const float f = ptx::ex2(m - top);
        m = top;
        l *= f;
#pragma unroll
        for (int c = 0; c < kC; ++c) acc[c] *= f;
#pragma unroll
        for (int u = 0; u < kAt; ++u)
            if (u < have) {
                const float w = ptx::ex2(ml[u].x - m);
                bad |= ml[u].y < 0.f;
                l += w * ml[u].y;
#pragma unroll
                for (int c = 0; c < kC; ++c) acc[c] += w * v[u][c];
            }
        z += have;
        if (z >= parts) break;
        have = min(kAt, parts - z);
        load(z, parts);
    }
    const bool zero = bad || l == 0.f;
    const int64_t row = static_cast<int64_t>(mw.x + rj) * p.num_heads + mw.z * p.group + rh;
    __half2 *o = reinterpret_cast<__half2 *>(p.out + row * kD + lane * kC);
#pragma unroll
    for (int c = 0; c < kC; c += 2)
        o[c / 2] = __floats2half2_rn(zero ? 0.f : acc[c] / l, zero ? 0.f : acc[c + 1] / l);
}

// -------------------------------------------------------------------- host
template <int kKv, int kD, int kN>
pkv_status launch_tree(const TreeCall &c)
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
    const int group = c.num_heads / c.num_kv_heads, tokens = kN / group;
    const uint64_t rows = static_cast<uint64_t>(c.num_blocks) * c.num_kv_heads * kPage;
    const int elem = M::kCodes ? 1 : 2, box = M::kCodes ? kD : 64;
    if (!encode_tmap_3d_f16(&tmq, c.query, kD, c.num_heads, c.num_tokens, 64, group,
                            tokens) ||
        !encode_tmap_2d(&tmk, c.kpool, elem, kD, rows, box, kPage, box * elem) ||
        !encode_tmap_2d(&tmv, c.vpool, elem, kD, rows, box, kPage, box * elem))
        return PKV_ERR_CUDA;
    constexpr int64_t ctas = kTreePieces;
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
    a.group = group;
    a.tokens = tokens;
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
    cfg.blockDim = dim3(tree_threads(kKv, kN));
    cfg.dynamicSmemBytes = M::kAsk;
    cfg.stream = static_cast<cudaStream_t>(c.stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a, tmq, tmk, tmv);
    if (e == cudaSuccess) {
        cfg.gridDim = dim3(static_cast<unsigned>(ctas), kN / kJoinWarps);
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

template <int kKv>
pkv_status launch_tree(const TreeCall &c, const TreePlan &plan)
{
    if (c.head_dim == 128)
        return plan.rows == 32 ? launch_tree<kKv, 128, 32>(c) : launch_tree<kKv, 128, 64>(c);
    return plan.rows == 32 ? launch_tree<kKv, 64, 32>(c) : launch_tree<kKv, 64, 64>(c);
}

#ifdef PKV_DEBUG
inline int set_waits(int give_role, int give_at, int slow_role, int slow_ns, int slow_warp)
{
    const WaitDebug d = {give_role < 0 ? -2 : give_role, give_at, slow_role < 0 ? -2 : slow_role,
                         slow_ns, slow_warp};
    return cudaMemcpyToSymbol(g_wait_debug, &d, sizeof(d)) == cudaSuccess ? 0 : -1;
}
#endif

}  // namespace
}  // namespace pkv
