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
//   P = 2^(S' - m)  (registers: one thread per row, two where scores are worked
//                    out first; back to TMEM as fp16)
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
// Roles of the warps: 0-7 the rows of the two tiles (0-15 with two threads per
// row, and the others 8 further on), 8 issues the products, 9 and 11 the TMA
// loads of Q, K and V (a ring of tiles of 128 keys, K and V in turn), 10 finds
// the next item.  INT8 / FP8 pages land in a second ring, and warps 12-15 widen
// them exactly to fp16; the K scales multiply the scores, the V scales enter
// the probabilities as a ratio to a reference per row (kVLazy).
//
// Measured on GB300, 32 / 8 heads, head_dim 128: 2048 tokens over 8192 in 171 us
// (1408 TFLOP/s, 0.75 of the measured bf16 rate), capped 274 (scores up to the
// cap 312, beyond it 452), INT8 203, FP8 204; 8 prompts of 2048 in 234 us (0.62;
// 245 among other inputs in turn), one of 4096 in 112 (0.65).
//
// Items are numbered by bounds that the host knows (pkv_ragged.cuh), the ones
// with the most keys first.  Few items over long contexts are split over their
// keys, and a second kernel joins the parts (plan_of).  An item whose rows
// fill one tile only (a few drafted tokens) then has the second tile work on
// the same rows, with every other tile of keys, as a part of its own.
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

namespace pkv {
namespace {

constexpr int kRows = 256;      // query rows per item: two tiles
constexpr int kTile = 128;      // rows per tile, keys per step
constexpr int kPage = 16;
constexpr int kPagesPerTile = kTile / kPage;

// Softmax threads per row.  One, with 128 scores each, where a score is one
// multiply-add and one exponential: nothing is exchanged.  Two, with 64 each,
// where a score is worked out first (cap, bias): one thread's row would take
// 2600 cycles, in which the tensor core has done its part of 1024 long since;
// the two exchange their maxima and sums.
__host__ __device__ constexpr int row_threads(bool mod)
{
    return mod ? 2 : 1;
}

__host__ __device__ constexpr int soft_warps(bool mod)
{
    return 8 * row_threads(mod);
}
constexpr int kSms = 152;       // GB300: what the split over the keys aims to fill
constexpr int kMaxSplits = 64;
constexpr uint64_t kWaitLimitNs = 1000000000ull;  // bounded waits: 1 s
constexpr float kLazy = 6.f;    // log2 growth of a maximum that is left in the sums
constexpr float kLift = 6.f;    // log2 factor of the probabilities
constexpr float kVLazy = 8.f;   // growth of a V scale that is left in the ratio

// V scales of code caches: the accumulators of a row are in units of a reference
// scale, and a page's scale over the reference multiplies its probabilities on
// their way to fp16.  The reference is at most kVLazy times the largest scale of
// the pages that the row sees, whose scales of earlier tiles count with the
// factor by which the maximum has grown since, and at least that over kVLazy.
// Products below 2^-14 (lifted by 2^6; the row's largest probability is 2^6 at
// least) are subnormal, and rounded by up to 2^-25: with P the row's largest
// probability and V that largest scale, a key's probability times its page's
// scale is off by up to 2^-28 P V and keeps fewer than 11 bits below 2^-17 P V.

constexpr int kKvF16 = 0, kKvI8 = 1, kKvF8 = 2;

struct PrefillArgs {
    __half *out;
    const __half *query;
    const int32_t *block_tables, *query_starts, *context_lens;
    const float *k_scales, *v_scales;
    const float *slopes;
    const int32_t *prefix_lens;
    float *part_acc;    // [2 splits][num_tokens * num_heads][head_dim]
    float2 *part_ml;    // [2 splits][num_tokens * num_heads]: maximum, sum
    int32_t *dev_status;
    int num_tokens, num_seqs, num_heads, num_kv_heads, group;
    int chunk, chunks;  // heads of a kv head per item (the group, at most 256), chunks of them
    int tokens;         // tokens per item: 256 / chunk
    int max_blocks_per_seq, num_blocks, ctx_cap, window, splits, units;
    float scale_log2, cap, cap_inv;
};

// ------------------------------------------------------------ shared memory
template <int kKv, int kD>
struct Smem {
    static constexpr bool kCodes = kKv != kKvF16;
    static constexpr int kHalves = kD / 64;
    static constexpr int kHalfBytes = kTile * 128;             // 64 values of 128 rows
    static constexpr int kTileBytes = kHalves * kHalfBytes;    // 128 rows of K or V
    static constexpr int kQHalfBytes = kRows * 128;            // 64 values of the item's rows
    static constexpr int kCodeBytes = kTile * kD;
    static constexpr int kStages = kCodes ? (kD == 128 ? 3 : 6) : (kD == 128 ? 4 : 8);
    static constexpr int kCodeStages = kCodes ? 3 : 0;
    static constexpr int kRing = 2 * kTileBytes;
    static constexpr int kCodeRing = kRing + kStages * kTileBytes;
    static constexpr int kOut = kCodeRing + kCodeStages * kCodeBytes;   // rows on their way out
    static constexpr int kOutBytes = 16 * 1024;
    static constexpr int kCtl = kOut + kOutBytes;
    static constexpr int kBars = 3 * kStages + 2 * kCodeStages + 16;
    // scales [kScaleTiles][K, V][8 pages].  The K warp writes both of a tile
    // before it arrives for the tile's K codes; their widening waits for that,
    // the product Q K^T for the widening and the softmax for the product, so
    // every read of a tile's scales is behind their writes.  (V's own barriers
    // are not on that way: the products wait for V only after the softmax.)
    // A slot is written again eight tiles later, when the K codes of three
    // elements before (V of tile n - 2) are widened: they went to a stage that
    // the products have given back, so the softmax is through with tile n - 5
    // at least (head_dim 128: n - 4; two tiles on the same rows: n - 5).
    static constexpr int kScaleTiles = 8;
    static constexpr int kNext = (kCtl + 8 * kBars + 15) & ~15;   // answer of the launch queue
    static constexpr int kScales = kNext + 16;
    static constexpr int kItems = kScales + (kCodes ? kScaleTiles * 2 * kPagesPerTile * 4 : 0);
    static constexpr int kFlags = kItems + 2 * 64;
    static constexpr int kSwap = kFlags + 16;   // [2 tiles][2 halves of the columns][128 rows]
    static constexpr int kIssued = kSwap + 2 * 2 * kTile * 4;   // see drain_copies
    static constexpr int kBytes = kIssued + 16;
    // a second CTA on the SM would wait for TMEM: ask for more than half
    static constexpr int kAsk = kBytes > 120 * 1024 ? kBytes : 120 * 1024;
    static_assert(kAsk <= 227 * 1024, "shared memory of one CTA");
};

// What a warp does; its waits are counted by role in the debug build.
enum Role { kRoleRows, kRoleProducts, kRoleLoadK, kRoleLoadV, kRoleItems, kRoleWiden, kRoles };

#ifdef PKV_DEBUG
// Settable through pkv_debug_set_prefill: wait number give_at of every warp of
// give_role gives up, as if its limit had run out, and every wait of slow_role
// begins slow_ns later (role -2: none; warps without a role have -1).
struct PrefillDebug {
    int give_role, give_at, slow_role, slow_ns;
};
__device__ PrefillDebug g_prefill_debug = {-2, 0, -2, 0};
#endif

struct Waiter {
    volatile int *abort;
    int32_t *dev_status;
#ifdef PKV_DEBUG
    int role = -1;
    mutable int waits = 0;
#endif
    __device__ __forceinline__ Waiter as([[maybe_unused]] Role r) const
    {
        Waiter w = *this;
#ifdef PKV_DEBUG
        w.role = r;
#endif
        return w;
    }
    // Bounded waits; false once any wait of the CTA ran out.  By one thread:
    __device__ __forceinline__ bool one(uint32_t bar, uint32_t parity) const
    {
        if (gives_up()) return false;
        return ptx::mbar_try_wait(bar, parity) || slow(bar, parity);
    }
    // by a whole warp, all lanes with the same outcome:
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const
    {
        if (gives_up()) return false;
        if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity))) return true;
        return __all_sync(0xffffffffu, slow(bar, parity));
    }
    __device__ __forceinline__ bool slow(uint32_t bar, uint32_t parity) const
    {
        uint64_t t0 = 0;  // the timer is slow to read: only after many tries
        for (;;) {
            for (int i = 0; i < 4096; ++i)
                if (ptx::mbar_try_wait(bar, parity)) return true;
            if (*abort) return false;
            const uint64_t now = ptx::globaltimer_ns();
            if (t0 == 0) t0 = now;
            if (now - t0 > kWaitLimitNs) give_up();
        }
    }
    __device__ __forceinline__ void give_up() const
    {
        *abort = 1;
        if (dev_status) atomicOr(dev_status, PKV_DEV_TIMEOUT);
    }
    __device__ __forceinline__ bool gives_up() const
    {
#ifdef PKV_DEBUG
        const PrefillDebug d = g_prefill_debug;
        if (role == d.slow_role) __nanosleep(d.slow_ns);
        if (role == d.give_role && waits++ == d.give_at) {
            give_up();
            return true;
        }
#endif
        return false;
    }
};

// ------------------------------------------------------------------- items
struct __align__(16) Item {
    int seq, kvh;
    int tok, toks;              // first token (of the batch) and tokens of the item
    int head;                   // first query head
    int16_t heads, dir;         // heads; order of the tiles (see tile)
    int pos;                    // position of the first token
    int z;                      // split
    int lo, hi, pre;            // keys of the item: lo .. hi and below pre
    int np1, gap, visited;      // pages: np1, a gap, the rest (see the decode)
    int ta;                     // tile of keys to begin with
    int nt;                     // tiles of keys; 0: no further item

    __device__ __forceinline__ int real(int v) const { return v + (v >= np1 ? gap : 0); }

    // the j-th tile of keys: with a bias by distance (dir -1) from the last one
    // to the first
    __device__ __forceinline__ int tile(int j) const { return ta + dir * j; }

    // whether a tile of keys holds some that no row sees
    __device__ __forceinline__ bool dirty(int tile) const
    {
        const int tmin = real(tile * kPagesPerTile) * kPage;
        const int tmax = real(tile * kPagesPerTile + kPagesPerTile - 1) * kPage + kPage - 1;
        return !((tmax <= hi && tmin >= lo) || tmax < pre);
    }

    // bits of a page's tokens (its first is t0) that some row may see
    __device__ __forceinline__ uint32_t live(int t0) const
    {
        return (below(hi + 1 - t0) & ~below(lo - t0)) | below(pre - t0);
    }
};

static_assert(sizeof(Item) == 64, "an item is 64 bytes of shared memory");

// Whether the two tiles share the rows of the item.
__device__ __forceinline__ bool paired(const PrefillArgs &p, const Item &it)
{
    return p.splits > 1 && it.toks * p.chunk <= kTile;
}

// The item of a block number: 1 an item with keys, 0 one without (its rows are
// then zeros), -1 none.  The units with the most keys (the last ones of a
// sequence) first; kv heads, chunks of heads and key splits side by side.
__device__ __forceinline__ int find_item(const PrefillArgs &p, int block, Item &it)
{
    const int per_unit = p.num_kv_heads * p.chunks * p.splits;
    const int u = p.units - 1 - block / per_unit;
    int sub = block % per_unit;
    it.z = sub % p.splits;
    sub /= p.splits;
    const int c = sub % p.chunks;
    it.kvh = sub / p.chunks;
    SeqRows sr;
    int pre = 0;   // visible prefix of the sequence
    if (p.num_seqs <= 32) {
        // a lane per sequence: all that is asked of the batch in one round trip
        const int lane = threadIdx.x & 31, s = min(lane, p.num_seqs - 1);
        const int st = __ldg(p.query_starts + s), en = __ldg(p.query_starts + s + 1);
        const int ln = __ldg(p.context_lens + s);
        const int pr = p.prefix_lens ? __ldg(p.prefix_lens + s) : 0;
        const bool le = lane < p.num_seqs && st / p.tokens + s <= u;
        const unsigned m = __ballot_sync(0xffffffffu, le);
        it.seq = (m == 0xffffffffu ? 32 : __ffs(~m) - 1) - 1;
        if (it.seq < 0) return -1;
        sr.set(__shfl_sync(0xffffffffu, st, it.seq), __shfl_sync(0xffffffffu, en, it.seq),
               __shfl_sync(0xffffffffu, ln, it.seq), p.num_tokens, p.ctx_cap);
        pre = __shfl_sync(0xffffffffu, pr, it.seq);
    } else {
        it.seq = warp_search(p.num_seqs, u, [&](int s) -> int64_t {
            return static_cast<int64_t>(__ldg(p.query_starts + s) / p.tokens) + s;
        });
        if (it.seq < 0) return -1;
        sr.load(p.query_starts, p.context_lens, it.seq, p.num_tokens, p.ctx_cap);
        if (p.prefix_lens) pre = __ldg(p.prefix_lens + it.seq);
    }
    const int base = sr.start / p.tokens + it.seq;
    const int64_t t0 = static_cast<int64_t>(u - base) * p.tokens;
    if (t0 < 0 || t0 >= sr.len) return -1;
    it.tok = sr.start + static_cast<int>(t0);
    it.toks = min(p.tokens, sr.len - static_cast<int>(t0));
    it.head = it.kvh * p.group + c * p.chunk;
    it.heads = static_cast<int16_t>(min(p.chunk, p.group - c * p.chunk));
    it.dir = p.slopes ? -1 : 1;
    it.ta = it.nt = 0;
    if (!sr.ok) return 0;
    it.pos = sr.ctx - sr.len + static_cast<int>(t0);
    it.hi = it.pos + it.toks - 1;
    it.lo = p.window > 0 && it.pos >= p.window ? it.pos - p.window + 1 : 0;
    it.pre = min(max(pre, 0), sr.ctx);
    const int fp = it.lo / kPage;
    it.np1 = min((it.pre + kPage - 1) / kPage, fp);
    it.gap = fp - it.np1;
    it.visited = max(it.hi, it.pre - 1) / kPage + 1 - it.gap;
    const int tiles = (it.visited + kPagesPerTile - 1) / kPagesPerTile;
    it.ta = static_cast<int>(static_cast<int64_t>(tiles) * it.z / p.splits);
    it.nt = static_cast<int>(static_cast<int64_t>(tiles) * (it.z + 1) / p.splits) - it.ta;
    if (it.dir < 0) it.ta += it.nt - 1;
    return it.nt > 0;
}

// Sequences that do not fit need not have an item.
__device__ __noinline__ void check_sequences(const PrefillArgs &p, int lane)
{
    report_bad_sequences(p.query_starts, p.context_lens, p.num_seqs, p.num_tokens, p.ctx_cap,
                         p.dev_status, lane, 32);
}

// After a wait that ran out, with every warp behind a barrier of the CTA: waits
// (bounded) for the copies that may still write into its shared memory.  K and
// V tile t are elements 2 t and 2 t + 1 of a ring of R stages, and a stage is
// filled again only after its element was used up, so only the last element of
// each stage can be in flight; of the queries only the last item's.
template <int R>
__device__ void drain_copies(uint32_t full0, uint32_t q_full, int k_tiles, int v_tiles, int items)
{
    for (int s = 0; s < R; ++s)
        for (int n = 2 * max(k_tiles, v_tiles) - 1; n >= 0; --n)
            if (n % R == s && n / 2 < (n & 1 ? v_tiles : k_tiles)) {
                ptx::mbar_wait_bounded(full0 + 8 * s, n / R & 1, kWaitLimitNs);
                break;
            }
    if (items > 0) ptx::mbar_wait_bounded(q_full, (items - 1) & 1, kWaitLimitNs);
}

// ------------------------------------------------------------------ kernel
// Softmax warps, four more (products, loads, items), and four that widen codes.
template <int kKv, bool kMod>
__host__ __device__ constexpr int prefill_threads()
{
    return 32 * (soft_warps(kMod) + (kKv == kKvF16 ? 4 : 8));
}

// Registers: all threads are launched with 65536 / threads, rounded down to a
// multiple of 8 (fp16: 168 for 384 threads, 96 for 640; codes: 128 for 512, 80
// for 768).  The softmax warps take what the others give back.
template <int kKv, bool kMod>
__device__ __forceinline__ void soft_registers()
{
    if constexpr (kKv == kKvF16 && !kMod) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    if constexpr (kKv == kKvF16 && kMod) asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    if constexpr (kKv != kKvF16 && !kMod) asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    if constexpr (kKv != kKvF16 && kMod) asm volatile("setmaxnreg.inc.sync.aligned.u32 96;");
}

template <int kKv, bool kMod>
__device__ __forceinline__ void issue_registers()
{
    if constexpr (kKv == kKvF16 && !kMod) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if constexpr (kKv == kKvF16 && kMod) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if constexpr (kKv != kKvF16 && !kMod) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if constexpr (kKv != kKvF16 && kMod) asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
}

template <bool kMod>
__device__ __forceinline__ void widen_registers()
{
    if constexpr (!kMod) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if constexpr (kMod) asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
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

// The largest of 16 values.
__device__ __forceinline__ float max16(const float *x)
{
    const float a = fmaxf(fmaxf(x[0], x[1]), x[2]), b = fmaxf(fmaxf(x[3], x[4]), x[5]);
    const float c = fmaxf(fmaxf(x[6], x[7]), x[8]), d = fmaxf(fmaxf(x[9], x[10]), x[11]);
    const float e = fmaxf(fmaxf(x[12], x[13]), x[14]);
    return fmaxf(fmaxf(fmaxf(a, b), fmaxf(c, d)), fmaxf(e, x[15]));
}

// tanh(u) of two values as u P(u^2): P of degree 6 for |u| <= 1 (tanh_coef),
// or of degree 3, from the same fit on [0, 0.35], whose relative error there
// is 6.1e-8 (2^-23.9) with its coefficients in fp32, 2^-22.6 as evaluated.
template <int kDegree>
__device__ __forceinline__ uint64_t tanh2(uint64_t u)
{
    constexpr float near[4] = {0.99999994f, -0.333324224f, 0.132957995f, -0.0489582308f};
    const uint64_t w = ptx::mul2(u, u);
    const float top = kDegree == 3 ? near[3] : tanh_coef(6);
    uint64_t q = ptx::f32x2(top, top);
#pragma unroll
    for (int k = kDegree - 1; k >= 0; --k) {
        const float c = kDegree == 3 ? near[k] : tanh_coef(k);
        q = ptx::fma2(q, w, ptx::f32x2(c, c));
    }
    return ptx::mul2(u, q);
}

// x <- tanh(x), by the largest |x| of the warp's rows: a short polynomial
// (the usual case: scores well inside the cap), a longer one, or the
// exponential for what lies beyond the cap.
template <int kN>
__device__ __forceinline__ void tanh_row(float (&x)[kN])
{
    float top[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < kN; c += 2)
        top[c / 2 & 3] = fmaxf(fmaxf(top[c / 2 & 3], fabsf(x[c])), fabsf(x[c + 1]));
    const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    if (__all_sync(0xffffffffu, most <= 0.35f)) {
#pragma unroll
        for (int c = 0; c < kN; c += 2) {
            const float2 y = ptx::f32x2_parts(tanh2<3>(ptx::f32x2(x[c], x[c + 1])));
            x[c] = y.x;
            x[c + 1] = y.y;
        }
    } else if (__all_sync(0xffffffffu, most <= 1.f)) {
#pragma unroll
        for (int c = 0; c < kN; c += 2) {
            const float2 y = ptx::f32x2_parts(tanh2<6>(ptx::f32x2(x[c], x[c + 1])));
            x[c] = y.x;
            x[c + 1] = y.y;
        }
    } else {
#pragma unroll
        for (int c = 0; c < kN; c += 2) {
            const float2 y = ptx::f32x2_parts(tanh2<6>(ptx::f32x2(x[c], x[c + 1])));
            x[c] = fabsf(x[c]) <= 1.f ? y.x : cap_far(x[c], 1.f);
            x[c + 1] = fabsf(x[c + 1]) <= 1.f ? y.y : cap_far(x[c + 1], 1.f);
        }
    }
}

// kMod: a cap, a bias, or a softmax scale that is not positive -- the scores are
// worked out before their maximum is taken.  Without it the products stay as
// they are and their scale (with codes, the page's K scale too) enters with the
// exponent: 2^(S f - m) is one multiply-add.
//
// With a bias by distance, keys are taken from the last tile to the first: the
// nearest keys have the largest scores, so that the accumulators are hardly
// ever rescaled.  (Without one the other way is faster, 254 against 263 us for
// 8 prompts of 2048 tokens: the tile with masks and stale rows, the last one,
// is then worked on while the pipeline is full.)
//
// One CTA per SM, which takes the block numbers of CTAs that have not started
// (cluster launch control) as long as there are any: a warp asks for the next
// one, works out its item and hands it to the others, so that loads and
// products of an item begin while the last one's rows are written.
template <int kKv, int kD, bool kMod>
__global__ void __launch_bounds__(prefill_threads<kKv, kMod>(), 1)
    prefill_kernel(const __grid_constant__ PrefillArgs p, const __grid_constant__ CUtensorMap tmq,
                   const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv)
{
    using M = Smem<kKv, kD>;
    constexpr bool kCodes = M::kCodes;
    constexpr int S = M::kStages;
    constexpr int kRowChunks = kD / 8;
    constexpr int kSoftWarps = soft_warps(kMod), T = row_threads(kMod);
    constexpr int kCols = kTile / T, kColPages = kCols / kPage;  // of S, per softmax thread
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = ptx::smem_addr(smem);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    // barriers: ring full / empty, code ring full / empty, then single ones
    auto full = [&](int s) { return base + M::kCtl + 8 * s; };
    auto empty = [&](int s) { return base + M::kCtl + 8 * (S + s); };
    [[maybe_unused]] auto cfull = [&](int s) { return base + M::kCtl + 8 * (2 * S + s); };
    [[maybe_unused]] auto cempty = [&](int s) {
        return base + M::kCtl + 8 * (2 * S + M::kCodeStages + s);
    };
    const uint32_t one = base + M::kCtl + 8 * (2 * S + 2 * M::kCodeStages);
    const uint32_t q_full = one, q_empty = one + 8, drain = one + 16, next_full = one + 24;
    auto s_full = [&](int i) { return one + 32 + 8 * i; };
    auto p_full = [&](int i) { return one + 48 + 8 * i; };
    auto o_full = [&](int i) { return one + 64 + 8 * i; };
    auto i_full = [&](int k) { return one + 80 + 8 * (k & 1); };
    auto i_empty = [&](int k) { return one + 96 + 8 * (k & 1); };
    [[maybe_unused]] auto swapped = [&](int i) { return one + 112 + 8 * i; };
    // one per stage: rows are zeroed tiles ahead of the products
    [[maybe_unused]] auto fixed = [&](int s) { return one + 128 + 8 * s; };
    volatile int *flags = reinterpret_cast<volatile int *>(smem + M::kFlags);
    // flags: abort, bad of item slot 0, of slot 1, TMEM address
    const Waiter waiter{flags, p.dev_status};
    // what was issued: K tiles, V tiles, items' queries
    volatile int *issued = reinterpret_cast<volatile int *>(smem + M::kIssued);
    // the k-th item of this CTA
    auto item = [&](int k) -> Item & {
        return *reinterpret_cast<Item *>(smem + M::kItems + 64 * (k & 1));
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            ptx::mbar_init(full(s), kCodes ? 4 : 1);
            ptx::mbar_init(empty(s), 1);
            ptx::mbar_init(fixed(s), 1);
        }
        for (int s = 0; s < M::kCodeStages; ++s) {
            ptx::mbar_init(cfull(s), 1);
            ptx::mbar_init(cempty(s), 4);
        }
        ptx::mbar_init(q_full, 1);
        ptx::mbar_init(q_empty, 1);
        ptx::mbar_init(drain, 1);
        ptx::mbar_init(next_full, 1);
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(s_full(i), 1);
            ptx::mbar_init(p_full(i), kSoftWarps / 2);
            ptx::mbar_init(o_full(i), 1);
            ptx::mbar_init(swapped(i), kSoftWarps / 2);
            ptx::mbar_init(i_full(i), 1);
            ptx::mbar_init(i_empty(i), kSoftWarps + 3 + (kCodes ? 4 : 0));
        }
        ptx::fence_mbar_init();
        flags[0] = flags[1] = flags[2] = 0;
        issued[0] = issued[1] = issued[2] = 0;
    }
    if (warp == kSoftWarps) umma::alloc(base + M::kFlags + 12, 512);
    umma::fence_before();
    __syncthreads();
    umma::fence_after();
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const uint32_t tmem = __shfl_sync(0xffffffffu, static_cast<uint32_t>(flags[3]), 0);
    auto t_s = [&](int i) { return tmem + kTile * i; };            // S, then P, of tile i
    auto t_o = [&](int i) { return tmem + 2 * kTile + kD * i; };   // O of tile i

    if (warp < kSoftWarps) {
        // ------------------------------------------------ rows of the tiles
        soft_registers<kKv, kMod>();
        const Waiter wait = waiter.as(kRoleRows);
        const int i = warp / (4 * T);                   // tile
        const int half = T == 2 ? warp >> 2 & 1 : 0;    // which of the row's columns
        const int rt = threadIdx.x & (kTile - 1);       // row of the tile
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // TMEM lane 32 (w mod 4)
        // token and head of the thread's row, in its own tile and in the first
        const int rj_own = (kTile * i + rt) / p.chunk, rj_first = rt / p.chunk;
        uint32_t steps = 0;   // tiles of keys of this tile of rows so far
        uint32_t outs = 0;
        // T == 2: the other thread's value of the row.  The buffer is free again
        // when the next one is due: in an item because S is not started before
        // both threads were through, behind its last one by a barrier that the
        // next item's first exchange waits for.
        [[maybe_unused]] uint32_t swaps = 0;
        [[maybe_unused]] bool held = false;
        [[maybe_unused]] float *sw = reinterpret_cast<float *>(smem + M::kSwap) + i * 2 * kTile;
        auto swap = [&](float v, float &other, bool last) -> bool {
            if (held && !wait(swapped(i), swaps++ & 1)) return false;
            sw[half * kTile + rt] = v;
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(swapped(i));
            if (!wait(swapped(i), swaps++ & 1)) return false;
            other = sw[(half ^ 1) * kTile + rt];
            held = last;
            __syncwarp();
            if (last && lane == 0) ptx::mbar_arrive(swapped(i));
            return true;
        };
        [[maybe_unused]] uint32_t tiles = 0;  // tiles of keys of the CTA so far
        bool ok = true;
        for (int k = 0; ok; ++k) {
            ok = wait(i_full(k), k >> 1 & 1);
            if (!ok) break;
            const Item &it = item(k);
            const int nt = it.nt;
            if (nt == 0) break;
            const int rows = it.toks * p.chunk;
            const bool pair = paired(p, it);
            if (i == 1 && rows <= kTile && !pair) {
                tiles += nt;
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(i_empty(k));
                continue;
            }
            const int row0 = pair ? 0 : kTile * i;          // first row of the tile
            const int rj = pair ? rj_first : rj_own;        // token of the row
            const int rh = row0 + rt - rj * p.chunk;        // head of the row
            const int j0 = pair ? i : 0, step = pair ? 2 : 1;  // its tiles of keys
            // Whether the row is one of the item's.  The others hold queries of
            // other tokens or heads, or what was in shared memory before.  So that
            // the item's results depend on its own rows alone, they have no say
            // where a warp decides something for its rows together: their maximum
            // begins at +inf, which nothing exceeds, and their capped scores are
            // 0 (or NaN, which a maximum leaves out).
            const bool mine = rj < it.toks && rh < it.heads;
            const int pos = it.pos + min(rj, it.toks - 1);
            const int lo = p.window > 0 ? max(pos - p.window + 1, 0) : 0;
            const int pre = it.pre;
            // positions of the tile's first and last row; all of its rows see
            // all keys of the tiles (of 8 pages) clean_a <= t < clean_b, which
            // lie behind the gap, and t < clean_p, in the prefix
            const int pos_a = it.pos + row0 / p.chunk;
            const int pos_b = it.pos + (min(row0 + kTile, rows) - 1) / p.chunk;
            const int first = p.window > 0 ? max(0, pos_b - p.window + kPage) / kPage - it.gap : 0;
            const int clean_a = (max(first, it.np1) + kPagesPerTile - 1) / kPagesPerTile;
            const int clean_b = max((pos_a + 1) / kPage - it.gap, 0) / kPagesPerTile;
            const int clean_p = (it.gap ? min(pre / kPage, it.np1) : pre / kPage) / kPagesPerTile;
            float slope = 0.f;
            if (kMod && p.slopes && rh < it.heads)
                slope = __ldg(p.slopes + it.head + rh) * 1.4426950408889634f;
            float m = mine ? -INFINITY : INFINITY, l = 0.f;
            [[maybe_unused]] float vref = 0.f, vinv = 0.f;
            for (int j = j0; j < nt; j += step) {
                const int tile = it.tile(j);
                const int v0 = tile * kPagesPerTile + half * kColPages;  // the thread's first page
                // K and V scales of the tile's pages
                const float *scales = reinterpret_cast<const float *>(smem + M::kScales) +
                                      ((tiles + j) & (M::kScaleTiles - 1)) * 2 * kPagesPerTile;
                [[maybe_unused]] const float *ks = scales + half * kColPages;
                [[maybe_unused]] const float *vs = ks + kPagesPerTile;
                ok = wait(s_full(i), steps & 1);
                if (!ok) break;
                ++steps;
                umma::fence_after();
                // Tiles in which some row does not see some key: the rows'
                // seen keys page by page; true if all rows see the whole page.
                const bool clean = (tile >= clean_a && tile < clean_b) || tile < clean_p;
                auto page_seen = [&](int g, uint32_t &seen) {
                    const int t0 = it.real(v0 + g) * kPage;
                    seen = (below(pos + 1 - t0) & ~below(lo - t0)) | below(pre - t0);
                    return (t0 + kPage - 1 <= pos_a && (p.window <= 0 || t0 > pos_b - p.window)) ||
                           t0 + kPage <= pre;
                };
                if constexpr (!kMod) {
                    // masked where they lie, by a loop of a few instructions.  Its
                    // own gain was not measured: the first masked tile took 2600
                    // cycles more than a clean one unrolled on registers and so
                    // alike.  Rolled together with the rows' way out: 8 prompts of
                    // 2048 in 239 against 243 us, 32 of 512 in 114 against 133.
                    if (!clean) {
#pragma unroll 1
                        for (int g = 0; g < kPagesPerTile; ++g) {
                            uint32_t seen;
                            if (page_seen(g, seen)) continue;
                            float s[kPage];
                            umma::ld16(t_s(i) + lanes + kPage * g, s);
                            umma::wait_ld();
#pragma unroll
                            for (int c = 0; c < kPage; ++c)
                                if (!(seen >> c & 1u)) s[c] = -INFINITY;
                            umma::st16(t_s(i) + lanes + kPage * g,
                                       reinterpret_cast<const uint32_t *>(s));
                        }
                        umma::wait_st();
                    }
                }
                float x[kCols];
#pragma unroll
                for (int c = 0; c < kCols; c += 32)
                    umma::ld32(t_s(i) + lanes + half * kCols + c, x + c);
                [[maybe_unused]] float most = 0.f;  // largest V scale of the tile's pages
                // what a product is multiplied with, in log2 units (a page of
                // zeros has scale 0: a masked score must stay -inf)
                auto factor = [&](int g) {
                    if constexpr (!kCodes) return p.scale_log2;
                    const float s = ks[g] * p.scale_log2;
                    return kMod ? s : fmaxf(s, 1e-30f);
                };
                if constexpr (kCodes) {
#pragma unroll
                    for (int g = 0; g < kPagesPerTile; ++g)
                        most = fmaxf(most, scales[kPagesPerTile + g]);
                }
                umma::wait_ld();
                float sl = 1.f;  // kMod: what x is to be multiplied with
                if constexpr (kMod) {
                    const float by = p.cap > 0.f ? (m < INFINITY ? p.cap_inv : 0.f) : 1.f;
#pragma unroll
                    for (int g = 0; g < kColPages; ++g) {
                        const float f = factor(g) * by;
#pragma unroll
                        for (int c = kPage * g; c < kPage * (g + 1); c += 2) {
                            const float2 y = ptx::f32x2_parts(
                                ptx::mul2(ptx::f32x2(x[c], x[c + 1]), ptx::f32x2(f, f)));
                            x[c] = y.x;
                            x[c + 1] = y.y;
                        }
                    }
                    if (p.cap > 0.f) {
                        tanh_row(x);
                        sl = p.cap;
                    }
                    if (p.slopes) {
                        // - slope |pos - t|; keys ahead of a row are seen in the
                        // prefix only
                        const bool ahead = it.real(v0) * kPage < pre;
#pragma unroll
                        for (int g = 0; g < kColPages; ++g) {
                            const float f = static_cast<float>(pos - it.real(v0 + g) * kPage);
                            if (ahead) {
#pragma unroll
                                for (int c = 0; c < kPage; ++c)
                                    x[kPage * g + c] =
                                        fmaf(x[kPage * g + c], sl, -slope * fabsf(f - c));
                            } else {
                                const uint64_t at = ptx::f32x2(-slope * f, -slope * f);
                                const uint64_t s2 = ptx::f32x2(slope, slope);
                                const uint64_t by2 = ptx::f32x2(sl, sl);
#pragma unroll
                                for (int c = 0; c < kPage; c += 2) {
                                    const int e = kPage * g + c;
                                    const float2 y = ptx::f32x2_parts(ptx::fma2(
                                        ptx::f32x2(x[e], x[e + 1]), by2,
                                        ptx::fma2(s2, ptx::f32x2(c, c + 1), at)));
                                    x[e] = y.x;
                                    x[e + 1] = y.y;
                                }
                            }
                        }
                        sl = 1.f;
                    }
                }
                if constexpr (kMod) {
                    if (!clean) {
#pragma unroll
                        for (int g = 0; g < kColPages; ++g) {
                            uint32_t seen;
                            if (page_seen(g, seen)) continue;
#pragma unroll
                            for (int c = 0; c < kPage; ++c)
                                if (!(seen >> c & 1u)) x[kPage * g + c] = -INFINITY;
                        }
                    }
                }
                float top = -INFINITY;
#pragma unroll
                for (int g = 0; g < kColPages; ++g) {
                    const float t = max16(x + kPage * g);
                    top = fmaxf(top, kMod || !kCodes ? t : t * factor(g));
                }
                if constexpr (kMod)
                    top *= sl;
                else if constexpr (!kCodes)
                    top *= p.scale_log2;
                if constexpr (T == 2) {
                    float other = 0.f;
                    ok = swap(top, other, false);
                    if (!ok) break;
                    top = fmaxf(top, other);
                }
                if (__any_sync(0xffffffffu, top > m + kLazy || (kCodes && most > kVLazy * vref))) {
                    const float mn = fmaxf(m, top);
                    const float f = m == -INFINITY ? 0.f : ptx::ex2(m - mn);
                    l *= f;
                    m = mn;
                    float fo = f;
                    if constexpr (kCodes) {
                        // the V reference: the largest of the tile's pages that the
                        // row sees, or what that of earlier pages weighs now
                        if (!clean && most > kVLazy * vref) {
                            float least = most;
#pragma unroll
                            for (int g = 0; g < kPagesPerTile; ++g) {
                                const float y = scales[kPagesPerTile + g];
                                least = y > 0.f ? fminf(least, y) : least;
                            }
                            // (scales that are nearly alike: no need to ask which)
                            if (most > kVLazy * least) {
                                most = 0.f;
#pragma unroll 1
                                for (int g = 0; g < kPagesPerTile; ++g) {
                                    const int t0 = it.real(tile * kPagesPerTile + g) * kPage;
                                    if ((t0 <= pos && t0 + kPage > lo) || t0 < pre)
                                        most = fmaxf(most, scales[kPagesPerTile + g]);
                                }
                            }
                        }
                        if (most <= kVLazy * vref) most = fminf(most, vref);
                        const float vn = fmaxf(fmaxf(most, vref * f), 1e-30f);
                        vinv = __frcp_rn(vn);
                        fo *= vref * vinv;
                        vref = vn;
                    }
                    if (j > j0) {
#pragma unroll 1
                        for (int c = half * (kD / T); c < (half + 1) * (kD / T); c += 16) {
                            float o[16];
                            umma::ld16(t_o(i) + lanes + c, o);
                            umma::wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] *= fo;
                            umma::st16(t_o(i) + lanes + c, reinterpret_cast<const uint32_t *>(o));
                        }
                    }
                }
                // a row that has seen nothing yet: every exponent is -inf
                const float off = kLift - (m == -INFINITY ? 0.f : m);
                const uint64_t off2 = ptx::f32x2(off, off);
                uint64_t sum[2] = {0, 0};
#pragma unroll
                for (int h = 0; h < kCols; h += 32) {
                    uint32_t pk[16];
#pragma unroll
                    for (int g = h / kPage; g < h / kPage + 2; ++g) {
                        const float fy = kMod ? sl : factor(g);
                        const uint64_t f2 = ptx::f32x2(fy, fy);
                        [[maybe_unused]] float vr = 0.f;
                        // (pages that the row does not see have probabilities of 0)
                        if constexpr (kCodes) vr = ptx::min_nan(vs[g] * vinv, 2.f * kVLazy);
#pragma unroll
                        for (int c = kPage * g; c < kPage * (g + 1); c += 2) {
                            const float2 z2 = ptx::f32x2_parts(
                                ptx::fma2(ptx::f32x2(x[c], x[c + 1]), f2, off2));
                            uint64_t y = ptx::f32x2(ptx::ex2(z2.x), ptx::ex2(z2.y));
                            sum[c / 2 & 1] = ptx::add2(sum[c / 2 & 1], y);
                            if constexpr (kCodes) y = ptx::mul2(y, ptx::f32x2(vr, vr));
                            const float2 pr = ptx::f32x2_parts(y);
                            pk[(c - h) / 2] = pack2(pr.x, pr.y);
                        }
                    }
                    umma::st16(t_s(i) + lanes + (half * kCols + h) / 2, pk);
                }
                const float2 both = ptx::f32x2_parts(ptx::add2(sum[0], sum[1]));
                l += both.x + both.y;
                umma::wait_st();
                umma::fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(p_full(i));
            }
            tiles += nt;
            const bool any = j0 < nt;  // the tile had keys to work on
            if (any) {
                ok = ok && wait(o_full(i), outs & 1);
                if (!ok) break;
                ++outs;
                umma::fence_after();
            }
            if constexpr (T == 2) {  // the row's sum, the halves in their order
                float other = 0.f;
                ok = swap(l, other, true);
                if (!ok) break;
                l = half == 0 ? l + other : other + l;
            }
            const bool bad = flags[1 + (k & 1)] != 0;
            int64_t row = static_cast<int64_t>(it.tok + rj) * p.num_heads + it.head + rh;
            if (p.splits > 1) {
                // part 2 z, or 2 z + 1 for the second tile of a pair; the latter
                // is empty where the tiles have rows of their own
                const int64_t all = static_cast<int64_t>(p.num_tokens) * p.num_heads;
                row += (2 * it.z + (pair ? i : 0)) * all;
                if (mine && half == 0) {
                    if (!pair) p.part_ml[row + all] = make_float2(-INFINITY, 0.f);
                    if (!any) p.part_ml[row] = make_float2(-INFINITY, 0.f);
                }
            }
            // the item is not needed any more (and this release waits for no
            // store of the rows)
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(i_empty(k));
            if (!any) continue;
            const float vs = kCodes ? vref : 1.f;
            // The warp's rows leave by way of its 2 KB (T == 2: 1 KB) of shared
            // memory, kPass bytes of each at a time, so that a store instruction
            // writes whole pieces of a few rows and not 16 bytes of 32.  By itself
            // that gained nothing (an item's end took 3700 cycles with direct
            // stores, 4000 staged, both unrolled); staged by a rolled loop it
            // takes 2700.  Direct stores by a rolled loop were not measured.
            // 16-byte chunk c of row r lies at kCh r + (c ^ r kCh / 8 mod kCh).
            constexpr int kPass = M::kOutBytes / (32 * kSoftWarps), kCh = kPass / 16;
            const uint32_t out = base + M::kOut + warp * (32 * kPass);
            const uint32_t put = out + lane * kPass, get = out + (lane / kCh) * kPass;
            const int px = lane * kCh / 8 % kCh, gx = (lane % kCh) ^ (lane / kCh * kCh / 8 % kCh);
            int64_t rows_of[kCh];   // the rows that this lane stores to, or -1
#pragma unroll
            for (int e = 0; e < kCh; ++e)
                rows_of[e] = __shfl_sync(0xffffffffu, mine ? row : int64_t(-1),
                                         32 / kCh * e + lane / kCh);
            auto store = [&](const uint4 (&v)[kCh], uint8_t *to, int row_bytes) {
#pragma unroll
                for (int c = 0; c < kCh; ++c) st_shared16(put + ((c ^ px) << 4), v[c]);
                __syncwarp();
#pragma unroll
                for (int e = 0; e < kCh; ++e) {
                    const uint4 w = ptx::lds128(get + e * (32 / kCh * kPass) + (gx << 4));
                    if (rows_of[e] >= 0)
                        *reinterpret_cast<uint4 *>(to + rows_of[e] * row_bytes +
                                                   (lane % kCh) * 16) = w;
                }
                __syncwarp();
            };
            const int c0 = half * (kD / T), c1 = c0 + kD / T;   // the thread's columns of O
            if (p.splits == 1) {
                const float f = l > 0.f ? vs / l : l;  // an empty row: zeros; NaN stays
#pragma unroll 1
                for (int c = c0; c < c1; c += kPass / 2) {
                    float o[kPass / 2];
#pragma unroll
                    for (int e = 0; e < kPass / 2; e += 16) umma::ld16(t_o(i) + lanes + c + e, o + e);
                    umma::wait_ld();
                    uint4 v[kCh];
#pragma unroll
                    for (int e = 0; e < kPass / 2; ++e) o[e] = bad ? 0.f : o[e] * f;
#pragma unroll
                    for (int e = 0; e < kCh; ++e)
                        v[e] = make_uint4(
                            pack2(o[8 * e], o[8 * e + 1]), pack2(o[8 * e + 2], o[8 * e + 3]),
                            pack2(o[8 * e + 4], o[8 * e + 5]), pack2(o[8 * e + 6], o[8 * e + 7]));
                    store(v, reinterpret_cast<uint8_t *>(p.out + c), kD * 2);
                }
            } else {
                if (mine && half == 0) p.part_ml[row] = make_float2(m, bad ? -1.f : l);
#pragma unroll 1
                for (int c = c0; c < c1; c += 16) {
                    float o[16];
                    umma::ld16(t_o(i) + lanes + c, o);
                    umma::wait_ld();
#pragma unroll
                    for (int q = 0; q < 16; q += kPass / 4) {
                        uint4 v[kCh];
#pragma unroll
                        for (int e = 0; e < kCh; ++e)
                            v[e] = make_uint4(__float_as_uint(o[q + 4 * e] * vs),
                                              __float_as_uint(o[q + 4 * e + 1] * vs),
                                              __float_as_uint(o[q + 4 * e + 2] * vs),
                                              __float_as_uint(o[q + 4 * e + 3] * vs));
                        store(v, reinterpret_cast<uint8_t *>(p.part_acc + c + q), kD * 4);
                    }
                }
            }
            // (the next item's first product into O waits for this tile's next
            // probabilities, which come after this)
            umma::fence_before();
        }
    } else if (warp < kSoftWarps + 4) {
        issue_registers<kKv, kMod>();
        if (warp == kSoftWarps) {
            // ------------------------------------------------ products
            const Waiter wait = waiter.as(kRoleProducts);
            if (umma::elect_one()) {
                constexpr uint32_t kQk = umma::f16_idesc(kTile, kTile, false);
                constexpr uint32_t kPv = umma::f16_idesc(kTile, kD, true);
                // low descriptor words; the ring advances by whole tiles
                const uint32_t q_lo = umma::desc_lo(base, 16);
                const uint32_t k_lo = umma::desc_lo(base + M::kRing, 16);
                const uint32_t v_lo = umma::desc_lo(base + M::kRing, M::kHalfBytes);
                auto qk = [&](int i, int rows, int s) {  // S_i = Q_rows K^T
                    const uint32_t a = q_lo + rows * (M::kHalfBytes >> 4);
                    const uint32_t b = k_lo + s * (M::kTileBytes >> 4);
#pragma unroll
                    for (int k = 0; k < kD / 16; ++k)
                        umma::mma_ss(
                            t_s(i),
                            umma::desc(a + (((k >> 2) * M::kQHalfBytes + (k & 3) * 32) >> 4)),
                            umma::desc(b + (((k >> 2) * M::kHalfBytes + (k & 3) * 32) >> 4)), kQk,
                            k > 0);
                    umma::commit(s_full(i));
                };
                auto pv = [&](int i, int s, bool more) {  // O_i += P_i V
                    const uint32_t b = v_lo + s * (M::kTileBytes >> 4);
#pragma unroll
                    for (int k = 0; k < kTile / 16; ++k)
                        umma::mma_ts(t_o(i), t_s(i) + 8 * k, umma::desc(b + k * (2048 >> 4)), kPv,
                                     more || k > 0);
                };
                int s = 0;                   // next stage of the ring
                uint32_t phase = 0;          // its parity
                auto advance = [&]() {
                    if (++s == S) {
                        s = 0;
                        phase ^= 1;
                    }
                };
                [[maybe_unused]] uint32_t fixes = 0;  // parity of each stage's fixes
                // K or V of the j-th tile of keys has landed in stage sv
                auto ready = [&](bool fix, const Item &it, int j, int sv, uint32_t ph) -> bool {
                    bool ok = wait.one(full(sv), ph);
                    if (!kCodes && fix && ok && it.dirty(it.tile(j))) {
                        ok = wait.one(fixed(sv), fixes >> sv & 1u);
                        fixes ^= 1u << sv;
                    }
                    return ok;
                };
                auto v_ready = [&](const Item &it, int j, int sv, uint32_t ph) -> bool {
                    return ready(true, it, j, sv, ph);
                };
                auto k_ready = [&](const Item &it, int j, int sv, uint32_t ph) -> bool {
                    return ready(kMod && p.cap > 0.f, it, j, sv, ph);
                };
                uint32_t steps[2] = {0, 0};
                bool ok = true;
                for (int k = 0; ok; ++k) {
                    ok = wait.one(i_full(k), k >> 1 & 1);
                    if (!ok) break;
                    const Item &it = item(k);
                    const int nt = it.nt;
                    if (nt == 0) break;
                    ok = wait.one(q_full, k & 1) && k_ready(it, 0, s, phase);
                    if (!ok) break;
                    umma::fence_after();
                    if (!paired(p, it)) {
                        // every tile of keys for one or two tiles of rows
                        const int last = it.toks * p.chunk > kTile ? 1 : 0;
                        qk(0, 0, s);
                        if (last) qk(1, 1, s);
                        umma::commit(empty(s));
                        if (nt == 1) umma::commit(q_empty);
                        advance();
                        for (int j = 0; j < nt && ok; ++j) {
                            const int sv = s;
                            ok = v_ready(it, j, sv, phase);
                            if (!ok) break;
                            advance();
                            for (int i = 0; i <= last; ++i) {
                                ok = wait.one(p_full(i), steps[i] & 1);
                                if (!ok) break;
                                ++steps[i];
                                umma::fence_after();
                                pv(i, sv, j > 0);
                                if (i == last) umma::commit(empty(sv));
                                if (j + 1 < nt) {
                                    if (i == 0) {
                                        ok = k_ready(it, j + 1, s, phase);
                                        if (!ok) break;
                                        umma::fence_after();
                                    }
                                    qk(i, i, s);
                                    if (i == last) {
                                        umma::commit(empty(s));
                                        if (j + 2 == nt) umma::commit(q_empty);
                                    }
                                } else {
                                    umma::commit(o_full(i));
                                }
                            }
                            if (j + 1 < nt) advance();
                        }
                    } else {
                        // the tiles of keys in turn for the two tiles, which
                        // share the rows; K is two elements of the ring ahead
                        qk(0, 0, s);
                        umma::commit(empty(s));
                        if (nt == 1) umma::commit(q_empty);
                        advance();
                        for (int j = -1; j < nt && ok; ++j) {
                            // (j = -1: only the second tile's first product)
                            const int i = j & 1, sv = s;
                            const uint32_t ph = phase;
                            if (j >= 0) {
                                ok = v_ready(it, j, sv, ph) && wait.one(p_full(i), steps[i] & 1);
                                if (!ok) break;
                                ++steps[i];
                                umma::fence_after();
                                pv(i, sv, j > 1);
                                umma::commit(empty(sv));
                                advance();          // K of j + 1, taken before
                                if (j + 1 < nt) advance();
                            }
                            if (j + 2 < nt) {
                                const int sk = s + 1 == S ? 0 : s + 1;
                                ok = k_ready(it, j + 2, sk, s + 1 == S ? phase ^ 1 : phase);
                                if (!ok) break;
                                umma::fence_after();
                                qk(i, 0, sk);
                                umma::commit(empty(sk));
                                if (j + 3 == nt) umma::commit(q_empty);
                            } else if (j >= 0) {
                                umma::commit(o_full(i));
                            }
                        }
                    }
                    ptx::mbar_arrive(i_empty(k));
                }
                // nothing of this thread's is in flight after this
                umma::commit(drain);
                ptx::mbar_wait_bounded(drain, 0, kWaitLimitNs);
            }
            __syncwarp();
        } else if (warp == kSoftWarps + 1 || warp == kSoftWarps + 3) {
            // ------------------------------------------------ loads of Q and the pages
            // One warp for K and Q, one for V.  A lane per page looks its
            // block up; one thread issues the copies, 2 KB of a page each (16
            // copies and the loop around them: 1000 to 1100 cycles, and 1600 to
            // 2000 when every lane issued its own).
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
                const Item &it = item(k);
                const int nt = it.nt;
                if (nt == 0) break;
                const int32_t *table =
                    p.block_tables + static_cast<int64_t>(it.seq) * p.max_blocks_per_seq;
                auto lookup = [&](int j) -> int32_t {  // block of the lane's page, -2: none
                    const int v = it.tile(j) * kPagesPerTile + lane;
                    return lane < kPagesPerTile && v < it.visited ? __ldg(table + it.real(v)) : -2;
                };
                int32_t blk = lookup(0);
                for (int j = 0; j < nt; ++j) {
                    const uint32_t n = 2 * tiles + (is_v ? 1 : 0);
                    const int s = n % R;
                    const bool have = blk >= 0 && blk < p.num_blocks;
                    if (blk != -2 && !have) {
                        flags[1 + (k & 1)] = 1;
                        if (p.dev_status) atomicOr(p.dev_status, PKV_DEV_BAD_BLOCK);
                    }
                    // both scales by the K warp: see Smem::kScales
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
                    ok = wait(eb, ((n / R) & 1) ^ 1);
                    if (!ok) break;
                    if (j + 1 < nt) blk = lookup(j + 1);
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
                    for (int g = 0; g < kPagesPerTile; ++g) {
                        const int y = __shfl_sync(0xffffffffu, row, g);
                        if ((pages >> g & 1u) && umma::elect_one()) {
#pragma unroll
                            for (int b = 0; b < kBoxes; ++b)
                                ptx::tma_load_2d(dst + b * M::kHalfBytes + g * kBoxBytes, tm,
                                                 b * kBox, y, fb);
                        }
                    }
                    __syncwarp();
                    ++tiles;
                    if (!is_v && j == 0) {
                        // the queries: tokens x heads x 64 values, which land as
                        // the item's rows in their order (rows of heads that
                        // are not the item's, or behind the batch, do not count)
                        ok = wait(q_empty, (k & 1) ^ 1);
                        if (!ok) break;
                        if (umma::elect_one()) {
                            ptx::mbar_arrive_expect_tx(q_full,
                                                       p.tokens * p.chunk * M::kHalves * 128);
#pragma unroll
                            for (int b = 0; b < M::kHalves; ++b)
                                ptx::tma_load_3d(base + b * M::kQHalfBytes, &tmq, b * 64, it.head,
                                                 it.tok, q_full);
                        }
                        __syncwarp();
                        ++queries;
                    }
                    if constexpr (!kCodes)
                        if ((is_v || (kMod && p.cap > 0.f)) && it.dirty(it.tile(j))) {
                            // rows of V that no row of the item sees may hold
                            // anything, NaN included (and are not loaded for
                            // pages past the last): zeros.  So are K's ahead of a
                            // cap, whose polynomial the largest score chooses (2048
                            // over 8192, capped: 271 us; with the scores of unseen
                            // keys set to 0 in TMEM 275, in registers 281).  The
                            // products wait for this, so the stage is not filled
                            // meanwhile.
                            ok = wait(fb, (n / R) & 1);
                            if (!ok) break;
                            const int v = it.tile(j) * kPagesPerTile + lane;
                            uint32_t lv = 0xffffu;
                            if (lane < kPagesPerTile)
                                lv = v < it.visited ? it.live(it.real(v) * kPage) : 0u;
                            unsigned todo = __ballot_sync(0xffffffffu, lv != 0xffffu);
                            while (todo) {
                                const int g = __ffs(todo) - 1;
                                todo &= todo - 1;
                                const uint32_t keep = __shfl_sync(0xffffffffu, lv, g);
                                for (int e = lane; e < kPage * kRowChunks; e += 32) {
                                    const int row = e / kRowChunks, ch = e % kRowChunks;
                                    if (!(keep >> row & 1u))
                                        st_shared16(dst + (ch >> 3) * M::kHalfBytes +
                                                        (g * kPage + row) * 128 + ((ch & 7) << 4),
                                                    make_uint4(0, 0, 0, 0));
                                }
                            }
                            ptx::fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) ptx::mbar_arrive(fixed(s));
                        }
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(i_empty(k));
            }
            // The products have waited for every copy, unless a wait ran out:
            // what was issued, for the drain behind it.
            if (lane == 0) {
                issued[is_v] = static_cast<int>(tiles);
                if (!is_v) issued[2] = queries;
            }
        } else {
            // ------------------------------------------------ the next items
            const Waiter wait = waiter.as(kRoleItems);
            int block = blockIdx.x;
            bool ok = true;
            int k = 0;
            // Where the sequences are looked at changes nothing but where the other
            // roles' code lies, and with it the time.  Out of line next to the item /
            // inlined behind the loop: INT8 with bias and window (12 chunks) 294 /
            // 283 us, 4 prompts capped at head_dim 64 116 / 108, 8 prompts capped
            // INT8 476 / 464; the other way around 8 prompts capped fp16 369 / 393,
            // INT8 299 / 307.
            constexpr bool kLate = kMod && (kCodes || kD == 64);
            [[maybe_unused]] bool first = false;
            for (uint32_t asked = 0; ok; ++asked) {
                if (umma::elect_one()) {
                    ptx::mbar_arrive_expect_tx(next_full, 16);
                    ptx::try_cancel(base + M::kNext, next_full);
                }
                __syncwarp();
                Item it;
                const int what = find_item(p, block, it);
                if (what > 0) {
                    ok = wait(i_empty(k), (k >> 1 & 1) ^ 1);
                    if (ok && lane == 0) {
                        item(k) = it;
                        flags[1 + (k & 1)] = 0;
                        ptx::mbar_arrive(i_full(k));
                    }
                    __syncwarp();
                    ++k;
                } else if (what == 0) {
                    // a sequence that does not fit (zeros), or a split without keys
                    for (int e = lane; e < it.toks * it.heads * kRowChunks; e += 32) {
                        const int q = e / kRowChunks, t = it.tok + q / it.heads;
                        const int64_t row =
                            static_cast<int64_t>(t) * p.num_heads + it.head + q % it.heads;
                        if (t < 0 || t >= p.num_tokens) continue;
                        if (p.splits == 1)
                            reinterpret_cast<uint4 *>(p.out + row * kD)[e % kRowChunks] =
                                make_uint4(0, 0, 0, 0);
                        else if (e % kRowChunks == 0)
                            for (int part = 2 * it.z; part < 2 * it.z + 2; ++part)
                                p.part_ml[static_cast<int64_t>(part) * p.num_tokens * p.num_heads +
                                          row] = make_float2(-INFINITY, 0.f);
                    }
                }
                if constexpr (kLate)
                    first |= block == 0;
                else if (block == 0 && p.dev_status)
                    check_sequences(p, lane);
                // (also after a wait that ran out: the answer must have come)
                if (!wait(next_full, asked & 1)) {
                    ptx::mbar_wait_bounded(next_full, asked & 1, kWaitLimitNs);
                    ok = false;
                }
                if (!ok || !ptx::cancelled_block(base + M::kNext, block)) break;
                ptx::fence_proxy_async_smem();  // read before the next answer is written
            }
            if (kLate && first && p.dev_status)
                report_bad_sequences(p.query_starts, p.context_lens, p.num_seqs, p.num_tokens,
                                     p.ctx_cap, p.dev_status, lane, 32);
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
            widen_registers<kMod>();
            const Waiter wait = waiter.as(kRoleWiden);
            constexpr int R = M::kCodeStages;
            constexpr int kCh = kD / 16;  // 16-byte chunks of codes per row
            constexpr int kStep = 128 / kCh;
            const int tid = threadIdx.x - 32 * (kSoftWarps + 4);
            uint32_t n = 0;
            bool ok = true;
            for (int k = 0; ok; ++k) {
                ok = wait(i_full(k), k >> 1 & 1);
                if (!ok) break;
                const Item &it = item(k);
                const int nt = it.nt;
                if (nt == 0) break;
                for (int j = 0; j < 2 * nt; ++j, ++n) {
                    ok = wait(cfull(n % R), (n / R) & 1) && wait(empty(n % S), ((n / S) & 1) ^ 1);
                    if (!ok) break;
                    const uint32_t src = base + M::kCodeRing + (n % R) * M::kCodeBytes;
                    const uint32_t dst = base + M::kRing + (n % S) * M::kTileBytes;
                    const int v0 = it.tile(j / 2) * kPagesPerTile;
                    // (INT8 codes are finite; for K see the load warps)
                    const bool dirty = (j & 1 ? kKv == kKvF8 : kMod && p.cap > 0.f) &&
                                       it.dirty(it.tile(j / 2));
                    // all loads first: the thread's row advances by kStep
                    const int ch = tid % kCh, row0 = tid / kCh;
                    constexpr int kAt = kMod && kCh > 4 ? 4 : kCh;   // registers
#pragma unroll
                    for (int e0 = 0; e0 < kCh; e0 += kAt) {
                        uint4 w[kAt];
#pragma unroll
                        for (int e = 0; e < kAt; ++e) {
                            const int row = row0 + (e0 + e) * kStep;
                            const uint32_t sx =
                                kD == 128 ? (ch ^ (row & 7)) : (ch ^ ((row >> 1) & 3));
                            w[e] = ptx::lds128(src + row * kD + (sx << 4));
                        }
#pragma unroll
                        for (int e = 0; e < kAt; ++e) {
                            const int row = row0 + (e0 + e) * kStep;
                            const uint4 a = widen<kKv>(w[e].x, w[e].y);
                            const uint4 b = widen<kKv>(w[e].z, w[e].w);
                            const uint32_t to = dst + (ch >> 2) * M::kHalfBytes + row * 128;
                            const int cc = (2 * ch) & 7;
                            st_shared16(to + ((cc ^ (row & 7)) << 4), a);
                            st_shared16(to + (((cc + 1) ^ (row & 7)) << 4), b);
                        }
                    }
                    // the thread's rows that no row of the item sees (in a loop of
                    // their own: next to the widening FP8 took 227 against 207 us)
                    if (dirty)
#pragma unroll 1
                        for (int row = row0; row < kTile; row += kStep) {
                            const int v = v0 + (row >> 4);
                            const uint32_t lv = v < it.visited ? it.live(it.real(v) * kPage) : 0u;
                            if (lv >> (row & 15) & 1u) continue;
                            const uint32_t to = dst + (ch >> 2) * M::kHalfBytes + row * 128;
                            const int cc = (2 * ch) & 7;
                            const uint4 zero = make_uint4(0, 0, 0, 0);
                            st_shared16(to + ((cc ^ (row & 7)) << 4), zero);
                            st_shared16(to + (((cc + 1) ^ (row & 7)) << 4), zero);
                        }
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        ptx::mbar_arrive(full(n % S));
                        ptx::mbar_arrive(cempty(n % R));
                    }
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(i_empty(k));
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

// Joins the parts of every row, four warps a row.
//   out = sum_z 2^(m_z - M) acc_z / sum_z 2^(m_z - M) l_z,  M = max_z m_z
// Every lane fetches the maxima and sums of its parts, then the lanes lie along
// head_dim: warp w adds up parts w, w + 4, .., eight loads in flight, and the
// warps' sums are added in their order.  A part with l < 0 (a bad block) makes
// the row zeros.  Rows that no sequence owns have no parts and are left alone.
constexpr int kJoinWarps = 4;

template <int kD>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const __grid_constant__ PrefillArgs p)
{
    constexpr int kC = kD / 32;
    __shared__ float sums[kJoinWarps][kD];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t all = static_cast<int64_t>(p.num_tokens) * p.num_heads;
    const int64_t row = blockIdx.x;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    // lane z: part z's (and z + 32's ..) maximum and sum
    constexpr int kPer = 2 * kMaxSplits / 32;
    const int parts = 2 * p.splits;
    float pm[kPer], pl[kPer], m = -INFINITY;
    bool bad = false;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        const int z = lane + 32 * e;
        const float2 ml =
            z < parts ? __ldcg(p.part_ml + z * all + row) : make_float2(-INFINITY, 0.f);
        pm[e] = ml.x;
        pl[e] = ml.y;
        m = fmaxf(m, ml.x);
        bad |= ml.y < 0.f;
    }
    // (whose row it is, while the parts' maxima are on their way)
    const int tok = static_cast<int>(row / p.num_heads);
    const int seq = warp_search(p.num_seqs, tok, [&](int s) { return __ldg(p.query_starts + s); });
    if (seq < 0) return;
    SeqRows sr;
    sr.load(p.query_starts, p.context_lens, seq, p.num_tokens, p.ctx_cap);
    if (tok - sr.start >= sr.len) return;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    bad = __any_sync(0xffffffffu, bad);
    float l = 0.f;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        // the part's factor (0 where no key was seen: it has no accumulators)
        pm[e] = pl[e] == 0.f ? 0.f : ptx::ex2(pm[e] - m);
        l += pm[e] * pl[e];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    float acc[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) acc[c] = 0.f;
    const float *src = p.part_acc + row * kD + lane * kC;
#pragma unroll
    for (int e = 0; e < kPer; ++e)
        if (32 * e < parts) {
            float v[8][kC], f[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int z = warp + kJoinWarps * u;   // of these 32
                f[u] = __shfl_sync(0xffffffffu, pm[e], z);
#pragma unroll
                for (int c = 0; c < kC; ++c) v[u][c] = 0.f;
                if (f[u] != 0.f) {
                    const float *a = src + (32 * e + z) * all * kD;
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
            }
#pragma unroll
            for (int u = 0; u < 8; ++u)
#pragma unroll
                for (int c = 0; c < kC; ++c) acc[c] += f[u] * v[u][c];
        }
#pragma unroll
    for (int c = 0; c < kC; ++c) sums[warp][lane * kC + c] = acc[c];
    __syncthreads();
    const int c = 2 * threadIdx.x;
    if (c < kD) {
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) {
            a += sums[w][c];
            b += sums[w][c + 1];
        }
        const bool zero = bad || l == 0.f;
        *reinterpret_cast<__half2 *>(p.out + row * kD + c) =
            __floats2half2_rn(zero ? 0.f : a / l, zero ? 0.f : b / l);
    }
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
    int chunk = 0, chunks = 0, tokens = 0;
    int64_t units = 0;
    int splits = 1;
    size_t bytes = 0;
};

// Units of the batch and the number of key splits, from the sizes alone: the one
// with the least time by this model, fitted to fp16 calls of 8 to 464 items with
// 1 to 19 splits (times in us).
//   A tile (128 keys for 256 rows) takes 1.45 at head_dim 128, half of that at
//   64, and an item 2 more (queries, epilogue).  Where items hold one tile of
//   rows on average and do not fill the SMs, split ones share theirs: 0.63 of it.
//   With contexts of max_context_len, whose last tokens the rows are, items have
//   from `least` to `most` tiles.  w = items / SMs of them come one after the
//   other on an SM, the longest first: the SMs are through after w mean items,
//   and where w is not whole some of them a short item later, but no earlier
//   than the longest item.
//   Splits write their accumulators in fp32 and a launch joins them: 1.5, and
//   1.05 + 0.125 splits for every 1000 rows (tokens times heads).
// Unsplit against two splits: one prompt of 4096 (32 / 8 heads, head_dim 128) 113
// and 277 us, of 2048 (28 / 4) 40 and 115, 4096 tokens over 16384 650 and 756
// (capped 1021 and 1089); the other way around, 256 over 4096: 51 and 44 (37 with
// three), 128 over 8192: 95 and 60 (33 with six).
pkv_status plan_of(int num_tokens, int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                   int max_context_len, Plan *plan)
{
    if (num_tokens < 0 || num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
        max_context_len < 0 || num_heads % num_kv_heads != 0)
        return PKV_ERR_INVALID_ARG;
    if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
    const int group = num_heads / num_kv_heads;
    plan->chunk = group < kRows ? group : kRows;
    plan->chunks = (group + plan->chunk - 1) / plan->chunk;
    plan->tokens = kRows / plan->chunk;
    plan->units = num_tokens / plan->tokens + static_cast<int64_t>(num_seqs);
    const int64_t items = plan->units * num_kv_heads * plan->chunks;
    const int64_t tiles = (static_cast<int64_t>(max_context_len) + kTile - 1) / kTile + 1;
    if (plan->units > INT32_MAX || items * kMaxSplits > INT32_MAX)
        return PKV_ERR_UNSUPPORTED;
    plan->splits = 1;
    if (num_seqs > 0 && items < 4 * kSms) {  // (beyond, at most a fourth of the time is idle)
        const double krows = static_cast<double>(num_tokens) * num_heads / 1000;
        const double own = static_cast<double>(num_tokens) / num_seqs;
        const double most = static_cast<double>(max_context_len) / kTile;
        const double least = most > own / kTile ? most - own / kTile : 0.0;
        const double tile = 1.45 * head_dim / 128, item = 2.0;
        double best = 0.0;
        for (int z = 1; z <= kMaxSplits && z <= tiles; ++z) {
            const double w = static_cast<double>(items) * z / kSms;
            const bool shared = z > 1 && w <= 1.0 && own * plan->chunk <= kTile;
            const double t = (shared ? 0.63 * tile : tile) / z;
            double us = w * ((most + least) / 2 * t + item) + (ceil(w) - w) * (least * t + item);
            if (us < most * t + item) us = most * t + item;
            if (z > 1) us += 1.5 + (1.05 + 0.125 * z) * krows;
            if (z == 1 || us < best) {
                best = us;
                plan->splits = z;
            }
        }
    }
    plan->bytes = plan->splits == 1 ? 0
                                    : static_cast<size_t>(2 * plan->splits) * num_tokens * num_heads *
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
    CUtensorMap tmq, tmk, tmv;
    const uint64_t rows = static_cast<uint64_t>(c.num_blocks) * c.num_kv_heads * kPage;
    const int elem = M::kCodes ? 1 : 2, box = M::kCodes ? kD : 64;
    const int swizzle = box * elem;
    if (!encode_tmap_3d_f16(&tmq, c.query, kD, c.num_heads, c.num_tokens, 64, plan.chunk, plan.tokens))
        return PKV_ERR_CUDA;
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
        a.part_acc + static_cast<size_t>(2 * plan.splits) * c.num_tokens * c.num_heads * kD);
    a.dev_status = c.dev_status;
    a.num_tokens = c.num_tokens;
    a.num_seqs = c.num_seqs;
    a.num_heads = c.num_heads;
    a.num_kv_heads = c.num_kv_heads;
    a.group = c.num_heads / c.num_kv_heads;
    a.chunk = plan.chunk;
    a.chunks = plan.chunks;
    a.tokens = plan.tokens;
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
    cfg.gridDim =
        dim3(static_cast<unsigned>(plan.units * c.num_kv_heads * plan.chunks * plan.splits));
    cfg.blockDim = dim3(prefill_threads<kKv, kMod>());
    cfg.dynamicSmemBytes = M::kAsk;
    cfg.stream = static_cast<cudaStream_t>(c.stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a, tmq, tmk, tmv);
    if (e == cudaSuccess && plan.splits > 1) {
        const int64_t all = static_cast<int64_t>(c.num_tokens) * c.num_heads;
        cfg.gridDim = dim3(static_cast<unsigned>(all));
        cfg.blockDim = dim3(32 * kJoinWarps);
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
    if (!c.kpool || !c.vpool || !c.query_starts) return PKV_ERR_INVALID_ARG;
    // (arrays without elements may be null)
    if (c.num_tokens != 0 && (!c.out || !c.query)) return PKV_ERR_INVALID_ARG;
    if (c.num_seqs != 0 && (!c.context_lens || (!c.block_tables && c.max_blocks_per_seq != 0)))
        return PKV_ERR_INVALID_ARG;
    if (codes && (!c.k_scales || !c.v_scales)) return PKV_ERR_INVALID_ARG;
    if (c.num_blocks <= 0 || c.block_size <= 0 || c.max_blocks_per_seq < 0 || c.window < 0)
        return PKV_ERR_INVALID_ARG;
    if (!(fabsf(c.softmax_scale) <= 2.0e38f) || !valid_cap(c.logit_cap)) return PKV_ERR_INVALID_ARG;
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
    const bool mod = c.logit_cap > 0.f || c.slopes || !(c.softmax_scale > 0.f);
    auto pick = [&](auto kind) -> pkv_status {
        constexpr int kKv = decltype(kind)::value;
        if (c.head_dim == 128)
            return mod ? launch_prefill<kKv, 128, true>(c, plan)
                       : launch_prefill<kKv, 128, false>(c, plan);
        return mod ? launch_prefill<kKv, 64, true>(c, plan)
                   : launch_prefill<kKv, 64, false>(c, plan);
    };
    if (kv == kKvF8) return pick(std::integral_constant<int, kKvF8>());
    if (kv == kKvI8) return pick(std::integral_constant<int, kKvI8>());
    return pick(std::integral_constant<int, kKvF16>());
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

#ifdef PKV_DEBUG
// Debug builds only: see PrefillDebug (roles 0 rows, 1 products, 2 K and query
// loads, 3 V loads, 4 items, 5 widening of codes).  A negative role resets its
// setting.  Synchronises with the device; returns 0, or -1 if the CUDA runtime
// fails or an argument is out of range.
extern "C" __attribute__((visibility("default"))) int pkv_debug_set_prefill(int give_role,
                                                                            int give_at,
                                                                            int slow_role,
                                                                            int slow_ns)
{
    if (give_role >= pkv::kRoles || slow_role >= pkv::kRoles || slow_ns < 0 || slow_ns > 1000000)
        return -1;
    const pkv::PrefillDebug d = {give_role < 0 ? -2 : give_role, give_at,
                                 slow_role < 0 ? -2 : slow_role, slow_ns};
    if (cudaDeviceSynchronize() != cudaSuccess ||
        cudaMemcpyToSymbol(pkv::g_prefill_debug, &d, sizeof(d)) != cudaSuccess)
        return -1;
    return 0;
}
#endif
