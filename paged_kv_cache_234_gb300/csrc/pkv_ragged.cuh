// pkv_ragged.cuh -- a ragged batch of new tokens: sequence s owns the rows
// query_starts[s] .. query_starts[s + 1) of the [num_tokens] arrays, and its
// tokens are the last ones of its context_lens[s] cached tokens.
//
// Work that is handed out in units of `per` rows (16 tokens, 256 query rows)
// is numbered without a prefix sum: with a = rows per token, sequence s owns
// the units from floor(starts[s] * a / per) + s * extra on.  `extra` units per
// sequence cover the rounding, so the ranges never meet, and a few numbers
// name no unit.  The owner of a unit is found by a search over
// query_starts, 32 candidates a step.
#pragma once

#include <stdint.h>

#include "../../include/pkv.h"

namespace pkv {

// Largest s in [0, n) with key(s) <= x for a nondecreasing key; -1 if there
// is none.  All 32 lanes of a warp call it with the same arguments.  Whatever
// key() returns, only arguments in [0, n) are asked for.
template <typename Key>
__device__ __forceinline__ int warp_search(int n, int64_t x, Key key)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, span = n;
    while (span > 32) {
        const int step = (span + 31) >> 5;
        const int off = lane * step;
        const bool le = off < span && key(lo + off) <= x;
        const unsigned m = __ballot_sync(0xffffffffu, le);
        const int c = __ffs(~m) - 1;  // leading run of candidates that pass
        if (c == 0) return lo - 1;
        const int run = c < 0 ? 32 : c;
        lo += (run - 1) * step;
        span = min(step, span - (run - 1) * step);
    }
    const bool le = lane < span && key(lo + lane) <= x;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    return lo + (m == 0xffffffffu ? 32 : __ffs(~m) - 1) - 1;
}

// One sequence of the batch, as the caller's arrays describe it.
struct SeqRows {
    int start = 0;   // first row
    int len = 0;     // rows (new tokens)
    int ctx = 0;     // cached tokens, the new ones included
    bool ok = false; // 0 <= start, start + len <= num_tokens, len <= ctx <= ctx_cap

    __device__ __forceinline__ void load(const int32_t *__restrict__ starts,
                                         const int32_t *__restrict__ lens, int s, int num_tokens,
                                         int ctx_cap)
    {
        set(__ldg(starts + s), __ldg(starts + s + 1), __ldg(lens + s), num_tokens, ctx_cap);
    }

    __device__ __forceinline__ void set(int first, int end, int cached, int num_tokens, int ctx_cap)
    {
        start = first;
        ctx = cached;
        const int64_t l = static_cast<int64_t>(end) - first;
        ok = start >= 0 && l >= 0 && start + l <= num_tokens && l <= ctx && ctx <= ctx_cap;
        len = l < 0 ? 0 : l > num_tokens ? num_tokens : static_cast<int>(l);
    }
};

// Sets PKV_DEV_BAD_CTX if a sequence with rows does not fit, wherever its rows
// would begin.  By `threads` threads, of which this is number t.
__device__ __forceinline__ void report_bad_sequences(const int32_t *__restrict__ starts,
                                                     const int32_t *__restrict__ lens, int num_seqs,
                                                     int num_tokens, int ctx_cap,
                                                     int32_t *dev_status, int t, int threads)
{
    bool bad = false;
    for (int s = t; s < num_seqs; s += threads) {
        SeqRows sr;
        const int first = __ldg(starts + s), end = __ldg(starts + s + 1);
        sr.set(first, end, __ldg(lens + s), num_tokens, ctx_cap);
        bad |= first != end && !sr.ok;
    }
    if (bad) atomicOr(dev_status, static_cast<int32_t>(PKV_DEV_BAD_CTX));
}

}  // namespace pkv
