// pkv_score.cuh -- what the attention kernels do to a score before the softmax:
// the cap by a tanh, and which tokens of a page are seen.
#pragma once

#include <stdint.h>

#include "pkv_ptx.cuh"

namespace pkv {

// The 16-bit mask of a page's tokens (its first is t0) below ctx that lie
// in the window (from lo on) or in the prefix (below pre).
__device__ __forceinline__ uint32_t below(int n)
{
    return n >= 16 ? 0xffffu : n <= 0 ? 0u : (1u << n) - 1u;
}

__device__ __forceinline__ uint32_t seen_mask(int t0, int ctx, int lo, int pre)
{
    return below(ctx - t0) & (~below(lo - t0) | below(pre - t0));
}

// cap * tanh(x / cap) of a score in log2 units.  Away from zero 1 - 2 / (1 +
// e^2u) has an absolute error of some 2^-23; near zero it would lose the
// score's relative precision, so |u| < 1/4 takes the series of tanh up to
// u^9, whose first omitted term, 1382/155925 u^11, is 1e-8 of u there.
__device__ __forceinline__ float cap_score(float x, float cap, float cap_inv)
{
    const float u = x * cap_inv, w = u * u;
    const float poly = x + x * w *
        fmaf(w, fmaf(w, fmaf(w, 62.f / 2835.f, -17.f / 315.f), 2.f / 15.f), -1.f / 3.f);
    const float e = ptx::ex2(u * 2.885390081777927f);
    const float far = fmaf(-2.f * cap, __fdividef(1.f, 1.f + e), cap);
    return w < 0.0625f ? poly : far;
}

}  // namespace pkv
