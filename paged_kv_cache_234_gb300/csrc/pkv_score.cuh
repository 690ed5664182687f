// pkv_score.cuh -- what the attention kernels do to a score before the softmax:
// the cap by a tanh, and which tokens of a page are seen.
#pragma once

#include <stdint.h>

#include "pkv_ptx.cuh"

namespace pkv {

// A cap that the host lets through: none, or one whose value and reciprocal in
// log2 units are normal fp32 numbers.
inline bool valid_cap(float cap)
{
    return cap == 0.f || (cap >= 1e-30f && cap <= 1e30f);
}

// The 16-bit mask of a page's tokens (its first is t0) below ctx that lie
// in the window (from lo on) or in the prefix (below pre).  None of the bounds
// is negative.
__device__ __forceinline__ uint32_t below(int n)
{
    return n >= 16 ? 0xffffu : n <= 0 ? 0u : (1u << n) - 1u;
}

__device__ __forceinline__ uint32_t seen_mask(int t0, int ctx, int lo, int pre)
{
    return below(ctx - t0) & (~below(lo - t0) | below(pre - t0));
}

// cap * tanh(x / cap) of a score in log2 units, u = x / cap.  For |u| <= 1 the
// polynomial x P(u^2), P of degree 6 with the least maximum relative error
// against tanh(u) / u on [0, 1] (iteratively reweighted least squares): 2^-23.1
// with its coefficients in fp32, 2^-22.2 as evaluated in fp32.  Beyond, 1 - 2 / (1 + e^2u), whose
// absolute error of some 2^-23 is relative there too.
__device__ __forceinline__ constexpr float tanh_coef(int k)
{
    constexpr float c[7] = {1.f, -0.333328396f, 0.13325204f, -0.0534570292f,
                            0.0202899799f, -0.00620337855f, 0.00104102236f};
    return c[k];
}

// The same for |u| <= 0.5, of degree 4: 2^-25 with its coefficients in fp32, 2^-23
// as evaluated.
__device__ __forceinline__ constexpr float tanh_close(int k)
{
    constexpr float close[5] = {1.f, -0.333330691f, 0.133247808f, -0.0529861338f, 0.0171351079f};
    return close[k];
}

__device__ __forceinline__ float cap_poly(float x, float u)
{
    const float w = u * u;
    float p = tanh_coef(6);
#pragma unroll
    for (int k = 5; k >= 0; --k) p = fmaf(p, w, tanh_coef(k));
    return x * p;
}

__device__ __forceinline__ float cap_far(float u, float cap)
{
    const float e = ptx::ex2(u * 2.885390081777927f);
    return fmaf(-2.f * cap, __fdividef(1.f, 1.f + e), cap);
}

__device__ __forceinline__ float cap_score(float x, float cap, float cap_inv)
{
    const float u = x * cap_inv;
    return fabsf(u) <= 1.f ? cap_poly(x, u) : cap_far(u, cap);
}

}  // namespace pkv
