// pkv_wait.cuh -- bounded waits of kernels whose warps have roles (loads, products,
// softmax ..): the first wait that runs out sets PKV_DEV_TIMEOUT and an abort flag
// that ends every role of the CTA; the copies that may still be in flight are then
// waited for behind a barrier.
#pragma once

#include <stdint.h>

#include "../../include/pkv.h"
#include "pkv_ptx.cuh"

namespace pkv {
namespace {

constexpr uint64_t kWaitLimitNs = 1000000000ull;  // bounded waits: 1 s

#ifdef PKV_DEBUG
// Settable by the debug build's entry points: wait number give_at of every warp of
// give_role gives up, as if its limit had run out, and every wait of slow_role
// begins slow_ns later (role -2: none; warps without a role have -1), or with
// slow_warp > 0 those of its warps number slow_warp - 1 modulo 4 alone.
struct WaitDebug {
    int give_role, give_at, slow_role, slow_ns, slow_warp;
};
static __device__ WaitDebug g_wait_debug = {-2, 0, -2, 0, 0};
#endif

struct Waiter {
    volatile int *abort;
    int32_t *dev_status;
#ifdef PKV_DEBUG
    int role = -1;
    mutable int waits = 0;
#endif
    __device__ __forceinline__ Waiter as([[maybe_unused]] int r) const
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
        const WaitDebug d = g_wait_debug;
        if (role == d.slow_role &&
            (d.slow_warp <= 0 || static_cast<int>(threadIdx.x >> 5 & 3) == d.slow_warp - 1))
            __nanosleep(d.slow_ns);
        if (role == d.give_role && waits++ == d.give_at) {
            give_up();
            return true;
        }
#endif
        return false;
    }
};

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

}  // namespace
}  // namespace pkv
