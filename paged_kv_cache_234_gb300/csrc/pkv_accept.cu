// pkv_accept.cu -- the path of every tree of drafted tokens that the model
// confirms: from row 0 on, the first row whose parent is the present one and
// whose token is the present one's target.
//
// Parents lie before their children, so the path rises, and the first child
// that fits is the first such row behind the present one: one pass over the
// rows finds the whole path.  A warp takes a sequence, 32 rows at a time with
// the next 32 on their way; within them a ballot finds the next row of the
// path and a shuffle its target.  Every row is read once (12 bytes) and its
// entry of the path written once (4 bytes); what is left is latency: the look at
// the sequence, the rows' loads and some 30 cycles for each row of the path.
#include <stdint.h>

#include "pkv_host.cuh"
#include "pkv_ptx.cuh"
#include "pkv_ragged.cuh"

namespace pkv {
namespace {

constexpr int kAcceptWarps = 4;

__global__ void __launch_bounds__(32 * kAcceptWarps)
    accept_kernel(int32_t *__restrict__ kept, int32_t *__restrict__ kept_lens,
                  int32_t *__restrict__ next_tokens, const int32_t *__restrict__ tokens,
                  const int32_t *__restrict__ targets, const int32_t *__restrict__ parents,
                  const int32_t *__restrict__ query_starts, int num_tokens, int num_seqs,
                  int32_t *dev_status)
{
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int s = blockIdx.x * kAcceptWarps + static_cast<int>(threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (s >= num_seqs) return;
    SeqRows sr;
    sr.set(__ldg(query_starts + s), __ldg(query_starts + s + 1), INT32_MAX, num_tokens, INT32_MAX);
    const int n = sr.ok ? sr.len : 0;
    const int32_t *par = parents + sr.start, *tok = tokens + sr.start, *tgt = targets + sr.start;
    int32_t *path = kept + sr.start;
    int here = -1, want = 0, m = 0;   // the present row and its target; rows of the path
    bool bad = false;
    int p1 = -1, t1 = 0, g1 = 0;      // the next 32 rows
    auto load = [&](int j) {
        p1 = -1;
        if (j < n) {
            p1 = __ldg(par + j);
            t1 = __ldg(tok + j);
            g1 = __ldg(tgt + j);
        }
    };
    load(lane);
    for (int j0 = 0; j0 < n; j0 += 32) {
        const int j = j0 + lane, p = p1, t = t1, g = g1;
        load(j + 32);
        bad |= j < n && (p < -1 || p >= j);
        unsigned on = 0;              // rows of the path among these
        unsigned ahead = 0xffffffffu; // rows behind the present one
        if (j0 == 0) {
            on = 1u;
            ahead = ~1u;
            here = 0;
            want = __shfl_sync(0xffffffffu, g, 0);
        }
        for (;;) {
            const unsigned fits =
                __ballot_sync(0xffffffffu, j < n && p == here && t == want) & ahead;
            if (!fits) break;
            const int b = __ffs(fits) - 1;
            on |= 1u << b;
            ahead = ~1u << b;   // (b = 31: none)
            here = j0 + b;
            want = __shfl_sync(0xffffffffu, g, b);
        }
        if (on >> lane & 1u) path[m + __popc(on & ((1u << lane) - 1u))] = j;
        m += __popc(on);
    }
    bad = __any_sync(0xffffffffu, bad);
    if (bad) m = 0;
    __syncwarp();
    for (int j = m + lane; j < n; j += 32) path[j] = -1;
    if (lane == 0) {
        kept_lens[s] = m;
        next_tokens[s] = m > 0 ? want : -1;
        if (dev_status) {
            if (bad) atomicOr(dev_status, static_cast<int32_t>(PKV_DEV_BAD_TREE));
            if (!sr.ok) atomicOr(dev_status, static_cast<int32_t>(PKV_DEV_BAD_CTX));
        }
    }
}

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_tree_accept(int32_t *kept, int32_t *kept_lens, int32_t *next_tokens,
                                      const int32_t *tokens, const int32_t *targets,
                                      const int32_t *parents, const int32_t *query_starts,
                                      int num_tokens, int num_seqs, int32_t *dev_status,
                                      void *stream)
{
    using namespace pkv;
    if (num_tokens < 0 || num_seqs < 0 || !query_starts) return PKV_ERR_INVALID_ARG;
    // (arrays without elements may be null)
    if (num_tokens != 0 && (!kept || !tokens || !targets || !parents)) return PKV_ERR_INVALID_ARG;
    if (num_seqs != 0 && (!kept_lens || !next_tokens)) return PKV_ERR_INVALID_ARG;
    if (!aligned(kept, 4) || !aligned(kept_lens, 4) || !aligned(next_tokens, 4) ||
        !aligned(tokens, 4) || !aligned(targets, 4) || !aligned(parents, 4) ||
        !aligned(query_starts, 4) || !aligned(dev_status, 4))
        return PKV_ERR_MISALIGNED;
    if (num_seqs == 0) return PKV_OK;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((num_seqs - 1) / kAcceptWarps + 1));
    cfg.blockDim = dim3(32 * kAcceptWarps);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, accept_kernel, kept, kept_lens, next_tokens, tokens, targets,
                           parents, query_starts, num_tokens, num_seqs, dev_status) !=
        cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    return PKV_OK;
}
