// pkv_umma.cuh -- tcgen05 wrappers (sm_103a): TMEM allocation, matrix
// products with fp16 operands and fp32 accumulation in TMEM, and the transfers
// between TMEM and registers.
#pragma once

#include <stdint.h>

namespace pkv {
namespace umma {

// ------------------------------------------------------------- allocation
// Whole warp; writes the TMEM address to shared memory.
__device__ __forceinline__ void alloc(uint32_t smem_dst, uint32_t columns)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_dst),
                 "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void dealloc(uint32_t tmem, uint32_t columns)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns)
                 : "memory");
}

// ------------------------------------------------------------- descriptors
// Shared-memory operand in rows of 128 bytes with the 128-byte swizzle, atoms
// of 8 rows (1024 bytes) one after the other.
//   K-major (rows are M or N, 64 values of K each): one 64-wide slice of K.
//   MN-major (rows are K, 64 values of N each): `next` is the distance from
//   one 64-wide block of N to the next.
// The low word holds the address and `next`, the high word is the same for
// all, so the operands of one product differ by an addition to the low word.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t next)
{
    return ((addr & 0x3ffffu) >> 4) | (next >> 4 << 16);
}

__device__ __forceinline__ uint64_t desc(uint32_t lo)
{
    constexpr uint32_t hi = (1024u >> 4) | (1u << 14) | (2u << 29);
    return static_cast<uint64_t>(hi) << 32 | lo;
}

// Shared-memory operand without a swizzle, MN-major: 8 values of M or N by 8 of K
// are 128 contiguous bytes, 8 rows (K) of 16.  The next 8 of K follow at once, the
// next 8 of M or N `block` bytes further on.
__device__ __forceinline__ uint64_t desc_plain(uint32_t addr, uint32_t block)
{
    const uint32_t lo = ((addr & 0x3ffffu) >> 4) | ((128u >> 4) << 16);
    const uint32_t hi = (block >> 4) | (1u << 14);
    return static_cast<uint64_t>(hi) << 32 | lo;
}

// fp16 x fp16 -> fp32, M x N per instruction (K = 16); b_mn: B is MN-major.
__host__ __device__ constexpr uint32_t f16_idesc(int m, int n, bool b_mn)
{
    return (1u << 4) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(m >> 4) << 24);
}

// The bit of an instruction descriptor that says that A is MN-major.
constexpr uint32_t kAMn = 1u << 15;

// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok));
    return ok != 0;
}

// ---------------------------------------------------------------- products
// One thread.  D[tmem] (+)= A . B with A and B in shared memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       bool accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}

// The same with A in TMEM (row i in lane i, two fp16 values per column).
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       bool accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}

// Arrive on an mbarrier when everything this thread issued so far is done.
__device__ __forceinline__ void commit(uint32_t bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
}

__device__ __forceinline__ void fence_after()
{
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void fence_before()
{
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void wait_ld()
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void wait_st()
{
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// ------------------------------------------------- registers <-> TMEM
// Whole warp; lane i of warp w reads and writes TMEM lane 32 (w mod 4) + i,
// 32 consecutive columns.  Loaded values are valid after wait_ld().
__device__ __forceinline__ void ld32(uint32_t tmem, float *v)
{
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(tmem)
        : "memory");
}

// The same, 16 columns.
__device__ __forceinline__ void ld16(uint32_t tmem, float *v)
{
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]),
          "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
          "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(tmem)
        : "memory");
}

__device__ __forceinline__ void st16(uint32_t tmem, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
        "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
        "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
        "r"(tmem)
        : "memory");
}

}  // namespace umma
}  // namespace pkv
