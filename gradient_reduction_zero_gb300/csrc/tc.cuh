// The tensor cores of sm_103a from one CTA: TMA tile loads, tcgen05 products
// with accumulators in tensor memory, and the mbarriers between them.
//
// Operands are bf16 in shared memory as TMA writes them with the 128-byte
// swizzle: blocks of 64 columns, 128 bytes a row, 128 rows (16 KB), on a
// boundary of 1024 bytes.  A product reads such a block either along its columns
// (the sum runs over columns: "K-major") or along its rows (the sum runs over
// rows: "MN-major"); the left operand can also lie in tensor memory, two bf16 in a
// 32-bit column.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "bulk.cuh"

namespace dpz {

constexpr int kTcRows = 128;                   // rows of an operand's block
constexpr int kTcCols = 64;                    // its columns
constexpr int kTcBlock = kTcRows * 128;        // its bytes
constexpr uint32_t kTmemCols = 512;

// ------------------------------------------------------------ barriers

__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t arrivals)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(arrivals)
                 : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// Waits of a block's warps on one another and on the copies and products in
// flight.  Each is bounded by the SM clock; one that runs out sets the block's
// `lost` flag, which ends every other wait of the block as well.
__device__ __forceinline__ bool tc_wait(uint64_t* bar, uint32_t parity, volatile int* lost)
{
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity)) {
        if (*lost != 0) return false;
        if (clock64() - t0 > kWaitLimitCycles) {
            if (mbar_try_wait(bar, parity)) return true;
            *lost = 1;
            return false;
        }
    }
    return true;
}

// The same for a warp, which goes on as one.
__device__ __forceinline__ bool tc_wait_warp(uint64_t* bar, uint32_t parity, volatile int* lost)
{
    return __all_sync(0xffffffffu, tc_wait(bar, parity, lost));
}

// ------------------------------------------------------------ TMA

__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, uint64_t* bar, int x,
                                         int y, int z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_addr(dst)),
        "l"(map), "r"(smem_addr(bar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}

__device__ __forceinline__ void tma_prefetch(const CUtensorMap* map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// Shared memory written by threads, before the tensor cores read it.
__device__ __forceinline__ void fence_async_proxy()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ------------------------------------------------------------ tensor memory

__device__ __forceinline__ void tmem_alloc(uint32_t* at)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(at)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_free(uint32_t at)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(kTmemCols)
                 : "memory");
}

// 32 columns of the warp's 32 lanes (lane l of the warp holds row l of them).
// The registers are there after tmem_wait.
__device__ __forceinline__ void tmem_load32(uint32_t at, uint32_t* r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at));
}

__device__ __forceinline__ void tmem_store32(uint32_t at, const uint32_t* r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
        "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

// Waits for the warp's loads and ties the registers to it, so that no use of
// them moves before the wait.
template <int N>
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[N])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

__device__ __forceinline__ void tmem_wait_stores()
{
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Around a barrier between threads that use tensor memory.
__device__ __forceinline__ void tc_fence_before()
{
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after()
{
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// ------------------------------------------------------------ registers
//
// A warpgroup's registers per thread from here on.  What some gain others must have
// given: the sum over the block's warpgroups is at most what it was launched with.

template <int N>
__device__ __forceinline__ void set_registers_up()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_registers_down()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// ------------------------------------------------------------ products

// What issues a product must be the same in the whole warp for the hardware's
// uniform registers; values that come through shared memory are made so here.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// One thread of a converged warp, always the same.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}

// Descriptor of an operand in blocks of 64 swizzled columns.  K-major: groups
// of 8 rows are 1024 bytes apart.  MN-major: the same groups follow one another
// along the sum, and blocks of 64 columns are kTcBlock bytes apart (which a K-major
// operand ignores).  The low word holds the address in units of 16 bytes, so that
// a step of the sum is an addition to it; the high word is the same for all.
constexpr uint32_t kTcDescHigh = (1024u >> 4) | 1u << 14 | 2u << 29;

__device__ __forceinline__ uint32_t tc_desc(const void* p)
{
    return (smem_addr(p) & 0x3ffffu) >> 4 | (uint32_t)(kTcBlock >> 4) << 16;
}

__device__ __forceinline__ uint64_t tc_whole(uint32_t low)
{
    return (uint64_t)kTcDescHigh << 32 | low;
}

// Instruction descriptor: bf16 x bf16 -> fp32, 128 rows, n columns; b_mn: the
// right operand is MN-major.
__device__ __forceinline__ uint32_t tc_idesc(int n, bool b_mn)
{
    return 1u << 4 | 1u << 7 | 1u << 10 | (b_mn ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 |
           (uint32_t)(kTcRows >> 4) << 24;
}

// d (+)= a b, the sum over 16 elements; one thread issues it.
__device__ __forceinline__ void tc_mma(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(tc_whole(a)), "l"(tc_whole(b)), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}

// The same with the left operand in tensor memory.
__device__ __forceinline__ void tc_mma_tmem(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                            bool add)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(tc_whole(b)), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}

// Arrives on the barrier once every product issued so far by this thread is
// complete.
__device__ __forceinline__ void tc_commit(uint64_t* bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     smem_addr(bar))
                 : "memory");
}

// d = a b^T over `steps` times 16 columns of two K-major operands of BLOCKS blocks.
template <int BLOCKS>
__device__ __forceinline__ void tc_dot(uint32_t d, const char* a, const char* b, int steps,
                                       uint32_t idesc)
{
    const uint32_t x = tc_desc(a), y = tc_desc(b);
#pragma unroll
    for (int k = 0; k < 4 * BLOCKS; ++k) {
        const uint32_t at = (uint32_t)((k >> 2) * kTcBlock + (k & 3) * 32) >> 4;
        if (k < steps) tc_mma(d, x + at, y + at, idesc, k > 0);
    }
}

// d (+)= a b over the 128 rows of an MN-major operand b; a in tensor memory, its
// k-th 16 elements 8 k columns on, and `gap` more from the fifth.
__device__ __forceinline__ void tc_rows(uint32_t d, uint32_t a, uint32_t gap, const char* b,
                                        uint32_t idesc, bool add)
{
    const uint32_t y = tc_desc(b);
#pragma unroll
    for (int k = 0; k < kTcRows / 16; ++k)
        tc_mma_tmem(d, a + 8 * k + (k >= 4 ? gap : 0), y + k * (2048 >> 4), idesc, add || k > 0);
}

// Zeros in rows [n, 128) of `blocks` blocks, by a warp.
__device__ __forceinline__ void clear_rows(char* p, int n, int blocks)
{
    const int lane = threadIdx.x & 31;
    for (int b = 0; b < blocks; ++b)
        for (int i = n * 8 + lane; i < kTcRows * 8; i += 32)
            *reinterpret_cast<uint4*>(p + b * kTcBlock + i * 16) = make_uint4(0, 0, 0, 0);
}

}  // namespace dpz
