// sm_103a building blocks of the 8-bit products: mbarriers with bounded waits,
// tensor-map copies, tcgen05 matrix instructions and tensor memory.
#pragma once

#include <cuda.h>

#include "expert_vec.cuh"

namespace arf {

__device__ __forceinline__ uint32_t smem_u32(const void* p)
{
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// ------------------------------------------------------------- mbarriers

// Limit of a wait, tries between two looks at the time, and how a try waits
// (try_wait: some time in hardware).  Constants: as a kernel argument the limit
// cost the product for many rows 1 to 2%.  The tests also build the kernels with
// waits that give up at once.
#ifndef ARF_WAIT_NS
#define ARF_WAIT_NS 2000000000ull
#define ARF_WAIT_TRIES 16u
#define ARF_WAIT_TRY "try_wait"
#endif

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar)
{
    asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0];\n\t}" ::"r"(bar)
                 : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile(
        "{\n\t.reg .b64 st;\n\tmbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(bar),
        "r"(bytes)
        : "memory");
}
// `bytes` that no copy will bring count as arrived
__device__ __forceinline__ void bar_forgo(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier." ARF_WAIT_TRY ".parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Every wait ends: after ARF_WAIT_NS, or as soon as another wait of the block gave
// up (its flag is set), it returns false, and the first one to give up records
// AR_ERR_TIMEOUT and `where` in the device's status words.
struct Bail {
    uint32_t dead;              // shared-memory address of the block's flag
    int* status;                // device status words: code, detail
};

__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, const Bail& b, int where)
{
    if (bar_try(bar, parity))
        return true;
    uint64_t t0 = 0;
    for (uint32_t n = 1; !bar_try(bar, parity); ++n) {
        if (n % ARF_WAIT_TRIES)
            continue;
        uint32_t dead;
        asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(dead) : "r"(b.dead) : "memory");
        if (dead)
            return false;
        const uint64_t t = globaltimer_ns();
        t0 = t0 ? t0 : t;
        if (t - t0 > ARF_WAIT_NS) {
            asm volatile("st.volatile.shared.u32 [%0], 1;" ::"r"(b.dead) : "memory");
            if (atomicCAS(b.status, 0, AR_ERR_TIMEOUT) == 0)
                atomicExch(b.status + 1, where);
            return false;
        }
    }
    return true;
}
// A last wait for work in flight, taken only after the block gave up.
__device__ __forceinline__ void bar_drain(uint32_t bar, uint32_t parity)
{
    const uint64_t t0 = globaltimer_ns();
    while (!bar_try(bar, parity) && globaltimer_ns() - t0 < 200000000ull) {
    }
}

// One lane of a converged warp, the same one every time.  Copies and products are
// issued under this rather than under lane == 0: the compiler then knows that
// one thread runs them, and keeps their descriptors in uniform registers.
__device__ __forceinline__ bool elect_one()
{
    uint32_t yes;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(yes));
    return yes != 0;
}

// ------------------------------------------------------ tensor-map copies

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int x, int y)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(y)
        : "memory");
}
// the same of data with an eviction priority in L2
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int x, int y, uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%0], [%1, {%3, %4}], [%2], %5;" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(y), "l"(policy)
        : "memory");
}
__device__ __forceinline__ uint64_t evict_first()
{
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ uint64_t evict_normal()
{
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap* map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// Pairs of blocks (cta_group::2): the address of `bar` in the pair's first
// block, copies into this block's memory that signal there, and stores.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr, uint32_t rank)
{
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(map_rank(addr, rank)) : "memory");
    return v;
}
__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t rank, uint32_t v)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_rank(addr, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void bar_arrive_remote(uint32_t cluster_bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar)
                 : "memory");
}
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map,
                                              uint32_t cluster_bar, int x, int y)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(map), "r"(cluster_bar), "r"(x), "r"(y)
        : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int x, int y)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];\n\t"
        "cp.async.bulk.commit_group;" ::"l"(map),
        "r"(src), "r"(x), "r"(y)
        : "memory");
}
// until all but `N` of this thread's stores have been read from shared memory
template <int N>
__device__ __forceinline__ void tma_store_wait_read()
{
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// -------------------------------------------------- tcgen05: tensor memory

__device__ __forceinline__ void tmem_alloc(uint32_t smem_slot, uint32_t cols)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_slot),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols)
                 : "memory");
}
// the same for a pair: one warp of each block
__device__ __forceinline__ void tmem_alloc_pair(uint32_t smem_slot, uint32_t cols)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_slot),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free_pair(uint32_t addr, uint32_t cols)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols)
                 : "memory");
}
__device__ __forceinline__ void tc_fence_before()
{
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after()
{
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// 16 columns of this warp's 32 lanes: register i is column i of the thread's
// lane.  The registers may be read after tmem_wait on the same array.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&d)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3]), "=r"(d[4]), "=r"(d[5]), "=r"(d[6]),
          "=r"(d[7]), "=r"(d[8]), "=r"(d[9]), "=r"(d[10]), "=r"(d[11]), "=r"(d[12]), "=r"(d[13]),
          "=r"(d[14]), "=r"(d[15])
        : "r"(addr));
}
// Waits for this thread's loads; naming the registers keeps their uses behind it.
__device__ __forceinline__ void tmem_wait(uint32_t (&d)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3]), "+r"(d[4]), "+r"(d[5]),
                   "+r"(d[6]), "+r"(d[7]), "+r"(d[8]), "+r"(d[9]), "+r"(d[10]), "+r"(d[11]),
                   "+r"(d[12]), "+r"(d[13]), "+r"(d[14]), "+r"(d[15])
                 :
                 : "memory");
}

// ----------------------------------------------- tcgen05: matrix products

// Shared-memory operand: K-major rows of 128 bytes in the 128-byte swizzle, 8
// rows per 1024-byte group (stride 1024 >> 4 = 64; the leading offset is
// unused for this layout; descriptor version 1; swizzle code 2).  A step of 32
// bytes along K within the 128 adds 2 to the address field.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr)
{
    return (uint64_t)((addr & 0x3ffffu) >> 4) | (1ull << 16) | (64ull << 32) | (1ull << 46) |
           (2ull << 61);
}
// E4M3 x E4M3 -> fp32, both K-major, M x N per instruction
__host__ __device__ constexpr uint32_t fp8_idesc(int M, int N)
{
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// Four products, 128 of K: d = a * b.  `a` and `b` are the low words of the
// descriptors, `hi` their common high word.  One asm block, and the loop around
// it run by one thread: with votes and descriptor arithmetic between them the
// products were issued every 110 cycles at best (64 is what 128 columns take),
// and later still while other warps of the scheduler had arithmetic to issue.
// GROUP: cta_group::1, or ::2 for a pair, whose first block issues; M then
// counts the rows of both blocks, each of which holds its rows of a and half
// the rows of b.
#define ARF_MMA4(GROUP)                                                              \
    asm volatile(                                                                    \
        "{\n\t.reg .b64 p, q;\n\t.reg .b32 x, y;\n\t.reg .pred no, yes;\n\t"           \
        "setp.ne.b32 no, 0, 0;\n\tsetp.ne.b32 yes, 1, 0;\n\t"                          \
        "mov.b64 p, {%1, %3};\n\tmov.b64 q, {%2, %3};\n\t"                             \
        "tcgen05.mma." GROUP ".kind::f8f6f4 [%0], p, q, %4, no;\n\t"                   \
        "add.u32 x, %1, 2;\n\tadd.u32 y, %2, 2;\n\t"                                   \
        "mov.b64 p, {x, %3};\n\tmov.b64 q, {y, %3};\n\t"                               \
        "tcgen05.mma." GROUP ".kind::f8f6f4 [%0], p, q, %4, yes;\n\t"                  \
        "add.u32 x, %1, 4;\n\tadd.u32 y, %2, 4;\n\t"                                   \
        "mov.b64 p, {x, %3};\n\tmov.b64 q, {y, %3};\n\t"                               \
        "tcgen05.mma." GROUP ".kind::f8f6f4 [%0], p, q, %4, yes;\n\t"                  \
        "add.u32 x, %1, 6;\n\tadd.u32 y, %2, 6;\n\t"                                   \
        "mov.b64 p, {x, %3};\n\tmov.b64 q, {y, %3};\n\t"                               \
        "tcgen05.mma." GROUP ".kind::f8f6f4 [%0], p, q, %4, yes;\n\t}" ::"r"(d),         \
        "r"(a), "r"(b), "r"(hi), "r"(idesc)                                          \
        : "memory")

__device__ __forceinline__ void mma4_fp8(uint32_t d, uint32_t a, uint32_t b, uint32_t hi,
                                         uint32_t idesc)
{
    ARF_MMA4("cta_group::1");
}
__device__ __forceinline__ void mma4_fp8_pair(uint32_t d, uint32_t a, uint32_t b, uint32_t hi,
                                              uint32_t idesc)
{
    ARF_MMA4("cta_group::2");
}
#undef ARF_MMA4
// one arrival on `bar` once every product issued so far by this thread is done
__device__ __forceinline__ void mma_commit(uint32_t bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
}

// The same of a pair's products, at a barrier of the issuing block alone.
__device__ __forceinline__ void mma_commit_pair_here(uint32_t bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
}
// The commit arrives at the same barrier of both blocks.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}

// Registers per thread of this warpgroup from here on.  The shares of a block's
// warpgroups may not exceed what it was launched with (threads x registers).
template <int N>
__device__ __forceinline__ void regs_fewer()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_more()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

}  // namespace arf
