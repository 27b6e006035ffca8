// tc.cuh -- sm_100a tensor-core, tensor-copy and barrier primitives used by
// the products on FP4 weights.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace fp4q {

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// One lane of a converged warp.  The warps that feed the tensor cores run their
// loops converged and issue under this predicate: addresses and descriptors
// then stay in the warp's uniform registers.
__device__ __forceinline__ bool elect_one()
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok));
    return ok != 0;
}

// A place in a ring of N stages and the parity of its current pass.
template <int N> struct Ring {
    uint32_t stage = 0, parity = 0;
    __device__ __forceinline__ void next()
    {
        if (++stage == N) {
            stage = 0;
            parity ^= 1;
        }
    }
};

// ---------------------------------------------------------------- mbarriers
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Arrival on the barrier at the same offset in thread block `rank` of the
// cluster.  It does not wait for the thread's ordinary writes to become visible
// there (a fence that takes over a thousand clocks under load): for signals
// about tensor memory, about shared memory that the tensor cores of its own SM
// read, and about data that has been read.
__device__ __forceinline__ void mbar_signal_peer(uint32_t bar, uint32_t rank)
{
    asm volatile(
        "{\n\t.reg .b32 a;\n\t"
        "mapa.shared::cluster.u32 a, %0, %1;\n\t"
        "mbarrier.arrive.shared::cluster.b64 _, [a];\n\t}" ::"r"(bar), "r"(rank)
        : "memory");
}
// Four or two words to the same offset in thread block `rank`, counted there as bytes on `bar`.
__device__ __forceinline__ void send(uint32_t addr, uint4 v, uint32_t bar, uint32_t rank)
{
    asm volatile(
        "{\n\t.reg .b32 a, b;\n\t"
        "mapa.shared::cluster.u32 a, %0, %6;\n\t"
        "mapa.shared::cluster.u32 b, %5, %6;\n\t"
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [a], {%1, %2, %3, %4}, [b];\n\t}" ::"r"(addr),
        "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "r"(bar), "r"(rank)
        : "memory");
}
__device__ __forceinline__ void send(uint32_t addr, uint2 v, uint32_t bar, uint32_t rank)
{
    asm volatile(
        "{\n\t.reg .b32 a, b;\n\t"
        "mapa.shared::cluster.u32 a, %0, %4;\n\t"
        "mapa.shared::cluster.u32 b, %3, %4;\n\t"
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [a], {%1, %2}, [b];\n\t}" ::"r"(addr),
        "r"(v.x), "r"(v.y), "r"(bar), "r"(rank)
        : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
// The barrier of group `e` of four epilogue warps; group_all also gives all of
// them whether `ok` held for every thread.
__device__ __forceinline__ void group_bar(int e) { asm volatile("bar.sync %0, 128;" ::"r"(1 + e) : "memory"); }
__device__ __forceinline__ bool group_all(int e, bool ok)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\t"
        "bar.red.and.pred q, %1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r) : "r"(1 + e), "r"((uint32_t)ok) : "memory");
    return r != 0;
}

}  // namespace fp4q

#include "mbar_wait.cuh"

namespace fp4q {

// ---------------------------------------------------------------- clusters
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}
// A barrier of all threads of the cluster that orders no ordinary writes: for
// what mbarrier initialisations (fenced by themselves) and allocations need, and
// so that no block ends while a peer uses its memory.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// ---------------------------------------------------------------- copies to shared memory
__device__ __forceinline__ void tma_prefetch_desc(const CUtensorMap* map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
// Tile at byte (or element) column x, row y; x * element size is a multiple of 16 bytes.
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst), "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
// `bytes` contiguous bytes; addresses and size are multiples of 16.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
// Shared memory written by ordinary stores, to be read by the tensor cores or copies.
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ---------------------------------------------------------------- tensor memory
// G: thread blocks that the tensor-core operations span (2: a cluster's pair,
// both of which allocate and free; the even one issues everything else).
// One warp allocates (and later frees) `cols` columns, a power of two from 32.
template <int G> __device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t cols)
{
    if (G == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
}
template <int G> __device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols)
{
    if (G == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Arrival on `bar` (of both thread blocks of a pair) when every tensor-core
// operation this thread issued has completed.
template <int G> __device__ __forceinline__ void tc_commit(uint32_t bar)
{
    if (G == 2)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                bar), "h"((uint16_t)3)
            : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                     : "memory");
}
// 32 lanes x 16 columns of binary32: register i of lane l is column i of the warp's lane l
// (the wait is part of the statement: nothing may use the registers before it).
__device__ __forceinline__ void tmem_load16(uint32_t (&r)[16], uint32_t addr)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr) : "memory");
}

// ---------------------------------------------------------------- tensor-core operations
// Shared-memory operand, K contiguous in 128-byte rows under the 128-byte
// swizzle, 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_k128(uint32_t addr)
{
    return (uint64_t)((addr & 0x3FFFF) >> 4) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) |
           (2ull << 61);
}
// A 512-byte scale tile: 32 lines of 16 bytes, 8-line groups 128 bytes apart, no swizzle.
__device__ __forceinline__ uint64_t desc_scales(uint32_t addr)
{
    return (uint64_t)((addr & 0x3FFFF) >> 4) | (1ull << 16) | ((uint64_t)(128 >> 4) << 32) | (1ull << 46);
}
// Scale tile -> 4 columns of tensor memory, repeated for the four lane quarters.
template <int G> __device__ __forceinline__ void tc_copy_scales(uint32_t tmem, uint64_t desc)
{
    if (G == 2)
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}
// D[128 G][N] (+)= A[128 G][64] * B[N][64]^T, E2M1 with block scales in tensor
// memory: NVFP4 four E4M3 scales per row, MXFP4 two E8M0 ones.  Of a pair,
// each thread block holds its 128 rows of A and D with their scales, half the
// rows of B and the scales of all of B.
template <bool MX, int G>
__device__ __forceinline__ void tc_mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                           uint32_t sfb, bool add)
{
    if (MX && G == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::
                "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"((uint32_t)add)
            : "memory");
    else if (MX)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::
                "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"((uint32_t)add)
            : "memory");
    else if (G == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::
                "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"((uint32_t)add)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::
                "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"((uint32_t)add)
            : "memory");
}
// Instruction descriptor of tc_mma_fp4: E2M1 operands (format 1), both K-major,
// m x n; scale type E8M0 for MXFP4; `id` the byte of a scale column that the
// operands' first scale is in.
__device__ __forceinline__ uint32_t idesc_fp4(bool mx, uint32_t m, uint32_t n, uint32_t id)
{
    return (id << 4) | (1u << 7) | (1u << 10) | ((n >> 3) << 17) | ((mx ? 1u : 0u) << 23) | ((m >> 4) << 24) |
           (id << 29);
}

}  // namespace fp4q
