// mbar_wait.cuh -- the products' bounded waits for mbarriers.
//
// Every wait is bounded by time: one that runs out sets the thread block's
// `dead` word, every other wait of the block then ends at its next look at it,
// and the kernel reports FP4Q_FLAG_TIMEOUT.
//
// A phase that completes about when the time runs out may be seen by one thread
// and missed by another, and what follows a wait is done together: elect.sync,
// tensor-memory loads and stores and the loops around them by a warp, barriers by
// a group of four.  So the lanes of a warp agree on every look, by a vote (2048 x
// 14336 x 4096 of fp4q_linear takes 1% longer by that; one vote after several
// waits, each lane by itself in between, took 3%), and a group of warps by the
// barrier that it meets at anyway (group_all), before its next one.
//
// Written on what the includer declares first, mbar_try (one look at an
// mbarrier's phase), so that it also compiles for the host.
#pragma once

#include <cstdint>

namespace fp4q {

constexpr long long kWaitClocks = 1ll << 32;    // longest wait: about two seconds of SM clocks

// Whether the block is dead or the wait that began at t0 has run out (which
// makes it dead), for the whole warp.
__device__ __forceinline__ bool gave_up(long long t0, volatile int* dead)
{
    if (__all_sync(~0u, !*dead && clock64() - t0 <= kWaitClocks)) return false;
    *dead = 1;
    return true;
}

// True once the barrier's phase `parity` has completed, false if the thread
// block is dead; called by a whole warp, whose lanes all get the same answer.
// Time is the SM's own clock.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* dead)
{
    if (__all_sync(~0u, mbar_try(bar, parity))) return true;
    const long long t0 = clock64();
    do {
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (__all_sync(~0u, mbar_try(bar, parity))) return true;
    } while (!gave_up(t0, dead));
    return false;
}
// For a long wait (the epilogue's for a tile's sums): looks seldom, so that the
// waiting warps leave the issue slots to the ones that work.
__device__ __forceinline__ bool mbar_wait_long(uint32_t bar, uint32_t parity, volatile int* dead)
{
    const long long t0 = clock64();
    while (!__all_sync(~0u, mbar_try(bar, parity))) {
        __nanosleep(64);
        if (gave_up(t0, dead)) return false;
    }
    return true;
}

// For the end of a dead thread block: the wait for what it has in flight.
__device__ __forceinline__ void mbar_drain(uint32_t bar, uint32_t parity)
{
    const long long t0 = clock64();
    while (!mbar_try(bar, parity) && clock64() - t0 < kWaitClocks / 16) {
    }
}
// And for all else that may still come: copies issued by a warp that ended
// before the block died, words and signals from its peers.
__device__ __forceinline__ void linger()
{
    const long long t0 = clock64();
    while (clock64() - t0 < kWaitClocks / 16) {
    }
}

}  // namespace fp4q
