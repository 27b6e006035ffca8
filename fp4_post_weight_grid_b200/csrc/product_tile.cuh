// product_tile.cuh -- what the tensor-core kernels of the products on FP4
// weights share: the list of output tiles, the sum over a cluster that splits
// K, and the way from tensor memory to y.
//
// A tile is 128 rows of W (features) by up to BN rows of x (tokens) of one
// group.  W is the operand that fills the 128 lanes of tensor memory and the
// tokens are its columns, so that the cost of a tile follows the number of
// tokens in steps of 16: the same kernel serves one token and thousands.
#pragma once

#include "product_epilogue.cuh"
#include "tc.cuh"

namespace fp4q {

struct TileArgs {
    const int32_t* offsets;       // [groups + 1] or null
    int64_t n;
    int m, k, groups;
    int n_tiles;                  // tiles of 128 features
    int k_steps;                  // steps of 256 columns
    int split;                    // thread blocks of the cluster that share a tile's k_steps
    int w_col_tiles;              // scale tiles of a row tile
    const uint8_t* x_scales;      // packed x
    const float* x_S;
    const uint8_t* w_scales;
    const float* w_S;
    int64_t w_scale_stride;
    EpilogueArgs ep;
    int32_t* status;
};

struct Tile {
    int group, feature, row, rows;      // first feature, first token row, token rows
};

// The token tiles of the groups before each group, in shared memory; built by
// one warp.  False if the offsets are out of order or range.
template <int BN>
__device__ __forceinline__ bool tile_table(const TileArgs& a, int* before)
{
    const int lane = threadIdx.x & 31;
    if (!a.offsets) {
        if (lane == 0) {
            before[0] = 0;
            before[1] = (a.m + BN - 1) / BN;
        }
        __syncwarp();
        return true;
    }
    bool ok = true;
    int total = 0;
    for (int g0 = 0; g0 < a.groups; g0 += 32) {
        const int g = g0 + lane;
        int count = 0;
        if (g < a.groups) {
            const int lo = __ldg(a.offsets + g), hi = __ldg(a.offsets + g + 1);
            ok = ok && lo >= 0 && lo <= hi && hi <= a.m;
            count = ok ? (hi - lo + BN - 1) / BN : 0;
        }
        int sum = count;
        for (int d = 1; d < 32; d *= 2) {
            const int v = __shfl_up_sync(~0u, sum, d);
            if (lane >= d) sum += v;
        }
        if (g < a.groups) before[g + 1] = total + sum;
        total += __shfl_sync(~0u, sum, 31);
    }
    if (lane == 0) before[0] = 0;
    ok = __all_sync(~0u, ok);
    __syncwarp();
    return ok;
}

// Tile t: the features vary fastest, so that neighbouring tiles share x.
template <int BN>
__device__ __forceinline__ Tile tile_at(const TileArgs& a, const int* before, int64_t t)
{
    const int mt = (int)(t / a.n_tiles);
    Tile r;
    r.feature = (int)(t % a.n_tiles) * 128;
    if (!a.offsets) {
        r.group = 0;
        r.row = mt * BN;
        r.rows = min(BN, a.m - r.row);
        return r;
    }
    int lo = 0, hi = a.groups;            // before[lo] <= mt < before[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (before[mid] <= mt)
            lo = mid;
        else
            hi = mid;
    }
    r.group = lo;
    r.row = __ldg(a.offsets + lo) + (mt - before[lo]) * BN;
    r.rows = min(BN, __ldg(a.offsets + lo + 1) - r.row);
    return r;
}

// This thread block's share of a tile's steps.
__device__ __forceinline__ void split_steps(const TileArgs& a, int rank, int& first, int& last)
{
    first = (int)((int64_t)a.k_steps * rank / a.split);
    last = (int)((int64_t)a.k_steps * (rank + 1) / a.split);
}

// From the accumulator (lane = feature, column = token) to y, by four warps
// that each own a quarter of the lanes.  A thread keeps its feature, so a
// store of a warp covers 32 neighbouring features of one token.
template <typename T>
__device__ __forceinline__ void write_tile(const TileArgs& a, const Tile& t, uint32_t acc, float S)
{
    const int quarter = (threadIdx.x / 32) % 4, lane = threadIdx.x & 31;
    const int64_t j = t.feature + quarter * 32 + lane;
    const bool in = j < a.n;
    float bias = 0.f;
    if (a.ep.bias && in) bias = to_f32<T>(static_cast<const T*>(a.ep.bias)[t.group * a.n + j]);
    for (int c = 0; c < t.rows; c += 16) {
        uint32_t r[16];
        tmem_load16(r, acc + ((uint32_t)quarter << 21) + c);
        if (in) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (c + i < t.rows)
                    finish<T>(a.ep, __uint_as_float(r[i]), S, bias, a.ep.bias != nullptr,
                              (int64_t)(t.row + c + i) * a.n + j);
        }
    }
}

// The same where a cluster split the steps: every thread block leaves its
// partial sums in shared memory, and each finishes its share of the tokens,
// adding the partials in rank order (the result does not depend on timing).
// `full`/`empty`: barriers of `split` arrivals, one from every thread block.
template <typename T>
__device__ __forceinline__ bool write_tile_split(const TileArgs& a, const Tile& t, uint32_t acc, float S, float* part,
                                                 uint32_t full, uint32_t empty, uint32_t parity, uint32_t rank,
                                                 volatile int* dead, uint32_t acc_empty)
{
    const int quarter = (threadIdx.x / 32) % 4, lane = threadIdx.x & 31, line = quarter * 32 + lane;
    bool ok = mbar_wait(empty, parity ^ 1, dead);       // every peer has read the tile before
    if (ok)
        for (int c = 0; c < t.rows; c += 16) {
            uint32_t r[16];
            tmem_load16(r, acc + ((uint32_t)quarter << 21) + c);
#pragma unroll
            for (int i = 0; i < 16; ++i) part[(c + i) * 128 + line] = __uint_as_float(r[i]);
        }
    tc_fence_before();
    asm volatile("bar.sync 1, 128;" ::: "memory");
    if (line == 0) mbar_arrive(acc_empty);
    if (line < a.split) mbar_arrive_peer(full, line);
    ok = mbar_wait(full, parity, dead) && ok;
    const int64_t j = t.feature + line;
    if (ok && j < a.n) {
        float bias = 0.f;
        if (a.ep.bias) bias = to_f32<T>(static_cast<const T*>(a.ep.bias)[t.group * a.n + j]);
        for (int c = (int)rank; c < t.rows; c += a.split) {
            const uint32_t at = smem_u32(part + c * 128 + line);
            float sum = ld_peer_f32(at, 0);
            for (int q = 1; q < a.split; ++q) sum += ld_peer_f32(at, q);
            finish<T>(a.ep, sum, S, bias, a.ep.bias != nullptr, (int64_t)(t.row + c) * a.n + j);
        }
    }
    asm volatile("bar.sync 1, 128;" ::: "memory");
    if (line < a.split) mbar_arrive_peer(empty, line);
    return ok;
}

}  // namespace fp4q
