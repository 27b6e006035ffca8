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
// that each own a quarter of the lanes, kChunk tokens at a time through
// shared memory: a thread writes its feature's sums of the chunk there (rows
// of 132 floats, so that neither side has bank conflicts) and then finishes 16
// bytes of y at a time, whose mul and residual it asked for before.
constexpr int kPartRow = 132;
template <typename T, int BN> struct Chunk {
    static constexpr int kTokens = BN < 4 * Lanes<T>::kCount ? BN : 4 * Lanes<T>::kCount;
};

__device__ __forceinline__ void tile_bar() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

__device__ __forceinline__ void to_part(uint32_t acc, int c0, int count, float* part)
{
    const int quarter = (threadIdx.x / 32) % 4, line = quarter * 32 + (threadIdx.x & 31);
    for (int c = 0; c < count; c += 16) {
        uint32_t r[16];
        tmem_load16(r, acc + ((uint32_t)quarter << 21) + c0 + c);
#pragma unroll
        for (int i = 0; i < 16; ++i) part[(c + i) * kPartRow + line] = __uint_as_float(r[i]);
    }
}

// Where one thread's 16 bytes of a chunk are.
template <typename T> struct Item {
    int token, lane;              // of the chunk; first feature of the tile
    int64_t at;                   // element of y
    int count;                    // features that exist
    bool whole;
    __device__ __forceinline__ Item(const TileArgs& a, const Tile& t, int c0, int i)
    {
        constexpr int kPer = 128 / Lanes<T>::kCount;
        token = i / kPer;
        lane = i % kPer * Lanes<T>::kCount;
        const int64_t j = t.feature + lane;
        count = (int)min((int64_t)Lanes<T>::kCount, a.n - j);
        at = (int64_t)(t.row + c0 + token) * a.n + j;
        whole = count == Lanes<T>::kCount && a.n % Lanes<T>::kCount == 0;
    }
};

template <typename T, int N>
__device__ __forceinline__ void load_bias(const TileArgs& a, const Tile& t, const Item<T>& it, float (&bias)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) bias[i] = 0.f;
    if (a.ep.bias && it.count > 0) {
        const int64_t j = t.group * a.n + t.feature + it.lane;
        unpack16(load_lanes<T>(a.ep.bias, j, it.count, it.whole), bias);
    }
}

// Tokens [0, t.rows) of a tile that one thread block summed.
template <typename T, int kChunk>
__device__ __forceinline__ void write_tile(const TileArgs& a, const Tile& t, uint32_t acc, float S, float* part)
{
    constexpr int N = Lanes<T>::kCount, kPer = 128 / N, kItems = kChunk * kPer / 128;
    const int tid = threadIdx.x & 127;
    float bias[N];
    load_bias<T>(a, t, Item<T>(a, t, 0, tid), bias);       // a thread keeps its features
    for (int c0 = 0; c0 < t.rows; c0 += kChunk) {
        const int rows = min(kChunk, t.rows - c0);
        Extra<T> x[kItems];
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const Item<T> it(a, t, c0, k * 128 + tid);
            if (it.token < rows && it.count > 0) x[k] = load_extra<T>(a.ep, it.at, it.count, it.whole);
        }
        to_part(acc, c0, rows, part);
        tile_bar();
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const Item<T> it(a, t, c0, k * 128 + tid);
            if (it.token >= rows || it.count <= 0) continue;
            float z[N];
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                const float4 f = *reinterpret_cast<const float4*>(part + it.token * kPartRow + it.lane + i);
                z[i] = f.x * S;
                z[i + 1] = f.y * S;
                z[i + 2] = f.z * S;
                z[i + 3] = f.w * S;
            }
            finish<T>(a.ep, z, bias, x[k], it.at, it.count, it.whole);
        }
        tile_bar();
    }
}

// The same where a cluster split the steps: every thread block leaves its
// partial sums in shared memory, and each finishes its share of the outputs,
// adding the partials in rank order (the result does not depend on timing).
// `full`/`empty`: barriers of `split` arrivals, one from every thread block.
template <typename T>
__device__ __forceinline__ bool write_tile_split(const TileArgs& a, const Tile& t, uint32_t acc, float S, float* part,
                                                 uint32_t full, uint32_t empty, uint32_t parity, uint32_t rank,
                                                 volatile int* dead, uint32_t acc_empty)
{
    constexpr int N = Lanes<T>::kCount, kPer = 128 / N;
    const int tid = threadIdx.x & 127;
    bool ok = mbar_wait(empty, parity ^ 1, dead);          // every peer has read the tile before
    const int first = (int)rank * 128 + tid;
    const Item<T> it0(a, t, 0, first);
    Extra<T> x;
    float bias[N];
    load_bias<T>(a, t, it0, bias);
    if (it0.token < t.rows && it0.count > 0) x = load_extra<T>(a.ep, it0.at, it0.count, it0.whole);
    if (ok) to_part(acc, 0, t.rows, part);
    tc_fence_before();
    tile_bar();
    if (tid == 0) mbar_arrive(acc_empty);
    if (tid < a.split) mbar_arrive_peer(full, tid);
    ok = mbar_wait(full, parity, dead) && ok;
    for (int i = first; ok && i < t.rows * kPer; i += a.split * 128) {
        const Item<T> it(a, t, 0, i);
        if (it.count <= 0) continue;
        if (i != first) x = load_extra<T>(a.ep, it.at, it.count, it.whole);
        const uint32_t from = smem_u32(part + it.token * kPartRow + it.lane);
        float z[N];
#pragma unroll
        for (int k = 0; k < N; ++k) z[k] = 0.f;
        for (int q = 0; q < a.split; ++q) {
#pragma unroll
            for (int k = 0; k < N; k += 4) {
                const float4 f = ld_peer_f32x4(from + 4 * k, q);
                z[k] += f.x;
                z[k + 1] += f.y;
                z[k + 2] += f.z;
                z[k + 3] += f.w;
            }
        }
#pragma unroll
        for (int k = 0; k < N; ++k) z[k] *= S;
        finish<T>(a.ep, z, bias, x, it.at, it.count, it.whole);
    }
    tile_bar();
    if (tid < a.split) mbar_arrive_peer(empty, tid);
    return ok;
}

}  // namespace fp4q
