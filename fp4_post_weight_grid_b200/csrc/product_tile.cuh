// product_tile.cuh -- what the tensor-core kernels of the products on FP4
// weights share: the list of output tiles, the sum over a cluster that splits
// K, and the way from tensor memory to y.
//
// A tile is 128 rows of W (features; 256 where a pair of thread blocks works on
// it) by up to `tokens` rows of x of one group.  W is the operand that fills the
// 128 lanes of tensor memory and the tokens are its columns, so that the cost of a
// tile follows the number of tokens in steps of 16: the same kernel serves one
// token and thousands.
#pragma once

#include <type_traits>

#include "product_epilogue.cuh"
#include "tc.cuh"

namespace fp4q {

struct TileArgs {
    const int32_t* offsets;       // [groups + 1] or null
    int64_t n;
    int m, k, groups;
    int n_tiles;                  // tiles of features
    int tokens;                   // rows of x per tile, at most the kernel's BN
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
__device__ __forceinline__ bool tile_table(const TileArgs& a, int* before)
{
    const int lane = threadIdx.x & 31;
    if (!a.offsets) {
        if (lane == 0) {
            before[0] = 0;
            before[1] = (a.m + a.tokens - 1) / a.tokens;
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
            count = ok ? (hi - lo + a.tokens - 1) / a.tokens : 0;
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
template <int kFeatures>
__device__ __forceinline__ Tile tile_at(const TileArgs& a, const int* before, int64_t t)
{
    const int mt = (int)(t / a.n_tiles);
    Tile r;
    r.feature = (int)(t % a.n_tiles) * kFeatures;
    if (!a.offsets) {
        r.group = 0;
        r.row = mt * a.tokens;
        r.rows = min(a.tokens, a.m - r.row);
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
    r.row = __ldg(a.offsets + lo) + (mt - before[lo]) * a.tokens;
    r.rows = min(a.tokens, __ldg(a.offsets + lo + 1) - r.row);
    return r;
}

// Bytes [at, at + count) of p, which has `total` bytes, as N words (2 or 4) with
// zeros behind them, in two halves: the loads of the two aligned vectors around
// them, and, when they are wanted, the shifts.  (Shifted at once, each row waited
// for its load: 777 x 1112 x 4128 of fp4q_matmul took 14.4 us, 11.6 this way.)
template <int N> struct Bytes {
    static_assert(N == 2 || N == 4, "vectors");
    uint32_t w[2 * N];
    int back, count;                                       // bytes before the first one, bytes of them
    // 4N aligned bytes, or zeros.
    __device__ __forceinline__ void load_whole(const uint8_t* p, bool in)
    {
        if (N == 4)
            put(0, in ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0));
        else
            put(0, in ? __ldg(reinterpret_cast<const uint2*>(p)) : make_uint2(0, 0));
    }
    __device__ __forceinline__ void load(const uint8_t* p, int64_t at, int64_t total, int n)
    {
        count = n;
        back = (int)(reinterpret_cast<uintptr_t>(p + at) & (4 * N - 1));
        const int64_t lo = at - back;
        if (n <= 0) return;
        if (lo >= 0 && lo + 8 * N <= total) {
            const uint8_t* q = p + lo;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (N == 4)
                    put(i * N, __ldg(reinterpret_cast<const uint4*>(q) + i));
                else
                    put(i * N, __ldg(reinterpret_cast<const uint2*>(q) + i));
            }
        } else {                                           // the ends of the matrix
            back = 0;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                w[i] = 0;
                for (int b = 0; b < 4; ++b)
                    if (4 * i + b < n) w[i] |= (uint32_t)__ldg(p + at + 4 * i + b) << (8 * b);
            }
        }
    }
    template <bool kWhole> __device__ __forceinline__ void words(uint32_t (&v)[N]) const
    {
        if constexpr (kWhole) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = w[i];
        } else {
            uint32_t u[2 * N];
#pragma unroll
            for (int i = 0; i < 2 * N; ++i) u[i] = w[i];
            if (N == 4)
#pragma unroll
                for (int i = 0; i + 2 < 2 * N; ++i) u[i] = back & 8 ? u[i + 2] : u[i];
#pragma unroll
            for (int i = 0; i + 1 < 2 * N; ++i) u[i] = back & 4 ? u[i + 1] : u[i];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int left = count - 4 * i;
                const uint32_t all = __funnelshift_r(u[i], u[i + 1], 8 * (back & 3));
                v[i] = left >= 4 ? all : left > 0 ? all & ((1u << (8 * left)) - 1) : 0;
            }
        }
    }

private:
    __device__ __forceinline__ void put(int i, uint2 u)
    {
        w[i] = u.x;
        w[i + 1] = u.y;
    }
    __device__ __forceinline__ void put(int i, uint4 u)
    {
        put(i, make_uint2(u.x, u.y));
        put(i + 2, make_uint2(u.z, u.w));
    }
};

// This thread block's share of a tile's steps.
__device__ __forceinline__ void split_steps(const TileArgs& a, int rank, int& first, int& last)
{
    first = (int)((int64_t)a.k_steps * rank / a.split);
    last = (int)((int64_t)a.k_steps * (rank + 1) / a.split);
}

// For a dead thread block: the last copies into a ring, whose phases may not
// have been waited for, end before the block does.
template <int N> __device__ __forceinline__ void drain_ring(Ring<N> r, uint32_t full, volatile int* dead)
{
    if (!*dead) return;
    for (int i = 0; i < N; ++i, r.next()) mbar_drain(full + 8 * r.stage, r.parity ^ 1);
}

// Before a block ends: every signal that a stage is free has arrived, as none
// may come after it (a pair's, from the other block).
template <int N> __device__ __forceinline__ void await_empty(Ring<N> r, uint32_t empty, volatile int* dead)
{
    for (int i = 0; i < N; ++i, r.next())
        if (!mbar_wait(empty + 8 * r.stage, r.parity ^ 1, dead)) return;
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

// Columns [c0, c0 + count) of the accumulator; S, bias and act are applied
// on the way where `last` (the sums are complete).
template <bool last>
__device__ __forceinline__ void to_part(uint32_t acc, int c0, int count, float* part, const Scale& S, float bias, int act)
{
    const int quarter = (threadIdx.x / 32) % 4, line = quarter * 32 + (threadIdx.x & 31);
#pragma unroll 1
    for (int c = 0; c < count; c += 16) {
        uint32_t r[16];
        tmem_load16(r, acc + ((uint32_t)quarter << 21) + c0 + c);
        float z[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) z[i] = __uint_as_float(r[i]);
        if (last) {
#pragma unroll
            for (int i = 0; i < 16; ++i) z[i] = S(z[i]) + bias;
            activate(z, act);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) part[(c + i) * kPartRow + line] = z[i];
    }
}

// Whether rows of y consist of whole 16-byte pieces.
template <typename T> __device__ __forceinline__ bool whole_rows(const TileArgs& a)
{
    return a.n % Lanes<T>::kCount == 0;
}

template <typename T> __device__ __forceinline__ float bias_of(const TileArgs& a, const Tile& t, int line)
{
    const int64_t j = t.feature + line;
    return a.ep.bias && j < a.n ? to_f32<T>(static_cast<const T*>(a.ep.bias)[t.group * a.n + j]) : 0.f;
}

// A tile that needs no sum over a cluster; group e of kGroups takes every
// kGroups-th chunk, through a `part` of its own.  `ok`, the warp's: the sums are
// there; the group writes where they are for all of its warps.
template <typename T, int kChunk, int kGroups>
__device__ __forceinline__ void write_tile(const TileArgs& a, const Tile& t, uint32_t acc, const Scale& S, float* part, int e,
                                           bool ok)
{
    constexpr int N = Lanes<T>::kCount, kPer = 128 / N, kItems = kChunk * kPer / 128;
    const int tid = threadIdx.x & 127, line = (threadIdx.x / 32) % 4 * 32 + (threadIdx.x & 31);
    const float bias = bias_of<T>(a, t, line);
    const bool whole = whole_rows<T>(a);
    const int lane = tid % kPer * N, token0 = tid / kPer;             // a thread keeps its features
    const bool in = whole && t.feature + lane < a.n;
    const int64_t at0 = (int64_t)(t.row + token0) * a.n + t.feature + lane, step = (int64_t)(128 / kPer) * a.n;
#pragma unroll 1
    for (int c0 = e * kChunk; c0 < t.rows; c0 += kGroups * kChunk) {
        const int rows = min(kChunk, t.rows - c0);
        const int64_t at = at0 + (int64_t)c0 * a.n;
        Extra x[kItems];
#pragma unroll
        for (int k = 0; k < kItems; ++k)
            if (in && token0 + k * (128 / kPer) < rows) x[k] = load_extra<T>(a.ep, at + k * step);
        if (ok) to_part<true>(acc, c0, rows, part, S, bias, a.ep.act);
        ok = group_all(e, ok);
        if (!ok) return;
        if (whole) {
#pragma unroll
            for (int k = 0; k < kItems; ++k) {
                const int token = token0 + k * (128 / kPer);
                if (!in || token >= rows) continue;
                float z[N];
#pragma unroll
                for (int i = 0; i < N; i += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(part + token * kPartRow + lane + i);
                    z[i] = f.x;
                    z[i + 1] = f.y;
                    z[i + 2] = f.z;
                    z[i + 3] = f.w;
                }
                finish<T>(a.ep, z, x[k], at + k * step);
            }
        } else if (t.feature + line < a.n) {
            // One feature a thread, 16 tokens' mul and residual asked for at once.
            // (Pieces from each row's first 16-byte boundary on took longer: the
            // rows' ends, element by element, held up every warp.)
            int64_t at1 = (int64_t)(t.row + c0) * a.n + t.feature + line;
            if (!a.ep.mul && !a.ep.residual) {
#pragma unroll 4
                for (int c = 0; c < rows; ++c, at1 += a.n)
                    static_cast<T*>(a.ep.y)[at1] = from_f32<T>(part[c * kPartRow + line]);
            } else {
#pragma unroll 1
                for (int c = 0; c < rows; c += 16, at1 += 16 * a.n) {
                    T m[16], r[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        m[i] = a.ep.mul && c + i < rows ? static_cast<const T*>(a.ep.mul)[at1 + i * a.n] : from_f32<T>(1.f);
                        r[i] = a.ep.residual && c + i < rows ? static_cast<const T*>(a.ep.residual)[at1 + i * a.n]
                                                             : from_f32<T>(-0.f);
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i)           // times 1 and plus -0 change nothing
                        if (c + i < rows)
                            static_cast<T*>(a.ep.y)[at1 + i * a.n] =
                                from_f32<T>(part[(c + i) * kPartRow + line] * to_f32<T>(m[i]) + to_f32<T>(r[i]));
                }
            }
        }
        group_bar(e);
    }
}

// A tile whose sums come in pieces: group e keeps every kGroups-th 16 tokens in
// its own `part`, one after the other.
template <int kGroups> __device__ __forceinline__ void add_to_part(uint32_t acc, int rows, float* part, int e, bool add)
{
    const int quarter = (threadIdx.x / 32) % 4, line = quarter * 32 + (threadIdx.x & 31);
#pragma unroll 1
    for (int c0 = 16 * e; c0 < rows; c0 += 16 * kGroups, part += 16 * kPartRow) {
        uint32_t r[16];
        tmem_load16(r, acc + ((uint32_t)quarter << 21) + c0);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float* p = part + i * kPartRow + line;
            *p = add ? *p + __uint_as_float(r[i]) : __uint_as_float(r[i]);
        }
    }
}
template <typename T, int kGroups>
__device__ __forceinline__ void finish_part(const TileArgs& a, const Tile& t, const Scale& S, const float* part, int e)
{
    constexpr int N = Lanes<T>::kCount, kPer = 128 / N;
    const int tid = threadIdx.x & 127;
    if (whole_rows<T>(a)) {
        const int lane = tid % kPer * N;                   // a thread keeps its features
        if (t.feature + lane < a.n) {
            float bias[N];
#pragma unroll
            for (int i = 0; i < N; ++i) bias[i] = bias_of<T>(a, t, lane + i);
#pragma unroll 1
            for (int l = tid / kPer;; l += 128 / kPer) {
                const int c = l / 16 * (16 * kGroups) + 16 * e + l % 16;
                if (l / 16 * (16 * kGroups) + 16 * e >= t.rows) break;
                if (c >= t.rows) continue;
                const int64_t at = (int64_t)(t.row + c) * a.n + t.feature + lane;
                const Extra x = load_extra<T>(a.ep, at);
                float z[N];
#pragma unroll
                for (int i = 0; i < N; ++i) z[i] = S(part[l * kPartRow + lane + i]) + bias[i];
                activate(z, a.ep.act);
                finish<T>(a.ep, z, x, at);
            }
        }
    } else if (t.feature + tid < a.n) {
        const float b = bias_of<T>(a, t, tid);
        for (int c0 = 16 * e, l = 0; c0 < t.rows; c0 += 16 * kGroups, l += 16)
            for (int i = 0; i < 16 && c0 + i < t.rows; ++i) {
                float z[1] = {S(part[(l + i) * kPartRow + tid]) + b};
                activate(z, a.ep.act);
                finish_one<T>(a.ep, z[0], (int64_t)(t.row + c0 + i) * a.n + t.feature + tid);
            }
    }
    group_bar(e);
}

// A tile whose steps a cluster of kSplit blocks shared: every block sends its
// partial sums of token c to block c % kSplit, which adds them in rank order (the
// result does not depend on timing) and finishes the token.  A thread sends its
// feature's sums of 4 (2, for 8 blocks) tokens at a time and finishes that
// feature of the block's own tokens; `part` is [rank][tokens / 4][128][4].
// (Sum by sum, and 16 bytes of y a thread, 512 x 1024 x 1024 of fp4q_linear took
// 13.3 us, 10.4 this way, 16 tokens 6.8 and 6.0; 128 x 4096 x 4096 of MXFP4 in
// fp4q_matmul 9.6 and 10.7, for the narrow stores.  Fetching the partials from
// the peers took two fences and a round trip more.)  `full` counts the bytes that
// arrive here, `empty` has an arrival from every block that sends here: this
// tile's have been read (`more`: there is a next one, which waits for that; no
// signal may reach a block that has ended).
// `ok`, the warp's: its sums are there; `before`: the sums of the runs before the
// one in the accumulator, as add_to_part leaves them, or null.  Returns, to all of
// the group, whether no wait gave up.
template <typename T, int kSplit>
__device__ __forceinline__ bool split_tile(const TileArgs& a, const Tile& t, uint32_t acc, const Scale& S, float* part,
                                           uint32_t full, uint32_t empty, uint32_t parity, uint32_t rank,
                                           volatile int* dead, uint32_t acc_empty, bool more, bool ok,
                                           const float* before)
{
    constexpr int V = kSplit == 8 ? 2 : 4, kEach = 16 / kSplit;      // tokens at a time, of 16 to each block
    using Vec = typename std::conditional<V == 4, uint4, uint2>::type;
    const int tid = threadIdx.x & 127, quarter = (threadIdx.x / 32) % 4, line = quarter * 32 + (threadIdx.x & 31);
    const int slots = (t.rows + 15) / 16 * kEach;          // tokens of a block, with those past the last row
    const int mine = (t.rows - (int)rank + kSplit - 1) / kSplit;
    if (tid == 0) mbar_expect(full, slots * kSplit * 512);
    ok = ok && mbar_wait(empty, parity ^ 1, dead);         // the tile before has been read everywhere
    if (ok)
#pragma unroll 1
        for (int c0 = 0; c0 < t.rows; c0 += 16) {
            uint32_t r[16];
            tmem_load16(r, acc + ((uint32_t)quarter << 21) + c0);
            if (before) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    r[i] = __float_as_uint(before[(c0 + i) * kPartRow + line] + __uint_as_float(r[i]));
            }
            const uint32_t to = smem_u32(part + ((int)rank * slots + c0 / kSplit) * 128 + line * V);
#pragma unroll
            for (int d = 0; d < kSplit; ++d)
#pragma unroll
                for (int j = 0; j < kEach; j += V) {
                    Vec v;
                    v.x = r[j * kSplit + d];
                    v.y = r[(j + 1) * kSplit + d];
                    if constexpr (V == 4) {
                        v.z = r[(j + 2) * kSplit + d];
                        v.w = r[(j + 3) * kSplit + d];
                    }
                    send(to + j * 512, v, full, d);
                }
        }
    tc_fence_before();
    group_bar(0);
    if (tid == 0) mbar_arrive(acc_empty);
    const float bias = bias_of<T>(a, t, tid);
    const bool in = t.feature + tid < a.n;
    auto at = [&](int s) { return (int64_t)(t.row + s * kSplit + (int)rank) * a.n + t.feature + tid; };
    T m[V], res[V];
    auto load = [&](int s0) {                              // times 1 and plus -0 change nothing
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const bool here = in && s0 + i < mine;
            m[i] = a.ep.mul && here ? static_cast<const T*>(a.ep.mul)[at(s0 + i)] : from_f32<T>(1.f);
            res[i] = a.ep.residual && here ? static_cast<const T*>(a.ep.residual)[at(s0 + i)] : from_f32<T>(-0.f);
        }
    };
    load(0);
    ok = ok && mbar_wait(full, parity, dead);
    if (ok && in)
#pragma unroll 1
        for (int s = 0; s < mine; s += V) {
            float z[V] = {};
#pragma unroll
            for (int q = 0; q < kSplit; ++q) {
                const Vec v = *reinterpret_cast<const Vec*>(part + (q * slots + s) * 128 + tid * V);
                z[0] += __uint_as_float(v.x);
                z[1] += __uint_as_float(v.y);
                if constexpr (V == 4) {
                    z[2] += __uint_as_float(v.z);
                    z[3] += __uint_as_float(v.w);
                }
            }
#pragma unroll
            for (int i = 0; i < V; ++i) z[i] = S(z[i]) + bias;
            activate(z, a.ep.act);
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (s + i < mine)
                    static_cast<T*>(a.ep.y)[at(s + i)] = from_f32<T>(z[i] * to_f32<T>(m[i]) + to_f32<T>(res[i]));
            if (s + V < mine) load(s + V);
        }
    ok = group_all(0, ok);
    if (more && tid < kSplit) mbar_signal_peer(empty, tid);
    return ok;
}
template <typename T>
__device__ __forceinline__ bool write_tile_split(const TileArgs& a, const Tile& t, uint32_t acc, const Scale& S, float* part,
                                                 uint32_t full, uint32_t empty, uint32_t parity, uint32_t rank,
                                                 volatile int* dead, uint32_t acc_empty, bool more, bool ok,
                                                 const float* before)
{
    if (a.split == 2) return split_tile<T, 2>(a, t, acc, S, part, full, empty, parity, rank, dead, acc_empty, more, ok, before);
    if (a.split == 4) return split_tile<T, 4>(a, t, acc, S, part, full, empty, parity, rank, dead, acc_empty, more, ok, before);
    return split_tile<T, 8>(a, t, acc, S, part, full, empty, parity, rank, dead, acc_empty, more, ok, before);
}

}  // namespace fp4q
