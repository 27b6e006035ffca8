// matmul.cu -- fp4q_matmul and fp4q_matmul_group: both operands FP4, on the
// block-scaled tensor-core instructions of sm_100a.
//
// One thread block works on tiles of 128 features x BN tokens (product_tile.cuh)
// in steps of 256 columns, in four roles that meet at mbarriers:
//   warp 0     copies the codes of both operands (128-byte rows, swizzled) and
//              the weight's tiled scales into a ring of kStages steps;
//   warps 2-3  bring the tokens' row-major scales into the tiled layout of the
//              ring, by way of registers;
//   warp 1     moves a step's scales to tensor memory and issues four products
//              of 64 columns;
//   warps 4..  in groups of four, take the accumulator to y.
// The products are exact (2 x 2 significant bits, block scales of 4 x 4) and
// summed in binary32 in tensor memory; the global scales multiply the sum.
//
// Many tokens: two thread blocks of a cluster share a tile of 256 features x
// 192 tokens.  Each holds its 128 features and half of the tokens' codes, and
// the tensor cores of both read both halves, so that a step brings 16 + 12 KB
// to an SM where a tile of its own (128 x 192) would bring 16 + 24 KB for the
// same products (at 4096 x 14336 x 4096 the path through L1 and shared memory is
// then the busiest unit, 67%, with the tensor pipe at 46% and L2 at 41%).  Two
// accumulators of 192 columns let the epilogue of one tile run under the products
// of the next.
#include "product_host.cuh"

namespace fp4q {

namespace {

constexpr int kStepCols = 256;             // columns of a step: 128 bytes of codes
constexpr int kMmaCols = 64;

// The tensor core truncates where it adds: a float result falls short by 4e-7 of
// its norm after 2048 columns, 9e-7 after 4096, 1.9e-5 after 65536 (a plain
// binary32 sum of 4096 is off by 4e-7).  So longer float sums come in runs of
// 4096 columns that are added in shared memory (RUNS), which leaves room for
// fewer stages: 4096 x 4096 x 14336 NVFP4 takes 145 us so, 128 with the one
// accumulator, 140 with the sums in the epilogue's registers.  bf16 ones, whose
// rounding is 2e-3, come in runs of 65536.
template <typename T> constexpr int kRun = (sizeof(T) == 4 ? 4096 : 65536) / kStepCols;      // steps

template <int BN, bool RUNS> struct Config {
    static constexpr int kPair = BN > 128 ? 2 : 1;                  // thread blocks of a tile
    static constexpr int kTokenTiles = (BN + 127) / 128;            // scale tiles over the tokens
    static constexpr int kW = 128 * 128, kX = BN / kPair * 128;     // bytes of a step
    static constexpr int kWS = 4 * 512, kXS = kTokenTiles * 4 * 512;
    static constexpr int kStage = kW + kX + kWS + kXS;
    static constexpr int kStages = BN > 128 && RUNS ? 3 : BN > 64 && RUNS ? 4 : BN > 32 ? 5 : 8;
    static constexpr int kAccs = 2;
    // Tensor memory: accumulators, then the scales of the last two steps.
    static constexpr int kScaleCols = 4 * 4 * (1 + kTokenTiles);
    static constexpr int kUsed = kAccs * BN + 2 * kScaleCols;
    static constexpr int kCols = kUsed <= 128 ? 128 : kUsed <= 256 ? 256 : 512;
    static constexpr bool kSplits = BN <= 64;
    static constexpr int kEpi = BN >= 128 ? 2 : 1;                  // groups of four epilogue warps
    static constexpr int kPart = (kSplits ? BN : RUNS ? BN / kEpi : 32) * kPartRow * 4;      // sums on their way to y, per group
    static constexpr int kThreads = (4 + 4 * kEpi) * 32;
    static constexpr int kSmem = kStages * kStage + (kSplits && RUNS ? 2 : kEpi) * kPart + 1024;
    static constexpr int kResident = 1;
    static_assert(kUsed <= 512 && kCols * kResident <= 512, "tensor memory");
    static_assert(kSmem <= 222 * 1024 && kStage % 1024 == 0, "shared memory");
};

template <bool MX, int BN, typename T, bool RUNS>
__global__ void __launch_bounds__(Config<BN, RUNS>::kThreads, Config<BN, RUNS>::kResident)
matmul_kernel(const __grid_constant__ CUtensorMap w_map, const __grid_constant__ CUtensorMap x_map,
              const __grid_constant__ TileArgs a)
{
    using C = Config<BN, RUNS>;
    constexpr int G = C::kPair;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t bars[3 * C::kStages + 2 * C::kAccs + 3];
    __shared__ int before[FP4Q_PRODUCT_GROUPS_MAX + 1];
    __shared__ uint32_t tmem_slot;
    __shared__ int dead_word, good_offsets;
    volatile int* dead = &dead_word;

    const int warp = __shfl_sync(~0u, threadIdx.x / 32, 0), lane = threadIdx.x & 31;
    uint8_t* ring = raw + (1024 - smem_u32(raw) % 1024) % 1024;
    float* part = reinterpret_cast<float*>(ring + C::kStages * C::kStage);
    const uint32_t ring0 = smem_u32(ring);
    const uint32_t full = smem_u32(bars), empty = full + 8 * C::kStages, peer_full = empty + 8 * C::kStages,
                   acc_full = peer_full + 8 * C::kStages, acc_empty = acc_full + 8 * C::kAccs,
                   part_full = acc_empty + 8 * C::kAccs, part_empty = part_full + 8, drain = part_empty + 8;
    const bool cluster = G > 1 || a.split > 1;
    const uint32_t rank = cluster ? cluster_rank() : 0;

    if (warp == 0) {
        if (lane == 0) {
            dead_word = 0;
            for (int i = 0; i < C::kStages; ++i) {
                mbar_init(full + 8 * i, 1 + 1);            // the copies, the warp of the token scales
                mbar_init(empty + 8 * i, 1);
                mbar_init(peer_full + 8 * i, 1);
            }
            for (int i = 0; i < C::kAccs; ++i) {
                mbar_init(acc_full + 8 * i, 1);
                mbar_init(acc_empty + 8 * i, G * C::kEpi);
            }
            mbar_init(part_full, 1);
            mbar_init(part_empty, a.split);
            mbar_init(drain, 1);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
            tma_prefetch_desc(&w_map);
            tma_prefetch_desc(&x_map);
        }
    } else if (warp == 1) {
        tmem_alloc<G>(smem_u32(&tmem_slot), C::kCols);
    } else if (warp == 2) {
        const bool ok = tile_table(a, before);
        if (lane == 0) good_offsets = ok;
    }
    tc_fence_before();
    __syncthreads();
    // A pair uses each other's memory from the start, a split tile in its epilogue.
    if (cluster) cluster_arrive();
    if (G > 1) cluster_wait();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const int64_t tiles = good_offsets ? (int64_t)before[a.groups] * a.n_tiles : 0;
    if (!good_offsets && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.status, FP4Q_FLAG_OFFSETS);
    const int blocks = G > 1 ? G : a.split;                // of a tile
    const int64_t first_tile = blockIdx.x / blocks, tile_step = gridDim.x / blocks;
    constexpr int kScaleTile = MX ? 128 : 64;              // columns of a scale tile
    constexpr int kScaleTiles = kStepCols / kScaleTile;    // of a step
    int k0, k1;
    split_steps(a, G > 1 ? 0 : (int)rank, k0, k1);
    // The tile with this thread block's features.
    auto my_tile = [&](int64_t t) {
        Tile r = tile_at<128 * G>(a, before, t);
        if (G > 1) r.feature += 128 * rank;
        return r;
    };
    // Tokens of a tile as the tensor core counts them.
    auto mma_cols = [&](const Tile& t) { return (t.rows + 16 * G - 1) / (16 * G) * (16 * G); };

    if (warp == 0) {
        Ring<C::kStages> g;
        bool ok = true;
        for (int64_t t = first_tile; ok && t < tiles; t += tile_step) {
            const Tile tl = my_tile(t);
            const int wrow = (int)(tl.group * a.n) + tl.feature;
            const int xrow = tl.row + (G > 1 ? (int)rank * (mma_cols(tl) / G) : 0);
            // Past the last feature (the second half of a pair's tile) any scales will do.
            const int64_t row_tile = min((int64_t)tl.feature, a.n - 1) / 128;
            const uint8_t* ws = a.w_scales + tl.group * a.w_scale_stride + row_tile * a.w_col_tiles * 512;
            for (int k = k0; k < k1; ++k, g.next()) {
                if (!(ok = mbar_wait(empty + 8 * g.stage, g.parity ^ 1, dead))) break;
                const uint32_t at = ring0 + g.stage * C::kStage, bar = full + 8 * g.stage;
                const int c0 = k * kScaleTiles;
                const uint32_t sb = (uint32_t)min(kScaleTiles, a.w_col_tiles - c0) * 512;
                if (elect_one()) {
                    mbar_expect(bar, C::kW + a.tokens / G * 128 + sb);
                    tma_load(at, &w_map, k * (kStepCols / 2), wrow, bar);
                    tma_load(at + C::kW, &x_map, k * (kStepCols / 2), xrow, bar);
                    bulk_load(at + C::kW + C::kX, ws + (int64_t)c0 * 512, sb, bar);
                }
                __syncwarp();
            }
        }
        await_empty(g, empty, dead);
        drain_ring(g, full, dead);
    } else if (warp == 1 && rank % G != 0) {
        // The odd block of a pair tells the even one, which issues for both,
        // that its half of a step is there.
        Ring<C::kStages> g;
        bool ok = true;
        for (int64_t t = first_tile; ok && t < tiles; t += tile_step)
            for (int k = k0; k < k1; ++k, g.next()) {
                if (!(ok = mbar_wait(full + 8 * g.stage, g.parity, dead))) break;
                __syncwarp();
                if (lane == 0) mbar_signal_peer(peer_full + 8 * g.stage, rank - 1);
            }
    } else if (warp == 1) {
        Ring<C::kStages> g, last2;                         // last2 follows two steps behind
        Ring<C::kAccs> ac;
        uint32_t step = 0;
        bool ok = true;
        for (int64_t t = first_tile; ok && t < tiles; t += tile_step, ac.next()) {
            const Tile tl = my_tile(t);
            const uint32_t cols = mma_cols(tl);
            uint32_t acc = tmem + ac.stage * BN;
            if (!(ok = mbar_wait(acc_empty + 8 * ac.stage, ac.parity ^ 1, dead))) break;
            for (int k = k0, first = k0; k < k1; ++k, g.next(), ++step) {
                if (RUNS && k - first == kRun<T>) {        // the next run, into the other accumulator
                    if (elect_one()) tc_commit<G>(acc_full + 8 * ac.stage);
                    __syncwarp();
                    ac.next();
                    acc = tmem + ac.stage * BN;
                    first = k;
                    if (!(ok = mbar_wait(acc_empty + 8 * ac.stage, ac.parity ^ 1, dead))) break;
                }
                ok = mbar_wait(full + 8 * g.stage, g.parity, dead);
                if (G > 1) ok = ok && mbar_wait(peer_full + 8 * g.stage, g.parity, dead);
                if (step >= 2) {                           // whose scales were where this step's go
                    ok = ok && mbar_wait(empty + 8 * last2.stage, last2.parity, dead);
                    last2.next();
                }
                if (!ok) break;
                tc_fence_after();
                const uint32_t at = ring0 + g.stage * C::kStage;
                const uint32_t sf = tmem + C::kAccs * BN + step % 2 * C::kScaleCols;
                const int parts = min(kStepCols / kMmaCols, (a.k - k * kStepCols + kMmaCols - 1) / kMmaCols);
                const uint64_t wd = desc_k128(at), xd = desc_k128(at + C::kW),
                               sd = desc_scales(at + C::kW + C::kX);
                if (elect_one()) {
#pragma unroll
                    for (int i = 0; i < kScaleTiles; ++i) {
                        if (i * (kScaleTile / kMmaCols) >= parts) break;
                        tc_copy_scales<G>(sf + i * 4, sd + i * (512 >> 4));
#pragma unroll
                        for (int h = 0; h < C::kTokenTiles; ++h)
                            tc_copy_scales<G>(sf + 16 + i * 4 * C::kTokenTiles + h * 4,
                                              sd + ((C::kWS + (i * C::kTokenTiles + h) * 512) >> 4));
                    }
#pragma unroll
                    for (int i = 0; i < kStepCols / kMmaCols; ++i) {
                        if (i >= parts) break;
                        const int st = MX ? i / 2 : i;
                        tc_mma_fp4<MX, G>(acc, wd + i * 2, xd + i * 2,
                                          idesc_fp4(MX, 128 * G, cols, MX ? (i % 2) * 2 : 0), sf + st * 4,
                                          sf + 16 + st * 4 * C::kTokenTiles, k > first || i > 0);
                    }
                    tc_commit<G>(empty + 8 * g.stage);
                }
                __syncwarp();
            }
            if (ok && elect_one()) tc_commit<G>(acc_full + 8 * ac.stage);
            __syncwarp();
        }
        await_empty(ac, acc_empty, dead);
        if (__any_sync(~0u, *dead)) {
            if (elect_one()) tc_commit<G>(drain);
            mbar_drain(drain, 0);
        }
    } else if (warp < 4) {
        // Token scales: the two warps take turns with the steps, a lane takes
        // rows lane, lane + 32, ...  A row's scales of one tile are 4
        // neighbouring bytes, at (r % 32) * 16 + (r / 32) * 4 of that tile.  A
        // step's loads are issued when the one before last has been stored, so
        // that they are on their way while the ring is waited for.  One load a
        // row where rows start on boundaries of a step's bytes, else two; a loop
        // for each (one for both, shifting by nothing, cost 4096 x 14336 x 4096 10%).
        constexpr int kRows = (BN + 31) / 32;
        const int64_t scols = a.k / (MX ? 32 : 16), total = (int64_t)a.m * scols;
        auto bring = [&](auto whole) {                     // whether rows start on boundaries
            constexpr bool kWhole = decltype(whole)::value;
            Bytes<kScaleTiles> v[kRows];
            auto load = [&](const Tile& tl, int k) {
                const int64_t c0 = (int64_t)k * kScaleTiles * 4;
#pragma unroll
                for (int q = 0; q < kRows; ++q) {
                    const int r = lane + 32 * q;
                    const bool in = r < tl.rows;
                    const int64_t at = (tl.row + r) * scols + c0;
                    if (kWhole)
                        v[q].load_whole(a.x_scales + at, in);
                    else
                        v[q].load(a.x_scales, at, total, in ? (int)min(scols - c0, (int64_t)4 * kScaleTiles) : 0);
                }
            };
            Ring<C::kStages> g;
            int64_t t = first_tile;
            int k = k0;
            Tile tl;
            auto next = [&] {                              // the step after (t, k)
                g.next();
                if (++k == k1) {
                    k = k0;
                    t += tile_step;
                    if (t < tiles) tl = my_tile(t);
                }
            };
            if (t < tiles) tl = my_tile(t);
            if (warp == 3 && t < tiles) next();
            if (t < tiles) load(tl, k);
            while (t < tiles) {
                if (!mbar_wait(empty + 8 * g.stage, g.parity ^ 1, dead)) break;
                uint8_t* xs = ring + g.stage * C::kStage + C::kW + C::kX + C::kWS;
#pragma unroll
                for (int q = 0; q < kRows; ++q) {
                    const int r = lane + 32 * q;
                    if (r >= BN) break;
                    uint32_t u[kScaleTiles];
                    v[q].template words<kWhole>(u);
#pragma unroll
                    for (int i = 0; i < kScaleTiles; ++i)
                        *reinterpret_cast<uint32_t*>(xs + (i * C::kTokenTiles + q / 4) * 512 + lane * 16 + q % 4 * 4) = u[i];
                }
                fence_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(full + 8 * g.stage);
                next();
                if (t < tiles) next();
                if (t < tiles) load(tl, k);
            }
        };
        if (scols % (4 * kScaleTiles) == 0 && (reinterpret_cast<uintptr_t>(a.x_scales) & (4 * kScaleTiles - 1)) == 0)
            bring(std::true_type{});
        else
            bring(std::false_type{});
    } else {
        const int e = (warp - 4) / 4;
        if (G == 1 && cluster) cluster_wait();
        Ring<C::kAccs> ac;
        uint32_t parity = 0;
        bool ok = true;
        for (int64_t t = first_tile; ok && t < tiles; t += tile_step, ac.next(), parity ^= 1) {
            const Tile tl = my_tile(t);
            const Scale S = MX ? scale_of(1.f) : scale_of(a.w_S[tl.group], *a.x_S);
            auto release = [&](uint32_t stage) {           // the accumulator has been read by this group
                tc_fence_before();
                ok = group_all(e, ok);
                if (warp % 4 == 0 && lane == 0) {
                    if (G > 1)
                        mbar_signal_peer(acc_empty + 8 * stage, rank & ~1u);
                    else
                        mbar_arrive(acc_empty + 8 * stage);
                }
            };
            if (RUNS) {
                // of a split tile behind its partial sums, which the last run's join
                const bool split = C::kSplits && a.split > 1;
                float* mine = part + (split ? 1 : e) * (C::kPart / 4);
                for (int k = k0; ok && k < k1; k += kRun<T>) {
                    if (k > k0) ac.next();
                    ok = mbar_wait_long(acc_full + 8 * ac.stage, ac.parity, dead);
                    tc_fence_after();
                    if (split && k + kRun<T> >= k1) break;
                    if (ok) add_to_part<C::kEpi>(tmem + ac.stage * BN, tl.rows, mine, e, k > k0);
                    release(ac.stage);
                }
                if (split)
                    ok = write_tile_split<T>(a, tl, tmem + ac.stage * BN, S, part, part_full, part_empty, parity, rank, dead,
                                             acc_empty + 8 * ac.stage, t + tile_step < tiles, ok,
                                             k1 - k0 > kRun<T> ? mine : nullptr);
                else if (ok)
                    finish_part<T, C::kEpi>(a, tl, S, mine, e);
                continue;
            }
            const uint32_t acc = tmem + ac.stage * BN;
            ok = mbar_wait_long(acc_full + 8 * ac.stage, ac.parity, dead);
            tc_fence_after();
            if (C::kSplits && a.split > 1) {
                ok = write_tile_split<T>(a, tl, acc, S, part, part_full, part_empty, parity, rank, dead,
                                         acc_empty + 8 * ac.stage, t + tile_step < tiles, ok, nullptr);
            } else {
                write_tile<T, Chunk<T, BN>::kTokens, C::kEpi>(a, tl, acc, S, part + e * (C::kPart / 4), e, ok);
                release(ac.stage);
            }
        }
    }
    __syncwarp();
    if (G == 1 && cluster && warp < 4) cluster_wait();
    tc_fence_before();
    __syncthreads();
    if (cluster) {                             // a peer may still use this block's shared or tensor memory
        cluster_arrive();
        cluster_wait();
    }
    tc_fence_after();
    if (warp == 1) tmem_free<G>(tmem, C::kCols);
    if (*dead) {
        linger();
        if (threadIdx.x == 0) atomicOr(a.status, FP4Q_FLAG_TIMEOUT);
    }
}

}  // namespace

template <bool MX, int BN, typename T, bool RUNS = false>
static cudaError_t launch_one(const Product& p, TileArgs& a, const TileShape& shape, cudaStream_t s)
{
    using C = Config<BN, RUNS>;
    auto kernel = matmul_kernel<MX, BN, T, RUNS>;
    CUtensorMap w_map, x_map;
    cudaError_t e = byte_tile_map(&w_map, p.w, p.n * p.groups, p.k / 2, 128);
    if (e == cudaSuccess) e = byte_tile_map(&x_map, p.x, p.m, p.k / 2, shape.tokens / C::kPair);
    if (e != cudaSuccess) return e;
    static Residency residency;
    const int per_sm = product_blocks_per_sm(residency, reinterpret_cast<const void*>(kernel), C::kThreads, C::kSmem);
    return launch_tiles(kernel, w_map, x_map, p, a, shape, C::kPair, per_sm, C::kThreads, C::kSmem, s);
}

template <bool MX, typename T> static cudaError_t launch_shape(const Product& p, cudaStream_t s)
{
    TileArgs a = tile_args(p, kStepCols, MX ? 128 : 64);
    const TileShape shape = tile_shape(p, a.k_steps, 2, {kRun<T>, sizeof(T) == 4 ? 192 : 64, true});
    if ((a.k_steps + shape.split - 1) / shape.split > kRun<T>) {
        if constexpr (sizeof(T) == 4) {
            if (shape.tokens > 128) return launch_one<MX, 192, T, true>(p, a, shape, s);
            if (shape.tokens > 64) return launch_one<MX, 128, T, true>(p, a, shape, s);
        }
        return launch_one<MX, 64, T, true>(p, a, shape, s);
    }
    if (shape.tokens <= 16) return launch_one<MX, 16, T>(p, a, shape, s);
    if (shape.tokens <= 32) return launch_one<MX, 32, T>(p, a, shape, s);
    if (shape.tokens <= 64) return launch_one<MX, 64, T>(p, a, shape, s);
    if (shape.tokens <= 128) return launch_one<MX, 128, T>(p, a, shape, s);
    return launch_one<MX, 192, T>(p, a, shape, s);
}

cudaError_t launch_matmul(const Product& p, cudaStream_t s)
{
    if (p.mx) return p.out_bf16 ? launch_shape<true, __nv_bfloat16>(p, s) : launch_shape<true, float>(p, s);
    return p.out_bf16 ? launch_shape<false, __nv_bfloat16>(p, s) : launch_shape<false, float>(p, s);
}

}  // namespace fp4q
