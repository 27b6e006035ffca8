// linear.cu -- fp4q_linear and fp4q_linear_group: bf16 activations times FP4
// weights on the bf16 tensor cores of sm_100a.
//
// q * s of an NVFP4 element has at most 2 + 4 significant bits and q * 2^e of an
// MXFP4 element 2, so a decoded weight is a bf16 value and the product needs no
// rounding of the weight.  The weight is decoded once per tile, by the thread
// that owns its row, from shared memory straight into tensor memory, where the
// tensor core takes it as the operand that fills the 128 lanes; x goes from
// global to shared memory as it is.  Roles of a thread block's warps, meeting
// at mbarriers:
//   warp 0     copies codes and scales into a ring (steps of 256 columns);
//   warp 3     copies x into another (sub-steps of 64 columns, 128-byte rows, swizzled);
//   warp 1     issues the products, 4 of 16 columns per sub-step;
//   warp 2     the tile table, then idle;
//   warps 4..  in kDq groups of four, decode, a sub-step per group at a time;
//   the last   in groups of four, take the accumulator to y (product_tile.cuh).
#include <climits>

#include "decode.cuh"
#include "product_host.cuh"

namespace fp4q {

namespace {

constexpr int kStepCols = 256;             // columns of a step of W: 128 bytes of codes
constexpr int kSubCols = 64;               // columns of a step of x and of decoded W
constexpr int kSubs = kStepCols / kSubCols;
constexpr int kTableBytes = 65536;
constexpr int kACols = kSubCols / 2;       // columns of tensor memory per decoded sub-step

// The tensor core truncates where it adds: a float result falls short by 1.2e-6
// of its norm after 2048 columns, by 3.3e-6 after 8192, 2.6e-5 after 65536 (a
// plain binary32 sum of 8192 is off by 8e-7).  So longer float sums come in runs
// of 2048 columns that are added in shared memory (RUNS); bf16 ones, whose
// rounding is 2e-3, in runs of 65536.
template <typename T> constexpr int kRun = (sizeof(T) == 4 ? 2048 : 65536) / kStepCols;      // steps

template <int BN, typename T, bool RUNS> struct Config {
    static constexpr bool kRuns = RUNS;
    static constexpr int kPair = BN > 128 ? 2 : 1;                  // thread blocks of a tile
    static constexpr int kW = 128 * 128, kWStage = kW + 4 * 512;
    static constexpr int kXSubs = BN > 64 ? 1 : 4;                  // sub-steps in a stage of x
    static constexpr int kXTile = BN / kPair * 128, kX = kXSubs * kXTile;
    // Few tokens: codes decoded by table (see decode8_table), which takes the
    // second 64 KB of shared memory; x and the sums lie before it, W behind.
    static constexpr bool kTable = BN <= 32;
    static constexpr int kWStages = BN > 64 ? (kRuns ? 4 : 5) : BN > 32 ? 6 : 5;
    static constexpr int kXStages = BN > 128 ? 6 : BN > 64 ? 4 : BN > 32 ? 2 : BN > 16 ? 2 : 4;
    static constexpr int kAccs = 2;
    static constexpr int kDq = BN <= 64 ? 4 : 2;                    // groups of four decoding warps
    static constexpr int kEpi = BN > 64 ? 2 : 1;                    // groups of four epilogue warps
    static constexpr int kThreads = (4 + 4 * kDq + 4 * kEpi) * 32;
    static constexpr int kADepth = 2;                               // decoded sets in tensor memory
    static constexpr int kUsed = kAccs * BN + kADepth * kDq * kACols;
    static constexpr int kCols = kUsed <= 256 ? 256 : 512;
    static constexpr bool kSplits = BN <= 64;
    static constexpr int kPart = (kSplits ? BN : kRuns ? BN / kEpi : 32) * kPartRow * 4;     // sums on their way to y, per group
    static constexpr int kSmem = kWStages * kWStage + (kTable ? 2 * kTableBytes : kXStages * kX + kEpi * kPart + 1024);
    static_assert(!kTable || kXStages * kX + kEpi * kPart + 1024 <= kTableBytes - 8192, "room before the table");
    static constexpr int kResident = 1;
    static_assert(kUsed <= 512 && kCols * kResident <= 512, "tensor memory");
    static_assert(kSmem <= (kTable ? 226 : 222) * 1024 && kWStage % 1024 == 0 && kX % 1024 == 0, "shared memory");
};

// The same by table, q itself times its half of `scale`: entry b of 256 holds
// the pair of code byte b, 32 times in a row, one for the bank of each lane (no
// conflicts whatever the codes).  Entries are 256 bytes apart and the table
// starts at a multiple of 65536, so that one permutation puts an address
// together: bits 15..8 the code byte, the rest `lane_base`.  One operation of
// the ALU pipe a pair and a load: 64 KB of shared memory, which few tokens
// leave free, and their products are the ones that wait for the decoding.
template <int J> __device__ __forceinline__ uint32_t lookup2(uint32_t w, uint32_t lane_base, uint32_t scale)
{
    uint32_t v;
    asm("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(prmt<4 | J << 4 | 6 << 8 | 7 << 12>(w, lane_base)));
    return mul_bf16x2(v, scale);
}
__device__ __forceinline__ void decode8_table(uint32_t w, uint32_t lane_base, uint32_t scale, uint32_t* out)
{
    out[0] = lookup2<0>(w, lane_base, scale);
    out[1] = lookup2<1>(w, lane_base, scale);
    out[2] = lookup2<2>(w, lane_base, scale);
    out[3] = lookup2<3>(w, lane_base, scale);
}
// Entry b of the table: the pair of its low and high nibble.
__device__ __forceinline__ uint32_t table_entry(uint32_t b)
{
    uint32_t out[4];
    decode8(b, 0x7E807E80u, out);                          // * 2^126
    return out[0];
}

// 64 columns of one row: 32 bytes of codes, and their scales.
template <bool TABLE>
__device__ __forceinline__ void decode_nvfp4(const uint32_t (&c)[8], uint32_t scales, uint32_t lane_base,
                                             uint32_t (&v)[32])
{
    uint32_t f[2];
    nv_factors<TABLE>(scales, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (TABLE)
            decode8_table(c[i], lane_base, one_factor(f[i / 4], i / 2 % 2), v + 4 * i);
        else
            decode8(c[i], one_factor(f[i / 4], i / 2 % 2), v + 4 * i);
    }
}
// The two E8M0 bytes in the low half of `scales`.
template <bool TABLE>
__device__ __forceinline__ void decode_mxfp4(const uint32_t (&c)[8], uint32_t scales, uint32_t lane_base,
                                             uint32_t (&v)[32])
{
    uint32_t rest = 0;
    const uint32_t f = TABLE ? mx_factors_table(scales) : mx_factors(scales, rest);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (TABLE)
            decode8_table(c[i], lane_base, one_factor(f, i / 4), v + 4 * i);
        else
            decode8(c[i], one_factor(f, i / 4), v + 4 * i);
    }
    if (!TABLE && rest) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = mul_bf16x2(v[i], one_factor(rest, i / 16));
    }
}

// D[128 G][N] (+)= A[128 G][16] * B[N][16]^T, bf16, A in tensor memory.  Of a
// pair, each thread block holds its 128 rows of A and D and half the rows of B.
template <int G>
__device__ __forceinline__ void tc_mma_bf16(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add)
{
    if (G == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
            "r"((uint32_t)add)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
            "r"((uint32_t)add)
            : "memory");
}
// Binary32 sums (1 << 4) of bf16 operands (1 << 7, 1 << 10), both K-major, m x n.
__device__ __forceinline__ uint32_t idesc_bf16(uint32_t m, uint32_t n)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | ((n >> 3) << 17) | ((m >> 4) << 24);
}
// One row's pairs, a column of tensor memory each; complete on return.
__device__ __forceinline__ void tmem_store(uint32_t addr, const uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};\n\t"
        "tcgen05.wait::st.sync.aligned;" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

template <bool MX, int BN, typename T, bool RUNS>
__global__ void __launch_bounds__(Config<BN, T, RUNS>::kThreads, Config<BN, T, RUNS>::kResident)
linear_kernel(const __grid_constant__ CUtensorMap w_map, const __grid_constant__ CUtensorMap x_map,
              const __grid_constant__ TileArgs a)
{
    using C = Config<BN, T, RUNS>;
    constexpr int G = C::kPair;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t bars[2 * (C::kWStages + C::kXStages + C::kAccs) + 3 * C::kADepth + 3];
    __shared__ int before[FP4Q_PRODUCT_GROUPS_MAX + 1];
    __shared__ uint32_t tmem_slot;
    __shared__ int dead_word, good_offsets;
    volatile int* dead = &dead_word;

    const int warp = __shfl_sync(~0u, threadIdx.x / 32, 0), lane = threadIdx.x & 31;
    uint8_t* aligned = raw + (1024 - smem_u32(raw) % 1024) % 1024;
    uint8_t* table = raw + (kTableBytes - smem_u32(raw) % kTableBytes);
    uint8_t* w_ring = C::kTable ? table + kTableBytes : aligned;
    uint8_t* x_ring = C::kTable ? aligned : w_ring + C::kWStages * C::kWStage;
    float* part = reinterpret_cast<float*>(x_ring + C::kXStages * C::kX);
    const uint32_t w_full = smem_u32(bars), w_empty = w_full + 8 * C::kWStages, x_full = w_empty + 8 * C::kWStages,
                   x_empty = x_full + 8 * C::kXStages, a_full = x_empty + 8 * C::kXStages, a_empty = a_full + 8 * C::kADepth,
                   acc_full = a_empty + 8 * C::kADepth, acc_empty = acc_full + 8 * C::kAccs,
                   peer_full = acc_empty + 8 * C::kAccs, part_full = peer_full + 8 * C::kADepth, part_empty = part_full + 8, drain = part_empty + 8;
    const bool cluster = G > 1 || a.split > 1;
    const uint32_t rank = cluster ? cluster_rank() : 0;

    if (warp == 0) {
        if (lane == 0) {
            dead_word = 0;
            for (int i = 0; i < C::kWStages; ++i) {
                mbar_init(w_full + 8 * i, 1);
                mbar_init(w_empty + 8 * i, 4 * C::kDq);
            }
            for (int i = 0; i < C::kXStages; ++i) {
                mbar_init(x_full + 8 * i, 1);
                mbar_init(x_empty + 8 * i, 1);
            }
            for (int i = 0; i < C::kADepth; ++i) {
                mbar_init(a_full + 8 * i, 4 * C::kDq);
                mbar_init(a_empty + 8 * i, 1);
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
    const uint32_t tmem = tmem_slot, a_tmem = tmem + C::kAccs * BN;
    const int64_t tiles = good_offsets ? (int64_t)before[a.groups] * a.n_tiles : 0;
    if (!good_offsets && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.status, FP4Q_FLAG_OFFSETS);
    const int blocks = G > 1 ? G : a.split;                // of a tile
    const int64_t first_tile = blockIdx.x / blocks, tile_step = gridDim.x / blocks;
    constexpr int kScaleTile = MX ? 128 : 64;              // columns of a scale tile
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
    const int run = C::kRuns && a.split == 1 ? kRun<T> : INT_MAX;       // steps of an accumulator
    // sub-steps of 64 columns of step k
    auto subs = [&](int k) { return min(kSubs, (a.k - k * kStepCols + kSubCols - 1) / kSubCols); };

    if (warp == 0) {
        Ring<C::kWStages> w;
        bool ok = true;
        for (int64_t t = first_tile; ok && t < tiles; t += tile_step) {
            const Tile tl = my_tile(t);
            const int wrow = (int)(tl.group * a.n) + tl.feature;
            const uint8_t* ws = a.w_scales + tl.group * a.w_scale_stride +
                                min((int64_t)tl.feature, a.n - 1) / 128 * a.w_col_tiles * 512;   // any, past the last feature
            for (int k = k0; k < k1; ++k, w.next()) {
                if (!(ok = mbar_wait(w_empty + 8 * w.stage, w.parity ^ 1, dead))) break;
                const uint32_t at = smem_u32(w_ring) + w.stage * C::kWStage, bar = w_full + 8 * w.stage;
                const int c0 = k * (kStepCols / kScaleTile);
                const uint32_t sb = (uint32_t)min(kStepCols / kScaleTile, a.w_col_tiles - c0) * 512;
                if (elect_one()) {
                    mbar_expect(bar, C::kW + sb);
                    tma_load(at, &w_map, k * (kStepCols / 2), wrow, bar);
                    bulk_load(at + C::kW, ws + (int64_t)c0 * 512, sb, bar);
                }
                __syncwarp();
            }
        }
        drain_ring(w, w_full, dead);
    } else if (warp == 3) {
        Ring<C::kXStages> x;
        bool ok = true;
        for (int64_t t = first_tile; ok && t < tiles; t += tile_step) {
            const Tile tl = my_tile(t);
            const int c1 = min(a.k, k1 * kStepCols);
            const int xrow = tl.row + (G > 1 ? (int)rank * (mma_cols(tl) / G) : 0);
            for (int c = k0 * kStepCols; c < c1; c += kSubCols * C::kXSubs, x.next()) {
                if (!(ok = mbar_wait(x_empty + 8 * x.stage, x.parity ^ 1, dead))) break;
                const uint32_t bar = x_full + 8 * x.stage;
                const int count = min(C::kXSubs, (c1 - c + kSubCols - 1) / kSubCols);
                if (elect_one()) {
                    mbar_expect(bar, count * (a.tokens / G) * 128);
#pragma unroll
                    for (int i = 0; i < C::kXSubs; ++i)
                        if (i < count)
                            tma_load(smem_u32(x_ring) + x.stage * C::kX + i * C::kXTile, &x_map,
                                     (c + i * kSubCols) * 2, xrow, bar);
                }
                __syncwarp();
            }
        }
        await_empty(x, x_empty, dead);
        drain_ring(x, x_full, dead);
    } else if (warp == 1 && rank % G != 0) {
        // The odd block of a pair tells the even one, which issues for both,
        // that its half of a set and of its x is there.
        Ring<C::kXStages> x;
        Ring<C::kADepth> d;
        bool ok = true;
        for (int64_t t = first_tile; ok && t < tiles; t += tile_step)
            for (int k = k0; ok && k < k1; ++k) {
                const int count = subs(k);
                for (int i = 0; ok && i < count; i += C::kDq, d.next()) {
                    for (int q = 0; q < C::kDq && i + q < count; ++q, x.next())
                        ok = ok && mbar_wait(x_full + 8 * x.stage, x.parity, dead);
                    ok = ok && mbar_wait(a_full + 8 * d.stage, d.parity, dead);
                    tc_fence_after();
                    tc_fence_before();
                    __syncwarp();
                    if (ok && lane == 0) mbar_signal_peer(peer_full + 8 * d.stage, rank - 1);
                }
            }
        await_empty(d, a_empty, dead);
    } else if (warp == 1) {
        Ring<C::kXStages> x;
        Ring<C::kADepth> d;
        Ring<C::kAccs> ac;
        bool ok = true;
        const uint64_t desc0 = desc_k128(smem_u32(x_ring));
        for (int64_t t = first_tile; ok && t < tiles; t += tile_step, ac.next()) {
            const Tile tl = my_tile(t);
            const uint32_t idesc = idesc_bf16(128 * G, mma_cols(tl));
            uint32_t acc = tmem + ac.stage * BN;
            if (!(ok = mbar_wait(acc_empty + 8 * ac.stage, ac.parity ^ 1, dead))) break;
            tc_fence_after();
            for (int k = k0, first = k0; ok && k < k1; ++k) {
                if (C::kRuns && k - first == run) {        // the next one, into the other accumulator
                    if (elect_one()) tc_commit<G>(acc_full + 8 * ac.stage);
                    __syncwarp();
                    ac.next();
                    acc = tmem + ac.stage * BN;
                    first = k;
                    if (!(ok = mbar_wait(acc_empty + 8 * ac.stage, ac.parity ^ 1, dead))) break;
                    tc_fence_after();
                }
                const int count = subs(k);
#pragma unroll
                for (int i = 0; i < kSubs; i += C::kDq) {  // a decoded set
                    if (i >= count) break;
                    Ring<C::kXStages> xs[C::kDq];          // where its sub-steps' x is
#pragma unroll
                    for (int q = 0; q < C::kDq; ++q) {
                        xs[q] = x;
                        if ((i + q) % C::kXSubs == C::kXSubs - 1 && i + q < count) x.next();
                    }
#pragma unroll
                    for (int q = 0; q < C::kDq; ++q)
                        if ((i + q) % C::kXSubs == 0 && i + q < count)
                            ok = ok && mbar_wait(x_full + 8 * xs[q].stage, xs[q].parity, dead);
                    ok = ok && mbar_wait(a_full + 8 * d.stage, d.parity, dead);
                    if (G > 1) ok = ok && mbar_wait(peer_full + 8 * d.stage, d.parity, dead);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int q = 0; q < C::kDq; ++q) {
                            if (i + q >= count) break;
                            const uint64_t desc = desc0 + (xs[q].stage * C::kX >> 4) + ((i + q) % C::kXSubs * C::kXTile >> 4);
                            const uint32_t at = a_tmem + (d.stage * C::kDq + q) * kACols;
#pragma unroll
                            for (int c = 0; c < kSubCols / 16; ++c)
                                tc_mma_bf16<G>(acc, at + c * 8, desc + c * 2, idesc, k > first || i + q + c > 0);
                            if ((i + q) % C::kXSubs == C::kXSubs - 1) tc_commit<G>(x_empty + 8 * xs[q].stage);
                        }
                        tc_commit<G>(a_empty + 8 * d.stage);
                        if (C::kXSubs > 1 && i + C::kDq >= count && count % C::kXSubs != 0)
                            tc_commit<G>(x_empty + 8 * x.stage);
                    }
                    __syncwarp();
                    d.next();
                }
                if (C::kXSubs > 1 && count % C::kXSubs != 0) x.next();     // a ragged step ends its stage
            }
            if (ok && elect_one()) tc_commit<G>(acc_full + 8 * ac.stage);
            __syncwarp();
        }
        await_empty(ac, acc_empty, dead);
        if (__any_sync(~0u, *dead)) {
            if (elect_one()) tc_commit<G>(drain);
            mbar_drain(drain, 0);
        }
    } else if (warp >= 4 && warp < 4 + 4 * C::kDq) {
        const int group = (warp - 4) / 4, quarter = warp % 4, row = quarter * 32 + lane;
        // Each group decodes one sub-step of every set, or none of the last one
        // of a ragged step, and waits and signals either way: a group that
        // skipped a set could take a later phase of its barriers for this one.
        const uint32_t lane_base = smem_u32(table) + 4 * lane;
        if (C::kTable) {                                   // filled while the first copies are on their way
            for (int b = warp - 4; b < 256; b += 4 * C::kDq)
                *reinterpret_cast<uint32_t*>(table + 256 * b + 4 * lane) = table_entry(b);
            asm volatile("bar.sync 7, %0;" ::"n"(4 * C::kDq * 32) : "memory");
        }
        Ring<C::kWStages> w;
        Ring<C::kADepth> d;
        bool ok = true;
        for (int64_t t = first_tile; ok && t < tiles; t += tile_step) {
            for (int k = k0; ok && k < k1; ++k, w.next()) {
                if (!(ok = mbar_wait(w_full + 8 * w.stage, w.parity, dead))) break;
                const uint8_t* codes = w_ring + w.stage * C::kWStage + row * 128;
                const uint8_t* scales = w_ring + w.stage * C::kWStage + C::kW + lane * 16 + quarter * 4;
                const int n = subs(k);
                for (int i = group; i < (n + C::kDq - 1) / C::kDq * C::kDq; i += C::kDq, d.next()) {
                    uint32_t v[32];
                    if (i < n) {
                        const uint4 c0 = *reinterpret_cast<const uint4*>(codes + ((2 * i) ^ (row & 7)) * 16);
                        const uint4 c1 = *reinterpret_cast<const uint4*>(codes + ((2 * i + 1) ^ (row & 7)) * 16);
                        const uint32_t sc = *reinterpret_cast<const uint32_t*>(scales + (MX ? i / 2 : i) * 512);
                        const uint32_t c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
                        if (MX)
                            decode_mxfp4<C::kTable>(c, sc >> (16 * (i & 1)), lane_base, v);
                        else
                            decode_nvfp4<C::kTable>(c, sc, lane_base, v);
                    }
                    if (!(ok = mbar_wait(a_empty + 8 * d.stage, d.parity ^ 1, dead))) break;
                    if (i < n) {
                        tc_fence_after();
                        tmem_store(a_tmem + (d.stage * C::kDq + group) * kACols + ((uint32_t)quarter << 21), v);
                        tc_fence_before();
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(a_full + 8 * d.stage);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(w_empty + 8 * w.stage);
            }
        }
    } else if (warp >= 4 + 4 * C::kDq) {
        const int e = (warp - 4 - 4 * C::kDq) / 4;
        if (G == 1 && cluster) cluster_wait();
        Ring<C::kAccs> ac;
        uint32_t parity = 0;
        bool ok = true;
        for (int64_t t = first_tile; ok && t < tiles; t += tile_step, ac.next(), parity ^= 1) {
            const Tile tl = my_tile(t);
            const Scale S = scale_of(MX ? 4.f : a.w_S[tl.group] * 128.f);       // the decoded weights are scaled down
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
            if (k1 - k0 > run) {
                float* mine = part + e * (C::kPart / 4);
                for (int k = k0; ok && k < k1; k += run) {
                    if (k > k0) ac.next();
                    ok = mbar_wait_long(acc_full + 8 * ac.stage, ac.parity, dead);
                    tc_fence_after();
                    if (ok) add_to_part<C::kEpi>(tmem + ac.stage * BN, tl.rows, mine, e, k > k0);
                    release(ac.stage);
                }
                if (ok) finish_part<T, C::kEpi>(a, tl, S, mine, e);
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
    if (G == 1 && cluster && warp < 4 + 4 * C::kDq) cluster_wait();
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

template <bool MX, int BN, typename T, bool RUNS = sizeof(T) == 4 && BN <= 128>
static cudaError_t launch_one(const Product& p, TileArgs& a, const TileShape& shape, cudaStream_t s)
{
    using C = Config<BN, T, RUNS>;
    auto kernel = linear_kernel<MX, BN, T, RUNS>;
    CUtensorMap w_map, x_map;
    cudaError_t e = byte_tile_map(&w_map, p.w, p.n * p.groups, p.k / 2, 128);
    if (e == cudaSuccess) e = byte_tile_map(&x_map, p.x, p.m, p.k * 2, shape.tokens / C::kPair);
    if (e != cudaSuccess) return e;
    static Residency residency;
    const int per_sm = product_blocks_per_sm(residency, reinterpret_cast<const void*>(kernel), C::kThreads, C::kSmem);
    return launch_tiles(kernel, w_map, x_map, p, a, shape, C::kPair, per_sm, C::kThreads, C::kSmem, s);
}

template <bool MX, typename T> static cudaError_t launch_shape(const Product& p, cudaStream_t s)
{
    TileArgs a = tile_args(p, kStepCols, MX ? 128 : 64);
    const TileShape shape = tile_shape(p, a.k_steps, 2, {kRun<T>, p.out_bf16 ? 64 : 128, false});
    if (p.out_bf16 && a.k_steps > kRun<T> && shape.split == 1) return launch_one<MX, 64, T, true>(p, a, shape, s);
    if (shape.tokens <= 16) return launch_one<MX, 16, T>(p, a, shape, s);
    if (shape.tokens <= 32) return launch_one<MX, 32, T>(p, a, shape, s);
    if (shape.tokens <= 64) return launch_one<MX, 64, T>(p, a, shape, s);
    if (shape.tokens <= 128) return launch_one<MX, 128, T>(p, a, shape, s);
    return launch_one<MX, 192, T>(p, a, shape, s);
}

cudaError_t launch_linear(const Product& p, cudaStream_t s)
{
    if (p.mx) return p.out_bf16 ? launch_shape<true, __nv_bfloat16>(p, s) : launch_shape<true, float>(p, s);
    return p.out_bf16 ? launch_shape<false, __nv_bfloat16>(p, s) : launch_shape<false, float>(p, s);
}

}  // namespace fp4q
