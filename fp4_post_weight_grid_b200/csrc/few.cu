// few.cu -- fp4q_linear for up to 8 tokens on a weight of moderate size, where
// what counts is how soon the weights are on their way and how little comes
// after them.
//
// A warp takes 16 rows of W and every ks-th stretch of 256 columns: codes go
// from global memory to registers, a stretch ahead, are decoded there in the
// layout of the first operand of mma.sync.m16n8k16, and meet the tokens'
// values.  The sum over k may run in any order as long as both operands agree,
// so of every 128 columns thread t of a quad takes 32t .. 32t+31: 16 contiguous
// bytes of codes of each of its two rows and 64 of its token.  x lies in shared
// memory, up to 4096 columns at a time, where 16-byte units change places so
// that the quads' reads meet different banks (read straight from L1, a read
// touched 32 lines).  The block's warps share x and, ks at a time, the rows,
// whose partial sums are added at the end; between phases of x they do not wait
// for one another, where the tensor-memory kernel of linear.cu hands every 64
// columns from copying to decoding to multiplying warps.
//
// Measured (NVFP4, us, here and there): 1024 x 4096, 1 and 8 tokens 3.9 and 5.2
// against 7.3 and 7.7; 4096 x 4096 5.5 and 6.7 against 9.4; 14336 x 4096 14.2 and
// 15.7 against 16.6 and 16.8; 4096 x 14336 15.1 and 19.8 against 16.5 and 16.9;
// 28672 x 8192 47.0 and 50.6 against 47.5.  It is bound by instructions (about
// 240 a warp for 2048 weights, 150 of them decoding, issue slots two thirds busy).
//
// The tensor core truncates where it adds, so a long sum in one accumulator
// falls short by an amount that grows with its length (by 3e-5 of it after 32768
// columns): after every 2048 columns of a warp the sums go to registers of their
// own, by additions that round, and stay within 2e-6 of the whole.  A count of
// stretches takes 1 x 4096 x 14336 from 14.8 to 15.1 us; at every end of a phase
// of x it took 15.6.
#include "decode.cuh"
#include "product_host.cuh"

namespace fp4q {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kStretch = 256;                  // columns a warp takes at a time
constexpr int kTokens = 8;
constexpr int kRun = 2048;                     // columns that one accumulator may sum
constexpr int kMostPhase = 4096;               // columns of x in shared memory: 64 KB

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 bytes that are read once: around L1.
__device__ __forceinline__ uint4 ld_once(const uint8_t* p)
{
    uint4 v;
    asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
        : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
// `bytes` 16, or 0 for zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// A thread's codes of a stretch, rows g and g + 8 and two runs of 32 columns,
// and the words that hold their scales.
template <bool MX> struct Part {
    uint4 codes[2][2];
    uint32_t words[2][2];
    // `left`: columns from the thread's first one on; past the last one there are zeros.
    __device__ __forceinline__ void load(const uint8_t* const (&row)[2], const uint8_t* const (&scales)[2], int s, int t,
                                         int left)
    {
        const int64_t tile = MX ? 2 * s : 4 * s + t / 2;
        if (left >= 160) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    codes[h][e] = ld_once(row[h] + (int64_t)s * (kStretch / 2) + 64 * e);
                    words[h][e] = __ldg(reinterpret_cast<const uint32_t*>(scales[h] + tile * 512 + (MX ? 512 : 1024) * e));
                }
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const bool in = 128 * e < left;
                    codes[h][e] = in ? ld_once(row[h] + (int64_t)s * (kStretch / 2) + 64 * e) : make_uint4(0, 0, 0, 0);
                    words[h][e] =
                        in ? __ldg(reinterpret_cast<const uint32_t*>(scales[h] + tile * 512 + (MX ? 512 : 1024) * e)) : 0;
                }
        }
    }
    // The scales of the two runs, side by side.
    __device__ __forceinline__ uint32_t scales(int h, int t) const
    {
        if (MX) return (words[h][0] >> (8 * t) & 255) | (words[h][1] >> (8 * t) & 255) << 8;
        return (words[h][0] >> (16 * (t & 1)) & 0xFFFF) | words[h][1] >> (16 * (t & 1)) << 16;
    }
};

// ODD: some factors want `rest` too (MXFP4 scales above 8).
template <bool MX, bool ODD>
__device__ __forceinline__ void multiply(float (&acc)[4], const Part<MX>& p, const uint32_t (&f)[2][2],
                                         const uint32_t (&rest)[2], uint32_t x, int g, int t)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {                          // 8 columns: a word of codes, 16 bytes of x
        uint32_t b[4];
        const int unit = (16 * (i / 4) + 4 * t + i % 4) ^ (t >> 1 | (g & 1) << 1);
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3])
                     : "r"(x + unit * 16)
                     : "memory");
        uint32_t v[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint4& q = p.codes[h][i / 4];
            const uint32_t word = i % 4 == 0 ? q.x : i % 4 == 1 ? q.y : i % 4 == 2 ? q.z : q.w;
            const int half = MX ? i / 4 : i / 2 % 2;
            decode8(word, one_factor(f[h][MX ? 0 : i / 4], half), v[h]);
            if (ODD && rest[h]) {
#pragma unroll
                for (int c = 0; c < 4; ++c) v[h][c] = mul_bf16x2(v[h][c], one_factor(rest[h], half));
            }
        }
        mma16816(acc, v[0][0], v[1][0], v[0][1], v[1][1], b[0], b[1]);
        mma16816(acc, v[0][2], v[1][2], v[0][3], v[1][3], b[2], b[3]);
    }
}

// ks warps share 16 rows, 8 / ks of which a block has.  `phase`: columns of x in
// shared memory at a time.
template <bool MX, typename T>
__global__ void __launch_bounds__(kThreads, 2)
few_kernel(const __grid_constant__ TileArgs a, const uint8_t* __restrict__ w, const __nv_bfloat16* __restrict__ x, int ks,
           int phase)
{
    constexpr int kRows = 16;
    extern __shared__ __align__(128) uint8_t raw[];
    __shared__ float sums[kWarps][kTokens][kRows + 1];
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, g = lane / 4, t = lane % 4;
    const int part = warp % ks, tiles = kWarps / ks;
    const int64_t block_row = (int64_t)blockIdx.x * (kRows * tiles), row0 = block_row + warp / ks * kRows;
    const int stretches = (a.k + kStretch - 1) / kStretch;
    const uint32_t xs = smem_u32(raw), token_bytes = 2 * phase;

    // Rows past the last one repeat it; their sums are not used.
    const uint8_t* row[2];
    const uint8_t* scale_row[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t j = min(row0 + 8 * h + g, a.n - 1);
        row[h] = w + j * (a.k / 2) + 16 * t;
        scale_row[h] = a.w_scales + j / 128 * a.w_col_tiles * 512 + j % 32 * 16 + j % 128 / 32 * 4;
    }
    float sum[4] = {}, acc[4] = {};
    int left = kRun / kStretch;
    Part<MX> next;
    if (part < stretches) next.load(row, scale_row, part, t, a.k - part * kStretch - 32 * t);
    int s = part;
    for (int k0 = 0; k0 < a.k; k0 += phase) {
        const int cols = min(phase, a.k - k0), units = cols / 8;
        const int padded = (cols + kStretch - 1) / kStretch * (kStretch / 8);      // to whole stretches, by zeros
        if (k0 > 0) __syncthreads();                       // the phase before has been read
        // Unit u of a token's 16-byte units goes to u ^ (bit 3 of u, bit 0 of the
        // token).  What lies where a token is missing goes into sums that are not used.
        for (int c = 0; c < a.m; ++c)
            for (int u = threadIdx.x; u < padded; u += kThreads)
                cp_async16(xs + c * token_bytes + (u ^ (((u >> 3) & 1) | (c & 1) << 1)) * 16,
                           x + (int64_t)c * a.k + k0 + (u < units ? 8 * u : 0), u < units ? 16 : 0);
        cp_async_wait_all();
        __syncthreads();
        for (; s * kStretch < k0 + cols; s += ks) {
            const Part<MX> cur = next;
            if (s + ks < stretches) next.load(row, scale_row, s + ks, t, a.k - (s + ks) * kStretch - 32 * t);
            uint32_t f[2][2], rest[2] = {0, 0};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (MX)
                    f[h][0] = f[h][1] = mx_factors(cur.scales(h, t), rest[h]);
                else
                    nv_factors<false>(cur.scales(h, t), f[h]);
            }
            const uint32_t at = xs + g * token_bytes + (s * kStretch - k0) * 2;
            if (MX && __any_sync(~0u, (rest[0] | rest[1]) != 0))
                multiply<MX, true>(acc, cur, f, rest, at, g, t);
            else
                multiply<MX, false>(acc, cur, f, rest, at, g, t);
            if (--left == 0) {                             // of this run
                left = kRun / kStretch;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sum[i] += acc[i];
                    acc[i] = 0.f;
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[i] += acc[i];
    // sum[0..3]: (row g, tokens 2t and 2t + 1), (row g + 8, the same)
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[warp][2 * t + i % 2][8 * (i / 2) + g] = sum[i];
    __syncthreads();
    const float S = MX ? 4.f : *a.w_S * 128.f;             // the decoded weights are scaled down
    for (int i = threadIdx.x; i < kRows * tiles * a.m; i += kThreads) {
        const int r = i % (kRows * tiles), c = i / (kRows * tiles);
        const int64_t j = block_row + r;
        if (j >= a.n) continue;
        float z[1] = {0.f};
        for (int q = 0; q < ks; ++q) z[0] += sums[r / kRows * ks + q][c][r % kRows];
        z[0] *= S;
        if (a.ep.bias) z[0] += to_f32<T>(static_cast<const T*>(a.ep.bias)[j]);
        activate(z, a.ep.act);
        finish_one<T>(a.ep, z[0], (int64_t)c * a.n + j);
    }
}

template <bool MX, typename T> cudaError_t launch_one(const Product& p, cudaStream_t s)
{
    const TileArgs a = tile_args(p, kStretch, MX ? 128 : 64);
    // As many warps to a row as leave all blocks resident at once: 4096 rows took
    // 6.3, 7.2, 11.3 and 19.2 us with 8, 4, 2 and 1, 14336 rows 22.5, 18.0, 16.1 and
    // 18.0.
    int ks = 8;
    while (ks > 1 && (p.n * ks + 127) / 128 > 2 * sm_count()) ks /= 2;
    const int phase = (int)std::min<int64_t>((p.k + kStretch - 1) / kStretch * kStretch, kMostPhase);
    static Residency residency;
    product_blocks_per_sm(residency, reinterpret_cast<const void*>(few_kernel<MX, T>), kThreads,
                          (size_t)kTokens * kMostPhase * 2);
    few_kernel<MX, T><<<(unsigned)((p.n * ks + 127) / 128), kThreads, (size_t)kTokens * phase * 2, s>>>(
        a, p.w, static_cast<const __nv_bfloat16*>(p.x), ks, phase);
    return cudaGetLastError();
}

}  // namespace

// Beyond 2^26 weights the two kernels are as fast as each other; columns over
// 8192 take so many phases of x that linear.cu's is faster from 5 tokens on.
bool few_tokens(const Product& p)
{
    return !p.offsets && p.m <= (p.k <= 8192 ? kTokens : 4) && p.n * p.k <= 1 << 26;
}

cudaError_t launch_few(const Product& p, cudaStream_t s)
{
    if (p.mx) return p.out_bf16 ? launch_one<true, __nv_bfloat16>(p, s) : launch_one<true, float>(p, s);
    return p.out_bf16 ? launch_one<false, __nv_bfloat16>(p, s) : launch_one<false, float>(p, s);
}

}  // namespace fp4q
