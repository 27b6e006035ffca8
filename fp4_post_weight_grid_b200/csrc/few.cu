// few.cu -- fp4q_linear and fp4q_linear_group for a few tokens: every weight is
// read and decoded once for at most 16 tokens, so that the product is bound by
// the weights' way from memory and, close behind, by their decoding.
//
// A warp takes 16 or 32 rows of W and every 8th stretch of 256 columns: codes
// go from global memory to registers, are decoded there in the layout of the
// first operand of mma.sync.m16n8k16, and meet the tokens' values loaded
// straight from x.  The sum over k may run in any order as long as both
// operands agree, so thread t of a quad takes columns 64t .. 64t+63 of the
// stretch: 32 contiguous bytes of codes of each of its rows, one word of scales
// and 128 contiguous bytes of its token.  Nothing is exchanged before the
// block's eight partial sums are added in shared memory: no barriers, no
// staging, and the loads of the next stretch are under way while one is decoded.
// (The tensor-memory kernel of linear.cu hands every 64 columns from copying to
// decoding to multiplying warps, and took twice as long for few tokens.)
#include "decode.cuh"
#include "product_host.cuh"

namespace fp4q {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kStretch = 256;                  // columns a warp takes at a time

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 bytes that are read once: around L1, which is left to x and the scales.
__device__ __forceinline__ uint4 ld_once(const uint8_t* p)
{
    uint4 v;
    asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
        : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// The codes and scales of a thread's part of a stretch: rows g and g + 8 of MT
// tiles of 16.
template <int MT> struct Part {
    uint4 codes[MT][2][2];
    uint32_t scales[MT][2];
};

// MT: tiles of 16 rows of W per warp; NT: tiles of 8 tokens.
template <bool MX, int MT, int NT, typename T>
__global__ void __launch_bounds__(kThreads, 2) few_kernel(const __grid_constant__ TileArgs a,
                                                          const uint8_t* __restrict__ w,
                                                          const __nv_bfloat16* __restrict__ x)
{
    constexpr int kRows = 16 * MT, kTokens = 8 * NT;
    __shared__ float sums[kWarps][kTokens][kRows + 1];
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, g = lane / 4, t = lane % 4;
    const int group = blockIdx.x / a.n_tiles;
    const int64_t row0 = (int64_t)(blockIdx.x % a.n_tiles) * kRows;
    int first = 0, last = a.m;
    if (a.offsets) {
        bool ok = true;
        for (int i = threadIdx.x; i < a.groups; i += kThreads) {
            const int lo = __ldg(a.offsets + i), hi = __ldg(a.offsets + i + 1);
            ok = ok && lo >= 0 && lo <= hi && hi <= a.m;
        }
        first = __ldg(a.offsets + group);
        last = __ldg(a.offsets + group + 1);
        if (!__syncthreads_and(ok)) {
            if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.status, FP4Q_FLAG_OFFSETS);
            return;
        }
        if (first == last) return;
    }
    const float S = MX ? 4.f : a.w_S[group] * 128.f;       // the decoded weights are scaled down
    const int stretches = (a.k + kStretch - 1) / kStretch;
    const int per_scale_tile = MX ? 128 : 64;

    // Rows past the last one repeat it; their sums are not used.
    const uint8_t* rows[MT][2];
    const uint8_t* scale_rows[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t j = min(row0 + 16 * mt + 8 * h + g, a.n - 1);
            rows[mt][h] = w + ((int64_t)group * a.n + j) * (a.k / 2) + t * 32;
            scale_rows[mt][h] = a.w_scales + group * a.w_scale_stride + j / 128 * a.w_col_tiles * 512 + j % 32 * 16 +
                                j % 128 / 32 * 4;
        }
    // Columns past the last one are zeros in both operands.
    auto load = [&](Part<MT>& p, int s) {
        const int k = s * kStretch + 64 * t;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint8_t* c = rows[mt][h] + (int64_t)s * (kStretch / 2);
                p.codes[mt][h][0] = k < a.k ? ld_once(c) : make_uint4(0, 0, 0, 0);
                p.codes[mt][h][1] = k + 32 < a.k ? ld_once(c + 16) : make_uint4(0, 0, 0, 0);
                p.scales[mt][h] =
                    k < a.k ? __ldg(reinterpret_cast<const uint32_t*>(scale_rows[mt][h] + k / per_scale_tile * 512)) : 0;
            }
    };

    for (int tok0 = first; tok0 < last; tok0 += kTokens) {
        float acc[MT][NT][4] = {};
        const __nv_bfloat16* xs[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) xs[nt] = x + (int64_t)min(tok0 + 8 * nt + g, last - 1) * a.k + 64 * t;
        Part<MT> cur, next;
        if (warp < stretches) load(cur, warp);
        for (int s = warp; s < stretches; s += kWarps) {
            if (s + kWarps < stretches) load(next, s + kWarps);
            const int k = s * kStretch + 64 * t;
            uint32_t f[MT][2][2], rest[MT][2];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    rest[mt][h] = 0;
                    if (MX)
                        f[mt][h][0] = f[mt][h][1] = mx_factors(cur.scales[mt][h] >> (16 * (t & 1)), rest[mt][h]);
                    else
                        nv_factors<false>(cur.scales[mt][h], f[mt][h]);
                }
#pragma unroll
            for (int i = 0; i < 8; ++i) {                  // 8 columns: a word of codes, 16 bytes of x
                uint4 b[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    b[nt] = k + 32 * (i / 4) < a.k
                                ? __ldg(reinterpret_cast<const uint4*>(xs[nt] + (int64_t)s * kStretch + 8 * i))
                                : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    uint32_t v[2][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint4& q = cur.codes[mt][h][i / 4];
                        const uint32_t word = i % 4 == 0 ? q.x : i % 4 == 1 ? q.y : i % 4 == 2 ? q.z : q.w;
                        const int half = MX ? i / 4 : i / 2 % 2;
                        decode8(word, one_factor(f[mt][h][MX ? 0 : i / 4], half), v[h]);
                        if (MX && rest[mt][h]) {
#pragma unroll
                            for (int q2 = 0; q2 < 4; ++q2) v[h][q2] = mul_bf16x2(v[h][q2], one_factor(rest[mt][h], half));
                        }
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma16816(acc[mt][nt], v[0][0], v[1][0], v[0][1], v[1][1], b[nt].x, b[nt].y);
                        mma16816(acc[mt][nt], v[0][2], v[1][2], v[0][3], v[1][3], b[nt].z, b[nt].w);
                    }
                }
            }
            cur = next;
        }
        // acc[0..3]: (row g, tokens 2t and 2t + 1), (row g + 8, the same)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sums[warp][8 * nt + 2 * t + i % 2][16 * mt + 8 * (i / 2) + g] = acc[mt][nt][i];
        __syncthreads();
        for (int i = threadIdx.x; i < kRows * kTokens; i += kThreads) {
            const int r = i % kRows, c = i / kRows;
            const int64_t j = row0 + r;
            if (tok0 + c >= last || j >= a.n) continue;
            float z[1] = {0.f};
#pragma unroll
            for (int q = 0; q < kWarps; ++q) z[0] += sums[q][c][r];
            z[0] *= S;
            if (a.ep.bias) z[0] += to_f32<T>(static_cast<const T*>(a.ep.bias)[group * a.n + j]);
            activate(z, a.ep.act);
            finish_one<T>(a.ep, z[0], (int64_t)(tok0 + c) * a.n + j);
        }
        __syncthreads();
    }
}

template <bool MX, int MT, int NT, typename T>
cudaError_t launch_one(const Product& p, TileArgs& a, cudaStream_t s)
{
    a.n_tiles = (int)((p.n + 16 * MT - 1) / (16 * MT));
    few_kernel<MX, MT, NT, T><<<(unsigned)((int64_t)a.n_tiles * p.groups), kThreads, 0, s>>>(
        a, p.w, static_cast<const __nv_bfloat16*>(p.x));
    return cudaGetLastError();
}

template <bool MX, typename T> cudaError_t launch_shape(const Product& p, cudaStream_t s)
{
    TileArgs a = tile_args(p, kStretch, MX ? 128 : 64);
    const bool two = p.m > 8 * (int64_t)p.groups;
    // 32 rows a warp halve the reads of x; 16 where 32 would leave less than two blocks for an SM.
    if ((p.n + 31) / 32 * std::min<int64_t>(p.groups, p.m) >= 2 * sm_count())
        return two ? launch_one<MX, 2, 2, T>(p, a, s) : launch_one<MX, 2, 1, T>(p, a, s);
    return two ? launch_one<MX, 1, 2, T>(p, a, s) : launch_one<MX, 1, 1, T>(p, a, s);
}

}  // namespace

bool few_tokens(const Product& p)
{
    return p.offsets ? p.m <= 64 && p.m <= 16 * (int64_t)p.groups : p.m <= 16;
}

cudaError_t launch_few(const Product& p, cudaStream_t s)
{
    if (p.mx) return p.out_bf16 ? launch_shape<true, __nv_bfloat16>(p, s) : launch_shape<true, float>(p, s);
    return p.out_bf16 ? launch_shape<false, __nv_bfloat16>(p, s) : launch_shape<false, float>(p, s);
}

}  // namespace fp4q
