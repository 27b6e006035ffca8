// product.cu -- the products on FP4 weights, y = act(S * x W^T + bias) * mul +
// residual, dense and grouped (include/fp4q.h): tensor maps, tile shapes and
// the choice of the kernel.
#include "product_host.cuh"

namespace fp4q {

namespace {

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder, looked up once (the library is not linked to the driver).
EncodeTiled encoder()
{
    static const EncodeTiled fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeTiled>(f);
    }();
    return fn;
}

}  // namespace

cudaError_t byte_tile_map(CUtensorMap* map, const void* base, int64_t rows, int64_t row_bytes, int box_rows)
{
    const EncodeTiled encode = encoder();
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {(cuuint64_t)row_bytes, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
    const cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
    const cuuint32_t steps[2] = {1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, steps,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

int product_blocks_per_sm(Residency& r, const void* kernel, int threads, size_t smem)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return resident_blocks_per_sm(kernel, threads, smem);
    int n = r.cached[dev].load(std::memory_order_relaxed);
    if (n <= 0) {
        n = resident_blocks_per_sm(kernel, threads, smem);
        r.cached[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

TileArgs tile_args(const Product& p, int step_cols, int scale_tile_cols)
{
    TileArgs a{};
    a.offsets = p.offsets;
    a.n = p.n;
    a.m = (int)p.m;
    a.k = (int)p.k;
    a.groups = p.groups;
    a.n_tiles = (int)((p.n + 127) / 128);
    a.k_steps = (int)((p.k + step_cols - 1) / step_cols);
    a.split = 1;
    a.w_col_tiles = (int)((p.k + scale_tile_cols - 1) / scale_tile_cols);
    a.x_scales = p.x_scales;
    a.x_S = p.x_S;
    a.w_scales = p.w_scales;
    a.w_S = p.w_S;
    a.w_scale_stride = p.w_scale_stride;
    a.ep = EpilogueArgs{p.ep.bias, p.ep.mul, p.ep.residual, p.y, (int)p.ep.act};
    a.status = p.status;
    return a;
}

TileShape tile_shape(const Product& p, int k_steps, int pair, const Runs& runs)
{
    const int64_t rows = p.offsets ? (p.m + p.groups - 1) / p.groups : p.m;       // of a group, on average
    const int64_t busy = p.offsets ? std::min<int64_t>(p.groups, p.m) : 1;
    const int sms = sm_count();
    auto tiles = [&](int tokens) {
        const int features = tokens > 128 ? 128 * pair : 128;
        return busy * ((rows + tokens - 1) / tokens) * ((p.n + features - 1) / features);
    };
    // Rounds of tiles over the SMs times the length of one, whose fixed part
    // (the weight's tile, decoded or copied) weighs as much as about 160 tokens:
    // 2048 tokens x 14336 x 4096 took 242, 208 and 201 us in tiles of 128, 160 and
    // 192, FP4 x FP4 on 4096 tokens 152, 136 and 128 us.  Blocks that would idle
    // may share a tile's steps, which costs them the exchange of the partial
    // sums, about 40 tokens' worth; only while all of them run at once, as the
    // exchange is not hidden: one in every round took 16 x 4096 x 14336 to 23 us
    // from 11 us in one.
    auto cost = [&](int tokens, int split) {
        const int64_t slots = tokens > 128 ? sms / pair : sms;
        return (tiles(tokens) * split + slots - 1) / slots * (tokens + 160) / split + (split > 1 ? 40 : 0);
    };
    const int most = k_steps > runs.steps ? runs.tokens : 192;
    TileShape t{16, 1};
    int64_t best = INT64_MAX;
    for (const int tokens : {16, 32, 64, 128, 160, 192}) {
        if (tokens > most || (tokens >= 32 && tokens / 2 >= rows)) break;
        for (int split = 1; split <= 8; split *= 2) {
            if (split > 1 && (tokens > 64 || split > k_steps || tiles(tokens) * split > sms)) break;
            if (split > 1 && !runs.split && (k_steps + split - 1) / split > runs.steps) continue;
            if (cost(tokens, split) <= best) {
                best = cost(tokens, split);
                t.tokens = tokens;
                t.split = split;
            }
        }
    }
    // Groups differ: no use in counting rounds of the average one.
    if (p.offsets && rows > 128 && t.tokens > 64) t.tokens = most;
    return t;
}

cudaError_t launch_product(const Product& p, cudaStream_t s)
{
    if (p.packed) return launch_matmul(p, s);
    return few_tokens(p) ? launch_few(p, s) : launch_linear(p, s);
}

}  // namespace fp4q
