// product.cu -- the products on FP4 weights, y = act(S * x W^T + bias) * mul +
// residual, dense and grouped (include/fp4q.h): both operands are decoded to
// binary32 in shared memory and multiplied there.
#include "device.cuh"
#include "launch.h"
#include "product_host.cuh"

namespace fp4q {

namespace {

constexpr int kTile = 64;        // rows of x, rows of W per thread block
constexpr int kStep = 32;        // columns per shared-memory step
constexpr int kThreads = 256;    // 16 x 16 threads, 4 x 4 outputs each

// A block scale; MXFP4's is a quarter of its value, so that code 6 (a quarter
// of 2^127 times 6) stays in range too: S gives the 4 back.
__device__ __forceinline__ float scale_value(uint8_t b, bool mx)
{
    if (mx) return b == 255 ? __int_as_float(0x7FC00000) : exp2f((float)b - 129.f);
    const __nv_bfloat16 h = __ushort_as_bfloat16((unsigned short)((b & 0x7F) << 4));
    return (b & 0x7F) == 0x7F ? __int_as_float(0x7FC00000) : __bfloat162float(h) * 0x1p120f;
}

__device__ __forceinline__ float code_value(uint32_t nib)
{
    const float h[8] = {0.f, 0.5f, 1.f, 1.5f, 2.f, 3.f, 4.f, 6.f};
    return (nib & 8) ? -h[nib & 7] : h[nib & 7];
}

template <typename T>
__global__ void __launch_bounds__(kThreads) product_kernel(Product p)
{
    __shared__ float xs[kStep][kTile + 1], ws[kStep][kTile + 1];
    const int g = blockIdx.z;
    int64_t r0 = 0, r1 = p.m;
    if (p.offsets) {
        bool ok = true;
        for (int i = threadIdx.x; i <= p.groups; i += kThreads) {
            const int64_t o = p.offsets[i], before = i ? p.offsets[i - 1] : 0;
            ok = ok && o >= before && o <= p.m;
        }
        if (!__syncthreads_and(ok)) {
            if (threadIdx.x == 0) atomicOr(p.status, FP4Q_FLAG_OFFSETS);
            return;
        }
        r0 = p.offsets[g];
        r1 = p.offsets[g + 1];
    }
    const int block = p.mx ? 32 : 16;
    const int64_t scols = p.k / block, col_tiles = (scols + 3) / 4;
    const uint8_t* w = p.w + (int64_t)g * p.n * (p.k / 2);
    const uint8_t* wsc = p.w_scales + g * p.w_scale_stride;
    float S = p.mx ? (p.packed ? 16.f : 4.f) : p.w_S[g];
    if (p.packed && !p.mx) S *= *p.x_S;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    const EpilogueArgs e{p.ep.bias, p.ep.mul, p.ep.residual, p.y, (int)p.ep.act};
    for (int64_t nt = blockIdx.x; nt * kTile < p.n; nt += gridDim.x)
        for (int64_t mt = r0 + (int64_t)blockIdx.y * kTile; mt < r1; mt += (int64_t)gridDim.y * kTile) {
            float acc[4][4] = {};
            for (int64_t k0 = 0; k0 < p.k; k0 += kStep) {
                for (int i = threadIdx.x; i < kTile * kStep; i += kThreads) {
                    const int c = i % kStep, r = i / kStep;
                    const int64_t row = mt + r, col = k0 + c, j = nt * kTile + r;
                    float v = 0.f;
                    if (row < r1) {
                        if (p.packed) {
                            const uint8_t b = static_cast<const uint8_t*>(p.x)[(row * p.k + col) / 2];
                            v = code_value((col & 1) ? b >> 4 : b & 15) *
                                scale_value(p.x_scales[row * scols + col / block], p.mx);
                        } else {
                            v = __bfloat162float(static_cast<const __nv_bfloat16*>(p.x)[row * p.k + col]);
                        }
                    }
                    xs[c][r] = v;
                    v = 0.f;
                    if (j < p.n) {
                        const uint8_t b = w[(j * p.k + col) / 2];
                        const int64_t sc = col / block;
                        const uint8_t s = wsc[((j / 128) * col_tiles + sc / 4) * 512 + (j % 32) * 16 +
                                              (j % 128) / 32 * 4 + sc % 4];
                        v = code_value((col & 1) ? b >> 4 : b & 15) * scale_value(s, p.mx);
                    }
                    ws[c][r] = v;
                }
                __syncthreads();
                for (int c = 0; c < kStep; ++c)
                    for (int a = 0; a < 4; ++a)
                        for (int b = 0; b < 4; ++b)
                            acc[a][b] = __fmaf_rn(xs[c][ty + 16 * a], ws[c][tx + 16 * b], acc[a][b]);
                __syncthreads();
            }
            for (int a = 0; a < 4; ++a)
                for (int b = 0; b < 4; ++b) {
                    const int64_t row = mt + ty + 16 * a, j = nt * kTile + tx + 16 * b;
                    if (row >= r1 || j >= p.n) continue;
                    const float bias = p.ep.bias ? to_f32<T>(static_cast<const T*>(p.ep.bias)[g * p.n + j]) : 0.f;
                    finish<T>(e, acc[a][b], S, bias, p.ep.bias != nullptr, row * p.n + j);
                }
        }
}

}  // namespace

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

TileShape tile_shape(const Product& p, int n_tiles, int k_steps)
{
    const int64_t rows = p.offsets ? (p.m + p.groups - 1) / p.groups : p.m;       // of a group, on average
    const int64_t busy = p.offsets ? std::min<int64_t>(p.groups, p.m) : 1;
    const int sms = sm_count();
    TileShape t{16, 1};
    while (t.tokens < 256 && t.tokens < rows) t.tokens *= 2;
    auto tiles = [&] { return busy * ((rows + t.tokens - 1) / t.tokens) * n_tiles; };
    while (t.tokens > 32 && tiles() < sms) t.tokens /= 2;
    if (t.tokens <= 64) {
        const int64_t slots = (int64_t)sms * (t.tokens <= 32 ? 2 : 1);
        while (t.split < 8 && t.split * 2 <= k_steps && tiles() * t.split * 2 <= slots) t.split *= 2;
    }
    return t;
}

cudaError_t launch_product(const Product& p, cudaStream_t s)
{
    if (p.packed) return launch_matmul(p, s);
    const int64_t nt = (p.n + kTile - 1) / kTile, mt = (p.m + kTile - 1) / kTile;
    const dim3 grid((unsigned)(nt < 65535 ? nt : 65535), (unsigned)(mt < 1024 ? mt : 1024), (unsigned)p.groups);
    if (p.out_bf16)
        product_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(p);
    else
        product_kernel<float><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace fp4q
