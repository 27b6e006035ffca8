// product.h -- what the four products on FP4 weights share on the host side:
// one problem description (a dense call is one group whose offsets pointer is
// null) and the launchers.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "fp4q.h"

namespace fp4q {

struct Product {
    bool mx;                      // MXFP4, else NVFP4
    bool packed;                  // x is FP4 (codes + row-major scales), else bf16
    const void* x;                // bf16 [m][k], or codes [m][k/2]
    const uint8_t* x_scales;      // packed: [m][k/block]
    const float* x_S;             // packed NVFP4
    const uint8_t* w;             // codes [groups][n][k/2]
    const uint8_t* w_scales;      // tiled, w_scale_stride bytes per group
    const float* w_S;             // NVFP4: [groups]
    const int32_t* offsets;       // [groups + 1], or null: one group of all m rows
    int64_t m, n, k;
    int groups;
    int64_t w_scale_stride;
    fp4q_epilogue ep;
    void* y;
    bool out_bf16;
    int32_t* status;
};

// All checks are done; m, n and groups are positive.
cudaError_t launch_product(const Product& p, cudaStream_t s);
cudaError_t launch_linear(const Product& p, cudaStream_t s);      // bf16 x
bool few_tokens(const Product& p);                                // bf16 x: whether launch_few is the faster one
cudaError_t launch_few(const Product& p, cudaStream_t s);
cudaError_t launch_matmul(const Product& p, cudaStream_t s);      // packed x

}  // namespace fp4q
