// product_epilogue.cuh -- the element-wise end of the products on FP4 weights:
// y = act(acc * S + bias) * mul + residual, each operation rounded in binary32
// and the result once to the output dtype.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "fp4q.h"

namespace fp4q {

struct EpilogueArgs {
    const void* bias;             // [groups][n]
    const void* mul;              // [m][n]
    const void* residual;         // [m][n]
    void* y;                      // [m][n]
    int act;
};

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// The GELUs in the forms without cancellation for negative z: Phi(z) =
// erfc(-z/sqrt 2)/2, and 1 + tanh(u) = 2/(1 + exp(-2u)).  A NaN stays a NaN
// in every one of them.
__device__ __forceinline__ float activate(float z, int act)
{
    switch (act) {
    case FP4Q_ACT_RELU:
        return z < 0.f ? 0.f : z;
    case FP4Q_ACT_GELU:
        return 0.5f * z * erfcf(z * -0.70710678f);
    case FP4Q_ACT_GELU_TANH:
        return z / (1.f + expf(-1.59576912f * (z + 0.044715f * z * z * z)));
    case FP4Q_ACT_SILU:
        return z / (1.f + expf(-z));
    default:
        return z;
    }
}

// One output element.  mul and residual may alias y: the element is read by
// the thread that then writes it.
template <typename T>
__device__ __forceinline__ void finish(const EpilogueArgs& e, float acc, float S, float bias, bool has_bias, int64_t at)
{
    float z = acc * S;
    if (has_bias) z += bias;
    z = activate(z, e.act);
    if (e.mul) z *= to_f32<T>(static_cast<const T*>(e.mul)[at]);
    if (e.residual) z += to_f32<T>(static_cast<const T*>(e.residual)[at]);
    static_cast<T*>(e.y)[at] = from_f32<T>(z);
}

}  // namespace fp4q
