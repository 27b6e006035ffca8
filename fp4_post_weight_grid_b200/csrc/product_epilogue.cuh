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

// The factor S of the sums.  The product of two global scales of the quantizers
// (2^-76 and up each) need not be a normal number; sums then take one after the
// other, which are.
struct Scale {
    float first, second;
    __device__ __forceinline__ float operator()(float z) const { return z * first * second; }
};
__device__ __forceinline__ Scale scale_of(float s) { return {s, 1.f}; }
__device__ __forceinline__ Scale scale_of(float w, float x)
{
    const float s = w * x;
    return fabsf(s) >= 1.17549435e-38f && fabsf(s) <= 3.40282347e38f ? Scale{s, 1.f} : Scale{w, x};
}

// Outputs that one thread finishes together: 16 bytes of y.
template <typename T> struct Lanes {
    static constexpr int kCount = 16 / sizeof(T);
};

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

__device__ __forceinline__ void unpack16(const uint4& u, float (&v)[4])
{
    v[0] = __uint_as_float(u.x);
    v[1] = __uint_as_float(u.y);
    v[2] = __uint_as_float(u.z);
    v[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ void unpack16(const uint4& u, float (&v)[8])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ uint4 pack16(const float (&v)[4])
{
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
__device__ __forceinline__ uint4 pack16(const float (&v)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// z * Phi(z) from the rational approximation of erfc by Abramowitz and Stegun,
// "Handbook of Mathematical Functions", 7.1.26 (absolute error 1.5e-7, a step
// of binary32 near 1): with x = |z|/sqrt 2, t = 1/(1 + p x), Phi(-|z|) =
// (a1 t + .. + a5 t^5) exp(-x^2) / 2, so that neither sign of z cancels.  The
// result is off by 2.1e-7 at most, by 3e-7 of it for |z| < 1; as the fit's error
// falls more slowly than the tail, by 5e-5 of it at z = -3 and 1.6e-3 at -5 (about
// half a step of bf16).
__device__ __forceinline__ float gelu(float z)
{
    const float x = fabsf(z) * 0.70710678f, t = __fdividef(1.f, 1.f + 0.3275911f * x);
    float p = 1.061405429f;
    p = p * t - 1.453152027f;
    p = p * t + 1.421413741f;
    p = p * t - 0.284496736f;
    p = p * t + 0.254829592f;
    const float phi = 0.5f * p * t * __expf(-x * x);
    return z < 0.f ? z * phi : phi == 0.f ? z : z - z * phi;       // z = +inf stays +inf
}

// The tanh GELU as z / (1 + exp(-2u)), as 1 + tanh(u) = 2/(1 + exp(-2u)) and
// this form does not cancel.  The hardware exponential and division (a few
// units in the last place of binary32; the exponential's grow with its
// argument where the result vanishes) keep the activation below the cost of
// the product.  A NaN stays a NaN in every one.
template <int N> __device__ __forceinline__ void activate(float (&z)[N], int act)
{
    if (act == FP4Q_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] = __fdividef(z[i], 1.f + __expf(-z[i]));
    } else if (act == FP4Q_ACT_GELU_TANH) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            z[i] = __fdividef(z[i], 1.f + __expf(-1.59576912f * (z[i] + 0.044715f * z[i] * z[i] * z[i])));
    } else if (act == FP4Q_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] = gelu(z[i]);
    } else if (act == FP4Q_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] = z[i] < 0.f ? 0.f : z[i];
    }
}

// mul and residual of 16 bytes of y, loaded ahead of their use.  y may be
// either of them: an element is read by the thread that then writes it.
struct Extra {
    uint4 mul, residual;
};
template <typename T> __device__ __forceinline__ Extra load_extra(const EpilogueArgs& e, int64_t at)
{
    Extra x;
    if (e.mul) x.mul = *reinterpret_cast<const uint4*>(static_cast<const T*>(e.mul) + at);
    if (e.residual) x.residual = *reinterpret_cast<const uint4*>(static_cast<const T*>(e.residual) + at);
    return x;
}
// The 16 bytes of y from sums that have their bias and activation.
template <typename T, int N>
__device__ __forceinline__ void finish(const EpilogueArgs& e, float (&z)[N], const Extra& x, int64_t at)
{
    static_assert(N == Lanes<T>::kCount, "16 bytes");
    float v[N];
    if (e.mul) {
        unpack16(x.mul, v);
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] *= v[i];
    }
    if (e.residual) {
        unpack16(x.residual, v);
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] += v[i];
    }
    *reinterpret_cast<uint4*>(static_cast<T*>(e.y) + at) = pack16(z);
}
// One element, for rows that do not start on 16-byte boundaries.
template <typename T> __device__ __forceinline__ void finish_one(const EpilogueArgs& e, float z, int64_t at)
{
    if (e.mul) z *= to_f32<T>(static_cast<const T*>(e.mul)[at]);
    if (e.residual) z += to_f32<T>(static_cast<const T*>(e.residual)[at]);
    static_cast<T*>(e.y)[at] = from_f32<T>(z);
}

}  // namespace fp4q
