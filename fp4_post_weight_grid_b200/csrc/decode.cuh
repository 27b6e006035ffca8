// decode.cuh -- FP4 weights as bf16 pairs, exactly.
//
// q * s of an NVFP4 element has at most 2 + 4 significant bits and q * 2^e of an
// MXFP4 element 2, so a decoded weight is a bf16 value.
#pragma once

#include <cstdint>

namespace fp4q {

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

template <uint32_t kSel> __device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "n"(kSel));
    return r;
}

// Eight codes -> four pairs of bf16 in column order, each q * 2^-126 times its
// half of `scale`.  Where bf16 keeps the low exponent bits and the first
// mantissa bit (8..6), the three magnitude bits of a code are its value under
// an exponent bias of 127 instead of 1 (the code 1/2 becomes a subnormal,
// which the multiplication takes exactly); the sign goes to bit 15.  A pair's
// nibbles come to bits 3..0 of the two halves (the permutation's sign mode
// gives the zero bytes between them), one integer multiplication by 2^6 + 2^12
// puts both copies of each in place, and a mask keeps the bits wanted: two
// operations of the ALU pipe a pair, which is what bounds the decoding, where
// shifting and merging took four (212 -> 125 ALU instructions per warp and step).
template <int J> __device__ __forceinline__ uint32_t decode2(uint32_t lo, uint32_t hi, uint32_t scale)
{
    const uint32_t p = prmt<J | (J | 8) << 4 | (4 + J) << 8 | (12 + J) << 12>(lo, hi);
    return mul_bf16x2((p * 0x1040u) & 0x81C081C0u, scale);
}
__device__ __forceinline__ void decode8(uint32_t w, uint32_t scale, uint32_t* out)
{
    const uint32_t lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;
    out[0] = decode2<0>(lo, hi, scale);
    out[1] = decode2<1>(lo, hi, scale);
    out[2] = decode2<2>(lo, hi, scale);
    out[3] = decode2<3>(lo, hi, scale);
}

// Half 0 or 1 of a pair of factors, in both halves.
__device__ __forceinline__ uint32_t one_factor(uint32_t f, int half)
{
    return half ? prmt<0x3232>(f, 0) : prmt<0x1010>(f, 0);
}

// NVFP4: the factors of four E4M3 bytes (the blocks of 64 columns), two pairs.
// The decoded weight is q * s * 2^-7, in range for every q and s: s * 2^119 for
// decode8, s * 2^-7 where q itself is multiplied (UNIT).  A byte in bits 10..4 of
// a half stands for s * 2^-120; two exact multiplications do the rest.
template <bool UNIT> __device__ __forceinline__ void nv_factors(uint32_t scales, uint32_t (&f)[2])
{
    const uint32_t s = scales & 0x7F7F7F7Fu;
    f[0] = prmt<0x4140>(s, 0) << 4;
    f[1] = prmt<0x4342>(s, 0) << 4;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        f[i] = mul_bf16x2(mul_bf16x2(f[i], 0x7F007F00u), UNIT ? 0x38803880u : 0x77807780u);   // 2^127, 2^-14 or 2^112
    if ((s + 0x01010101u) & 0x80808080u) {                 // a byte 0x7F is a NaN
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (((s >> (8 * i)) & 0x7F) == 0x7F) f[i / 2] |= 0x7FFFu << (16 * (i % 2));
    }
}
// MXFP4: the factors of the two E8M0 bytes in the low half of `scales`.  The
// decoded weight is q * 2^(b-129), in range up to b = 254.  decode8 takes
// 2^(b-129+126), which is up to b = 130; above, `rest` (else 0) holds what must
// still multiply the result.
__device__ __forceinline__ uint32_t mx_factors(uint32_t scales, uint32_t& rest)
{
    const uint32_t b = prmt<0x4140>(scales, 0);
    const bool large = ((b + 0x007D007Du) & 0x01000100u) != 0;         // a byte above 130
    rest = 0;
    if (large) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t e = (b >> (16 * i)) & 255;
            rest |= (e == 255 ? 0x7FC0u : (max(e, 130u) - 130 + 127) << 7) << (16 * i);
        }
    }
    return (large ? __vminu2(b, 0x00820082u) : b) * 128u + 0x3E003E00u;
}
// The same for q itself: 2^(b-129), a normal number from b = 3.
__device__ __forceinline__ uint32_t mx_factors_table(uint32_t scales)
{
    const uint32_t b = prmt<0x4140>(scales, 0);
    uint32_t f = b * 128u - 0x01000100u;
    const uint32_t odd = (b + 0x00010001u) & 0x00FC00FCu;
    if ((odd & 0xFFFFu) == 0 || odd >> 16 == 0) {          // a byte below 3 (a subnormal factor) or 255 (a NaN)
        f = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t e = (b >> (16 * i)) & 255;
            f |= (e == 255 ? 0x7FC0u : e < 3 ? 0x10u << e : (e - 2) << 7) << (16 * i);
        }
    }
    return f;
}

}  // namespace fp4q
