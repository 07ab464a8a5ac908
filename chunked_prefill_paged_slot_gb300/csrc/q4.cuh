// q4.cuh -- the 4-bit cache's numbers: what its writer and its readers share.
//
// A number is code * scale, one scale for every 16 columns of a place and head. Codes are
// e2m1 (sign; 0, 0.5, 1, 1.5, 2, 3, 4, 6), two to a byte, the even column in the low half.
// Scale bytes have 5 bits of exponent and 3 of mantissa and no sign: byte << 7 are the
// bits of the f16 number that it stands for, 2^-17 to 61440 (248 is infinity, above NaN).
// Why this and not e4m3 scales: decoding is a shift, the exponent reaches down to 2^-17
// (e4m3's 2^-9 needs another scale per tensor beside it), and with scales of at most 10240,
// which is what the writer stores, every number is exact in f16 (2 significant bits times
// 4, a multiple of 2^-18 below 61440) and in bf16: readers need no common exponents.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace cpsa {

constexpr int kQ4Group = 16;              // columns that share a scale
constexpr uint32_t kQ4NanScale = 255;
constexpr float kQ4MinScale = 0x1p-17f, kQ4MaxScale = 10240.f;

// Largest magnitude of eight numbers, as its bits: those of a NaN are above infinity's, and
// these above any finite number's.
__device__ __forceinline__ uint32_t q4_amax(const float (&x)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
    return m;
}

// The scale of a group: amax / 6 rounded to the nearest scale (ties to even), and its
// reciprocal in two parts. A quotient a / b by a two-part reciprocal, fma(a, hi, a * lo),
// is off by some 2^-47 of itself before its one rounding to fp32. So where it is a tie
// between two numbers of few bits (often: bf16 numbers over scales of 4 bits) it comes out
// as that tie, and elsewhere on the right side of it: for such a tie t, t * b has few bits
// too, so an fp32 a other than t * b is at least 2^-24 of itself away.
struct Q4Scale {
    float hi, lo;
    uint32_t byte;
    __device__ __forceinline__ explicit Q4Scale(uint32_t amax_bits)
    {
        constexpr float s_hi = (float)(1.0 / 6.0), s_lo = (float)(1.0 / 6.0 - (double)s_hi);
        const float amax = __uint_as_float(amax_bits);
        const float w = fmaf(amax, s_hi, amax * s_lo);
        const uint32_t b = __float_as_uint(w);
        float f = __uint_as_float((b + 0x7ffffu + ((b >> 20) & 1u)) & 0xfff00000u);
        if (w < 0x1p-14f)
            f = rintf(w * 0x1p17f) * 0x1p-17f;
        f = fminf(fmaxf(f, kQ4MinScale), kQ4MaxScale);
        hi = __frcp_rn(f);
        lo = fmaf(-hi, f, 1.f) * hi;
        byte = amax_bits >= 0x7f800000u ? kQ4NanScale : (uint32_t)__half_as_ushort(__float2half_rn(f)) >> 7;
    }
};

// The codes of eight columns: x / scale to the nearest (ties to even), at most 6 in size.
__device__ __forceinline__ uint32_t q4_codes(const float (&x)[8], const Q4Scale &f)
{
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = fmaf(x[i], f.hi, x[i] * f.lo);
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
    return r;
}

// The four code pairs of a word as f16 pairs (without their scale); exact.
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t (&r)[4])
{
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(w));
}

__device__ __forceinline__ uint32_t lds_u16(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}

// A scale byte as an f16 pair.
__device__ __forceinline__ uint32_t q4_scale2(uint32_t byte) { return byte * 0x00800080u; }

__device__ __forceinline__ uint32_t q4_mul(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Eight columns of one group as bf16.
__device__ __forceinline__ uint4 q4_bf16x8(uint32_t codes, uint32_t scale_byte)
{
    const uint32_t f = q4_scale2(scale_byte);
    uint32_t h[4], o[4];
    e2m1x8(codes, h);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t x = q4_mul(h[i], f);
        const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&x));
        o[i] = pack_bf16x2(y.x, y.y);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace cpsa
