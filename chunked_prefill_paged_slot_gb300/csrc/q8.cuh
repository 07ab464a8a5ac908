// q8.cuh -- device helpers of the 8-bit cache's readers: scale bytes, powers of two,
// e4m3 and bf16 to f16.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace cpsa {

// Read-only loads that stay where they are written: the compiler may move __ldg down
// to its use, behind the waits that a prefetch is meant to overlap.
__device__ __forceinline__ uint4 ldg_here(const uint4 *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

__device__ __forceinline__ int ldg_here(const int32_t *p)
{
    int v;
    asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

__device__ __forceinline__ uint32_t ldg_here(const uint8_t *p)
{
    uint32_t v;
    asm volatile("ld.global.nc.u8 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

__device__ __forceinline__ void sts128(uint32_t a, const uint4 &v)
{
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// The exponent a scale byte stands for (0 and 255, which the writer never stores, as
// their neighbours: every exponent is that of a normal fp32 number).
__device__ __forceinline__ int q8_exp(uint32_t byte) { return min(max((int)byte, 1), 254) - 127; }

// 2^x, -126 <= x <= 127
__device__ __forceinline__ float exp2i(int x) { return __uint_as_float((uint32_t)(x + 127) << 23); }

// Two e4m3 bytes (the low or the high half of w) as an f16 pair; exact.
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t w)
{
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

__device__ __forceinline__ uint32_t e4m3_hi(uint32_t w)
{
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Largest finite magnitude of eight bf16 numbers. Magnitudes of one format order like
// their bits, so pairs of 16-bit integer maxima do; only where an infinity or NaN turns
// up (which sets `others`) are the finite ones sorted out one by one.
__device__ __forceinline__ float bf16x8_amax(const uint4 &v, bool &others)
{
    const uint32_t k = 0x7fff7fffu;
    const uint32_t w = __vmaxu2(__vmaxu2(v.x & k, v.y & k), __vmaxu2(v.z & k, v.w & k));
    uint32_t m = max(w & 0xffffu, w >> 16);
    if (m >= 0x7f80u) {
        others = true;
        const uint32_t x[4] = {v.x & k, v.y & k, v.z & k, v.w & k};
        m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = x[i] & 0xffffu, hi = x[i] >> 16;
            m = max(m, lo < 0x7f80u ? lo : 0u);
            m = max(m, hi < 0x7f80u ? hi : 0u);
        }
    }
    return __uint_as_float(m << 16);
}

__device__ __forceinline__ float bf16x8_amax(const uint4 &v)
{
    bool others = false;
    return bf16x8_amax(v, others);
}

// Exponent x with amax * 2^-x in [2^14, 2^15) (where the range of exp2i allows it).
__device__ __forceinline__ int q_exponent(float amax)
{
    const int e = (int)(__float_as_uint(amax) >> 23) - 127 - 14;
    return amax > 0.f ? max(e, -126) : 0;
}

// A bf16 pair times f, as an f16 pair.
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w, float f)
{
    return pack_f16x2(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xffff0000u) * f);
}

}  // namespace cpsa
