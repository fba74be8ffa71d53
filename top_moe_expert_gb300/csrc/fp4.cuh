// fp4.cuh -- NVFP4 / MXFP4 element and scale conversions.
#pragma once

#include "common.cuh"

namespace moe {
namespace fp4 {

// Elements that share a scale, and scale bytes of a row of K: K / block,
// rounded up to whole 16-byte words so that every row starts aligned.
__host__ __device__ constexpr int block_of(int fmt) { return fmt == MOE_FP4_NVFP4 ? 16 : 32; }
__host__ __device__ constexpr int scale_cols(int K, int fmt) { return (K / block_of(fmt) + 15) / 16 * 16; }

// 16-byte load of data that is read once.  Not of the non-coherent kind, here and
// in the other kernels that start before their predecessor on the stream has
// ended: what they read may be what it wrote.
__device__ __forceinline__ uint4 ld_once_u4(const void *p)
{
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }

// UE4M3 byte of a non-negative value: nearest, ties to even, at most 448.
__device__ __forceinline__ uint32_t to_ue4m3(float v)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(v));
    return r & 0x7Fu;
}

__device__ __forceinline__ float ue4m3_value(uint32_t b)
{
    return __half2float(__low2half(e4m3x2_to_half2(static_cast<uint16_t>(b))));
}

// The two values of a byte of codes, low nibble first (exact).
__device__ __forceinline__ float2 e2m1_values(uint32_t b)
{
    uint32_t r;
    asm("{\n .reg .b8 b, z;\n mov.b16 {b, z}, %1;\n cvt.rn.f16x2.e2m1x2 %0, b;\n}"
        : "=r"(r) : "h"(static_cast<uint16_t>(b)));
    return __half22float2(*reinterpret_cast<__half2 *>(&r));
}

// Scale byte of a block from the bits of its amax; inv is the factor that
// takes a value onto the E2M1 grid.  NVFP4: g = 1 / (6 alpha).
__device__ __forceinline__ uint32_t block_scale_nv(uint32_t amax, float alpha, float g, float &inv)
{
    inv = 0.f;
    if (amax >= 0x7F800000u)
        return 0x7Fu;
    const uint32_t b = amax ? to_ue4m3(__uint_as_float(amax) * g) : 0u;
    if (b)
        inv = 1.0f / (alpha * ue4m3_value(b));
    return b;
}

__device__ __forceinline__ uint32_t block_scale_mx(uint32_t amax, float &inv)
{
    inv = 0.f;
    if (amax >= 0x7F800000u)
        return 0xFFu;
    const int ef = static_cast<int>(amax >> 23);
    const int X = ef == 0 ? -127 : max(ef - 129, -127);       // at most 125
    inv = __uint_as_float(static_cast<uint32_t>(127 - X) << 23);
    return static_cast<uint32_t>(X + 127);
}

// The product a * b of two constants as two factors to apply one after the
// other, v * f * g: each may lie anywhere in 2^-100 .. 2^100, where a * b alone
// can leave FP32 while v * a * b does not.  f carries the significands and half
// of the exponent, g the other half, a power of two.  For v of a product of codes
// (0, or 2^-20 .. 2^60) neither f, g nor v * f is subnormal, and v * f overflows
// only where the result does, so that the roundings are those of a * b and of its
// product with v, with one more where the result itself is subnormal.
__host__ __device__ __forceinline__ void factors(float a, float b, float &f, float &g)
{
    const int ia = ilogbf(a), ib = ilogbf(b);           // of 0, infinity and NaN far outside the limits
    const int ea = ia < -100 ? -100 : ia > 100 ? 100 : ia, eb = ib < -100 ? -100 : ib > 100 ? 100 : ib;
    const int half = (ea + eb) / 2;
    f = ldexpf(ldexpf(a, -ea) * ldexpf(b, -eb), half);
    g = ldexpf(1.f, ea + eb - half);
}

template <int FMT>
__device__ __forceinline__ float scale_value(uint32_t b)
{
    if constexpr (FMT == MOE_FP4_NVFP4)
        return ue4m3_value(b);
    else
        return b == 0xFFu ? __uint_as_float(0x7FC00000u) : e8m0_to_float(b);
}

}  // namespace fp4
}  // namespace moe
