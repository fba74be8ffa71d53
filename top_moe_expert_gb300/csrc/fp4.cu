// fp4.cu -- NVFP4 and MXFP4 quantization of rows, and the values back.
//
// Per block of B consecutive elements of a row (NVFP4: B = 16, MXFP4: B =
// 32), amax = max |v|:
//   NVFP4: S = UE4M3(binary32(amax * binary32(1 / (6 alpha)))), the nearest
//     value (ties to even), at most 448; code_i = E2M1(binary32(v_i *
//     binary32(1 / binary32(alpha S)))), all magnitudes 0 where S = 0.  The
//     decisions are those of the paired-sparse NVFP4 path's activation
//     quantizer, on 16-element blocks.
//   MXFP4: X = floor(log2 amax) - 2 (2 = emax of E2M1) clamped to [-127,
//     127], amax = 0 giving -127; code_i = E2M1(v_i 2^-X).  v 2^-X is exact
//     in FP32 for every value that can round to a non-zero code.
// E2M1 rounds to nearest, ties to even, at most 6, the sign kept.  A block
// that holds a NaN or an infinity gets the scale NaN (0x7F / 0xFF) and zero
// codes, so it reads back, and multiplies, as NaN.
#include "common.cuh"
#include "fp4.cuh"
#include "gmm_common.cuh"

namespace moe {
namespace fp4 {

// Every thread takes 32 consecutive elements of a row (one block of MXFP4, two
// of NVFP4) with 16-byte loads, keeps them in registers and writes their 16
// bytes of codes at once; a warp reads 2 or 4 KB in one go.  Both kernels are
// streams: the conversions are a few instructions per element (packed cvt),
// less than the memory time of the 16-bit types.
template <typename VT>
struct Vec32 {
    static constexpr int kWords = sizeof(VT) * 32 / 16;
    uint4 w[kWords];
};

__device__ __forceinline__ void unpack(const Vec32<float> &v, float (&x)[32])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[4 * i] = __uint_as_float(v.w[i].x);
        x[4 * i + 1] = __uint_as_float(v.w[i].y);
        x[4 * i + 2] = __uint_as_float(v.w[i].z);
        x[4 * i + 3] = __uint_as_float(v.w[i].w);
    }
}

template <typename VT>
__device__ __forceinline__ void unpack(const Vec32<VT> &v, float (&x)[32])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w[4] = {v.w[i].x, v.w[i].y, v.w[i].z, v.w[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (std::is_same<VT, __half>::value)
                f16x2_to_float(w[j], x[8 * i + 2 * j], x[8 * i + 2 * j + 1]);
            else
                bf16x2_to_float(w[j], x[8 * i + 2 * j], x[8 * i + 2 * j + 1]);
        }
    }
}

// The largest magnitude's bits of B values.
template <int B>
__device__ __forceinline__ uint32_t amax_bits(const float *x)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < B; ++i)
        m = max(m, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    return m;
}

// 8 values onto the E2M1 grid: one 32-bit word of codes.
__device__ __forceinline__ uint32_t codes8(const float *x, float inv)
{
    uint32_t r;
    asm("{\n .reg .b8 a, b, c, d;\n"
        " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
        " mov.b32 %0, {a, b, c, d};\n}"
        : "=r"(r)
        : "f"(x[0] * inv), "f"(x[1] * inv), "f"(x[2] * inv), "f"(x[3] * inv), "f"(x[4] * inv), "f"(x[5] * inv),
          "f"(x[6] * inv), "f"(x[7] * inv));
    return r;
}

template <typename VT, int FMT>
__global__ void __launch_bounds__(256)
quantize_kernel(const VT *__restrict__ v, int64_t rows, int nq, int Ks, const float *__restrict__ alpha,
                int64_t rows_per_alpha, uint4 *__restrict__ q, uint8_t *__restrict__ s)
{
    // nq 32-element pieces in a row; the row's scale bytes past its blocks are
    // zeroed by the threads past them
    constexpr int kPer = 32 / block_of(FMT);              // scale bytes of a piece
    const int np = Ks / kPer;
    for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < rows * np;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t r = i / np;
        const int c = static_cast<int>(i - r * np);
        uint32_t bytes = 0;
        if (c < nq) {
            Vec32<VT> in;
            const uint4 *p = reinterpret_cast<const uint4 *>(v) + (r * nq + c) * Vec32<VT>::kWords;
#pragma unroll
            for (int k = 0; k < Vec32<VT>::kWords; ++k)
                in.w[k] = ld_stream_u4(p + k);
            float x[32];
            unpack(in, x);
            uint32_t w[4];
            if constexpr (FMT == MOE_FP4_NVFP4) {
                const float a = __ldg(alpha + r / rows_per_alpha), g = 1.0f / (6.0f * a);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float inv;
                    const uint32_t b = block_scale_nv(amax_bits<16>(x + 16 * h), a, g, inv);
                    bytes |= b << (8 * h);
                    w[2 * h] = b == 0x7Fu ? 0u : codes8(x + 16 * h, inv);
                    w[2 * h + 1] = b == 0x7Fu ? 0u : codes8(x + 16 * h + 8, inv);
                }
            } else {
                float inv;
                bytes = block_scale_mx(amax_bits<32>(x), inv);
#pragma unroll
                for (int h = 0; h < 4; ++h)
                    w[h] = bytes == 0xFFu ? 0u : codes8(x + 8 * h, inv);
            }
            q[r * nq + c] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if constexpr (kPer == 2)
            reinterpret_cast<uint16_t *>(s)[i] = static_cast<uint16_t>(bytes);
        else
            s[i] = static_cast<uint8_t>(bytes);
    }
}

template <typename VT, int FMT>
__global__ void __launch_bounds__(256)
dequantize_kernel(const uint4 *__restrict__ q, const uint8_t *__restrict__ s, int64_t rows, int nq, int Ks,
                  const float *__restrict__ alpha, int64_t rows_per_alpha, VT *__restrict__ v)
{
    constexpr int kPer = 32 / block_of(FMT);
    for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < rows * nq;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t r = i / nq;
        const int c = static_cast<int>(i - r * nq);
        const uint4 in = ld_stream_u4(q + i);
        const uint32_t w[4] = {in.x, in.y, in.z, in.w};
        const float a = FMT == MOE_FP4_NVFP4 ? __ldg(alpha + r / rows_per_alpha) : 1.f;
        float f[kPer];
        if constexpr (kPer == 2) {
            const uint32_t b = reinterpret_cast<const uint16_t *>(s + r * Ks)[c];
            f[0] = ue4m3_value(b & 0xFFu);
            f[1] = ue4m3_value(b >> 8);
        } else {
            f[0] = scale_value<FMT>(s[r * Ks + c]);
        }
        uint4 *o = reinterpret_cast<uint4 *>(v) + i * Vec32<VT>::kWords;
#pragma unroll
        for (int h = 0; h < 4; ++h) {                       // 8 elements, a word of codes
            float x[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 e = e2m1_values((w[h] >> (8 * j)) & 0xFFu);
                x[2 * j] = e.x * f[h * kPer / 4] * a;
                x[2 * j + 1] = e.y * f[h * kPer / 4] * a;
            }
            if constexpr (sizeof(VT) == 4) {
                o[2 * h] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
                o[2 * h + 1] = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
            } else {
                o[h] = make_uint4(gmm::pack2<VT>(x[0], x[1]), gmm::pack2<VT>(x[2], x[3]), gmm::pack2<VT>(x[4], x[5]),
                                  gmm::pack2<VT>(x[6], x[7]));
            }
        }
    }
}

constexpr int64_t kMostBlocks = 152 * 64;

template <typename F>
static bool by_type(int32_t dt, F f)
{
    switch (dt) {
    case MOE_FP32: f(float{}); return true;
    case MOE_BF16: f(__nv_bfloat16{}); return true;
    case MOE_FP16: f(__half{}); return true;
    }
    return false;
}

static moe_status_t check(const void *v, int32_t vdt, int64_t rows, int32_t K, int32_t fmt, const float *alpha,
                          int64_t groups, const uint8_t *q, const uint8_t *s)
{
    if (rows < 0 || K <= 0 || groups < 1 || rows % groups != 0)
        return MOE_ERR_INVALID_ARG;
    if (fmt != MOE_FP4_NVFP4 && fmt != MOE_FP4_MXFP4)
        return MOE_ERR_UNSUPPORTED;
    if (K % 32 != 0)
        return MOE_ERR_INVALID_ARG;
    if (vdt != MOE_FP32 && vdt != MOE_BF16 && vdt != MOE_FP16)
        return MOE_ERR_UNSUPPORTED;
    if ((fmt == MOE_FP4_NVFP4) != (alpha != nullptr) && rows)
        return MOE_ERR_INVALID_ARG;
    if (rows && (!v || !q || !s || !aligned(v, 16) || !aligned(q, 16) || !aligned(s, 16)))
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

}  // namespace fp4
}  // namespace moe

using namespace moe;
using namespace moe::fp4;

MOE_API moe_status_t moe_fp4_scale_cols(int32_t K, int32_t fmt, int32_t *cols)
{
    if (K <= 0 || K % 32 != 0 || !cols)
        return MOE_ERR_INVALID_ARG;
    if (fmt != MOE_FP4_NVFP4 && fmt != MOE_FP4_MXFP4)
        return MOE_ERR_UNSUPPORTED;
    *cols = scale_cols(K, fmt);
    return MOE_OK;
}

MOE_API moe_status_t moe_fp4_quantize(const void *v, int32_t vdt, int64_t rows, int32_t K, int32_t fmt,
                                      const float *alpha, int64_t groups, uint8_t *q, uint8_t *s, void *stream)
{
    const moe_status_t st = check(v, vdt, rows, K, fmt, alpha, groups, q, s);
    if (st != MOE_OK || rows == 0)
        return st;
    const int Ks = scale_cols(K, fmt), np = Ks * block_of(fmt) / 32;
    const int64_t blocks = (rows * np + 255) / 256;
    const int grid = static_cast<int>(blocks < kMostBlocks ? blocks : kMostBlocks);
    by_type(vdt, [&](auto t) {
        using T = decltype(t);
        auto k = fmt == MOE_FP4_NVFP4 ? quantize_kernel<T, MOE_FP4_NVFP4> : quantize_kernel<T, MOE_FP4_MXFP4>;
        k<<<grid, 256, 0, as_stream(stream)>>>(static_cast<const T *>(v), rows, K / 32, Ks, alpha, rows / groups,
                                               reinterpret_cast<uint4 *>(q), s);
    });
    return launch_status();
}

MOE_API moe_status_t moe_fp4_dequantize(const uint8_t *q, const uint8_t *s, int64_t rows, int32_t K, int32_t fmt,
                                        const float *alpha, int64_t groups, void *v, int32_t vdt, void *stream)
{
    const moe_status_t st = check(v, vdt, rows, K, fmt, alpha, groups, q, s);
    if (st != MOE_OK || rows == 0)
        return st;
    const int Ks = scale_cols(K, fmt);
    const int64_t blocks = (rows * (K / 32) + 255) / 256;
    const int grid = static_cast<int>(blocks < kMostBlocks ? blocks : kMostBlocks);
    by_type(vdt, [&](auto t) {
        using T = decltype(t);
        auto k = fmt == MOE_FP4_NVFP4 ? dequantize_kernel<T, MOE_FP4_NVFP4> : dequantize_kernel<T, MOE_FP4_MXFP4>;
        k<<<grid, 256, 0, as_stream(stream)>>>(reinterpret_cast<const uint4 *>(q), s, rows, K / 32, Ks, alpha,
                                               rows / groups, static_cast<T *>(v));
    });
    return launch_status();
}
