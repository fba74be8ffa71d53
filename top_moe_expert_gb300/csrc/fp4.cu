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

namespace moe {
namespace fp4 {

// One thread per block.
template <typename VT, int FMT>
__global__ void __launch_bounds__(256)
quantize_kernel(const VT *__restrict__ v, int64_t rows, int K, int Ks, const float *__restrict__ alpha,
                int64_t rows_per_alpha, uint8_t *__restrict__ q, uint8_t *__restrict__ s)
{
    constexpr int B = block_of(FMT);
    const int nb = K / B;
    for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < rows * Ks;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t r = i / Ks;
        const int b = static_cast<int>(i - r * Ks);
        if (b >= nb) {                            // the row's padding
            s[i] = 0;
            continue;
        }
        const VT *p = v + r * K + static_cast<int64_t>(b) * B;
        float x[B];
        uint32_t amax = 0;
        for (int j = 0; j < B; ++j) {
            x[j] = to_float(p[j]);
            amax = max(amax, __float_as_uint(x[j]) & 0x7FFFFFFFu);
        }
        float inv;
        const uint32_t byte = block_scale<FMT>(amax, FMT == MOE_FP4_NVFP4 ? alpha[r / rows_per_alpha] : 1.f, inv);
        uint8_t *o = q + r * (K / 2) + static_cast<int64_t>(b) * (B / 2);
        for (int j = 0; j < B / 2; ++j)
            o[j] = static_cast<uint8_t>(amax >= 0x7F800000u ? 0u : e2m1_pair(x[2 * j] * inv, x[2 * j + 1] * inv));
        s[i] = static_cast<uint8_t>(byte);
    }
}

template <typename VT, int FMT>
__global__ void __launch_bounds__(256)
dequantize_kernel(const uint8_t *__restrict__ q, const uint8_t *__restrict__ s, int64_t rows, int K, int Ks,
                  const float *__restrict__ alpha, int64_t rows_per_alpha, VT *__restrict__ v)
{
    constexpr int B = block_of(FMT);
    const int nb = K / B;
    for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < rows * nb;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t r = i / nb;
        const int b = static_cast<int>(i - r * nb);
        const float f = scale_value<FMT>(s[r * Ks + b]);
        const float a = FMT == MOE_FP4_NVFP4 ? alpha[r / rows_per_alpha] : 1.f;
        const uint8_t *p = q + r * (K / 2) + static_cast<int64_t>(b) * (B / 2);
        VT *o = v + r * K + static_cast<int64_t>(b) * B;
        for (int j = 0; j < B / 2; ++j) {
            const float2 c = e2m1_values(p[j]);
            o[2 * j] = from_float<VT>(c.x * f * a);
            o[2 * j + 1] = from_float<VT>(c.y * f * a);
        }
    }
}

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
    const int Ks = scale_cols(K, fmt);
    const int64_t blocks = (rows * Ks + 255) / 256;
    const int grid = static_cast<int>(blocks < 152 * 64 ? blocks : 152 * 64);
    by_type(vdt, [&](auto t) {
        using T = decltype(t);
        auto k = fmt == MOE_FP4_NVFP4 ? quantize_kernel<T, MOE_FP4_NVFP4> : quantize_kernel<T, MOE_FP4_MXFP4>;
        k<<<grid, 256, 0, as_stream(stream)>>>(static_cast<const T *>(v), rows, K, Ks, alpha, rows / groups, q, s);
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
    const int64_t blocks = (rows * (K / block_of(fmt)) + 255) / 256;
    const int grid = static_cast<int>(blocks < 152 * 64 ? blocks : 152 * 64);
    by_type(vdt, [&](auto t) {
        using T = decltype(t);
        auto k = fmt == MOE_FP4_NVFP4 ? dequantize_kernel<T, MOE_FP4_NVFP4> : dequantize_kernel<T, MOE_FP4_MXFP4>;
        k<<<grid, 256, 0, as_stream(stream)>>>(q, s, rows, K, Ks, alpha, rows / groups, static_cast<T *>(v));
    });
    return launch_status();
}
