// gmm_fp4.cu -- products of rows grouped by expert with the experts'
// matrices, both NVFP4 or both MXFP4:
//   y[r][n] = a_x a_w[e] sum over blocks of Sx Sw (sum in the block of cx cw)
// with E2M1 codes c, a scale S per block along K and, for NVFP4, the two
// constants.  Sums are FP32, rounded once.
#include "common.cuh"
#include "fp4.cuh"
#include "ragged.cuh"

namespace moe {
namespace gmm4 {

constexpr int kT = 32;

template <int FMT>
__device__ __forceinline__ float value(const uint8_t *q, const uint8_t *s, int64_t row, int K, int Ks, int k)
{
    const float2 c = fp4::e2m1_values(q[row * (K / 2) + k / 2]);
    return (k & 1 ? c.y : c.x) * fp4::scale_value<FMT>(s[row * Ks + k / fp4::block_of(FMT)]);
}

template <int FMT, typename YT>
__global__ void __launch_bounds__(1024)
rows_kernel(const uint8_t *__restrict__ xq, const uint8_t *__restrict__ xs, const float *__restrict__ xa,
            const uint8_t *__restrict__ wq, const uint8_t *__restrict__ ws, const float *__restrict__ wa,
            const int32_t *__restrict__ off, int R, int E, int N, int K, YT *__restrict__ y, int32_t *dev_status)
{
    __shared__ float sa[kT][kT + 1], sb[kT][kT + 1];
    const int e = blockIdx.y, c0 = blockIdx.x * kT, tx = threadIdx.x, ty = threadIdx.y;
    const int Ks = fp4::scale_cols(K, FMT);
    int lo, hi;
    ragged::group(off, e, R, lo, hi);
    if (blockIdx.x == 0 && tx == 0 && ty == 0)
        ragged::report_bad(off, R, e, dev_status);
    const float f = FMT == MOE_FP4_NVFP4 ? *xa * wa[e] : 1.f;
    for (int r0 = lo; r0 < hi; r0 += kT) {
        float acc = 0.f;
        for (int j0 = 0; j0 < K; j0 += kT) {
            sa[ty][tx] = r0 + ty < hi ? value<FMT>(xq, xs, r0 + ty, K, Ks, j0 + tx) : 0.f;
            sb[tx][ty] = c0 + ty < N ? value<FMT>(wq, ws, static_cast<int64_t>(e) * N + c0 + ty, K, Ks, j0 + tx) : 0.f;
            __syncthreads();
            for (int j = 0; j < kT; ++j)
                acc += sa[ty][j] * sb[j][tx];
            __syncthreads();
        }
        if (r0 + ty < hi && c0 + tx < N)
            y[static_cast<int64_t>(r0 + ty) * N + c0 + tx] = fp4::from_float<YT>(acc * f);
    }
    const int first = min(max(off[0], 0), R), last = max(min(off[E], R), 0);
    if (c0 + tx < N) {
        for (int r = e * kT + ty; r < first; r += gridDim.y * kT)
            y[static_cast<int64_t>(r) * N + c0 + tx] = fp4::from_float<YT>(0.f);
        for (int r = last + e * kT + ty; r < R; r += gridDim.y * kT)
            y[static_cast<int64_t>(r) * N + c0 + tx] = fp4::from_float<YT>(0.f);
    }
}

}  // namespace gmm4
}  // namespace moe

using namespace moe;
using namespace moe::gmm4;

MOE_API moe_status_t moe_grouped_mm_fp4(const uint8_t *xq, const uint8_t *xs, const float *x_alpha, const uint8_t *wq,
                                        const uint8_t *ws, const float *w_alpha, int32_t fmt, const int32_t *offsets,
                                        int32_t R, int32_t E, int32_t N, int32_t K, void *y, int32_t ydt,
                                        int32_t *dev_status, void *stream)
{
    if (R < 0 || E < 1 || N < 1 || K < 1)
        return MOE_ERR_INVALID_ARG;
    if ((fmt != MOE_FP4_NVFP4 && fmt != MOE_FP4_MXFP4) || (ydt != MOE_BF16 && ydt != MOE_FP16 && ydt != MOE_FP32) ||
        E > ragged::kMaxExperts || N % 8 || K % 32)
        return MOE_ERR_UNSUPPORTED;
    if (R == 0)
        return MOE_OK;
    if (!xq || !xs || !wq || !ws || !offsets || !y || (fmt == MOE_FP4_NVFP4) != (x_alpha != nullptr) ||
        (fmt == MOE_FP4_NVFP4) != (w_alpha != nullptr) || !aligned(xq, 16) || !aligned(xs, 16) || !aligned(wq, 16) ||
        !aligned(ws, 16) || !aligned(y, 16) || !aligned(offsets, 4))
        return MOE_ERR_INVALID_ARG;
    const dim3 grid((N + kT - 1) / kT, E), block(kT, kT);
    auto go = [&](auto t) {
        using T = decltype(t);
        auto k = fmt == MOE_FP4_NVFP4 ? rows_kernel<MOE_FP4_NVFP4, T> : rows_kernel<MOE_FP4_MXFP4, T>;
        k<<<grid, block, 0, as_stream(stream)>>>(xq, xs, x_alpha, wq, ws, w_alpha, offsets, R, E, N, K, static_cast<T *>(y),
                                                 dev_status);
    };
    if (ydt == MOE_FP32)
        go(float{});
    else if (ydt == MOE_BF16)
        go(__nv_bfloat16{});
    else
        go(__half{});
    return launch_status();
}
