// gmm.cu -- products of rows grouped by expert with the experts' 16-bit
// matrices, and their gradients:
//   y[r][n]     = sum_k x[r][k]  w[e][n][k]     moe_grouped_mm
//   dx[r][k]    = sum_n dy[r][n] w[e][n][k]     moe_grouped_mm_dgrad
//   dw[e][n][k] = sum_r dy[r][n] x[r][k]        moe_grouped_mm_wgrad
// for the rows r of expert e.  Sums are FP32, rounded once.
#include "common.cuh"
#include "fp4.cuh"
#include "ragged.cuh"

namespace moe {
namespace gmm {

constexpr int kT = 32;                  // tile side

// out[r][c] = sum_j a[r][j] * b(e, c, j); b(e, c, j) = w[e][c][j] (TRANS = 0, w
// [E][C][J]) or w[e][j][c] (TRANS = 1, w [E][J][C]).  One block per (32
// columns, expert) walks the expert's rows.
template <typename T, typename YT, int TRANS>
__global__ void __launch_bounds__(1024)
rows_kernel(const T *__restrict__ a, const T *__restrict__ w, const int32_t *__restrict__ off, int R, int E, int C, int J,
            YT *__restrict__ out, int32_t *dev_status)
{
    __shared__ float sa[kT][kT + 1], sb[kT][kT + 1];
    const int e = blockIdx.y, c0 = blockIdx.x * kT, tx = threadIdx.x, ty = threadIdx.y;
    int lo, hi;
    ragged::group(off, e, R, lo, hi);
    if (blockIdx.x == 0 && tx == 0 && ty == 0)
        ragged::report_bad(off, E, R, e, dev_status);
    const T *we = w + static_cast<int64_t>(e) * C * J;
    for (int r0 = lo; r0 < hi; r0 += kT) {
        float acc = 0.f;
        for (int j0 = 0; j0 < J; j0 += kT) {
            sa[ty][tx] = r0 + ty < hi && j0 + tx < J ? fp4::to_float(a[static_cast<int64_t>(r0 + ty) * J + j0 + tx]) : 0.f;
            if (TRANS)
                sb[ty][tx] = j0 + ty < J && c0 + tx < C ? fp4::to_float(we[static_cast<int64_t>(j0 + ty) * C + c0 + tx]) : 0.f;
            else
                sb[tx][ty] = j0 + tx < J && c0 + ty < C ? fp4::to_float(we[static_cast<int64_t>(c0 + ty) * J + j0 + tx]) : 0.f;
            __syncthreads();
            for (int j = 0; j < kT; ++j)
                acc += sa[ty][j] * sb[j][tx];
            __syncthreads();
        }
        if (r0 + ty < hi && c0 + tx < C)
            out[static_cast<int64_t>(r0 + ty) * C + c0 + tx] = fp4::from_float<YT>(acc);
    }
    // rows outside every group
    const int first = min(max(off[0], 0), R), last = max(min(off[E], R), 0);
    if (c0 + tx < C) {
        for (int r = e * kT + ty; r < first; r += gridDim.y * kT)
            out[static_cast<int64_t>(r) * C + c0 + tx] = fp4::from_float<YT>(0.f);
        for (int r = last + e * kT + ty; r < R; r += gridDim.y * kT)
            out[static_cast<int64_t>(r) * C + c0 + tx] = fp4::from_float<YT>(0.f);
    }
}

template <typename T, typename YT>
__global__ void __launch_bounds__(1024)
wgrad_kernel(const T *__restrict__ dy, const T *__restrict__ x, const int32_t *__restrict__ off, int R, int E, int N, int K,
             YT *__restrict__ dw, int accumulate, int32_t *dev_status)
{
    __shared__ float sa[kT][kT + 1], sb[kT][kT + 1];
    const int e = blockIdx.z, n0 = blockIdx.y * kT, k0 = blockIdx.x * kT, tx = threadIdx.x, ty = threadIdx.y;
    int lo, hi;
    ragged::group(off, e, R, lo, hi);
    if (blockIdx.x == 0 && blockIdx.y == 0 && tx == 0 && ty == 0)
        ragged::report_bad(off, E, R, e, dev_status);
    float acc = 0.f;
    for (int r0 = lo; r0 < hi; r0 += kT) {
        sa[ty][tx] = r0 + ty < hi && n0 + tx < N ? fp4::to_float(dy[static_cast<int64_t>(r0 + ty) * N + n0 + tx]) : 0.f;
        sb[ty][tx] = r0 + ty < hi && k0 + tx < K ? fp4::to_float(x[static_cast<int64_t>(r0 + ty) * K + k0 + tx]) : 0.f;
        __syncthreads();
        for (int j = 0; j < kT; ++j)
            acc += sa[j][ty] * sb[j][tx];
        __syncthreads();
    }
    if (n0 + ty < N && k0 + tx < K) {
        YT *o = dw + (static_cast<int64_t>(e) * N + n0 + ty) * K + k0 + tx;
        *o = fp4::from_float<YT>(accumulate ? acc + fp4::to_float(*o) : acc);
    }
}

static bool type16(int32_t dt) { return dt == MOE_BF16 || dt == MOE_FP16; }
static bool out_type(int32_t t, int32_t dt) { return t == MOE_FP32 || t == dt; }

// The checks that the three products share.
static moe_status_t check(const void *a, const void *b, const void *out, int32_t dt, int32_t odt, int32_t R, int32_t E,
                          int32_t N, int32_t K, const int32_t *offsets)
{
    if (R < 0 || E < 1 || N < 1 || K < 1)
        return MOE_ERR_INVALID_ARG;
    if (!type16(dt) || !out_type(odt, dt) || E > ragged::kMaxExperts || N % 8 || K % 8)
        return MOE_ERR_UNSUPPORTED;
    if (!offsets || !out || !aligned(out, 16) || !aligned(offsets, 4))
        return MOE_ERR_INVALID_ARG;
    if (R && (!a || !b || !aligned(a, 16) || !aligned(b, 16)))
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

template <int TRANS>
static moe_status_t rows(const void *a, const void *w, int32_t dt, int32_t R, int32_t E, int32_t C, int32_t J,
                         const int32_t *off, void *y, int32_t ydt, int32_t *dev_status, cudaStream_t s)
{
    const dim3 grid((C + kT - 1) / kT, E), block(kT, kT);
    auto go = [&](auto t, auto u) {
        using T = decltype(t);
        using U = decltype(u);
        rows_kernel<T, U, TRANS><<<grid, block, 0, s>>>(static_cast<const T *>(a), static_cast<const T *>(w), off, R, E, C, J,
                                                        static_cast<U *>(y), dev_status);
    };
    if (dt == MOE_BF16)
        ydt == MOE_FP32 ? go(__nv_bfloat16{}, float{}) : go(__nv_bfloat16{}, __nv_bfloat16{});
    else
        ydt == MOE_FP32 ? go(__half{}, float{}) : go(__half{}, __half{});
    return launch_status();
}

}  // namespace gmm
}  // namespace moe

using namespace moe;
using namespace moe::gmm;

MOE_API moe_status_t moe_grouped_mm(const void *x, const void *w, int32_t dt, const int32_t *offsets, int32_t R, int32_t E,
                                    int32_t N, int32_t K, void *y, int32_t ydt, int32_t *dev_status, void *stream)
{
    if (R == 0 && E >= 1 && N >= 1 && K >= 1)
        return type16(dt) && out_type(ydt, dt) ? MOE_OK : MOE_ERR_UNSUPPORTED;
    const moe_status_t st = check(x, w, y, dt, ydt, R, E, N, K, offsets);
    return st != MOE_OK ? st : rows<0>(x, w, dt, R, E, N, K, offsets, y, ydt, dev_status, as_stream(stream));
}

MOE_API moe_status_t moe_grouped_mm_dgrad(const void *dy, const void *w, int32_t dt, const int32_t *offsets, int32_t R,
                                          int32_t E, int32_t N, int32_t K, void *dx, int32_t xdt, int32_t *dev_status,
                                          void *stream)
{
    if (R == 0 && E >= 1 && N >= 1 && K >= 1)
        return type16(dt) && out_type(xdt, dt) ? MOE_OK : MOE_ERR_UNSUPPORTED;
    const moe_status_t st = check(dy, w, dx, dt, xdt, R, E, N, K, offsets);
    return st != MOE_OK ? st : rows<1>(dy, w, dt, R, E, K, N, offsets, dx, xdt, dev_status, as_stream(stream));
}

MOE_API moe_status_t moe_grouped_mm_wgrad(const void *dy, const void *x, int32_t dt, const int32_t *offsets, int32_t R,
                                          int32_t E, int32_t N, int32_t K, void *dw, int32_t wdt, int32_t accumulate,
                                          int32_t *dev_status, void *stream)
{
    if (accumulate != 0 && accumulate != 1)
        return MOE_ERR_INVALID_ARG;
    const moe_status_t st = check(dy, x, dw, dt, wdt, R, E, N, K, offsets);
    if (st != MOE_OK)
        return st;
    const dim3 grid((K + kT - 1) / kT, (N + kT - 1) / kT, E), block(kT, kT);
    auto go = [&](auto t, auto u) {
        using T = decltype(t);
        using U = decltype(u);
        wgrad_kernel<T, U><<<grid, block, 0, as_stream(stream)>>>(static_cast<const T *>(dy), static_cast<const T *>(x),
                                                                  offsets, R, E, N, K, static_cast<U *>(dw), accumulate,
                                                                  dev_status);
    };
    if (dt == MOE_BF16)
        wdt == MOE_FP32 ? go(__nv_bfloat16{}, float{}) : go(__nv_bfloat16{}, __nv_bfloat16{});
    else
        wdt == MOE_FP32 ? go(__half{}, float{}) : go(__half{}, __half{});
    return launch_status();
}
