// gmm_small.cu -- the grouped product y[r][n] = sum_k x[r][k] w[e][n][k] for at most
// four rows (a token's routes to a few experts), bf16 or fp16.
//
// The work is reading the weights of the experts that have rows, and with few
// experts the tiled kernel of gmm.cu has too few tiles to keep the SMs loading
// (6 pairs of CTAs for one expert's 1536 x 2048).  Here every warp takes an even,
// contiguous share of the (expert, pair of n) list and forms the two rows' dot
// products across its lanes: 16-byte loads, 8 steps of both rows under way,
// products and sums in FP32 in a fixed order.  Measured (us, this kernel / the
// tiled one; K = 2048, N = 1536 and K = 7168, N = 4096): one row 3.9 / 8.8 and
// 12.6 / 25.4, two rows of each of two experts 4.8 / 8.8 and 24.3 / 28.1; from
// eight rows of eight experts on the tiled kernel is as fast or faster.
#include <type_traits>

#include "attr.h"
#include "common.cuh"
#include "fp4.cuh"
#include "gmm_small.h"
#include "ragged.cuh"

namespace moe {
namespace gmm_small {

constexpr int kRows = kSmallRows;
constexpr int kThreads = 256, kWarps = kThreads / 32, kPerSm = 2, kUnroll = 8;

struct Groups {
    int expert[kRows];                  // of each row, -1 for none
    int e[kRows], r0[kRows], n[kRows], count;
};

// The groups that have rows, the same list in every CTA.  Offsets are clamped
// as in ragged.cuh.
__device__ __forceinline__ void make_groups(Groups &g, const int32_t *off, int E, int R)
{
    if (threadIdx.x < kRows)
        g.expert[threadIdx.x] = -1;
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kThreads) {
        const int lo = min(max(off[e], 0), R), hi = min(max(off[e + 1], 0), R);
        for (int r = lo; r < hi; ++r)
            g.expert[r] = e;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        int m = 0;
        for (int r = 0; r < R;) {
            const int e = g.expert[r];
            int n = 1;
            while (r + n < R && g.expert[r + n] == e)
                ++n;
            if (e >= 0) {
                g.e[m] = e;
                g.r0[m] = r;
                g.n[m++] = n;
            }
            r += n;
        }
        g.count = m;
    }
    __syncthreads();
}

struct Args {
    const void *x, *w;
    const int32_t *off;
    void *y;
    int32_t *dev_status;
    int R, E, N, K;
};

template <typename T>
__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (std::is_same<T, __half>::value)
            f16x2_to_float(w[i], f[2 * i], f[2 * i + 1]);
        else
            bf16x2_to_float(w[i], f[2 * i], f[2 * i + 1]);
    }
}

// Two rows of w with NT rows of x: lane l takes elements 8 l .. 8 l + 7 of every 256.
template <typename T, typename OT, int NT>
__device__ __forceinline__ void pair_of(const Args &a, int e, int r0, int n, int lane)
{
    const T *x = static_cast<const T *>(a.x) + static_cast<int64_t>(r0) * a.K;
    const T *w = static_cast<const T *>(a.w) + (static_cast<int64_t>(e) * a.N + n) * a.K;
    float acc[2][NT] = {};
#pragma unroll kUnroll
    for (int k = lane * 8; k < a.K; k += 256) {
        const uint4 w0 = fp4::ld_once_u4(w + k), w1 = fp4::ld_once_u4(w + a.K + k);
        uint4 xv[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t)
            xv[t] = *reinterpret_cast<const uint4 *>(x + static_cast<int64_t>(t) * a.K + k);
        float f0[8], f1[8];
        unpack8<T>(w0, f0);
        unpack8<T>(w1, f1);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float xf[8];
            unpack8<T>(xv[t], xf);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                acc[0][t] = fmaf(f0[j], xf[j], acc[0][t]);
                acc[1][t] = fmaf(f1[j], xf[j], acc[1][t]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const float v = warp_sum(acc[i][t]);
            if (lane == 0)
                static_cast<OT *>(a.y)[static_cast<int64_t>(r0 + t) * a.N + n + i] = fp4::from_float<OT>(v);
        }
}

template <typename T, typename OT>
__global__ void __launch_bounds__(kThreads, kPerSm) small_kernel(const Args a)
{
    __shared__ Groups c;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    make_groups(c, a.off, a.E, a.R);
    const int lane = threadIdx.x & 31;
    const uint32_t half = a.N / 2;                       // N is even: pairs of rows
    const int64_t total = static_cast<int64_t>(c.count) * half, warps = static_cast<int64_t>(gridDim.x) * kWarps;
    const int64_t me = static_cast<int64_t>(threadIdx.x >> 5) * gridDim.x + blockIdx.x;
    const uint32_t end = static_cast<uint32_t>(total * (me + 1) / warps);
    for (uint32_t i = static_cast<uint32_t>(total * me / warps); i < end; ++i) {
        const int m = i / half, n = 2 * (i - m * half);
        switch (c.n[m]) {
        case 1: pair_of<T, OT, 1>(a, c.e[m], c.r0[m], n, lane); break;
        case 2: pair_of<T, OT, 2>(a, c.e[m], c.r0[m], n, lane); break;
        case 3: pair_of<T, OT, 3>(a, c.e[m], c.r0[m], n, lane); break;
        default: pair_of<T, OT, 4>(a, c.e[m], c.r0[m], n, lane); break;
        }
    }
    // rows outside every group
    for (int r = 0; r < a.R; ++r)
        if (c.expert[r] < 0)
            for (int64_t i = blockIdx.x * kThreads + threadIdx.x; i < a.N; i += gridDim.x * kThreads)
                static_cast<OT *>(a.y)[static_cast<int64_t>(r) * a.N + i] = fp4::from_float<OT>(0.f);
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e < a.E; e += kThreads)
            ragged::report_bad(a.off, a.R, e, a.dev_status);
}

template <typename T, typename OT>
static moe_status_t launch(const Args &a, cudaStream_t s)
{
    return launch_pdl(small_kernel<T, OT>, dim3(device_sm_count() * kPerSm), dim3(kThreads), 0, s, a) == cudaSuccess
               ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace gmm_small

moe_status_t grouped_mm_small(const void *x, const void *w, int dt, const int32_t *off, int R, int E, int N, int K, void *y,
                              int ydt, int32_t *dev_status, cudaStream_t s)
{
    using namespace gmm_small;
    const Args a{x, w, off, y, dev_status, R, E, N, K};
    if (dt == MOE_BF16)
        return ydt == MOE_FP32 ? launch<__nv_bfloat16, float>(a, s) : launch<__nv_bfloat16, __nv_bfloat16>(a, s);
    return ydt == MOE_FP32 ? launch<__half, float>(a, s) : launch<__half, __half>(a, s);
}

}  // namespace moe
