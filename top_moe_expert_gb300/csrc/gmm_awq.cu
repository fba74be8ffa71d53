// gmm_awq.cu -- the grouped product of few rows per expert with 4-bit AWQ weights:
// y[r][n] = sum_k x[r][k] (q[e][n][k] - zero) scale for the rows r of expert e.
//
// The work is reading the weights of the experts that have rows once, 0.52 bytes
// each, and widening them.  A CTA takes 16 rows of an expert's weights and up to
// 8 NT of its rows of x, and its warps divide K.  The codes less their zero, whole
// numbers up to 15, are exact in x's own type, and so are the products: the
// tensor cores (m16n8k16, the weights as the left operand) add a group of 128 in
// FP32, and the group's scale comes to the sum.  Against multiplications on the
// CUDA cores that saves the conversion to FP32 and, for more than one row, widens
// each weight once for all rows.
//
// The order of k inside a group is free as long as both operands agree: lane t of
// a row's four takes 16 bytes of codes, k = 32 t .. 32 t + 31, and of each word of
// 8 the pairs (0, 4), (1, 5), (2, 6), (3, 7), which one AND and OR turn into two
// numbers 1024 + q (fp16) or 128 + q (bf16).
#include <type_traits>

#include "common.cuh"
#include "fp4.cuh"
#include "ragged.cuh"

namespace moe {
namespace gmm_awq {

constexpr int kWarps = 8, kThreads = kWarps * 32, kRowsW = 16;

struct Args {
    const void *x;
    const uint32_t *q;
    const __half *scale;
    const uint32_t *zero;
    const int32_t *off;
    void *y;
    int32_t *dev_status;
    int R, E, N, K;
};

__device__ __forceinline__ int clamp_off(const Args &a, int e) { return min(max(a.off[e], 0), a.R); }

// The slot-th run of at most `most` rows of one expert, found by one warp: expert
// (-1: there is none), first row, rows.
struct Run {
    int e, r0, n;
};

__device__ __forceinline__ Run find_run(const Args &a, int slot, int most, int lane)
{
    const int per = (a.E + 31) / 32, e0 = min(lane * per, a.E), e1 = min(e0 + per, a.E);
    int sum = 0;
    for (int e = e0; e < e1; ++e)
        sum += (max(clamp_off(a, e + 1) - clamp_off(a, e), 0) + most - 1) / most;
    int run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o)
            run += v;
    }
    Run f{-1, 0, 0};
    const unsigned past = __ballot_sync(0xffffffffu, run > slot);
    if (past == 0)
        return f;
    const int src = __ffs(past) - 1;
    if (lane == src) {
        int at = run - sum;
        for (int e = e0; e < e1; ++e) {
            const int lo = clamp_off(a, e), n = max(clamp_off(a, e + 1) - lo, 0), runs = (n + most - 1) / most;
            if (slot < at + runs) {
                f.e = e;
                f.r0 = lo + (slot - at) * most;
                f.n = min(most, lo + n - f.r0);
                break;
            }
            at += runs;
        }
    }
    f.e = __shfl_sync(0xffffffffu, f.e, src);
    f.r0 = __shfl_sync(0xffffffffu, f.r0, src);
    f.n = __shfl_sync(0xffffffffu, f.n, src);
    return f;
}

template <typename T>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    if constexpr (std::is_same<T, __half>::value)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Pairs of codes (i, i + 4) of a word less the zero, i = 0 .. 3, exact in T.
template <typename T>
struct Zero;

template <>
struct Zero<__half> {
    __half2 low, high;                       // 1024 + z, and -(64 + z) for the codes in the upper nibbles
    __device__ __forceinline__ explicit Zero(uint32_t z)
    {
        low = __half2half2(__ushort_as_half(static_cast<uint16_t>(0x6400u | z)));
        high = __half2half2(__float2half_rn(-64.f - static_cast<float>(z)));
    }
    __device__ __forceinline__ void widen(uint32_t w, uint32_t (&p)[4]) const
    {
        const __half2 r16 = __half2half2(__ushort_as_half(0x2C00u));           // 1 / 16
#pragma unroll
        for (int i = 0; i < 2; ++i, w >>= 8) {
            const uint32_t lo = (w & 0x000F000Fu) | 0x64006400u, hi = (w & 0x00F000F0u) | 0x64006400u;
            const __half2 a = __hsub2(*reinterpret_cast<const __half2 *>(&lo), low);
            const __half2 b = __hfma2(*reinterpret_cast<const __half2 *>(&hi), r16, high);   // 64 + q - 64 - z
            p[2 * i] = *reinterpret_cast<const uint32_t *>(&a);
            p[2 * i + 1] = *reinterpret_cast<const uint32_t *>(&b);
        }
    }
};

template <>
struct Zero<__nv_bfloat16> {
    __nv_bfloat162 low;                      // 128 + z
    __device__ __forceinline__ explicit Zero(uint32_t z)
    {
        low = __bfloat162bfloat162(__ushort_as_bfloat16(static_cast<uint16_t>(0x4300u | z)));
    }
    __device__ __forceinline__ void widen(uint32_t w, uint32_t (&p)[4]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i, w >>= 4) {
            const uint32_t v = (w & 0x000F000Fu) | 0x43004300u;
            const __nv_bfloat162 a = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v), low);
            p[i] = *reinterpret_cast<const uint32_t *>(&a);
        }
    }
};

template <typename T, typename OT, int NT>
__global__ void __launch_bounds__(kThreads) gmm_awq_kernel(const Args a)
{
    __shared__ Run s_run;
    __shared__ float part[kWarps][8 * NT][kRowsW + 1];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int n0 = blockIdx.x * kRowsW, G = a.K / 128;
    for (int slot = blockIdx.y;; slot += gridDim.y) {
        if (warp == 0) {
            const Run f = find_run(a, slot, 8 * NT, lane);
            if (lane == 0)
                s_run = f;
        }
        __syncthreads();
        const Run f = s_run;
        if (f.e < 0)
            break;
        const bool second = n0 + 8 < a.N;                       // N is a multiple of 8: the tile's lower half may be past it
        const int64_t row0 = static_cast<int64_t>(f.e) * a.N + n0 + g, row1 = second ? row0 + 8 : row0;
        const uint4 *q0 = reinterpret_cast<const uint4 *>(a.q + row0 * (a.K / 8)) + t;
        const uint4 *q1 = reinterpret_cast<const uint4 *>(a.q + row1 * (a.K / 8)) + t;
        const __half *s0 = a.scale + row0 * G, *s1 = a.scale + row1 * G;
        const uint32_t *z0 = a.zero + (row0 >> 3) * G, *z1 = a.zero + (row1 >> 3) * G;
        const int nt = (f.n + 7) / 8;
        const T *x = static_cast<const T *>(a.x) + static_cast<int64_t>(f.r0 + g) * a.K + 32 * t;
        float acc[NT][4] = {};
        const int k0 = static_cast<int>(static_cast<int64_t>(G) * warp / kWarps);
        const int k1 = static_cast<int>(static_cast<int64_t>(G) * (warp + 1) / kWarps);
#pragma unroll 2
        for (int k = k0; k < k1; ++k) {
            const uint4 w0 = fp4::ld_once_u4(q0 + 4 * k), w1 = fp4::ld_once_u4(q1 + 4 * k);
            const float f0 = __half2float(s0[k]), f1 = __half2float(s1[k]);
            const Zero<T> c0(z0[k] >> (4 * g) & 15u), c1(z1[k] >> (4 * g) & 15u);
            float sum[NT][4] = {};
            const uint32_t v0[4] = {w0.x, w0.y, w0.z, w0.w}, v1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t p0[4], p1[4];
                c0.widen(v0[i], p0);
                c1.widen(v1[i], p1);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    if (j < nt) {
                        uint4 xv = make_uint4(0, 0, 0, 0);
                        if (8 * j + g < f.n)
                            xv = *reinterpret_cast<const uint4 *>(x + static_cast<int64_t>(8 * j) * a.K + 128 * k + 8 * i);
                        mma<T>(sum[j], p0[0], p1[0], p0[1], p1[1], __byte_perm(xv.x, xv.z, 0x5410), __byte_perm(xv.x, xv.z, 0x7632));
                        mma<T>(sum[j], p0[2], p1[2], p0[3], p1[3], __byte_perm(xv.y, xv.w, 0x5410), __byte_perm(xv.y, xv.w, 0x7632));
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                acc[j][0] = fmaf(sum[j][0], f0, acc[j][0]);
                acc[j][1] = fmaf(sum[j][1], f0, acc[j][1]);
                acc[j][2] = fmaf(sum[j][2], f1, acc[j][2]);
                acc[j][3] = fmaf(sum[j][3], f1, acc[j][3]);
            }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            part[warp][8 * j + 2 * t][g] = acc[j][0];
            part[warp][8 * j + 2 * t + 1][g] = acc[j][1];
            part[warp][8 * j + 2 * t][g + 8] = acc[j][2];
            part[warp][8 * j + 2 * t + 1][g + 8] = acc[j][3];
        }
        __syncthreads();
        for (int i = threadIdx.x; i < kRowsW * f.n; i += kThreads) {
            const int n = i & (kRowsW - 1), r = i / kRowsW;
            float sum = part[0][r][n];
#pragma unroll
            for (int w = 1; w < kWarps; ++w)
                sum += part[w][r][n];
            if (n0 + n < a.N)
                static_cast<OT *>(a.y)[static_cast<int64_t>(f.r0 + r) * a.N + n0 + n] = fp4::from_float<OT>(sum);
        }
        __syncthreads();
    }
    // rows outside every group, divided among the CTAs of a column of tiles
    const int first = clamp_off(a, 0), last = clamp_off(a, a.E), outside = first + a.R - last;
    for (int64_t i = static_cast<int64_t>(blockIdx.y) * kThreads + threadIdx.x; i < static_cast<int64_t>(outside) * kRowsW;
         i += static_cast<int64_t>(gridDim.y) * kThreads) {
        const int n = n0 + static_cast<int>(i & (kRowsW - 1)), j = static_cast<int>(i / kRowsW), r = j < first ? j : last + j - first;
        if (n < a.N)
            static_cast<OT *>(a.y)[static_cast<int64_t>(r) * a.N + n] = fp4::from_float<OT>(0.f);
    }
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int e = threadIdx.x; e < a.E; e += kThreads)
            ragged::report_bad(a.off, a.R, e, a.dev_status);
}

template <typename T, typename OT>
static moe_status_t launch(const Args &a, cudaStream_t s)
{
    const int most = a.R <= 8 ? 8 : 32;
    const int64_t live = a.E < a.R ? a.E : a.R, runs = (a.R + live * (most - 1)) / most;
    const dim3 grid(static_cast<unsigned>((a.N + kRowsW - 1) / kRowsW), static_cast<unsigned>(runs < 65535 ? runs : 65535));
    const cudaError_t e = most == 8 ? launch_pdl(gmm_awq_kernel<T, OT, 1>, grid, dim3(kThreads), 0, s, a)
                                    : launch_pdl(gmm_awq_kernel<T, OT, 4>, grid, dim3(kThreads), 0, s, a);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace gmm_awq
}  // namespace moe

using namespace moe;

MOE_API moe_status_t moe_grouped_mm_awq(const void *x, int32_t dt, const moe_weights_t *w, const int32_t *offsets, int32_t R,
                                        void *y, int32_t ydt, int32_t *dev_status, void *stream)
{
    if (R < 0 || !w || w->E < 1 || w->N < 1 || w->K < 1)
        return MOE_ERR_INVALID_ARG;
    if (w->fmt != MOE_W_AWQ4 || (dt != MOE_BF16 && dt != MOE_FP16) || (ydt != dt && ydt != MOE_FP32))
        return MOE_ERR_UNSUPPORTED;
    if (w->N % 8 != 0 || w->K % 128 != 0)
        return MOE_ERR_INVALID_ARG;
    if (w->E > ragged::kMaxExperts || R > ragged::kMaxSide || w->N > ragged::kMaxSide || w->K > ragged::kMaxSide ||
        !ragged::list_fits(w->E, R, 1, 8))
        return MOE_ERR_UNSUPPORTED;
    if (R == 0)
        return MOE_OK;
    if (!x || !y || !offsets || !w->q || !w->scale || !w->zero || !aligned(x, 16) || !aligned(y, 16) || !aligned(offsets, 4) ||
        !aligned(w->q, 16) || !aligned(w->scale, 16) || !aligned(w->zero, 16) || !aligned(dev_status, 4))
        return MOE_ERR_INVALID_ARG;
    const gmm_awq::Args a{x, static_cast<const uint32_t *>(w->q), static_cast<const __half *>(w->scale),
                          static_cast<const uint32_t *>(w->zero), offsets, y, dev_status, R, w->E, w->N, w->K};
    cudaStream_t s = as_stream(stream);
    if (dt == MOE_BF16)
        return ydt == MOE_FP32 ? gmm_awq::launch<__nv_bfloat16, float>(a, s) : gmm_awq::launch<__nv_bfloat16, __nv_bfloat16>(a, s);
    return ydt == MOE_FP32 ? gmm_awq::launch<__half, float>(a, s) : gmm_awq::launch<__half, __half>(a, s);
}
