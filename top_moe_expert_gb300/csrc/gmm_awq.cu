// gmm_awq.cu -- the grouped product of few rows per expert with 4-bit AWQ weights:
// y[r][n] = sum_k x[r][k] (q[e][n][k] - zero) scale for the rows r of expert e.
//
// The work is reading the weights of the experts that have rows once, 0.52 bytes
// each, and widening them.  A CTA takes 16 or 32 rows of an expert's weights and up to
// 8 or 16 of its rows of x; its two or four warps divide K (by K alone, so that a
// row's result does not depend on the other rows), each with a ring of its own that
// cp.async fills two groups ahead, and add their sums in order at the end.  The codes
// less their zero, whole numbers up to 15, are exact in x's own type, and so are the
// products: the tensor cores (m16n8k16, the weights as the left operand) add a group
// of 128 in FP32, and the group's scale comes to the sum.  Against multiplications on
// the CUDA cores that saves the conversion to FP32 and, for more than one row, widens
// each weight once for all rows.
//
// The order of k inside a group is free as long as both operands agree: lane t of
// a row's four takes 16 bytes of codes, k = 32 t .. 32 t + 31, and of each word of
// 8 the pairs (0, 4), (1, 5), (2, 6), (3, 7), which one AND and OR turn into two
// numbers 1024 + q (fp16) or 128 + q (bf16): a whole number in the low bits of a
// float's fraction (Kim, Henry, Fahim, Hassan Awadalla: "Who says elephants can't run",
// 2022, widen 4-bit weights to fp16 so).
//
// Bound in two parts.  The widening: some 145 instructions for 16 rows by a group, half
// of them shifts and masks of the pipe that runs at half rate, which is 66 % busy.  The
// rest is latency: with 120 registers a quarter of the warps are resident, 58 % of the
// issue slots are used, and what warps wait for first are global loads (x, in the loop),
// then that pipe, then the barriers around each tile.  One row by 65536 x 8192 takes 76
// us (3.7 TB/s), one row of each of 128 experts of 1536 x 2048 63 us (3.4 TB/s), 512
// rows, Zipf over them, 57.2 us.  What did not help there: deeper rings or weights
// straight into registers, a group ahead or not; x a group ahead; one CTA per SM that
// walks all its tiles with x staged in shared memory (102 us); the zero taken off the
// sums instead of the codes would save a fifth of the instructions, but the sums of 128 +
// q lose four bits.  Few rows are bound by one warp's chain of instructions, near half of
// it waits for global loads: 8 rows of 8 of 128 experts 8.1 us, one row by 4096 x 7168
// 8.1 us.
#include <atomic>
#include <type_traits>

#include "attr.h"
#include "common.cuh"
#include "fp4.cuh"
#include "ragged.cuh"

namespace moe {
namespace gmm_awq {

constexpr int kMaxK = 1 << 24, kDepth = 3;

struct Args {
    const void *x;
    const uint32_t *q;
    const __half *scale;
    const uint32_t *zero;
    const int32_t *off;
    void *y;
    int32_t *dev_status;
    int R, E, N, K;
    bool y32;
};

__device__ __forceinline__ int clamp_off(const Args &a, int e) { return min(max(a.off[e], 0), a.R); }

// The slot-th run of at most `most` rows of one expert, found by one warp: expert
// (-1: there is none), first row, rows; and how many such runs there are.
struct Run {
    int e, r0, n, runs;
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
    Run f{-1, 0, 0, __shfl_sync(0xffffffffu, run, 31)};
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
    uint32_t low, high;                      // 1024 + z, and -(64 + z) for the codes in the upper nibbles
    __device__ __forceinline__ explicit Zero(uint32_t z) : low(0x64006400u | z | z << 16)
    {
        asm("sub.f16x2 %0, %1, %2;" : "=r"(high) : "r"(0x63806380u), "r"(low));                    // 960 - 1024 - z
    }
    __device__ __forceinline__ void widen(uint32_t w, uint32_t (&p)[4]) const
    {
#pragma unroll
        for (int i = 0; i < 2; ++i, w >>= 8) {
            const uint32_t lo = (w & 0x000F000Fu) | 0x64006400u, hi = (w & 0x00F000F0u) | 0x64006400u;
            asm("sub.f16x2 %0, %1, %2;" : "=r"(p[2 * i]) : "r"(lo), "r"(low));
            asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(p[2 * i + 1]) : "r"(hi), "r"(0x2C002C00u), "r"(high));   // / 16 - 64 - z
        }
    }
};

template <>
struct Zero<__nv_bfloat16> {
    uint32_t low;                            // -(128 + z)
    __device__ __forceinline__ explicit Zero(uint32_t z) : low(0xC300C300u | z | z << 16) {}
    __device__ __forceinline__ void widen(uint32_t w, uint32_t (&p)[4]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i, w >>= 4) {
            const uint32_t v = (w & 0x000F000Fu) | 0x43004300u;
            asm("add.bf16x2 %0, %1, %2;" : "=r"(p[i]) : "r"(v), "r"(low));
        }
    }
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void cp4(uint32_t dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// A stage of a warp's ring: 16 MT rows of w by a group of 128, 64 bytes each; the
// words that hold the rows' scales; the words of zeros of every 8 rows.
template <int MT>
constexpr int kStage = MT * 1024 + 16 * MT * 4 + 16;

// The loads of a warp's part of w: the groups k0 .. k1 - 1 of the rows from n0 on, a
// stage at a time.  Rows past N are left out: what their places hold reaches only
// their own sums, which are not stored.
template <int MT, int D>
struct Loader {
    uint32_t ring;
    const uint8_t *q, *scale;
    const uint32_t *zero;
    int64_t eight;                                     // bytes to the rows 8 further
    int blocks, left, odd, put;
    __device__ __forceinline__ Loader(const Args &a, uint32_t at, int e, int n0, int k0, int k1, int lane)
    {
        const int G = a.K / 128;
        const int64_t row = static_cast<int64_t>(e) * a.N + n0, first = (row + lane) * G + k0;
        ring = at;
        q = reinterpret_cast<const uint8_t *>(a.q) + (row + (lane >> 2)) * (a.K / 2) + (lane & 3) * 16 + k0 * 64;
        eight = static_cast<int64_t>(a.K) * 4;
        odd = static_cast<int>(first & 1);             // a scale is half of an aligned word
        scale = reinterpret_cast<const uint8_t *>(a.scale) + (first - odd) * 2;
        zero = a.zero + ((row >> 3) + lane) * G + k0;
        blocks = min((a.N - n0) / 8, 2 * MT);
        left = k1 - k0;
        put = 0;
    }
    __device__ __forceinline__ void next(int lane)
    {
        if (left > 0) {
            const uint32_t at = ring + put * kStage<MT>;
#pragma unroll
            for (int m = 0; m < 2 * MT; ++m)
                if (m < blocks)
                    cp16(at + m * 512 + lane * 16, q + m * eight);
            if (lane < 8 * blocks)
                cp4(at + MT * 1024 + lane * 4, scale);
            if (lane < blocks)
                cp4(at + MT * 1024 + MT * 64 + lane * 4, zero);
            q += 64;
            odd ^= 1;
            scale += odd ? 0 : 4;
            ++zero;
            --left;
            put = put + 1 == D ? 0 : put + 1;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
};

// One warp's sums of 16 MT rows of w by 8 NT rows of x over its groups.
template <typename T, int MT, int NT, int D>
__device__ __forceinline__ void dot(const Args &a, const Run &f, Loader<MT, D> &load, const uint8_t *ring, int k0, int k1, int lane,
                                    float (&acc)[MT][NT][4])
{
    const int g = lane >> 2, t = lane & 3, odd = a.K / 128 & g & 1;
    const uint4 *x[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j)                       // a lane without a row reads the last one: its column is not used
        x[j] = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.x) +
                                               static_cast<int64_t>(f.r0 + min(8 * j + g, f.n - 1)) * a.K + 32 * t) + 16 * k0;
    int get = 0;
    for (int k = k0; k < k1; ++k) {
        uint4 xv[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j, x[j - 1] += 16)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                xv[j][i] = x[j][i];
        asm volatile("cp.async.wait_group %0;" ::"n"(D - 2) : "memory");
        __syncwarp();
        load.next(lane);
        const uint8_t *st = ring + get * kStage<MT>;
        get = get + 1 == D ? 0 : get + 1;
        const uint8_t *meta = st + MT * 1024;
        const int shift = ((odd ^ k) & 1) << 4;         // the scale's half of its word: rows of odd K / 128 alternate
        uint4 w[2 * MT];
        float s[2 * MT];
        uint32_t z[2 * MT];
#pragma unroll
        for (int m = 0; m < 2 * MT; ++m) {
            w[m] = *reinterpret_cast<const uint4 *>(st + m * 512 + lane * 16);
            s[m] = __half2float(__ushort_as_half(static_cast<uint16_t>(*reinterpret_cast<const uint32_t *>(meta + (8 * m + g) * 4) >> shift)));
            z[m] = *reinterpret_cast<const uint32_t *>(meta + MT * 64 + m * 4) >> (4 * g) & 15u;
        }
        float sum[MT][NT][4] = {};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t p[2 * MT][4];
#pragma unroll
            for (int m = 0; m < 2 * MT; ++m)
                Zero<T>(z[m]).widen(i == 0 ? w[m].x : i == 1 ? w[m].y : i == 2 ? w[m].z : w[m].w, p[m]);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const uint4 v = xv[j][i];
                const uint32_t b0 = __byte_perm(v.x, v.z, 0x5410), b1 = __byte_perm(v.x, v.z, 0x7632);
                const uint32_t b2 = __byte_perm(v.y, v.w, 0x5410), b3 = __byte_perm(v.y, v.w, 0x7632);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    mma<T>(sum[m][j], p[2 * m][0], p[2 * m + 1][0], p[2 * m][1], p[2 * m + 1][1], b0, b1);
                    mma<T>(sum[m][j], p[2 * m][2], p[2 * m + 1][2], p[2 * m][3], p[2 * m + 1][3], b2, b3);
                }
            }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    acc[m][j][c] = fmaf(sum[m][j][c], s[2 * m + (c >> 1)], acc[m][j][c]);
    }
}

// W warps divide K; a CTA takes 16 MT rows of w and a run of up to 8 NT rows of x.
template <typename T, int W, int MT, int NT>
__global__ void __launch_bounds__(32 * W, (W == 2 && MT * NT == 1 ? 24 : 16) / W) gmm_awq_kernel(const Args a)
{
    constexpr int kThreads = 32 * W, kRowsW = 16 * MT, D = kDepth;
    __shared__ Run s_run;
    __shared__ float part[W][8 * NT][kRowsW + 1];
    extern __shared__ __align__(16) uint8_t rings[];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const uint8_t *ring = rings + warp * D * kStage<MT>;
    const int n0 = blockIdx.x * kRowsW, G = a.K / 128;
    const int k0 = G * warp / W, k1 = G * (warp + 1) / W;
    const int first = clamp_off(a, 0), last = clamp_off(a, a.E);
    const int64_t outside = static_cast<int64_t>(first) + a.R - last;
    for (int64_t slot = blockIdx.y, runs = slot + 1; slot < runs; slot += gridDim.y) {
        if (warp == 0) {
            const Run f = find_run(a, static_cast<int>(slot), 8 * NT, lane);
            if (lane == 0)
                s_run = f;
        }
        __syncthreads();
        const Run f = s_run;
        runs = f.runs;                                                   // the grid has as many where offsets are in order
        if (f.e < 0)
            break;
        Loader<MT, D> load(a, static_cast<uint32_t>(__cvta_generic_to_shared(ring)), f.e, n0, k0, k1, lane);
#pragma unroll
        for (int i = 0; i < D - 1; ++i)
            load.next(lane);
        float (*mine)[kRowsW + 1] = part[warp];
        if (NT == 1 || f.n <= 8) {
            float acc[MT][1][4] = {};
            dot<T, MT, 1, D>(a, f, load, ring, k0, k1, lane, acc);
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    mine[2 * t + (c & 1)][16 * m + g + 8 * (c >> 1)] = acc[m][0][c];
        } else {
            float acc[MT][NT][4] = {};
            dot<T, MT, NT, D>(a, f, load, ring, k0, k1, lane, acc);
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        mine[8 * j + 2 * t + (c & 1)][16 * m + g + 8 * (c >> 1)] = acc[m][j][c];
        }
        __syncthreads();
        for (int i = threadIdx.x; i < kRowsW * f.n; i += kThreads) {
            const int n = i & (kRowsW - 1), r = i / kRowsW;
            float sum = part[0][r][n];
#pragma unroll
            for (int w = 1; w < W; ++w)
                sum += part[w][r][n];
            if (n0 + n < a.N) {
                const int64_t o = static_cast<int64_t>(f.r0 + r) * a.N + n0 + n;
                if (a.y32)
                    static_cast<float *>(a.y)[o] = sum;
                else
                    static_cast<T *>(a.y)[o] = fp4::from_float<T>(sum);
            }
        }
        __syncthreads();
    }
    // rows outside every group, divided among the CTAs of a column of tiles
    for (int64_t i = static_cast<int64_t>(blockIdx.y) * kThreads + threadIdx.x; i < outside * kRowsW;
         i += static_cast<int64_t>(gridDim.y) * kThreads) {
        const int n = n0 + static_cast<int>(i & (kRowsW - 1));
        const int64_t j = i / kRowsW, r = j < first ? j : last + j - first;
        if (n < a.N) {
            if (a.y32)
                static_cast<float *>(a.y)[r * a.N + n] = 0.f;
            else
                static_cast<T *>(a.y)[r * a.N + n] = fp4::from_float<T>(0.f);
        }
    }
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int e = threadIdx.x; e < a.E; e += kThreads)
            ragged::report_bad(a.off, a.R, e, a.dev_status);
}

template <typename T, int W, int MT, int NT>
static moe_status_t launch(const Args &a, cudaStream_t s)
{
    static std::atomic<uint64_t> done{0};
    constexpr int bytes = W * kDepth * kStage<MT>;
    if (!smem_attr_once(done, reinterpret_cast<const void *>(gmm_awq_kernel<T, W, MT, NT>), bytes))
        return MOE_ERR_CUDA;
    const int64_t live = a.E < a.R ? a.E : a.R, most = 8 * NT, runs = (a.R + live * (most - 1)) / most;
    const dim3 grid(static_cast<unsigned>((a.N + 16 * MT - 1) / (16 * MT)), static_cast<unsigned>(runs < 65535 ? runs : 65535));
    return launch_pdl(gmm_awq_kernel<T, W, MT, NT>, grid, dim3(32 * W), bytes, s, a) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <typename T>
static moe_status_t run(const Args &a, cudaStream_t s)
{
    const int64_t live = a.E < a.R ? a.E : a.R;
    // 32 rows of w per CTA halve the work on x, where that leaves eight CTAs for every
    // SM: 512 rows over 128 experts 57.2 us, 74.5 with 16 rows; for 8 rows of 8 experts
    // (2.5 CTAs per SM) 8.7 us with 32 rows, 8.1 with 16
    const bool wide = live * ((a.N + 31) / 32) >= 8 * device_sm_count();
    // Groups per warp: 512 such rows take 33.0, 54.9, 65.5, 98.6 and 163.1 us with two
    // warps at K = 1024, 2048, 2560, 4096 and 7168, and 41.0, 61.4, 71.3, 102.6 and 164.1
    // with four; one row by 4096 x K takes 4.0, 5.5, 6.2, 10.1 and 15.9 with two and 3.5,
    // 4.2, 4.5, 6.6 and 9.5 with four.  (So few tiles with a K just below the border lose:
    // 9.1 us at K = 3584, 5.7 with four.)  Runs of up to 16 rows of x widen the weights
    // once where an expert has that many, and cost registers where R could not fill one of
    // 8.
    if (a.K >= 4096)
        return a.R <= 8 ? (wide ? launch<T, 4, 2, 1>(a, s) : launch<T, 4, 1, 1>(a, s))
                        : (wide ? launch<T, 4, 2, 2>(a, s) : launch<T, 4, 1, 2>(a, s));
    return a.R <= 8 ? (wide ? launch<T, 2, 2, 1>(a, s) : launch<T, 2, 1, 1>(a, s))
                    : (wide ? launch<T, 2, 2, 2>(a, s) : launch<T, 2, 1, 2>(a, s));
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
    if (w->E > ragged::kMaxExperts || R > ragged::kMaxSide || w->N > ragged::kMaxSide || w->K > gmm_awq::kMaxK ||
        !ragged::list_fits(w->E, R, 1, 8))
        return MOE_ERR_UNSUPPORTED;
    if (R == 0)
        return MOE_OK;
    if (!x || !y || !offsets || !w->q || !w->scale || !w->zero || !aligned(x, 16) || !aligned(y, 16) || !aligned(offsets, 4) ||
        !aligned(w->q, 16) || !aligned(w->scale, 16) || !aligned(w->zero, 16) || !aligned(dev_status, 4))
        return MOE_ERR_INVALID_ARG;
    const gmm_awq::Args a{x, static_cast<const uint32_t *>(w->q), static_cast<const __half *>(w->scale),
                          static_cast<const uint32_t *>(w->zero), offsets, y, dev_status, R, w->E, w->N, w->K, ydt == MOE_FP32};
    cudaStream_t s = as_stream(stream);
    return dt == MOE_BF16 ? gmm_awq::run<__nv_bfloat16>(a, s) : gmm_awq::run<__half>(a, s);
}
