// swiglu.cu -- the experts' activation with dropout, and its gradient, on rows
// [g | u] of the fused gate/up projection:
//
//   h  = f silu(g) u,      silu(g) = g s, s = 1 / (1 + exp(-g))
//   du = f dh silu(g),     dg = f dh u s (1 + g (1 - s))
//
// f is 0 for a dropped element and 65536 / (65536 - T) for a kept one, T = p
// 65536 rounded: the chance is T / 65536 and the factor is its own, so that the
// mean of f is 1.  The choice is made anew in both directions from a counter:
// element (r, i) takes the 16 bits i % 8 of Philox4x32 with 10 rounds (Salmon,
// Moraes, Dror, Shaw: "Parallel random numbers: as easy as 1, 2, 3", 2011) of the
// counter (i / 8, r, offset), key = seed, and is kept where they are not below T.
// So one generator call serves 8 elements, the unit of a thread's loads.
#include <type_traits>

#include "attr.h"
#include "common.cuh"
#include "fp4.cuh"
#include "gmm_common.cuh"
#include "ragged.cuh"

namespace moe {
namespace swiglu {

constexpr int kThreads = 256, kPerSm = 64;

// The generator's keys of the rounds and the offset, formed once per thread.
struct Rng {
    uint32_t k0[10], k1[10], o0, o1;
    __device__ __forceinline__ explicit Rng(const uint64_t *p)
    {
        const uint64_t seed = p[0], offset = p[1];
#pragma unroll
        for (uint32_t i = 0; i < 10; ++i) {
            k0[i] = static_cast<uint32_t>(seed) + i * 0x9E3779B9u;
            k1[i] = static_cast<uint32_t>(seed >> 32) + i * 0xBB67AE85u;
        }
        o0 = static_cast<uint32_t>(offset);
        o1 = static_cast<uint32_t>(offset >> 32);
    }
    __device__ __forceinline__ void draw(uint32_t column, uint32_t row, uint32_t (&v)[4]) const
    {
        uint32_t a = column, b = row, c = o0, d = o1;
#pragma unroll
        for (int i = 0; i < 10; ++i) {
            const uint64_t p0 = static_cast<uint64_t>(a) * 0xD2511F53u, p1 = static_cast<uint64_t>(c) * 0xCD9E8D57u;
            a = static_cast<uint32_t>(p1 >> 32) ^ b ^ k0[i];
            c = static_cast<uint32_t>(p0 >> 32) ^ d ^ k1[i];
            b = static_cast<uint32_t>(p1);
            d = static_cast<uint32_t>(p0);
        }
        v[0] = a;
        v[1] = b;
        v[2] = c;
        v[3] = d;
    }
};

// s and 1 - s from exp(-|g|), which does not overflow, and is subnormal rather than
// 0 far out.  FP32 tensors take the accurate functions.  For the 16-bit types 1 - s is
// off by 2^-24, which the gradient's 1 + g (1 - s) does not see.
template <typename T>
__device__ __forceinline__ void sigmoid(float g, float &s, float &c)
{
    if constexpr (sizeof(T) == 4) {
        const float t = expf(-fabsf(g)), r = 1.0f / (1.0f + t), q = t * r;
        s = g >= 0.f ? r : q;
        c = g >= 0.f ? q : r;
    } else {
        const float t = __expf(-fabsf(g));
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + t));
        s = g >= 0.f ? r : t * r;
        c = 1.0f - s;
    }
}

struct Args {
    const void *gu, *dh;
    const uint64_t *rng;
    void *out;                       // h, or the gradient of gu
    int64_t R, I;
    uint32_t units;                  // of 8 columns, of all rows
    uint32_t per_row, threshold;     // units of a row; T << 16
    uint32_t step, step_rows, step_units;    // units from a thread's one to its next, as rows and units of a row
    float factor;
};

// Whether each of a unit's 8 elements is kept.
template <bool DROP>
__device__ __forceinline__ void kept(const Args &a, const Rng &rng, uint32_t j, uint32_t r, bool (&keep)[8])
{
    if constexpr (DROP) {
        uint32_t v[4];
        rng.draw(j, r, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            keep[2 * i] = v[i] << 16 >= a.threshold;
            keep[2 * i + 1] = v[i] >= a.threshold;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            keep[i] = true;
    }
}

// A dropped element is 0 whatever g, u and dh hold.
template <typename T>
__device__ __forceinline__ float forward(float g, float u, bool keep, float f)
{
    float s, c;
    sigmoid<T>(g, s, c);
    return keep ? g * s * u * f : 0.f;
}

template <typename T>
__device__ __forceinline__ void backward(float g, float u, float dh, bool keep, float f, float &dg, float &du)
{
    float s, c;
    sigmoid<T>(g, s, c);
    const float d = dh * f;
    dg = keep ? s * fmaf(g, c, 1.0f) * u * d : 0.f;
    du = keep ? g * s * d : 0.f;
}

// 8 consecutive elements.
template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&x)[8])
{
    if constexpr (sizeof(T) == 4) {
        const float4 lo = __ldcs(reinterpret_cast<const float4 *>(p)), hi = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
        x[0] = lo.x, x[1] = lo.y, x[2] = lo.z, x[3] = lo.w;
        x[4] = hi.x, x[5] = hi.y, x[6] = hi.z, x[7] = hi.w;
    } else {
        const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (std::is_same<T, __half>::value)
                f16x2_to_float(w[i], x[2 * i], x[2 * i + 1]);
            else
                bf16x2_to_float(w[i], x[2 * i], x[2 * i + 1]);
        }
    }
}

template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&x)[8])
{
    if constexpr (sizeof(T) == 4) {
        __stcs(reinterpret_cast<float4 *>(p), make_float4(x[0], x[1], x[2], x[3]));
        __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
    } else {
        __stcs(reinterpret_cast<uint4 *>(p), make_uint4(gmm::pack2<T>(x[0], x[1]), gmm::pack2<T>(x[2], x[3]),
                                                        gmm::pack2<T>(x[4], x[5]), gmm::pack2<T>(x[6], x[7])));
    }
}

// Whole units at 16-byte accesses: a thread takes one unit after the other, each
// `step` further.  38400 x 2048 bf16, p = 0.3, takes 80.2 us forward (5.9 TB/s) and
// 111.9 us backward (7.0 TB/s; a part of the tensors is still in the L2 from call to
// call).  Backward is bound by HBM; forward, with the same generator for three fifths of
// the bytes, by both: DRAM at 66 % of its nominal rate, 75 % of the issue slots used.  With 16 CTAs per SM rather than 64 83.3 and 117.3; with a
// division per unit and the generator's keys formed anew 88.4 and 114.8.
template <typename T, bool DROP, bool BWD>
__global__ void __launch_bounds__(kThreads) swiglu_kernel(const Args a)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const uint64_t none[2] = {0, 0};
    const Rng rng(DROP ? a.rng : none);
    uint64_t at = static_cast<uint64_t>(blockIdx.x) * kThreads + threadIdx.x;
    uint32_t r = static_cast<uint32_t>(at) / a.per_row, j = static_cast<uint32_t>(at) - r * a.per_row;
    for (; at < a.units; at += a.step) {
        const int64_t h_at = static_cast<int64_t>(r) * a.I + 8 * static_cast<int64_t>(j);
        const T *g_at = static_cast<const T *>(a.gu) + h_at + static_cast<int64_t>(r) * a.I;
        float g[8], u[8], d[8];
        load8<T>(g_at, g);
        load8<T>(g_at + a.I, u);
        if constexpr (BWD)
            load8<T>(static_cast<const T *>(a.dh) + h_at, d);
        bool keep[8];
        kept<DROP>(a, rng, j, r, keep);
        if constexpr (BWD) {
            T *out = static_cast<T *>(a.out) + h_at + static_cast<int64_t>(r) * a.I;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                backward<T>(g[i], u[i], d[i], keep[i], a.factor, g[i], u[i]);
            store8<T>(out, g);
            store8<T>(out + a.I, u);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                g[i] = forward<T>(g[i], u[i], keep[i], a.factor);
            store8<T>(static_cast<T *>(a.out) + h_at, g);
        }
        r += a.step_rows;
        j += a.step_units;
        if (j >= a.per_row) {
            j -= a.per_row;
            ++r;
        }
    }
}

// Rows of any width and alignment: a warp takes 32 units of a row, element l + 32 i
// of them in lane l so that its accesses are neighbours; each lane makes the choice
// for one unit, and the others take it from there (777 x 1001 fp16 3.3 us forward and
// 4.8 backward; with a unit's elements in one lane 4.2 and 7.6).
template <typename T, bool DROP, bool BWD>
__global__ void __launch_bounds__(kThreads) swiglu_odd_kernel(const Args a)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const uint64_t none[2] = {0, 0};
    const Rng rng(DROP ? a.rng : none);
    const int lane = threadIdx.x & 31;
    const uint32_t blocks = (a.per_row + 31) / 32;                      // of 256 columns
    const uint64_t total = blocks * static_cast<uint64_t>(a.R), warps = static_cast<uint64_t>(gridDim.x) * (kThreads / 32);
    for (uint64_t at = static_cast<uint64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); at < total; at += warps) {
        const uint32_t r = static_cast<uint32_t>(at / blocks), b = static_cast<uint32_t>(at - static_cast<uint64_t>(r) * blocks);
        const int64_t col = 256 * static_cast<int64_t>(b) + lane, h_at = static_cast<int64_t>(r) * a.I + col;
        const T *g_at = static_cast<const T *>(a.gu) + h_at + static_cast<int64_t>(r) * a.I;
        float g[8], u[8], d[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool in = col + 32 * i < a.I;
            g[i] = in ? static_cast<float>(g_at[32 * i]) : 0.f;
            u[i] = in ? static_cast<float>(g_at[a.I + 32 * i]) : 0.f;
            d[i] = BWD && in ? static_cast<float>((static_cast<const T *>(a.dh) + h_at)[32 * i]) : 0.f;
        }
        bool keep[8];
        kept<DROP>(a, rng, 32 * b + lane, r, keep);
        uint32_t mine = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            mine |= keep[i] ? 1u << i : 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool k = !DROP || (__shfl_sync(0xffffffffu, mine, 4 * i + (lane >> 3)) >> (lane & 7) & 1u);
            if (BWD)
                backward<T>(g[i], u[i], d[i], k, a.factor, g[i], u[i]);
            else
                g[i] = forward<T>(g[i], u[i], k, a.factor);
        }
        T *out = static_cast<T *>(a.out) + h_at + (BWD ? static_cast<int64_t>(r) * a.I : 0);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (col + 32 * i < a.I) {
                out[32 * i] = fp4::from_float<T>(g[i]);
                if (BWD)
                    out[a.I + 32 * i] = fp4::from_float<T>(u[i]);
            }
    }
}

template <typename T, bool BWD>
static cudaError_t launch(Args &a, cudaStream_t s)
{
    const bool drop = a.threshold != 0, vec = a.I % 8 == 0 && aligned(a.gu, 16) && aligned(a.out, 16) && aligned(a.dh, 16);
    const int64_t wanted = vec ? (static_cast<int64_t>(a.units) + kThreads - 1) / kThreads
                               : (static_cast<int64_t>(a.per_row + 31) / 32 * a.R + kThreads / 32 - 1) / (kThreads / 32);
    const int64_t most = static_cast<int64_t>(device_sm_count()) * kPerSm;
    const dim3 grid(static_cast<unsigned>(wanted < most ? wanted : most)), block(kThreads);
    a.step = grid.x * kThreads;
    a.step_rows = a.step / a.per_row;
    a.step_units = a.step % a.per_row;
    auto k = vec ? (drop ? swiglu_kernel<T, true, BWD> : swiglu_kernel<T, false, BWD>)
                 : (drop ? swiglu_odd_kernel<T, true, BWD> : swiglu_odd_kernel<T, false, BWD>);
    return launch_pdl(k, grid, block, 0, s, a);
}

static moe_status_t call(const void *dh, const void *gu, int32_t dt, int32_t R, int32_t I, double p, const int64_t *rng,
                         void *out, bool bwd, void *stream)
{
    if (R < 0 || I < 1 || !(p >= 0.0 && p < 1.0))
        return MOE_ERR_INVALID_ARG;
    if (dt != MOE_BF16 && dt != MOE_FP16 && dt != MOE_FP32)
        return MOE_ERR_UNSUPPORTED;
    const uint32_t threshold = static_cast<uint32_t>(p * 65536.0 + 0.5);
    if (threshold > 65535)                            // nothing would be kept
        return MOE_ERR_INVALID_ARG;
    const uint32_t per_row = (static_cast<uint32_t>(I) + 7) / 8;
    if (I > ragged::kMaxSide || static_cast<uint32_t>(R) > UINT32_MAX / per_row)
        return MOE_ERR_UNSUPPORTED;
    if (R == 0)
        return MOE_OK;
    const size_t size = dt == MOE_FP32 ? 4 : 2;
    if (!gu || !out || (bwd && !dh) || (threshold && !rng) || !aligned(gu, size) || !aligned(out, size) ||
        !aligned(dh, size) || !aligned(rng, 8))
        return MOE_ERR_INVALID_ARG;
    Args a{gu, dh, reinterpret_cast<const uint64_t *>(rng), out, R, I, static_cast<uint32_t>(R) * per_row, per_row,
           threshold << 16, 0, 0, 0, static_cast<float>(65536.0 / (65536 - threshold))};
    cudaStream_t s = as_stream(stream);
    cudaError_t e;
    if (dt == MOE_BF16)
        e = bwd ? launch<__nv_bfloat16, true>(a, s) : launch<__nv_bfloat16, false>(a, s);
    else if (dt == MOE_FP16)
        e = bwd ? launch<__half, true>(a, s) : launch<__half, false>(a, s);
    else
        e = bwd ? launch<float, true>(a, s) : launch<float, false>(a, s);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace swiglu
}  // namespace moe

using namespace moe;

MOE_API moe_status_t moe_swiglu_dropout(const void *gu, int32_t dt, int32_t R, int32_t I, double p, const int64_t *rng,
                                        void *h, void *stream)
{
    return swiglu::call(nullptr, gu, dt, R, I, p, rng, h, false, stream);
}

MOE_API moe_status_t moe_swiglu_dropout_bwd(const void *dh, const void *gu, int32_t dt, int32_t R, int32_t I, double p,
                                            const int64_t *rng, void *dgu, void *stream)
{
    return swiglu::call(dh, gu, dt, R, I, p, rng, dgu, true, stream);
}
