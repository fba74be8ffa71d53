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
#include "common.cuh"
#include "fp4.cuh"
#include "gmm_common.cuh"
#include "ragged.cuh"

namespace moe {
namespace swiglu {

constexpr int kThreads = 256;

// The generator's key and offset, read once per thread.
struct Rng {
    uint32_t k0, k1, o0, o1;
    __device__ __forceinline__ explicit Rng(const uint64_t *p)
    {
        const uint64_t seed = p[0], offset = p[1];
        k0 = static_cast<uint32_t>(seed);
        k1 = static_cast<uint32_t>(seed >> 32);
        o0 = static_cast<uint32_t>(offset);
        o1 = static_cast<uint32_t>(offset >> 32);
    }
    __device__ __forceinline__ void draw(uint32_t column, uint32_t row, uint32_t (&v)[4]) const
    {
        uint32_t a = column, b = row, c = o0, d = o1, ka = k0, kb = k1;
#pragma unroll
        for (int i = 0; i < 10; ++i) {
            const uint64_t p0 = static_cast<uint64_t>(a) * 0xD2511F53u, p1 = static_cast<uint64_t>(c) * 0xCD9E8D57u;
            a = static_cast<uint32_t>(p1 >> 32) ^ b ^ ka;
            c = static_cast<uint32_t>(p0 >> 32) ^ d ^ kb;
            b = static_cast<uint32_t>(p1);
            d = static_cast<uint32_t>(p0);
            ka += 0x9E3779B9u;
            kb += 0xBB67AE85u;
        }
        v[0] = a;
        v[1] = b;
        v[2] = c;
        v[3] = d;
    }
};

// s and 1 - s, each to its own precision: from exp(-|g|), which neither
// overflows nor cancels.  FP32 tensors take the accurate functions.
template <typename T>
__device__ __forceinline__ void sigmoid(float g, float &s, float &c)
{
    float t, r;
    if constexpr (sizeof(T) == 4) {
        t = expf(-fabsf(g));
        r = 1.0f / (1.0f + t);
    } else {
        t = __expf(-fabsf(g));
        r = __fdividef(1.0f, 1.0f + t);
    }
    const float q = t * r;
    s = g >= 0.f ? r : q;
    c = g >= 0.f ? q : r;
}

struct Args {
    const void *gu, *dh;
    const uint64_t *rng;
    void *out;                       // h, or the gradient of gu
    int64_t R, I;
    uint32_t units;                  // of 8 columns, of all rows
    uint32_t per_row, threshold;
    float factor;
};

// The factors of a unit's 8 elements.
template <bool DROP>
__device__ __forceinline__ void factors(const Args &a, const Rng &rng, uint32_t j, uint32_t r, float (&f)[8])
{
    if constexpr (DROP) {
        uint32_t v[4];
        rng.draw(j, r, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = (v[i] & 0xFFFFu) >= a.threshold ? a.factor : 0.f;
            f[2 * i + 1] = (v[i] >> 16) >= a.threshold ? a.factor : 0.f;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = 1.f;
    }
}

// A dropped element is 0 whatever g, u and dh hold.
template <typename T>
__device__ __forceinline__ float forward(float g, float u, float f)
{
    float s, c;
    sigmoid<T>(g, s, c);
    return f == 0.f ? 0.f : g * s * u * f;
}

template <typename T>
__device__ __forceinline__ void backward(float g, float u, float dh, float f, float &dg, float &du)
{
    float s, c;
    sigmoid<T>(g, s, c);
    const float d = dh * f;
    dg = f == 0.f ? 0.f : s * fmaf(g, c, 1.0f) * u * d;
    du = f == 0.f ? 0.f : g * s * d;
}

// 8 consecutive elements, whole (VEC: 16-byte accesses) or the first n of them.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T *p, int n, float (&x)[8])
{
    if constexpr (VEC) {
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
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = i < n ? static_cast<float>(p[i]) : 0.f;
    }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T *p, int n, const float (&x)[8])
{
    if constexpr (VEC) {
        if constexpr (sizeof(T) == 4) {
            __stcs(reinterpret_cast<float4 *>(p), make_float4(x[0], x[1], x[2], x[3]));
            __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
        } else {
            __stcs(reinterpret_cast<uint4 *>(p), make_uint4(gmm::pack2<T>(x[0], x[1]), gmm::pack2<T>(x[2], x[3]),
                                                            gmm::pack2<T>(x[4], x[5]), gmm::pack2<T>(x[6], x[7])));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n)
                p[i] = fp4::from_float<T>(x[i]);
    }
}

template <typename T, bool DROP, bool VEC, bool BWD>
__global__ void __launch_bounds__(kThreads) swiglu_kernel(const Args a)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const uint64_t none[2] = {0, 0};
    const Rng rng(DROP ? a.rng : none);
    const T *gu = static_cast<const T *>(a.gu);
    const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
    for (int64_t at = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; at < a.units; at += step) {
        const uint32_t u = static_cast<uint32_t>(at), r = u / a.per_row, j = u - r * a.per_row;
        const int n = static_cast<int>(min(a.I - 8 * static_cast<int64_t>(j), static_cast<int64_t>(8)));
        const int64_t row = static_cast<int64_t>(r) * 2 * a.I, g_at = row + 8 * static_cast<int64_t>(j), u_at = g_at + a.I;
        const int64_t h_at = static_cast<int64_t>(r) * a.I + 8 * static_cast<int64_t>(j);
        float g[8], v[8], f[8], d[8];
        load8<T, VEC>(gu + g_at, n, g);
        load8<T, VEC>(gu + u_at, n, v);
        if constexpr (BWD)
            load8<T, VEC>(static_cast<const T *>(a.dh) + h_at, n, d);
        factors<DROP>(a, rng, j, r, f);
        if constexpr (BWD) {
            float dg[8], du[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                backward<T>(g[i], v[i], d[i], f[i], dg[i], du[i]);
            store8<T, VEC>(static_cast<T *>(a.out) + g_at, n, dg);
            store8<T, VEC>(static_cast<T *>(a.out) + u_at, n, du);
        } else {
            float h[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                h[i] = forward<T>(g[i], v[i], f[i]);
            store8<T, VEC>(static_cast<T *>(a.out) + h_at, n, h);
        }
    }
}

template <typename T, bool BWD>
static cudaError_t launch(const Args &a, cudaStream_t s)
{
    const bool vec = a.I % 8 == 0 && aligned(a.gu, 16) && aligned(a.out, 16) && aligned(a.dh, 16);
    const int64_t blocks = (static_cast<int64_t>(a.units) + kThreads - 1) / kThreads;
    const dim3 grid(static_cast<unsigned>(blocks < 152 * 64 ? blocks : 152 * 64)), block(kThreads);
    const bool drop = a.threshold != 0;
    auto k = drop ? (vec ? swiglu_kernel<T, true, true, BWD> : swiglu_kernel<T, true, false, BWD>)
                  : (vec ? swiglu_kernel<T, false, true, BWD> : swiglu_kernel<T, false, false, BWD>);
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
    const Args a{gu, dh, reinterpret_cast<const uint64_t *>(rng), out, R, I, static_cast<uint32_t>(R) * per_row, per_row,
                 threshold, static_cast<float>(65536.0 / (65536 - threshold))};
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
