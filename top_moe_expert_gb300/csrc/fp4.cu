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
#include "ragged.cuh"

namespace moe {
namespace fp4 {

// Both kernels are streams.  A lane takes 8 consecutive elements at a time, so
// that a warp's loads and stores are whole lines whatever the alignment past 16
// bytes, and has four such units under way; a block's two or four lanes agree
// on its amax by shuffles.  (32 elements per lane, without shuffles but with
// half-used sectors, took 408 us for 196608 x 2048 bf16 both ways.)
constexpr int kUnits = 4;

template <typename VT>
struct Unit {
    uint4 w[sizeof(VT) / 2];
};

// 8 FP32 values in one 32-byte access where the array starts on 32 bytes: two
// of 16 bytes each leave half of every sector to the next instruction (181 us
// rather than 142 for 98304 x 2048 values back).
__device__ __forceinline__ void ld32(const void *p, uint4 &a, uint4 &b)
{
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w) : "l"(p));
}

__device__ __forceinline__ void st32(void *p, const uint4 &a, const uint4 &b)
{
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w) : "memory");
}

// alpha of a row and 1 / (6 alpha), kept while the row's run stays the same.
// (The dequantizer loads alpha anew for each unit: without the division, a
// branch between its loads costs more, 199 us against 160.)
struct Alpha {
    const float *alpha;
    uint32_t rows_per, at;
    float a, g;
    __device__ __forceinline__ Alpha(const float *p, uint32_t per) : alpha(p), rows_per(per), at(~0u), a(1.f), g(0.f) {}
    __device__ __forceinline__ void row(uint32_t r)
    {
        const uint32_t i = rows_per ? r / rows_per : 0;            // 0: one alpha for all rows
        if (i != at) {
            at = i;
            a = alpha[i];
            g = 1.0f / (6.0f * a);
        }
    }
};

// A unit's largest magnitude, as the bits of its type (two halves of a word for
// the 16-bit types, to be folded after the shuffles), and its values.
__device__ __forceinline__ uint32_t amax_bits(const Unit<float> &u)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        m = max(m, max(max(u.w[i].x & 0x7FFFFFFFu, u.w[i].y & 0x7FFFFFFFu), max(u.w[i].z & 0x7FFFFFFFu, u.w[i].w & 0x7FFFFFFFu)));
    return m;
}

template <typename VT>
__device__ __forceinline__ uint32_t amax_bits(const Unit<VT> &u)
{
    constexpr uint32_t k = 0x7FFF7FFFu;
    return __vmaxu2(__vmaxu2(u.w[0].x & k, u.w[0].y & k), __vmaxu2(u.w[0].z & k, u.w[0].w & k));
}

template <typename VT>
__device__ __forceinline__ uint32_t amax_join(uint32_t a, uint32_t b)
{
    return sizeof(VT) == 4 ? max(a, b) : __vmaxu2(a, b);
}

// The FP32 bits of an amax.
template <typename VT>
__device__ __forceinline__ uint32_t amax_float(uint32_t a)
{
    if constexpr (sizeof(VT) == 4)
        return a;
    a = max(a & 0xFFFFu, a >> 16);
    if constexpr (std::is_same<VT, __half>::value)
        return __float_as_uint(__half2float(__ushort_as_half(static_cast<uint16_t>(a))));
    return a << 16;
}

__device__ __forceinline__ void unpack(const Unit<float> &u, float (&x)[8])
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        x[4 * i] = __uint_as_float(u.w[i].x);
        x[4 * i + 1] = __uint_as_float(u.w[i].y);
        x[4 * i + 2] = __uint_as_float(u.w[i].z);
        x[4 * i + 3] = __uint_as_float(u.w[i].w);
    }
}

template <typename VT>
__device__ __forceinline__ void unpack(const Unit<VT> &u, float (&x)[8])
{
    const uint32_t w[4] = {u.w[0].x, u.w[0].y, u.w[0].z, u.w[0].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (std::is_same<VT, __half>::value)
            f16x2_to_float(w[j], x[2 * j], x[2 * j + 1]);
        else
            bf16x2_to_float(w[j], x[2 * j], x[2 * j + 1]);
    }
}

// 8 values onto the E2M1 grid: one 32-bit word of codes.
__device__ __forceinline__ uint32_t codes8(const float (&x)[8], float inv)
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

// Row and 32-element piece of the row of a lane's units: one division for the
// first, steps of 8 pieces (32 units) after it.
struct Place {
    uint32_t row, piece;
    __device__ __forceinline__ Place(uint32_t p, uint32_t nq) : row(p / nq), piece(p - row * nq) {}
    __device__ __forceinline__ void step(uint32_t nq)
    {
        piece += 8;
        while (piece >= nq) {
            piece -= nq;
            ++row;
        }
    }
};

template <typename VT, int FMT>
__global__ void __launch_bounds__(256)
quantize_kernel(const VT *v, int64_t units, uint32_t nq, int Ks, const float *alpha,
                uint32_t rows_per_alpha, bool wide, uint32_t *q, uint8_t *s)
{
    // chained by programmatic dependent launch
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    Alpha al(alpha, rows_per_alpha);
    constexpr int kLanes = block_of(FMT) / 8, kPer = 32 / block_of(FMT);
    const int lane = threadIdx.x & 31;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
    for (int64_t base = (blockIdx.x * static_cast<int64_t>(blockDim.x >> 5) + (threadIdx.x >> 5)) * (32 * kUnits); base < units;
         base += warps * (32 * kUnits)) {
        Unit<VT> in[kUnits];
#pragma unroll
        for (int j = 0; j < kUnits; ++j) {
            const int64_t u = base + 32 * j + lane;
#pragma unroll
            for (int k = 0; k < static_cast<int>(sizeof(VT) / 2); ++k)
                in[j].w[k] = make_uint4(0, 0, 0, 0);
            if (u < units) {
                const uint4 *p = reinterpret_cast<const uint4 *>(v) + u * (sizeof(VT) / 2);
                if (sizeof(VT) == 4 && wide) {
                    ld32(p, in[j].w[0], in[j].w[sizeof(VT) / 2 - 1]);
                } else {
#pragma unroll
                    for (int k = 0; k < static_cast<int>(sizeof(VT) / 2); ++k)
                        in[j].w[k] = ld_once_u4(p + k);
                }
            }
        }
        Place at(static_cast<uint32_t>((base + lane) >> 2), nq);
#pragma unroll
        for (int j = 0; j < kUnits; ++j, at.step(nq)) {
            const int64_t u = base + 32 * j + lane;
            uint32_t m = amax_bits(in[j]);
#pragma unroll
            for (int o = 1; o < kLanes; o <<= 1)
                m = amax_join<VT>(m, __shfl_xor_sync(0xffffffffu, m, o));
            m = amax_float<VT>(m);
            if (u < units) {
                float inv;
                uint32_t byte;
                if constexpr (FMT == MOE_FP4_NVFP4) {
                    al.row(at.row);
                    byte = block_scale_nv(m, al.a, al.g, inv);
                } else {
                    byte = block_scale_mx(m, inv);
                }
                float x[8];
                unpack(in[j], x);
                q[u] = m >= 0x7F800000u ? 0u : codes8(x, inv);
                if ((lane & (kLanes - 1)) == 0) {
                    uint8_t *row = s + static_cast<int64_t>(at.row) * Ks;
                    const int b = at.piece * kPer + (kPer == 2 ? (lane >> 1) & 1 : 0);
                    row[b] = static_cast<uint8_t>(byte);
                    if (b == static_cast<int>(nq) * kPer - 1)      // the last block zeroes the row's padding
                        for (int i = b + 1; i < Ks; ++i)
                            row[i] = 0;
                }
            }
        }
    }
}

template <typename VT, int FMT>
__global__ void __launch_bounds__(256)
dequantize_kernel(const uint32_t *q, const uint8_t *s, int64_t units, uint32_t nq, int Ks,
                  const float *alpha, uint32_t rows_per_alpha, bool wide, VT *v)
{
    // chained by programmatic dependent launch
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    constexpr int kPer = 32 / block_of(FMT);
    const int lane = threadIdx.x & 31;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
    for (int64_t base = (blockIdx.x * static_cast<int64_t>(blockDim.x >> 5) + (threadIdx.x >> 5)) * (32 * kUnits); base < units;
         base += warps * (32 * kUnits)) {
        uint32_t c[kUnits];
        float f[kUnits], al[kUnits];
        Place at(static_cast<uint32_t>((base + lane) >> 2), nq);
#pragma unroll
        for (int j = 0; j < kUnits; ++j, at.step(nq)) {
            const int64_t u = base + 32 * j + lane;
            if (u < units) {
                c[j] = __ldcs(q + u);
                f[j] = scale_value<FMT>(s[static_cast<int64_t>(at.row) * Ks + at.piece * kPer + (kPer == 2 ? (lane >> 1) & 1 : 0)]);
                al[j] = FMT == MOE_FP4_NVFP4 ? alpha[rows_per_alpha ? at.row / rows_per_alpha : 0u] : 1.f;
            }
        }
#pragma unroll
        for (int j = 0; j < kUnits; ++j) {
            const int64_t u = base + 32 * j + lane;
            if (u < units) {
                float x[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 e = e2m1_values((c[j] >> (8 * i)) & 0xFFu);
                    x[2 * i] = e.x * f[j] * al[j];
                    x[2 * i + 1] = e.y * f[j] * al[j];
                }
                uint4 *o = reinterpret_cast<uint4 *>(v) + u * (sizeof(VT) / 2);
                if constexpr (sizeof(VT) == 4) {
                    const uint4 lo = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
                    const uint4 hi = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
                    if (wide) {
                        st32(o, lo, hi);
                    } else {
                        __stcs(o, lo);
                        __stcs(o + 1, hi);
                    }
                } else {
                    __stcs(o, make_uint4(gmm::pack2<VT>(x[0], x[1]), gmm::pack2<VT>(x[2], x[3]), gmm::pack2<VT>(x[4], x[5]),
                                         gmm::pack2<VT>(x[6], x[7])));
                }
            }
        }
    }
}

// One warp takes 32 * kUnits units of 8 elements.
static int grid_of(int64_t units)
{
    const int64_t blocks = (units + 32 * kUnits * 8 - 1) / (32 * kUnits * 8);
    return static_cast<int>(blocks < 152 * 64 ? blocks : 152 * 64);
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
    if (K > ragged::kMaxSide || rows > UINT32_MAX / (K / 32))
        return MOE_ERR_UNSUPPORTED;
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
    const int64_t units = rows * (K / 8);
    cudaError_t e = cudaSuccess;
    by_type(vdt, [&](auto t) {
        using T = decltype(t);
        auto k = fmt == MOE_FP4_NVFP4 ? quantize_kernel<T, MOE_FP4_NVFP4> : quantize_kernel<T, MOE_FP4_MXFP4>;
        e = launch_pdl(k, dim3(grid_of(units)), dim3(256), 0, as_stream(stream), static_cast<const T *>(v), units,
                       static_cast<uint32_t>(K / 32), scale_cols(K, fmt), alpha,
                       groups == 1 ? 0u : static_cast<uint32_t>(rows / groups), aligned(v, 32),
                       reinterpret_cast<uint32_t *>(q), s);
    });
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

MOE_API moe_status_t moe_fp4_dequantize(const uint8_t *q, const uint8_t *s, int64_t rows, int32_t K, int32_t fmt,
                                        const float *alpha, int64_t groups, void *v, int32_t vdt, void *stream)
{
    const moe_status_t st = check(v, vdt, rows, K, fmt, alpha, groups, q, s);
    if (st != MOE_OK || rows == 0)
        return st;
    const int64_t units = rows * (K / 8);
    cudaError_t e = cudaSuccess;
    by_type(vdt, [&](auto t) {
        using T = decltype(t);
        auto k = fmt == MOE_FP4_NVFP4 ? dequantize_kernel<T, MOE_FP4_NVFP4> : dequantize_kernel<T, MOE_FP4_MXFP4>;
        e = launch_pdl(k, dim3(grid_of(units)), dim3(256), 0, as_stream(stream), reinterpret_cast<const uint32_t *>(q), s, units,
                       static_cast<uint32_t>(K / 32), scale_cols(K, fmt), alpha,
                       groups == 1 ? 0u : static_cast<uint32_t>(rows / groups), aligned(v, 32), static_cast<T *>(v));
    });
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
