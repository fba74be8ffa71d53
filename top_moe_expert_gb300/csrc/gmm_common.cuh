// gmm_common.cuh -- epilogue pieces of the ragged grouped products.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "tc_pair.cuh"

namespace moe {
namespace gmm {

template <typename OT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    if constexpr (sizeof(OT) == 4) {
        return 0;
    } else if constexpr (std::is_same<OT, __half>::value) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

// 32 accumulator columns (rows of y or dx) of this lane's output element:
// neighbouring lanes exchange halves so that each stores two elements of one
// row, 64 contiguous bytes per row and warp.  f, g: factors of every element,
// applied in that order.
template <typename OT>
__device__ __forceinline__ void store_rows(const uint32_t (&v)[32], OT *out, int64_t ld, int m, int M, int n, int lane,
                                           float f = 1.f, float g = 1.f)
{
    if constexpr (sizeof(OT) == 4) {
        if (m < M) {
#pragma unroll
            for (int c = 0; c < 32; ++c)
                if (c < n)
                    out[c * ld + m] = __uint_as_float(v[c]) * f * g;
        }
    } else {
        const int odd = lane & 1;
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
            const uint32_t own = pack2<OT>(__uint_as_float(v[c]) * f * g, __uint_as_float(v[c + 1]) * f * g);
            const uint32_t other = __shfl_xor_sync(0xffffffffu, own, 1);
            const uint32_t w = odd ? __byte_perm(other, own, 0x7632) : __byte_perm(own, other, 0x5410);
            if (m < M && c + odd < n)
                *reinterpret_cast<uint32_t *>(out + (c + odd) * ld + (m & ~1)) = w;
        }
    }
}

// The same for 32 whole rows, through a staging tile of this warp's and TMA: 32
// rows of the warp's 32 elements (64 or 128 bytes, swizzled so that the warp's
// words of a row or two fall into different banks).  tiles: 4096 bytes; m0:
// the warp's first element, r0 the first row.
template <typename OT>
__device__ __forceinline__ void drain_rows(const uint32_t (&v)[32], uint8_t *tiles, int &flip, const CUtensorMap *map, int m0,
                                           int r0, int M, int lane, float f = 1.f, float g = 1.f)
{
    if constexpr (sizeof(OT) == 4) {
        tc::bulk_wait_read<0>();
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 32; ++c)
            *reinterpret_cast<float *>(tiles + c * 128 + ((lane * 4) ^ ((c & 7) << 4))) = __uint_as_float(v[c]) * f * g;
    } else {
        tiles += flip * 2048;
        flip ^= 1;
        tc::bulk_wait_read<1>();
        __syncwarp();
        const int odd = lane & 1;
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
            const uint32_t own = pack2<OT>(__uint_as_float(v[c]) * f * g, __uint_as_float(v[c + 1]) * f * g);
            const uint32_t other = __shfl_xor_sync(0xffffffffu, own, 1);
            const uint32_t w = odd ? __byte_perm(other, own, 0x7632) : __byte_perm(own, other, 0x5410);
            *reinterpret_cast<uint32_t *>(tiles + (c + odd) * 64 + (((lane & ~1) * 2) ^ (((c >> 1) & 3) << 4))) = w;
        }
    }
    tc::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
        if (m0 < M)
            tc::tma_store_2d(map, tc::smem_u32(tiles), m0, r0);
        tc::bulk_commit();
    }
}

}  // namespace gmm
}  // namespace moe
