// host_products.cu -- host-side arithmetic of the ragged and 4-bit products
// (top_moe_expert_gb300/csrc), run on the CPU for the CPU tests.
#include <cstdint>
#include "fp4.cuh"
#include "ragged.cuh"

extern "C" void fp4_factors(int64_t n, const float *a, const float *b, float *f, float *g)
{
    for (int64_t i = 0; i < n; ++i)
        moe::fp4::factors(a[i], b[i], f[i], g[i]);
}

// The index of the first poll at which the limit has expired, n if none.
extern "C" int64_t limit_expires(int64_t n, const int64_t *now, const int32_t *progress, int64_t limit)
{
    moe::ragged::Limit l{now[0], progress[0]};
    for (int64_t i = 0; i < n; ++i)
        if (l.expired(now[i], progress[i], limit))
            return i;
    return n;
}
