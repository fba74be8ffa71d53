// host_products.cu -- host-side arithmetic of the ragged and 4-bit products
// (top_moe_expert_gb300/csrc), run on the CPU for the CPU tests.
#include <cstdint>
#include "fp4.cuh"

extern "C" void fp4_factors(int64_t n, const float *a, const float *b, float *f, float *g)
{
    for (int64_t i = 0; i < n; ++i)
        moe::fp4::factors(a[i], b[i], f[i], g[i]);
}
