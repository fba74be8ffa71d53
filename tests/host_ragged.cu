// host_ragged.cu -- the order of the grouped products' tiles (ragged::place in
// top_moe_expert_gb300/csrc/ragged.cuh), run on the CPU for the CPU tests.
#include <cstdint>
#include "ragged.cuh"

extern "C" void place_all(int n_mt, int n_nt, int32_t *out)
{
    for (int at = 0; at < n_mt * n_nt; ++at) {
        int mt, nt;
        moe::ragged::place(at, n_mt, n_nt, mt, nt);
        out[2 * at] = mt;
        out[2 * at + 1] = nt;
    }
}
