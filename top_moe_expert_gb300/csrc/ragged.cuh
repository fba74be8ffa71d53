// ragged.cuh -- rows grouped by expert: offsets[e] .. offsets[e+1] are the
// rows of expert e among R rows, of any count, zero among them.
#pragma once

#include "common.cuh"

namespace moe {
namespace ragged {

constexpr int kMaxExperts = 1024;

// Rows [lo, hi) of expert e.  offsets are device data: they are clamped to
// [0, R] and a group that would run backwards is empty, so no value of them
// takes an access out of its buffer.
__device__ __forceinline__ void group(const int32_t *__restrict__ off, int e, int R, int &lo, int &hi)
{
    lo = min(max(off[e], 0), R);
    hi = max(min(off[e + 1], R), lo);
}

// Whether offsets are what the contract says; a call reports it once.
__device__ __forceinline__ void report_bad(const int32_t *__restrict__ off, int E, int R, int e, int32_t *dev_status)
{
    if (dev_status && (off[e] < 0 || off[e] > off[e + 1] || off[e + 1] > R || (e == 0 && off[0] != 0)))
        atomicCAS(dev_status + 1, 0, static_cast<int32_t>(MOE_ERR_BOUNDS));
}

}  // namespace ragged
}  // namespace moe
