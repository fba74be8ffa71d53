// ragged.cuh -- rows grouped by expert: offsets[e] .. offsets[e+1] are the
// rows of expert e among R rows, of any count, zero among them.
#pragma once

#include "common.cuh"

namespace moe {
namespace ragged {

constexpr int kMaxExperts = 1024;
constexpr int kMaxSide = INT32_MAX - 1023;         // of a matrix, so that rounding a side up to a tile stays in 32 bits
constexpr int kMaxTiles = kMaxSide;                // so that a step past the last does too

// Whether the list of tiles (mt x ceil(rows / nt) for each expert) counts in 32
// bits whatever the offsets hold: a group has at most R rows.
inline bool list_fits(int E, int R, int64_t mt, int nt) { return mt * E <= kMaxTiles / (R / nt + 1); }

// Whether offsets are what the contract says; a call reports it once.
__device__ __forceinline__ void report_bad(const int32_t *off, int R, int e, int32_t *dev_status)
{
    if (dev_status && (off[e] < 0 || off[e] > off[e + 1] || off[e + 1] > R || (e == 0 && off[0] != 0)))
        atomicCAS(dev_status + 1, 0, static_cast<int32_t>(MOE_ERR_BOUNDS));
}

// The persistent kernels' list of tiles, in shared memory: expert e's first
// row, and the number of tiles before its own (mt tiles across for every nt
// rows); tiles[E] is the total.  Every CTA makes its own.  Offsets are device
// data: they are clamped to [0, R] and a group that would run backwards is
// empty, so no value of them takes an access out of its buffer.
struct List {
    int lo[kMaxExperts + 1], tiles[kMaxExperts + 1];
    int warp_sum[32];
    __device__ __forceinline__ int rows(int e) const { return max(lo[e + 1] - lo[e], 0); }
};

__device__ __forceinline__ void make_list(List &l, const int32_t *off, int E, int R, int mt, int nt)
{
    const int per = (E + blockDim.x - 1) / blockDim.x;
    const int e0 = min(static_cast<int>(threadIdx.x) * per, E), e1 = min(e0 + per, E);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int sum = 0;
    for (int e = e0; e < e1; ++e) {
        l.lo[e] = min(max(off[e], 0), R);
        if (e == E - 1)
            l.lo[E] = min(max(off[E], 0), R);
    }
    __syncthreads();
    for (int e = e0; e < e1; ++e)
        sum += mt * ((l.rows(e) + nt - 1) / nt);
    int run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o)
            run += v;
    }
    if (lane == 31)
        l.warp_sum[warp] = run;
    __syncthreads();
    int at = run - sum;
    for (int w = 0; w < warp; ++w)
        at += l.warp_sum[w];
    for (int e = e0; e < e1; ++e) {
        l.tiles[e] = at;
        at += mt * ((l.rows(e) + nt - 1) / nt);
    }
    if (e1 == E && e0 < E)
        l.tiles[E] = at;
    __syncthreads();
}

// The expert of tile t < tiles[E].
__device__ __forceinline__ int expert_of(const List &l, int E, int t)
{
    int a = 0, b = E;                       // tiles[a] <= t < tiles[b]
    while (b - a > 1) {
        const int m = (a + b) >> 1;
        if (l.tiles[m] <= t)
            a = m;
        else
            b = m;
    }
    return a;
}

// The place of the at-th tile of a grid of n_mt x n_nt tiles: bands of kBand tiles
// along mt, each walked along nt, so that the tiles that run at the same time
// form a near-square of the grid and share their operands' rows in the L2 (one
// product of 8192 x 8192 x 8192 in bf16: 567 us, 611 along mt first; at half and
// at twice the band 582 and 579).
constexpr int kBand = 8;
__host__ __device__ __forceinline__ void place(int at, int n_mt, int n_nt, int &mt, int &nt)
{
    const int band = at / (kBand * n_nt), left = n_mt - band * kBand;
    const int width = left < kBand ? left : kBand;
    at -= band * kBand * n_nt;
    nt = at / width;
    mt = band * kBand + at - nt * width;
}

// The limit of a wait for what another role brings after an unknown amount of
// work: it runs from the last time that role was seen to have moved on.
struct Limit {
    long long since;
    int seen;
    __host__ __device__ __forceinline__ bool expired(long long now, int progress, long long limit)
    {
        if (progress != seen) {
            seen = progress;
            since = now;
        }
        return now - since > limit;
    }
};

}  // namespace ragged
}  // namespace moe
