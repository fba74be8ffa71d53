// gmm_fp4.cu -- products of rows grouped by expert with the experts'
// matrices, both NVFP4 or both MXFP4:
//   y[r][n] = a_x a_w[e] sum over blocks of Sx Sw (sum in the block of cx cw)
// with E2M1 codes c, a scale S per block along K and, for NVFP4, the two
// constants.  Sums are FP32 on the tensor cores, rounded once.
//
// The structure of gmm.cu on tcgen05 kind::mxf4nvf4: one persistent kernel, two
// CTAs per tile of 256 rows of w (128 each) x 192 (or 128) rows of x (half each),
// a stage of 256 along K (128 bytes of codes a row, 4 MMAs of 64).  192 rather
// than 256 rows leave tensor memory for two accumulators and two stages of
// scales.
//
// Scales lie in memory row by row; the MMA wants them in tensor memory with a
// row's 4 bytes in lane row % 32, column row / 32.  Groups start at any row, so
// that arrangement cannot be made beforehand for x: 32 natural bytes of each
// row (a slot: 512 elements of NVFP4, 1024 of MXFP4) come by TMA, a warp turns
// them into the arrangement in place (a 4 x 4 transpose of words in registers;
// a lane holds rows l, l + 32, l + 64, l + 96), and tcgen05.cp copies a stage's
// part into every quadrant of tensor memory.  TMA is paid by the row: slots of
// a stage's 16 bytes took 261 us at 8192 x 8192 x 8192 (NVFP4), of 64 bytes
// with the room for only two of them 183 us, five of 32 bytes 164 us.
// Both CTAs hold the scales of all 192 rows of x and of their own 128 of w.
//
// The accumulator does not round to nearest (gmm.cu): each MMA of 64 along K can
// lose 2^-23 of the sum.  For quantized normal values little of that adds up (3e-8
// to 4e-7 at K = 7168), for values of one sign with scales over the whole range it
// does: 3.9e-6 at K = 7168, 1.5e-5 at 32768, 5.3e-5 at 131072.  So the sum ends
// every kSpan steps and the parts are added in registers, rounded to nearest, where
// K is past kLong (FP32 results) or kLong16 (16-bit ones, whose own rounding is
// 2^-9 or 2^-12).  Parts need the tiles of 128 rows, whose sums fit the registers:
// with many rows 220 us rather than 180 (8192 rows over 4 experts of 4096 x 16384,
// NVFP4; MXFP4 189 and 170), with few the time of one accumulation.
//
// Roles: warp 0 loads codes, warp 2 loads scales, warps 8..10 arrange them (w,
// the first 128 rows of x, the rest) and warp 3 tells the leader, whose warp 1
// issues copies and MMAs; warps 4..7 drain the accumulators.  Every wait is
// bounded, and an expired one is reported, as in gmm.cu.
//
// Bound by feeding the tiles: 168 us at 8192 x 8192 x 8192 (NVFP4; MXFP4 151) in
// runs of a few calls, 128 us with every copy left out; back to back for 3 s 186
// and 165 us under the power cap.  By HBM for few rows per expert (42 us for 4096
// rows over 128 experts of 1536 x 2048, 34 us of bytes).
#include <cuda.h>

#include "attr.h"
#include "common.cuh"
#include "fp4.cuh"
#include "gmm_common.cuh"
#include "gmm_internal.h"
#include "gmm_stall.h"
#include "ragged.cuh"
#include "tc_pair.cuh"

namespace moe {
namespace gmm4 {

constexpr int kSlotRow = 32;                   // bytes of a row's scales in a slot
constexpr int kTileM = 256, kStep = 256;
constexpr int kSpan = 8;                       // steps of a part: 2048 elements
constexpr int kLong = 8192, kLong16 = 32768;
constexpr int kABytes = 128 * 128;
constexpr int kBlockBytes = 128 * kSlotRow;    // scales of 128 rows
constexpr int kDrainBytes = 16384;
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kWaitNs = 2000000000ull;

// FEW kernels, for at most 64 rows per expert as in gmm.cu, take tiles of 128
// rows of x and have more stages of codes on the way: 39.6 us rather than 41.1
// for 512 rows over 128 experts of 1536 x 2048 (NVFP4), 40.9 rather than 42.4 for
// 4096 (MXFP4); past that many rows more groups take two tiles.  As there, rows
// on a few of many experts get these tiles all the same (16384 rows on 8 of 256
// experts of 1536 x 2048, MXFP4: 31 us rather than 27).
enum Kind { kWide = 0, kFew = 1, kSum = 2 };   // kSum: FEW's shape, sums in parts
constexpr bool few_of(int kind) { return kind != kWide; }

template <bool FEW>
struct Shape {
    static constexpr int kTileN = FEW ? 128 : 192, kStages = FEW ? 7 : 5, kSlots = FEW ? 4 : 5;
    static constexpr int kBlocks = FEW ? 2 : 3;            // of scales in a slot: w, then x
    static constexpr int kStageBytes = kABytes + kTileN / 2 * 128, kSlotBytes = kBlocks * kBlockBytes;
    static constexpr int kThreads = 32 * (8 + kBlocks);
    static constexpr uint32_t kTmemScales = 2 * kTileN;    // accumulators first, then two stages of scales
};
constexpr int kMaxStages = 7, kMaxSlots = 5;

struct Args {
    const int32_t *off;
    const float *xa, *wa;
    void *out;
    int32_t *dev_status;
    int R, E, N, K;
    MOE_STALL_ARG
};

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t sfull[kMaxSlots], sdone[kMaxSlots], sready[kMaxSlots], sempty[kMaxSlots];
    uint64_t accf[2], acce[2], fin;
    uint32_t tmem;
    int abort;
    MOE_STALL_BARRIER
    ragged::List list;
};

template <bool FEW>
constexpr int smem_of()
{
    using S = Shape<FEW>;
    return 1024 + S::kStages * S::kStageBytes + S::kSlots * S::kSlotBytes + kDrainBytes + static_cast<int>(sizeof(Shared));
}
static_assert(smem_of<false>() <= 232448 && smem_of<true>() <= 232448, "shared memory of one CTA");

struct Tile {
    int e, m0, r0, n;          // expert, first row of w, first row of x and how many
};

template <int kTileN>
__device__ __forceinline__ Tile tile_of(const Args &a, const Shared &s, int t, int n_mt)
{
    Tile T;
    T.e = ragged::expert_of(s.list, a.E, t);
    const int at = t - s.list.tiles[T.e], nt = at / n_mt;
    T.m0 = (at - nt * n_mt) * kTileM;
    T.r0 = s.list.lo[T.e] + nt * kTileN;
    T.n = min(kTileN, s.list.rows(T.e) - nt * kTileN);
    return T;
}

__device__ __forceinline__ int n_mma(int n) { return (n + 31) & ~31; }

template <int FMT, typename OT, int KIND>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Shape<few_of(KIND)>::kThreads, 1)
gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
            const __grid_constant__ CUtensorMap tmB16, const __grid_constant__ CUtensorMap tmSA,
            const __grid_constant__ CUtensorMap tmSB, const __grid_constant__ CUtensorMap tmY, const Args a)
{
    constexpr bool FEW = few_of(KIND), SUM = KIND == kSum;
    using S = Shape<FEW>;
    constexpr int kTileN = S::kTileN, kStages = S::kStages, kSlots = S::kSlots, kBlocks = S::kBlocks;
    constexpr int kStageBytes = S::kStageBytes, kSlotBytes = S::kSlotBytes;
    constexpr uint32_t kTmemScales = S::kTmemScales;
    constexpr bool kMx = FMT == MOE_FP4_MXFP4;
    constexpr int kWords = kMx ? 2 : 4;                 // words of scales of a row in a stage
    constexpr int kSlotSteps = kSlotRow / 4 / kWords;             // stages in a slot
    extern __shared__ uint8_t smem_raw[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = tc::cluster_rank();
    const uint32_t raw = tc::smem_u32(smem_raw);
    uint8_t *smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    uint8_t *sf = smem + kStages * kStageBytes;
    const uint32_t ring = tc::smem_u32(smem), sfring = tc::smem_u32(sf);
    Shared &s = *reinterpret_cast<Shared *>(sf + kSlots * kSlotBytes + kDrainBytes);
    volatile int *abort = &s.abort;
    auto bar = [](uint64_t &b) { return tc::smem_u32(&b); };

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            tc::mbar_init(bar(s.full[i]), 1);
            tc::mbar_init(bar(s.empty[i]), 1);
        }
        for (int i = 0; i < kSlots; ++i) {
            tc::mbar_init(bar(s.sfull[i]), 1);
            tc::mbar_init(bar(s.sdone[i]), kBlocks);     // the arranging warps
            tc::mbar_init(bar(s.sready[i]), 2);          // each CTA's relay
            tc::mbar_init(bar(s.sempty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(bar(s.accf[i]), 1);
            tc::mbar_init(bar(s.acce[i]), 8);
        }
        tc::mbar_init(bar(s.fin), 1);
        MOE_STALL_INIT(s);
        s.abort = 0;
        tc::fence_mbar_init();
        tc::prefetch_tmap(&tmA);
        tc::prefetch_tmap(&tmB);
        tc::prefetch_tmap(&tmB16);
        tc::prefetch_tmap(&tmSA);
        tc::prefetch_tmap(&tmSB);
        tc::prefetch_tmap(&tmY);
    }
    if (warp == 1) {
        tc::tmem_alloc_pair(tc::smem_u32(&s.tmem), kTmemCols);
        tc::tmem_relinquish_pair();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int n_mt = (a.N + kTileM - 1) / kTileM, steps = (a.K + kStep - 1) / kStep;
    const int slots = (steps + kSlotSteps - 1) / kSlotSteps;
    ragged::make_list(s.list, a.off, a.E, a.R, n_mt, kTileN);
    tc::tc_fence_before();
    __syncthreads();
    tc::cluster_sync();
    tc::tc_fence_after();
    const uint32_t tmem = s.tmem;
    const int total = s.list.tiles[a.E];
    const int cid = blockIdx.x >> 1, n_cl = gridDim.x >> 1;

    if (warp == 0) {
        if (tc::elect_one()) {
            int st = 0, issued = 0;
            uint32_t ph = 0;
            const uint32_t full_lead = tc::mapa(bar(s.full[0]), 0);
            for (int t = cid; t < total && !*abort; t += n_cl) {
                const Tile T = tile_of<kTileN>(a, s, t, n_mt);
                const int m0 = T.m0 + 128 * rank, nh = n_mma(T.n) / 2, r0 = T.r0 + rank * nh;
                const uint32_t bytes = kABytes + (nh > kTileN / 4 ? kTileN / 2 : nh) * 128;
                for (int j = 0; j < steps; ++j, ++issued) {
                    if (!tc::mbar_wait(bar(s.empty[st]), ph ^ 1u, abort, kWaitNs))
                        break;
                    const uint32_t sa = ring + st * kStageBytes, sb = sa + kABytes, fb = full_lead + 8 * st;
                    if (rank == 0)
                        tc::mbar_arrive_expect_tx(fb, 2 * bytes);
                    tc::tma_load_3d_pair(sa, &tmA, j * 128, m0, T.e, fb);
                    if (nh > kTileN / 4)
                        tc::tma_load_2d_pair(sb, &tmB, j * 128, r0, fb);
                    else
                        for (int i = 0; i < nh; i += 16)
                            tc::tma_load_2d_pair(sb + i * 128, &tmB16, j * 128, r0 + i, fb);
                    if (++st == kStages) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (rank == 0) {
                // every copy has landed before the CTAs may finish
                volatile int never = 0;
                for (int i = 1; i <= min(issued, kStages); ++i) {
                    const int q = st - i < 0 ? st - i + kStages : st - i;
                    tc::mbar_wait(bar(s.full[q]), st - i < 0 ? ph ^ 1u : ph, &never, kWaitNs);
                }
                if (never)
                    *abort = 1;
            }
        }
    } else if (warp == 2) {
        if (tc::elect_one()) {
            int st = 0, issued = 0;
            uint32_t ph = 0;
            for (int t = cid; t < total && !*abort; t += n_cl) {
                const Tile T = tile_of<kTileN>(a, s, t, n_mt);
                const int m0 = T.m0 + 128 * rank, n = n_mma(T.n);
                for (int j = 0; j < slots; ++j, ++issued) {
                    if (!tc::mbar_wait(bar(s.sempty[st]), ph ^ 1u, abort, kWaitNs))
                        break;
                    const uint32_t sa = sfring + st * kSlotBytes, fb = bar(s.sfull[st]);
                    tc::mbar_arrive_expect_tx(fb, kBlockBytes + n * kSlotRow);
                    tc::tma_load_3d(sa, &tmSA, j * kSlotRow, m0, T.e, fb);
                    for (int i = 0; i < n; i += 32)
                        tc::tma_load_2d(sa + kBlockBytes + i * kSlotRow, &tmSB, j * kSlotRow, T.r0 + i, fb);
                    if (++st == kSlots) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
            }
            volatile int never = 0;
            for (int i = 1; i <= min(issued, kSlots); ++i) {
                const int q = st - i < 0 ? st - i + kSlots : st - i;
                tc::mbar_wait(bar(s.sfull[q]), st - i < 0 ? ph ^ 1u : ph, &never, kWaitNs);
            }
            if (never)
                *abort = 1;
        }
    } else if (warp == 1) {
        if (rank == 0 && tc::elect_one()) {
            // descriptors of stage 0; a stage or step further adds to the
            // address field (forming them anew costs more than the MMA takes)
            const uint64_t a0 = tc::smem_desc(ring, 16, 1024, tc::kLayoutSw128);
            const uint64_t b0 = tc::smem_desc(ring + kABytes, 16, 1024, tc::kLayoutSw128);
            const uint64_t s0 = tc::smem_desc(sfring, 0, 128, tc::kLayoutNone);
            int st = 0, sst = 0, tix = 0, g = 0;
            uint32_t ph = 0, sph = 0;
            for (int t = cid; t < total && !*abort; t += n_cl) {
                const Tile T = tile_of<kTileN>(a, s, t, n_mt);
                const int n = n_mma(T.n);
                const uint32_t id0 = tc::idesc_fp4(256, n, kMx, 0), id1 = kMx ? tc::idesc_fp4(256, n, kMx, 2) : id0;
                for (int j0 = 0; j0 < steps; j0 += SUM ? kSpan : steps, ++tix) {
                    const int buf = tix & 1, j1 = SUM ? min(j0 + kSpan, steps) : steps;
                    if (!tc::mbar_wait_cluster(bar(s.acce[buf]), ((tix >> 1) & 1) ^ 1u, abort, kWaitNs))
                        break;
                    tc::tc_fence_after();
                    const uint32_t acc = tmem + kTileN * buf;
                    MOE_STALL(a, s, t >= n_cl);
                    bool ok = true;
                    for (int j = j0; j < j1; ++j, ++g) {
                        const int js = j % kSlotSteps;
                        ok = (js != 0 || tc::mbar_wait_cluster(bar(s.sready[sst]), sph, abort, kWaitNs)) &&
                             tc::mbar_wait(bar(s.full[st]), ph, abort, kWaitNs);
                        if (!ok)
                            break;
                        tc::tc_fence_after();
                        const uint64_t ad = a0 + st * (kStageBytes >> 4), bd = b0 + st * (kStageBytes >> 4);
                        const uint64_t sd = s0 + (sst * kSlotBytes + js * kWords * 512) / 16;
                        const uint32_t ta = tmem + kTmemScales + (g & 1) * 48, tb = ta + 16;
#pragma unroll
                        for (int w = 0; w < kWords; ++w) {
                            tc::tc_cp_32x128b_x4_pair(ta + 4 * w, sd + 32 * w);
                            tc::tc_cp_32x128b_x4_pair(tb + 8 * w, sd + kBlockBytes / 16 + 32 * w);
                            if (!FEW && n > 128)
                                tc::tc_cp_32x128b_x4_pair(tb + 8 * w + 4, sd + 2 * kBlockBytes / 16 + 32 * w);
                        }
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            const int w = kMx ? kk >> 1 : kk;
                            tc::mma_fp4_pair<kMx>(acc, ad + 2 * kk, bd + 2 * kk, kk & 1 ? id1 : id0, ta + 4 * w, tb + 8 * w,
                                                  ((j - j0) | kk) != 0 ? 1u : 0u);
                        }
                        tc::tc_commit_pair(bar(s.empty[st]));
                        if (++st == kStages) {
                            st = 0;
                            ph ^= 1u;
                        }
                        if (js == kSlotSteps - 1 || j == steps - 1) {
                            tc::tc_commit_pair(bar(s.sempty[sst]));
                            if (++sst == kSlots) {
                                sst = 0;
                                sph ^= 1u;
                            }
                        }
                    }
                    if (!ok)                             // a part of the sums: not to be drained
                        break;
                    tc::tc_commit_pair(bar(s.accf[buf]));
                }
            }
            tc::tc_commit_pair(bar(s.fin));
        }
    } else if (warp == 3) {
        // tell the leader of every arranged slot, one thread for the three
        // warps' writes (each is through its own proxy fence by then)
        if (lane == 0) {
            int st = 0;
            uint32_t ph = 0;
            const uint32_t ready_lead = tc::mapa(bar(s.sready[0]), 0);
            for (int t = cid; t < total && !*abort; t += n_cl) {
                for (int j = 0; j < slots; ++j) {
                    if (!tc::mbar_wait(bar(s.sdone[st]), ph, abort, kWaitNs))
                        break;
                    tc::fence_proxy_async_smem();
                    tc::mbar_arrive_cluster_smem(ready_lead + 8 * st);
                    if (++st == kSlots) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
            }
        }
    } else if (warp >= 8) {
        // arrange the scales: each warp its block of 128 rows of every slot
        const int b = warp - 8;
        int st = 0;
        uint32_t ph = 0;
        for (int t = cid; t < total && !*abort; t += n_cl) {
            const Tile T = tile_of<kTileN>(a, s, t, n_mt);
            for (int j = 0; j < slots; ++j) {
                if (!tc::mbar_wait(bar(s.sfull[st]), ph, abort, kWaitNs))
                    break;
                if (b < 2 || T.n > 128) {
                    uint8_t *p = sf + st * kSlotBytes + b * kBlockBytes;
                    constexpr int kChunks = kSlotRow / 16;
                    uint4 v[4][kChunks];                 // [row l + 32 i][16-byte chunk]
                    const int x = (lane >> 2) & 1;       // the 32-byte swizzle of rows l + 32 i
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int c = 0; c < kChunks; ++c)
                            v[i][c] = *reinterpret_cast<const uint4 *>(p + (lane + 32 * i) * kSlotRow + ((c ^ x) << 4));
                    __syncwarp();
                    uint4 *o = reinterpret_cast<uint4 *>(p) + lane;
#pragma unroll
                    for (int c = 0; c < kChunks; ++c) {
                        o[128 * c] = make_uint4(v[0][c].x, v[1][c].x, v[2][c].x, v[3][c].x);
                        o[128 * c + 32] = make_uint4(v[0][c].y, v[1][c].y, v[2][c].y, v[3][c].y);
                        o[128 * c + 64] = make_uint4(v[0][c].z, v[1][c].z, v[2][c].z, v[3][c].z);
                        o[128 * c + 96] = make_uint4(v[0][c].w, v[1][c].w, v[2][c].w, v[3][c].w);
                    }
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                }
                if (lane == 0)
                    tc::mbar_arrive(bar(s.sdone[st]));
                if (++st == kSlots) {
                    st = 0;
                    ph ^= 1u;
                }
            }
        }
    } else if (warp >= 4) {
        const int q = warp & 3;                         // TMEM lane quadrant
        int tix = 0, flip = 0;
        OT *out = static_cast<OT *>(a.out);
        for (int t = cid; t < total; t += n_cl) {
            const Tile T = tile_of<kTileN>(a, s, t, n_mt);
            const int m = T.m0 + 128 * rank + 32 * q + lane;
            float f = 1.f, g = 1.f;
            if (!kMx)
                fp4::factors(*a.xa, a.wa[T.e], f, g);
            uint8_t *tiles = sf + kSlots * kSlotBytes + q * 4096;
            auto store = [&](int c0, const uint32_t (&v)[32]) {
                if (T.n - c0 < 32)                       // a TMA store would reach into the next group's rows
                    gmm::store_rows<OT>(v, out + static_cast<int64_t>(T.r0 + c0) * a.N, a.N, m, a.N, T.n - c0, lane, f, g);
                else
                    gmm::drain_rows<OT>(v, tiles, flip, &tmY, m - lane, T.r0 + c0, a.N, lane, f, g);
            };
            constexpr int kGroups = kTileN / 32;
            float sum[SUM ? kGroups : 1][32] = {};
            bool ok = true;
            for (int j0 = 0; j0 < steps; j0 += SUM ? kSpan : steps, ++tix) {
                const int buf = tix & 1;
                ok = tc::mbar_wait_cluster(bar(s.accf[buf]), (tix >> 1) & 1, abort, kWaitNs);
                if (!ok)
                    break;
                tc::tc_fence_after();
                const uint32_t acc = tmem + kTileN * buf + (static_cast<uint32_t>(32 * q) << 16);
                if constexpr (SUM) {
#pragma unroll
                    for (int c = 0; c < kGroups; ++c) {
                        if (32 * c < T.n) {
#pragma unroll
                            for (int h = 0; h < 32; h += 16) {
                                uint32_t v[16];
                                tc::tmem_ld_32x32b_x16(acc + 32 * c + h, v);
                                tc::tmem_ld_wait_for(v);
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    sum[c][h + i] += __uint_as_float(v[i]);
                            }
                        }
                    }
                } else {
                    for (int c0 = 0; c0 < T.n; c0 += 32) {
                        uint32_t v[32];
                        tc::tmem_ld_32x32b_x32(acc + c0, v);
                        tc::tmem_ld_wait_for(v);
                        store(c0, v);
                    }
                }
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    tc::mbar_arrive_cluster_relaxed(tc::mapa(bar(s.acce[buf]), 0));
            }
            if (!ok)
                break;
            if constexpr (SUM) {
#pragma unroll
                for (int c = 0; c < kGroups; ++c) {
                    if (32 * c < T.n) {
                        uint32_t v[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            v[i] = __float_as_uint(sum[c][i]);
                        store(32 * c, v);
                    }
                }
            }
        }
        tc::bulk_wait<0>();
        // rows outside every group
        const int first = min(max(a.off[0], 0), a.R), last = min(max(a.off[a.E], 0), a.R);
        const int64_t per = static_cast<int64_t>(a.N) * sizeof(OT) / 16;
        uint4 *o = static_cast<uint4 *>(a.out);
        const int64_t at = static_cast<int64_t>(blockIdx.x) * 128 + (threadIdx.x - 128), by = static_cast<int64_t>(gridDim.x) * 128;
        for (int64_t i = at; i < first * per; i += by)
            o[i] = make_uint4(0, 0, 0, 0);
        for (int64_t i = last * per + at; i < a.R * per; i += by)
            o[i] = make_uint4(0, 0, 0, 0);
        if (blockIdx.x == 0)
            for (int e = threadIdx.x - 128; e < a.E; e += 128)
                ragged::report_bad(a.off, a.R, e, a.dev_status);
    }
    __syncwarp();
    tc::tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) {
        // the leader's last MMA is done and has told both CTAs so
        volatile int never = 0;
        tc::mbar_wait(bar(s.fin), 0, &never, kWaitNs);
        if ((never || *abort) && a.dev_status)
            atomicCAS(a.dev_status + 1, 0, static_cast<int>(MOE_ERR_TIMEOUT));
    }
    tc::cluster_sync();                                  // neither CTA ends while the other still reaches into it
    if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc_pair(tmem, kTmemCols);
    }
}

// ---------------------------------------------------------------- host

template <int FMT, typename OT, int KIND>
static moe_status_t launch(const CUtensorMap (&tm)[6], const Args &a, cudaStream_t s)
{
    constexpr bool FEW = few_of(KIND);
    using S = Shape<FEW>;
    auto k = gemm_kernel<FMT, OT, KIND>;
    static std::atomic<uint64_t> done{0};
    if (!smem_attr_once(done, reinterpret_cast<const void *>(k), smem_of<FEW>()))
        return MOE_ERR_CUDA;
    const int64_t most = static_cast<int64_t>((a.N + kTileM - 1) / kTileM) * (a.R / S::kTileN + (a.E < a.R ? a.E : a.R));
    const int pairs = device_sm_count() / 2;
    const int grid = 2 * static_cast<int>(most < pairs ? most : pairs);
    return launch_pdl(k, dim3(grid), dim3(S::kThreads), smem_of<FEW>(), s, tm[0], tm[1], tm[2], tm[3], tm[4], tm[5], a) ==
                   cudaSuccess
               ? MOE_OK : MOE_ERR_CUDA;
}

template <int FMT, int KIND>
static moe_status_t launch_type(const CUtensorMap (&tm)[6], const Args &a, int32_t ydt, cudaStream_t s)
{
    if (ydt == MOE_FP32)
        return launch<FMT, float, KIND>(tm, a, s);
    return ydt == MOE_BF16 ? launch<FMT, __nv_bfloat16, KIND>(tm, a, s) : launch<FMT, __half, KIND>(tm, a, s);
}

template <int FMT>
static moe_status_t launch_kind(const CUtensorMap (&tm)[6], const Args &a, int32_t ydt, int kind, cudaStream_t s)
{
    if (kind == kSum)
        return launch_type<FMT, kSum>(tm, a, ydt, s);
    return kind == kFew ? launch_type<FMT, kFew>(tm, a, ydt, s) : launch_type<FMT, kWide>(tm, a, ydt, s);
}

}  // namespace gmm4
}  // namespace moe

using namespace moe;
using namespace moe::gmm4;

MOE_API moe_status_t moe_grouped_mm_fp4(const uint8_t *xq, const uint8_t *xs, const float *x_alpha, const uint8_t *wq,
                                        const uint8_t *ws, const float *w_alpha, int32_t fmt, const int32_t *offsets,
                                        int32_t R, int32_t E, int32_t N, int32_t K, void *y, int32_t ydt,
                                        int32_t *dev_status, void *stream)
{
    if (R < 0 || E < 1 || N < 1 || K < 1)
        return MOE_ERR_INVALID_ARG;
    if ((fmt != MOE_FP4_NVFP4 && fmt != MOE_FP4_MXFP4) || (ydt != MOE_BF16 && ydt != MOE_FP16 && ydt != MOE_FP32) ||
        E > ragged::kMaxExperts || N % 8 || K % 32 || R > ragged::kMaxSide || N > ragged::kMaxSide || K > ragged::kMaxSide)
        return MOE_ERR_UNSUPPORTED;
    if (R == 0)
        return MOE_OK;
    if (!xq || !xs || !wq || !ws || !offsets || !y || (fmt == MOE_FP4_NVFP4) != (x_alpha != nullptr) ||
        (fmt == MOE_FP4_NVFP4) != (w_alpha != nullptr) || !aligned(xq, 16) || !aligned(xs, 16) || !aligned(wq, 16) ||
        !aligned(ws, 16) || !aligned(y, 16) || !aligned(offsets, 4))
        return MOE_ERR_INVALID_ARG;
    const int Ks = fp4::scale_cols(K, fmt);
    const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_32B;
    const CUtensorMapDataType ty = ydt == MOE_FP32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : ydt == MOE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const int kind = K > (ydt == MOE_FP32 ? kLong : kLong16) ? kSum : R <= 64 * static_cast<int64_t>(E) ? kFew : kWide;
    const int tn = few_of(kind) ? Shape<true>::kTileN : Shape<false>::kTileN;
    if (!ragged::list_fits(E, R, (N + kTileM - 1) / kTileM, tn))
        return MOE_ERR_UNSUPPORTED;
    CUtensorMap tm[6];
    if (!tmap_tile(&tm[0], 3, u8, 1, wq, K / 2, N, E, 128, 128) || !tmap_tile(&tm[1], 2, u8, 1, xq, K / 2, R, 1, 128, tn / 2) ||
        !tmap_tile(&tm[2], 2, u8, 1, xq, K / 2, R, 1, 128, 16) || !tmap_tile(&tm[3], 3, u8, 1, ws, Ks, N, E, kSlotRow, 128, sw) ||
        !tmap_tile(&tm[4], 2, u8, 1, xs, Ks, R, 1, kSlotRow, 32, sw) ||
        !tmap_rows_out(&tm[5], ty, ydt == MOE_FP32 ? 4 : 2, y, N, R))
        return MOE_ERR_CUDA;
    const Args a{offsets, x_alpha, w_alpha, y, dev_status, R, E, N, K MOE_STALL_VALUE};
    return fmt == MOE_FP4_NVFP4 ? launch_kind<MOE_FP4_NVFP4>(tm, a, ydt, kind, as_stream(stream))
                                : launch_kind<MOE_FP4_MXFP4>(tm, a, ydt, kind, as_stream(stream));
}
