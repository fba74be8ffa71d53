// gmm.cu -- products of rows grouped by expert with the experts' 16-bit
// matrices, and their gradients:
//   y[r][n]     = sum_k x[r][k]  w[e][n][k]     moe_grouped_mm
//   dx[r][k]    = sum_n dy[r][n] w[e][n][k]     moe_grouped_mm_dgrad
//   dw[e][n][k] = sum_r dy[r][n] x[r][k]        moe_grouped_mm_wgrad
// for the rows r of expert e.  Sums are FP32, rounded once.
//
// One persistent kernel on the tensor cores (tcgen05 kind::f16), one CTA per
// SM, two CTAs (a cluster) per tile of 256 x 256 (256 x 128).  The left operand
// is the expert's matrix (w, w^T, or dy^T), 128 of its rows per CTA; the rows of
// x or dy -- or, for wgrad, the columns of x -- are the right operand's N, half
// of them held by each CTA.  A group's last tile takes N down to the next 32, so
// a group of few rows costs few columns of MMA, and a row's result is its own
// column of the accumulator: what the other columns hold does not reach it.
// Where an operand's contracted dimension is not its contiguous one (w^T, dy^T
// and x of wgrad) the tile is loaded as it lies and the MMA reads it
// MN-major; nothing is transposed in memory.
//
// wgrad contracts over the expert's rows, whose count is ragged: the rows of
// the last step that belong to the next expert are zeroed in shared memory up
// to the next 16 (both operands, so that a NaN there stays out) and the 16-row
// MMA steps past them are left out.
//
// Roles: warp 0 loads (TMA, 128-byte swizzle, a ring of 5 to 8 stages of 64
// along the contraction), warp 1 of the pair's leader issues the MMAs into two
// accumulators of 256 TMEM columns, warps from 4 on drain one while the next
// tile fills the other, warp 2 zeroes wgrad's row tails.  Every wait is bounded.  A
// role whose wait expires sets its CTA's abort flag, which ends the CTA's other
// roles at their next wait; an unfinished accumulator is not handed on, so the
// other CTA's waits expire too.  Each CTA reports its flag at its end, as
// MOE_ERR_TIMEOUT in dev_status[1].
//
// Bound by the tensor pipe for many rows per expert, at the clock that the power
// cap leaves: 8192 x 8192 x 8192 bf16 in runs of a few calls forward 572, dgrad
// 566, wgrad (FP32) 589 us, 1.9 PFLOP/s; back to back for 3 s 644, 641 and 663 us,
// 1.7 PFLOP/s.  By HBM for few: 4096 rows (Zipf) over 128 experts of 1536 x 2048
// in bf16 128 us, 6.5 TB/s; dgrad 125; wgrad 161, its 805 MB of dw (154 with the
// ragged tails announced at CTA scope, which PTX does not order).
#include <cuda.h>

#include "attr.h"
#include "common.cuh"
#include "fp4.cuh"
#include "gmm_common.cuh"
#include "gmm_internal.h"
#include "gmm_small.h"
#include "gmm_stall.h"
#include "ragged.cuh"
#include "tc_pair.cuh"

namespace moe {
namespace gmm {

enum { kFwd = 0, kDgrad = 1, kWgrad = 2 };

constexpr int kMaxStages = 8;

// The tensor cores add to an FP32 accumulator without rounding to nearest, so a
// long sum drifts (measured: 1.1e-9 of the result per contracted element, 4.4e-6
// at 4096).  Sum kernels end the accumulation every kSpan steps (512 elements)
// and add the parts in registers, rounded to nearest.  What is left grows with the
// parts' own roundings alone: terms of one sign, drawn at random, are at worst
// 9e-7 off at 4096 terms, 1.2e-6 at 65536 and 2.4e-6 at 2^20; equal terms, whose
// parts all round the same way, 3.1e-5 at 2^20.  FP32 results take them always,
// 16-bit ones -- whose own rounding is 2^-9 or 2^-12 -- where the contraction can
// be longer than kLong.
constexpr int kSpan = 8;
constexpr int kLong = 16384;

// Draining warps, one to a quadrant of tensor memory, or two with half of the
// columns each where they hold the sums; ring stages; bytes of a draining
// warp's staging tiles.  wgrad writes far more per tile of MMA work and has
// two tiles of 128-byte rows in place of a stage (4 stages: 8 to 12 % slower
// where the MMAs bound it; 64-byte rows or one tile: 10 to 25 % slower where
// dw does).
//
// Narrow kernels take tiles of 128 rows of x or dy and use the room for more
// stages: with few rows per expert the time is that of streaming the weights,
// and more of them are on the way (8 stages of 24 KB; 16 KB each are weights).
// 127 us rather than 132 for 4096 rows over 128 experts of 1536 x 2048, 13.6
// rather than 16.1 (dgrad) for 800 rows over 40 of 1000 x 520.  Past 64 rows per
// expert more and more groups take two tiles, which read the weights twice: 169
// rather than 158 us at 80 rows (Zipf) over 16 of 4096 x 7168.  The rule knows the
// mean alone, as the counts are on the device: rows that all go to a few of many
// experts get narrow tiles where wide ones are faster (16384 rows on 8 of 256
// experts: 74 rather than 66 us at 1536 x 2048, 317 rather than 287 at 4096 x
// 4096).
//
// Sum kernels have both forms: of the forward and dgrad with tiles of 128 rows,
// of wgrad with a second staging tile per warp in place of a stage, as with few
// rows per expert dw's stream bounds it (FP32 results, 32 rows for each of 128
// experts of 1536 x 2048: forward 132 rather than 137 us, wgrad 287 rather than
// 292; 20 rows for each of 40 of 1000 x 520: wgrad 19.6 rather than 20.6,
// and 20.3 since its tails are handed over at cluster scope).
enum Kind { kPlain = 0, kNarrow = 1, kSum = 2, kSumFew = 3 };
constexpr bool sums(int kind) { return kind == kSum || kind == kSumFew; }
constexpr int drain_of(int kind) { return sums(kind) ? 8 : 4; }
constexpr int tile_n(int op, int kind) { return kind == kNarrow || (kind == kSumFew && op != kWgrad) ? 128 : 256; }
constexpr int stages_of(int op, int kind)
{
    return kind == kNarrow ? 8 : kind == kSumFew ? (op == kWgrad ? 4 : 7) : op == kWgrad || kind == kSum ? 5 : 6;
}
constexpr int stage_bytes(int op, int kind) { return 16384 + 64 * tile_n(op, kind); }   // 128 rows and half a tile's
constexpr int staging_of(int op, int kind) { return op == kWgrad && kind != kSum ? 8192 : 4096; }
constexpr int threads_of(int kind) { return 32 * (4 + drain_of(kind)); }

constexpr int kTileM = 256, kStep = 64;
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kWaitNs = 2000000000ull;

struct Args {
    const int32_t *off;
    void *out;
    int32_t *dev_status;
    int R, E;
    int M;                     // rows of the left operand of one expert: N (fwd, wgrad) or K (dgrad)
    int C;                     // wgrad: columns of dw (K)
    int J;                     // fwd, dgrad: the contraction
    int accumulate;
    int bf16;
    MOE_STALL_ARG
};

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages], tail[kMaxStages], peer[kMaxStages], accf[2], acce[2], fin;
    uint32_t tmem;
    int abort, loaded;         // loaded: stages that the loader has begun (wgrad)
    MOE_STALL_BARRIER
    ragged::List list;
};

constexpr int smem_of(int op, int kind)
{
    return 1024 + stages_of(op, kind) * stage_bytes(op, kind) + drain_of(kind) * staging_of(op, kind) + static_cast<int>(sizeof(Shared));
}
static_assert(smem_of(kFwd, kPlain) <= 232448 && smem_of(kFwd, kNarrow) <= 232448 && smem_of(kWgrad, kPlain) <= 232448 &&
              smem_of(kFwd, kSum) <= 232448 && smem_of(kFwd, kSumFew) <= 232448 && smem_of(kWgrad, kSumFew) <= 232448,
              "shared memory of one CTA");

struct Tile {
    int e, m0, lo, rows;       // expert, first left row, the expert's rows
    int n0, n;                 // first column (row of the group, or column of dw) and how many
    int steps;
};

template <int OP, int kTileN>
__device__ __forceinline__ Tile tile_of(const Args &a, const Shared &s, int t, int n_mt, int n_nt)
{
    Tile T;
    int at;
    if (OP == kWgrad) {
        T.e = t / (n_mt * n_nt);
        at = t - T.e * n_mt * n_nt;
    } else {
        T.e = ragged::expert_of(s.list, a.E, t);
        at = t - s.list.tiles[T.e];
    }
    T.lo = s.list.lo[T.e];
    T.rows = s.list.rows(T.e);
    int mt, nt;
    ragged::place(at, n_mt, OP == kWgrad ? n_nt : (T.rows + kTileN - 1) / kTileN, mt, nt);
    T.m0 = mt * kTileM;
    T.n0 = nt * kTileN;
    T.n = min(kTileN, (OP == kWgrad ? a.C : T.rows) - T.n0);
    T.steps = ((OP == kWgrad ? T.rows : a.J) + kStep - 1) / kStep;
    return T;
}

__device__ __forceinline__ int n_mma(int n) { return (n + 31) & ~31; }

// Up to 32 rows of y or dx from row r0 on (n of them are the group's): through
// TMA where all 32 are, which would reach into the next group's rows otherwise.
template <typename OT>
__device__ __forceinline__ void store_y(const uint32_t (&v)[32], uint8_t *tiles, int &flip, const CUtensorMap *map, OT *out,
                                        int r0, int n, int m, int M, int lane)
{
    if (n < 32)
        store_rows<OT>(v, out + static_cast<int64_t>(r0) * M, M, m, M, n, lane);
    else
        drain_rows<OT>(v, tiles, flip, map, m - lane, r0, M, lane);
}

// 128 bytes of this lane's row of dw (row m of expert e, columns from c on) in
// w: through a staging tile (32 rows, 128-byte swizzle) and out, or added, by
// TMA, which cuts them at the expert's last row and column.  TWO: the warp has
// two tiles and alternates; the last but one store has read its tile by then.
template <typename OT, bool TWO>
__device__ __forceinline__ void store_tile(const uint32_t (&w)[32], uint8_t *tiles, int &flip, const CUtensorMap *map, int c, int m,
                                           int e, int M, int lane, bool add)
{
    uint8_t *tile = tiles + (TWO ? 4096 * flip : 0);
    flip ^= 1;
    tc::bulk_wait_read<TWO ? 1 : 0>();
    __syncwarp();
#pragma unroll
    for (int u = 0; u < 8; ++u)
        *reinterpret_cast<uint4 *>(tile + lane * 128 + ((u ^ (lane & 7)) << 4)) =
            make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
    tc::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
        if (m < M) {
            if (add)
                tc::tma_add_3d(map, tc::smem_u32(tile), c, m, e);
            else
                tc::tma_store_3d(map, tc::smem_u32(tile), c, m, e);
        }
        tc::bulk_commit();
    }
}

// 32 FP32 sums of this lane's row of dw as 16-bit values in w; accumulate: plus
// the old elements, rounded once (C % 8 == 0).
template <typename OT>
__device__ __forceinline__ void round_dw(const uint32_t (&v)[32], uint32_t *w, const OT *out, int c, int m, int e, int M, int C,
                                         bool accumulate)
{
#pragma unroll
    for (int i = 0; i < 16; ++i)
        w[i] = pack2<OT>(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
    if (accumulate && m < M) {
        const OT *old = out + (static_cast<int64_t>(e) * M + m) * C + c;
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
            if (c + i < C) {
                const uint4 o = *reinterpret_cast<const uint4 *>(old + i);
                const OT *p = reinterpret_cast<const OT *>(&o);
#pragma unroll
                for (int j = 0; j < 8; j += 2)
                    w[(i + j) / 2] = pack2<OT>(__uint_as_float(v[i + j]) + fp4::to_float(p[j]),
                                               __uint_as_float(v[i + j + 1]) + fp4::to_float(p[j + 1]));
            }
        }
    }
}

// tc::mbar_wait for the next ragged tail.  Experts whose rows are a multiple of 16
// have none, so it may be as far away as the end of the call: the limit runs anew
// with each stage that the loader begins.
__device__ __forceinline__ bool wait_tail(uint32_t bar, uint32_t parity, volatile int *loaded, volatile int *abort)
{
    ragged::Limit limit{clock64(), *loaded};
    for (uint32_t i = 1; !tc::mbar_try_wait(bar, parity); ++i) {
        if ((i & 3) == 0) {
            if (*abort)
                return false;
            if (limit.expired(clock64(), *loaded, static_cast<long long>(kWaitNs) * 5 / 2)) {
                *abort = 1;
                return false;
            }
        }
    }
    return true;
}

template <int OP, typename OT, int KIND>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(threads_of(KIND), 1)
gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
            const __grid_constant__ CUtensorMap tmB16, const __grid_constant__ CUtensorMap tmY, const Args a)
{
    // tmB16: B in boxes of 16 rows (fwd, dgrad); tmY: the result
    constexpr bool SUM = sums(KIND);
    constexpr int kStages = stages_of(OP, KIND), kDrain = drain_of(KIND), kStaging = staging_of(OP, KIND);
    constexpr bool kTwo = kStaging == 8192;             // wgrad: two staging tiles of 128-byte rows
    constexpr int kTileN = tile_n(OP, KIND), kStageBytes = stage_bytes(OP, KIND);
    extern __shared__ uint8_t smem_raw[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = tc::cluster_rank();
    const uint32_t raw = tc::smem_u32(smem_raw);
    uint8_t *smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);      // the same offset in both CTAs
    const uint32_t ring = tc::smem_u32(smem);
    Shared &s = *reinterpret_cast<Shared *>(smem + kStages * kStageBytes + kDrain * kStaging);
    volatile int *abort = &s.abort;
    auto bar = [](uint64_t &b) { return tc::smem_u32(&b); };

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            tc::mbar_init(bar(s.full[i]), 1);          // the leader's loader or tail warp
            tc::mbar_init(bar(s.empty[i]), 1);
            tc::mbar_init(bar(s.tail[i]), 1);
            tc::mbar_init(bar(s.peer[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(bar(s.accf[i]), 1);
            tc::mbar_init(bar(s.acce[i]), 2 * kDrain); // of both CTAs
        }
        tc::mbar_init(bar(s.fin), 1);
        MOE_STALL_INIT(s);
        s.abort = 0;
        s.loaded = 0;
        tc::fence_mbar_init();
        tc::prefetch_tmap(&tmA);
        tc::prefetch_tmap(&tmB);
        if (OP != kWgrad)
            tc::prefetch_tmap(&tmB16);
        tc::prefetch_tmap(&tmY);
    }
    if (warp == 1) {
        tc::tmem_alloc_pair(tc::smem_u32(&s.tmem), kTmemCols);
        tc::tmem_relinquish_pair();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int n_mt = (a.M + kTileM - 1) / kTileM, n_nt = (a.C + kTileN - 1) / kTileN;
    ragged::make_list(s.list, a.off, a.E, a.R, n_mt, kTileN);
    tc::tc_fence_before();
    __syncthreads();
    tc::cluster_sync();
    tc::tc_fence_after();
    const uint32_t tmem = s.tmem;
    const int total = OP == kWgrad ? a.E * n_mt * n_nt : s.list.tiles[a.E];
    const int cid = blockIdx.x >> 1, n_cl = gridDim.x >> 1;

    if (warp == 0) {
        if (tc::elect_one()) {
            int st = 0, issued = 0;
            uint32_t ph = 0;
            const uint32_t full_lead = tc::mapa(bar(s.full[0]), 0);
            for (int t = cid; t < total && !*abort; t += n_cl) {
                const Tile T = tile_of<OP, kTileN>(a, s, t, n_mt, n_nt);
                const int m0 = T.m0 + 128 * rank, nh = n_mma(T.n) / 2;
                const int tail = OP == kWgrad && (T.rows & 15) ? T.steps - 1 : -1;
                uint32_t bytes = 16384;
                if (OP == kWgrad)
                    bytes += nh > 64 ? 16384 : 8192;
                else
                    bytes += (nh > kTileN / 4 ? kTileN / 2 : nh) * 128;
                for (int j = 0; j < T.steps; ++j, ++issued) {
                    if (!tc::mbar_wait(bar(s.empty[st]), ph ^ 1u, abort, kWaitNs))
                        break;
                    const uint32_t sa = ring + st * kStageBytes, sb = sa + 16384;
                    uint32_t fb;
                    if (OP == kWgrad)
                        *const_cast<volatile int *>(&s.loaded) = issued + 1;
                    if (j == tail) {
                        // this CTA's tail warp hears of the data first
                        fb = bar(s.tail[st]);
                        tc::mbar_arrive_expect_tx(fb, bytes);
                    } else {
                        // the leader expects both CTAs' bytes; the other CTA
                        // cannot be a phase ahead, as the leader's MMAs empty
                        // the stage in both
                        fb = full_lead + 8 * st;
                        if (rank == 0)
                            tc::mbar_arrive_expect_tx(fb, 2 * bytes);
                    }
                    if (OP == kFwd) {
                        tc::tma_load_3d_pair(sa, &tmA, j * kStep, m0, T.e, fb);
                    } else if (OP == kDgrad) {
                        tc::tma_load_3d_pair(sa, &tmA, m0, j * kStep, T.e, fb);
                        tc::tma_load_3d_pair(sa + 8192, &tmA, m0 + 64, j * kStep, T.e, fb);
                    } else {
                        tc::tma_load_2d_pair(sa, &tmA, m0, T.lo + j * kStep, fb);
                        tc::tma_load_2d_pair(sa + 8192, &tmA, m0 + 64, T.lo + j * kStep, fb);
                    }
                    if (OP == kWgrad) {
                        const int c0 = T.n0 + rank * nh;
                        tc::tma_load_2d_pair(sb, &tmB, c0, T.lo + j * kStep, fb);
                        if (nh > 64)
                            tc::tma_load_2d_pair(sb + 8192, &tmB, c0 + 64, T.lo + j * kStep, fb);
                    } else {
                        const int r0 = T.lo + T.n0 + rank * nh;
                        if (nh > kTileN / 4)
                            tc::tma_load_2d_pair(sb, &tmB, j * kStep, r0, fb);
                        else
                            for (int i = 0; i < nh; i += 16)
                                tc::tma_load_2d_pair(sb + i * 128, &tmB16, j * kStep, r0 + i, fb);
                    }
                    if (++st == kStages) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
            }
            // every copy has landed before the CTAs may finish (a wait that is
            // over at once unless a role gave up)
            if (rank == 0) {
                volatile int never = 0;
                for (int i = 1; i <= min(issued, kStages); ++i) {
                    const int q = st - i < 0 ? st - i + kStages : st - i;
                    tc::mbar_wait(bar(s.full[q]), st - i < 0 ? ph ^ 1u : ph, &never, kWaitNs);
                }
                if (never)
                    *abort = 1;
            }
        }
    } else if (warp == 1) {
        if (rank == 0 && tc::elect_one()) {
            // descriptors of stage 0; a stage or step further adds to the
            // address field, so that an MMA costs a few instructions to issue
            const uint64_t a0 = OP == kFwd ? tc::smem_desc(ring, 16, 1024, tc::kLayoutSw128)
                                           : tc::smem_desc(ring, 8192, 1024, tc::kLayoutSw128);
            const uint64_t b0 = OP != kWgrad ? tc::smem_desc(ring + 16384, 16, 1024, tc::kLayoutSw128)
                                             : tc::smem_desc(ring + 16384, 8192, 1024, tc::kLayoutSw128);
            constexpr int kAStep = (OP == kFwd ? 32 : 2048) >> 4, kBStep = (OP != kWgrad ? 32 : 2048) >> 4;
            int st = 0, tix = 0;
            uint32_t ph = 0;
            for (int t = cid; t < total && !*abort; t += n_cl) {
                const Tile T = tile_of<OP, kTileN>(a, s, t, n_mt, n_nt);
                if (T.steps == 0)
                    continue;
                const uint32_t id = tc::idesc_f16_major(256, n_mma(T.n), a.bf16, OP != kFwd, OP == kWgrad);
                for (int j0 = 0; j0 < T.steps; j0 += SUM ? kSpan : T.steps) {
                    const int buf = tix & 1, j1 = SUM ? min(j0 + kSpan, T.steps) : T.steps;
                    if (!tc::mbar_wait_cluster(bar(s.acce[buf]), ((tix >> 1) & 1) ^ 1u, abort, kWaitNs))
                        break;
                    tc::tc_fence_after();
                    ++tix;
                    const uint32_t acc = tmem + 256 * buf;
                    MOE_STALL(a, s, t >= n_cl);
                    bool ok = true;
                    for (int j = j0; j < j1; ++j) {
                        ok = tc::mbar_wait(bar(s.full[st]), ph, abort, kWaitNs);
                        if (!ok)
                            break;
                        tc::tc_fence_after();
                        const uint64_t ad = a0 + st * (kStageBytes >> 4), bd = b0 + st * (kStageBytes >> 4);
                        const int nk = OP == kWgrad ? min(4, (T.rows - j * kStep + 15) >> 4) : 4;
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            if (OP != kWgrad || kk < nk)
                                tc::mma_f16_pair(acc, ad + kk * kAStep, bd + kk * kBStep, id, (j - j0) | kk ? 1u : 0u);
                        tc::tc_commit_pair(bar(s.empty[st]));
                        if (++st == kStages) {
                            st = 0;
                            ph ^= 1u;
                        }
                    }
                    if (!ok)                             // a part of the sums: not to be drained
                        break;
                    tc::tc_commit_pair(bar(s.accf[buf]));
                }
            }
            tc::tc_commit_pair(bar(s.fin));
        }
    } else if (warp == 2) {
        if (OP == kWgrad) {
            // zero the last step's rows past the expert's, up to the next 16
            int st = 0;
            uint32_t phases = 0;
            for (int t = cid; t < total; t += n_cl) {
                const Tile T = tile_of<OP, kTileN>(a, s, t, n_mt, n_nt);
                if (T.steps == 0)
                    continue;
                const int q = (st + T.steps - 1) % kStages;
                st = (st + T.steps) % kStages;
                if (!(T.rows & 15))
                    continue;
                const uint32_t ph = (phases >> q) & 1u;
                phases ^= 1u << q;
                if (!wait_tail(bar(s.tail[q]), ph, &s.loaded, abort))
                    break;
                const int r0 = T.rows - (T.steps - 1) * kStep, r1 = (r0 + 15) & ~15;
                for (int i = lane; i < (r1 - r0) * 32; i += 32) {
                    const int r = r0 + (i >> 5), part = (i >> 3) & 3, col = i & 7;     // 4 chunks of 64 x 128 bytes
                    *reinterpret_cast<uint4 *>(smem + q * kStageBytes + part * 8192 + r * 128 + col * 16) = make_uint4(0, 0, 0, 0);
                }
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (rank == 0) {
                    // both CTAs' tails are zeroed: the stage is full
                    if (!tc::mbar_wait_cluster(bar(s.peer[q]), ph, abort, kWaitNs))
                        break;
                    if (lane == 0)
                        tc::mbar_arrive(bar(s.full[q]));
                } else if (lane == 0) {
                    tc::mbar_arrive_cluster(tc::mapa(bar(s.peer[q]), 0));
                }
            }
        }
    } else if (warp >= 4) {
        const int q = warp & 3;                         // TMEM lane quadrant
        int tix = 0, flip = 0;
        OT *out = static_cast<OT *>(a.out);
        uint8_t *tiles = smem + kStages * kStageBytes + (warp - 4) * kStaging;
        for (int t = cid; t < total; t += n_cl) {
            const Tile T = tile_of<OP, kTileN>(a, s, t, n_mt, n_nt);
            const int m = T.m0 + 128 * rank + 32 * q + lane;
            if constexpr (SUM) {
                // this warp's half of the columns: the spans' parts added in
                // registers
                constexpr int kGroups = kTileN / 64;
                const int half = (warp - 4) >> 2;
                // the column of group g: alternate 128 bytes of dw, so that the
                // quadrant's two warps write next to each other
                auto col = [&](int g) {
                    return OP == kWgrad && sizeof(OT) == 2 ? (g / 2) * 128 + 64 * half + (g & 1) * 32 : 64 * g + 32 * half;
                };
                float sum[kGroups][32];
#pragma unroll
                for (int g = 0; g < kGroups; ++g)
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        sum[g][i] = 0.f;
                bool ok = true;
                for (int j0 = 0; j0 < T.steps; j0 += kSpan, ++tix) {
                    const int buf = tix & 1;
                    ok = tc::mbar_wait_cluster(bar(s.accf[buf]), (tix >> 1) & 1, abort, kWaitNs);
                    if (!ok)
                        break;
                    tc::tc_fence_after();
                    const uint32_t acc = tmem + 256 * buf + (static_cast<uint32_t>(32 * q) << 16);
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) {
                        if (col(g) < T.n) {
#pragma unroll
                            for (int h = 0; h < 32; h += 16) {
                                uint32_t v[16];
                                tc::tmem_ld_32x32b_x16(acc + col(g) + h, v);
                                tc::tmem_ld_wait_for(v);
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    sum[g][h + i] += __uint_as_float(v[i]);
                            }
                        }
                    }
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        tc::mbar_arrive_cluster_relaxed(tc::mapa(bar(s.acce[buf]), 0));
                }
                if (!ok)
                    break;
                auto bits = [&](int g, uint32_t (&v)[32]) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        v[i] = __float_as_uint(sum[g][i]);
                };
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    const int c0 = col(g);
                    if (c0 >= T.n || (OP == kWgrad && T.steps == 0 && a.accumulate))
                        continue;
                    uint32_t v[32];
                    bits(g, v);
                    if constexpr (OP != kWgrad) {
                        store_y<OT>(v, tiles, flip, &tmY, out, T.lo + T.n0 + c0, T.n - c0, m, a.M, lane);
                    } else if constexpr (sizeof(OT) == 4) {
                        store_tile<OT, kTwo>(v, tiles, flip, &tmY, T.n0 + c0, m, T.e, a.M, lane, a.accumulate);
                    } else if (g % 2 == 0) {
                        uint32_t w[32];
                        round_dw<OT>(v, w, out, T.n0 + c0, m, T.e, a.M, a.C, a.accumulate);
                        bits(g + 1 < kGroups ? g + 1 : g, v);
                        round_dw<OT>(v, w + 16, out, T.n0 + c0 + 32, m, T.e, a.M, a.C, a.accumulate);
                        store_tile<OT, kTwo>(w, tiles, flip, &tmY, T.n0 + c0, m, T.e, a.M, lane, false);
                    }
                }
            } else {
                const int buf = tix & 1;
                if (T.steps) {
                    if (!tc::mbar_wait_cluster(bar(s.accf[buf]), (tix >> 1) & 1, abort, kWaitNs))
                        break;
                    tc::tc_fence_after();
                    ++tix;
                }
                const uint32_t acc = tmem + 256 * buf + (static_cast<uint32_t>(32 * q) << 16);
                if (OP == kWgrad) {
                    if (T.steps || !a.accumulate) {
                        for (int c0 = 0; c0 < T.n; c0 += 64) {
                            uint32_t v[2][32], w[32];
                            if (T.steps) {
                                tc::tmem_ld_32x32b_x32(acc + c0, v[0]);
                                tc::tmem_ld_32x32b_x32(acc + c0 + 32, v[1]);
                                tc::tmem_ld_wait_for(v[0]);
                                tc::tmem_ld_wait_for(v[1]);
                            } else {
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    v[0][i] = v[1][i] = 0;
                            }
                            round_dw<OT>(v[0], w, out, T.n0 + c0, m, T.e, a.M, a.C, a.accumulate);
                            round_dw<OT>(v[1], w + 16, out, T.n0 + c0 + 32, m, T.e, a.M, a.C, a.accumulate);
                            store_tile<OT, kTwo>(w, tiles, flip, &tmY, T.n0 + c0, m, T.e, a.M, lane, false);
                        }
                    }
                } else {
                    for (int c0 = 0; c0 < T.n; c0 += 32) {
                        uint32_t v[32];
                        tc::tmem_ld_32x32b_x32(acc + c0, v);
                        tc::tmem_ld_wait_for(v);
                        store_y<OT>(v, tiles, flip, &tmY, out, T.lo + T.n0 + c0, T.n - c0, m, a.M, lane);
                    }
                }
                if (T.steps) {
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        tc::mbar_arrive_cluster_relaxed(tc::mapa(bar(s.acce[buf]), 0));
                }
            }
        }
        tc::bulk_wait<0>();
        if (OP != kWgrad) {
            // rows outside every group
            const int first = min(max(a.off[0], 0), a.R), last = min(max(a.off[a.E], 0), a.R);
            const int64_t per = static_cast<int64_t>(a.M) * sizeof(OT) / 16;
            uint4 *o = static_cast<uint4 *>(a.out);
            const int64_t at = static_cast<int64_t>(blockIdx.x) * (32 * kDrain) + (threadIdx.x - 128);
            const int64_t by = static_cast<int64_t>(gridDim.x) * (32 * kDrain);
            for (int64_t i = at; i < first * per; i += by)
                o[i] = make_uint4(0, 0, 0, 0);
            for (int64_t i = last * per + at; i < a.R * per; i += by)
                o[i] = make_uint4(0, 0, 0, 0);
        }
        if (blockIdx.x == 0)
            for (int e = threadIdx.x - 128; e < a.E; e += 32 * kDrain)
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

static bool type16(int32_t dt) { return dt == MOE_BF16 || dt == MOE_FP16; }
static bool out_type(int32_t t, int32_t dt) { return t == MOE_FP32 || t == dt; }

// The checks that the three products share.
static moe_status_t check(const void *a, const void *b, const void *out, int32_t dt, int32_t odt, int32_t R, int32_t E,
                          int32_t N, int32_t K, const int32_t *offsets)
{
    if (R < 0 || E < 1 || N < 1 || K < 1)
        return MOE_ERR_INVALID_ARG;
    if (!type16(dt) || !out_type(odt, dt) || E > ragged::kMaxExperts || N % 8 || K % 8 || R > ragged::kMaxSide ||
        N > ragged::kMaxSide || K > ragged::kMaxSide)
        return MOE_ERR_UNSUPPORTED;
    if (!offsets || !out || !aligned(out, 16) || !aligned(offsets, 4))
        return MOE_ERR_INVALID_ARG;
    if (R && (!a || !b || !aligned(a, 16) || !aligned(b, 16)))
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

template <int OP, typename OT, int KIND>
static moe_status_t launch(const CUtensorMap (&tm)[4], const Args &a, int64_t most_tiles, cudaStream_t s)
{
    auto k = gemm_kernel<OP, OT, KIND>;
    constexpr int kSmem = smem_of(OP, KIND);
    static std::atomic<uint64_t> done{0};
    if (!smem_attr_once(done, reinterpret_cast<const void *>(k), kSmem))
        return MOE_ERR_CUDA;
    const int pairs = device_sm_count() / 2;
    const int grid = 2 * static_cast<int>(most_tiles < pairs ? most_tiles : pairs);
    return launch_pdl(k, dim3(grid), dim3(threads_of(KIND)), kSmem, s, tm[0], tm[1], tm[2], tm[3], a) == cudaSuccess ? MOE_OK
                                                                                                               : MOE_ERR_CUDA;
}

template <int OP, int KIND>
static moe_status_t launch_as(const CUtensorMap (&tm)[4], const Args &a, int32_t odt, int64_t most_tiles, cudaStream_t s)
{
    if constexpr (sums(KIND))
        if (odt == MOE_FP32)
            return launch<OP, float, KIND>(tm, a, most_tiles, s);
    return odt == MOE_BF16 ? launch<OP, __nv_bfloat16, KIND>(tm, a, most_tiles, s) : launch<OP, __half, KIND>(tm, a, most_tiles, s);
}

template <int OP>
static moe_status_t launch_kind(const CUtensorMap (&tm)[4], const Args &a, int32_t odt, int kind, int64_t most_tiles,
                                cudaStream_t s)
{
    if (kind == kSum)
        return launch_as<OP, kSum>(tm, a, odt, most_tiles, s);
    if (kind == kSumFew)
        return launch_as<OP, kSumFew>(tm, a, odt, most_tiles, s);
    if constexpr (OP != kWgrad)
        if (kind == kNarrow)
            return launch_as<OP, kNarrow>(tm, a, odt, most_tiles, s);
    return launch_as<OP, kPlain>(tm, a, odt, most_tiles, s);
}

static CUtensorMapDataType map_type(int32_t dt)
{
    return dt == MOE_FP32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                          : dt == MOE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

// y or dx: C outputs per row from J contracted values; w [E][C][J] (OP kFwd)
// or [E][J][C] (OP kDgrad).
template <int OP>
static moe_status_t rows(const void *x, const void *w, int32_t dt, int32_t R, int32_t E, int32_t C, int32_t J,
                         const int32_t *off, void *y, int32_t ydt, int32_t *dev_status, cudaStream_t s)
{
    const CUtensorMapDataType t = map_type(dt);
    const bool few = R <= 64 * static_cast<int64_t>(E), sum = ydt == MOE_FP32 || J > kLong;
    const int kind = sum ? (few ? kSumFew : kSum) : few ? kNarrow : kPlain;
    const int tn = tile_n(OP, kind);
    const int64_t n_mt = (C + kTileM - 1) / kTileM;
    if (!ragged::list_fits(E, R, n_mt, tn))
        return MOE_ERR_UNSUPPORTED;
    CUtensorMap tm[4];
    const bool ok = OP == kFwd ? tmap_tile(&tm[0], 3, t, 2, w, J, C, E, 64, 128) : tmap_tile(&tm[0], 3, t, 2, w, C, J, E, 64, 64);
    if (!ok || !tmap_tile(&tm[1], 2, t, 2, x, J, R, 1, 64, tn / 2) || !tmap_tile(&tm[2], 2, t, 2, x, J, R, 1, 64, 16) ||
        !tmap_rows_out(&tm[3], map_type(ydt), ydt == MOE_FP32 ? 4 : 2, y, C, R))
        return MOE_ERR_CUDA;
    const Args a{off, y, dev_status, R, E, C, 0, J, 0, dt == MOE_BF16 MOE_STALL_VALUE};
    const int64_t tiles = n_mt * (static_cast<int64_t>(R) / tn + (E < R ? E : R));
    return launch_kind<OP>(tm, a, ydt, kind, tiles, s);
}

}  // namespace gmm
}  // namespace moe

using namespace moe;
using namespace moe::gmm;

#ifdef MOE_DEBUG_BOUNDS
std::atomic<int> moe::g_products_stall{0};

MOE_API moe_status_t moe_debug_products_stall(int32_t on)
{
    if (on != 0 && on != 1)
        return MOE_ERR_INVALID_ARG;
    g_products_stall.store(on, std::memory_order_relaxed);
    return MOE_OK;
}
#endif

MOE_API moe_status_t moe_grouped_mm(const void *x, const void *w, int32_t dt, const int32_t *offsets, int32_t R, int32_t E,
                                    int32_t N, int32_t K, void *y, int32_t ydt, int32_t *dev_status, void *stream)
{
    if (R == 0 && E >= 1 && N >= 1 && K >= 1)
        return type16(dt) && out_type(ydt, dt) ? MOE_OK : MOE_ERR_UNSUPPORTED;
    const moe_status_t st = check(x, w, y, dt, ydt, R, E, N, K, offsets);
    if (st == MOE_OK && R <= kSmallRows)
        return grouped_mm_small(x, w, dt, offsets, R, E, N, K, y, ydt, dev_status, as_stream(stream));
    return st != MOE_OK ? st : rows<kFwd>(x, w, dt, R, E, N, K, offsets, y, ydt, dev_status, as_stream(stream));
}

MOE_API moe_status_t moe_grouped_mm_dgrad(const void *dy, const void *w, int32_t dt, const int32_t *offsets, int32_t R,
                                          int32_t E, int32_t N, int32_t K, void *dx, int32_t xdt, int32_t *dev_status,
                                          void *stream)
{
    if (R == 0 && E >= 1 && N >= 1 && K >= 1)
        return type16(dt) && out_type(xdt, dt) ? MOE_OK : MOE_ERR_UNSUPPORTED;
    const moe_status_t st = check(dy, w, dx, dt, xdt, R, E, N, K, offsets);
    return st != MOE_OK ? st : rows<kDgrad>(dy, w, dt, R, E, K, N, offsets, dx, xdt, dev_status, as_stream(stream));
}

MOE_API moe_status_t moe_grouped_mm_wgrad(const void *dy, const void *x, int32_t dt, const int32_t *offsets, int32_t R,
                                          int32_t E, int32_t N, int32_t K, void *dw, int32_t wdt, int32_t accumulate,
                                          int32_t *dev_status, void *stream)
{
    if (accumulate != 0 && accumulate != 1)
        return MOE_ERR_INVALID_ARG;
    const moe_status_t st = check(dy, x, dw, dt, wdt, R, E, N, K, offsets);
    if (st != MOE_OK)
        return st;
    const int64_t tiles = static_cast<int64_t>(E) * ((N + kTileM - 1) / kTileM) * ((K + 255) / 256);
    if (tiles > ragged::kMaxTiles)
        return MOE_ERR_UNSUPPORTED;
    const CUtensorMapDataType t = map_type(dt);
    const int size = wdt == MOE_FP32 ? 4 : 2;
    CUtensorMap tm[4];
    // without rows nothing is loaded; the maps still need an address
    if (!tmap_tile(&tm[0], 2, t, 2, R ? dy : dw, N, R ? R : 1, 1, 64, 64) ||
        !tmap_tile(&tm[1], 2, t, 2, R ? x : dw, K, R ? R : 1, 1, 64, 64) ||
        !tmap_tile(&tm[3], 3, map_type(wdt), size, dw, K, N, E, 128 / size, 32))
        return MOE_ERR_CUDA;
    tm[2] = tm[1];
    const Args a{offsets, dw, dev_status, R, E, N, K, 0, accumulate, dt == MOE_BF16 MOE_STALL_VALUE};
    const bool few = R <= 64 * static_cast<int64_t>(E), sum = wdt == MOE_FP32 || R > kLong;
    return launch_kind<kWgrad>(tm, a, wdt, sum ? (few ? kSumFew : kSum) : kPlain, tiles, as_stream(stream));
}
