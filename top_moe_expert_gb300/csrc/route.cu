// route.cu -- the general router: k experts of each token by softmax or sigmoid
// scores, with a bias that only the choice sees and a limit to the best groups of
// experts, their weights, and the gradient of the logits from the weights'.
//
//   score s_e = exp(l_e) / sum exp(l)  or  1 / (1 + exp(-l_e))
//   choice    by v_e = s_e + b_e, or by l_e where there is no bias (scores rise
//             with the logit); a group of E / groups consecutive experts is worth
//             its best v, or the sum of its two best (of s without a bias), and
//             only the topk_groups best groups are in; equal values go by index
//   weights   w_j = scale s_j, or scale s_j / sum of the chosen s
//
// What is compared are the values in binary64.  A warp takes a token and forms
// them in binary32; where two that decide something are nearer than their errors
// can be (a share of about 1e-3 of the tokens at logits of spread 1), those and
// their rivals alone are formed anew in binary64, whose instructions take a warp some
// 60 cycles each.  Logits without a bias are compared as they are.
//
// A lane holds consecutive experts of one group, and a group takes a power of two
// of neighbouring lanes, so that the lowest lane that holds a maximum also holds
// the lowest index.
//
// Bound by instruction issue (0.73 per cycle and scheduler), 746 of a warp for a token
// of 256 experts (in parts, roughly: 50 for the loads, 110 for the scores, 140 for the
// groups, 90 for the bound, 90 to collect what is above it, 160 to rank it, 100 for the
// weights).  65536 tokens, 8 of 256 in 4 of 8 groups, bf16 with a bias: 55.2 us, where the
// bytes take 5.6; 4096 tokens, 8 of 128, FP32: 4.8 us.  Before: k rounds of a maximum over
// sorted lanes 100 us; candidates placed by a ballot for each of a lane's experts 74;
// all of an undecided token in binary64 at the end 69.  Two tokens in the halves of a
// warp, whose maxima take shuffles, gained nothing (52 us against 48 without groups).
//
// The time depends on the data.  What binary32 leaves open costs binary64 values, and a
// softmax with a bias, or more than 64 candidates, the whole token anew (route_exact).
// The same 65536 tokens in FP32, all logits equal (a router that starts at zero): 1.51 ms
// by sigmoids, 1.35 by softmax with a bias, 1.50 without groups or bias.  The groups'
// margin is one for all: a finite bias of -1e9 or the type's lowest value on one group
// makes it wider than all scores, and every token's groups are settled in binary64, in
// 0.85 ms (softmax 1.36); -inf on that group leaves them to binary32, in 61 us (95).
#include <cfloat>
#include <climits>
#include <type_traits>

#include "attr.h"
#include "common.cuh"
#include "fp4.cuh"
#include "gmm_common.cuh"
#include "ragged.cuh"
#include "topk.cuh"

namespace moe {
namespace route {

constexpr int kWarps = 16, kBwdWarps = 4;
constexpr int kMaxExperts = ragged::kMaxExperts;
constexpr int kMaxK = 32, kMaxGroups = 32, kMaxPer = 64, kMaxFound = 64;

struct Args {
    const void *logits;
    const float *bias;
    int M, E, k, groups, topk_groups, group_top, sigmoid, renorm;
    float scale;
    int of_group, lanes, shift, per;     // experts of a group, lanes of a group (2^shift), experts of a lane (at most)
    int32_t *ids;
    float *w;
    int32_t *load;
};

template <typename T>
__device__ __forceinline__ float value(T v) { return static_cast<float>(v); }

// NaN and +inf are out of the choice, as -inf is.
__device__ __forceinline__ float clean(float v) { return v < INFINITY ? v : -INFINITY; }

__device__ __forceinline__ float warp_max(float v)
{
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// The two best of two pairs (a1 >= a2, b1 >= b2).
__device__ __forceinline__ void best_two(float &a1, float &a2, float b1, float b2)
{
    a2 = fmaxf(fminf(a1, b1), fmaxf(a2, b2));
    a1 = fmaxf(a1, b1);
}

__device__ __forceinline__ void best_two(uint64_t &a1, uint64_t &a2, uint64_t b1, uint64_t b2)
{
    const uint64_t lo = a1 < b1 ? a1 : b1, hi = a1 < b1 ? b1 : a1, s = a2 < b2 ? b2 : a2;
    a1 = hi;
    a2 = lo < s ? s : lo;
}

// A lane's place: its first expert, how many it has.
struct Place {
    int group, base, count;
    __device__ __forceinline__ Place(const Args &a, int lane)
    {
        group = lane >> a.shift;
        const int first = (lane & (a.lanes - 1)) * a.per;
        base = group * a.of_group + first;
        count = group < a.groups ? min(max(a.of_group - first, 0), a.per) : 0;
    }
};

// The sigmoid of a logit from exp(-|l|), which does not overflow.
__device__ __forceinline__ float sigmoid(float l)
{
    const float t = expf(-fabsf(l)), r = __fdividef(1.0f, 1.0f + t);
    return l >= 0.f ? r : t * r;
}

// Lane j < k: weight of slot j from its logit (live: it has an expert).  m, z:
// the row's maximum and sum of exp(l - m), for softmax weights as they are.
__device__ __forceinline__ float weight(bool sigmoid_score, bool renorm, float scale, float l, bool live, float m, float z)
{
    if (!renorm) {
        const float s = sigmoid_score ? sigmoid(l) : expf(l - m) / z;
        return live ? s * scale : 0.f;
    }
    // the chosen scores over their sum.  Sigmoids of logits below -18 are exp(l) to
    // within 2^-25, and a softmax of the logits loses none of them, nor their bits to
    // the subnormal range, before it is divided.
    const float top = warp_max(live ? l : -INFINITY);
    const float s = !live ? 0.f : sigmoid_score && top > -18.f ? sigmoid(l) : expf(l - top);
    const float sum = warp_sum(s);
    return live ? __fdividef(s, sum) * scale : 0.f;         // sum is at least e^-18 / 2
}

// A token's candidates, one to a lane or two; then in their order.
struct Slots {
    uint64_t found[kMaxFound];                         // key64, or order64 of the exact value
    uint64_t sorted[kMaxK + 1];
    int expert[kMaxFound];
};

// A value and its place among the candidates as one number: larger values first,
// then lower places.
__device__ __forceinline__ uint64_t key64(float v, int place)
{
    return static_cast<uint64_t>(topk_key(v)) << 32 | ~static_cast<uint32_t>(place);
}
// Comparisons of binary64 take a warp some 60 cycles, those of whole numbers 4.
__device__ __forceinline__ uint64_t order64(double v)
{
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
    return u ^ (u >> 63 ? ~0ull : 0x8000000000000000ull);
}
__device__ __forceinline__ double value64(uint64_t k)
{
    return __longlong_as_double(static_cast<long long>(k ^ (k >> 63 ? 0x8000000000000000ull : ~0ull)));
}
__device__ __forceinline__ double sigmoid64(float l) { return 1.0 / (1.0 + exp(-static_cast<double>(l))); }
// A score in binary64.  Not inlined: what runs for a few tokens only should be
// little code, which every SM fetches anew.
__device__ __noinline__ double score64(double l, bool sigmoid_score, double m, double z)
{
    const double t = exp(sigmoid_score ? -l : l - m);
    return (sigmoid_score ? 1.0 : t) / (sigmoid_score ? 1.0 + t : z);
}
__device__ __forceinline__ int index_of(uint64_t k) { return static_cast<int>(~static_cast<uint32_t>(k)); }
__device__ __forceinline__ float value_of(uint64_t k) { return topk_unkey(static_cast<uint32_t>(k >> 32)); }

// The errors that the values of the choice may have in binary32.
//   sigmoid  2^-21: exp to (2 + 1.7 |l|) ulp moves it by at most 0.7 2^-23, the sum
//            and the reciprocal by 1.5 2^-23
//   softmax  (20 + PER / 2) 2^-23 of the largest score 1 / z: its own 3, the sum's
//            terms' 2 + 1.7 |x| ulp, |x| weighed by the scores at most ln E, and its
//            additions'
// Two values that are closer than twice that and their additions' rounding may be
// in the other order.
__device__ __forceinline__ float slack_of(const Args &a, float rz)
{
    return a.sigmoid ? 0x1p-20f : (40 + a.per) * 0x1p-23f * rz;
}

// exp(-x) / (1 + exp(-x)) as far as that error; 0 below -88.
__device__ __forceinline__ float fast_sigmoid(float l)
{
    float t, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(l * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + t));
    return r;
}

// The same in binary64 for one token, by one warp: what it may choose is found in
// binary32 as the kernel does, with those errors to spare, and the values of these
// candidates alone are formed in binary64, one to a lane (a warp's instruction takes
// some 60 cycles).  Lane j < k receives slot j's expert, or -1.
template <typename T>
struct Exact {
    const Args &a;
    const T *l;
    Slots &slots;
    const Place at;
    const int lane;
    double m, z;                                       // of a softmax
    float slack, rz, kept_x = NAN, kept_b = 0.f;
    uint64_t kept = 0;
    float own[kMaxPer];                                // the lane's experts' values in binary32

    __device__ __forceinline__ Exact(const Args &args, const T *row, Slots &s, int my_lane)
        : a(args), l(row), slots(s), at(args, my_lane), lane(my_lane), m(0.0), z(1.0)
    {
        if (!a.sigmoid) {
            float top = -INFINITY;
#pragma unroll 1
            for (int i = 0; i < at.count; ++i)
                top = fmaxf(top, logit(at.base + i));
            m = warp_max(top);
            z = 0.0;
            if (m > -INFINITY)
#pragma unroll 1
                for (int i = 0; i < at.count; ++i)
                    z += score64(logit(at.base + i), false, m, 1.0);
#pragma unroll 1
            for (int o = 16; o > 0; o >>= 1)
                z += __shfl_xor_sync(0xffffffffu, z, o);
        }
        rz = 1.0f / static_cast<float>(z);
        slack = slack_of(a, rz);
    }
    __device__ __forceinline__ float logit(int e) const { return clean(value(l[e])); }
    __device__ __forceinline__ float bias(int e) const { return clean(a.bias[e]); }
    __device__ __forceinline__ float near_score(int e) const
    {
        const float x = logit(e);
        return !(x > -INFINITY) ? -INFINITY
               : a.sigmoid      ? fast_sigmoid(x)
                                : __expf(x - static_cast<float>(m)) * rz;
    }
    // What a group's value is made of, and what experts are chosen by.
    __device__ __forceinline__ float near(int e, bool of_group) const
    {
        if (a.bias)
            return near_score(e) + bias(e);
        return of_group && a.group_top == 2 ? near_score(e) : logit(e);
    }
    // The same exactly, as its order.  The last one is kept: of many equal experts
    // (a router that starts at zero) one is formed.
    __device__ __forceinline__ uint64_t exact(int e, bool of_group)
    {
        const float x = logit(e), b = a.bias ? bias(e) : 0.f;
        if (!a.bias && !(of_group && a.group_top == 2))
            return order64(x);
        if (x != kept_x || b != kept_b) {
            kept_x = x;
            kept_b = b;
            kept = order64(score64(x, a.sigmoid, m, z) + static_cast<double>(b));
        }
        return kept;
    }
    __device__ __forceinline__ void form(bool of_group)
    {
#pragma unroll 4
        for (int i = 0; i < at.count; ++i)
            own[i] = near(at.base + i, of_group);
    }
    // All experts of the lane with a value of at least its bound as candidates;
    // their number, which may be above what there is room for.
    __device__ __forceinline__ int collect(bool live, float bound, bool of_group)
    {
        int found = 0;
#pragma unroll 1
        for (int i = 0; i < a.per; ++i) {
            const float v = live && i < at.count ? own[i] : -INFINITY;
            const bool is = v > -INFINITY && v >= bound;
            const unsigned lanes = __ballot_sync(0xffffffffu, is);
            const int to = found + __popc(lanes & ((1u << lane) - 1u));
            if (is && to < kMaxFound)
                slots.expert[to] = at.base + i;
            found += __popc(lanes);
        }
        __syncwarp();
#pragma unroll 1
        for (int i = lane; i < min(found, kMaxFound); i += 32)
            slots.found[i] = exact(slots.expert[i], of_group);
        __syncwarp();
        return found;
    }
    // A bound with the values' errors to spare.
    __device__ __forceinline__ float below(float v) const { return v - (slack + 0x1p-21f * fabsf(v)); }

    __device__ __forceinline__ unsigned groups()         // a bit for each group that is in
    {
        if (a.groups == 1)
            return 1u;
        form(true);
        float b1 = -INFINITY, b2 = -INFINITY;
#pragma unroll 1
        for (int i = 0; i < at.count; ++i)
            best_two(b1, b2, own[i], -INFINITY);
#pragma unroll 1
        for (int o = 1; o < a.lanes; o <<= 1) {
            const float o1 = __shfl_xor_sync(0xffffffffu, b1, o), o2 = __shfl_xor_sync(0xffffffffu, b2, o);
            best_two(b1, b2, o1, o2);
        }
        const int found = collect(at.group < a.groups, below(a.group_top == 2 ? b2 : b1), true);
        // lane g: group g's value, from the candidates or from all of its experts
        uint64_t e1 = 0, e2 = 0;
        if (lane < a.groups) {
            if (found <= kMaxFound) {
                const int lo = lane * a.of_group, hi = lo + a.of_group;
#pragma unroll 1
                for (int i = 0; i < found; ++i)
                    if (slots.expert[i] >= lo && slots.expert[i] < hi)
                        best_two(e1, e2, slots.found[i], static_cast<uint64_t>(0));
            } else {
#pragma unroll 1
                for (int e = lane * a.of_group; e < (lane + 1) * a.of_group; ++e)
                    if (near(e, true) > -INFINITY)
                        best_two(e1, e2, exact(e, true), static_cast<uint64_t>(0));
            }
        }
        const uint64_t v = a.group_top == 2 && e2 ? order64(value64(e1) + value64(e2)) : e1;
        int better = 0;
#pragma unroll 1
        for (int g = 0; g < a.groups; ++g) {
            const uint64_t o = __shfl_sync(0xffffffffu, v, g);
            better += o > v || (o == v && g < lane);
        }
        return __ballot_sync(0xffffffffu, lane < a.groups && better < a.topk_groups);
    }
    __device__ __forceinline__ int choose()
    {
        const unsigned in = groups();                    // by all lanes, also those without a group
        const bool live = at.group < a.groups && (in >> at.group & 1u);
        if (a.groups == 1 || !a.bias)
            form(false);
        float top = -INFINITY, last = -INFINITY;
#pragma unroll 1
        for (int i = 0; live && i < at.count; ++i)
            top = fmaxf(top, own[i]);
#pragma unroll 1
        for (int lanes = 0; lanes <= a.k;) {
            last = warp_max(top);
            if (last == -INFINITY)
                break;
            lanes += __popc(__ballot_sync(0xffffffffu, top == last));
            top = top == last ? -INFINITY : top;
        }
        const int found = collect(live, a.bias && last > -INFINITY ? below(last) : last, false);
        if (found <= kMaxFound) {
#pragma unroll 1
            for (int i = lane; i < found; i += 32) {
                const uint64_t v = slots.found[i];
                const int e = slots.expert[i];
                int rank = 0;
#pragma unroll 4
                for (int j = 0; j < found; ++j)
                    rank += slots.found[j] > v || (slots.found[j] == v && slots.expert[j] < e);
                if (rank < a.k)
                    slots.sorted[rank] = e;
            }
            __syncwarp();
            return lane < a.k && lane < found ? static_cast<int>(slots.sorted[lane]) : -1;
        }
        // that many equal values: one slot after the other, over all experts
        uint64_t taken = live ? 0ull : ~0ull;
        int slot = -1;
#pragma unroll 1
        for (int j = 0; j < a.k; ++j) {
            uint64_t best = 0;
            int at_best = -1;
#pragma unroll 1
            for (int i = 0; i < at.count; ++i)
                if (!(taken >> i & 1) && own[i] > -INFINITY) {
                    const uint64_t v = exact(at.base + i, false);
                    if (v > best) {
                        best = v;
                        at_best = i;
                    }
                }
            uint64_t first = best;
#pragma unroll 1
            for (int o = 16; o > 0; o >>= 1) {
                const uint64_t n = __shfl_xor_sync(0xffffffffu, first, o);
                first = n > first ? n : first;
            }
            const unsigned have = __ballot_sync(0xffffffffu, at_best >= 0 && best == first);
            if (!have)
                break;
            const int wl = __ffs(have) - 1;
            const int e = __shfl_sync(0xffffffffu, at.base + at_best, wl);
            if (lane == wl)
                taken |= 1ull << at_best;
            if (lane == j)
                slot = e;
        }
        return slot;
    }
};

// A token's ids and weights, and its part of the load.
__device__ __forceinline__ void put(const Args &a, uint32_t t, int slot, float w, bool bad, int lane, int *load)
{
    if (lane < a.k) {
        a.ids[static_cast<int64_t>(t) * a.k + lane] = slot;
        a.w[static_cast<int64_t>(t) * a.k + lane] = bad ? __uint_as_float(0x7FC00000u) : w;
        if (a.load && slot >= 0)
            atomicAdd(load + slot, 1);
    }
}

// All of a token by the exact choice.
template <typename T>
__device__ __noinline__ void route_exact(const Args &a, uint32_t t, Slots &slots, int *load, int lane)
{
    const T *l = static_cast<const T *>(a.logits) + static_cast<int64_t>(t) * a.E;
    bool bad = false;
    for (int e = lane; e < a.E; e += 32)
        bad |= !(value(l[e]) < INFINITY) || (a.bias && !(a.bias[e] < INFINITY));
    bad = __any_sync(0xffffffffu, bad);
    Exact<T> exact(a, l, slots, lane);
    const int slot = exact.choose();
    const float my_l = slot >= 0 ? value(l[slot]) : 0.f;
    put(a, t, slot, weight(a.sigmoid, a.renorm, a.scale, my_l, slot >= 0, static_cast<float>(exact.m), static_cast<float>(exact.z)), bad,
        lane, load);
    __syncwarp();
}

// Whether any of the n candidates behind the expert of the last slot is nearer to it
// than the values' errors, and not by equal inputs, whose order is known.
template <typename T>
__device__ __noinline__ bool others_near(const Args &a, const T *l, const Slots &slots, int n, float slack, int lane)
{
    const uint64_t last = slots.sorted[a.k - 1];
    const float x = value_of(last);
    const int e = slots.expert[index_of(last)];
    bool near = false;
    for (int i = lane; i < n; i += 32) {
        const float y = value_of(slots.found[i]);
        const int o = slots.expert[i];
        if (slots.found[i] < last && x - y <= slack + 0x1p-23f * fmaxf(fabsf(x), fabsf(y)))
            near = near || value(l[e]) != value(l[o]) || a.bias[e] != a.bias[o];
    }
    return __any_sync(0xffffffffu, near);
}

// A bit for each of a lane's experts.
template <int PER>
using Mask = std::conditional_t<(PER > 32), uint64_t, uint32_t>;
__device__ __forceinline__ int popc(uint32_t m) { return __popc(m); }
__device__ __forceinline__ int popc(uint64_t m) { return __popcll(m); }
__device__ __forceinline__ int first_of(uint32_t m) { return __ffs(m) - 1; }
__device__ __forceinline__ int first_of(uint64_t m) { return __ffsll(m) - 1; }

// Consecutive elements of a row: 16 bytes at a time where FULL says that every
// lane has PER of them, on their natural alignment.
template <typename T, int PER, bool FULL>
__device__ __forceinline__ void load_row(const T *p, int count, float (&v)[PER])
{
    constexpr int kWords = PER * static_cast<int>(sizeof(T)) / 4;
    if constexpr (FULL && kWords >= 1) {
        uint32_t w[kWords];
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if constexpr (kWords % 4 == 0) {
                if (i % 4 == 0) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(reinterpret_cast<const uint32_t *>(p) + i);
                    w[i] = x.x, w[i + 1] = x.y, w[i + 2] = x.z, w[i + 3] = x.w;
                }
            } else if constexpr (kWords == 2) {
                if (i == 0) {
                    const uint2 x = *reinterpret_cast<const uint2 *>(p);
                    w[0] = x.x, w[1] = x.y;
                }
            } else {
                w[i] = reinterpret_cast<const uint32_t *>(p)[i];
            }
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if constexpr (sizeof(T) == 4) {
                v[i] = __uint_as_float(w[i]);
            } else {
                float lo, hi;
                if constexpr (std::is_same<T, __half>::value)
                    f16x2_to_float(w[i / 2], lo, hi);
                else
                    bf16x2_to_float(w[i / 2], lo, hi);
                v[i] = i % 2 ? hi : lo;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            v[i] = i < count ? value(p[i]) : -INFINITY;
    }
}

template <typename T, int PER>
__device__ __forceinline__ void store_row(T *p, const float (&v)[PER])
{
    constexpr int kWords = PER * static_cast<int>(sizeof(T)) / 4;
    uint32_t w[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
        if constexpr (sizeof(T) == 4)
            w[i] = __float_as_uint(v[i]);
        else
            w[i] = gmm::pack2<T>(v[2 * i], v[2 * i + 1]);
    }
#pragma unroll
    for (int i = 0; i < kWords; i += 4) {
        uint32_t *to = reinterpret_cast<uint32_t *>(p) + i;
        if constexpr (kWords % 4 == 0)
            *reinterpret_cast<uint4 *>(to) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
        else if constexpr (kWords == 2)
            *reinterpret_cast<uint2 *>(to) = make_uint2(w[0], w[1]);
        else
            *to = w[0];
    }
}

// Warps go over the tokens.  Of a token, each lane finds its best value; the
// (k + 1)-th best of those bounds what can be chosen, usually some ten values,
// which the lanes then take one each and rank.  Tokens that binary32 cannot decide
// are marked, and done at the end, so that their code is out of this loop.
constexpr int kLater = INT_MIN;

template <typename T, int PER, bool FULL>
__global__ void __launch_bounds__(kWarps * 32, PER <= 8 ? 2 : 1) route_kernel(const Args a)
{
    __shared__ Slots all[kWarps];
    __shared__ int load[kMaxExperts];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int lane = threadIdx.x & 31;
    Slots &slots = all[threadIdx.x >> 5];
    if (a.load) {
        for (int e = threadIdx.x; e < a.E; e += kWarps * 32)
            load[e] = 0;
        __syncthreads();
    }
    const Place at(a, lane);
    const bool two = a.groups > 1 && a.group_top == 2 && !a.bias;      // group values from scores, choice by logits
    const int rounds = a.bias ? a.k + 1 : a.k;
    constexpr bool kKeep = PER <= 16;                                   // the biases stay in registers
    float b[PER];
    if (kKeep && a.bias)
        load_row<float, PER, FULL>(a.bias + at.base, at.count, b);
    const uint32_t M = a.M, step = gridDim.x * kWarps, begin = blockIdx.x * kWarps + (threadIdx.x >> 5);
    bool later = false;

    for (uint32_t t = begin; t < M; t += step) {
        const T *l = static_cast<const T *>(a.logits) + static_cast<int64_t>(t) * a.E;
        float v[PER], c[PER];
        load_row<T, PER, FULL>(l + at.base, at.count, v);
        bool bad = false, finite = FULL;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            finite = finite && fabsf(v[i]) < INFINITY;
        if (!__all_sync(0xffffffffu, finite)) {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (!(v[i] < INFINITY)) {              // the token's weights will be NaN
                    bad = true;
                    v[i] = -INFINITY;
                }
        }
        // row maximum and sum
        float m = -INFINITY, z = 1.f;
        if (!a.sigmoid && (a.bias || two || !a.renorm)) {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                m = fmaxf(m, v[i]);
            m = warp_max(m);
            z = 0.f;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                z += v[i] > -INFINITY ? __expf(v[i] - m) : 0.f;
            z = warp_sum(z);
        }
        const float rz = 1.f / z, slack = slack_of(a, rz);
        float b1 = -INFINITY, b2 = -INFINITY;          // the lane's best, of what group values are made of
        if (a.bias || two) {
            if (!kKeep && a.bias)
                load_row<float, PER, FULL>(a.bias + at.base, at.count, b);
            bool plain = finite;
            if (a.sigmoid) {
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    c[i] = fast_sigmoid(v[i]);
            } else {
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    c[i] = __expf(v[i] - m) * rz;
            }
            if (a.bias) {
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    c[i] += b[i];
                    plain = plain && fabsf(c[i]) < INFINITY;
                }
            }
            if (!__all_sync(0xffffffffu, plain)) {
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    if (a.bias && i < at.count && !(b[i] < INFINITY))
                        bad = true;
                    if (!(v[i] > -INFINITY) || !(fabsf(c[i]) < INFINITY))
                        c[i] = -INFINITY;
                }
            }
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                b2 = fmaxf(b2, fminf(b1, c[i]));
                b1 = fmaxf(b1, c[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                b1 = fmaxf(b1, v[i]);
        }
        float top = b1, second = b2;                   // the lane's best, of what experts are chosen by
        if (!a.bias) {
            top = second = -INFINITY;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                c[i] = v[i];
                if (a.groups > 1)                      // all lanes are in otherwise, mostly more than are needed
                    second = fmaxf(second, fminf(top, v[i]));
                top = fmaxf(top, v[i]);
            }
        }
        bool close = false;                            // in this lane's view; what follows from it is decided together
        bool live = at.group < a.groups;
        if (a.groups > 1) {
            for (int o = 1; o < a.lanes; o <<= 1) {
                const float o1 = __shfl_xor_sync(0xffffffffu, b1, o), o2 = __shfl_xor_sync(0xffffffffu, b2, o);
                best_two(b1, b2, o1, o2);
            }
            // half the sum of the two best: it stays finite whatever the biases, and groups without experts alone are at -inf
            const float part = a.group_top == 2 ? 0.5f : 1.f;
            const float h1 = part * b1, h2 = a.group_top == 2 && b2 > -INFINITY ? part * b2 : 0.f, whole = h1 + h2;
            float g = whole, in = -INFINITY;
            live = false;
            for (int j = 0; j < a.topk_groups; ++j) {  // the best of the groups that are left
                in = warp_max(g);
                const bool is = g == in;
                live = live || is;
                g = is ? -INFINITY : g;
            }
            if (__popc(__ballot_sync(0xffffffffu, live)) != a.topk_groups << a.shift) {
                // equal groups came in together, or there were none left: one by one, the first of equal ones first
                g = whole;
                live = false;
                for (int j = 0; j < a.topk_groups; ++j) {
                    in = warp_max(g);
                    const int best = __ffs(__ballot_sync(0xffffffffu, g == in)) - 1;
                    if (in > -INFINITY && (lane ^ best) >> a.shift == 0) {
                        live = true;
                        g = -INFINITY;
                    }
                }
            }
            if (a.bias || two) {
                const float size = h1 > -INFINITY ? fabsf(h1) + fabsf(h2) : 0.f;
                const float out = warp_max(g), apart = slack + 0x1p-22f * warp_max(size);
                close = in - out <= apart;
                if (close && a.sigmoid) {
                    // the groups that are in or out by less than their errors, by their values in binary64
                    const bool open = live ? whole - out <= apart : in - whole <= apart;
                    const int left = __popc(__ballot_sync(0xffffffffu, live && open)) >> a.shift;
                    float least = a.group_top == 2 ? b2 : b1;
                    least = fmaxf(least - 2.f * apart, -FLT_MAX);
                    Mask<PER> which = 0;
#pragma unroll
                    for (int i = 0; i < PER; ++i)
                        which |= open && (two ? fast_sigmoid(v[i]) : c[i]) >= least && v[i] > -INFINITY ? static_cast<Mask<PER>>(1) << i : 0;
                    uint64_t e1 = 0, e2 = 0;
                    for (; which; which &= which - 1) {
                        const int e = at.base + first_of(which);
                        const double x = sigmoid64(value(l[e])) + (a.bias ? static_cast<double>(a.bias[e]) : 0.0);
                        best_two(e1, e2, order64(x), static_cast<uint64_t>(0));
                    }
                    __syncwarp();
                    for (int o = 1; o < a.lanes; o <<= 1) {
                        const uint64_t o1 = __shfl_xor_sync(0xffffffffu, e1, o), o2 = __shfl_xor_sync(0xffffffffu, e2, o);
                        best_two(e1, e2, o1, o2);
                    }
                    const uint64_t exact = a.group_top == 2 && e2 ? order64(value64(e1) + value64(e2)) : e1;
                    int better = 0;
                    for (int i = 0; i < a.groups; ++i) {
                        const uint64_t o = __shfl_sync(0xffffffffu, exact, i << a.shift);
                        better += o > exact || (o == exact && i < at.group);
                    }
                    live = open ? better < left : live;
                    close = false;
                }
            }
        }
        // a bound of what can be chosen: as many of the lanes' two best as are needed are not below it
        float bound = -INFINITY;
        if (!live)
            top = second = -INFINITY;
#pragma unroll 3
        for (int j = 0; j < rounds; ++j) {             // (fewer than that: -inf, no bound)
            bound = warp_max(top);
            const bool is = top == bound;
            top = is ? second : top;
            second = is ? -INFINITY : second;
        }
        if (bound == -INFINITY && __popc(__ballot_sync(0xffffffffu, live)) * a.per > kMaxFound) {
            // few lanes, of one or two groups, with many experts each: their values in turn
            top = -INFINITY;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                top = live ? fmaxf(top, c[i]) : top;
            for (int j = 0; j < rounds; ++j) {
                bound = warp_max(top);
                if (top == bound) {
                    top = -INFINITY;
#pragma unroll
                    for (int i = 0; i < PER; ++i)
                        top = c[i] < bound ? fmaxf(top, c[i]) : top;
                }
            }
        }
        if (a.bias)                                    // and what may be as good
            bound -= slack + 0x1p-22f * fabsf(bound);
        bound = live ? fmaxf(bound, -FLT_MAX) : INFINITY;
        // what is not below it, by expert: the lanes' counts give each its place
        Mask<PER> which = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            which |= c[i] >= bound ? static_cast<Mask<PER>>(1) << i : 0;
        int to = popc(which);
        const int own = to;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int n = __shfl_up_sync(0xffffffffu, to, o);
            to += lane >= o ? n : 0;
        }
        const int found = __shfl_sync(0xffffffffu, to, 31);
        bool near = false;                             // the order may not be the exact values'
        int slot = -1;
        float my_l = 0.f;
        const int n = found <= kMaxFound ? found : 0;  // more: all that equal values
        if (n)
            for (to -= own; which; which &= which - 1)
                slots.expert[to++] = at.base + first_of(which);
        __syncwarp();
        // each lane takes one after the other, and finds its rank; equal ones are in order already
        for (int i = lane; i < n; i += 32) {
            const int e = slots.expert[i];
            const float x = value(l[e]);
            float y = x;
            if (a.bias)
                y = (a.sigmoid ? fast_sigmoid(x) : __expf(x - m) * rz) + a.bias[e];
            slots.found[i] = key64(y, i);
        }
        __syncwarp();
        for (int i = lane; i < n; i += 32) {
            const uint64_t own = slots.found[i];
            int rank = 0, j = 0;
            for (; j + 4 <= n; j += 4)
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    rank += slots.found[j + u] > own;
            for (; j < n; ++j)
                rank += slots.found[j] > own;
            if (rank <= a.k)
                slots.sorted[rank] = own;
        }
        __syncwarp();
        if (lane < min(a.k, n)) {
            const uint64_t own = slots.sorted[lane];
            slot = slots.expert[index_of(own)];
            my_l = value(l[slot]);
            if (a.bias && lane + 1 < n) {
                const uint64_t after = slots.sorted[lane + 1];
                const float x = value_of(own), y = value_of(after);
                // equal inputs have equal values, and are in order; behind the last slot others may follow them
                if (x - y <= slack + 0x1p-23f * fmaxf(fabsf(x), fabsf(y))) {
                    const int e = slots.expert[index_of(after)];
                    near = my_l != value(l[e]) || a.bias[slot] != a.bias[e] || lane == a.k - 1;
                }
            }
        }
        bool undecided = found > kMaxFound || close;
        if (__any_sync(0xffffffffu, near)) {
            near = __any_sync(0xffffffffu, near && lane != a.k - 1) || others_near<T>(a, l, slots, n, slack, lane);
            undecided = undecided || (near && !a.sigmoid);
            // the candidates' values in binary64, one to a lane
            const int again = near && a.sigmoid ? n : 0;
            for (int i = lane; i < again; i += 32) {
                const int e = slots.expert[i];
                slots.found[i] = order64(sigmoid64(value(l[e])) + static_cast<double>(a.bias[e]));
            }
            __syncwarp();
            for (int i = lane; i < again; i += 32) {
                int rank = 0;
                for (int j = 0; j < again; ++j)
                    rank += slots.found[j] > slots.found[i] || (slots.found[j] == slots.found[i] && j < i);
                if (rank < a.k)
                    slots.sorted[rank] = slots.expert[i];
            }
            __syncwarp();
            if (lane < min(a.k, again)) {
                slot = static_cast<int>(slots.sorted[lane]);
                my_l = value(l[slot]);
            }
        }
        const float w = weight(a.sigmoid, a.renorm, a.scale, my_l, slot >= 0, m, z);
        if (!undecided)
            put(a, t, slot, w, __any_sync(0xffffffffu, bad), lane, load);
        else if (lane == 0)
            a.ids[static_cast<int64_t>(t) * a.k] = kLater;
        later = later || undecided;
        __syncwarp();                                  // the slots are the next token's
    }
    if (later)
        for (uint32_t t = begin; t < M; t += step) {
            if (a.ids[static_cast<int64_t>(t) * a.k] == kLater)
                route_exact<T>(a, t, slots, load, lane);
            __syncwarp();
        }
    if (a.load) {
        __syncthreads();
        for (int e = threadIdx.x; e < a.E; e += kWarps * 32)
            if (load[e])
                atomicAdd(a.load + e, load[e]);
    }
}

// ---- gradient of the logits ------------------------------------------------
// With s the score of a slot, w its weight, D = sum w_i dw_i / scale (renorm):
//   softmax, renorm   dl_j = w_j (dw_j - D) at the chosen, 0 elsewhere
//   softmax           dl_e = s_e (scale dw_e [chosen] - sum scale s_i dw_i)
//   sigmoid, renorm   dl_j = w_j (1 - s_j) (dw_j - D)
//   sigmoid           dl_j = scale s_j (1 - s_j) dw_j
// An expert in several slots gets their sum.
struct BwdArgs {
    const float *dw;
    const void *logits;
    const int32_t *ids;
    int M, E, k, sigmoid, renorm;
    float scale;
    void *dl;
};

// Where a row of the gradient holds expert e: the pieces of four of a lane's PER
// experts lie apart, so that the lanes' pieces are neighbours.
template <int PER>
__device__ __forceinline__ int place_of(int e)
{
    return PER < 4 ? e : e % PER / 4 * 128 + e / PER * 4 + e % 4;
}

// PER: experts of a lane, neighbouring ones that it loads and stores as vectors; 0:
// any number, every 32nd one.
template <typename T, int PER>
__global__ void __launch_bounds__(kBwdWarps * 32) route_bwd_kernel(const BwdArgs a)
{
    extern __shared__ __align__(16) float rows[];      // a row of E for each warp
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int lane = threadIdx.x & 31;
    float *row = rows + (threadIdx.x >> 5) * a.E;
    const uint32_t t = blockIdx.x * kBwdWarps + (threadIdx.x >> 5);
    if (t >= static_cast<uint32_t>(a.M))
        return;
    const T *l = static_cast<const T *>(a.logits) + static_cast<int64_t>(t) * a.E;
    T *dl = static_cast<T *>(a.dl) + static_cast<int64_t>(t) * a.E;
    const bool dense = !a.sigmoid && !a.renorm;
    int e = -1;
    float dw = 0.f, lj = 0.f;
    if (lane < a.k) {
        e = a.ids[static_cast<int64_t>(t) * a.k + lane];
        if (e < 0 || e >= a.E) {
            e = -1;
        } else {
            dw = a.dw[static_cast<int64_t>(t) * a.k + lane];
            lj = value(l[e]);
            if (lj == -INFINITY)
                e = -1;                                // not an expert that the choice can have given
        }
    }
    float m = -INFINITY, z = 0.f;
    bool bad = false;
    constexpr int kOwn = PER ? PER : 1;
    float v[kOwn];                                     // logits, then exp(logit - m)
    if constexpr (PER > 0) {
        load_row<T, kOwn, true>(l + lane * PER, PER, v);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            bad |= !(v[i] < INFINITY);
            if (PER < 4)
                row[lane * PER + i] = 0.f;
            else if (i % 4 == 0)
                reinterpret_cast<float4 *>(row)[i * 8 + lane] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if (dense) {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                m = fmaxf(m, v[i]);
            m = warp_max(m);
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                v[i] = v[i] > -INFINITY ? expf(v[i] - m) : 0.f;
                z += v[i];
            }
            z = warp_sum(z);
        }
    } else {
        for (int i = lane; i < a.E; i += 32) {
            const float x = value(l[i]);
            bad |= !(x < INFINITY);
            m = fmaxf(m, x);
            row[i] = 0.f;
        }
        if (dense) {
            m = warp_max(m);
            for (int i = lane; i < a.E; i += 32)
                z += m > -INFINITY ? expf(value(l[i]) - m) : 0.f;
            z = warp_sum(z);
        }
    }
    bad = __any_sync(0xffffffffu, bad);
    const float w = weight(a.sigmoid, a.renorm, a.scale, lj, e >= 0, m, z);
    float g = e >= 0 ? w * dw : 0.f;
    const float sum = warp_sum(g);
    if (a.renorm)
        g -= w * (sum / a.scale);
    if (a.sigmoid)
        g *= sigmoid(-lj);
    // slots that share an expert: the lowest adds them up
    const unsigned peers = __match_any_sync(0xffffffffu, e);
    if (__any_sync(0xffffffffu, e >= 0 && peers != 1u << lane)) {
        float total = 0.f;
        for (int j = 0; j < a.k; ++j) {
            const float o = __shfl_sync(0xffffffffu, g, j);
            if (peers >> j & 1)
                total += o;
        }
        if (e >= 0 && (peers & ((1u << lane) - 1u)))
            e = -1;
        g = total;
    }
    __syncwarp();
    if (e >= 0)
        row[PER ? place_of<kOwn>(e) : e] = g;
    __syncwarp();
    const float f = z > 0.f ? sum / z : 0.f;           // z is 0 where no expert is left, else at least 1
    if constexpr (PER > 0) {
        float d[kOwn];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (PER < 4) {
                d[i] = row[lane * PER + i];
            } else if (i % 4 == 0) {
                const float4 q = reinterpret_cast<const float4 *>(row)[i * 8 + lane];
                d[i] = q.x, d[(i + 1) % kOwn] = q.y, d[(i + 2) % kOwn] = q.z, d[(i + 3) % kOwn] = q.w;
            }
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (dense)
                d[i] -= v[i] * f;
            d[i] = bad ? __uint_as_float(0x7FC00000u) : d[i];
        }
        store_row<T, kOwn>(dl + lane * PER, d);
    } else {
        for (int i = lane; i < a.E; i += 32) {
            float d = row[i];
            if (dense) {
                const float x = value(l[i]);
                d -= x > -INFINITY ? expf(x - m) * f : 0.f;
            }
            dl[i] = fp4::from_float<T>(bad ? __uint_as_float(0x7FC00000u) : d);
        }
    }
}

template <typename T>
static cudaError_t launch(Args &a, cudaStream_t s)
{
    int lanes = 32, shift = 5;
    for (int g = 1; g < a.groups; g <<= 1, --shift)
        lanes >>= 1;
    a.lanes = lanes;
    a.shift = shift;
    a.of_group = a.E / a.groups;
    a.per = (a.of_group + lanes - 1) / lanes;
    // every lane has all of its experts, and they begin on the alignment of its loads
    auto full = [&](int per) {
        const size_t unit = sizeof(T) * per < 16 ? sizeof(T) * per : 16;
        return a.per == per && a.of_group == per * lanes && a.groups * lanes == 32 && aligned(a.logits, unit) &&
               aligned(a.bias, per * 4 < 16 ? per * 4 : 16);
    };
    const int64_t wanted = (static_cast<int64_t>(a.M) + kWarps - 1) / kWarps, most = device_sm_count() * (a.per <= 8 ? 2 : 1);
    const dim3 grid(static_cast<unsigned>(wanted < most ? wanted : most)), block(kWarps * 32);
    auto k = full(2)       ? route_kernel<T, 2, true>
             : full(4)     ? route_kernel<T, 4, true>
             : full(8)     ? route_kernel<T, 8, true>
             : full(16)    ? route_kernel<T, 16, true>
             : a.per <= 2  ? route_kernel<T, 2, false>
             : a.per <= 4  ? route_kernel<T, 4, false>
             : a.per <= 8  ? route_kernel<T, 8, false>
             : a.per <= 16 ? route_kernel<T, 16, false>
             : a.per <= 32 ? route_kernel<T, 32, false>
                           : route_kernel<T, kMaxPer, false>;
    return launch_pdl(k, grid, block, 0, s, a);
}

template <typename T>
static cudaError_t launch_bwd(const BwdArgs &a, dim3 grid, dim3 block, size_t smem, cudaStream_t s)
{
    auto full = [&](int per) {
        const size_t unit = sizeof(T) * per < 16 ? sizeof(T) * per : 16;
        return a.E == 32 * per && aligned(a.logits, unit) && aligned(a.dl, unit);
    };
    auto k = full(2)    ? route_bwd_kernel<T, 2>
             : full(4)  ? route_bwd_kernel<T, 4>
             : full(8)  ? route_bwd_kernel<T, 8>
             : full(16) ? route_bwd_kernel<T, 16>
                        : route_bwd_kernel<T, 0>;
    return launch_pdl(k, grid, block, smem, s, a);
}

static bool how(int32_t E, int32_t k, int32_t score, int32_t renorm, float scale)
{
    return E >= 1 && k >= 1 && k <= E && (score == MOE_SCORE_SOFTMAX || score == MOE_SCORE_SIGMOID) &&
           (renorm == 0 || renorm == 1) && scale > 0.f && scale < INFINITY;
}

}  // namespace route
}  // namespace moe

using namespace moe;

MOE_API moe_status_t moe_route(const void *logits, int32_t ldt, const float *bias, int32_t M, int32_t E, int32_t k,
                               int32_t score, int32_t groups, int32_t topk_groups, int32_t group_top, int32_t renorm,
                               float scale, int32_t *topk_ids, float *topk_w, int32_t *load, void *stream)
{
    if (M < 0 || !route::how(E, k, score, renorm, scale) || groups < 1 || E % groups != 0 || topk_groups < 1 ||
        topk_groups > groups || k > static_cast<int64_t>(topk_groups) * (E / groups) || group_top < 1 || group_top > 2)
        return MOE_ERR_INVALID_ARG;
    if ((ldt != MOE_BF16 && ldt != MOE_FP16 && ldt != MOE_FP32) || E > route::kMaxExperts || k > route::kMaxK ||
        groups > route::kMaxGroups || M > INT32_MAX / k)
        return MOE_ERR_UNSUPPORTED;
    if (M == 0)
        return MOE_OK;
    if (!logits || !topk_ids || !topk_w || !aligned(logits, ldt == MOE_FP32 ? 4 : 2) || !aligned(bias, 4) ||
        !aligned(topk_ids, 4) || !aligned(topk_w, 4) || !aligned(load, 4))
        return MOE_ERR_INVALID_ARG;
    route::Args a{logits, bias, M, E, k, groups, topk_groups, group_top, score == MOE_SCORE_SIGMOID, renorm, scale,
                  0, 0, 0, 0, topk_ids, topk_w, load};
    cudaStream_t s = as_stream(stream);
    const cudaError_t e = ldt == MOE_BF16   ? route::launch<__nv_bfloat16>(a, s)
                          : ldt == MOE_FP16 ? route::launch<__half>(a, s)
                                            : route::launch<float>(a, s);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

MOE_API moe_status_t moe_route_bwd(const float *dw, const void *logits, int32_t ldt, const int32_t *topk_ids, int32_t M,
                                   int32_t E, int32_t k, int32_t score, int32_t renorm, float scale, void *dlogits,
                                   void *stream)
{
    if (M < 0 || !route::how(E, k, score, renorm, scale))
        return MOE_ERR_INVALID_ARG;
    if ((ldt != MOE_BF16 && ldt != MOE_FP16 && ldt != MOE_FP32) || E > route::kMaxExperts || k > route::kMaxK ||
        M > INT32_MAX / k)
        return MOE_ERR_UNSUPPORTED;
    if (M == 0)
        return MOE_OK;
    const size_t size = ldt == MOE_FP32 ? 4 : 2;
    if (!dw || !logits || !topk_ids || !dlogits || !aligned(dw, 4) || !aligned(logits, size) || !aligned(topk_ids, 4) ||
        !aligned(dlogits, size))
        return MOE_ERR_INVALID_ARG;
    const route::BwdArgs a{dw, logits, topk_ids, M, E, k, score == MOE_SCORE_SIGMOID, renorm, scale, dlogits};
    const int64_t ctas = (static_cast<int64_t>(M) + route::kBwdWarps - 1) / route::kBwdWarps;
    const dim3 grid(static_cast<unsigned>(ctas)), block(route::kBwdWarps * 32);
    const size_t smem = sizeof(float) * route::kBwdWarps * E;                  // at most 16 KB
    cudaStream_t s = as_stream(stream);
    const cudaError_t e = ldt == MOE_BF16   ? route::launch_bwd<__nv_bfloat16>(a, grid, block, smem, s)
                          : ldt == MOE_FP16 ? route::launch_bwd<__half>(a, grid, block, smem, s)
                                            : route::launch_bwd<float>(a, grid, block, smem, s);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
