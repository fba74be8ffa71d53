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
// can be (a share of about 1e-3 of the tokens at logits of spread 1), it forms
// that token's anew in binary64.  Logits without a bias are compared as they are.
//
// A lane holds consecutive experts of one group, and a group takes a power of two
// of neighbouring lanes, so that the lowest lane that holds a maximum also holds
// the lowest index.
#include "common.cuh"
#include "fp4.cuh"
#include "gmm_common.cuh"
#include "ragged.cuh"
#include "topk.cuh"

namespace moe {
namespace route {

constexpr int kWarps = 4;
constexpr int kMaxExperts = ragged::kMaxExperts;
constexpr int kMaxK = 32, kMaxGroups = 32, kMaxPer = 64;

struct Args {
    const void *logits;
    const float *bias;
    int M, E, k, groups, topk_groups, group_top, sigmoid, renorm;
    float scale;
    int of_group, lanes, per;            // experts of a group, lanes of a group, experts of a lane (at most)
    int32_t *ids;
    float *w;
    int32_t *load;
};

template <typename T>
__device__ __forceinline__ float value(T v) { return static_cast<float>(v); }

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// The two best of two pairs (a1 >= a2, b1 >= b2).
template <typename F>
__device__ __forceinline__ void best_two(F &a1, F &a2, F b1, F b2)
{
    const F lo = a1 < b1 ? a1 : b1, hi = a1 < b1 ? b1 : a1, s = a2 < b2 ? b2 : a2;
    a1 = hi;
    a2 = lo < s ? s : lo;
}

// A lane's place: its first expert, how many it has.
struct Place {
    int group, base, count;
    __device__ __forceinline__ Place(const Args &a, int lane)
    {
        group = lane / a.lanes;
        const int first = (lane - group * a.lanes) * a.per;
        base = group * a.of_group + first;
        count = group < a.groups ? min(max(a.of_group - first, 0), a.per) : 0;
    }
};

// Whether the lane's group is among the best: its value against every other's,
// the lower group first among equal ones.  Values of 0 experts are -inf.
template <typename F>
__device__ __forceinline__ bool in_best(const Args &a, int group, F v)
{
    int better = 0;
    for (int g = 0; g < a.groups; ++g) {
        const F o = __shfl_sync(0xffffffffu, v, g * a.lanes);
        better += o > v || (o == v && g < group);
    }
    return group < a.groups && better < a.topk_groups;
}

// The choice of one token in binary64: lane j < k receives slot j's expert, or -1.
template <typename T>
__device__ __noinline__ int choose_exact(const Args &a, const T *l, int lane)
{
    const Place at(a, lane);
    double v[kMaxPer];                  // what the choice goes by
    double m = -INFINITY, z = 1.0;
    if (!a.sigmoid) {
        for (int i = 0; i < at.count; ++i)
            m = fmax(m, static_cast<double>(value(l[at.base + i])));
        for (int o = 16; o > 0; o >>= 1)
            m = fmax(m, __shfl_xor_sync(0xffffffffu, m, o));
        z = 0.0;
        if (m > -INFINITY)
            for (int i = 0; i < at.count; ++i)
                z += exp(static_cast<double>(value(l[at.base + i])) - m);
        for (int o = 16; o > 0; o >>= 1)
            z += __shfl_xor_sync(0xffffffffu, z, o);
    }
    double b1 = -INFINITY, b2 = -INFINITY;
    for (int i = 0; i < at.count; ++i) {
        const double x = value(l[at.base + i]);
        double s = -INFINITY;
        if (x > -INFINITY)
            s = a.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - m) / z;
        v[i] = a.bias ? s + static_cast<double>(a.bias[at.base + i]) : x;
        best_two(b1, b2, a.bias || a.group_top == 2 ? (a.bias ? v[i] : s) : x, -static_cast<double>(INFINITY));
    }
    bool live = at.group < a.groups;
    if (a.groups > 1) {
        for (int o = 1; o < a.lanes; o <<= 1) {
            const double o1 = __shfl_xor_sync(0xffffffffu, b1, o), o2 = __shfl_xor_sync(0xffffffffu, b2, o);
            best_two(b1, b2, o1, o2);
        }
        live = in_best(a, at.group, a.group_top == 2 && b2 > -INFINITY ? b1 + b2 : b1);
    }
    uint64_t taken = live ? 0ull : ~0ull;
    int slot = -1;
    for (int j = 0; j < a.k; ++j) {
        double bv = -INFINITY;
        int bi = -1;
        for (int i = 0; i < at.count; ++i)
            if (!(taken >> i & 1) && v[i] > bv) {
                bv = v[i];
                bi = i;
            }
        double top = bv;
        for (int o = 16; o > 0; o >>= 1)
            top = fmax(top, __shfl_xor_sync(0xffffffffu, top, o));
        const unsigned have = __ballot_sync(0xffffffffu, bi >= 0 && bv == top);
        if (!have)
            break;
        const int wl = __ffs(have) - 1;
        const int e = __shfl_sync(0xffffffffu, at.base + bi, wl);
        if (lane == wl)
            taken |= 1ull << bi;
        if (lane == j)
            slot = e;
    }
    return slot;
}

// The sigmoid of a logit from exp(-|l|), which does not overflow.
__device__ __forceinline__ float sigmoid(float l)
{
    const float t = expf(-fabsf(l)), r = 1.0f / (1.0f + t);
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
    // the chosen scores over their sum.  Sigmoids of logits below -60 are exp(l)
    // to within 2^-86, and a softmax of the logits does not lose them to zero.
    const float top = warp_max(live ? l : -INFINITY);
    const float s = !live ? 0.f : sigmoid_score && top > -60.f ? sigmoid(l) : expf(l - top);
    const float sum = warp_sum(s);
    return live ? s / sum * scale : 0.f;
}

template <typename T, int PER, bool SORT>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const Args a)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (t >= a.M)
        return;
    const T *l = static_cast<const T *>(a.logits) + static_cast<int64_t>(t) * a.E;
    const Place at(a, lane);
    float v[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i)
        v[i] = i < at.count ? value(l[at.base + i]) : -INFINITY;
    bool bad = false;                          // NaN or +inf: out of the choice, and the token's weights are NaN
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (!(v[i] < INFINITY)) {
            bad = true;
            v[i] = -INFINITY;
        }
    // row maximum and sum
    const bool two = a.groups > 1 && a.group_top == 2 && !a.bias;      // group values from scores, choice by logits
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
    const float rz = 1.f / z;
    // Largest error of a score: sigmoids 2^-21 (exp to 2 ulp where it is near 1,
    // the quotient); of a softmax (20 + PER / 2) 2^-23 of the largest score, the
    // sum's own error (its terms' 2 + 1.7 |x| ulp, |x| weighed by the scores at
    // most ln E; the additions') included.  Two values closer than twice that
    // and their additions' rounding may be in the other order.
    const float slack = a.sigmoid ? 0x1p-20f : (40 + PER) * 0x1p-23f * rz;
    float c[PER];
    float b1 = -INFINITY, b2 = -INFINITY;
    if (a.bias || two) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            float s;
            if (a.sigmoid) {
                const float e = __expf(-fabsf(v[i])), r = __fdividef(1.f, 1.f + e);
                s = v[i] >= 0.f ? r : e * r;
            } else {
                s = __expf(v[i] - m) * rz;
            }
            if (!(v[i] > -INFINITY))
                s = -INFINITY;
            if (a.bias) {
                float b = i < at.count ? a.bias[at.base + i] : 0.f;
                if (!(b < INFINITY)) {
                    bad = true;
                    b = -INFINITY;
                }
                s += b;
                c[i] = s;
            } else {
                c[i] = v[i];
            }
            best_two(b1, b2, s, -INFINITY);
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            c[i] = v[i];
            best_two(b1, b2, v[i], -INFINITY);
        }
    }
    bad = __any_sync(0xffffffffu, bad);
    bool close = false;
    bool live = at.group < a.groups;
    if (a.groups > 1) {
        for (int o = 1; o < a.lanes; o <<= 1) {
            const float o1 = __shfl_xor_sync(0xffffffffu, b1, o), o2 = __shfl_xor_sync(0xffffffffu, b2, o);
            best_two(b1, b2, o1, o2);
        }
        const float g = a.group_top == 2 && b2 > -INFINITY ? b1 + b2 : b1;
        live = in_best(a, at.group, g);
        if (a.bias || two) {
            const float in = -warp_max(live ? -g : -INFINITY), out = warp_max(live ? -INFINITY : g);
            const float size = warp_max((b1 > -INFINITY ? fabsf(b1) : 0.f) + (b2 > -INFINITY ? fabsf(b2) : 0.f));
            close = in - out <= 2.f * slack + 0x1p-22f * size;
        }
    }
    // selection: keys of the experts that are in, the rest 0
    uint32_t key[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i)
        key[i] = live && c[i] > -INFINITY ? topk_key(c[i]) : 0u;
    int idx[PER];
    uint64_t taken = 0;
    if constexpr (SORT) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            idx[i] = i;
#pragma unroll
        for (int i = 1; i < PER; ++i)
#pragma unroll
            for (int j = i; j > 0; --j) {
                const bool sw = key[j] > key[j - 1];
                const uint32_t ka = key[j - 1], kb = key[j];
                const int ia = idx[j - 1], ib = idx[j];
                key[j - 1] = sw ? kb : ka;
                key[j] = sw ? ka : kb;
                idx[j - 1] = sw ? ib : ia;
                idx[j] = sw ? ia : ib;
            }
    }
    int slot = -1, next = -1;
    float mine = -INFINITY, after = -INFINITY;
    const int rounds = a.bias ? a.k + 1 : a.k;
    for (int j = 0; j < rounds; ++j) {
        uint32_t head = 0;
        int hi = 0;
        if constexpr (SORT) {
            head = key[0];
            hi = idx[0];
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (!(taken >> i & 1) && key[i] > head) {
                    head = key[i];
                    hi = i;
                }
        }
        const uint32_t top = __reduce_max_sync(0xffffffffu, head);
        if (top == 0)
            break;
        const int wl = __ffs(__ballot_sync(0xffffffffu, head == top)) - 1;
        const int e = __shfl_sync(0xffffffffu, at.base + hi, wl);
        if (lane == wl) {
            if constexpr (SORT) {
#pragma unroll
                for (int i = 0; i + 1 < PER; ++i) {
                    key[i] = key[i + 1];
                    idx[i] = idx[i + 1];
                }
                key[PER - 1] = 0u;
            } else {
                taken |= 1ull << hi;
            }
        }
        if (lane == j) {
            slot = e;
            mine = topk_unkey(top);
        }
        if (lane == j - 1) {
            next = e;
            after = topk_unkey(top);
        }
    }
    if (lane >= a.k)
        slot = next = -1;
    float my_l = slot >= 0 ? value(l[slot]) : 0.f;
    if (a.bias && next >= 0) {
        // equal inputs have equal values, and are in order
        const bool same = my_l == value(l[next]) && a.bias[slot] == a.bias[next];
        close |= !same && mine - after <= slack + 0x1p-23f * fmaxf(fabsf(mine), fabsf(after));
    }
    if (__any_sync(0xffffffffu, close) && !bad) {
        slot = choose_exact<T>(a, l, lane);
        my_l = slot >= 0 ? value(l[slot]) : 0.f;
    }
    float w = weight(a.sigmoid, a.renorm, a.scale, my_l, slot >= 0, m, z);
    if (bad)
        w = __uint_as_float(0x7FC00000u);
    if (lane < a.k) {
        a.ids[static_cast<int64_t>(t) * a.k + lane] = slot;
        a.w[static_cast<int64_t>(t) * a.k + lane] = w;
        if (a.load && slot >= 0)
            atomicAdd(a.load + slot, 1);
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

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) route_bwd_kernel(const BwdArgs a)
{
    extern __shared__ float rows[];                    // a row of E for each warp
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int lane = threadIdx.x & 31;
    float *row = rows + (threadIdx.x >> 5) * a.E;
    const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (t >= a.M)
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
    for (int i = lane; i < a.E; i += 32) {
        const float x = value(l[i]);
        bad |= !(x < INFINITY);
        m = fmaxf(m, x);
        row[i] = 0.f;
    }
    bad = __any_sync(0xffffffffu, bad);
    if (dense) {
        m = warp_max(m);
        for (int i = lane; i < a.E; i += 32)
            z += m > -INFINITY ? expf(value(l[i]) - m) : 0.f;
        z = warp_sum(z);
    }
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
        row[e] = g;
    __syncwarp();
    for (int i = lane; i < a.E; i += 32) {
        float d = row[i];
        if (dense) {
            const float x = value(l[i]);
            d -= x > -INFINITY ? expf(x - m) / z * sum : 0.f;
        }
        dl[i] = fp4::from_float<T>(bad ? __uint_as_float(0x7FC00000u) : d);
    }
}

template <typename T>
static cudaError_t launch(Args &a, cudaStream_t s)
{
    int lanes = 32;
    for (int g = 1; g < a.groups; g <<= 1)
        lanes >>= 1;
    a.lanes = lanes;
    a.of_group = a.E / a.groups;
    a.per = (a.of_group + lanes - 1) / lanes;
    const dim3 grid((a.M + kWarps - 1) / kWarps), block(kWarps * 32);
    auto k = a.per <= 2   ? route_kernel<T, 2, true>
             : a.per <= 4 ? route_kernel<T, 4, true>
             : a.per <= 8 ? route_kernel<T, 8, true>
             : a.per <= 16 ? route_kernel<T, 16, false>
             : a.per <= 32 ? route_kernel<T, 32, false>
                           : route_kernel<T, kMaxPer, false>;
    return launch_pdl(k, grid, block, 0, s, a);
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
                  0, 0, 0, topk_ids, topk_w, load};
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
    const dim3 grid((M + route::kWarps - 1) / route::kWarps), block(route::kWarps * 32);
    const size_t smem = sizeof(float) * route::kWarps * E;                  // at most 16 KB
    cudaStream_t s = as_stream(stream);
    const cudaError_t e = ldt == MOE_BF16   ? launch_pdl(route::route_bwd_kernel<__nv_bfloat16>, grid, block, smem, s, a)
                          : ldt == MOE_FP16 ? launch_pdl(route::route_bwd_kernel<__half>, grid, block, smem, s, a)
                                            : launch_pdl(route::route_bwd_kernel<float>, grid, block, smem, s, a);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
