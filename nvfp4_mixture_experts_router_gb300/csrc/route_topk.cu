// Experts chosen from logits, and the gradient of the logits.
//
//   s = softmax(l) or sigmoid(l),  c = s + bias (l without a bias)
//   group score = max c, or the sum of the two largest s (+ bias)
//   ids = the K largest c in the topk_groups best groups
//   w_k = scale s_k, or scale s_k / sum_j s_j
//
// A warp has a token: EPL consecutive experts a lane, so that the order of the
// lanes and of a lane's registers is the order of the experts and ties fall to
// the lower one.  -infinity is an expert that cannot be
// chosen.  The K-th largest of the lanes' own largest is a
// border below which none of the K largest lies: the experts above it, few more
// than K, go to a lane each, which counts those before its own.  (Where they are
// more than the lanes, many being equal or K large, K rounds of a warp-wide
// maximum.)
//
// The choice has to be that of exact scores: an expert more or less is not a
// rounding.  Logits compare exactly.  Scores with a bias, and sums of two
// scores, are computed in FP32 with a bound of their error, and the border lies
// lower by twice that; where two values that decide are closer than their bounds,
// each lane computes its own again in FP64 (about one token in 700 with 256
// experts, standard normal logits and a bias: 2 of 17 us, as such a token ends last).
//
// Bound by a token's instructions and their latency, 6 times what the logits' bytes
// take: 760 with a bias, groups and 256 experts, which would be 10 of 17 us if the
// schedulers issued all the time; they do 47 % of it, as sorts and prefix sums are
// chains of dependent shuffles.  Measured on GB300, 16384 tokens, FP32: 256
// experts, top-8, sigmoid, bias, 4 of 8 groups 17 us (29 for 32768 tokens); without
// groups 13, softmax without a bias 10.4 and with one 18 (its FP64 sums); 64 experts,
// top-6 8.1; 1024 with a bias 48; top-32 of 256 46 (in rounds).  Backward
// 4.8 (3.8 TB/s: a launch's 2.6 and the latency of ids, their logits and the rows'
// stores), softmax not renormalized 8.4.  One token: 2.8 and 2.6.
#include <float.h>
#include <limits.h>
#include <math.h>

#include "row_vec.cuh"
#include "train_kernels.h"

namespace moe {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kRouteWarps = 8;      // tokens of a block, at most

struct RouteArgs {
    int T, E, K;
    const void* logits;
    int64_t stride;
    const float* bias;
    moe_route_rule rule;
    int* ids;
    float* w;
    bool wide, wide_bias;      // rows, and the bias, in vectors
    int size, span;            // experts of a group; log2 of its lanes, or -1
};

// The unsigned integer in the order of a float that is no NaN; not 0.
__device__ __forceinline__ uint32_t order_of(float v) {
    const int b = __float_as_int(v);
    return (uint32_t)(b ^ ((b >> 31) | (int)0x80000000));
}

// A logit as it counts: NaN as -infinity, at most the largest FP32 number.
__device__ __forceinline__ float as_logit(float v) { return fminf(fmaxf(v, -INFINITY), FLT_MAX); }

__device__ __forceinline__ float load_logit(const float* p) { return as_logit(*p); }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) { return as_logit(__bfloat162float(*p)); }

// The lane's EPL values, -infinity past the row's end.
template <typename T_, int EPL>
__device__ __forceinline__ void load_row(const T_* row, int E, bool wide, float (&l)[EPL]) {
    const int e0 = (threadIdx.x & 31) * EPL;
    constexpr int kMost = 16 / sizeof(T_), VEC = EPL < kMost ? EPL : kMost;
    if (VEC > 1 && wide) {
#pragma unroll
        for (int i = 0; i < EPL; i += VEC) {
            float u[VEC];
            if (e0 + i < E) {       // E is a multiple of VEC then
                RowVec<T_, VEC>::unpack(*reinterpret_cast<const typename RowVec<T_, VEC>::Raw*>(row + e0 + i), u);
            } else {
#pragma unroll
                for (int k = 0; k < VEC; ++k) u[k] = -INFINITY;
            }
#pragma unroll
            for (int k = 0; k < VEC; ++k) l[i + k] = u[k];
        }
    } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) l[i] = e0 + i < E ? (float)row[e0 + i] : -INFINITY;
    }
}

template <int EPL>
__device__ __forceinline__ void as_logits(float (&l)[EPL]) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) l[i] = as_logit(l[i]);
}

// Scores in FP32.  Of sigmoid the absolute error is below kSigmoidErr: e^-l is
// off by (3 + 1.18 |l|) 2^-23 of itself at most (the product with log2 e and ex2's
// documented 2^-22), which s (1 - s) takes to 0.75 + 0.27 units of 2^-23, and the
// sum and the reciprocal (documented 2^-23) add 2.5.  Of softmax, p = e^x / S with
// x = l - max, it is below (kSoftmaxErr + 1.18 |x|) 2^-23 p: 3 + 1.18 |x| of e^x as
// above; of S half a unit for each of its EPL + 4 roundings and 3 + 1.18 log E by its
// terms (their mean |x| is log E at most); 2.5 of the reciprocal and the product.  In
// all 15.1, 16.4, 18.2, 21.1, 25.9 and 34.7 for EPL = 1 to 32.  That is largest at x = 0.
constexpr float kUnit = 1.1920929e-07f;     // 2^-23
constexpr float kSigmoidErr = 4.0f * kUnit;
template <int EPL>
constexpr float kSoftmaxErr = (17.0f + 0.65f * EPL) * kUnit;    // times the largest p
constexpr float kTiny = 7.5e-37f;           // 2^-120, where the approximations flush to zero
__device__ __forceinline__ float exp_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.44269504f));
    return r;
}
__device__ __forceinline__ float sigmoid_fast(float l) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + exp_fast(-l)));
    return r;
}

struct Softmax {
    float max, inv;     // of the row; p = e^(l - max) inv
    __device__ __forceinline__ float of(float l) const { return exp_fast(l - max) * inv; }
};
template <int EPL>
__device__ __forceinline__ Softmax softmax_of(const float (&l)[EPL]) {
    float m = l[0], s = 0.0f;
#pragma unroll
    for (int i = 1; i < EPL; ++i) m = fmaxf(m, l[i]);
    m = warp_max(m);
    if (!(m > -INFINITY)) m = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) s += exp_fast(l[i] - m);
    s = warp_sum(s);
    return Softmax{m, s > 0.0f ? __fdividef(1.0f, s) : 0.0f};
}

// The scores of the lane's logits, in their place.
template <int EPL>
__device__ __forceinline__ void scores(bool sigmoid, const Softmax& soft, float (&l)[EPL]) {
    if (sigmoid) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) l[i] = sigmoid_fast(l[i]);
    } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) l[i] = soft.of(l[i]);
    }
}

// The first `lanes` lanes' values from the largest down, with those of the lanes up
// to the next power of two (a bitonic sort: Batcher 1968).
__device__ __forceinline__ float sorted_lanes(float v, int lanes) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1) {
        if (size >= 2 * lanes) break;
#pragma unroll
        for (int o = size >> 1; o > 0; o >>= 1) {
            const float u = __shfl_xor_sync(kAll, v, o);
            v = ((lane & o) == 0) == ((lane & size) == 0 || size == 32) ? fmaxf(v, u) : fminf(v, u);
        }
    }
    return v;
}
// The lane's number of `mine` things before its own in the order of the lanes, and of all.
__device__ __forceinline__ int before_lane(int mine, int* all) {
    int sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kAll, sum, o);
        if ((int)(threadIdx.x & 31) >= o) sum += v;
    }
    *all = __shfl_sync(kAll, sum, 31);
    return sum - mine;
}

// The two largest of a group of lanes' values, a >= b.
__device__ __forceinline__ void join_top2(float& a, float& b, float a2, float b2) {
    b = fmaxf(fminf(a, a2), fmaxf(b, b2));
    a = fmaxf(a, a2);
}
__device__ __forceinline__ void into_top2(float& a, float& b, float v) {
    b = fmaxf(b, fminf(a, v));
    a = fmaxf(a, v);
}

// ---- what FP32 cannot decide --------------------------------------------------------

// A token's scores in FP64: c of expert e, with the warp's S of a softmax.
template <typename T_>
struct Exact {
    const T_* row;
    const float* bias;
    bool sigmoid;
    double max, sum;
    __device__ __forceinline__ double operator()(int e) const {
        const double l = (double)load_logit(row + e);
        const double s = sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - max) / sum;
        return bias ? s + (double)bias[e] : s;
    }
};
template <typename T_, int EPL>
__device__ __forceinline__ Exact<T_> exact_of(const T_* row, const float* bias, bool sigmoid, int E, float max) {
    double s = 0.0;
    if (!sigmoid) {
        const int e0 = (threadIdx.x & 31) * EPL;
#pragma unroll 1
        for (int i = 0; i < EPL && e0 + i < E; ++i) s += exp((double)load_logit(row + e0 + i) - (double)max);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
    }
    return Exact<T_>{row, bias, sigmoid, (double)max, s};
}

// FP64 values are compared as integers in their order (FP64 runs at a 64th of the
// rate): those of all that is no NaN lie above kNoKey.
constexpr long long kNoKey = LLONG_MIN;
__device__ __forceinline__ long long key_of(double v) {
    const long long b = __double_as_longlong(v + 0.0);      // zeros alike
    return b ^ ((b >> 63) & LLONG_MAX);
}
__device__ __forceinline__ double of_key(long long k) { return __longlong_as_double(k ^ ((k >> 63) & LLONG_MAX)); }

// The topk_groups best groups, as a mask: lane g has group g's score, or NaN
// (kNoKey) for a group that does not exist.
template <typename F>
__device__ __forceinline__ uint32_t best_groups(F score, int groups, int take) {
    const int lane = threadIdx.x & 31;
    int above = 0;
    for (int g0 = 0; g0 < groups; g0 += 4)
#pragma unroll
        for (int g = g0; g < g0 + 4; ++g) {         // (NaN past the last group)
            const F v = __shfl_sync(kAll, score, g);
            above += v > score || (v == score && g < lane);
        }
    return __ballot_sync(kAll, lane < groups && above < take);
}

// The lane's experts in the taken groups of `size`, as a mask.
template <int EPL>
__device__ __forceinline__ uint32_t lane_mask(uint32_t taken, int size) {
    const int e0 = (threadIdx.x & 31) * EPL;
    int g = e0 / size, r = e0 - g * size;
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        m |= ((taken >> (g & 31)) & 1u) << i;       // past the last group: no experts
        if (++r == size) {
            r = 0;
            ++g;
        }
    }
    return m;
}

// The groups by FP64 scores.  can: a mask of the lane's experts that may be among
// their group's largest; s_c: E doubles of this warp; s_list: 32 entries.
template <typename T_, int EPL>
__device__ __noinline__ uint32_t exact_groups(const T_* row, const float* bias, bool sigmoid, int E, float max, int groups,
                                              int take, bool pair, uint32_t can, double* s_c, uint2* s_list) {
    const int lane = threadIdx.x & 31, e0 = lane * EPL, size = E / groups;
    const Exact<T_> f = exact_of<T_, EPL>(row, bias, sigmoid, E, max);
    int n, pos = before_lane(__popc(can), &n);
#pragma unroll 1
    for (int i = 0; i < EPL && e0 + i < E; ++i) {
        const bool look = (can >> i) & 1u;
        s_c[e0 + i] = look && n > 32 ? f(e0 + i) : -INFINITY;
        if (look && n <= 32) s_list[pos++].x = (uint32_t)(e0 + i);
    }
    __syncwarp();
    if (n <= 32 && lane < n) s_c[s_list[lane].x] = f((int)s_list[lane].x);     // one each
    __syncwarp();
    long long a = kNoKey, b = kNoKey;
    if (lane < groups) {
#pragma unroll 4
        for (int i = 0; i < size; ++i) {
            const long long v = key_of(s_c[lane * size + i]);
            const long long low = v > a ? a : v;
            if (v > a) a = v;
            if (low > b) b = low;
        }
        if (pair && b > key_of(-INFINITY)) a = key_of(of_key(a) + of_key(b));
    }
    __syncwarp();
    return best_groups(a, groups, take);
}

// The rank of the lane's expert e (-1: none) among the warp's, by FP64.
template <typename T_, int EPL>
__device__ __noinline__ int exact_rank(const T_* row, const float* bias, bool sigmoid, int E, float max, int e, int n) {
    const int lane = threadIdx.x & 31;
    const Exact<T_> f = exact_of<T_, EPL>(row, bias, sigmoid, E, max);
    const long long c = e >= 0 ? key_of(f(e)) : kNoKey;
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
        const long long v = __shfl_sync(kAll, c, j);
        rank += v > c || (v == c && j < lane);
    }
    return rank;
}

// The K largest c among the lane's experts `near` (a mask; every expert that may
// be one of them), in FP64.  Slot k's expert in lane k, or -1.
template <typename T_, int EPL>
__device__ __noinline__ int exact_choice(const T_* row, const float* bias, bool sigmoid, int E, float max, int K, uint32_t near,
                                         double* s_c) {
    const int lane = threadIdx.x & 31, e0 = lane * EPL;
    const Exact<T_> f = exact_of<T_, EPL>(row, bias, sigmoid, E, max);
#pragma unroll 1
    for (int i = 0; i < EPL && e0 + i < E; ++i) s_c[e0 + i] = (near >> i) & 1u ? f(e0 + i) : -INFINITY;
    __syncwarp();
    int mine = -1;
#pragma unroll 1
    for (int k = 0; k < K; ++k) {
        double v = -INFINITY;
        int e = E;
#pragma unroll 1
        for (int i = 0; i < EPL && e0 + i < E; ++i)
            if (s_c[e0 + i] > v) {
                v = s_c[e0 + i];
                e = e0 + i;
            }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const double v2 = __shfl_xor_sync(kAll, v, o);
            const int e2 = __shfl_xor_sync(kAll, e, o);
            if (v2 > v || (v2 == v && e2 < e)) {
                v = v2;
                e = e2;
            }
        }
        if (e == E) break;      // the same in every lane
        if (lane == k) mine = e;
        __syncwarp();
        if (lane == 0) s_c[e] = -INFINITY;
        __syncwarp();
    }
    return mine;
}

// The K largest of exact values in K rounds.  Slot k's expert in lane k, or -1.
template <int EPL>
__device__ __forceinline__ int rounds_choice(float (&c)[EPL], int K) {
    const int lane = threadIdx.x & 31;
    int mine = -1;
#pragma unroll 1
    for (int k = 0; k < K; ++k) {
        float best = c[0];
        int at = 0;
#pragma unroll
        for (int i = 1; i < EPL; ++i)
            if (c[i] > best) {
                best = c[i];
                at = i;
            }
        const float m = warp_largest(best);
        if (!(m > -INFINITY)) break;
        const int src = __ffs(__ballot_sync(kAll, best == m)) - 1;
        const int e = src * EPL + __shfl_sync(kAll, at, src);
        if (lane == k) mine = e;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (lane == src && i == at) c[i] = -INFINITY;
    }
    return mine;
}

// ---- forward ------------------------------------------------------------------------

// Tokens of a block of the forward kernel.  (16384 tokens of 1024 experts with a bias
// 48 us with four and 53 with eight, of 512 with groups 25.9 and 23.9.)
template <int EPL>
constexpr int kForwardWarps = EPL == 32 ? 4 : kRouteWarps;

template <typename T_, int EPL>
__global__ void __launch_bounds__(32 * kForwardWarps<EPL>, EPL == 16 ? 3 : 4) route_topk_kernel(const RouteArgs a) {
    __shared__ uint2 s_near[kForwardWarps<EPL>][33];   // key and expert; then the keys by rank
    extern __shared__ double s_exact[];         // [warps][E], with a bias or sums of two
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.E, K = a.K, e0 = lane * EPL;
    const int t = blockIdx.x * (blockDim.x >> 5) + warp;
    if (t >= a.T) return;
    const T_* row = static_cast<const T_*>(a.logits) + (int64_t)t * a.stride;
    double* s_c = s_exact + (size_t)warp * E;
    const bool sigmoid = a.rule.score == MOE_SCORE_SIGMOID, grouped = a.rule.topk_groups < a.rule.groups;
    const bool pair = grouped && a.rule.group_score == MOE_GROUP_TOP2, biased = a.bias != nullptr;
    float l[EPL], b[EPL];
    load_row<T_, EPL>(row, E, a.wide, l);
    if (biased) load_row<float, EPL>(a.bias, E, a.wide_bias, b);
    if (!(sigmoid && biased)) as_logits<EPL>(l);        // (sigmoid takes infinity as it is, and NaN is compared away)
    Softmax soft{0.0f, 0.0f};
    if (!sigmoid && (biased || pair || !a.rule.renormalize)) soft = softmax_of<EPL>(l);
    float c[EPL];       // -infinity: cannot be chosen
#pragma unroll
    for (int i = 0; i < EPL; ++i) c[i] = l[i];
    if (biased) {
        scores<EPL>(sigmoid, soft, c);
#pragma unroll
        for (int i = 0; i < EPL; ++i) c[i] = l[i] > -INFINITY && b[i] > -INFINITY ? c[i] + b[i] : -INFINITY;
    }
    // a bound of the error of c: its score's, and c's own rounding
    const float most = sigmoid ? kSigmoidErr : kSoftmaxErr<EPL> * soft.inv;
    auto err_of = [&](float v) { return most + kTiny + 2.0f * kUnit * fabsf(v); };

    if (grouped) {
        const int groups = a.rule.groups;
        const bool whole = a.span >= 0;         // a group is 2^span whole lanes
        const bool plain = pair && !biased;     // sums of the scores
        float x = -INFINITY, y = -INFINITY, border = -INFINITY;     // lane g: the two largest of group g
        float v[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) v[i] = c[i];
        if (plain) {
            scores<EPL>(sigmoid, soft, v);
#pragma unroll
            for (int i = 0; i < EPL; ++i) v[i] = l[i] > -INFINITY ? v[i] : -INFINITY;
        }
        if (whole) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) into_top2(x, y, v[i]);
            for (int o = 1; o < 1 << a.span; o <<= 1) {
                const float x2 = __shfl_xor_sync(kAll, x, o), y2 = __shfl_xor_sync(kAll, y, o);
                join_top2(x, y, x2, y2);
            }
            border = pair ? y : x;              // of the lane's own group
            const int src = lane << a.span & 31;
            x = __shfl_sync(kAll, x, src);
            y = __shfl_sync(kAll, y, src);
        } else {
            float* s_v = reinterpret_cast<float*>(s_c);
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (e0 + i < E) s_v[e0 + i] = v[i];
            __syncwarp();
            if (lane < groups)
                for (int i = 0; i < a.size; ++i) into_top2(x, y, s_v[lane * a.size + i]);
            __syncwarp();
        }
        const float score = lane >= groups ? -INFINITY : pair && y > -INFINITY ? x + y : x;
        // the worst that is taken and the best that is not
        const int take = a.rule.topk_groups;
        const float ranked = sorted_lanes(score, groups);
        const float low = __shfl_sync(kAll, ranked, take - 1), high = __shfl_sync(kAll, ranked, take);
        uint32_t taken = __ballot_sync(kAll, score >= low);
        if (high > -INFINITY) {
            const float size = biased || pair ? warp_largest(lane < groups && score > -INFINITY ? fabsf(score) + fabsf(x) : 0.0f) : 0.0f;
            const float err = biased || pair ? 2.0f * err_of(size) : 0.0f;      // of each score
            if (biased || pair ? !(low - high > 2.0f * err) : low == high) {
                border = fmaxf(border - 2.1f * err_of(border), -FLT_MAX);      // (none: all that can be chosen)
                uint32_t can = 0;
#pragma unroll
                for (int i = 0; i < EPL; ++i) can |= v[i] >= border ? 1u << i : 0u;
                taken = biased || pair ? exact_groups<T_, EPL>(row, a.bias, sigmoid, E, soft.max, groups, take, pair, can, s_c, s_near[warp])
                                       : best_groups(lane < groups ? score : NAN, groups, take);
            }
        }
        const uint32_t open = whole ? (taken >> (lane >> a.span)) & 1u ? kAll : 0u : lane_mask<EPL>(taken, a.size);
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (!((open >> i) & 1u)) c[i] = -INFINITY;
    }

    // the border: the K-th largest of the lanes' largest, lower by the bounds
    float mine_best = c[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) mine_best = fmaxf(mine_best, c[i]);
    float border = __shfl_sync(kAll, sorted_lanes(mine_best, 32), K - 1);
    if (biased) border -= 2.1f * err_of(border);
    border = fmaxf(border, -FLT_MAX);           // (-infinity, or less and so NaN: all that can be chosen)
    // the experts from there on, in their order
    uint32_t near = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) near |= c[i] >= border ? 1u << i : 0u;
    int n, pos = before_lane(__popc(near), &n);
    int mine = -1, slot = lane;     // this lane's expert and its place
    if (n <= 32) {
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if ((near >> i) & 1u) s_near[warp][pos++] = make_uint2(__float_as_uint(c[i]), (uint32_t)(e0 + i));
        __syncwarp();
        uint2 own = lane < n ? s_near[warp][lane] : make_uint2(0u, 0u);
        const float my_c = __uint_as_float(own.x);
        if (lane < n) {
            mine = (int)own.y;
            own.x = order_of(my_c + 0.0f);      // zeros alike
        }
        slot = 0;
        for (int j0 = 0; j0 < n; j0 += 4)
#pragma unroll
            for (int j = j0; j < j0 + 4; ++j) slot += __shfl_sync(kAll, own.x, j) > own.x;      // (0 in the lanes past n - 1)
        if (__reduce_or_sync(kAll, lane < n ? 1u << slot : 0u) != (n ? kAll >> (32 - n) : 0u))     // equal ones in their order
            for (int j = 0; j < n; ++j) slot += __shfl_sync(kAll, own.x, j) == own.x && j < lane;
        if (biased) {
            // is the order of the chosen beyond doubt, and the last of them ahead of every one that is not?
            __syncwarp();
            if (lane < n) s_near[warp][slot] = make_uint2(__float_as_uint(my_c), own.y);
            __syncwarp();
            bool doubt = false;
            if (lane < n && lane != K - 1 && (lane >= K || lane + 1 < n)) {
                const uint2 u = s_near[warp][min(lane, K - 1)], v = s_near[warp][lane < K ? lane + 1 : lane];
                const float cu = __uint_as_float(u.x), cv = __uint_as_float(v.x);
                // equal inputs are equal exactly, in the lower expert's favour
                doubt = !(cu - cv > err_of(cu) + err_of(cv)) &&
                        !(load_logit(row + u.y) == load_logit(row + v.y) && as_logit(a.bias[u.y]) == as_logit(a.bias[v.y]));
            }
            if (__any_sync(kAll, doubt)) slot = exact_rank<T_, EPL>(row, a.bias, sigmoid, E, soft.max, mine, n);
        }
        if (slot >= K) mine = -1;
    } else if (biased) {
        mine = exact_choice<T_, EPL>(row, a.bias, sigmoid, E, soft.max, K, near, s_c);
    } else {
        mine = rounds_choice<EPL>(c, K);
    }

    // weights: of renormalized sigmoids the common factor e^-min(max, 0) is left
    // out, so that they do not underflow together
    const float my_l = mine >= 0 ? load_logit(row + mine) : -INFINITY;
    float s;
    if (a.rule.renormalize) {
        const float m = fmaxf(warp_largest(my_l), -FLT_MAX);
        s = sigmoid ? __fdividef(exp_fast(fminf(my_l, 0.0f) - fminf(m, 0.0f)), 1.0f + exp_fast(-fabsf(my_l))) : exp_fast(my_l - m);
        s = __fdividef(s, warp_sum(mine >= 0 ? s : 0.0f));
    } else if (sigmoid) {
        s = 1.0f / (1.0f + expf(-my_l));
    } else {
        s = expf(my_l - soft.max) * soft.inv;
    }
    int* ids = a.ids + (int64_t)t * K;
    float* w = a.w + (int64_t)t * K;
    if (mine >= 0) {
        ids[slot] = mine;
        w[slot] = s * a.rule.scale;
    }
    const int chosen = __popc(__ballot_sync(kAll, mine >= 0));
    if (lane >= chosen && lane < K) {
        ids[lane] = -1;
        w[lane] = 0.0f;
    }
    pdl_launch_dependents();
}

// ---- backward -----------------------------------------------------------------------

struct RouteGradArgs {
    int T, E, K;
    const void* logits;
    int64_t stride;
    const int* ids;
    const float* dw;
    moe_route_rule rule;
    void* out;
    int64_t out_stride;
    bool wide;
};

template <typename T_>
__device__ __forceinline__ void put(T_* p, float v) { *p = (T_)v; }

// Slot k:
//   softmax, renormalized   w (u - sum w u)                u = scale dw
//   softmax                 p_e (u_e - sum_k p_k u_k)      over all experts
//   sigmoid, renormalized   w (1 - s) (u - sum w u)
//   sigmoid                 u s (1 - s)
// The row is written as if no expert were chosen, and then the chosen ones, by
// the same warp.

// A softmax that is not renormalized: a warp a token, slot k in lane k.
template <typename T_, int EPL>
__global__ void __launch_bounds__(32 * kRouteWarps) route_softmax_backward_kernel(const RouteGradArgs a) {
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.E, K = a.K, e0 = lane * EPL;
    const int t = blockIdx.x * (blockDim.x >> 5) + warp;
    if (t >= a.T) return;
    const T_* row = static_cast<const T_*>(a.logits) + (int64_t)t * a.stride;
    T_* out = static_cast<T_*>(a.out) + (int64_t)t * a.out_stride;
    int e = lane < K ? a.ids[(int64_t)t * K + lane] : -1;
    const float dw = lane < K ? a.dw[(int64_t)t * K + lane] : 0.0f;
    if (e < 0 || e >= E) e = -1;
    const float u = e >= 0 ? dw * a.rule.scale : 0.0f;
    const float my_l = e >= 0 ? load_logit(row + e) : -INFINITY;
    float l[EPL];
    load_row<T_, EPL>(row, E, a.wide, l);
    as_logits<EPL>(l);
    const Softmax soft = softmax_of<EPL>(l);
    const float base = -warp_sum(e >= 0 ? soft.of(my_l) * u : 0.0f);
    // slots of one expert add up
    float sum = 0.0f;
    for (int k = 0; k < K; ++k) {
        const int e2 = __shfl_sync(kAll, e, k);
        const float u2 = __shfl_sync(kAll, u, k);
        if (e2 == e) sum += u2;
    }
    __syncwarp();       // dlogits may be the logits: every lane has read them
    constexpr int kMost = 16 / sizeof(T_), VEC = EPL < kMost ? EPL : kMost;
    if (VEC > 1 && a.wide) {
#pragma unroll
        for (int i = 0; i < EPL; i += VEC) {
            float v[VEC];
#pragma unroll
            for (int k = 0; k < VEC; ++k) v[k] = soft.of(l[i + k]) * base;
            if (e0 + i < E)
                *reinterpret_cast<typename RowVec<T_, VEC>::Raw*>(out + e0 + i) = RowVec<T_, VEC>::pack(v);
        }
    } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (e0 + i < E) put(out + e0 + i, soft.of(l[i]) * base);
    }
    __syncwarp();
    if (e >= 0) put(out + e, soft.of(my_l) * (sum + base));
    pdl_launch_dependents();
}

// The others need the chosen logits alone: LANES lanes a token, so that a warp's loads
// are of all its lanes and a token takes a share of its instructions (16384 tokens of
// 256 experts, top-8: 4.8 us against 7.0 with a warp each; of 1024: 13.0 and 25.3).
template <typename T_, int LANES>
__global__ void __launch_bounds__(32 * kRouteWarps) route_slots_backward_kernel(const RouteGradArgs a) {
    pdl_wait();
    constexpr int N = 32 / LANES, VEC = 16 / sizeof(T_);
    const int lane = threadIdx.x & 31, j = lane % LANES, E = a.E, K = a.K;
    const int first = (blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) * N, t = first + lane / LANES;
    if (first >= a.T) return;
    const bool has = j < K && t < a.T;
    const int64_t slot = (int64_t)t * K + j;
    int e = has ? a.ids[slot] : -1;
    const float dw = has ? a.dw[slot] : 0.0f;
    if (e < 0 || e >= E) e = -1;
    const float u = e >= 0 ? dw * a.rule.scale : 0.0f;
    const float l = e >= 0 ? load_logit(static_cast<const T_*>(a.logits) + t * a.stride + e) : -INFINITY;
    auto sum_of = [](float v) {
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
        return v;
    };
    const bool sigmoid = a.rule.score == MOE_SCORE_SIGMOID;
    float d;
    if (a.rule.renormalize) {
        float m = l;
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
        if (!(m > -INFINITY)) m = 0.0f;
        float w = sigmoid ? expf(fminf(l, 0.0f) - fminf(m, 0.0f)) / (1.0f + expf(-fabsf(l))) : expf(l - m);
        const float all = sum_of(e >= 0 ? w : 0.0f);
        w = e >= 0 ? w / all : 0.0f;
        d = w * (u - sum_of(w * u));
        if (sigmoid) d *= 1.0f / (1.0f + expf(l));
    } else {
        const float x = expf(-fabsf(l));
        d = u * (x / ((1.0f + x) * (1.0f + x)));
    }
    float sum = 0.0f;       // slots of one expert add up
#pragma unroll
    for (int k = 0; k < LANES; ++k) {
        const int e2 = __shfl_sync(kAll, e, k, LANES);
        const float d2 = __shfl_sync(kAll, d, k, LANES);
        if (e2 == e) sum += d2;
    }
    __syncwarp();           // dlogits may be the logits: every lane has read them
    T_* out = static_cast<T_*>(a.out) + first * a.out_stride;
#pragma unroll
    for (int r = 0; r < N; ++r, out += a.out_stride) {
        if (first + r >= a.T) break;
        if (a.wide) {
            for (int c = lane; c < E / VEC; c += 32) reinterpret_cast<uint4*>(out)[c] = make_uint4(0, 0, 0, 0);
        } else {
            for (int c = lane; c < E; c += 32) put(out + c, 0.0f);
        }
    }
    __syncwarp();
    if (e >= 0) put(static_cast<T_*>(a.out) + t * a.out_stride + e, sum);
    pdl_launch_dependents();
}

// Tokens of a block: as many blocks as SMs first.
int route_warps(int T, int most = kRouteWarps) {
    int w = most;
    while (w > 1 && T <= 152 * (w / 2)) w /= 2;
    return w;
}

// Calls f<EPL>() for the smallest EPL that holds E experts in a warp.
#define MOE_ROUTE_EPL(E, f, T_, ...)                  \
    do {                                              \
        if ((E) <= 32) return f<T_, 1>(__VA_ARGS__);  \
        if ((E) <= 64) return f<T_, 2>(__VA_ARGS__);  \
        if ((E) <= 128) return f<T_, 4>(__VA_ARGS__); \
        if ((E) <= 256) return f<T_, 8>(__VA_ARGS__); \
        if ((E) <= 512) return f<T_, 16>(__VA_ARGS__);\
        return f<T_, 32>(__VA_ARGS__);                \
    } while (0)

template <typename T_, int EPL>
cudaError_t forward_epl(const LaunchCtx& c, RouteArgs a) {
    constexpr int kMost = 16 / sizeof(T_), VEC = EPL < kMost ? EPL : kMost;
    a.wide = a.E % VEC == 0 && row_at(a.logits, a.stride, sizeof(T_)) % (VEC * sizeof(T_)) == 0;
    a.size = a.E / a.rule.groups;
    a.span = -1;
    for (int n = 0; n < 6; ++n)
        if (a.size == EPL << n) a.span = n;
    const int warps = route_warps(a.T, kForwardWarps<EPL>);
    const bool scratch = a.bias || a.rule.topk_groups < a.rule.groups;
    constexpr int kBias = EPL < 4 ? EPL : 4;
    a.wide_bias = a.E % kBias == 0 && row_at(a.bias) % (kBias * 4) == 0;
    const size_t smem = scratch ? (size_t)warps * a.E * 8 : 0;     // 32 KB at most, which needs no leave
    static_assert(kForwardWarps<EPL> * EPL * 32 * 8 <= 32 * 1024, "beside s_near within 48 KB");
    return c.launch(route_topk_kernel<T_, EPL>, dim3((unsigned)((a.T + warps - 1) / warps)), dim3(32 * warps), smem, a);
}
template <typename T_>
cudaError_t forward_of(const LaunchCtx& c, const RouteArgs& a) {
    MOE_ROUTE_EPL(a.E, forward_epl, T_, c, a);
}

template <typename T_, int EPL>
cudaError_t backward_epl(const LaunchCtx& c, RouteGradArgs a) {
    constexpr int kMost = 16 / sizeof(T_), VEC = EPL < kMost ? EPL : kMost;
    a.wide = a.E % VEC == 0 &&
             (row_at(a.logits, a.stride, sizeof(T_)) | row_at(a.out, a.out_stride, sizeof(T_))) % (VEC * sizeof(T_)) == 0;
    const int warps = route_warps(a.T);
    return c.launch(route_softmax_backward_kernel<T_, EPL>, dim3((unsigned)((a.T + warps - 1) / warps)), dim3(32 * warps),
                    0, a);
}
template <typename T_, int LANES>
cudaError_t backward_slots(const LaunchCtx& c, RouteGradArgs a) {
    constexpr int VEC = 16 / sizeof(T_), N = 32 / LANES;
    a.wide = a.E % VEC == 0 && row_at(a.out, a.out_stride, sizeof(T_)) % 16 == 0;
    const int warps = route_warps((a.T + N - 1) / N), tokens = warps * N;
    return c.launch(route_slots_backward_kernel<T_, LANES>, dim3((unsigned)((a.T + tokens - 1) / tokens)), dim3(32 * warps), 0, a);
}
template <typename T_>
cudaError_t backward_of(const LaunchCtx& c, const RouteGradArgs& a) {
    if (a.rule.score == MOE_SCORE_SIGMOID || a.rule.renormalize)
        return a.K <= 8 ? backward_slots<T_, 8>(c, a) : a.K <= 16 ? backward_slots<T_, 16>(c, a) : backward_slots<T_, 32>(c, a);
    MOE_ROUTE_EPL(a.E, backward_epl, T_, c, a);
}

}  // namespace

cudaError_t launch_route_topk(const LaunchCtx& c, int T, int E, int K, int elem, const void* logits, int64_t stride,
                              const float* bias, const moe_route_rule& rule, int* ids, float* w) {
    const RouteArgs a{T, E, K, logits, stride, bias, rule, ids, w, false, false, 0, 0};
    return elem == 2 ? forward_of<__nv_bfloat16>(c, a) : forward_of<float>(c, a);
}

cudaError_t launch_route_topk_backward(const LaunchCtx& c, int T, int E, int K, int elem, const void* logits,
                                       int64_t stride, const int* ids, const float* dw, const moe_route_rule& rule,
                                       void* out, int64_t out_stride) {
    const RouteGradArgs a{T, E, K, logits, stride, ids, dw, rule, out, out_stride, false};
    return elem == 2 ? backward_of<__nv_bfloat16>(c, a) : backward_of<float>(c, a);
}

}  // namespace moe
