// Routing to experts and its gradient: rows of router logits -> the k experts of a row and
// their weights (gemm355_softmax.h states the formulas).
//
// The row softmax is the one of "Kernel optimisation guide" (section on softmax
// optimisation); the choice adds a bias, keeps the best groups and takes the k best, ties
// to the lowest index.
//
// One wave takes a row, Q = experts / 64 of its experts per lane.  A row is a few hundred
// bytes, so the time goes into instructions, not memory.  The ids are whole numbers and have
// to be those of exact scores, but only rows with two candidates closer than binary32 can
// tell apart need better: a row is first decided on 32-bit keys (the logits themselves where
// no bias is added, so exactly; else binary32 scores plus bias), and where two neighbours of
// the resulting order, or two groups, are closer than the bound of the scores' error, the
// row is decided again on binary64 scores.  Each round takes the largest key (a maximum over
// registers, four register exchanges within 16 lanes, a scalar maximum of four lanes) and
// the lowest expert that holds it (a ballot per register).
//
// Bound by the vector unit: about 660 instructions a row of 256 experts in groups with a bias
// and 8 places (binary64 throughout: over 2000).  16384 such rows take 36 us (29 without the
// counts, whose per-workgroup sums are added to memory by atomics; whole numbers, so in any
// order), 15 us without groups and bias; reading the logits alone would take 4.
#include "../../include/gemm355_softmax.h"
#include "common.hpp"
#include "launch.hpp"
#include "wave_reduce.hpp"

namespace g355 {

namespace {

constexpr int kMaxExperts = 1024, kMaxGroups = 64, kMaxK = 64, kMaxRouteRows = 1 << 30;
constexpr unsigned kRouteFlags = GEMM355_ROUTE_SIGMOID | GEMM355_ROUTE_RENORM;
constexpr double kLow = -__builtin_huge_val();

struct RouteArgs {
    int rows, experts, k, groups, top_groups, group_top;
    const void *X;
    int ldx;
    const float *bias;
    float scale;
    int32_t *ids;
    float *weights;
    int32_t *counts;
};

// The arguments (the kernel's first) as they lie in memory, behind a pointer the compiler
// cannot see through: what is rarely needed is loaded where it is used instead of being held
// in scalar registers from the kernel's start.
#ifdef __HIP_DEVICE_COMPILE__
typedef const __attribute__((address_space(4))) RouteArgs *ArgsPtr;
#else
typedef const RouteArgs *ArgsPtr;  // the host pass only parses the kernels
#endif
__device__ __forceinline__ ArgsPtr args_in_memory() {
    ArgsPtr p = (ArgsPtr)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return p;
}

template <typename T>
__device__ __forceinline__ float load_elem(const void *p, size_t i) {
    return to_float(((const T *)p)[i]);
}
template <typename T>
__device__ __forceinline__ void store_elem(void *p, size_t i, float v) {
    if constexpr (std::is_same<T, float>::value) ((float *)p)[i] = v;
    else ((uint16_t *)p)[i] = to_bits(v, T{});
}

// The same value in every lane: the other lane's copy of a binary64 value at xor distance d.
__device__ __forceinline__ double shfl_xor64(double v, int d) { return __shfl_xor(v, d, 64); }

template <class X>
__device__ __forceinline__ double exchange64(double v) {
    const unsigned long long u = __builtin_bit_cast(unsigned long long, v);
    const float lo = X::get(__builtin_bit_cast(float, (uint32_t)u)), hi = X::get(__builtin_bit_cast(float, (uint32_t)(u >> 32)));
    return __builtin_bit_cast(double, (unsigned long long)__builtin_bit_cast(uint32_t, lo) |
                                          (unsigned long long)__builtin_bit_cast(uint32_t, hi) << 32);
}

// The sum over the first n lanes of an aligned run (n a power of two), in every one of them.
__device__ __forceinline__ double lanes_sum64(double v, int n) {
    if (n > 1) v += exchange64<DppXchg<kDppQuadXor1>>(v);
    if (n > 2) v += exchange64<DppXchg<kDppQuadXor2>>(v);
    if (n > 4) v += exchange64<DppXchg<kDppRowHalfMirror>>(v);
    if (n > 8) v += exchange64<DppXchg<kDppRowMirror>>(v);
    if (n > 16) v += exchange64<SwapHalves16>(v);
    if (n > 32) v += shfl_xor64(v, 32);
    return v;
}
__device__ __forceinline__ double wave_sum64(double v) { return lanes_sum64(v, 64); }

__global__ void zero_counts_kernel(int n, int32_t *counts) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n) counts[i] = 0;
}

// Binary32 in an order-preserving 32-bit form; 0 is below every value's.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t u = __builtin_bit_cast(uint32_t, x + 0.0f);  // -0 as +0
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
    return __builtin_bit_cast(float, k ^ ((uint32_t)((int32_t)~k >> 31) | 0x80000000u));
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}

// The wave's largest v, as a scalar.
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
    v = max(v, dpp_u32<kDppQuadXor1>(v));
    v = max(v, dpp_u32<kDppQuadXor2>(v));
    v = max(v, dpp_u32<kDppRowHalfMirror>(v));
    v = max(v, dpp_u32<kDppRowMirror>(v));
    const uint32_t a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16);
    const uint32_t c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
    uint32_t e, f;   // on the scalar unit (left to itself the compiler takes these to the vector one)
    asm("s_max_u32 %0, %1, %2" : "=s"(e) : "s"(a), "s"(b) : "scc");
    asm("s_max_u32 %0, %1, %2" : "=s"(f) : "s"(c), "s"(d) : "scc");
    asm("s_max_u32 %0, %0, %1" : "+s"(e) : "s"(f) : "scc");
    return e;
}

__device__ __forceinline__ float wave_max(float v) { return of_key(wave_max_u32(key_of(v))); }

// The two largest of a lane's values and of those the other lane of an exchange holds.
template <typename F>
__device__ __forceinline__ void merge_two(F &best, F &second, F bo, F so) {
    second = fmax(fmax(second, so), fmin(best, bo));
    best = fmax(best, bo);
}

template <class X>
__device__ __forceinline__ float exchange(float v) { return X::get(v); }
template <class X>
__device__ __forceinline__ double exchange(double v) { return exchange64<X>(v); }

// A group's score, in every one of its lanes: group g of `per` experts (choices in LDS) is
// scanned by the S = 64 / (groups rounded up to a power of two) lanes from g S on.
template <typename F>
__device__ __forceinline__ F group_score(const F *choice, int per, int S, int sub, int group_top) {
    constexpr F low = (F)kLow;
    F best = low, second = low;
#pragma unroll 1
    for (int i = sub; i < per; i += S) merge_two(best, second, choice[i], low);
    if (S > 1) merge_two(best, second, exchange<DppXchg<kDppQuadXor1>>(best), exchange<DppXchg<kDppQuadXor1>>(second));
    if (S > 2) merge_two(best, second, exchange<DppXchg<kDppQuadXor2>>(best), exchange<DppXchg<kDppQuadXor2>>(second));
    if (S > 4)
        merge_two(best, second, exchange<DppXchg<kDppRowHalfMirror>>(best), exchange<DppXchg<kDppRowHalfMirror>>(second));
    if (S > 8) merge_two(best, second, exchange<DppXchg<kDppRowMirror>>(best), exchange<DppXchg<kDppRowMirror>>(second));
    if (S > 16) merge_two(best, second, exchange<SwapHalves16>(best), exchange<SwapHalves16>(second));
    return group_top == 2 && second > low ? best + second : best;
}

__device__ __forceinline__ float lane_value(float v, int lane) { return read_lane(v, lane); }
__device__ __forceinline__ double lane_value(double v, int lane) {
    const unsigned long long u = __builtin_bit_cast(unsigned long long, v);
    return __builtin_bit_cast(double, (unsigned long long)(uint32_t)__builtin_amdgcn_readlane((int)u, lane) |
                                          (unsigned long long)(uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), lane)
                                              << 32);
}

// Which of the groups are among the `top` of the largest score, ties to the lowest group;
// near: a kept score lies within `margin` of one that is not.  A lane holds the score of
// group lane >> shift.
template <typename F>
__device__ __forceinline__ unsigned long long best_groups(F score, int groups, int top, int shift, F margin,
                                                          bool &near) {
    const int mine = (int)(threadIdx.x % 64) >> shift;
    int rank = 0;
    int close = 0;   // groups ahead of mine by no more than the margin
#pragma unroll 1
    for (int g = 0; g < groups; ++g) {
        const F o = lane_value(score, g << shift);
        const bool ahead = o > score || (o == score && g < mine);
        rank += ahead;
        close += ahead && o - score <= margin;
    }
    // not kept, and one that is (ranks below top) among those just ahead
    near = __any(mine < groups && rank >= top && rank - close < top);
    const unsigned long long in = __ballot(rank < top);   // 2^shift lanes a group
    unsigned long long kept = 0;
#pragma unroll 1
    for (int g = 0; g < groups; ++g) kept |= ((in >> (g << shift)) & 1) << g;
    return kept;
}

__device__ __forceinline__ void wave_lds_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// exp in binary64: x = n log 2 + r with |r| <= log 2 / 2 (log 2 in two parts, the first short
// enough for n times it to be exact), the Taylor sum of exp(r) to r^13 / 13! (the next term
// is below 2^-57), times 2^n.  The coefficients 1 / 13!, 1 / 12!, ... 1 lie in LDS: held in
// registers across a kernel's loop over rows they take 28 scalar ones.
constexpr int kTaylor = 14;
__device__ __forceinline__ void taylor_to_lds(double *coef) {
    if (threadIdx.x < kTaylor) {
        double f = 1.0;
        for (int i = kTaylor - 1 - (int)threadIdx.x; i > 1; --i) f *= (double)i;
        coef[threadIdx.x] = 1.0 / f;
    }
}
__device__ __forceinline__ double exp64(double x, const double *coef) {
    x = fmin(fmax(x, -1000.0), 1000.0);
    const double n = rint(x * 1.4426950408889634074);
    double r = fma(n, -0x1.62e42fefap-1, x);
    r = fma(n, -0x1.cf79abc9e3b3ap-40, r);
    double p = coef[0];
#pragma unroll
    for (int i = 1; i < kTaylor; ++i) p = fma(p, r, coef[i]);
    return ldexp(p, (int)n);
}

// The score of a logit in binary64, for softmax before the division by the row's sum.
template <bool SIGMOID>
__device__ __forceinline__ double score64(float x, float m, const double *coef) {
    const bool masked = !(x > -__builtin_huge_valf());
    const double d = masked ? 0.0 : (double)x - (SIGMOID ? 0.0 : (double)m);
    const double v = exp64(SIGMOID ? -d : d, coef);
    return masked ? 0.0 : SIGMOID ? 1.0 / (1.0 + v) : v;
}

// A row's logit, -infinity past its experts.
template <typename T>
__device__ __forceinline__ float logit_at(const void *X, size_t x0, int e, int experts) {
    const float x = load_elem<T>(X, x0 + min(e, experts - 1));
    return e < experts ? x : -__builtin_huge_valf();
}

// What the scores of a row are divided by: softmax's sum, or 1.
template <typename T, bool SIGMOID>
__device__ __forceinline__ double divisor64(const void *X, size_t x0, int experts, float m, const double *coef) {
    if constexpr (SIGMOID) return 1.0;
    double sum = 0.0;
#pragma unroll 1
    for (int e0 = 0; e0 < experts; e0 += 64)
        sum += score64<false>(logit_at<T>(X, x0, e0 + (int)(threadIdx.x % 64), experts), m, coef);
    return wave_sum64(sum);
}

// An expert's choice in binary64, -infinity for a masked or absent one and for a NaN bias.
template <typename T, bool SIGMOID>
__device__ __forceinline__ double choice64(const void *X, size_t x0, const float *bias, int e, int experts, float m,
                                           double sum, const double *coef) {
    const float x = logit_at<T>(X, x0, e, experts);
    const double c = score64<SIGMOID>(x, m, coef) / sum + (bias != nullptr ? (double)bias[min(e, experts - 1)] : 0.0);
    return x > -__builtin_huge_valf() && c > kLow ? c : kLow;
}

// The lanes a group's score is found by: 2^shift of them.
__device__ __forceinline__ int group_shift(int groups) {
    return groups > 1 ? __builtin_clz((unsigned)groups - 1) - 26 : 6;
}

// The row's kept groups by binary64 choices, which are left in the wave's row of LDS.
template <typename T, int Q, bool SIGMOID>
__device__ __forceinline__ unsigned long long exact_groups(size_t row, float m, double *choice, const double *coef) {
    const ArgsPtr a = args_in_memory();
    const int lane = threadIdx.x % 64, experts = a->experts, groups = a->groups;
    const void *X = a->X;
    const float *bias = a->bias;
    const size_t x0 = row * a->ldx;
    const double sum = divisor64<T, SIGMOID>(X, x0, experts, m, coef);
#pragma unroll 1
    for (int e0 = 0; e0 < Q * 64; e0 += 64)
        choice[e0 + lane] = choice64<T, SIGMOID>(X, x0, bias, e0 + lane, experts, m, sum, coef);
    if (a->top_groups >= groups) return ~0ull;
    wave_lds_sync();
    const int shift = group_shift(groups), mine = min(lane >> shift, groups - 1), per = experts / groups;
    const double score = group_score(choice + mine * per, per, 1 << shift, lane & ((1 << shift) - 1), a->group_top);
    wave_lds_sync();
    bool near;
    return best_groups(score, groups, a->top_groups, shift, 0.0, near);
}

// The ids of the row's first places put in the order of their binary64 choices.
template <typename T, bool SIGMOID>
__device__ __forceinline__ int exact_order(size_t row, float m, int id, const double *coef) {
    const ArgsPtr a = args_in_memory();
    const int lane = threadIdx.x % 64;
    const size_t x0 = row * a->ldx;
    const double sum = divisor64<T, SIGMOID>(a->X, x0, a->experts, m, coef);
    const bool in = id >= 0;   // of the first lanes
    const double c = in ? choice64<T, SIGMOID>(a->X, x0, a->bias, max(id, 0), a->experts, m, sum, coef) : kLow;
    const int n = __builtin_popcountll(__ballot(in));
    int rank = 0;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        const double o = lane_value(c, i);
        const int oid = __builtin_amdgcn_readlane(id, i);
        rank += o > c || (o == c && oid < id);
    }
    return __builtin_amdgcn_ds_permute(4 * (in ? rank : lane), id);
}

// The row's ids wholly by binary64 choices: id of place i in lane i.  choice: the wave's row
// of LDS, of which a lane touches its own experts only, but for the groups' scores.
template <typename T, int Q, bool SIGMOID>
__device__ __forceinline__ int exact_ids(size_t row, float m, double *choice, const double *coef) {
    const unsigned long long kept = exact_groups<T, Q, SIGMOID>(row, m, choice, coef);
    const ArgsPtr a = args_in_memory();
    const int lane = threadIdx.x % 64, experts = a->experts, per = experts / a->groups, k = a->k;
    const bool by_logit = a->bias == nullptr;
#pragma unroll 1
    for (int e0 = 0; e0 < experts; e0 += 64) {
        const int e = e0 + lane;
        double c = choice[e];
        // without a bias the order within the kept groups is the logits'
        if (by_logit && c > kLow) c = (double)logit_at<T>(a->X, row * a->ldx, e, experts);
        choice[e] = (kept >> ((e / per) & 63)) & 1 ? c : kLow;
    }
    int id = -1;
#pragma unroll 1
    for (int i = 0; i < k; ++i) {
        double v = kLow;
        int at = 0x7fffffff;
#pragma unroll 1
        for (int e0 = 0; e0 < experts; e0 += 64) {
            const double c = choice[e0 + lane];
            at = c > v ? e0 + lane : at;
            v = fmax(c, v);
        }
#pragma unroll 1
        for (int d = 1; d < 64; d *= 2) {
            const double vo = shfl_xor64(v, d);
            const int ao = __shfl_xor(at, d, 64);
            const bool theirs = vo > v || (vo == v && ao < at);
            v = theirs ? vo : v;
            at = theirs ? ao : at;
        }
        at = __builtin_amdgcn_readfirstlane(at);
        if (at == 0x7fffffff) break;   // no expert left
        id = lane == i ? at : id;
        if (at % 64 == lane) choice[at] = kLow;
    }
    return id;
}

// Rows of more than 512 experts are always decided on binary64 scores: 16 keys and their lane
// masks per lane do not fit the scalar registers.
constexpr bool has_keys(int Q) { return Q <= 8; }

constexpr int kRouteWaves = 16;
constexpr int kRouteGrid = 512;  // workgroups; each takes every kRouteGrid-th group of rows

// BIAS: choices add a.bias.  GROUPS: a.top_groups < a.groups.  SINGLE: one workgroup takes
// every row, and writes the counts; else they are added to.
template <typename T, int Q, bool SIGMOID, bool BIAS, bool GROUPS>
__global__ __launch_bounds__(64 * kRouteWaves) void route_kernel(RouteArgs a, bool renorm, bool single) {
    constexpr bool kExact = BIAS || GROUPS || !has_keys(Q);
    __shared__ double choice_lds[kExact ? kRouteWaves : 1][kExact ? Q * 64 : 1];
    __shared__ int hist[Q * 64];
    __shared__ double coef[kTaylor];
    const int wave = threadIdx.x / 64, lane0 = threadIdx.x % 64;
    constexpr float kNegInf = -__builtin_huge_valf();
    const bool count = a.counts != nullptr;
    taylor_to_lds(coef);
    if (count)
        for (int e = threadIdx.x; e < a.experts; e += 64 * kRouteWaves) hist[e] = 0;
    __syncthreads();
    float b[Q], top_b = 0.0f;
    if constexpr (BIAS && has_keys(Q)) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int e = q * 64 + lane0;
            b[q] = e < a.experts ? a.bias[e] : 0.0f;
            // a masked expert's bias bounds nothing (NaN: the maximum ignores it)
            top_b = fmaxf(top_b, b[q] == kNegInf ? 0.0f : fabsf(b[q]));
        }
        top_b = wave_max(top_b);
    }
    int per = 1, group_of[Q];   // of an absent expert, whose key is 0: any group
    if constexpr (GROUPS && has_keys(Q)) {
        per = a.experts / a.groups;
#pragma unroll
        for (int q = 0; q < Q; ++q) group_of[q] = ((q * 64 + lane0) / per) & 63;
    }
    for (int row = blockIdx.x * kRouteWaves + wave; row < a.rows; row += gridDim.x * kRouteWaves) {
        // the lane as each row's own value, or the masks of absent experts, two scalar registers
        // each, are kept across rows
        int lane = lane0;
        asm volatile("" : "+v"(lane));
        float x[Q], m = kNegInf;
        bool bad = false;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            x[q] = logit_at<T>(a.X, (size_t)row * a.ldx, q * 64 + lane, a.experts);
            // NaN, and for softmax +infinity
            bad |= __builtin_amdgcn_classf(x[q], SIGMOID ? 0x003 : 0x203);
            m = fmaxf(m, x[q]);
        }
        bad = __any(bad);
        if constexpr (!SIGMOID) m = wave_max(m);
        int id = -1;
        if (!bad && (SIGMOID || m > kNegInf)) {
            bool near = true;
            if constexpr (has_keys(Q)) {
                // binary32 scores s, each within 2^-24 (1 + (E / 64 + 32) s) of the exact one: a
                // score's relative error is at most 2^-24 (2 |x| + 8), for softmax 2^-24 (2 |x - m|
                // + E / 64 + 32) with the sum's, and 2 d exp(-d) < 1
                uint32_t key[Q];
                float s[Q];
                float margin = 0.0f;
                if constexpr (BIAS || GROUPS) {
                    float largest = 1.0f;
                    if constexpr (SIGMOID) {
#pragma unroll
                        for (int q = 0; q < Q; ++q) s[q] = __builtin_amdgcn_rcpf(1.0f + __expf(-x[q]));
                    } else {
                        float sum = 0.0f;
#pragma unroll
                        for (int q = 0; q < Q; ++q) {
                            s[q] = __expf(x[q] - m);
                            sum += s[q];
                        }
                        largest = 1.0f / wave_allreduce_sum(sum);
#pragma unroll
                        for (int q = 0; q < Q; ++q) s[q] *= largest;
                    }
                    // two choices' errors, with the sum's with the bias
                    margin = 2.0f * 0x1p-24f * (1.0f + (Q + 34.0f) * largest + 2.0f * top_b);
                }
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    if constexpr (BIAS) s[q] += b[q];
                    const float c = BIAS ? s[q] : x[q];
                    const bool out = !(x[q] > kNegInf) || (BIAS && !(c > kNegInf));
                    key[q] = out ? 0u : key_of(c);
                    if constexpr (GROUPS) s[q] = out ? kNegInf : s[q];
                }
                near = false;
                if constexpr (GROUPS) {
                    const ArgsPtr am = args_in_memory();
                    const int groups = am->groups;
                    float *choice = (float *)choice_lds[wave];
#pragma unroll
                    for (int q = 0; q < Q; ++q) choice[q * 64 + lane] = s[q];
                    wave_lds_sync();
                    const int shift = group_shift(groups);
                    const int mine = min(lane >> shift, groups - 1);
                    const float score = group_score((const float *)choice + mine * per, per, 1 << shift,
                                                    lane & ((1 << shift) - 1), am->group_top);
                    wave_lds_sync();
                    bool close;
                    unsigned long long kept = best_groups(score, groups, am->top_groups, shift, 2.5f * margin, close);
                    if (close) kept = exact_groups<T, Q, SIGMOID>(row, m, choice_lds[wave], coef);
#pragma unroll
                    for (int q = 0; q < Q; ++q) key[q] = (kept >> group_of[q]) & 1 ? key[q] : 0u;
                }
                // The places, the i-th key in lane i as its id.  With a bias, one more to see
                // how far the last is from what stays out: neighbours closer than the margin
                // are put in order in binary64, and if the one after the last is as close to
                // the next, the row is left to binary64 choices altogether.
                uint32_t my_key = 0, v = 0;
                const auto next = [&]() {
                    v = key[0];
#pragma unroll
                    for (int q = 1; q < Q; ++q) v = max(v, key[q]);
                    v = wave_max_u32(v);
                };
                const int places = BIAS ? min(a.k + 1, 64) : a.k;
                for (int i = 0; i < places; ++i) {
                    next();
                    if (v == 0) break;
                    int at = 0;
#pragma unroll
                    for (int q = Q - 1; q >= 0; --q) {
                        const unsigned long long w = __ballot(key[q] == v);
                        at = w != 0 ? q * 64 + __builtin_ctzll(w) : at;
                    }
                    const bool here = lane == i;
                    id = here ? at : id;
                    if constexpr (BIAS) my_key = here ? v : my_key;
#pragma unroll
                    for (int q = 0; q < Q; ++q)
                        if (at >> 6 == q) key[q] = lane == (at & 63) ? 0u : key[q];   // one q: a scalar branch
                }
                if constexpr (BIAS) {
                    const uint32_t after = __shfl_down(my_key, 1, 64);
                    const bool close = lane < 63 && after != 0 && of_key(my_key) - of_key(after) <= margin;
                    const unsigned long long w = __ballot(close);   // lane i: places i and i + 1
                    if (w != 0) {
                        bool lost = places == 64;   // no lane for the one after the last
                        if (!lost && ((w >> (places - 2)) & 1)) {
                            const uint32_t last = __builtin_amdgcn_readlane(my_key, places - 1);
                            next();
                            lost = v != 0 && of_key(last) - of_key(v) <= margin;
                        }
                        near = lost;
                        if (!lost) id = exact_order<T, SIGMOID>(row, m, id, coef);
                    }
                    id = lane < a.k ? id : -1;
                }
            }
            if constexpr (kExact)
                if (near) id = exact_ids<T, Q, SIGMOID>(row, m, choice_lds[wave], coef);
        }
        // the weights, in binary64: place i in lane i
        const float xi = id >= 0 ? logit_at<T>(a.X, (size_t)row * a.ldx, id, a.experts) : kNegInf;
        double w = score64<SIGMOID>(xi, m, coef);
        if (renorm) {
            const double total = lanes_sum64(w, a.k <= 8 ? 8 : 64);
            w = total > 0.0 ? w / total : 0.0;
        } else if constexpr (!SIGMOID) {
            double sum = 0.0;
#pragma unroll 1
            for (int e0 = 0; e0 < a.experts; e0 += 64)
                sum += score64<false>(logit_at<T>(a.X, (size_t)row * a.ldx, e0 + lane, a.experts), m, coef);
            sum = wave_sum64(sum);
            w = sum > 0.0 ? w / sum : 0.0;
        }
        const ArgsPtr am = args_in_memory();
        w *= (double)am->scale;
        if (id < 0) w = bad ? __builtin_nan("") : 0.0;
        if (lane < a.k) {
            am->ids[(size_t)row * a.k + lane] = id;
            am->weights[(size_t)row * a.k + lane] = (float)w;
            if (count && id >= 0) atomicAdd(&hist[id], 1);
        }
    }
    if (!count) return;
    __syncthreads();
    int32_t *counts = args_in_memory()->counts;
    for (int e = threadIdx.x; e < a.experts; e += 64 * kRouteWaves) {
        const int n = hist[e];
        if (single) counts[e] = n;
        else if (n > 0) atomicAdd(counts + e, n);
    }
}

// Sums and maxima over aligned runs of n lanes, n a power of two; in every lane.
template <typename Op>
__device__ __forceinline__ float over_lanes(float v, int n, Op op) {
    if (n > 1) v = op(v, DppXchg<kDppQuadXor1>::get(v));
    if (n > 2) v = op(v, DppXchg<kDppQuadXor2>::get(v));
    if (n > 4) v = op(v, DppXchg<kDppRowHalfMirror>::get(v));
    if (n > 8) v = op(v, DppXchg<kDppRowMirror>::get(v));
    if (n > 16) v = op(v, SwapHalves16::get(v));
    if (n > 32) v = op(v, __shfl_xor(v, 32, 64));
    return v;
}
__device__ __forceinline__ float lanes_sum(float v, int n) {
    return over_lanes(v, n, [](float x, float y) { return x + y; });
}
__device__ __forceinline__ float lanes_max(float v, int n) {
    return over_lanes(v, n, [](float x, float y) { return fmaxf(x, y); });
}

// Adds each lane's v at its place (an index into the wave's row of LDS, -1 for none), places
// that several lanes of a row share in the order of their slots.  The row holds zeros.
__device__ __forceinline__ void scatter_add(float *row, int place, float v, int slot, int k) {
    const int lane = threadIdx.x % 64;
    int *tag = (int *)row;
    if (place >= 0) tag[place] = lane;
    wave_lds_sync();
    const bool shared = place >= 0 && tag[place] != lane;
    wave_lds_sync();
    if (!__any(shared)) {
        if (place >= 0) row[place] = v;
    } else {
        if (place >= 0) row[place] = 0.0f;
        wave_lds_sync();
        for (int j = 0; j < k; ++j) {
            if (slot == j && place >= 0) row[place] += v;
            wave_lds_sync();
        }
    }
    wave_lds_sync();
}

constexpr int kGradLds = 2048;  // floats of LDS per wave: the rows it takes at once

// The gradient where only chosen experts have one: sigmoid scores, and renormalised softmax
// (sum_f ds_f s_f is 0 there, and q_i s_i = w_i (dw_i - sum_j w_j dw_j) with w the softmax of
// the chosen logits alone).  Only k logits of a row are read.  A wave takes R rows, n lanes a
// row (n a power of two, at least k), a chosen expert per lane; the rows are put together in
// LDS and written whole: 6.7 us for 16384 binary32 rows of 256, 16.8 MB written at 2.5 TB/s
// (with a row per wave and every expert compared with every place the arithmetic took 18.8).
template <typename T, bool SIGMOID, bool VEC>
__global__ __launch_bounds__(256) void route_grad_chosen_kernel(int rows, int experts, int k, const void *X, int ldx,
                                                                const int32_t *ids, const float *dweights,
                                                                float scale, void *dX, int lddx, bool renorm,
                                                                int n, int R) {
    __shared__ __attribute__((aligned(16))) float lds[4][kGradLds];
    const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    const int row0 = (blockIdx.x * 4 + wave) * R;
    if (row0 >= rows) return;  // a whole wave; no barrier in this kernel
    float *out = lds[wave];
    const int live = min(R, rows - row0);
    for (int c = 4 * lane; c < live * experts; c += 256) *(floatx4 *)(out + c) = floatx4{0.f, 0.f, 0.f, 0.f};
    const int r = lane / n, slot = lane & (n - 1);
    int id = -1;
    float g = 0.0f;
    if (r < live && slot < k) {
        id = ids[(size_t)(row0 + r) * k + slot];
        g = scale * dweights[(size_t)(row0 + r) * k + slot];
    }
    const bool on = id >= 0 && id < experts;
    const float x = on ? load_elem<T>(X, (size_t)(row0 + r) * ldx + id) : -__builtin_huge_valf();
    g = on ? g : 0.0f;
    float v;
    if constexpr (SIGMOID) {
        const float s = on ? 1.0f / (1.0f + expf(-x)) : 0.0f;
        if (renorm) {
            const float sum = lanes_sum(s, n), inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            g = (g - lanes_sum(g * s, n) * inv) * inv;
        }
        v = g * s * (1.0f - s);
    } else {
        const float m = lanes_max(x, n);
        const float e = x > -__builtin_huge_valf() ? expf(x - m) : x != x ? x : 0.0f;
        const float sum = lanes_sum(e, n), w = sum == 0.0f ? 0.0f : e / sum;
        v = w * (g - lanes_sum(g * w, n));
    }
    wave_lds_sync();
    scatter_add(out, on ? r * experts + id : -1, v, slot, k);
    for (int i = 0; i < live; ++i) {
        const float *o = out + i * experts;
        const size_t at = (size_t)(row0 + i) * lddx;
        if constexpr (VEC) {
            for (int c = 4 * lane; c < experts; c += 256) {
                const floatx4 f = *(const floatx4 *)(o + c);
                if constexpr (std::is_same<T, float>::value) {
                    *(floatx4 *)((float *)dX + at + c) = f;
                } else {
                    const uint2 h = make_uint2((uint32_t)to_bits(f[0], T{}) | (uint32_t)to_bits(f[1], T{}) << 16,
                                               (uint32_t)to_bits(f[2], T{}) | (uint32_t)to_bits(f[3], T{}) << 16);
                    *(uint2 *)((uint16_t *)dX + at + c) = h;
                }
            }
        } else {
            for (int c = lane; c < experts; c += 64) store_elem<T>(dX, at + c, o[c]);
        }
    }
}

// The gradient of plain softmax weights, where every expert has one: one wave per row, Q
// experts per lane, the places' gradients gathered per expert through LDS.  4095 bf16 rows of
// 64 take 3.2 us, most of it the launch.
template <typename T, int Q>
__global__ __launch_bounds__(256) void route_grad_kernel(int rows, int experts, int k, const void *X, int ldx,
                                                         const int32_t *ids, const float *dweights, float scale,
                                                         void *dX, int lddx) {
    __shared__ __attribute__((aligned(16))) float lds[4][Q * 64];
    const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    const int row = blockIdx.x * 4 + wave;
    if (row >= rows) return;  // a whole wave; no barrier in this kernel
    float *sum_of = lds[wave];
    float s[Q], m = -__builtin_huge_valf();
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        s[q] = logit_at<T>(X, (size_t)row * ldx, q * 64 + lane, experts);
        sum_of[q * 64 + lane] = 0.0f;
        m = fmaxf(m, s[q]);
    }
    const int id = lane < k ? ids[(size_t)row * k + lane] : -1;
    const float g = lane < k ? scale * dweights[(size_t)row * k + lane] : 0.0f;
    wave_lds_sync();
    scatter_add(sum_of, id >= 0 && id < experts ? id : -1, g, lane, k);
    m = lanes_max(m, 64);
    const float shift = m == -__builtin_huge_valf() ? 0.0f : m;
    float sum = 0.0f;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        s[q] = expf(s[q] - shift);
        sum += s[q];
    }
    sum = wave_allreduce_sum(sum);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;   // a NaN row stays NaN
    float dot = 0.0f;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        s[q] *= inv;
        dot += sum_of[q * 64 + lane] * s[q];
    }
    dot = wave_allreduce_sum(dot);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int e = q * 64 + lane;
        if (e < experts) store_elem<T>(dX, (size_t)row * lddx + e, s[q] * (sum_of[e] - dot));
    }
}

// f(T{}) for the storage type.
template <typename F>
hipError_t by_type(int dtype, F f) {
    if (dtype == kF32) return f(0.0f);
    if (dtype == kF16) return f(f16_t{});
    return f(bf16_t{});
}

// f(T{}, integral_constant<int, Q>) for the storage type and the experts per lane.
template <typename F>
hipError_t by_type_and_width(int dtype, int experts, F f) {
    return by_type(dtype, [&](auto t) -> hipError_t {
        if (experts <= 64) return f(t, std::integral_constant<int, 1>{});
        if (experts <= 128) return f(t, std::integral_constant<int, 2>{});
        if (experts <= 256) return f(t, std::integral_constant<int, 4>{});
        if (experts <= 512) return f(t, std::integral_constant<int, 8>{});
        return f(t, std::integral_constant<int, 16>{});
    });
}

}  // namespace

}  // namespace g355

using namespace g355;

extern "C" {

gemm355_status gemm355_route(int dtype, unsigned flags, int rows, int experts, int k, int groups,
                             int top_groups, int group_top, const void *X, int ldx,
                             const float *bias, float scale, int32_t *ids, float *weights,
                             int32_t *counts, hipStream_t stream) {
    if (dtype < kF32 || dtype > kBF16 || (flags & ~kRouteFlags)) return GEMM355_ERR_INVALID_ARG;
    if (rows < 0 || rows > kMaxRouteRows || experts < 1 || experts > kMaxExperts || ldx < experts)
        return GEMM355_ERR_INVALID_ARG;
    if (groups < 1 || groups > kMaxGroups || experts % groups != 0 || top_groups < 1 ||
        top_groups > groups || group_top < 1 || group_top > 2)
        return GEMM355_ERR_INVALID_ARG;
    if (k < 1 || k > kMaxK || k > top_groups * (experts / groups)) return GEMM355_ERR_INVALID_ARG;
    if (rows > 0 && (X == nullptr || ids == nullptr || weights == nullptr)) return GEMM355_ERR_INVALID_ARG;
    const size_t es = dtype == kF32 ? 4 : 2;
    const Span out[3] = {{ids, ids ? (size_t)rows * k * 4 : 0},
                         {weights, weights ? (size_t)rows * k * 4 : 0},
                         {counts, counts ? (size_t)experts * 4 : 0}};
    const Span in[2] = {{X, matrix_bytes(rows, experts, ldx, es)},
                        {bias, bias ? (size_t)experts * 4 : 0}};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < 2; ++j)
            if (out[i].meets(in[j])) return GEMM355_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (out[i].meets(out[j])) return GEMM355_ERR_INVALID_ARG;
    }
    if (rows == 0 && counts == nullptr) return GEMM355_OK;
    if (!current_device_is_gfx950()) return GEMM355_ERR_DEVICE;
    const bool single = rows > 0 && rows <= kRouteWaves;  // one workgroup writes the counts itself
    if (counts != nullptr && !single) {
        hipLaunchKernelGGL(zero_counts_kernel, dim3(cdiv(experts, 256)), dim3(256), 0, stream, experts, counts);
        if (hipGetLastError() != hipSuccess) return GEMM355_ERR_LAUNCH;
    }
    if (rows == 0) return GEMM355_OK;
    const RouteArgs a{rows, experts, k, groups, top_groups, group_top, X, ldx, bias, scale, ids, weights, counts};
    const bool renorm = flags & GEMM355_ROUTE_RENORM;
    const dim3 grid(cdiv(rows, kRouteWaves) < kRouteGrid ? cdiv(rows, kRouteWaves) : kRouteGrid), block(64 * kRouteWaves);
    const hipError_t e = by_type_and_width(dtype, experts, [&](auto t, auto q) {
        using T = decltype(t);
        constexpr int Q = decltype(q)::value;
        const auto go = [&](auto sig, auto has_bias, auto in_groups) {
            hipLaunchKernelGGL((route_kernel<T, Q, decltype(sig)::value, decltype(has_bias)::value,
                                             decltype(in_groups)::value>),
                               grid, block, 0, stream, a, renorm, single);
        };
        const auto with = [&](auto sig, auto has_bias) {
            top_groups < groups ? go(sig, has_bias, std::true_type{}) : go(sig, has_bias, std::false_type{});
        };
        if (flags & GEMM355_ROUTE_SIGMOID)
            bias != nullptr ? with(std::true_type{}, std::true_type{}) : with(std::true_type{}, std::false_type{});
        else
            bias != nullptr ? with(std::false_type{}, std::true_type{}) : with(std::false_type{}, std::false_type{});
        return hipGetLastError();
    });
    return e == hipSuccess ? GEMM355_OK : GEMM355_ERR_LAUNCH;
}

gemm355_status gemm355_route_grad(int dtype, unsigned flags, int rows, int experts, int k,
                                  const void *X, int ldx, const int32_t *ids,
                                  const float *dweights, float scale, void *dX, int lddx,
                                  hipStream_t stream) {
    if (dtype < kF32 || dtype > kBF16 || (flags & ~kRouteFlags)) return GEMM355_ERR_INVALID_ARG;
    if (rows < 0 || rows > kMaxRouteRows || experts < 1 || experts > kMaxExperts || ldx < experts ||
        lddx < experts || k < 1 || k > kMaxK || k > experts)
        return GEMM355_ERR_INVALID_ARG;
    if (rows == 0) return GEMM355_OK;
    if (X == nullptr || ids == nullptr || dweights == nullptr || dX == nullptr) return GEMM355_ERR_INVALID_ARG;
    const size_t es = dtype == kF32 ? 4 : 2;
    const Span d(dX, matrix_bytes(rows, experts, lddx, es));
    if (X == (const void *)dX) {
        if (ldx != lddx) return GEMM355_ERR_INVALID_ARG;
    } else if (d.meets(Span(X, matrix_bytes(rows, experts, ldx, es)))) {
        return GEMM355_ERR_INVALID_ARG;
    }
    if (d.meets(Span(ids, (size_t)rows * k * 4)) || d.meets(Span(dweights, (size_t)rows * k * 4)))
        return GEMM355_ERR_INVALID_ARG;
    if (!current_device_is_gfx950()) return GEMM355_ERR_DEVICE;
    const bool renorm = flags & GEMM355_ROUTE_RENORM, sigmoid = flags & GEMM355_ROUTE_SIGMOID;
    hipError_t e;
    if (sigmoid || renorm) {
        int n = 1;
        while (n < k) n *= 2;
        const int fit = kGradLds / experts, R = fit < 64 / n ? fit : 64 / n;
        const bool vec = experts % 4 == 0 && lddx % 4 == 0 && (uintptr_t)dX % (4 * es) == 0;
        const dim3 grid(cdiv(rows, 4 * R));
        e = by_type(dtype, [&](auto t) {
            using T = decltype(t);
            const auto go = [&](auto sig, auto v) {
                hipLaunchKernelGGL((route_grad_chosen_kernel<T, decltype(sig)::value, decltype(v)::value>), grid,
                                   dim3(256), 0, stream, rows, experts, k, X, ldx, ids, dweights, scale, dX, lddx,
                                   renorm, n, R);
            };
            if (sigmoid) vec ? go(std::true_type{}, std::true_type{}) : go(std::true_type{}, std::false_type{});
            else vec ? go(std::false_type{}, std::true_type{}) : go(std::false_type{}, std::false_type{});
            return hipGetLastError();
        });
    } else {
        e = by_type_and_width(dtype, experts, [&](auto t, auto q) {
            hipLaunchKernelGGL((route_grad_kernel<decltype(t), decltype(q)::value>), dim3(cdiv(rows, 4)), dim3(256), 0,
                               stream, rows, experts, k, X, ldx, ids, dweights, scale, dX, lddx);
            return hipGetLastError();
        });
    }
    return e == hipSuccess ? GEMM355_OK : GEMM355_ERR_LAUNCH;
}

}  // extern "C"
