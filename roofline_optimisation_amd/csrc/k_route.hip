// Routing to experts and its gradient: rows of router logits -> the k experts of a row and
// their weights (gemm355_softmax.h states the formulas).
//
// The row softmax is the one of "Kernel optimisation guide" (section on softmax
// optimisation); the choice adds a bias, keeps the best groups and takes the k best, ties
// to the lowest index.
//
// One wave takes a row, Q = experts / 64 neighbouring ones per lane.  A row is a few hundred
// bytes, so the time goes into instructions, not memory.  The ids are whole numbers and have
// to be those of exact scores, but only rows with two candidates closer than binary32 can
// tell apart need better: a row is first decided on 32-bit keys (the logits themselves where
// no bias is added, so exactly; else binary32 scores plus bias), and where two neighbours of
// the resulting order, or two groups, are closer than the bound of the scores' error, the
// row is decided again on binary64 scores.  Each lane sorts its keys; a round then takes the
// largest first key (four register exchanges within 16 lanes, a scalar maximum of four lanes)
// and the lowest lane that holds it (a ballot), whose next key moves up.
//
// Bound by vector instructions, 530 a row of 256 experts in groups with a bias and 8
// places (binary64 throughout: four times as many).  16384 such rows take 22.2 us and their
// counts 3.9 more, a call 24.3 us and without groups and bias 11.6; reading the logits alone
// would take 4.  With rounds that look through all of a lane's keys, groups ranked one after
// the other, the weights of one row at a time and counts added up by each workgroup's atomics
// it was 36.  Registers (88) leave five waves on a SIMD; a bound of six makes the compiler
// spill.
#include <algorithm>

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

// A group's score, in every one of its S lanes (a power of two, aligned), from the two largest
// choices that each of them has seen.
template <typename F>
__device__ __forceinline__ F group_score(F best, F second, int S, int group_top) {
    if (S > 1) merge_two(best, second, exchange<DppXchg<kDppQuadXor1>>(best), exchange<DppXchg<kDppQuadXor1>>(second));
    if (S > 2) merge_two(best, second, exchange<DppXchg<kDppQuadXor2>>(best), exchange<DppXchg<kDppQuadXor2>>(second));
    if (S > 4)
        merge_two(best, second, exchange<DppXchg<kDppRowHalfMirror>>(best), exchange<DppXchg<kDppRowHalfMirror>>(second));
    if (S > 8) merge_two(best, second, exchange<DppXchg<kDppRowMirror>>(best), exchange<DppXchg<kDppRowMirror>>(second));
    if (S > 16) merge_two(best, second, exchange<SwapHalves16>(best), exchange<SwapHalves16>(second));
    return group_top == 2 && second > (F)kLow ? best + second : best;
}

// The same for a group of `per` experts whose choices lie in LDS, scanned by its S lanes.
template <typename F>
__device__ __forceinline__ F group_score(const F *choice, int per, int S, int sub, int group_top) {
    constexpr F low = (F)kLow;
    F best = low, second = low;
#pragma unroll 1
    for (int i = sub; i < per; i += S) merge_two(best, second, choice[i], low);
    return group_score(best, second, S, group_top);
}

__device__ __forceinline__ float lane_value(float v, int lane) { return read_lane(v, lane); }
__device__ __forceinline__ double lane_value(double v, int lane) {
    const unsigned long long u = __builtin_bit_cast(unsigned long long, v);
    return __builtin_bit_cast(double, (unsigned long long)(uint32_t)__builtin_amdgcn_readlane((int)u, lane) |
                                          (unsigned long long)(uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), lane)
                                              << 32);
}

// Which of the groups are among the `top` of the largest score, ties to the lowest group, as
// the lanes of those groups; near: a kept score lies within `margin` of one that is not.  A
// lane holds the score of group lane >> shift (shift < 6), and compares it with that of every
// 2^shift-th group.
template <typename F>
__device__ __forceinline__ unsigned long long best_groups(F score, int groups, int top, int shift, F margin,
                                                          bool &near) {
    const int lane = threadIdx.x % 64, mine = lane >> shift, S = 1 << shift, first = lane & -S;
    const uint32_t group_lanes = 0xffffffffu >> (32 - S);
    int rank = 0;
    int close = 0;   // groups ahead of mine by no more than the margin
#pragma unroll 1
    for (int g0 = 0; g0 < groups; g0 += S) {
        const int g = g0 + (lane & (S - 1));
        const F o = __shfl(score, (g << shift) & 63, 64);
        const bool ahead = (g < groups) & ((o > score) | ((o == score) & (g < mine)));   // no branches
        rank += __builtin_popcount((uint32_t)(__ballot(ahead) >> first) & group_lanes);
        close += __builtin_popcount((uint32_t)(__ballot(ahead & (o - score <= margin)) >> first) & group_lanes);
    }
    // not kept, and one that is (ranks below top) among those just ahead
    near = __any(mine < groups && rank >= top && rank - close < top);
    return __ballot(mine < groups && rank < top);
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
struct TaylorTable {
    double v[kTaylor];
    constexpr TaylorTable() : v{} {
        double f = 1.0;
        for (int n = 0; n < kTaylor; ++n) {
            f *= n > 1 ? (double)n : 1.0;
            v[kTaylor - 1 - n] = 1.0 / f;
        }
    }
};
__constant__ const TaylorTable kTaylorTable;
__device__ __forceinline__ void taylor_to_lds(double *coef) {
    if (threadIdx.x < kTaylor) coef[threadIdx.x] = kTaylorTable.v[threadIdx.x];
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

// The lanes of the row's kept groups by binary64 choices, which are left in the wave's row of
// LDS.
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
    const int shift = group_shift(a->groups);
    const bool by_logit = a->bias == nullptr;
#pragma unroll 1
    for (int e0 = 0; e0 < experts; e0 += 64) {
        const int e = e0 + lane;
        double c = choice[e];
        // without a bias the order within the kept groups is the logits'
        if (by_logit && c > kLow) c = (double)logit_at<T>(a->X, row * a->ldx, e, experts);
        choice[e] = (kept >> (((e / per) << shift) & 63)) & 1 ? c : kLow;
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

// Rows of more than 512 experts are always decided on binary64 scores: 16 keys per lane, and
// the order of them, would take more registers than the rest of the kernel.
constexpr bool has_keys(int Q) { return Q <= 8; }

// Logits lane Q ... lane Q + Q - 1 of a row, -infinity past its experts.  vec: whole chunks of
// Q, aligned to their bytes or 16.
template <typename T, int Q>
__device__ __forceinline__ void load_logits(const void *X, size_t x0, int lane, int experts, bool vec, float (&x)[Q]) {
    struct alignas(Q * sizeof(T) < 16 ? Q * sizeof(T) : 16) Chunk {
        T v[Q];
    };
    if (vec) {
        const Chunk c = *(const Chunk *)((const T *)X + x0 + min(lane * Q, experts - Q));
#pragma unroll
        for (int q = 0; q < Q; ++q) x[q] = lane * Q < experts ? to_float(c.v[q]) : -__builtin_huge_valf();
    } else {
#pragma unroll
        for (int q = 0; q < Q; ++q) x[q] = logit_at<T>(X, x0, lane * Q + q, experts);
    }
}

// A lane's keys in descending order, equal ones by expert; returns (four bits each, the first
// key's lowest) which of the lane's experts they are: a bitonic network of compare-exchanges
// on 64-bit pairs of key and the expert's place from the lane's end.
template <int Q>
__device__ __forceinline__ uint32_t sort_keys(uint32_t (&key)[Q]) {
    unsigned long long p[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) p[q] = (unsigned long long)key[q] << 32 | (unsigned)(Q - 1 - q);
#pragma unroll
    for (int size = 2; size <= Q; size *= 2)
#pragma unroll
        for (int d = size / 2; d > 0; d /= 2)
#pragma unroll
            for (int q = 0; q < Q; ++q)
                if (!(q & d)) {
                    const unsigned long long a = p[q], b = p[q | d];
                    const bool swap = (q & size) ? a > b : a < b;
                    p[q] = swap ? b : a;
                    p[q | d] = swap ? a : b;
                }
    uint32_t order = 0;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        key[q] = (uint32_t)(p[q] >> 32);
        order |= (Q - 1 - (uint32_t)p[q]) << 4 * q;
    }
    return order;
}

// Waves of a workgroup that takes every row, with at most half a CU's LDS.
constexpr int route_waves(int experts) { return experts <= 256 ? 16 : experts <= 512 ? 8 : 4; }
// Workgroups of 4 waves at most.  With 1024 the two calls above take 24.4 and 13.5 us, with
// 4096, where 16384 rows leave no wave a second one, 26.0 and 12.7.
constexpr int kRouteGrid = 2048;

// The ids of a row: place i in lane i, -1 for none.  m: softmax's maximum; bad: no routing
// (NaN, for softmax +infinity).  b, top_b: the lane's biases and a bound of all; group_at: the
// first lane of each expert's group; choice: the wave's row of LDS.
template <typename T, int Q, bool SIGMOID, bool BIAS, bool GROUPS>
__device__ __forceinline__ int choose(const RouteArgs &a, size_t row, bool vec, const float (&b)[Q], float top_b,
                                      const int (&group_at)[Q], int per, double *choice, const double *coef, float &m,
                                      bool &bad) {
    constexpr float kNegInf = -__builtin_huge_valf();
    // the lane as each row's own value, or the masks of absent experts, two scalar registers
    // each, are kept across rows
    int lane = threadIdx.x % 64;
    asm volatile("" : "+v"(lane));
    float x[Q];
    load_logits<T, Q>(a.X, row * a.ldx, lane, a.experts, vec, x);
    m = kNegInf;
    bad = false;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        bad |= __builtin_amdgcn_classf(x[q], SIGMOID ? 0x003 : 0x203);   // NaN, +infinity
        m = fmaxf(m, x[q]);
    }
    bad = __any(bad);
    if constexpr (!SIGMOID) m = wave_max(m);
    if (bad || (!SIGMOID && !(m > kNegInf))) return -1;
    int id = -1;
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
            const int groups = am->groups, shift = group_shift(groups), S = 1 << shift;
            float score;
            if (per == Q << shift) {   // a group's experts are those of its own lanes
                float best = s[0], second = kNegInf;
#pragma unroll
                for (int q = 1; q < Q; ++q) merge_two(best, second, s[q], kNegInf);
                score = group_score(best, second, S, am->group_top);
            } else {
                float *c = (float *)choice;
#pragma unroll
                for (int q = 0; q < Q; ++q) c[lane * Q + q] = s[q];
                wave_lds_sync();
                score = group_score((const float *)c + min(lane >> shift, groups - 1) * per, per, S, lane & (S - 1),
                                    am->group_top);
                wave_lds_sync();
            }
            bool close;
            unsigned long long kept = best_groups(score, groups, am->top_groups, shift, 2.5f * margin, close);
            if (close) kept = exact_groups<T, Q, SIGMOID>(row, m, choice, coef);
#pragma unroll
            for (int q = 0; q < Q; ++q) key[q] = (kept >> group_at[q]) & 1 ? key[q] : 0u;
        }
        // The places, the i-th key in lane i as its id.  Each lane's first key is the largest
        // it has left; the lowest lane that holds the wave's largest is taken, and its next
        // key moves up.  With a bias, one more place to see how far the last is from what
        // stays out: neighbours closer than the margin are put in order in binary64, and if
        // the one after the last is as close to the next, the row is left to binary64 choices
        // altogether.
        uint32_t order = sort_keys(key);
        uint32_t my_key = 0;
        const int places = BIAS ? min(a.k + 1, 64) : a.k;
        for (int i = 0; i < places; ++i) {
            const uint32_t v = wave_max_u32(key[0]);
            if (v == 0) break;
            const int from = __builtin_ctzll(__ballot(key[0] == v));
            const int at = from * Q + (__builtin_amdgcn_readlane(order, from) & 15);
            const bool here = lane == i;
            id = here ? at : id;
            if constexpr (BIAS) my_key = here ? v : my_key;
            const bool taken = lane == from;
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                // values, not elements: a choice between elements becomes one of their index
                const uint32_t held = key[q];
                uint32_t after = 0;
                if (q + 1 < Q) after = key[q + 1 < Q ? q + 1 : q];
                key[q] = taken ? after : held;
            }
            order = taken ? order >> 4 : order;
        }
        if constexpr (BIAS) {
            const uint32_t after = __shfl_down(my_key, 1, 64);
            const bool close = lane < 63 && after != 0 && of_key(my_key) - of_key(after) <= margin;
            const unsigned long long w = __ballot(close);   // lane i: places i and i + 1
            if (w != 0) {
                bool lost = places == 64;   // no lane for the one after the last
                if (!lost && ((w >> (places - 2)) & 1)) {
                    const uint32_t last = __builtin_amdgcn_readlane(my_key, places - 1);
                    const uint32_t v = wave_max_u32(key[0]);
                    lost = v != 0 && of_key(last) - of_key(v) <= margin;
                }
                near = lost;
                if (!lost) id = exact_order<T, SIGMOID>(row, m, id, coef);
            }
            id = lane < a.k ? id : -1;
        }
    }
    if constexpr (BIAS || GROUPS || !has_keys(Q))
        if (near) id = exact_ids<T, Q, SIGMOID>(row, m, choice, coef);
    return id;
}

// BIAS: choices add a.bias.  GROUPS: a.top_groups < a.groups.  vec: load_logits.  A wave
// chooses for two rows one after the other (one where k > 32), and finds the weights of both
// at once, a place per lane.  single: one workgroup takes every row and writes the counts;
// else they are set to zero here, for route_count_kernel.
template <typename T, int Q, bool SIGMOID, bool BIAS, bool GROUPS>
__global__ __launch_bounds__(1024) void route_kernel(RouteArgs a, bool renorm, bool single, bool vec) {
    constexpr bool kExact = BIAS || GROUPS || !has_keys(Q);
    extern __shared__ double choice_lds[];   // kExact: Q * 64 per wave
    __shared__ int hist[Q * 64];
    __shared__ double coef[kTaylor];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane0 = threadIdx.x % 64;
    const int waves = blockDim.x / 64;
    constexpr float kNegInf = -__builtin_huge_valf();
    const bool count = a.counts != nullptr && single;
    taylor_to_lds(coef);
    if (count)
        for (int e = threadIdx.x; e < a.experts; e += blockDim.x) hist[e] = 0;
    if (a.counts != nullptr && !single && blockIdx.x == 0)
        for (int e = threadIdx.x; e < a.experts; e += blockDim.x) a.counts[e] = 0;
    __syncthreads();
    float b[Q], top_b = 0.0f;
    if constexpr (BIAS && has_keys(Q)) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int e = lane0 * Q + q;
            b[q] = e < a.experts ? a.bias[e] : 0.0f;
            // a masked expert's bias bounds nothing (NaN: the maximum ignores it)
            top_b = fmaxf(top_b, b[q] == kNegInf ? 0.0f : fabsf(b[q]));
        }
        top_b = wave_max(top_b);
    }
    int per = 1, group_at[Q];   // of an absent expert, whose key is 0: any lane
    if constexpr (GROUPS && has_keys(Q)) {
        per = a.experts / a.groups;
        // e / per for e below 1024: e + 1/2 is 1 / (2 per) off any multiple, far above the rounding
        const float inv = 1.0f / (float)per;
#pragma unroll
        for (int q = 0; q < Q; ++q)
            group_at[q] = ((int)(((float)(lane0 * Q + q) + 0.5f) * inv) << group_shift(a.groups)) & 63;
    }
    const int span = a.k <= 32 ? 32 : 64;   // lanes of a row's places
    const int half = lane0 / span, slot = lane0 & (span - 1);
    const int stride = gridDim.x * waves;
    for (int first = blockIdx.x * waves + wave; first < a.rows; first += stride * (64 / span)) {
        int id = -1;
        float m = kNegInf;
        bool bad = false;
        double sum = 1.0;
#pragma unroll 1
        for (int h = 0; h < 64 / span; ++h) {
            const int row = first + h * stride;
            if (row >= args_in_memory()->rows) break;
            float m_h;
            bool bad_h;
            int id_h = choose<T, Q, SIGMOID, BIAS, GROUPS>(a, row, vec, b, top_b, group_at, per,
                                                           choice_lds + wave * (Q * 64), coef, m_h, bad_h);
            if (h > 0) id_h = __shfl(id_h, slot, 64);
            double sum_h = 1.0;
            if (!SIGMOID && !renorm) sum_h = divisor64<T, SIGMOID>(a.X, (size_t)row * a.ldx, a.experts, m_h, coef);
            id = half == h ? id_h : id;
            m = half == h ? m_h : m;
            bad = half == h ? bad_h : bad;
            sum = half == h ? sum_h : sum;
        }
        // the weights, in binary64
        const ArgsPtr am = args_in_memory();
        const int row = first + half * stride;
        const float xi = id >= 0 ? logit_at<T>(am->X, (size_t)row * am->ldx, id, am->experts) : kNegInf;
        double w = score64<SIGMOID>(xi, m, coef);
        if (renorm) sum = lanes_sum64(w, am->k <= 8 ? 8 : span);
        w = sum > 0.0 ? w / sum : 0.0;
        w *= (double)am->scale;
        if (id < 0) w = bad ? __builtin_nan("") : 0.0;
        if (slot < am->k && row < am->rows) {
            am->ids[(size_t)row * am->k + slot] = id;
            am->weights[(size_t)row * am->k + slot] = (float)w;
            if (count && id >= 0) atomicAdd(&hist[id], 1);
        }
    }
    if (!count) return;
    __syncthreads();
    int32_t *counts = args_in_memory()->counts;
    for (int e = threadIdx.x; e < a.experts; e += blockDim.x) counts[e] = hist[e];
}

// counts (zeros before) += how often each expert is among the n ids.  Per workgroup in LDS, then
// added in memory: whole numbers, so in any order.
constexpr int kCountGrid = 256, kCountIds = 4096;  // workgroups at most, ids of one at least
__global__ __launch_bounds__(1024) void route_count_kernel(size_t n, int experts, const int32_t *__restrict__ ids,
                                                           int32_t *counts) {
    __shared__ int hist[kMaxExperts];
    for (int e = threadIdx.x; e < experts; e += 1024) hist[e] = 0;
    __syncthreads();
    for (size_t i0 = (size_t)blockIdx.x * kCountIds; i0 < n; i0 += (size_t)gridDim.x * kCountIds) {
        int id[kCountIds / 1024];
#pragma unroll
        for (int j = 0; j < kCountIds / 1024; ++j) {
            const size_t i = i0 + j * 1024 + threadIdx.x;
            id[j] = i < n ? ids[i] : -1;
        }
#pragma unroll
        for (int j = 0; j < kCountIds / 1024; ++j)
            if (id[j] >= 0) atomicAdd(&hist[id[j]], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < experts; e += 1024)
        if (hist[e] > 0) atomicAdd(counts + e, hist[e]);
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
    const bool single = rows > 0 && rows <= route_waves(experts);  // one workgroup writes the counts itself
    if (rows == 0) {
        hipLaunchKernelGGL(zero_counts_kernel, dim3(cdiv(experts, 256)), dim3(256), 0, stream, experts, counts);
        return hipGetLastError() == hipSuccess ? GEMM355_OK : GEMM355_ERR_LAUNCH;
    }
    const RouteArgs a{rows, experts, k, groups, top_groups, group_top, X, ldx, bias, scale, ids, weights, counts};
    const bool renorm = flags & GEMM355_ROUTE_RENORM;
    const int waves = single ? route_waves(experts) : 4;
    const dim3 grid(std::min(cdiv(rows, waves), kRouteGrid)), block(64 * waves);
    hipError_t e = by_type_and_width(dtype, experts, [&](auto t, auto q) -> hipError_t {
        using T = decltype(t);
        constexpr int Q = decltype(q)::value;
        const bool vec = experts % Q == 0 && ldx % Q == 0 && (uintptr_t)X % (Q * es < 16 ? Q * es : 16) == 0;
        const auto go = [&](auto sig, auto has_bias, auto in_groups) {
            constexpr bool exact = decltype(has_bias)::value || decltype(in_groups)::value || !has_keys(Q);
            hipLaunchKernelGGL((route_kernel<T, Q, decltype(sig)::value, decltype(has_bias)::value,
                                             decltype(in_groups)::value>),
                               grid, block, exact ? waves * Q * 512 : 0, stream, a, renorm, single, vec);
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
    if (e == hipSuccess && counts != nullptr && !single) {
        const size_t n = (size_t)rows * k, parts = (n + kCountIds - 1) / kCountIds;
        hipLaunchKernelGGL(route_count_kernel, dim3(parts < kCountGrid ? parts : kCountGrid), dim3(1024), 0, stream, n,
                           experts, ids, counts);
        e = hipGetLastError();
    }
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
    // rows of one launch: its threads (64 a row at most) number fewer than 2^32
    constexpr int kRows = 1 << 25;
    for (int r0 = 0; r0 < rows; r0 += kRows) {
        const int live = std::min(rows - r0, kRows);
        const char *x = (const char *)X + (size_t)r0 * ldx * es;
        char *dx = (char *)dX + (size_t)r0 * lddx * es;
        const int32_t *id = ids + (size_t)r0 * k;
        const float *dw = dweights + (size_t)r0 * k;
        hipError_t e;
        if (sigmoid || renorm) {
            int n = 1;
            while (n < k) n *= 2;
            const int fit = kGradLds / experts, R = fit < 64 / n ? fit : 64 / n;
            const bool vec = experts % 4 == 0 && lddx % 4 == 0 && (uintptr_t)dX % (4 * es) == 0;
            const dim3 grid(cdiv(live, 4 * R));
            e = by_type(dtype, [&](auto t) {
                using T = decltype(t);
                const auto go = [&](auto sig, auto v) {
                    hipLaunchKernelGGL((route_grad_chosen_kernel<T, decltype(sig)::value, decltype(v)::value>), grid,
                                       dim3(256), 0, stream, live, experts, k, x, ldx, id, dw, scale, dx, lddx, renorm,
                                       n, R);
                };
                if (sigmoid) vec ? go(std::true_type{}, std::true_type{}) : go(std::true_type{}, std::false_type{});
                else vec ? go(std::false_type{}, std::true_type{}) : go(std::false_type{}, std::false_type{});
                return hipGetLastError();
            });
        } else {
            e = by_type_and_width(dtype, experts, [&](auto t, auto q) {
                hipLaunchKernelGGL((route_grad_kernel<decltype(t), decltype(q)::value>), dim3(cdiv(live, 4)), dim3(256),
                                   0, stream, live, experts, k, x, ldx, id, dw, scale, dx, lddx);
                return hipGetLastError();
            });
        }
        if (e != hipSuccess) return GEMM355_ERR_LAUNCH;
    }
    return GEMM355_OK;
}

}  // extern "C"
