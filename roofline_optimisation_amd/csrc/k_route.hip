// Routing to experts and its gradient: rows of router logits -> the k experts of a row and
// their weights (gemm355_softmax.h states the formulas).
//
// The row softmax is the one of "Kernel optimisation guide" (section on softmax
// optimisation); the choice adds a bias, keeps the best groups and takes the k best, ties
// to the lowest index.  Scores are computed in binary64: the ids are whole numbers, and two
// choices that differ by less than a binary32 rounding would otherwise be ordered by the
// order of a sum.
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

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) v += shfl_xor64(v, d);
    return v;
}

__global__ void zero_counts_kernel(int n, int32_t *counts) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n) counts[i] = 0;
}

// One wave per row, Q experts per lane (expert q * 64 + lane), four rows per workgroup.
template <typename T, int Q, bool SIGMOID>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs a, bool renorm) {
    __shared__ double choice_lds[4][Q * 64];
    const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    const int row = blockIdx.x * 4 + wave;
    const bool live = row < a.rows;   // every wave stays for the barrier
    double s[Q], c[Q];
    bool bad = false;
    float m = -__builtin_huge_valf();
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int e = q * 64 + lane;
        const float x = live && e < a.experts ? load_elem<T>(a.X, (size_t)row * a.ldx + e)
                                              : -__builtin_huge_valf();
        bad |= x != x || (!SIGMOID && x == __builtin_huge_valf());
        m = fmaxf(m, x);
        s[q] = (double)x;
    }
    bad = __any(bad);
    if constexpr (SIGMOID) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            c[q] = s[q];
            s[q] = 1.0 / (1.0 + exp(-s[q]));
        }
    } else {
        for (int d = 1; d < 64; d *= 2) m = fmaxf(m, __shfl_xor(m, d, 64));
        double sum = 0.0;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            c[q] = s[q];
            s[q] = s[q] == kLow ? 0.0 : exp(s[q] - (double)m);
            sum += s[q];
        }
        sum = wave_sum64(sum);
#pragma unroll
        for (int q = 0; q < Q; ++q) s[q] = sum > 0.0 ? s[q] / sum : 0.0;
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int e = q * 64 + lane;
        const double v = s[q] + (a.bias != nullptr && e < a.experts ? (double)a.bias[e] : 0.0);
        c[q] = c[q] > kLow && v > kLow ? v : kLow;   // masked, absent and NaN choices
    }
    if (a.top_groups < a.groups) {
        const int per = a.experts / a.groups;
#pragma unroll
        for (int q = 0; q < Q; ++q) choice_lds[wave][q * 64 + lane] = c[q];
        __syncthreads();
        double best = kLow, second = kLow;
        if (lane < a.groups)
            for (int i = 0; i < per; ++i) {
                const double v = choice_lds[wave][lane * per + i];
                if (v > best) {
                    second = best;
                    best = v;
                } else if (v > second) {
                    second = v;
                }
            }
        const double score = a.group_top == 2 && second > kLow ? best + second : best;
        int rank = 0;
        for (int g = 0; g < a.groups; ++g) {
            const double o = __shfl(score, g, 64);
            rank += o > score || (o == score && g < lane);
        }
        const unsigned long long kept = __ballot(lane < a.groups && rank < a.top_groups);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int g = (q * 64 + lane) / per;
            if (g >= a.groups || !((kept >> g) & 1)) c[q] = kLow;
        }
    }
    int my_id = -1;
    double my_s = 0.0, total = 0.0;
    for (int i = 0; i < a.k; ++i) {
        double v = kLow, sv = 0.0;
        int at = 0x7fffffff;
#pragma unroll
        for (int q = 0; q < Q; ++q)
            if (c[q] > v) {
                v = c[q];
                sv = s[q];
                at = q * 64 + lane;
            }
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const double vo = shfl_xor64(v, d), so = shfl_xor64(sv, d);
            const int ao = __shfl_xor(at, d, 64);
            if (vo > v || (vo == v && ao < at)) {
                v = vo;
                sv = so;
                at = ao;
            }
        }
        if (at == 0x7fffffff || bad) break;   // no expert left (the same in every lane)
        if (lane == i) {
            my_id = at;
            my_s = sv;
        }
        total += sv;
#pragma unroll
        for (int q = 0; q < Q; ++q)
            if (at == q * 64 + lane) c[q] = kLow;
    }
    if (live && lane < a.k) {
        double w = my_s;
        if (renorm) w = total > 0.0 ? w / total : 0.0;
        w *= (double)a.scale;
        if (my_id < 0) w = bad ? __builtin_nan("") : 0.0;
        a.ids[(size_t)row * a.k + lane] = my_id;
        a.weights[(size_t)row * a.k + lane] = (float)w;
        if (a.counts != nullptr && my_id >= 0) atomicAdd(a.counts + my_id, 1);
    }
}

// The gradient: one wave per row, Q experts per lane.
template <typename T, int Q, bool SIGMOID>
__global__ __launch_bounds__(256) void route_grad_kernel(int rows, int experts, int k, const void *X,
                                                         int ldx, const int32_t *ids,
                                                         const float *dweights, float scale, void *dX,
                                                         int lddx, bool renorm) {
    const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    const int row = blockIdx.x * 4 + wave;
    if (row >= rows) return;
    float s[Q], ds[Q];
    float m = -__builtin_huge_valf();
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int e = q * 64 + lane;
        s[q] = e < experts ? load_elem<T>(X, (size_t)row * ldx + e) : -__builtin_huge_valf();
        ds[q] = 0.0f;
        m = fmaxf(m, s[q]);
    }
    if constexpr (SIGMOID) {
#pragma unroll
        for (int q = 0; q < Q; ++q) s[q] = 1.0f / (1.0f + expf(-s[q]));
    } else {
        for (int d = 1; d < 64; d *= 2) m = fmaxf(m, __shfl_xor(m, d, 64));
        const float shift = m == -__builtin_huge_valf() ? 0.0f : m;
        float sum = 0.0f;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            s[q] = expf(s[q] - shift);
            sum += s[q];
        }
        sum = wave_allreduce_sum(sum);
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;   // a NaN row stays NaN
#pragma unroll
        for (int q = 0; q < Q; ++q) s[q] *= inv;
    }
    const int32_t *id = ids + (size_t)row * k;
    const float *dw = dweights + (size_t)row * k;
    float sum_s = 0.0f, sum_qs = 0.0f;   // this lane's share over its chosen experts
    for (int i = 0; i < k; ++i) {
        const int e = id[i];
        const float g = scale * dw[i];
#pragma unroll
        for (int q = 0; q < Q; ++q)
            if (e == q * 64 + lane && e < experts) {
                ds[q] += g;
                sum_s += s[q];
                sum_qs += g * s[q];
            }
    }
    if (renorm) {
        sum_s = wave_allreduce_sum(sum_s);
        sum_qs = wave_allreduce_sum(sum_qs);
        const float inv = sum_s == 0.0f ? 0.0f : 1.0f / sum_s;
        const float mean = sum_qs * inv;
#pragma unroll
        for (int q = 0; q < Q; ++q) ds[q] = 0.0f;
        for (int i = 0; i < k; ++i) {
            const int e = id[i];
            const float g = (scale * dw[i] - mean) * inv;
#pragma unroll
            for (int q = 0; q < Q; ++q)
                if (e == q * 64 + lane && e < experts) ds[q] += g;
        }
    }
    float dot = 0.0f;
    if constexpr (!SIGMOID) {
#pragma unroll
        for (int q = 0; q < Q; ++q) dot += ds[q] * s[q];
        dot = wave_allreduce_sum(dot);
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int e = q * 64 + lane;
        const float d = SIGMOID ? ds[q] * s[q] * (1.0f - s[q]) : s[q] * (ds[q] - dot);
        if (e < experts) store_elem<T>(dX, (size_t)row * lddx + e, d);
    }
}

// f(T{}, integral_constant<int, Q>) for the storage type and the experts per lane.
template <typename F>
hipError_t by_type_and_width(int dtype, int experts, F f) {
    const auto width = [&](auto t) -> hipError_t {
        if (experts <= 64) return f(t, std::integral_constant<int, 1>{});
        if (experts <= 128) return f(t, std::integral_constant<int, 2>{});
        if (experts <= 256) return f(t, std::integral_constant<int, 4>{});
        if (experts <= 512) return f(t, std::integral_constant<int, 8>{});
        return f(t, std::integral_constant<int, 16>{});
    };
    if (dtype == kF32) return width(0.0f);
    if (dtype == kF16) return width(f16_t{});
    return width(bf16_t{});
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
    if (counts != nullptr) {
        hipLaunchKernelGGL(zero_counts_kernel, dim3(cdiv(experts, 256)), dim3(256), 0, stream, experts, counts);
        if (hipGetLastError() != hipSuccess) return GEMM355_ERR_LAUNCH;
    }
    if (rows == 0) return GEMM355_OK;
    const RouteArgs a{rows, experts, k, groups, top_groups, group_top, X, ldx, bias, scale, ids, weights, counts};
    const bool renorm = flags & GEMM355_ROUTE_RENORM;
    const hipError_t e = by_type_and_width(dtype, experts, [&](auto t, auto q) {
        using T = decltype(t);
        constexpr int Q = decltype(q)::value;
        const dim3 grid(cdiv(rows, 4));
        if (flags & GEMM355_ROUTE_SIGMOID)
            hipLaunchKernelGGL((route_kernel<T, Q, true>), grid, dim3(256), 0, stream, a, renorm);
        else
            hipLaunchKernelGGL((route_kernel<T, Q, false>), grid, dim3(256), 0, stream, a, renorm);
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
    const bool renorm = flags & GEMM355_ROUTE_RENORM;
    const hipError_t e = by_type_and_width(dtype, experts, [&](auto t, auto q) {
        using T = decltype(t);
        constexpr int Q = decltype(q)::value;
        const dim3 grid(cdiv(rows, 4));
        if (flags & GEMM355_ROUTE_SIGMOID)
            hipLaunchKernelGGL((route_grad_kernel<T, Q, true>), grid, dim3(256), 0, stream, rows, experts, k, X,
                               ldx, ids, dweights, scale, dX, lddx, renorm);
        else
            hipLaunchKernelGGL((route_grad_kernel<T, Q, false>), grid, dim3(256), 0, stream, rows, experts, k, X,
                               ldx, ids, dweights, scale, dX, lddx, renorm);
        return hipGetLastError();
    });
    return e == hipSuccess ? GEMM355_OK : GEMM355_ERR_LAUNCH;
}

}  // extern "C"
