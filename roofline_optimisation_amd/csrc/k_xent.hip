// Softmax cross entropy of a projection and its gradient, piece by piece of the vocabulary
// (gemm355_softmax.h states the formulas).
//
// Forward: the online softmax of "Kernel optimisation guide" (section on softmax
// optimisation) over pieces of columns: each piece's (maximum, sum of exponentials) pair is
// merged into the row's, the sum of the smaller maximum rescaled, and the logit of the
// label is kept when its column passes.  Backward: dZ = g (exp(Z - lse) - onehot) of each
// piece, rounded to the operands' type, is the left operand of dX += dZ.op(W)^T and of the
// piece's columns (or rows) of dW = X^T.dZ.
//
// This file: the rows' kernels, the plan that lays out a call's workspace, and the entry
// points.  The products run in this library's GEMM kernels.
#include "../../include/gemm355_softmax.h"
#include "common.hpp"
#include "launch.hpp"
#include "wave_reduce.hpp"

namespace g355 {

namespace {

constexpr float kNegInf = -__builtin_huge_valf();
constexpr int kMaxDim = (1 << 30) - 1;

// A row's running statistics: maximum m, sum l of exp(z - m), the label's logit.
struct RowState { float m, l, z; };

// What the gradient needs of a row: its log-sum-exp, the upstream gradient (scaled) and the
// label, -1 for a row without one (whose g is 0 and whose copy of X is 0).
struct RowGrad { float lse, g; int label, unused; };

// (m, l) merged with another pair; an empty pair is (-infinity, 0).
__device__ __forceinline__ void merge_pair(float &m, float &l, float mo, float lo) {
    const bool mine = m >= mo;
    const float hi = mine ? m : mo, low = mine ? mo : m;
    const float lhi = mine ? l : lo, llo = mine ? lo : l;
    l = lhi + llo * (low == hi ? 1.0f : expf(low - hi));
    m = hi;
}

struct MergePair {
    __device__ __forceinline__ void operator()(float &m, float &l, float mo, float lo) const {
        merge_pair(m, l, mo, lo);
    }
};

// loss and lse of a row from its statistics.  label: the given one.
__device__ __forceinline__ void finish_row(int row, float m, float l, float z, int64_t label, int64_t ignore,
                                           int N, float *loss, float *lse) {
    const float s = m + logf(l);
    if (lse != nullptr) lse[row] = s;
    if (loss != nullptr)
        loss[row] = label == ignore ? 0.0f
                    : label < 0 || label >= N ? __builtin_nanf("")
                    : s - z;
}

// One workgroup per row of a piece Z (columns v0 .. v0 + nc of the logits): its statistics
// merged into state[row] (or started, at v0 == 0); the last piece writes the results.
__global__ __launch_bounds__(256) void xent_rows_kernel(int nc, int v0, int N, const float *__restrict__ Z,
                                                        int ldz, const int64_t *__restrict__ labels,
                                                        int64_t ignore, RowState *state, float *loss,
                                                        float *lse) {
    __shared__ float sm[4], sl[4];
    const int row = blockIdx.x, wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    const float *z = Z + (size_t)row * ldz;
    float m = kNegInf, l = 0.0f;
    for (int base = 0; base < nc; base += 1024) {
        float v[4], cm = kNegInf;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int c = base + 256 * u + (int)threadIdx.x;
            v[u] = c < nc ? z[c] : kNegInf;
            cm = fmaxf(cm, v[u]);
        }
        if (cm > m) {
            l *= expf(m - cm);
            m = cm;
        }
        const float shift = m == kNegInf ? 0.0f : m;
#pragma unroll
        for (int u = 0; u < 4; ++u) l += expf(v[u] - shift);
    }
    wave_allreduce2(m, l, MergePair{});
    if (lane == 0) {
        sm[wave] = m;
        sl[wave] = l;
    }
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int w = 1; w < 4; ++w) merge_pair(m, l, sm[w], sl[w]);
    RowState s{kNegInf, 0.0f, 0.0f};
    if (v0 > 0) s = state[row];
    merge_pair(s.m, s.l, m, l);
    const int64_t label = labels[row];
    if (label >= v0 && label < (int64_t)v0 + nc) s.z = z[label - v0];
    if (v0 + nc < N) state[row] = s;
    else finish_row(row, s.m, s.l, s.z, label, ignore, N, loss, lse);
}

// Before the gradient's pieces: scale[0] = S and scale[1] = 1 / S (S = 1 unless `rescale`:
// then the power of two that puts the largest |dloss| in [2^13, 2^14), from 2^-100 to
// 2^100), the rows' RowGrad, and Xm = X with the rows without a label set to zero (their
// products with a zero row of dZ would not be zero where X holds an infinity or NaN).
// Every workgroup finds the same maximum over all rows, then does its share of the rows.
template <typename E>
__global__ __launch_bounds__(256) void xent_prep_kernel(int M, int N, int K, const E *__restrict__ X, int ldx,
                                                        const int64_t *__restrict__ labels, int64_t ignore,
                                                        const float *__restrict__ lse,
                                                        const float *__restrict__ dloss, int rescale,
                                                        float *scale, RowGrad *rows, E *Xm, int ldm) {
    __shared__ float sm[4];
    float S = 1.0f;
    if (rescale) {
        float top = 0.0f;
        for (int r = threadIdx.x; r < M; r += 256) {
            const int64_t y = labels[r];
            if (y != ignore && y >= 0 && y < N) top = fmaxf(top, fabsf(dloss[r]));
        }
        for (int d = 1; d < 64; d *= 2) top = fmaxf(top, __shfl_xor(top, d, 64));
        if (threadIdx.x % 64 == 0) sm[threadIdx.x / 64] = top;
        __syncthreads();
        top = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
        if (top > 0.0f && top < __builtin_huge_valf())
            S = ldexpf(1.0f, max(-100, min(100, 13 - ilogbf(top))));
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        scale[0] = S;
        scale[1] = 1.0f / S;
    }
    for (int r = blockIdx.x; r < M; r += gridDim.x) {
        const int64_t y = labels[r];
        const bool live = y != ignore && y >= 0 && y < N;
        if (threadIdx.x == 0)
            rows[r] = live ? RowGrad{lse[r], dloss[r] * S, (int)y, 0} : RowGrad{0.0f, 0.0f, -1, 0};
        const E *x = X + (size_t)r * ldx;
        E *o = Xm + (size_t)r * ldm;
        for (int c = threadIdx.x; c < ldm; c += 256) o[c] = live && c < K ? x[c] : E{};
    }
}

// dZ of a piece from its logits: column v of the piece is class v0 + v.  Grid: (columns /
// 1024, rows).  Out may be Z itself (binary32).
template <typename T>
__global__ __launch_bounds__(256) void xent_dz_kernel(int nc, int v0, const float *Z, int ldz,
                                                      const RowGrad *__restrict__ rows, void *out, int ldo) {
    const int row = blockIdx.y;
    const RowGrad r = rows[row];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int c = blockIdx.x * 1024 + 256 * u + (int)threadIdx.x;
        if (c >= nc) break;
        const float p = expf(Z[(size_t)row * ldz + c] - r.lse);
        const float d = r.g * (p - (v0 + c == r.label ? 1.0f : 0.0f));
        if constexpr (std::is_same<T, float>::value) ((float *)out)[(size_t)row * ldo + c] = d;
        else ((uint16_t *)out)[(size_t)row * ldo + c] = to_bits(d, T{});
    }
}

// out = scale[1] * acc, rounded to the 16-bit type.  Grid: (columns / 1024, rows).
template <typename T>
__global__ __launch_bounds__(256) void xent_round_kernel(int cols, const float *__restrict__ acc, int lda,
                                                         const float *__restrict__ scale, uint16_t *out,
                                                         int ldo) {
    const float f = scale[1];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int c = blockIdx.x * 1024 + 256 * u + (int)threadIdx.x;
        if (c >= cols) break;
        out[(size_t)blockIdx.y * ldo + c] = to_bits(f * acc[(size_t)blockIdx.y * lda + c], T{});
    }
}

template <typename E>
__global__ void zero_matrix_kernel(int cols, E *out, int ld) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c < cols) out[(size_t)blockIdx.y * ld + c] = E{};
}

// Rows of a grid's y axis; more rows than that take several launches.
constexpr int kGridRows = 65535;

// launch(first row, rows) over blocks of rows that fit a grid's y axis.
template <typename F>
hipError_t over_rows(int rows, F launch) {
    for (int r = 0; r < rows; r += kGridRows) {
        launch(r, rows - r < kGridRows ? rows - r : kGridRows);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

size_t up(size_t v, size_t to) { return (v + to - 1) / to * to; }

// Carves 256-byte aligned pieces off the workspace; with base NULL it only counts.
struct Carver {
    char *base;
    size_t used = 0;
    void *take(size_t bytes) {
        void *p = base == nullptr ? nullptr : base + used;
        used += up(bytes, 256);
        return p;
    }
};

// Columns of a piece: about 64 Mi logits, a multiple of 256, at least 256.
int piece_cols(int M, int N) {
    const long fit = (1L << 26) / (M > 0 ? M : 1) / 256 * 256;
    const long all = (long)up((size_t)N, 256);
    const long c = fit < 256 ? 256 : fit;
    return (int)(c < all ? c : all);
}

constexpr int kRowBlock = 8192;  // rows whose logits are held at once in the forward pass

struct ForwardPlan {
    int rows, cols;
    float *Z;
    RowState *state;
    size_t bytes;
    ForwardPlan(int M, int N, void *ws) {
        rows = M < kRowBlock ? M : kRowBlock;
        cols = piece_cols(rows, N);
        Carver c{(char *)ws};
        Z = (float *)c.take((size_t)rows * cols * 4);
        state = (RowState *)c.take((size_t)rows * sizeof(RowState));
        bytes = c.used;
    }
};

struct GradPlan {
    int cols, ldm;
    float *scale, *Z, *dX, *dW;
    RowGrad *rows;
    void *Xm, *dZ;
    size_t bytes;
    GradPlan(int dtype, int M, int N, int K, void *ws) {
        const bool h16 = dtype != kF32;
        const size_t es = h16 ? 2 : 4;
        cols = piece_cols(M, N);
        ldm = (int)up((size_t)(K > 0 ? K : 1), 16 / es);
        Carver c{(char *)ws};
        scale = (float *)c.take(8);
        rows = (RowGrad *)c.take((size_t)M * sizeof(RowGrad));
        Xm = c.take((size_t)M * ldm * es);
        Z = (float *)c.take((size_t)M * cols * 4);
        dZ = h16 ? c.take((size_t)M * cols * 2) : Z;
        dX = h16 ? (float *)c.take((size_t)M * K * 4) : nullptr;
        dW = h16 ? (float *)c.take((size_t)cols * K * 4) : nullptr;
        bytes = c.used;
    }
};

bool valid_shape(int dtype, unsigned flags, int M, int N, int K) {
    if (dtype < kF32 || dtype > kBF16 || (flags & ~(unsigned)GEMM355_TRANS_B)) return false;
    if (M < 0 || N < 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim) return false;
    return N >= 1 || M == 0;
}

bool valid_operands(unsigned flags, int M, int N, int K, const void *X, int ldx, const void *W, int ldw,
                    const int64_t *labels) {
    const int w = flags & GEMM355_TRANS_B ? K : N;
    if (ldx < (K > 1 ? K : 1) || ldw < (w > 1 ? w : 1)) return false;
    if (M > 0 && (labels == nullptr || (K > 0 && (X == nullptr || W == nullptr)))) return false;
    return true;
}

const char *at(const void *p, size_t elem, size_t es) { return (const char *)p + elem * es; }
char *at(void *p, size_t elem, size_t es) { return (char *)p + elem * es; }

// The piece of op(W) that starts at class v0 (its first row with TRANS_B, else column).
size_t w_offset(unsigned flags, int v0, int ldw) {
    return flags & GEMM355_TRANS_B ? (size_t)v0 * ldw : (size_t)v0;
}

gemm355_status status_of(hipError_t e) { return e == hipSuccess ? GEMM355_OK : GEMM355_ERR_LAUNCH; }

gemm355_status forward(int dtype, unsigned flags, int M, int N, int K, const void *X, int ldx, const void *W,
                       int ldw, const int64_t *labels, int64_t ignore, float *loss, float *lse, void *ws,
                       hipStream_t s) {
    const ForwardPlan p(M, N, ws);
    const size_t es = dtype == kF32 ? 4 : 2;
    for (int r0 = 0; r0 < M; r0 += p.rows) {
        const int rows = M - r0 < p.rows ? M - r0 : p.rows;
        for (int v0 = 0; v0 < N; v0 += p.cols) {
            const int nc = N - v0 < p.cols ? N - v0 : p.cols;
            const gemm355_status st =
                gemm355_gemm_ex(GEMM355_VARIANT_AUTO, dtype, flags, rows, nc, K, at(X, (size_t)r0 * ldx, es), ldx,
                                at(W, w_offset(flags, v0, ldw), es), ldw, p.Z, p.cols, s);
            if (st != GEMM355_OK) return st;
            hipLaunchKernelGGL(xent_rows_kernel, dim3(rows), dim3(256), 0, s, nc, v0, N, p.Z, p.cols,
                               labels + r0, ignore, p.state, loss ? loss + r0 : nullptr, lse ? lse + r0 : nullptr);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return status_of(e);
        }
    }
    return GEMM355_OK;
}

// The rows' kernels of the gradient for one storage type.
struct GradCall {
    int dtype;
    unsigned flags;
    int M, N, K;
    const void *X;
    int ldx;
    const void *W;
    int ldw;
    const int64_t *labels;
    int64_t ignore;
    const float *lse, *dloss;
    void *dX;
    int lddx;
    void *dW;
    int lddw;
    hipStream_t s;
};

hipError_t prep(const GradCall &a, const GradPlan &p) {
    const dim3 grid(a.M < 1024 ? a.M : 1024);
    if (a.dtype == kF32)
        hipLaunchKernelGGL((xent_prep_kernel<float>), grid, dim3(256), 0, a.s, a.M, a.N, a.K, (const float *)a.X,
                           a.ldx, a.labels, a.ignore, a.lse, a.dloss, 0, p.scale, p.rows, (float *)p.Xm, p.ldm);
    else
        hipLaunchKernelGGL((xent_prep_kernel<uint16_t>), grid, dim3(256), 0, a.s, a.M, a.N, a.K,
                           (const uint16_t *)a.X, a.ldx, a.labels, a.ignore, a.lse, a.dloss,
                           a.dtype == kF16 ? 1 : 0, p.scale, p.rows, (uint16_t *)p.Xm, p.ldm);
    return hipGetLastError();
}

hipError_t piece_dz(const GradCall &a, const GradPlan &p, int v0, int nc) {
    return over_rows(a.M, [&](int r, int n) {
        const dim3 grid(cdiv(nc, 1024), n);
        const float *Z = p.Z + (size_t)r * p.cols;
        if (a.dtype == kF32)
            hipLaunchKernelGGL((xent_dz_kernel<float>), grid, dim3(256), 0, a.s, nc, v0, Z, p.cols, p.rows + r,
                               (void *)Z, p.cols);
        else if (a.dtype == kF16)
            hipLaunchKernelGGL((xent_dz_kernel<f16_t>), grid, dim3(256), 0, a.s, nc, v0, Z, p.cols, p.rows + r,
                               at(p.dZ, (size_t)r * p.cols, 2), p.cols);
        else
            hipLaunchKernelGGL((xent_dz_kernel<bf16_t>), grid, dim3(256), 0, a.s, nc, v0, Z, p.cols, p.rows + r,
                               at(p.dZ, (size_t)r * p.cols, 2), p.cols);
    });
}

hipError_t round16(const GradCall &a, const GradPlan &p, int rows, int cols, const float *acc, int lda, void *out,
                   int ldo) {
    return over_rows(rows, [&](int r, int n) {
        const dim3 grid(cdiv(cols, 1024), n);
        if (a.dtype == kF16)
            hipLaunchKernelGGL((xent_round_kernel<f16_t>), grid, dim3(256), 0, a.s, cols, acc + (size_t)r * lda, lda,
                               p.scale, (uint16_t *)out + (size_t)r * ldo, ldo);
        else
            hipLaunchKernelGGL((xent_round_kernel<bf16_t>), grid, dim3(256), 0, a.s, cols, acc + (size_t)r * lda, lda,
                               p.scale, (uint16_t *)out + (size_t)r * ldo, ldo);
    });
}

gemm355_status gradient(const GradCall &a, void *ws) {
    const GradPlan p(a.dtype, a.M, a.N, a.K, ws);
    const bool h16 = a.dtype != kF32, tb = a.flags & GEMM355_TRANS_B;
    const size_t es = h16 ? 2 : 4;
    hipError_t e = prep(a, p);
    if (e != hipSuccess) return status_of(e);
    float *dx = h16 ? p.dX : (float *)a.dX;
    const int lddx = h16 ? a.K : a.lddx;
    for (int v0 = 0; v0 < a.N; v0 += p.cols) {
        const int nc = a.N - v0 < p.cols ? a.N - v0 : p.cols;
        const char *w = at(a.W, w_offset(a.flags, v0, a.ldw), es);
        gemm355_status st = gemm355_gemm_ex(GEMM355_VARIANT_AUTO, a.dtype, a.flags, a.M, nc, a.K, p.Xm, p.ldm, w,
                                            a.ldw, p.Z, p.cols, a.s);
        if (st != GEMM355_OK) return st;
        e = piece_dz(a, p, v0, nc);
        if (e != hipSuccess) return status_of(e);
        if (a.dX != nullptr) {
            st = gemm355_gemm_ex(GEMM355_VARIANT_AUTO, a.dtype,
                                 (tb ? 0u : (unsigned)GEMM355_TRANS_B) | (v0 > 0 ? (unsigned)GEMM355_ACCUMULATE : 0u),
                                 a.M, a.K, nc, p.dZ, p.cols, w, a.ldw, dx, lddx, a.s);
            if (st != GEMM355_OK) return st;
        }
        if (a.dW != nullptr) {
            // the piece's rows (TRANS_B) or columns of dW
            const int rows = tb ? nc : a.K, cols = tb ? a.K : nc;
            char *dw = at(a.dW, w_offset(a.flags, v0, a.lddw), es);
            float *out = h16 ? p.dW : (float *)dw;
            const int ldo = h16 ? cols : a.lddw;
            st = tb ? gemm355_gemm_ex(GEMM355_VARIANT_AUTO, a.dtype, GEMM355_TRANS_A, rows, cols, a.M, p.dZ, p.cols,
                                      p.Xm, p.ldm, out, ldo, a.s)
                    : gemm355_gemm_ex(GEMM355_VARIANT_AUTO, a.dtype, GEMM355_TRANS_A, rows, cols, a.M, p.Xm, p.ldm,
                                      p.dZ, p.cols, out, ldo, a.s);
            if (st != GEMM355_OK) return st;
            if (h16) {
                e = round16(a, p, rows, cols, out, ldo, dw, a.lddw);
                if (e != hipSuccess) return status_of(e);
            }
        }
    }
    if (h16 && a.dX != nullptr) return status_of(round16(a, p, a.M, a.K, p.dX, a.K, a.dX, a.lddx));
    return GEMM355_OK;
}

}  // namespace

}  // namespace g355

using namespace g355;

extern "C" {

size_t gemm355_xent_workspace(int dtype, unsigned flags, int M, int N, int K) {
    if (!valid_shape(dtype, flags, M, N, K) || M == 0) return 0;
    return ForwardPlan(M, N, nullptr).bytes;
}

gemm355_status gemm355_xent(int dtype, unsigned flags, int M, int N, int K, const void *X, int ldx, const void *W,
                            int ldw, const int64_t *labels, int64_t ignore, float *loss, float *lse,
                            void *workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!valid_shape(dtype, flags, M, N, K) || !valid_operands(flags, M, N, K, X, ldx, W, ldw, labels))
        return GEMM355_ERR_INVALID_ARG;
    if (M == 0 || (loss == nullptr && lse == nullptr)) return GEMM355_OK;
    const size_t need = gemm355_xent_workspace(dtype, flags, M, N, K);
    if (workspace_bytes < need || (need > 0 && workspace == nullptr) || (uintptr_t)workspace % 16 != 0)
        return GEMM355_ERR_INVALID_ARG;
    const size_t es = dtype == kF32 ? 4 : 2;
    const bool tb = flags & GEMM355_TRANS_B;
    const Span in[3] = {{X, matrix_bytes(M, K, ldx, es)},
                        {W, tb ? matrix_bytes(N, K, ldw, es) : matrix_bytes(K, N, ldw, es)},
                        {labels, (size_t)M * 8}};
    const Span out[3] = {{loss, loss ? (size_t)M * 4 : 0}, {lse, lse ? (size_t)M * 4 : 0}, {workspace, need}};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < 3; ++j)
            if (out[i].meets(in[j])) return GEMM355_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (out[i].meets(out[j])) return GEMM355_ERR_INVALID_ARG;
    }
    if (!current_device_is_gfx950()) return GEMM355_ERR_DEVICE;
    return forward(dtype, flags, M, N, K, X, ldx, W, ldw, labels, ignore, loss, lse, workspace, stream);
}

size_t gemm355_xent_grad_workspace(int dtype, unsigned flags, int M, int N, int K) {
    if (!valid_shape(dtype, flags, M, N, K) || M == 0) return 0;
    return GradPlan(dtype, M, N, K, nullptr).bytes;
}

gemm355_status gemm355_xent_grad(int dtype, unsigned flags, int M, int N, int K, const void *X, int ldx,
                                 const void *W, int ldw, const int64_t *labels, int64_t ignore, const float *lse,
                                 const float *dloss, void *dX, int lddx, void *dW, int lddw, void *workspace,
                                 size_t workspace_bytes, hipStream_t stream) {
    if (!valid_shape(dtype, flags, M, N, K) || !valid_operands(flags, M, N, K, X, ldx, W, ldw, labels))
        return GEMM355_ERR_INVALID_ARG;
    const bool tb = flags & GEMM355_TRANS_B;
    const int w = tb ? K : N;
    if ((dX != nullptr && lddx < (K > 1 ? K : 1)) || (dW != nullptr && lddw < (w > 1 ? w : 1)))
        return GEMM355_ERR_INVALID_ARG;
    if (M > 0 && (lse == nullptr || dloss == nullptr)) return GEMM355_ERR_INVALID_ARG;
    if (K == 0 || N == 0 || (dX == nullptr && dW == nullptr)) return GEMM355_OK;
    const size_t need = gemm355_xent_grad_workspace(dtype, flags, M, N, K);
    if (workspace_bytes < need || (need > 0 && workspace == nullptr) || (uintptr_t)workspace % 16 != 0)
        return GEMM355_ERR_INVALID_ARG;
    const size_t es = dtype == kF32 ? 4 : 2;
    const int wr = tb ? N : K, wc = tb ? K : N;
    const Span in[5] = {{X, matrix_bytes(M, K, ldx, es)},
                        {W, matrix_bytes(wr, wc, ldw, es)},
                        {labels, (size_t)M * 8},
                        {lse, (size_t)M * 4},
                        {dloss, (size_t)M * 4}};
    const Span out[3] = {{dX, dX ? matrix_bytes(M, K, lddx, es) : 0},
                         {dW, dW ? matrix_bytes(wr, wc, lddw, es) : 0},
                         {workspace, need}};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < 5; ++j)
            if (out[i].meets(in[j])) return GEMM355_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (out[i].meets(out[j])) return GEMM355_ERR_INVALID_ARG;
    }
    if (M == 0 && dW == nullptr) return GEMM355_OK;
    if (!current_device_is_gfx950()) return GEMM355_ERR_DEVICE;
    if (M == 0)
        return status_of(over_rows(wr, [&](int r, int n) {
            const dim3 grid(cdiv(wc, 256), n);
            if (dtype == kF32)
                hipLaunchKernelGGL((zero_matrix_kernel<float>), grid, dim3(256), 0, stream, wc,
                                   (float *)dW + (size_t)r * lddw, lddw);
            else
                hipLaunchKernelGGL((zero_matrix_kernel<uint16_t>), grid, dim3(256), 0, stream, wc,
                                   (uint16_t *)dW + (size_t)r * lddw, lddw);
        }));
    const GradCall a{dtype, flags, M, N, K, X, ldx, W, ldw, labels, ignore, lse, dloss, dX, lddx, dW, lddw, stream};
    return gradient(a, workspace);
}

}  // extern "C"
