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
// Two paths.  16-bit types with 256 classes or more run on the direct-to-LDS tiles with
// epilogues of their own (xent_dma.hpp): the forward pass writes one (maximum, sum) pair per
// row and 32 to 128 classes, the backward pass dZ of a piece of the vocabulary (512 MiB at
// most) and two products that read it; what those tiles cannot load where it lies (rows not
// 16-byte aligned, K not a multiple of 8) is copied to aligned rows first, W a piece of 128
// MiB at a time.  Everything else (binary32; few classes) writes a piece of binary32 logits
// with the library's GEMM kernels and reads it back.
//
// This file: the rows' kernels, the plans that lay out a call's workspace, and the entry
// points.  Every kernel here is bound by memory; all of them together take 1-2 % of a large
// call and half of the smallest ones (4-5 us each, launch included).
#include <algorithm>

#include "../../include/gemm355_softmax.h"
#include "common.hpp"
#include "launch.hpp"
#include "wave_reduce.hpp"
#include "xent.hpp"

namespace g355 {

namespace {

constexpr float kNegInf = -__builtin_huge_valf();
constexpr int kMaxDim = (1 << 30) - 1;

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

constexpr int kChunk = 4096;  // columns of a row that one workgroup takes the statistics of

// The statistics of columns [4096 b, + 4096) of row r of a piece Z, workgroup (b, r), to
// part[b * ldp + r]; zl[r] = the label's logit where it is one of them (the piece starts at
// class v0).  Bound by reading the logits: 1000 x 32000 28.9 us, 4.4 TB/s.
__global__ __launch_bounds__(256) void xent_chunk_kernel(int nc, int v0, const float *__restrict__ Z, int ldz,
                                                         const int64_t *__restrict__ labels, float2 *part, int ldp,
                                                         float *zl) {
    __shared__ float sm[4], sl[4];
    const int row = blockIdx.y, wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    const int c0 = blockIdx.x * kChunk, c1 = min(c0 + kChunk, nc);
    const float *z = Z + (size_t)row * ldz;
    float m = kNegInf, l = 0.0f;
    for (int base = c0; base < c1; base += 2048) {
        float v[8], cm = kNegInf;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int c = base + 256 * u + (int)threadIdx.x;
            v[u] = c < c1 ? z[c] : kNegInf;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) cm = fmaxf(cm, v[u]);
        if (cm > m) {
            l *= expf(m - cm);
            m = cm;
        }
        const float shift = m == kNegInf ? 0.0f : m;
#pragma unroll
        for (int u = 0; u < 8; ++u) l += expf(v[u] - shift);
    }
    wave_allreduce2(m, l, MergePair{});
    if (lane == 0) {
        sm[wave] = m;
        sl[wave] = l;
    }
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int w = 1; w < 4; ++w) merge_pair(m, l, sm[w], sl[w]);
    part[(size_t)blockIdx.x * ldp + row] = make_float2(m, l);
    const int64_t at = labels[row] - v0;
    if (at >= c0 && at < c1) zl[row] = z[at];
}

// The statistics of the tiles or chunks: `blocks` pairs per row (part[block * ldp + row]) merged,
// and the row's results written.  A workgroup takes R rows, 1024 / R threads a row: each
// merges every (1024 / R)-th block, then the threads' pairs are merged in halves.  8192 rows of
// 1024 pairs 13.4 us (67 MB, 5 TB/s); 16 rows of 1000 with R = 4 3.9 us, mostly the launch.
template <int R>
__global__ __launch_bounds__(1024) void xent_merge_kernel(int M, int N, int blocks, const float2 *__restrict__ part,
                                                          int ldp, const float *__restrict__ zl,
                                                          const int64_t *__restrict__ labels, int64_t ignore,
                                                          float *loss, float *lse) {
    constexpr int kPer = 1024 / R;
    __shared__ float sm[1024], sl[1024];
    const int t = threadIdx.x, row = blockIdx.x * R + t % R;
    float m = kNegInf, l = 0.0f;
    if (row < M)
        for (int b = t / R; b < blocks; b += 4 * kPer) {
            float2 v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                v[u] = b + u * kPer < blocks ? part[(size_t)(b + u * kPer) * ldp + row] : make_float2(kNegInf, 0.0f);
#pragma unroll
            for (int u = 0; u < 4; ++u) merge_pair(m, l, v[u].x, v[u].y);
        }
    sm[t] = m;
    sl[t] = l;
#pragma unroll
    for (int h = 512; h >= R; h /= 2) {
        __syncthreads();
        if (t < h) {
            merge_pair(m, l, sm[t + h], sl[t + h]);
            sm[t] = m;
            sl[t] = l;
        }
    }
    if (t >= R || row >= M) return;
    const int64_t label = labels[row];
    finish_row(row, m, l, label >= 0 && label < N ? zl[row] : 0.0f, label, ignore, N, loss, lse);
}

// src (rows x cols, row stride lds, any alignment) copied to aligned rows of ldd elements (a
// multiple of 8), zeros past the last column and in the rows from `rows` to `all`.  Grid: (16-
// byte chunks of a row / 256, all).
__global__ __launch_bounds__(256) void xent_copy_kernel(int rows, int cols, const uint16_t *__restrict__ src, int lds,
                                                        uint16_t *dst, int ldd) {
    const int c = 8 * (blockIdx.x * 256 + (int)threadIdx.x), r = blockIdx.y;
    if (c >= ldd) return;
    const uint16_t *x = src + (size_t)r * lds + c;
    u16x8 v = {0, 0, 0, 0, 0, 0, 0, 0};
    if (r < rows && c + 8 <= cols) v = *(const u16x8_ua *)x;
    else if (r < rows)
        for (int i = 0; i < 8 && c + i < cols; ++i) v[i] = x[i];
    *(u16x8 *)(dst + (size_t)r * ldd + c) = v;
}

// Before the gradient's pieces: scale[0] = S and scale[1] = 1 / S (S = 1 unless `rescale`:
// then the power of two that puts the largest |dloss| in [2^13, 2^14), from 2^-100 to
// 2^100), the rows' RowGrad, and Xm = X with the rows without a label set to zero (their
// products with a zero row of dZ would not be zero where X holds an infinity or NaN).
// Every workgroup finds the same maximum over all rows, then does its share of the rows.
// Rows from M to Mp are rows without a label; with `again`, rows from `again` on are the
// first ones' X again.  512 x 1024 5.0 us, the launch and two reads that wait for each other.
template <typename E>
__global__ __launch_bounds__(256) void xent_prep_kernel(int M, int Mp, int again, int N, int K, const E *__restrict__ X, int ldx,
                                                        const int64_t *__restrict__ labels, int64_t ignore,
                                                        const float *__restrict__ lse,
                                                        const float *__restrict__ dloss, int rescale,
                                                        float *scale, RowGrad *rows, E *Xm, int ldm, int vec) {
    __shared__ float sm[4];
    float S = 1.0f;
    if (rescale) {
        float top = 0.0f;
        for (int r0 = threadIdx.x; r0 < M; r0 += 8 * 256) {   // eight rows' loads in flight
            int64_t y[8];
            float g[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int r = min(r0 + 256 * u, M - 1);   // the last row again: the same maximum
                y[u] = labels[r];
                g[u] = dloss[r];
            }
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (y[u] != ignore && y[u] >= 0 && y[u] < N) top = fmaxf(top, fabsf(g[u]));
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
    for (int r = blockIdx.x; r < Mp; r += gridDim.x) {
        const int from = again > 0 && r >= again ? r - again : r;
        const int64_t y = from < M ? labels[from] : -1;
        const bool live = from < M && y != ignore && y >= 0 && y < N;
        if (threadIdx.x == 0)
            rows[r] = RowGrad{live ? lse[from] : 0.0f, live ? dloss[from] * S : 0.0f, live ? (int)y : -1, 0};
        const E *x = X + (size_t)from * ldx;
        E *o = Xm + (size_t)r * ldm;
        if (vec) {   // rows of X and Xm 16-byte aligned, K a whole number of 16-byte chunks
            constexpr int kV = 16 / sizeof(E);
            for (int c = kV * threadIdx.x; c < ldm; c += kV * 256) {
                u32x4 v = {0, 0, 0, 0};
                if (live && c < K) v = *(const u32x4 *)(x + c);
                *(u32x4 *)(o + c) = v;
            }
        } else {
            for (int c = threadIdx.x; c < ldm; c += 256) o[c] = live && c < K ? x[c] : E{};
        }
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

// out = scale[1] * (the sum of `splits` partial sums, `stride` apart, and with `other` of those
// that many elements further on), rounded to the 16-bit type; four columns per thread (VEC:
// loaded in one access; wide: stored in one).  Grid: (columns / 1024, rows).  8192 x 4096 from
// one sum 34 us, 5.9 TB/s; 512 x 1024 from 16 6.6 us.
template <typename T, bool VEC>
__global__ __launch_bounds__(256) void xent_round_kernel(int cols, const float *__restrict__ acc, int lda,
                                                         int splits, size_t stride, size_t other,
                                                         const float *__restrict__ scale, uint16_t *out,
                                                         int ldo, int wide) {
    const int c = blockIdx.x * 1024 + 4 * (int)threadIdx.x;
    if (c >= cols) return;
    const float f = scale[1];
    const float *a = acc + (size_t)blockIdx.y * lda + c;
    uint16_t *o = out + (size_t)blockIdx.y * ldo + c;
    if constexpr (VEC) {   // acc's rows hold cols rounded up to 4
        floatx4 v = *(const floatx4 *)a;
        int i = 1;
        for (; i + 8 <= splits; i += 8) {   // eight loads in flight, added in order
            floatx4 w[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) w[u] = *(const floatx4 *)(a + (i + u) * stride);
#pragma unroll
            for (int u = 0; u < 8; ++u) v += w[u];
        }
        for (; i < splits; ++i) v += *(const floatx4 *)(a + i * stride);
        if (other > 0) {   // the remainders' sums
            floatx4 w = *(const floatx4 *)(a + other);
#pragma unroll 4
            for (int k = 1; k < splits; ++k) w += *(const floatx4 *)(a + other + k * stride);
            v += w;
        }
        if (wide && c + 4 <= cols)
            *(uint2 *)o = make_uint2((uint32_t)to_bits(f * v[0], T{}) | (uint32_t)to_bits(f * v[1], T{}) << 16,
                                     (uint32_t)to_bits(f * v[2], T{}) | (uint32_t)to_bits(f * v[3], T{}) << 16);
        else
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (c + u < cols) o[u] = to_bits(f * v[u], T{});
    } else {               // one product's sums
        for (int u = 0; u < 4 && c + u < cols; ++u) o[u] = to_bits(f * a[u], T{});
    }
}

// out = the sum of n partial sums, `stride` apart.  Grid: (columns / 256, rows).
__global__ __launch_bounds__(256) void xent_sum_kernel(int cols, const float *__restrict__ part, int n, size_t stride,
                                                       float *out, int ldo) {
    const int c = blockIdx.x * 256 + (int)threadIdx.x;
    if (c >= cols) return;
    const float *p = part + (size_t)blockIdx.y * cols + c;
    float v = p[0];
#pragma unroll 8
    for (int i = 1; i < n; ++i) v += p[i * stride];
    out[(size_t)blockIdx.y * ldo + c] = v;
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

// The ranges of `step` terms that a binary32 product of M x cols is summed over: four
// workgroups a CU where there are fewer than 512 tiles of 64 x 64, each of 256 terms or more.
// One range: an ordinary product.  Logits of 5 x 11952 x 3973 (187 tiles) as one product 134
// us, in 5 ranges 80 with their sum; of 8 x 91440 x 1344 (1429 tiles) the whole loss 153 as
// one, 185 in 2; of 863 x 1152 x 1728 (252 tiles) 55 in 4, 61 in 7.  With dX, from the logits
// on: 300 x 20000 x 4096 (320 tiles) 1058 as one, 941 in 3; 512 x 8000 x 2048 267 and 273.
struct F32Ranges {
    int count = 1, step = 0;
    F32Ranges(int M, int cols, int n) {
        const long tiles = (long)cdiv(M, 64) * cdiv(cols, 64);
        if (tiles >= 512 || n < 512) return;
        step = (int)up((size_t)std::max(cdiv(n, (int)(1024 / tiles)), 256), 32);
        count = cdiv(n, step);
    }
    size_t bytes(int M, int cols) const { return count > 1 ? (size_t)count * M * cols * 4 : 0; }
};

constexpr int kRowBlock = 8192;  // rows whose logits are held at once in the forward pass

struct ForwardPlan {
    int rows, cols, blocks, ldm;
    F32Ranges ranges{1, 1, 0};   // of the logits' sums
    float *Z, *zl, *sums;
    float2 *part;
    void *Xm;
    size_t bytes;
    ForwardPlan(int dtype, int M, int N, int K, void *ws) {
        const size_t es = dtype == kF32 ? 4 : 2;
        ldm = (int)up((size_t)(K > 0 ? K : 1), 16 / es);
        rows = M < kRowBlock ? M : kRowBlock;
        cols = piece_cols(rows, N);
        blocks = 0;
        for (int v0 = 0; v0 < N; v0 += cols) blocks += cdiv(N - v0 < cols ? N - v0 : cols, kChunk);
        Carver c{(char *)ws};
        Z = (float *)c.take((size_t)rows * cols * 4);
        part = (float2 *)c.take((size_t)blocks * rows * sizeof(float2));
        zl = (float *)c.take((size_t)rows * 4);
        Xm = c.take((size_t)rows * ldm * es);
        const int nc = cols < N ? cols : N;
        if (dtype == kF32) ranges = F32Ranges(rows, nc, K);
        sums = (float *)c.take(ranges.bytes(rows, nc));
        bytes = c.used;
    }
};

struct GradPlan {
    int Mp, cols, ldm;  // Mp: rows, with those of zeros that make dW's sum whole k-steps
    F32Ranges zr{1, 1, 0}, dxr{1, 1, 0};   // of the logits' and dX's sums
    float *scale, *Z, *sums, *dX, *dW;
    RowGrad *rows;
    void *Xm, *dZ;
    size_t bytes;
    GradPlan(int dtype, int M, int N, int K, void *ws) {
        const bool h16 = dtype != kF32;
        const size_t es = h16 ? 2 : 4;
        // binary32: dW over 294 rows of 11483 x 2944 258 us, over 320 238; a few rows gain
        // nothing from it and pay for writing more logits (5 x 11952 x 3973 270 us, 32 rows 310)
        Mp = h16 || M <= 64 ? M : (int)up((size_t)M, 32);
        cols = piece_cols(Mp, N);
        ldm = (int)up((size_t)(K > 0 ? K : 1), 16 / es);
        const int nc = cols < N ? cols : N;
        if (!h16) {
            zr = F32Ranges(Mp, nc, K);
            dxr = F32Ranges(M, K, nc);
        }
        Carver c{(char *)ws};
        scale = (float *)c.take(8);
        rows = (RowGrad *)c.take((size_t)Mp * sizeof(RowGrad));
        Xm = c.take((size_t)Mp * ldm * es);
        Z = (float *)c.take((size_t)Mp * cols * 4);
        dZ = h16 ? c.take((size_t)Mp * cols * 2) : Z;
        sums = (float *)c.take(zr.bytes(Mp, nc));
        dX = (float *)c.take(h16 ? (size_t)M * K * 4 : dxr.bytes(M, K));
        dW = h16 ? (float *)c.take((size_t)cols * K * 4) : nullptr;
        bytes = c.used;
    }
};

// Whether the matrix-core tiles with fused epilogues take these shapes: 16-bit types, as many
// classes as a product over them needs for a ring trip and more, and 256 rows of K within the
// range of a tile's offsets.
bool fused_shape(int dtype, int N, int K) { return dtype != kF32 && N >= 256 && K <= 1 << 20; }

// The hidden size the tiles work with: whole 16-byte chunks, a ring trip at least.
int padded_hidden(int K) { return (int)up((size_t)(K < 128 ? 128 : K), 8); }

// Byte offsets of `rows` rows of stride ld (and the ring trip past them) below 2^31.
bool offsets_fit(long rows, long ld) { return (rows + 256) * ld * 2 < (1L << 31); }

// Whether the tiles can load W where it lies: rows of whole chunks, 16-byte aligned, offsets
// within a tile (TRANS_B) or of all K rows in range.  Else each piece of it is copied to the
// workspace first.
bool weights_load(unsigned flags, int N, int K, const void *W, int ldw) {
    return K == padded_hidden(K) && (flags & GEMM355_TRANS_B || N % 8 == 0) && rows_aligned16(W, ldw, 2) &&
           offsets_fit(flags & GEMM355_TRANS_B ? 256 : K, ldw);
}

// The time of M x N logits in one kind of tile, in rounds of 256 x 256 tiles (one per CU):
// rounds of resident tiles times what a round takes, measured at K = 2048 (bf16, us: 256 x
// 256 46, 128 x 256 33, 64 x 256 29 with one per CU and 60 with two, 64 x 128 12, 64 x 64 8
// and 14, 128 x 128 17 and 30).  Few rows are bound by reading W, for which many small tiles
// do best: 16 x 32000 x 2048 51 / 41 / 38 / 26 / 26 us in this order, 256 x 8000 x 2048 48 /
// 36 / 32 / 17 / 21, 256 x 32000 x 2048 54 / 43 / 44 / 52 / 59, 512 x 32000 x 1024 37 / 45 /
// 47.  128 x 128 two per CU has neither the largest tile's rate nor its last rows' waste: 276
// x 104940 x 640 72 against 78 us in 128 x 256 and 92 in 256 x 256, 4096 x 32000 x 2048 474
// against 392.
double head_cost(int tile, int M, int N) {
    constexpr double kOne[kHeadTiles] = {1.0, 0.72, 0.63, 0.27, 0.17, 0.36};
    constexpr double kTwo[kHeadTiles] = {0, 0, 1.2, 0, 0.3, 0.6};
    const long tiles = (long)cdiv(M, kHeadRows[tile]) * cdiv(N, kHeadCols[tile]);
    if (kTwo[tile] > 0 && tiles > 256) return (double)((tiles + 511) / 512) * kTwo[tile];
    return (double)((tiles + 255) / 256) * kOne[tile];
}

int head_tile(int M, int N, int K) {
    int best = kHead256;
    for (int t = kHead128; t < kHeadTiles; ++t)
        if (K >= kHeadTrip[t] && head_cost(t, M, N) < head_cost(best, M, N)) best = t;
    return best;
}

// Columns [v0, v0 + cols) of a product in one kind of tile.
struct Section { int v0, cols, tile; };

// The columns of M x N logits in one section, or, where that leaves a last round of few
// tiles, the whole rounds and the rest in the tiles that suit it (2047 x 50003 x 2048: 1568
// tiles of 256 x 256 are 6 rounds and 32 tiles, 360 us; 6 rounds and 224 tiles of 64 x 128
// 338).
int head_sections(int M, int N, int K, Section out[2]) {
    const int tile = head_tile(M, N, K);
    out[0] = {0, N, tile};
    const long down = cdiv(M, kHeadRows[tile]), rounds = down * cdiv(N, kHeadCols[tile]) / 256;
    const int whole = (int)(rounds * 256 / down) * kHeadCols[tile];
    if (tile > kHead128 || whole == 0 || whole >= N) return 1;
    const int rest = head_tile(M, N - whole, K);
    if (head_cost(tile, M, whole) + head_cost(rest, M, N - whole) > 0.97 * head_cost(tile, M, N)) return 1;
    out[0].cols = whole;
    out[1] = {whole, N - whole, rest};
    return 2;
}

// dX's product: its 16-bit result is a sum over ranges of classes, whose partial sums grow
// with the number of ranges that fill the CUs, so fewer rows take smaller tiles (M = 512, K
// = 1024 in 16 ranges of 128 x 256 tiles against 32 of 256 x 256: 80 against 86 us with the
// dZ before it; 1024 x 2048 the same, 2047 x 2048 479 against 436).
int dx_tile(int M) { return M <= 512 ? kHead128 : kHead256; }

// dW's product, `across` tiles of 256 over the hidden size: 128 x 128 tiles two per CU where
// the sum over the rows is short and the stores of one tile hide behind the other's sum (512
// x 32000 x 1024 81 against 85 us with the dZ before it, 16 x 32000 x 2048 75 against 85,
// 1024 x 32000 x 2048 the same, 2047 457 against 489 the other way), and for the rest of a
// longer one where whole rounds of 256 x 256 tiles leave less than half a round.
int dw_sections(int M, int N, int K, Section out[2]) {
    const long across = cdiv(K, 256), tiles = across * cdiv(N, 256);
    out[0] = {0, N, M <= 1024 || tiles < 128 ? 128 : 256};
    const int whole = (int)(tiles / 256 * 256 / across) * 256;
    if (out[0].tile == 128 || whole == 0 || whole >= N || 2 * (tiles - across * (whole / 256)) > 256) return 1;
    out[0].cols = whole;
    out[1] = {whole, N - whole, 128};
    return 2;
}

constexpr int kStatRows = 32768;  // rows whose block statistics are held at once

int stat_blocks(const Section &c) {
    return cdiv(c.cols, kHeadCols[c.tile]) * (kHeadCols[c.tile] / kStatCols[c.tile]);
}

constexpr long kCopyBytes = 1L << 27;  // of W at once, where it has to be copied

// Columns of a piece: a multiple of 256, at most `fit` (but at least 256), the last piece not
// below 256 either unless it is the only one.
int even_pieces(int N, long fit) {
    fit = fit < 256 ? 256 : fit / 256 * 256;
    const int pieces = (int)((N + fit - 1) / fit);
    int cols = (int)up((size_t)cdiv(N, pieces), 256);
    while (cols < N && N % cols != 0 && N % cols < 256) cols += 256;
    return cols;
}

struct FusedForwardPlan {
    int rows, cols, Kp, ldw;
    float2 *part;
    float *zl;
    uint16_t *Xm, *Wm;
    size_t bytes;
    // `cols` classes at a time, which keep a launch's threads below 2^32, or, where W is copied,
    // the copy to kCopyBytes
    FusedForwardPlan(bool copied, unsigned flags, int M, int N, int K, void *ws) {
        rows = M < kStatRows ? M : kStatRows;
        Kp = padded_hidden(K);
        cols = even_pieces(N, copied ? kCopyBytes / 2 / Kp : 1L << 22);
        ldw = flags & GEMM355_TRANS_B ? Kp : (int)up((size_t)cols, 8);
        // the last rows may take smaller tiles, and so more blocks, than the others
        const int rest = M % rows;
        Carver c{(char *)ws};
        part = (float2 *)c.take(std::max(pairs(rows, N), rest > 0 ? pairs(rest, N) : 0) * sizeof(float2));
        zl = (float *)c.take((size_t)rows * 4);
        Xm = (uint16_t *)c.take((size_t)rows * Kp * 2);
        Wm = (uint16_t *)c.take(copied ? (size_t)(flags & GEMM355_TRANS_B ? cols : Kp) * ldw * 2 : 0);
        bytes = c.used;
    }
    // the (maximum, sum) pairs of n rows
    size_t pairs(int n, int N) const {
        size_t blocks = 0;
        for (int v0 = 0; v0 < N; v0 += cols) {
            Section part[2];
            const int sections = head_sections(n, N - v0 < cols ? N - v0 : cols, Kp, part);
            for (int i = 0; i < sections; ++i) blocks += stat_blocks(part[i]);
        }
        return blocks * n;
    }
};

// The ranges of K one product is split into: `want` of them at most, each a whole number of
// ring trips and none but a single one shorter than 256.
struct Splits {
    int count, step;
    Splits(int K, int want) {
        if (want > K / 512) want = K / 512;
        if (want < 1) want = 1;
        step = (int)up((size_t)cdiv(K, want), 128);
        while (step < K && K % step != 0 && K % step < 256) step += 128;
        count = cdiv(K, step);
    }
};

constexpr long kDzBytes = 1L << 29;  // dZ of a piece

// Up to this many rows dZ is kept in two parts, the rounded values in rows [0, 64) and what
// the rounding leaves in rows [64, 128), which the products read as rows of their own (X's
// again): dW's needs 128 rows of a ring trip in any case, and with few rows all the products
// are bound by reading W and writing dW.  dX and dW are then off by little more than their own
// rounding, where one part adds as much again.
constexpr int kFewRows = 64;

// Ranges of the rows that dW's product is summed over, 1 for none: with few 128 x 128 tiles
// and many rows, as many as fill the CUs twice (6948 rows, 1175 classes, K = 576: 50 tiles of
// 55 trips each on as many CUs).
int dw_splits(int Mp, int nc, int K) {
    const long tiles = (long)cdiv(nc, 128) * cdiv(K, 128);
    return tiles < 256 ? Splits(Mp, (int)(512 / tiles)).count : 1;
}

struct FusedGradPlan {
    bool few;
    int cols, Mp, Kp, ldw, dx, dx_rows, splits, ldx;
    float *scale, *dX, *dW;
    RowGrad *rows;
    uint16_t *Xm, *dZ, *Wm;
    size_t dx_stride, bytes;
    FusedGradPlan(bool copied, unsigned flags, int M, int N, int K, void *ws) {
        Mp = (int)up((size_t)M, 128);  // whole ring trips of dW's product, zeros past M
        Kp = padded_hidden(K);
        few = M <= kFewRows;
        dx_rows = few ? 2 * kFewRows : M;
        dx = dx_tile(dx_rows);
        long fit = kDzBytes / 2 / Mp;
        if (copied && kCopyBytes / 2 / Kp < fit) fit = kCopyBytes / 2 / Kp;
        cols = even_pieces(N, fit);
        ldw = flags & GEMM355_TRANS_B ? Kp : cols;
        // dX's product: as many ranges of a piece's classes as fill the 256 CUs
        const int nc = cols < N ? cols : N;
        splits = Splits(nc, 256 / (cdiv(dx_rows, kHeadRows[dx]) * cdiv(K, kHeadCols[dx]))).count;
        ldx = (int)up((size_t)K, 4);
        dx_stride = (size_t)dx_rows * ldx;
        Carver c{(char *)ws};
        scale = (float *)c.take(8);
        rows = (RowGrad *)c.take((size_t)Mp * sizeof(RowGrad));
        Xm = (uint16_t *)c.take((size_t)Mp * Kp * 2);
        dZ = (uint16_t *)c.take((size_t)Mp * cols * 2);
        dX = (float *)c.take((size_t)splits * dx_stride * 4);
        Wm = (uint16_t *)c.take(copied ? (size_t)(flags & GEMM355_TRANS_B ? cols : Kp) * ldw * 2 : 0);
        const bool tb = flags & GEMM355_TRANS_B;
        dW = (float *)c.take(std::max(dw_bytes(tb, nc, K), N % cols != 0 ? dw_bytes(tb, N % cols, K) : 0));
        bytes = c.used;
    }
    // dW's partial sums for a piece of nc classes
    size_t dw_bytes(bool tb, int nc, int K) const {
        const int n = dw_splits(Mp, nc, K);
        return n > 1 ? (size_t)n * (tb ? nc : K) * up((size_t)(tb ? K : nc), 4) * 4 : 0;
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

#define G355_TRY(call)                                    \
    do {                                                  \
        const hipError_t try_e = (call);                  \
        if (try_e != hipSuccess) return GEMM355_ERR_LAUNCH; \
    } while (0)

hipError_t merge(int M, int N, int blocks, const float2 *part, int ldp, const float *zl, const int64_t *labels,
                 int64_t ignore, float *loss, float *lse, hipStream_t s) {
    if (M >= 32)
        hipLaunchKernelGGL((xent_merge_kernel<32>), dim3(cdiv(M, 32)), dim3(1024), 0, s, M, N, blocks, part, ldp, zl,
                           labels, ignore, loss, lse);
    else
        hipLaunchKernelGGL((xent_merge_kernel<4>), dim3(cdiv(M, 4)), dim3(1024), 0, s, M, N, blocks, part, ldp, zl,
                           labels, ignore, loss, lse);
    return hipGetLastError();
}

hipError_t copy_rows(int rows, int all, int cols, const void *src, int lds, uint16_t *dst, int ldd, hipStream_t s) {
    return over_rows(all, [&](int r, int n) {
        hipLaunchKernelGGL(xent_copy_kernel, dim3(cdiv(ldd / 8, 256), n), dim3(256), 0, s, rows - r, cols,
                           (const uint16_t *)src + (size_t)r * lds, lds, dst + (size_t)r * ldd, ldd);
    });
}

// The piece of W from class v0 on, nc classes, copied: K x nc or nc x K to aligned rows,
// zeros from K to Kp.
hipError_t copy_weights(unsigned flags, int nc, int K, int Kp, const void *w, int ldw, uint16_t *Wm, int ldm,
                        hipStream_t s) {
    if (flags & GEMM355_TRANS_B) return copy_rows(nc, nc, K, w, ldw, Wm, ldm, s);
    return copy_rows(K, Kp, nc, w, ldw, Wm, ldm, s);
}

gemm355_status sum_ranges(const F32Ranges &ranges, const float *sums, int M, int cols, float *out, int ldo,
                          hipStream_t s) {
    return status_of(over_rows(M, [&](int r, int n) {
        hipLaunchKernelGGL(xent_sum_kernel, dim3(cdiv(cols, 256), n), dim3(256), 0, s, cols, sums + (size_t)r * cols,
                           ranges.count, (size_t)M * cols, out + (size_t)r * ldo, ldo);
    }));
}

gemm355_status forward_fused(int dtype, unsigned flags, int M, int N, int K, const void *X, int ldx, const void *W,
                             int ldw, const int64_t *labels, int64_t ignore, float *loss, float *lse, void *ws,
                             hipStream_t s) {
    const bool copied = !weights_load(flags, N, K, W, ldw), tb = flags & GEMM355_TRANS_B;
    const FusedForwardPlan p(copied, flags, M, N, K, ws);
    const bool copy_x = K != p.Kp || !rows_aligned16(X, ldx, 2) || !offsets_fit(256, ldx);
    for (int r0 = 0; r0 < M; r0 += p.rows) {
        const int rows = M - r0 < p.rows ? M - r0 : p.rows;
        const void *x = at(X, (size_t)r0 * ldx, 2);
        if (copy_x) G355_TRY(copy_rows(rows, rows, K, x, ldx, p.Xm, p.Kp, s));
        float2 *part = p.part;
        int blocks = 0;
        for (int v0 = 0; v0 < N; v0 += p.cols) {
            const int nc = N - v0 < p.cols ? N - v0 : p.cols;
            const void *w = at(W, w_offset(flags, v0, ldw), 2);
            if (copied) G355_TRY(copy_weights(flags, nc, K, p.Kp, w, ldw, p.Wm, p.ldw, s));
            if (copied) w = p.Wm;
            const int lw = copied ? p.ldw : ldw;
            Section sec[2];
            const int n = head_sections(rows, nc, p.Kp, sec);
            for (int i = 0; i < n; ++i) {
                const Section &c = sec[i];
                const HeadArgs h{rows, c.cols, p.Kp, copy_x ? p.Xm : x, copy_x ? p.Kp : ldx,
                                 at(w, w_offset(flags, c.v0, lw), 2), lw, tb};
                G355_TRY(dtype == kF16
                             ? launch_xent_stats_f16(c.tile, h, labels + r0, v0 + c.v0, part, rows, p.zl, s)
                             : launch_xent_stats_bf16(c.tile, h, labels + r0, v0 + c.v0, part, rows, p.zl, s));
                part += (size_t)stat_blocks(c) * rows;
                blocks += stat_blocks(c);
            }
        }
        G355_TRY(merge(rows, N, blocks, p.part, rows, p.zl, labels + r0, ignore, loss ? loss + r0 : nullptr,
                       lse ? lse + r0 : nullptr, s));
    }
    return GEMM355_OK;
}

// The logits of a piece, in ranges of the hidden size or as one product.
gemm355_status piece_logits(int dtype, unsigned flags, const F32Ranges &ranges, float *sums, int M, int nc, int K,
                            const void *X, int ldx, const void *w, int ldw, float *Z, int ldz, hipStream_t s) {
    if (ranges.count == 1)
        return gemm355_gemm_ex(GEMM355_VARIANT_AUTO, dtype, flags, M, nc, K, X, ldx, w, ldw, Z, ldz, s);
    const F32SplitArgs q{M, nc, K, (const float *)X, ldx, (const float *)w, ldw, sums, ranges.step, 0};
    G355_TRY(launch_xent_split_f32(!(flags & GEMM355_TRANS_B), q, s));
    return sum_ranges(ranges, sums, M, nc, Z, ldz, s);
}

gemm355_status forward(int dtype, unsigned flags, int M, int N, int K, const void *X, int ldx, const void *W,
                       int ldw, const int64_t *labels, int64_t ignore, float *loss, float *lse, void *ws,
                       hipStream_t s) {
    const ForwardPlan p(dtype, M, N, K, ws);
    const size_t es = dtype == kF32 ? 4 : 2;
    // rows of X that are not 16-byte aligned are copied: the copy is M x K, and every tile of
    // the product would load its rows element by element
    const bool copy_x = !rows_aligned16(X, ldx, (int)es);
    for (int r0 = 0; r0 < M; r0 += p.rows) {
        const int rows = M - r0 < p.rows ? M - r0 : p.rows;
        const void *x = at(X, (size_t)r0 * ldx, es);
        const int u = (int)es / 2;   // 16-bit units an element
        if (copy_x) G355_TRY(copy_rows(rows, rows, K * u, x, ldx * u, (uint16_t *)p.Xm, p.ldm * u, s));
        int blocks = 0;
        for (int v0 = 0; v0 < N; v0 += p.cols) {
            const int nc = N - v0 < p.cols ? N - v0 : p.cols;
            const gemm355_status st =
                piece_logits(dtype, flags, p.ranges, p.sums, rows, nc, K, copy_x ? p.Xm : x, copy_x ? p.ldm : ldx,
                             at(W, w_offset(flags, v0, ldw), es), ldw, p.Z, p.cols, s);
            if (st != GEMM355_OK) return st;
            hipLaunchKernelGGL(xent_chunk_kernel, dim3(cdiv(nc, kChunk), rows), dim3(256), 0, s, nc, v0, p.Z, p.cols,
                               labels + r0, p.part + (size_t)blocks * p.rows, p.rows, p.zl);
            G355_TRY(hipGetLastError());
            blocks += cdiv(nc, kChunk);
        }
        G355_TRY(merge(rows, N, blocks, p.part, p.rows, p.zl, labels + r0, ignore, loss ? loss + r0 : nullptr,
                       lse ? lse + r0 : nullptr, s));
    }
    return GEMM355_OK;
}

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

hipError_t prep(const GradCall &a, int Mp, int again, float *scale, RowGrad *rows, void *Xm, int ldm) {
    const dim3 grid(Mp < 1024 ? Mp : 1024);
    const size_t es = a.dtype == kF32 ? 4 : 2;
    const int vec = rows_aligned16(a.X, a.ldx, (int)es) && a.K % (16 / es) == 0;
    if (a.dtype == kF32)
        hipLaunchKernelGGL((xent_prep_kernel<float>), grid, dim3(256), 0, a.s, a.M, Mp, again, a.N, a.K, (const float *)a.X,
                           a.ldx, a.labels, a.ignore, a.lse, a.dloss, 0, scale, rows, (float *)Xm, ldm, vec);
    else
        hipLaunchKernelGGL((xent_prep_kernel<uint16_t>), grid, dim3(256), 0, a.s, a.M, Mp, again, a.N, a.K,
                           (const uint16_t *)a.X, a.ldx, a.labels, a.ignore, a.lse, a.dloss,
                           a.dtype == kF16 ? 1 : 0, scale, rows, (uint16_t *)Xm, ldm, vec);
    return hipGetLastError();
}

hipError_t piece_dz(const GradCall &a, const GradPlan &p, int v0, int nc) {
    return over_rows(p.Mp, [&](int r, int n) {
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

hipError_t round16(const GradCall &a, int rows, int cols, const float *acc, int lda, int splits, size_t stride,
                   size_t other, const float *scale, void *out, int ldo) {
    const bool vec = lda % 4 == 0 && stride % 4 == 0 && other % 4 == 0;
    if (!vec && (splits > 1 || other > 0)) return hipErrorInvalidValue;
    const int wide = ldo % 4 == 0 && (uintptr_t)out % 8 == 0;
    return over_rows(rows, [&](int r, int n) {
        const auto go = [&](auto t, auto v) {
            hipLaunchKernelGGL((xent_round_kernel<decltype(t), decltype(v)::value>), dim3(cdiv(cols, 1024), n),
                               dim3(256), 0, a.s, cols, acc + (size_t)r * lda, lda, splits, stride, other, scale,
                               (uint16_t *)out + (size_t)r * ldo, ldo, wide);
        };
        const auto typed = [&](auto t) { vec ? go(t, std::true_type{}) : go(t, std::false_type{}); };
        if (a.dtype == kF16) typed(f16_t{});
        else typed(bf16_t{});
    });
}

gemm355_status gradient_fused(const GradCall &a, bool copied, void *ws) {
    const FusedGradPlan p(copied, a.flags, a.M, a.N, a.K, ws);
    const bool tb = a.flags & GEMM355_TRANS_B, f16 = a.dtype == kF16;
    G355_TRY(prep(a, p.Mp, p.few ? kFewRows : 0, p.scale, p.rows, p.Xm, p.Kp));
    const bool one = !p.few && p.cols >= a.N && p.splits == 1;  // dX in one product
    for (int v0 = 0; v0 < a.N; v0 += p.cols) {
        const int nc = a.N - v0 < p.cols ? a.N - v0 : p.cols;
        const auto *w = (const uint16_t *)at(a.W, w_offset(a.flags, v0, a.ldw), 2);
        if (copied) G355_TRY(copy_weights(a.flags, nc, a.K, p.Kp, w, a.ldw, p.Wm, p.ldw, a.s));
        if (copied) w = p.Wm;
        const int lw = copied ? p.ldw : a.ldw;
        Section part[2];
        const int dz_rows = p.few ? kFewRows : p.Mp;
        const int dz_parts = head_sections(dz_rows, nc, p.Kp, part);
        for (int i = 0; i < dz_parts; ++i) {
            const Section &c = part[i];
            const HeadArgs h{dz_rows, c.cols, p.Kp, p.Xm, p.Kp, w + w_offset(a.flags, c.v0, lw), lw, tb};
            uint16_t *dZ = p.dZ + c.v0, *lo = p.few ? dZ + (size_t)kFewRows * p.cols : nullptr;
            G355_TRY(f16 ? launch_xent_dz_f16(c.tile, h, p.rows, v0 + c.v0, dZ, lo, p.cols, a.s)
                         : launch_xent_dz_bf16(c.tile, h, p.rows, v0 + c.v0, dZ, lo, p.cols, a.s));
        }
        if (a.dX != nullptr) {
            const Splits sp(nc, p.splits);
            ProductArgs q{};
            q.M = q.rows = p.dx_rows;
            q.N = p.Kp;
            q.cols = a.K;
            q.K = nc;
            q.A = p.dZ;
            q.lda = p.cols;
            q.B = w;
            q.ldb = lw;
            q.splits = sp.count;
            q.step = sp.step;
            if (one) {
                q.out = (uint16_t *)a.dX;
                q.ldo = a.lddx;
                q.factor = p.scale + 1;
            } else {
                q.part = p.dX;
                q.part_stride = p.dx_stride;
                q.ldo = p.ldx;
                q.accumulate = v0 > 0;
            }
            G355_TRY(f16 ? launch_xent_dx_f16(p.dx, tb, q, a.s) : launch_xent_dx_bf16(p.dx, tb, q, a.s));
        }
        const int dw_ranges = dw_splits(p.Mp, nc, a.K);
        int dw_parts = a.dW != nullptr ? dw_sections(a.M, nc, a.K, part) : 0;
        if (dw_parts > 0 && dw_ranges > 1) {
            part[0] = {0, nc, 128};
            dw_parts = 1;
        }
        for (int i = 0; i < dw_parts; ++i) {
            const Section &c = part[i];
            const int padded = (int)up((size_t)c.cols, 8);
            const uint16_t *dZ = p.dZ + c.v0;
            ProductArgs q{};
            q.K = p.Mp;
            q.A = tb ? dZ : p.Xm;
            q.lda = tb ? p.cols : p.Kp;
            q.B = tb ? p.Xm : dZ;
            q.ldb = tb ? p.Kp : p.cols;
            q.M = tb ? padded : p.Kp;
            q.N = tb ? p.Kp : padded;
            q.rows = tb ? c.cols : a.K;
            q.cols = tb ? a.K : c.cols;
            q.out = (uint16_t *)at(a.dW, w_offset(a.flags, v0 + c.v0, a.lddw), 2);
            q.ldo = a.lddw;
            q.factor = p.scale + 1;
            if (dw_ranges > 1) {
                const Splits sp(p.Mp, dw_ranges);
                q.splits = sp.count;
                q.step = sp.step;
                q.part = p.dW;
                q.ldo = (int)up((size_t)q.cols, 4);
                q.part_stride = (size_t)q.rows * q.ldo;
            }
            G355_TRY(f16 ? launch_xent_dw_f16(c.tile, q, a.s) : launch_xent_dw_bf16(c.tile, q, a.s));
            if (dw_ranges > 1)
                G355_TRY(round16(a, q.rows, q.cols, p.dW, q.ldo, q.splits, q.part_stride, 0, p.scale, q.out, a.lddw));
        }
    }
    if (!one && a.dX != nullptr)
        G355_TRY(round16(a, a.M, a.K, p.dX, p.ldx, p.splits, p.dx_stride, p.few ? (size_t)kFewRows * p.ldx : 0, p.scale,
                         a.dX, a.lddx));
    return GEMM355_OK;
}

// Whether the fused gradient takes this call: every operand's offsets in range.
bool fused_gradient(const GradCall &a, bool copied) {
    if (!fused_shape(a.dtype, a.N, a.K)) return false;
    const FusedGradPlan p(copied, a.flags, a.M, a.N, a.K, nullptr);
    return offsets_fit(p.Mp, p.cols) && offsets_fit(p.Mp, p.Kp) &&
           (!(a.flags & GEMM355_TRANS_B) || offsets_fit(p.cols, copied ? p.ldw : a.ldw)) &&
           (!copied || offsets_fit(p.Kp, p.ldw));
}

gemm355_status gradient(const GradCall &a, void *ws) {
    const GradPlan p(a.dtype, a.M, a.N, a.K, ws);
    const bool h16 = a.dtype != kF32, tb = a.flags & GEMM355_TRANS_B;
    const size_t es = h16 ? 2 : 4;
    hipError_t e = prep(a, p.Mp, 0, p.scale, p.rows, p.Xm, p.ldm);
    if (e != hipSuccess) return status_of(e);
    float *dx = h16 ? p.dX : (float *)a.dX;
    const int lddx = h16 ? a.K : a.lddx;
    for (int v0 = 0; v0 < a.N; v0 += p.cols) {
        const int nc = a.N - v0 < p.cols ? a.N - v0 : p.cols;
        const char *w = at(a.W, w_offset(a.flags, v0, a.ldw), es);
        gemm355_status st = piece_logits(a.dtype, a.flags, p.zr, p.sums, p.Mp, nc, a.K, p.Xm, p.ldm, w, a.ldw, p.Z,
                                         p.cols, a.s);
        if (st != GEMM355_OK) return st;
        e = piece_dz(a, p, v0, nc);
        if (e != hipSuccess) return status_of(e);
        if (a.dX != nullptr && p.dxr.count > 1) {
            const F32SplitArgs q{a.M, a.K, nc, p.Z, p.cols, (const float *)w, a.ldw, p.dX, p.dxr.step, v0 > 0};
            G355_TRY(launch_xent_split_f32(tb, q, a.s));
        } else if (a.dX != nullptr) {
            // whole k-steps, then the rest of the classes added: with a number of classes that is
            // no multiple of 4 every load of the one product would be predicated (binary32 2048
            // x 960 over 6649 classes 285 us, 213 + 7 in two)
            const unsigned fl = tb ? 0u : (unsigned)GEMM355_TRANS_B;
            const int whole = !h16 && nc > 32 ? nc / 32 * 32 : nc;
            st = gemm355_gemm_ex(GEMM355_VARIANT_AUTO, a.dtype, fl | (v0 > 0 ? (unsigned)GEMM355_ACCUMULATE : 0u), a.M,
                                 a.K, whole, p.dZ, p.cols, w, a.ldw, dx, lddx, a.s);
            if (st == GEMM355_OK && whole < nc)
                st = gemm355_gemm_ex(GEMM355_VARIANT_AUTO, a.dtype, fl | (unsigned)GEMM355_ACCUMULATE, a.M, a.K,
                                     nc - whole, at(p.dZ, whole, es), p.cols,
                                     at(w, w_offset(a.flags, whole, a.ldw), es), a.ldw, dx, lddx, a.s);
            if (st != GEMM355_OK) return st;
        }
        if (a.dW != nullptr) {
            // the piece's rows (TRANS_B) or columns of dW
            const int rows = tb ? nc : a.K, cols = tb ? a.K : nc;
            char *dw = at(a.dW, w_offset(a.flags, v0, a.lddw), es);
            float *out = h16 ? p.dW : (float *)dw;
            const int ldo = h16 ? cols : a.lddw;
            st = tb ? gemm355_gemm_ex(GEMM355_VARIANT_AUTO, a.dtype, GEMM355_TRANS_A, rows, cols, p.Mp, p.dZ, p.cols,
                                      p.Xm, p.ldm, out, ldo, a.s)
                    : gemm355_gemm_ex(GEMM355_VARIANT_AUTO, a.dtype, GEMM355_TRANS_A, rows, cols, p.Mp, p.Xm, p.ldm,
                                      p.dZ, p.cols, out, ldo, a.s);
            if (st != GEMM355_OK) return st;
            if (h16) {
                e = round16(a, rows, cols, out, ldo, 1, 0, 0, p.scale, dw, a.lddw);
                if (e != hipSuccess) return status_of(e);
            }
        }
    }
    if (a.dX != nullptr && p.dxr.count > 1) return sum_ranges(p.dxr, p.dX, a.M, a.K, (float *)a.dX, a.lddx, a.s);
    if (h16 && a.dX != nullptr) return status_of(round16(a, a.M, a.K, p.dX, a.K, 1, 0, 0, p.scale, a.dX, a.lddx));
    return GEMM355_OK;
}

}  // namespace

}  // namespace g355

using namespace g355;

extern "C" {

size_t gemm355_xent_workspace(int dtype, unsigned flags, int M, int N, int K) {
    if (!valid_shape(dtype, flags, M, N, K) || M == 0) return 0;
    const size_t any = ForwardPlan(dtype, M, N, K, nullptr).bytes;
    if (!fused_shape(dtype, N, K)) return any;
    // which one runs depends on W's alignment
    return std::max({any, FusedForwardPlan(false, flags, M, N, K, nullptr).bytes,
                     FusedForwardPlan(true, flags, M, N, K, nullptr).bytes});
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
    return (fused_shape(dtype, N, K) ? forward_fused : forward)(dtype, flags, M, N, K, X, ldx, W, ldw, labels, ignore, loss, lse,
                                                             workspace, stream);
}

size_t gemm355_xent_grad_workspace(int dtype, unsigned flags, int M, int N, int K) {
    if (!valid_shape(dtype, flags, M, N, K) || M == 0 || K == 0) return 0;
    const size_t any = GradPlan(dtype, M, N, K, nullptr).bytes;
    if (!fused_shape(dtype, N, K)) return any;
    return std::max({any, FusedGradPlan(false, flags, M, N, K, nullptr).bytes,
                     FusedGradPlan(true, flags, M, N, K, nullptr).bytes});
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
    const bool copied = !weights_load(flags, N, K, W, ldw);
    return fused_gradient(a, copied) ? gradient_fused(a, copied, workspace) : gradient(a, workspace);
}

}  // extern "C"
