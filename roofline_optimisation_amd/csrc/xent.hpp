// What the softmax cross entropy's files share: a row's data for the gradient, and the
// matrix-core launches of the 16-bit types (xent_dma.hpp).
#pragma once

#include <hip/hip_runtime.h>

#include "common.hpp"

namespace g355 {

// What the gradient needs of a row: its log-sum-exp, the upstream gradient (scaled) and the
// label, -1 for a row without one (whose lse and g are 0 and whose copy of X is 0).
struct alignas(16) RowGrad { float lse, g; int label, unused; };

// Z = X.op(W) of M rows and N classes; with trans_b W holds a class per row.  Rows start on
// 16-byte boundaries, K is a multiple of 8 and at least 128, and a K x N W has N a multiple
// of 8.
struct HeadArgs {
    int M, N, K;
    const void *X;
    int ldx;
    const void *W;
    int ldw;
    bool trans_b;
};

// The tiles of a head's products, EM rows x EN columns.
enum HeadTiles : int { kHead256 = 0, kHead128, kHead64, kHead64x128, kHead64x64, kHead128x128, kHeadTiles };
constexpr int kHeadRows[kHeadTiles] = {256, 128, 64, 64, 64, 128};
constexpr int kHeadCols[kHeadTiles] = {256, 256, 256, 128, 64, 128};
// A trip of the tile's ring of loads; K is at least one.
constexpr int kHeadTrip[kHeadTiles] = {128, 128, 128, 256, 256, 128};
// Columns of one wave, a block of the row statistics.
constexpr int kStatCols[kHeadTiles] = {128, 128, 64, 64, 32, 64};

// Statistics of Z, W pointing at class v0, by blocks of kStatCols[tile] columns: part[block *
// ldp + row] = (maximum, sum of exp(z - maximum)) and, where a row's label is one of these
// classes, zl[row] = its logit.
hipError_t launch_xent_stats_f16(int tile, const HeadArgs &h, const int64_t *labels, int v0, float2 *part,
                                 int ldp, float *zl, hipStream_t s);
hipError_t launch_xent_stats_bf16(int tile, const HeadArgs &h, const int64_t *labels, int v0, float2 *part,
                                  int ldp, float *zl, hipStream_t s);

// dZ (M x N rounded up to a multiple of 8, row stride ldz, the added columns 0) of the
// classes v0 .. v0 + N, W pointing at the first of them.  lo, if not NULL, takes what the
// rounding of dZ leaves over, rounded in turn.
hipError_t launch_xent_dz_f16(int tile, const HeadArgs &h, const RowGrad *rows, int v0, uint16_t *dZ, uint16_t *lo,
                              int ldz, hipStream_t s);
hipError_t launch_xent_dz_bf16(int tile, const HeadArgs &h, const RowGrad *rows, int v0, uint16_t *dZ, uint16_t *lo,
                               int ldz, hipStream_t s);

// A product of the gradient: op(A).op(B) over K.  A is M x K (k-contiguous), or K x M with
// a_mn; B is N x K, or K x N with b_mn.  M and N bound the loads (multiples of 8 where the
// operand is m/n-contiguous); rows x cols of the result are stored.
struct ProductArgs {
    int M, N, K;
    const uint16_t *A;
    int lda;
    const uint16_t *B;
    int ldb;
    int rows, cols;
    // 16-bit result: out = round(*factor * product)
    uint16_t *out;
    int ldo;
    const float *factor;
    // or binary32 partial sums: K walked in `splits` ranges of `step`, range r's sums at
    // part + r * part_stride, row stride ldo, added to what is there when `accumulate`
    float *part;
    size_t part_stride;
    int splits, step, accumulate;
};

// dX's product: A = dZ (k-contiguous), B m/n-contiguous or not; partial sums, or the 16-bit
// result when p.part is NULL.  Tiles
// kHead256 and kHead128.
hipError_t launch_xent_dx_f16(int tile, bool b_mn, const ProductArgs &p, hipStream_t s);
hipError_t launch_xent_dx_bf16(int tile, bool b_mn, const ProductArgs &p, hipStream_t s);
// dW's product: both operands m/n-contiguous, K a multiple of 128; square tiles of extent 128
// or 256 for the 16-bit result, 128 for partial sums (not accumulated).
hipError_t launch_xent_dw_f16(int tile, const ProductArgs &p, hipStream_t s);
hipError_t launch_xent_dw_bf16(int tile, const ProductArgs &p, hipStream_t s);

// A binary32 product of few tiles summed over ranges of `step` (a multiple of 32) of its n
// terms: M x cols = A.B, range r's sums at part + r M cols, added to what is there when `add`.
// A (M x n, row stride lda) has rows on 16-byte boundaries; B is n x cols (rows), or cols x n.
struct F32SplitArgs {
    int M, cols, n;
    const float *A;
    int lda;
    const float *B;
    int ldb;
    float *part;
    int step, add;
};
hipError_t launch_xent_split_f32(bool rows, const F32SplitArgs &p, hipStream_t s);

}  // namespace g355
