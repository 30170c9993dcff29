// The softmax cross entropy's products for the 16-bit types: the direct-to-LDS tile routine
// (h16_dma.hpp) with epilogues that turn a tile of logits into row statistics, or into dZ,
// in the registers the tile was summed in, so that the logits are never written.
//
// Bound: the matrix cores' rate at the part's power limit, and per tile the epilogue, which
// with one 256 x 256 tile per CU nothing hides.  At 8192 rows, K = 4096, bf16 (256 x 256
// tiles, us per tile, 94 of it the sum alone): statistics 99.5, of which a quarter is the
// exponentials (256 per lane at a quarter of the vector rate); dZ 105, whose stores leave
// from all CUs at once (33.5 MB a round); dW 89 (a sum over 8192 rows, per 4096 of them).
// Whole passes: 8192 x 131072 x 4096 statistics 6.2-6.4 ms (1.38-1.42 PFLOP/s), dZ 4 x 1.68-1.74,
// dX 4 x 1.49-1.55, dW 4 x 1.42-1.46 ms; the same product alone in the vendor's library 5.8-6.2 ms.
#pragma once

#include "h16_gemm.hpp"
#include "wave_reduce.hpp"
#include "xent.hpp"

namespace g355 {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;

// Another lane's value within the 16 lanes that hold a row of a 16 x 16 accumulator quad.
template <int CTRL>
__device__ __forceinline__ float of_lane(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
// The larger of two values; as the median with +infinity it costs one instruction, where
// fmaxf first quiets operands that could be signalling.  A NaN operand gives either value.
__device__ __forceinline__ float max2(float a, float b) {
    return __builtin_amdgcn_fmed3f(a, b, __builtin_huge_valf());
}

// Maximum and sum over those 16 lanes; every one of them gets the result.
__device__ __forceinline__ float row16_max(float v) {
    v = max2(v, of_lane<kDppQuadXor1>(v));
    v = max2(v, of_lane<kDppQuadXor2>(v));
    v = max2(v, of_lane<kDppRowHalfMirror>(v));
    return max2(v, of_lane<kDppRowMirror>(v));
}
__device__ __forceinline__ float row16_sum(float v) {
    v += of_lane<kDppQuadXor1>(v);
    v += of_lane<kDppQuadXor2>(v);
    v += of_lane<kDppRowHalfMirror>(v);
    return v + of_lane<kDppRowMirror>(v);
}

// An accumulator register, read where it is used (left to itself the compiler copies all 256
// of a 256 x 256 tile out of the accumulator file at once, which does not fit).
__device__ __forceinline__ float acc_read(float v) {
    float a;
    asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(a) : "a"(v));
    return a;
}

// Row statistics of the wave's tile.  Quad (i, j) holds rows row0 + 16 i + 4 (l/16) + r,
// columns col0 + 16 j + l%16: a row's values are kNB registers of 16 lanes.  Per row the
// maximum over registers and lanes, then the sum of exponentials.  Of every 16 results of a
// lane's 4 quad rows, lane l%16 = c keeps the one of quad row c / 4, register c % 4, so that
// 64 consecutive rows leave in one store.
struct StatsEpilogue {
    int M, N, v0;
    const int64_t *labels;
    float2 *part;
    int ldp;
    float *zl;
    __device__ int rows() const { return M; }
    __device__ int cols() const { return N; }

    template <bool EDGE, int kMB, int kNB>
    __device__ __forceinline__ void apply(floatx4 (&acc)[kMB][kNB], int row0, int col0, char *lds) const {
        const int lane = dma::lane_here(), c16 = lane & 15, q4 = lane >> 4;
        float2 *const out = part + (size_t)(col0 / (16 * kNB)) * ldp;
        constexpr float kNegInf = -__builtin_huge_valf();
        // the four labels of a lane's next quad row are loaded while this one's are used
        int64_t next[4];
        const auto load_labels = [&](int i) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = row0 + 16 * i + 4 * q4 + r;
                next[r] = labels[!EDGE || row < M ? row : 0];
            }
        };
        load_labels(0);
#pragma unroll
        for (int g = 0; g < kMB; g += 4) {
            constexpr int kI = kMB < 4 ? kMB : 4;
            float km = kNegInf, kl = 0.0f;
#pragma unroll
            for (int ii = 0; ii < kI; ++ii) {
                const int i = g + ii, r0 = row0 + 16 * i + 4 * q4;
                int rel[4];   // the label's column within the tile, -1 outside
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int64_t d = next[r] - v0 - col0;
                    rel[r] = d >= 0 && d < 16 * kNB && (!EDGE || (r0 + r < M && d < N - col0)) ? (int)d : -1;
                }
                if (i + 1 < kMB) load_labels(i + 1);
                __builtin_amdgcn_sched_barrier(0);
                // the four rows in straight-line code, so that their chains of dependent
                // instructions overlap: with one wave per SIMD nothing else does
                float x[4][kNB], m[4], l[4];
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int j = 0; j < kNB; ++j) {
                        x[r][j] = acc_read(acc[i][j][r]);
                        if (EDGE && col0 + 16 * j + c16 >= N) x[r][j] = kNegInf;
                    }
                // the labels' logits (of rows of many columns few tiles hold any label's)
                if (__any(max(max(rel[0], rel[1]), max(rel[2], rel[3])) >= 0)) {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
#pragma unroll
                        for (int j = 0; j < kNB; ++j)
                            if (rel[r] == 16 * j + c16) zl[r0 + r] = x[r][j];
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    m[r] = x[r][0];   // three-operand maxima: fewer instructions than max2's
#pragma unroll
                    for (int j = 1; j < kNB; ++j) m[r] = fmaxf(m[r], x[r][j]);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) m[r] = row16_max(m[r]);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    // exp(x - m) as 2^(x log2 e - m log2 e): the rounding of m log2 e moves all of
                    // the sum by |m| 2^-24 of it
                    const float shift = m[r] == kNegInf ? 0.0f : -m[r] * kLog2e;
                    l[r] = __builtin_amdgcn_exp2f(fmaf(x[r][0], kLog2e, shift));
#pragma unroll
                    for (int j = 1; j < kNB; ++j) l[r] += __builtin_amdgcn_exp2f(fmaf(x[r][j], kLog2e, shift));
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) l[r] = row16_sum(l[r]);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (c16 == 4 * ii + r) {
                        km = m[r];
                        kl = l[r];
                    }
            }
            const int row = row0 + 16 * (g + (c16 >> 2)) + 4 * q4 + (c16 & 3);
            if (c16 < 4 * kI && (!EDGE || row < M)) out[row] = make_float2(km, kl);
        }
    }
};

// Two values rounded to the 16-bit type, the first in the low half.
typedef float floatx2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 halfx2 __attribute__((ext_vector_type(2)));
template <typename T>
__device__ __forceinline__ uint32_t round_pair(float a, float b) {
    if constexpr (std::is_same<T, bf16_t>::value)
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((floatx2{a, b}), bf16x2));
    else
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((floatx2{a, b}), halfx2));
}

// One row of a pair of quads as 4-byte words of two 16-bit values: lanes 2m and 2m + 1
// exchange their rounded pairs, the even lane keeps columns 2m, 2m + 1 of the first quad (the
// low halves), the odd lane those of the second.  sel: pair_select(odd).
__device__ __forceinline__ uint32_t pair_select(int odd) { return odd ? 0x03020706u : 0x05040100u; }
template <typename T>
__device__ __forceinline__ uint32_t pair_word(float a0, float a1, uint32_t sel) {
    const uint32_t own = round_pair<T>(a0, a1);
    const uint32_t other = (uint32_t)__builtin_amdgcn_mov_dpp((int)own, kDppQuadXor1, 0xF, 0xF, true);
    return __builtin_amdgcn_perm(other, own, sel);
}

// 16 rows of a wave's 16-bit results, put together in its own part of LDS (rows of 16 kNB
// elements and 16 bytes) so that they leave as 16-byte pieces of whole lines: as 4-byte words
// out of the accumulators' layout each store instruction writes 64-byte pieces of four rows.
template <int kNB>
struct Strip {
    static constexpr int kRow = 32 * kNB + 16;   // bytes
    static constexpr int kChunks = 2 * kNB;      // 16-byte chunks of a row
    char *base;
    __device__ Strip(char *lds) : base(lds + (threadIdx.x / 64) * 16 * kRow) {}
    // columns 2 c, 2 c + 1 of row r
    __device__ __forceinline__ void put(int r, int c, uint32_t word) { *(uint32_t *)(base + r * kRow + 4 * c) = word; }
    // store(r, c, v): chunk c of row r, each of them once
    template <class F>
    __device__ __forceinline__ void each(int lane, F store) {
#pragma unroll
        for (int k = 0; k < 16 * kChunks / 64; ++k) {
            const int q = 64 * k + lane, r = q / kChunks, c = q % kChunks;
            store(r, c, *(const u32x4 *)(base + r * kRow + 16 * c));
        }
    }
};

// dZ of the wave's tile: g (exp(z - lse) - [column is the label]), rounded to T.  Columns
// from N to the next multiple of 8 are written as 0.  lo: the rounding's remainders, too.
template <typename T>
struct DzEpilogue {
    int M, N, v0;
    const RowGrad *rg;
    uint16_t *out, *lo;
    int ldo;
    __device__ int rows() const { return M; }
    __device__ int cols() const { return N; }

    template <bool EDGE, int kMB, int kNB>
    __device__ __forceinline__ void apply(floatx4 (&acc)[kMB][kNB], int row0, int col0, char *lds) const {
        const int lane = dma::lane_here(), c16 = lane & 15, q4 = lane >> 4, odd = lane & 1;
        const int cw = col0 + (lane & 14) + 16 * odd, padded = (N + 7) & ~7;
        const uint32_t sel = pair_select(odd);
        Strip<kNB> strip(lds);
        __syncthreads();
        // the data of a lane's next four rows are loaded while this quad row is computed
        floatx4 next[4];
        const auto load_rows = [&](int i) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = row0 + 16 * i + 4 * q4 + r;
                next[r] = *(const floatx4 *)(rg + (!EDGE || row < M ? row : 0));
            }
        };
        load_rows(0);
#pragma unroll
        for (int i = 0; i < kMB; ++i) {
            floatx4 now[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) now[r] = next[r];
            if (i + 1 < kMB) load_rows(i + 1);
            __builtin_amdgcn_sched_barrier(0);
            float d[4][kNB];
            int hot[4];   // the label's column relative to the lane's first
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const RowGrad w = __builtin_bit_cast(RowGrad, now[r]);
                const float shift = -w.lse * kLog2e;
                hot[r] = w.label - v0 - col0 - c16;
#pragma unroll
                for (int j = 0; j < kNB; ++j)
                    d[r][j] = w.g * __builtin_amdgcn_exp2f(fmaf(acc_read(acc[i][j][r]), kLog2e, shift));
            }
            // - g at the labels' columns: of rows of many columns few tiles hold any
            const unsigned last = 16 * (kNB - 1);
            if (__any((unsigned)hot[0] <= last || (unsigned)hot[1] <= last || (unsigned)hot[2] <= last ||
                      (unsigned)hot[3] <= last)) {
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int j = 0; j < kNB; ++j)
                        if (hot[r] == 16 * j) d[r][j] -= __builtin_bit_cast(RowGrad, now[r]).g;
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if constexpr (EDGE) {
#pragma unroll
                    for (int j = 0; j < kNB; ++j)
                        if (col0 + 16 * j + c16 >= N) d[r][j] = 0.0f;
                }
#pragma unroll
                for (int j = 0; j < kNB; j += 2)
                    strip.put(4 * q4 + r, (lane & 14) / 2 + 8 * (j + odd), pair_word<T>(d[r][j], d[r][j + 1], sel));
                if (lo != nullptr) {
                    const int row = row0 + 16 * i + 4 * q4 + r;
#pragma unroll
                    for (int j = 0; j < kNB; j += 2) {
                        const uint32_t v = pair_word<T>(d[r][j] - to_float(T{to_bits(d[r][j], T{})}),
                                                        d[r][j + 1] - to_float(T{to_bits(d[r][j + 1], T{})}), sel);
                        if (!EDGE || (row < M && cw + 16 * j < padded))
                            *(uint32_t *)(lo + (size_t)row * ldo + cw + 16 * j) = v;
                    }
                }
            }
            strip.each(lane, [&](int r, int c, u32x4 v) {
                const int row = row0 + 16 * i + r, col = col0 + 8 * c;
                if (!EDGE || (row < M && col < padded)) *(u32x4 *)(out + (size_t)row * ldo + col) = v;
            });
        }
    }
};

// The 16-bit result of a product: round(factor * sum), in 16-byte pieces at whatever alignment
// the output has (gfx950 under the HSA ABI runs with unaligned global access enabled).
template <typename T>
struct RoundEpilogue {
    int nrows, ncols;
    uint16_t *out;
    int ldo;
    const float *factor;
    __device__ int rows() const { return nrows; }
    __device__ int cols() const { return ncols; }

    template <bool EDGE, int kMB, int kNB>
    __device__ __forceinline__ void apply(floatx4 (&acc)[kMB][kNB], int row0, int col0, char *lds) const {
        const int lane = dma::lane_here(), q4 = lane >> 4, odd = lane & 1;
        const float f = *factor;
        const uint32_t sel = pair_select(odd);
        Strip<kNB> strip(lds);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kMB; ++i) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int j = 0; j < kNB; j += 2)
                    strip.put(4 * q4 + r, (lane & 14) / 2 + 8 * (j + odd),
                              pair_word<T>(f * acc_read(acc[i][j][r]), f * acc_read(acc[i][j + 1][r]), sel));
            strip.each(lane, [&](int r, int c, u32x4 v) {
                const int row = row0 + 16 * i + r, col = col0 + 8 * c;
                uint16_t *o = out + (size_t)row * ldo + col;
                if (!EDGE || (row < nrows && col + 8 <= ncols)) *(u16x8_ua *)o = __builtin_bit_cast(u16x8, v);
                else if (row < nrows)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (col + e < ncols) o[e] = (uint16_t)(v[e / 2] >> (16 * (e % 2)));
            });
        }
    }
};

// Binary32 partial sums, stored (EPI 0) or added to what is there (EPI 1).
template <typename T, int EPI>
struct PartialEpilogue {
    int nrows, ncols;
    float *part;
    int ldo;
    __device__ int rows() const { return nrows; }
    __device__ int cols() const { return ncols; }

    template <bool EDGE, int kMB, int kNB>
    __device__ __forceinline__ void apply(floatx4 (&acc)[kMB][kNB], int row0, int col0, char *lds) const {
        dma::store_tile<EPI, T, EDGE>(acc, part, ldo, row0, col0, nrows, ncols, 1.0f, EPI);
    }
};

// The tiles' waves and ring stages: 256 x 256 on 2 x 2 waves of 128 x 128, 128 x 256 on 2 x 2
// of 64 x 128, 64 x 256 on 1 x 4 of 64 x 64, 64 x 128 and 64 x 64 on 2 x 2.
template <int TILE>
struct HeadTile {
    static constexpr int kEM = kHeadRows[TILE], kEN = kHeadCols[TILE];
    static constexpr int kWM = TILE == kHead64 ? 1 : 2, kWN = 4 / kWM;
    static constexpr int kNs = kHeadTrip[TILE] / dma::kBK;
    static constexpr int kPerSimd = TILE == kHead64 || TILE == kHead64x64 || TILE == kHead128x128 ? 2 : 1;  // waves: workgroups per CU
    using G = dma::Geo<kEM, kEN, kWM, kWN, kNs, 0>;
    static_assert(kEN / kWN == kStatCols[TILE], "a statistics block is a wave's columns");
};

template <typename T, bool W_MN, int TILE, bool KR, class EX>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(HeadTile<TILE>::kPerSimd)))
void xent_head_kernel(int M, int N, int K, const uint16_t *__restrict__ X, int ldx,
                      const uint16_t *__restrict__ W, int ldw, EX ex) {
    using H = HeadTile<TILE>;
    __shared__ __attribute__((aligned(1024))) char lds[H::G::kLds];
    int tm, tn;
    grouped_tile(xcd_contiguous_id(blockIdx.x, gridDim.x), cdiv(M, H::kEM), cdiv(N, H::kEN), 4, tm, tn);
    // a K x N W is loaded in whole chunks of 8 classes; what lies past N in the last is masked
    dma::dma_tile<T, false, W_MN, 0, H::kEM, H::kEN, H::kWM, H::kWN, H::kNs, 0, false, KR, EX>(
        M, W_MN ? (N + 7) & ~7 : N, K, X, ldx, W, ldw, nullptr, 0, 1.0f, 0, tm * H::kEM, tn * H::kEN, lds, ex);
}

// dX's product over one of p.splits ranges of K: partial sums (EPI 0 or, adding to what is
// there, 1), or the rounded result.
template <typename T, bool B_MN, int TILE, bool KR, int EPI>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(HeadTile<TILE>::kPerSimd)))
void xent_dx_kernel(ProductArgs p) {
    using H = HeadTile<TILE>;
    constexpr int EM = H::kEM, EN = H::kEN;
    __shared__ __attribute__((aligned(1024))) char lds[H::G::kLds];
    const int tiles = cdiv(p.rows, EM) * cdiv(p.cols, EN);
    const int id = xcd_contiguous_id(blockIdx.x, gridDim.x);
    const int split = id / tiles;
    int tm, tn;
    grouped_tile(id - split * tiles, cdiv(p.rows, EM), cdiv(p.cols, EN), 4, tm, tn);
    const int k0 = split * p.step;
    const int K = split + 1 < p.splits ? p.step : p.K - k0;
    const uint16_t *A = p.A + k0, *B = p.B + (B_MN ? (size_t)k0 * p.ldb : (size_t)k0);
    if constexpr (EPI < 2) {
        using EX = PartialEpilogue<T, EPI>;
        dma::dma_tile<T, false, B_MN, 0, EM, EN, H::kWM, H::kWN, H::kNs, 0, false, KR, EX>(
            p.M, p.N, K, A, p.lda, B, p.ldb, nullptr, 0, 1.0f, 0, tm * EM, tn * EN, lds,
            EX{p.rows, p.cols, p.part + split * p.part_stride, p.ldo});
    } else {
        using EX = RoundEpilogue<T>;
        dma::dma_tile<T, false, B_MN, 0, EM, EN, H::kWM, H::kWN, H::kNs, 0, false, KR, EX>(
            p.M, p.N, K, A, p.lda, B, p.ldb, nullptr, 0, 1.0f, 0, tm * EM, tn * EN, lds,
            EX{p.rows, p.cols, p.out, p.ldo, p.factor});
    }
}

// dW's product: the rounded result, or (PART) the partial sums of one of p.splits ranges of
// the rows.
template <typename T, int E, bool PART>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(E == 128 ? 2 : 1)))
void xent_dw_kernel(ProductArgs p) {
    using G = dma::Geo<E, E, 2, 2, 4, 0>;
    __shared__ __attribute__((aligned(1024))) char lds[G::kLds];
    const int tiles = cdiv(p.rows, E) * cdiv(p.cols, E);
    const int id = xcd_contiguous_id(blockIdx.x, gridDim.x), split = PART ? id / tiles : 0;
    int tm, tn;
    grouped_tile(id - split * tiles, cdiv(p.rows, E), cdiv(p.cols, E), 4, tm, tn);
    if constexpr (PART) {
        using EX = PartialEpilogue<T, 0>;
        const int k0 = split * p.step, K = split + 1 < p.splits ? p.step : p.K - k0;
        dma::dma_tile<T, true, true, 0, E, E, 2, 2, 4, 0, false, false, EX>(
            p.M, p.N, K, p.A + (size_t)k0 * p.lda, p.lda, p.B + (size_t)k0 * p.ldb, p.ldb, nullptr, 0, 1.0f, 0, tm * E,
            tn * E, lds, EX{p.rows, p.cols, p.part + split * p.part_stride, p.ldo});
    } else {
        using EX = RoundEpilogue<T>;
        dma::dma_tile<T, true, true, 0, E, E, 2, 2, 4, 0, false, false, EX>(
            p.M, p.N, p.K, p.A, p.lda, p.B, p.ldb, nullptr, 0, 1.0f, 0, tm * E, tn * E, lds,
            EX{p.rows, p.cols, p.out, p.ldo, p.factor});
    }
}

template <typename T, bool W_MN, int TILE, class EX>
hipError_t launch_head_tile(const HeadArgs &h, const EX &ex, hipStream_t s) {
    const dim3 grid(cdiv(h.M, kHeadRows[TILE]) * cdiv(h.N, kHeadCols[TILE]));
    const auto *X = (const uint16_t *)h.X, *W = (const uint16_t *)h.W;
    if (h.K % kHeadTrip[TILE] != 0)
        hipLaunchKernelGGL((xent_head_kernel<T, W_MN, TILE, true, EX>), grid, dim3(256), 0, s, h.M, h.N, h.K, X,
                           h.ldx, W, h.ldw, ex);
    else
        hipLaunchKernelGGL((xent_head_kernel<T, W_MN, TILE, false, EX>), grid, dim3(256), 0, s, h.M, h.N, h.K, X,
                           h.ldx, W, h.ldw, ex);
    return hipGetLastError();
}

template <typename T, bool W_MN, class EX>
hipError_t launch_head_layout(int tile, const HeadArgs &h, const EX &ex, hipStream_t s) {
    switch (tile) {
    case kHead256: return launch_head_tile<T, W_MN, kHead256>(h, ex, s);
    case kHead128: return launch_head_tile<T, W_MN, kHead128>(h, ex, s);
    case kHead64: return launch_head_tile<T, W_MN, kHead64>(h, ex, s);
    case kHead64x128: return launch_head_tile<T, W_MN, kHead64x128>(h, ex, s);
    case kHead64x64: return launch_head_tile<T, W_MN, kHead64x64>(h, ex, s);
    default: return launch_head_tile<T, W_MN, kHead128x128>(h, ex, s);
    }
}

template <typename T, class EX>
hipError_t launch_head(int tile, const HeadArgs &h, const EX &ex, hipStream_t s) {
    return h.trans_b ? launch_head_layout<T, false>(tile, h, ex, s) : launch_head_layout<T, true>(tile, h, ex, s);
}

template <typename T, bool B_MN, int TILE, bool KR>
hipError_t launch_dx_epi(const ProductArgs &p, hipStream_t s) {
    const dim3 grid(cdiv(p.rows, kHeadRows[TILE]) * cdiv(p.cols, kHeadCols[TILE]) * p.splits);
    if (p.part == nullptr)
        hipLaunchKernelGGL((xent_dx_kernel<T, B_MN, TILE, KR, 2>), grid, dim3(256), 0, s, p);
    else if (p.accumulate)
        hipLaunchKernelGGL((xent_dx_kernel<T, B_MN, TILE, KR, 1>), grid, dim3(256), 0, s, p);
    else
        hipLaunchKernelGGL((xent_dx_kernel<T, B_MN, TILE, KR, 0>), grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

template <typename T, bool B_MN>
hipError_t launch_dx_layout(int tile, const ProductArgs &p, hipStream_t s) {
    // the ranges before the last are whole ring trips
    const bool kr = p.K % 128 != 0;
    if (tile == kHead128)
        return kr ? launch_dx_epi<T, B_MN, kHead128, true>(p, s) : launch_dx_epi<T, B_MN, kHead128, false>(p, s);
    return kr ? launch_dx_epi<T, B_MN, kHead256, true>(p, s) : launch_dx_epi<T, B_MN, kHead256, false>(p, s);
}

template <typename T>
hipError_t launch_dx(int tile, bool b_mn, const ProductArgs &p, hipStream_t s) {
    return b_mn ? launch_dx_layout<T, true>(tile, p, s) : launch_dx_layout<T, false>(tile, p, s);
}

template <typename T>
hipError_t launch_dw(int tile, const ProductArgs &p, hipStream_t s) {
    const dim3 grid(cdiv(p.rows, tile) * cdiv(p.cols, tile) * (p.part != nullptr ? p.splits : 1));
    if (p.part != nullptr) hipLaunchKernelGGL((xent_dw_kernel<T, 128, true>), grid, dim3(256), 0, s, p);
    else if (tile == 128) hipLaunchKernelGGL((xent_dw_kernel<T, 128, false>), grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((xent_dw_kernel<T, 256, false>), grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace

}  // namespace g355
