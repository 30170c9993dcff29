// Binary32 products of a head whose tiles leave CUs idle (dX of few rows, logits of few rows
// or classes): the sum is split into ranges, one workgroup of the FP32 tile routine
// (f32_gemm.hpp) per tile and range, and the ranges' partial sums are added afterwards.  As one
// product, dX of 16 rows of 704 over 53476 classes runs on 11 CUs.  With few
// rows it reads W, at 2.6 TB/s where W's rows are not 16-byte aligned (dX of 5 x 11952 x 3973 73
// us) and 3.4 where they are (5 x 82770 x 1984 196 us).
#include "f32_gemm.hpp"
#include "xent.hpp"

namespace g355 {

namespace {

// FAST: rows of B 16-byte aligned and, where they are the sum's terms (B_MN), cols a multiple
// of 4: whole k-steps unpredicated, the rest of the last range added to their sums; else every
// load predicated.
template <bool B_MN, bool FAST>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(4)))
void xent_split_f32_kernel(F32SplitArgs p) {
    using Cfg = F32Cfg<64, 64, 2, 2, false, B_MN>;
    __shared__ __attribute__((aligned(16))) float lds[2 * (Cfg::kLdsA + Cfg::kLdsB)];
    const int tiles = cdiv(p.M, 64) * cdiv(p.cols, 64);
    const int id = xcd_contiguous_id(blockIdx.x, gridDim.x), split = id / tiles;
    int tm, tn;
    grouped_tile(id - split * tiles, cdiv(p.M, 64), cdiv(p.cols, 64), 4, tm, tn);
    const int k0 = split * p.step, n = min(p.step, p.n - k0);
    const float *A = p.A + k0, *B = p.B + (B_MN ? (size_t)k0 * p.ldb : (size_t)k0);
    float *C = p.part + (size_t)split * p.M * p.cols;
    const int whole = FAST ? n / kBK * kBK : 0;
    if constexpr (FAST) {
        if (whole > 0)
            f32_tile<64, 64, 2, 2, 1, false, false, false, B_MN, true>(p.M, p.cols, whole, A, p.lda, B, p.ldb, C,
                                                                       p.cols, 1.0f, p.add, tm * 64, tn * 64, lds);
        if (whole == n) return;   // the same in every thread
        __syncthreads();
    }
    f32_tile<64, 64, 2, 2, FAST ? 1 : 0, true, false, false, B_MN, true>(
        p.M, p.cols, n - whole, A + whole, p.lda, B + (B_MN ? (size_t)whole * p.ldb : (size_t)whole), p.ldb, C, p.cols,
        1.0f, p.add || whole > 0, tm * 64, tn * 64, lds);
}

}  // namespace

hipError_t launch_xent_split_f32(bool rows, const F32SplitArgs &p, hipStream_t s) {
    const dim3 grid(cdiv(p.M, 64) * cdiv(p.cols, 64) * cdiv(p.n, p.step));
    const bool fast = rows_aligned16(p.B, p.ldb, 4) && (!rows || p.cols % 4 == 0);
    if (rows) {
        if (fast) hipLaunchKernelGGL((xent_split_f32_kernel<true, true>), grid, dim3(256), 0, s, p);
        else hipLaunchKernelGGL((xent_split_f32_kernel<true, false>), grid, dim3(256), 0, s, p);
    } else {
        if (fast) hipLaunchKernelGGL((xent_split_f32_kernel<false, true>), grid, dim3(256), 0, s, p);
        else hipLaunchKernelGGL((xent_split_f32_kernel<false, false>), grid, dim3(256), 0, s, p);
    }
    return hipGetLastError();
}

}  // namespace g355
