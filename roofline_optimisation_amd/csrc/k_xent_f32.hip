// dX of a binary32 head whose M x K tiles leave CUs idle: the sum over the classes is split
// into ranges, one workgroup of the FP32 tile routine (f32_gemm.hpp) per tile and range, and
// the ranges' partial sums are added afterwards.  As one product, 16 rows of 704 over 53476
// classes run on 11 CUs.
#include "f32_gemm.hpp"
#include "xent.hpp"

namespace g355 {

namespace {

// Ranges of p.step classes (a multiple of kBK).  FAST: rows of W 16-byte aligned and, where
// its classes are rows, K a multiple of 4: whole k-steps unpredicated, the rest of the last
// range added to their sums; else every load predicated.
template <bool B_MN, bool FAST>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(4)))
void xent_dx_f32_kernel(F32SplitArgs p) {
    using Cfg = F32Cfg<64, 64, 2, 2, false, B_MN>;
    __shared__ __attribute__((aligned(16))) float lds[2 * (Cfg::kLdsA + Cfg::kLdsB)];
    const int tiles = cdiv(p.M, 64) * cdiv(p.K, 64);
    const int id = xcd_contiguous_id(blockIdx.x, gridDim.x), split = id / tiles;
    int tm, tn;
    grouped_tile(id - split * tiles, cdiv(p.M, 64), cdiv(p.K, 64), 4, tm, tn);
    const int v0 = split * p.step, n = min(p.step, p.nc - v0);
    const float *A = p.dZ + v0, *B = p.W + (B_MN ? (size_t)v0 * p.ldw : (size_t)v0);
    float *C = p.part + (size_t)split * p.M * p.K;
    const int whole = FAST ? n / kBK * kBK : 0;
    if constexpr (FAST) {
        if (whole > 0)
            f32_tile<64, 64, 2, 2, 1, false, false, false, B_MN, true>(p.M, p.K, whole, A, p.ldz, B, p.ldw, C, p.K,
                                                                       1.0f, p.add, tm * 64, tn * 64, lds);
        if (whole == n) return;   // the same in every thread
        __syncthreads();
    }
    f32_tile<64, 64, 2, 2, FAST ? 1 : 0, true, false, false, B_MN, true>(
        p.M, p.K, n - whole, A + whole, p.ldz, B + (B_MN ? (size_t)whole * p.ldw : (size_t)whole), p.ldw, C, p.K, 1.0f,
        p.add || whole > 0, tm * 64, tn * 64, lds);
}

}  // namespace

hipError_t launch_xent_dx_f32(bool trans_b, const F32SplitArgs &p, hipStream_t s) {
    const dim3 grid(cdiv(p.M, 64) * cdiv(p.K, 64) * cdiv(p.nc, p.step));
    const bool fast = rows_aligned16(p.W, p.ldw, 4) && (!trans_b || p.K % 4 == 0);
    if (trans_b) {
        if (fast) hipLaunchKernelGGL((xent_dx_f32_kernel<true, true>), grid, dim3(256), 0, s, p);
        else hipLaunchKernelGGL((xent_dx_f32_kernel<true, false>), grid, dim3(256), 0, s, p);
    } else {
        if (fast) hipLaunchKernelGGL((xent_dx_f32_kernel<false, true>), grid, dim3(256), 0, s, p);
        else hipLaunchKernelGGL((xent_dx_f32_kernel<false, false>), grid, dim3(256), 0, s, p);
    }
    return hipGetLastError();
}

}  // namespace g355
