// Launchers of the norm and its backward (rmsnorm.cuh).
#include <algorithm>
#include <atomic>

#include "kernels.h"
#include "rmsnorm.cuh"

namespace gemm_epi {

namespace {
template <class Kern, class P>
cudaError_t launch(Kern kern, int64_t grid, int threads, const P &p, bool pdl, cudaStream_t s, int smem = 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    if (pdl) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int DT, int OUT, int TPR, int VPT>
cudaError_t fwd(const NormParams &p, bool pdl, cudaStream_t s) {
    constexpr int T = norm_threads(TPR), RPB = T / TPR;
    return launch(rmsnorm_kernel<DT, OUT, TPR, VPT>, (p.m + RPB - 1) / RPB, T, p, pdl, s);
}

template <int DT, int OUT>
cudaError_t fwd_shape(const NormParams &p, bool pdl, cudaStream_t s) {
    const int nv = p.d / 8;
    if (nv <= 8) return fwd<DT, OUT, 8, 1>(p, pdl, s);
    if (nv <= 16) return fwd<DT, OUT, 16, 1>(p, pdl, s);
    if (nv <= 32) return fwd<DT, OUT, 32, 1>(p, pdl, s);
    if (nv <= 64) return fwd<DT, OUT, 32, 2>(p, pdl, s);
    if (nv <= 128) return fwd<DT, OUT, 32, 4>(p, pdl, s);
    if (nv <= 256) return fwd<DT, OUT, 128, 2>(p, pdl, s);
    if (nv <= 512) return fwd<DT, OUT, 128, 4>(p, pdl, s);
    if (nv <= 1024) return fwd<DT, OUT, 256, 4>(p, pdl, s);
    return fwd<DT, OUT, 512, 4>(p, pdl, s);
}

template <int DT>
cudaError_t fwd_out(int out, const NormParams &p, bool pdl, cudaStream_t s) {
    switch (out) {
    case NORM_SAME: return fwd_shape<DT, NORM_SAME>(p, pdl, s);
    case NORM_E4M3: return fwd_shape<DT, NORM_E4M3>(p, pdl, s);
    default: return fwd_shape<DT, NORM_E4M3_ROWS>(p, pdl, s);
    }
}

// Threads a row and vectors a thread of the backward kernel for rows of d elements.
struct BwdShape {
    int tpr, vpt;
};
BwdShape bwd_shape(int64_t d) {
    const int64_t nv = d / 8;
    if (nv <= 8) return {8, 1};
    if (nv <= 16) return {16, 1};
    if (nv <= 32) return {32, 1};
    if (nv <= 64) return {32, 2};
    if (nv <= 128) return {128, 1};
    if (nv <= 256) return {128, 2};
    if (nv <= 512) return {128, 4};
    if (nv <= 1024) return {256, 4};
    return {512, 4};
}

// Longer rows: the ring's depth, so that 512 threads an SM have 192 KB of it between them.
template <int DT, int T, int VPT>
cudaError_t bwd_rows(const NormBwdParams &p, int64_t grid, bool pdl, cudaStream_t s) {
    constexpr int STAGES = 2, SMEM = STAGES * 3 * T * VPT * 16;
    auto kern = rmsnorm_bwd_rows_kernel<DT, T, VPT, STAGES>;
    static std::atomic<bool> attr_done[64];
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_done[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_done[dev].store(true, std::memory_order_release);
    }
    return launch(kern, grid, T, p, pdl, s, SMEM);
}

template <int DT>
cudaError_t bwd(const NormBwdParams &p, bool pdl, cudaStream_t s) {
    const BwdShape b = bwd_shape(p.d);
    const int64_t grid = norm_bwd_parts(p.m, p.d);
    const int threads = norm_threads(b.tpr);
#define GEMM_EPI_NORM_BWD(T, V) \
    if (b.tpr == T && b.vpt == V) return launch(rmsnorm_bwd_kernel<DT, T, V>, grid, threads, p, pdl, s)
    GEMM_EPI_NORM_BWD(8, 1);
    GEMM_EPI_NORM_BWD(16, 1);
    GEMM_EPI_NORM_BWD(32, 1);
    GEMM_EPI_NORM_BWD(32, 2);
#undef GEMM_EPI_NORM_BWD
    if (b.tpr == 128 && b.vpt == 1) return bwd_rows<DT, 128, 1>(p, grid, pdl, s);
    if (b.tpr == 128) return b.vpt == 2 ? bwd_rows<DT, 128, 2>(p, grid, pdl, s) : bwd_rows<DT, 128, 4>(p, grid, pdl, s);
    return b.tpr == 256 ? bwd_rows<DT, 256, 4>(p, grid, pdl, s) : bwd_rows<DT, 512, 4>(p, grid, pdl, s);
}
}  // namespace

int64_t norm_bwd_parts(int64_t m, int64_t d) {
    const BwdShape b = bwd_shape(d);
    const int64_t rpb = norm_threads(b.tpr) / b.tpr;
    // as many as a B200's 148 SMs hold at once
    const int64_t resident = 148 * (b.tpr <= 32 ? 4 : norm_rows_per_sm(b.tpr, b.vpt));
    return std::min<int64_t>((m + rpb - 1) / rpb, resident);
}

cudaError_t launch_rmsnorm(int dt, int out, const NormParams &p, bool pdl, cudaStream_t s) {
    return dt == DT_F16 ? fwd_out<DT_F16>(out, p, pdl, s) : fwd_out<DT_BF16>(out, p, pdl, s);
}

cudaError_t launch_rmsnorm_bwd(int dt, const NormBwdParams &p, bool pdl, cudaStream_t s) {
    return dt == DT_F16 ? bwd<DT_F16>(p, pdl, s) : bwd<DT_BF16>(p, pdl, s);
}

}  // namespace gemm_epi
