// Launchers of the norm and its backward (rmsnorm.cuh).
#include <algorithm>

#include "kernels.h"
#include "rmsnorm.cuh"

namespace gemm_epi {

namespace {
template <class Kern, class P>
cudaError_t launch(Kern kern, int64_t grid, int threads, const P &p, bool pdl, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
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
    if (nv <= 128) return {32, 4};
    if (nv <= 256) return {128, 2};
    if (nv <= 512) return {128, 4};
    if (nv <= 1024) return {256, 4};
    return {512, 4};
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
    GEMM_EPI_NORM_BWD(32, 4);
    GEMM_EPI_NORM_BWD(128, 2);
    GEMM_EPI_NORM_BWD(128, 4);
    GEMM_EPI_NORM_BWD(256, 4);
    GEMM_EPI_NORM_BWD(512, 4);
#undef GEMM_EPI_NORM_BWD
    return cudaErrorInvalidValue;
}
}  // namespace

int64_t norm_bwd_parts(int64_t m, int64_t d) {
    const int threads = norm_threads(bwd_shape(d).tpr);
    const int64_t rpb = threads / bwd_shape(d).tpr;
    const int64_t resident = 148 * std::max(1, 512 / threads);     // a B200's SMs, 512 threads each
    return std::min<int64_t>((m + rpb - 1) / rpb, resident);
}

cudaError_t launch_rmsnorm(int dt, int out, const NormParams &p, bool pdl, cudaStream_t s) {
    return dt == DT_F16 ? fwd_out<DT_F16>(out, p, pdl, s) : fwd_out<DT_BF16>(out, p, pdl, s);
}

cudaError_t launch_rmsnorm_bwd(int dt, const NormBwdParams &p, bool pdl, cudaStream_t s) {
    return dt == DT_F16 ? bwd<DT_F16>(p, pdl, s) : bwd<DT_BF16>(p, pdl, s);
}

}  // namespace gemm_epi
