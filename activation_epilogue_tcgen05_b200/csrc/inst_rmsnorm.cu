// Launchers of the norm and its backward (rmsnorm.cuh).
#include <algorithm>

#include "kernels.h"
#include "rmsnorm.cuh"

namespace gemm_epi {

namespace {
template <int DT, int OUT, int TPR, int VPT>
cudaError_t fwd(const NormParams &p, bool pdl, cudaStream_t s) {
    constexpr int T = norm_threads(TPR), RPB = T / TPR;
    static std::atomic<bool> attr_done[64];
    return launch_as(rmsnorm_kernel<DT, OUT, TPR, VPT>, attr_done, dim3((unsigned)((p.m + RPB - 1) / RPB)), T, 0, pdl, s, p);
}

// Four vectors a thread at every size: with one vector and more threads few rows were not done
// sooner (1 x 4096 1.4 us either way, 300 x 4096 2.3 against 3.1 us) and many were slower (65536 x
// 256 without a residual 12.4 against 17.4 us).  Rows of up to 64 take two, so that a row's threads still
// read 64 bytes at a time (262144 x 64 with a residual 21.2 us, with four 25.9).
template <int DT, int OUT>
cudaError_t fwd_shape(const NormParams &p, bool pdl, cudaStream_t s) {
    const int nv = p.d / 8;
    if (nv <= 8) return fwd<DT, OUT, 4, 2>(p, pdl, s);
    if (nv <= 16) return fwd<DT, OUT, 4, 4>(p, pdl, s);
    if (nv <= 32) return fwd<DT, OUT, 8, 4>(p, pdl, s);
    if (nv <= 64) return fwd<DT, OUT, 16, 4>(p, pdl, s);
    if (nv <= 128) return fwd<DT, OUT, 32, 4>(p, pdl, s);
    if (nv <= 256) return fwd<DT, OUT, 64, 4>(p, pdl, s);
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

// Whether a backward call has few rows: up to one vector of 8 to each of 1024 threads an SM.  Then a
// thread takes one vector, so that a row is done soonest (with partial rows 37 x 1000: 3.2 us, with four vectors 6.2;
// 64 x 4096 4.7 against 6.0); above, four (300 x 4096 the same, 1200 x 1024 6.3 against 6.7).
bool few_rows(int64_t m, int64_t d) { return m * (d / 8) <= 148 * 1024; }

// Threads a row and vectors a thread of the backward kernel.
struct BwdShape {
    int tpr, vpt;
};
int64_t bwd_blocks(int64_t m, BwdShape b) {
    const int rpb = norm_bwd_threads(b.tpr, b.vpt) / b.tpr;
    return std::min<int64_t>((m + rpb - 1) / rpb, NORM_BWD_BLOCKS);
}
BwdShape bwd_shape(int64_t m, int64_t d) {
    const int64_t nv = d / 8;
    if (few_rows(m, d)) {
        if (nv <= 8) return {8, 1};
        if (nv <= 32) return {32, 1};
        if (nv <= 128) return {128, 1};
        if (nv <= 512) return {512, 1};
        return {512, 4};
    }
    if (nv <= 8) return {4, 2};
    if (nv <= 16) return {4, 4};
    if (nv <= 32) return {8, 4};
    if (nv <= 64) return {16, 4};
    if (nv <= 128) return {32, 4};
    if (nv <= 256) return {64, 4};
    if (nv <= 512) return {128, 4};
    if (nv <= 1024) return {256, 4};
    return {512, 4};
}

template <int DT, int TPR, int VPT>
cudaError_t bwd_one(const NormBwdParams &p, int64_t grid, bool pdl, cudaStream_t s) {
    constexpr int T = norm_bwd_threads(TPR, VPT), SMEM = norm_ring_bytes(T, VPT);
    static std::atomic<bool> attr_done[64];
    return launch_as(rmsnorm_bwd_kernel<DT, TPR, VPT>, attr_done, dim3((unsigned)grid), T, SMEM, pdl, s, p);
}

template <int DT, int TPR>
cudaError_t bwd_cluster(const NormBwdParams &p, bool pdl, cudaStream_t s) {
    constexpr int SMEM = norm_ring_bytes(NORM_CLUSTER_T, 1);
    static std::atomic<bool> attr_done[64];
    return launch_as_cluster(rmsnorm_bwd_kernel<DT, TPR, 1, true>, attr_done, dim3(NORM_CLUSTER), NORM_CLUSTER_T, SMEM, pdl,
                             NORM_CLUSTER, s, p);
}

template <int DT>
cudaError_t bwd(const NormBwdParams &p, bool pdl, cudaStream_t s) {
    const BwdShape b = bwd_shape(p.m, p.d);
    if (p.dgamma != nullptr) {
        switch (b.tpr) {
        case 8: return bwd_cluster<DT, 8>(p, pdl, s);
        case 32: return bwd_cluster<DT, 32>(p, pdl, s);
        case 128: return bwd_cluster<DT, 128>(p, pdl, s);
        default: return bwd_cluster<DT, 512>(p, pdl, s);
        }
    }
    const int64_t grid = bwd_blocks(p.m, b);
    if (b.vpt == 1) {
        switch (b.tpr) {
        case 8: return bwd_one<DT, 8, 1>(p, grid, pdl, s);
        case 32: return bwd_one<DT, 32, 1>(p, grid, pdl, s);
        case 128: return bwd_one<DT, 128, 1>(p, grid, pdl, s);
        default: return bwd_one<DT, 512, 1>(p, grid, pdl, s);
        }
    }
    switch (b.tpr) {
    case 4: return b.vpt == 2 ? bwd_one<DT, 4, 2>(p, grid, pdl, s) : bwd_one<DT, 4, 4>(p, grid, pdl, s);
    case 8: return bwd_one<DT, 8, 4>(p, grid, pdl, s);
    case 16: return bwd_one<DT, 16, 4>(p, grid, pdl, s);
    case 32: return bwd_one<DT, 32, 4>(p, grid, pdl, s);
    case 64: return bwd_one<DT, 64, 4>(p, grid, pdl, s);
    case 128: return bwd_one<DT, 128, 4>(p, grid, pdl, s);
    case 256: return bwd_one<DT, 256, 4>(p, grid, pdl, s);
    default: return bwd_one<DT, 512, 4>(p, grid, pdl, s);
    }
}

// Sets the word that a launch max-reduces into to 0: a launch of the library's own, since a memset
// between two launches keeps the second from being set up during the first (4 us a call).
__global__ void zero_word_kernel(unsigned int *w) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    if (threadIdx.x == 0) *w = 0u;
}
}  // namespace

int64_t norm_bwd_parts(int64_t m, int64_t d) {
    const BwdShape b = bwd_shape(m, d);
    // one vector a thread and at most two turns of a cluster's rows: no partial rows
    if (b.vpt == 1 && m <= 2 * NORM_CLUSTER * (NORM_CLUSTER_T / b.tpr)) return 0;
    return bwd_blocks(m, b);
}

cudaError_t launch_rmsnorm(int dt, int out, const NormParams &p, bool pdl, cudaStream_t s) {
    return dt == DT_F16 ? fwd_out<DT_F16>(out, p, pdl, s) : fwd_out<DT_BF16>(out, p, pdl, s);
}

cudaError_t launch_rmsnorm_bwd(int dt, const NormBwdParams &p, bool pdl, cudaStream_t s) {
    return dt == DT_F16 ? bwd<DT_F16>(p, pdl, s) : bwd<DT_BF16>(p, pdl, s);
}

namespace {
template <int DT, int Y>
cudaError_t add_parts(const float *src, int64_t parts, int64_t len, void *out, bool pdl, cudaStream_t s) {
    static std::atomic<bool> attr_done[64];
    return launch_as(add_parts_kernel<DT, Y>, attr_done, dim3((unsigned)((len + 31) / 32)), 8 * Y, 0, pdl, s, src, parts, len, out);
}
template <int DT>
cudaError_t add_parts(const float *src, int64_t parts, int64_t len, void *out, bool pdl, cudaStream_t s) {
    return parts <= 320 ? add_parts<DT, 32>(src, parts, len, out, pdl, s) : add_parts<DT, 64>(src, parts, len, out, pdl, s);
}
}  // namespace

cudaError_t launch_add_parts(int dt, const float *src, int64_t parts, int64_t len, void *out, bool pdl, cudaStream_t s) {
    return dt == DT_F16 ? add_parts<DT_F16>(src, parts, len, out, pdl, s) : add_parts<DT_BF16>(src, parts, len, out, pdl, s);
}

cudaError_t launch_zero_word(unsigned int *w, bool pdl, cudaStream_t s) {
    static std::atomic<bool> attr_done[64];
    return launch_as(zero_word_kernel, attr_done, dim3(1), 32, 0, pdl, s, w);
}

}  // namespace gemm_epi
