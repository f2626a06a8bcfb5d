// Launchers of the layer norm, its backward and the quantisation of rows (layernorm.cuh).
#include <algorithm>

#include "kernels.h"
#include "layernorm.cuh"

namespace gemm_epi {

namespace {
template <int DT, int OUT, int TPR, int VPT>
cudaError_t fwd(const LnParams &p, bool pdl, cudaStream_t s) {
    constexpr int T = norm_threads(TPR), RPB = T / TPR;
    static std::atomic<bool> attr_done[64];
    const dim3 grid((unsigned)((p.m + RPB - 1) / RPB));
    return p.d == 8 * TPR * VPT ? launch_as(layernorm_kernel<DT, OUT, TPR, VPT, true>, attr_done, grid, T, 0, pdl, s, p)
                                : launch_as(layernorm_kernel<DT, OUT, TPR, VPT, false>, attr_done, grid, T, 0, pdl, s, p);
}

// The root-mean-square norm's shapes, and three vectors a thread where a fourth of long rows would be missing (6710 x 5000 bf16 with
// residual 49 us, with the fourth 60).
template <int DT, int OUT>
cudaError_t fwd_shape(const LnParams &p, bool pdl, cudaStream_t s) {
    const int nv = p.d / 8;
    if (nv <= 8) return fwd<DT, OUT, 4, 2>(p, pdl, s);
    if (nv <= 16) return fwd<DT, OUT, 4, 4>(p, pdl, s);
    if (nv <= 32) return fwd<DT, OUT, 8, 4>(p, pdl, s);
    if (nv <= 64) return fwd<DT, OUT, 16, 4>(p, pdl, s);
    if (nv <= 128) return fwd<DT, OUT, 32, 4>(p, pdl, s);
    if (nv <= 256) return fwd<DT, OUT, 64, 4>(p, pdl, s);
    if (nv <= 512) return fwd<DT, OUT, 128, 4>(p, pdl, s);
    if (nv <= 768) return fwd<DT, OUT, 256, 3>(p, pdl, s);
    if (nv <= 1024) return fwd<DT, OUT, 256, 4>(p, pdl, s);
    if (nv <= 1536) return fwd<DT, OUT, 512, 3>(p, pdl, s);
    return fwd<DT, OUT, 512, 4>(p, pdl, s);
}

template <int DT>
cudaError_t fwd_out(int out, const LnParams &p, bool pdl, cudaStream_t s) {
    switch (out) {
    case NORM_SAME: return fwd_shape<DT, NORM_SAME>(p, pdl, s);
    case NORM_E4M3: return fwd_shape<DT, NORM_E4M3>(p, pdl, s);
    case NORM_I8_ROWS: return fwd_shape<DT, NORM_I8_ROWS>(p, pdl, s);
    default: return fwd_shape<DT, NORM_E4M3_ROWS>(p, pdl, s);
    }
}

template <int DT, int OUT, int TPR, int VPT, bool LONG = false>
cudaError_t quant(const NormParams &p, bool pdl, cudaStream_t s) {
    constexpr int T = norm_threads(TPR), RPB = T / TPR;
    static std::atomic<bool> attr_done[64];
    return launch_as(quant_rows_kernel<DT, OUT, TPR, VPT, LONG>, attr_done, dim3((unsigned)((p.m + RPB - 1) / RPB)), T, 0, pdl, s, p);
}
template <int DT, int OUT>
cudaError_t quant_shape(const NormParams &p, bool pdl, cudaStream_t s) {
    const int nv = p.d / 8;
    if (nv <= 16) return quant<DT, OUT, 4, 4>(p, pdl, s);
    if (nv <= 32) return quant<DT, OUT, 8, 4>(p, pdl, s);
    if (nv <= 64) return quant<DT, OUT, 16, 4>(p, pdl, s);
    if (nv <= 128) return quant<DT, OUT, 32, 4>(p, pdl, s);
    if (nv <= 256) return quant<DT, OUT, 64, 4>(p, pdl, s);
    if (nv <= 512) return quant<DT, OUT, 128, 4>(p, pdl, s);
    if (nv <= 1024) return quant<DT, OUT, 256, 4>(p, pdl, s);
    if (nv <= 2048) return quant<DT, OUT, 512, 4>(p, pdl, s);
    return quant<DT, OUT, 512, 4, true>(p, pdl, s);
}

// Whether a backward call has few rows, one vector a thread: the root-mean-square norm's rule.  With the sums by partial rows, as few
// and as many rows: 128 x 1024 3.9 us and 5.3, 300 x 256 3.5 and 5.0, 17 x 4096 5.3 and 5.9, 2000 x 64 3.6 and 5.4; near the rule's end
// 1180 x 1024 7.6 and 7.9, 4700 x 256 6.6 and 7.5, but 290 x 4096 8.6 and 8.0, 600 x 1024 6.0 and 5.7.
bool few_rows(int64_t m, int64_t d) { return m * (d / 8) <= 148 * 1024; }

// The backward kernel's threads a row, vectors a thread and threads a block: one block an SM.
struct BwdShape {
    int tpr, vpt, t;
};
int64_t bwd_blocks(int64_t m, BwdShape b) {
    const int rpb = b.t / b.tpr;
    return std::min<int64_t>((m + rpb - 1) / rpb, NORM_BWD_BLOCKS);
}
BwdShape bwd_shape(int64_t m, int64_t d) {
    const int64_t nv = d / 8;
    if (few_rows(m, d)) {
        if (nv <= 8) return {8, 1, 128};
        if (nv <= 32) return {32, 1, 128};
        if (nv <= 128) return {128, 1, 128};
        if (nv <= 512) return {512, 1, 512};
    }
    if (nv <= 8) return {4, 2, 512};
    if (nv <= 16) return {8, 2, 512};
    if (nv <= 32) return {16, 2, 512};
    if (nv <= 64) return {32, 2, 512};
    if (nv <= 128) return {64, 2, 512};
    if (nv <= 256) return {128, 2, 512};
    if (nv <= 512) return {256, 2, 512};
    if (nv <= 768) return {256, 3, 512};              // (6710 x 5000 65 us, by 512 threads of two vectors 76)
    if (nv <= 1024) return {512, 2, 512};
    if (nv <= 1536) return {512, 3, 512};             // (3355 x 10000 65 us, with a fourth that is missing 73)
    return {512, 4, 512};
}

template <int DT, int TPR, int VPT, int T = 512>
cudaError_t bwd_one(const LnBwdParams &p, int64_t grid, bool pdl, cudaStream_t s) {
    constexpr int SMEM = ln_ring_bytes(T, VPT, false);
    static std::atomic<bool> attr_done[64], attr_done_full[64];
    if constexpr (VPT > 1)                            // (few rows: the call's latency, whatever their length)
        if (p.d == 8 * TPR * VPT)
            return launch_as(layernorm_bwd_kernel<DT, TPR, VPT, T, true>, attr_done_full, dim3((unsigned)grid), T, SMEM, pdl, s, p);
    return launch_as(layernorm_bwd_kernel<DT, TPR, VPT, T, false>, attr_done, dim3((unsigned)grid), T, SMEM, pdl, s, p);
}

template <int DT, int TPR>
cudaError_t bwd_cluster(const LnBwdParams &p, bool pdl, cudaStream_t s) {
    constexpr int SMEM = ln_ring_bytes(NORM_CLUSTER_T, 1, true);
    static std::atomic<bool> attr_done[64];
    return launch_as_cluster(layernorm_bwd_kernel<DT, TPR, 1, NORM_CLUSTER_T, false, true>, attr_done, dim3(NORM_CLUSTER), NORM_CLUSTER_T, SMEM, pdl,
                             NORM_CLUSTER, s, p);
}

template <int DT>
cudaError_t bwd(const LnBwdParams &p, bool pdl, cudaStream_t s) {
    const BwdShape b = bwd_shape(p.m, p.d);
    if (p.dgamma != nullptr || p.dbeta != nullptr) {
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
        case 8: return bwd_one<DT, 8, 1, 128>(p, grid, pdl, s);
        case 32: return bwd_one<DT, 32, 1, 128>(p, grid, pdl, s);
        case 128: return bwd_one<DT, 128, 1, 128>(p, grid, pdl, s);
        default: return bwd_one<DT, 512, 1>(p, grid, pdl, s);
        }
    }
    switch (b.tpr) {
    case 4: return bwd_one<DT, 4, 2>(p, grid, pdl, s);
    case 8: return bwd_one<DT, 8, 2>(p, grid, pdl, s);
    case 16: return bwd_one<DT, 16, 2>(p, grid, pdl, s);
    case 32: return bwd_one<DT, 32, 2>(p, grid, pdl, s);
    case 64: return bwd_one<DT, 64, 2>(p, grid, pdl, s);
    case 128: return bwd_one<DT, 128, 2>(p, grid, pdl, s);
    case 256: return b.vpt == 2 ? bwd_one<DT, 256, 2>(p, grid, pdl, s) : bwd_one<DT, 256, 3>(p, grid, pdl, s);
    default:
        return b.vpt == 2 ? bwd_one<DT, 512, 2>(p, grid, pdl, s)
             : b.vpt == 3 ? bwd_one<DT, 512, 3>(p, grid, pdl, s) : bwd_one<DT, 512, 4>(p, grid, pdl, s);
    }
}
}  // namespace

int64_t ln_bwd_parts(int64_t m, int64_t d) {
    const BwdShape b = bwd_shape(m, d);
    // One vector a thread and at most two turns of a cluster's rows: no partial rows, the root-mean-square norm's rule (it saves the
    // host's second launch, and the scratch).  The cluster against partial rows in a graph, and as called from Python with
    // scratch given: 37 x 1000 5.4 and 3.5 us, 5.8 and 7.4; 256 x 256 4.1 and 3.2, 4.7 and 7.4; 1000 x 64 3.9 and 3.3, 4.7 and 7.4;
    // at 512 threads a row it loses both ways: 8 x 4096 7.4 and 5.1, 7.8 and 7.4; 16 x 4096 8.4 and 5.2, 8.8 and 7.3.
    if (b.vpt == 1 && m <= 2 * NORM_CLUSTER * (NORM_CLUSTER_T / b.tpr)) return 0;
    return bwd_blocks(m, b);
}

cudaError_t launch_layernorm(int dt, int out, const LnParams &p, bool pdl, cudaStream_t s) {
    return dt == DT_F16 ? fwd_out<DT_F16>(out, p, pdl, s) : fwd_out<DT_BF16>(out, p, pdl, s);
}

cudaError_t launch_layernorm_bwd(int dt, const LnBwdParams &p, bool pdl, cudaStream_t s) {
    return dt == DT_F16 ? bwd<DT_F16>(p, pdl, s) : bwd<DT_BF16>(p, pdl, s);
}

cudaError_t launch_quant_rows(int dt, int out, const NormParams &p, bool pdl, cudaStream_t s) {
    if (out == NORM_I8_ROWS)
        return dt == DT_F16 ? quant_shape<DT_F16, NORM_I8_ROWS>(p, pdl, s) : quant_shape<DT_BF16, NORM_I8_ROWS>(p, pdl, s);
    return dt == DT_F16 ? quant_shape<DT_F16, NORM_E4M3_ROWS>(p, pdl, s) : quant_shape<DT_BF16, NORM_E4M3_ROWS>(p, pdl, s);
}

}  // namespace gemm_epi
