// Launcher of the epilogue's backward (dact.cuh).
#include <algorithm>

#include "dact.cuh"
#include "kernels.h"

namespace gemm_epi {

// Runs of rows so that the launch has about 148 x 8 blocks, each run a whole number of the 32
// rows that a block has in flight.
int64_t dact_rows(int64_t m, int64_t n) {
    const int64_t strips = (n + DACT_COLS - 1) / DACT_COLS;
    const int64_t runs = std::max<int64_t>(1, std::min<int64_t>(148 * 8 / strips, 4096));
    const int64_t rows = (m + runs - 1) / runs;
    return (rows + 31) / 32 * 32;
}

namespace {
template <int DT, int ACT>
cudaError_t dact(int axis, const DactParams &p, bool pdl, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.n + DACT_COLS - 1) / DACT_COLS), (unsigned)((p.m + p.rows - 1) / p.rows), 1);
    cfg.blockDim = dim3(32 * DACT_WARPS, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    if (pdl) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    return axis == AXIS_COL ? cudaLaunchKernelEx(&cfg, dact_kernel<DT, ACT, AXIS_COL>, p)
                            : cudaLaunchKernelEx(&cfg, dact_kernel<DT, ACT, AXIS_ROW>, p);
}

template <int DT>
cudaError_t dact_of(int act, int axis, const DactParams &p, bool pdl, cudaStream_t s) {
    switch (act) {
    case DACT_NONE: return dact<DT, DACT_NONE>(axis, p, pdl, s);
    case DACT_RELU: return dact<DT, DACT_RELU>(axis, p, pdl, s);
    case DACT_RELU_MASK: return dact<DT, DACT_RELU_MASK>(axis, p, pdl, s);
    case DACT_GELU: return dact<DT, DACT_GELU>(axis, p, pdl, s);
    default: return dact<DT, DACT_TANH>(axis, p, pdl, s);
    }
}
}  // namespace

cudaError_t launch_dact(int dt, int act, int axis, const DactParams &p, bool pdl, cudaStream_t s) {
    return dt == DT_F16 ? dact_of<DT_F16>(act, axis, p, pdl, s) : dact_of<DT_BF16>(act, axis, p, pdl, s);
}

}  // namespace gemm_epi
