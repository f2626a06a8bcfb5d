// Launcher of the epilogue's backward (dact.cuh).
#include <algorithm>

#include "dact.cuh"
#include "kernels.h"

namespace gemm_epi {

// Rows of a run: nearly whole waves of blocks -- three of three blocks an SM where z is read, two of
// four elsewhere and four of two from a checkpoint, on 148 SMs -- or runs of one batch of 32 rows.  With one wave some SMs have a block more
// than others, and nothing evens that out (8192 x 14336 GELU: 392 blocks 135 us, 1288 blocks 115); a wave
// with few blocks costs most of one (from the mask: 1120 blocks 86 us, 1232 blocks 99).  Up to 64 rows are
// one run, which writes dbias itself (64 x 4096 GELU: 3.6 us, 6.7 a call from Python; by two launches 4.1 and
// 11; 128 x 4096 would take 6.1 us against 4.3).
int64_t dact_rows(int64_t m, int64_t n, int blocks_sm) {
    const int64_t strips = (n + DACT_COLS - 1) / DACT_COLS, batches = (m + 31) / 32;
    if (batches <= 2) return batches * 32;
    const int64_t blocks = 148 * (blocks_sm == 3 ? 9 : 8);
    const int64_t runs = std::max<int64_t>(1, std::min<int64_t>(blocks / strips, batches));
    return (batches + runs - 1) / runs * 32;
}

// Whole rows to a block: where their blocks fill the GPU (148 SMs, three each), or rows of up to three
// passes (8192 x 14336 GELU 108 us, by strips 117; 1023 x 4104 from the mask 4.7 against 5.5, 64 x 4096 2.9
// against 3.4; not 300 x 16384, 12.5 against 11.0, nor 16 x 16384, 10.3 against 4.0).  Rows below 2048 columns leave
// threads without any: up to a few thousand rows the one launch still wins (300 x 128 1.9 against 4.0, 4096 x 1024
// 6.4 against 8.4, 8192 x 512 9.1 and 8.5), many such rows lose (16384 x 512 20.6 against 14.7, 65536 x 128 63 against 25).
bool dact_by_rows(int64_t m, int64_t n) { return m >= 148 * 3 * DACT_U || n <= 3 * DACT_WARPS * DACT_COLS; }

namespace {
template <int DT, int ACT, int AXIS>
cudaError_t dact(const DactParams &p, bool pdl, cudaStream_t s) {
    static std::atomic<bool> attr_done[64];
    const dim3 grid((unsigned)((p.n + DACT_COLS - 1) / DACT_COLS), (unsigned)((p.m + p.rows - 1) / p.rows), 1);
    constexpr int SMEM = dact_reads_z(ACT) ? dact_smem(false) : 0;
    return launch_as(dact_kernel<DT, ACT, AXIS>, attr_done, grid, 32 * DACT_WARPS, SMEM, pdl, s, p);
}

template <int DT, int ACT>
cudaError_t dact_whole_rows(const DactParams &p, bool pdl, cudaStream_t s) {
    static std::atomic<bool> attr_done[64];
    constexpr int SMEM = dact_reads_z(ACT) ? dact_smem(false) : 0;
    return launch_as(dact_rows_kernel<DT, ACT>, attr_done, dim3((unsigned)((p.m + DACT_U - 1) / DACT_U)), 32 * DACT_WARPS, SMEM,
                     pdl, s, p);
}

template <int DT, int ACT>
cudaError_t dact(int axis, const DactParams &p, bool pdl, cudaStream_t s) {
    if (axis == AXIS_ROW && p.dbias != nullptr) return dact_whole_rows<DT, ACT>(p, pdl, s);
    return axis == AXIS_COL ? dact<DT, ACT, AXIS_COL>(p, pdl, s) : dact<DT, ACT, AXIS_ROW>(p, pdl, s);
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
