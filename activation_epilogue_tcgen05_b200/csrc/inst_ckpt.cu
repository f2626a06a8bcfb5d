// Launchers of the 8-bit checkpoints (ckpt.cuh) and of the epilogue's backward from them (dact.cuh).
#include <algorithm>

#include "ckpt.cuh"
#include "dact.cuh"
#include "kernels.h"

namespace gemm_epi {

namespace {
template <int DT, int EPI, int U>
cudaError_t ckpt(bool save, const CkptParams &p, bool pdl, cudaStream_t s) {
    static std::atomic<bool> attr_done[64];
    const dim3 grid((p.total + CKPT_T / 4 * U - 1) / (CKPT_T / 4 * U));
    return save ? launch_as(ckpt_save_kernel<DT, EPI, U>, attr_done, grid, CKPT_T, 0, pdl, s, p)
                : launch_as(ckpt_load_kernel<DT, EPI, U>, attr_done, grid, CKPT_T, 0, pdl, s, p);
}
template <int DT, int EPI>
cudaError_t ckpt(bool save, const CkptParams &p, bool pdl, cudaStream_t s) {
    // four groups a thread, or one where that leaves SMs without a block.  Saved and loaded as GELU's, bf16, by ones and by fours: 64 x 4096
    // 3.2 and 4.4 us, 512 x 4096 5.5 and 6.1, 1023 x 4104 9.0 and 10.8 (f16 tanh 9.2 and 10.9), 32768 x 128 9.0 and 10.8, 1184 x 4096 10.3 and 11.2;
    // beyond, 2048 x 4096 16.5 and 16.0, 1024 x 14336 27.0 and 25.3, 4096 x 4096 30.4 and 27.7, 8192 x 14336 206 and 177.
    return p.total <= 148 * 8 * 2 * (CKPT_T / 4) ? ckpt<DT, EPI, 1>(save, p, pdl, s) : ckpt<DT, EPI, 4>(save, p, pdl, s);
}
template <int DT>
cudaError_t ckpt_of(bool save, int epi, const CkptParams &p, bool pdl, cudaStream_t s) {
    switch (epi) {
    case EPI_RELU: return ckpt<DT, EPI_RELU>(save, p, pdl, s);
    case EPI_GELU: return ckpt<DT, EPI_GELU>(save, p, pdl, s);
    case EPI_TANH: return ckpt<DT, EPI_TANH>(save, p, pdl, s);
    default: return ckpt<DT, EPI_NONE>(save, p, pdl, s);
    }
}

template <int DT, int ACT, bool VAL>
cudaError_t dact_ckpt(int axis, const DactParams &p, bool pdl, cudaStream_t s) {
    constexpr int SMEM = dact_smem(true), T = 32 * DACT_WARPS;
    const dim3 grid((unsigned)((p.n + DACT_COLS - 1) / DACT_COLS), (unsigned)((p.m + p.rows - 1) / p.rows), 1);
    if (axis == AXIS_ROW && p.dbias != nullptr) {
        static std::atomic<bool> attr_done[64], attr_done2[64], attr_done3[64];
        // narrow rows by warps: 16384 x 1024 GELU 28 us for 34, x 256 16 for 29, 65536 x 128 30 for 106; up to 1024 rows the same
        if (p.n <= 4 * DACT_COLS && p.m >= 1024)
            return launch_as(dact_narrow_kernel<DT, ACT, VAL>, attr_done3,
                             dim3((unsigned)std::min<int64_t>((p.m + DACT_WARPS - 1) / DACT_WARPS, 148 * dact_blocks(ACT, true))), T, SMEM,
                             pdl, s, p);
        // two rows a block where four leave SMs with one block or none.  GELU by twos and by fours: 64 x 4096 2.3 and 3.6 us, 300 x 4104 3.8 and
        // 4.3, 1023 x 4104 6.4 and 6.6, 1500 x 4104 9.3 and 10.3 (1023 x 1024 3.1 and 2.9); fours are not faster beyond (2500 x 4104 14.2 and
        // 16.1, 4096 x 4096 19.2 and 20.2): the limit is where they were thought to be.
        if (p.m < 148 * 3 * DACT_U)
            return launch_as(dact_rows_kernel<DT, ACT, true, VAL, 2>, attr_done2, dim3((unsigned)((p.m + 1) / 2)), T, dact_smem(true, 2),
                             pdl, s, p);
        return launch_as(dact_rows_kernel<DT, ACT, true, VAL>, attr_done, dim3((unsigned)((p.m + DACT_U - 1) / DACT_U)), T, SMEM, pdl,
                         s, p);
    }
    if (axis == AXIS_COL) {
        static std::atomic<bool> attr_done[64];
        return launch_as(dact_kernel<DT, ACT, AXIS_COL, true, VAL>, attr_done, grid, T, SMEM, pdl, s, p);
    }
    static std::atomic<bool> attr_done[64];
    return launch_as(dact_kernel<DT, ACT, AXIS_ROW, true, VAL>, attr_done, grid, T, SMEM, pdl, s, p);
}
template <int DT, int ACT>
cudaError_t dact_ckpt(int axis, const DactParams &p, bool pdl, cudaStream_t s) {
    return p.h != nullptr ? dact_ckpt<DT, ACT, true>(axis, p, pdl, s) : dact_ckpt<DT, ACT, false>(axis, p, pdl, s);
}
template <int DT>
cudaError_t dact_ckpt_of(int act, int axis, const DactParams &p, bool pdl, cudaStream_t s) {
    switch (act) {
    case DACT_RELU: return dact_ckpt<DT, DACT_RELU>(axis, p, pdl, s);
    case DACT_GELU: return dact_ckpt<DT, DACT_GELU>(axis, p, pdl, s);
    default: return dact_ckpt<DT, DACT_TANH>(axis, p, pdl, s);
    }
}
}  // namespace

cudaError_t launch_ckpt(int dt, bool save, int epi, const CkptParams &p, bool pdl, cudaStream_t s) {
    return dt == DT_F16 ? ckpt_of<DT_F16>(save, epi, p, pdl, s) : ckpt_of<DT_BF16>(save, epi, p, pdl, s);
}

cudaError_t launch_dact_ckpt(int dt, int act, int axis, const DactParams &p, bool pdl, cudaStream_t s) {
    return dt == DT_F16 ? dact_ckpt_of<DT_F16>(act, axis, p, pdl, s) : dact_ckpt_of<DT_BF16>(act, axis, p, pdl, s);
}

}  // namespace gemm_epi
