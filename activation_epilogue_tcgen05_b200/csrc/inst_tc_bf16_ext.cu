// Instantiations of the persistent kernel with the extended epilogue, bf16 operands.
#include "find_ext.cuh"
namespace gemm_epi {
bool find_tc_bf16_ext(int cg, int epi, bool bmn, int bn, TcLauncher *l, KernelInfo *i) {
    return TcFindExt<DT_BF16, false>::find(cg, epi, bmn, bn, l, i);
}
}  // namespace gemm_epi
