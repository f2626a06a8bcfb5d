// Instantiations of the persistent kernel with the extended epilogue, e4m3 operands.
#include "find_ext.cuh"
namespace gemm_epi {
bool find_tc_e4m3_ext(int cg, int epi, bool bmn, int bn, TcLauncher *l, KernelInfo *i) {
    return TcFindExt<DT_E4M3, false>::find(cg, epi, bmn, bn, l, i);
}
}  // namespace gemm_epi
