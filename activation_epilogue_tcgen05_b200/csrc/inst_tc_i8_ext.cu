// Instantiations of the persistent kernel with the extended epilogue, 8-bit integer operands.
#include "find_ext.cuh"
namespace gemm_epi {
bool find_tc_i8_ext(int cg, int epi, bool bmn, int bn, TcLauncher *l, KernelInfo *i) {
    return TcFindExt<DT_I8, false>::find(cg, epi, bmn, bn, l, i);
}
}  // namespace gemm_epi
