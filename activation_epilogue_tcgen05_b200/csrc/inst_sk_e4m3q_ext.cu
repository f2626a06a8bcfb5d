// Instantiations of the small-m split-K kernel with the extended epilogue, e4m3 operands with an e4m3 output.
#include "find_ext.cuh"
namespace gemm_epi {
bool find_sk_e4m3q_ext(int epi, bool wmn, int nm, SkLauncher *l, KernelInfo *i) {
    return SkFindExt<DT_E4M3, true>::find(epi, wmn, nm, l, i);
}
}  // namespace gemm_epi
