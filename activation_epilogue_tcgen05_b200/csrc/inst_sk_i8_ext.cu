// Instantiations of the small-m split-K kernel with the extended epilogue, 8-bit integer operands.
#include "find_ext.cuh"
namespace gemm_epi {
bool find_sk_i8_ext(int epi, bool wmn, int nm, SkLauncher *l, KernelInfo *i) {
    return SkFindExt<DT_I8, false>::find(epi, wmn, nm, l, i);
}
}  // namespace gemm_epi
