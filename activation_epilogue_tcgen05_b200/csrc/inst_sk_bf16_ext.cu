// Instantiations of the small-m split-K kernel with the extended epilogue, bf16 operands.
#include "find_ext.cuh"
namespace gemm_epi {
bool find_sk_bf16_ext(int epi, bool wmn, int nm, SkLauncher *l, KernelInfo *i) {
    return SkFindExt<DT_BF16, false>::find(epi, wmn, nm, l, i);
}
}  // namespace gemm_epi
