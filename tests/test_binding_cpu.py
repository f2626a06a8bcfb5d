"""The compiled checks of operands beside the Python ones: what memory they hand out, and where they stand aside."""
import pytest
import torch

from activation_epilogue_tcgen05_b200 import build, gemm_epi as g

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def compiled():
    assert build.build_operands() and g._compiled_checks()
    from activation_epilogue_tcgen05_b200 import _operands
    return _operands


@pytest.mark.parametrize("form", ["compiled", "python"])
def test_a_lazy_clone_gets_memory_of_its_own(compiled, form):
    """A kernel may write where an operand lies: a copy-on-write tensor's memory is its own by then, as data_ptr() has it."""
    operand = compiled.operand if form == "compiled" else g._python_forms[0]
    source = torch.arange(256, dtype=BF16).view(4, 64)
    clone = torch._lazy_clone(source)
    at = operand(clone, "X", BF16, (4, 64), -1)
    assert at == clone.data_ptr() and at != source.data_ptr() and not torch._C._is_cow_tensor(clone) and torch.equal(clone, source)
