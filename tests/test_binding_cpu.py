"""The compiled checks of operands beside the Python ones: what memory they hand out, and where they stand aside."""
import os
import subprocess
import sys

import pytest
import torch

from activation_epilogue_tcgen05_b200 import build, gemm_epi as g

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def compiled():
    assert build.build_operands()
    from activation_epilogue_tcgen05_b200 import _operands
    _operands.set_python_forms(*g._python_forms)          # (as the first call does, which also puts the compiled forms in place)
    return _operands


def fresh(code):
    """Run in a process where nothing has been put in place yet."""
    r = subprocess.run([sys.executable, "-c", "import torch\nfrom activation_epilogue_tcgen05_b200 import build, gemm_epi as g\n" + code],
                       cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]


@pytest.mark.parametrize("form", ["compiled", "python"])
def test_a_lazy_clone_gets_memory_of_its_own(compiled, form):
    """A kernel may write where an operand lies: a copy-on-write tensor's memory is its own by then, as data_ptr() has it."""
    operand = compiled.operand if form == "compiled" else g._python_forms[0]
    source = torch.arange(256, dtype=BF16).view(4, 64)
    clone = torch._lazy_clone(source)
    at = operand(clone, "X", BF16, (4, 64), -1)
    assert at == clone.data_ptr() and at != source.data_ptr() and not torch._C._is_cow_tensor(clone) and torch.equal(clone, source)


def test_a_module_that_was_built_for_another_torch_stands_aside(compiled):
    assert torch.__version__ in compiled.built_for and sys.version in compiled.built_for
    fresh("""
from activation_epilogue_tcgen05_b200 import _operands
right, _operands.built_for = _operands.built_for, _operands.built_for.replace(torch.__version__, "1.0")
assert not g._compiled_checks() and (g._operand, g._device_and_stream) == g._python_forms
_operands.built_for = right
assert g._compiled_checks() and g._operand is _operands.operand
""")


def test_without_its_python_forms_the_module_says_so(compiled):
    fresh("""
from activation_epilogue_tcgen05_b200 import _operands
for call in (lambda: _operands.operand(None, "X", torch.int8, (4,), -1), lambda: _operands.device_and_stream(7)):
    try:
        call()
        raise SystemExit("went on")
    except RuntimeError as e:
        assert "set_python_forms" in str(e)
""")
