"""The compiled checks of operands against the Python ones (CPU tensors: the device index of one is -1)."""
import itertools

import pytest
import torch

from activation_epilogue_tcgen05_b200 import build, gemm_epi as g

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def forms():
    """(Python form, compiled form) of _operand."""
    assert build.build_operands()
    from activation_epilogue_tcgen05_b200 import _operands
    python = g._operand
    if g._compiled_checks() and python is _operands.operand:
        pytest.skip("the compiled form is in place already: its Python form is not at hand")
    yield python, _operands.operand
    assert g._operand is _operands.operand


def outcome(f, *args):
    try:
        return f(*args)
    except g.GemmEpiError as e:
        return e.status, str(e)


def test_the_compiled_form_answers_as_the_python_form(forms):
    python, compiled = forms
    wide = torch.zeros(8, 64, dtype=BF16)
    tensors = [torch.zeros(4, 64, dtype=BF16), torch.zeros(256, dtype=BF16), torch.zeros(2, 2, 64, dtype=BF16), torch.zeros(64, 4, dtype=BF16),
               torch.zeros(64, 4, dtype=BF16).t(), wide[:4], wide[::2], wide[2:6, :], torch.zeros(4, 64), torch.zeros(4, 64, dtype=torch.int8),
               torch.nn.Parameter(torch.zeros(4, 64, dtype=BF16)), torch.zeros(4, 64, dtype=BF16, device="meta"), torch.zeros(0, 64, dtype=BF16),
               torch.zeros((), dtype=BF16), torch.zeros(4, 64, dtype=BF16).to_sparse(), None]
    for t, shape, device, optional in itertools.product(tensors, [(4, 64), (256,), (0, 64), ()], [-1, 0], [False, True]):
        args = (t, "Op.run: X", BF16, shape, device, optional)
        assert outcome(compiled, *args) == outcome(python, *args), args[1:] + (None if t is None else t.shape,)
    assert compiled(tensors[0], "X", BF16, (4, 64), -1) == tensors[0].data_ptr() and compiled(wide[2:6], "X", BF16, (4, 64), -1) == wide[2:].data_ptr()


def test_what_is_no_tensor_is_an_error(forms):
    python, compiled = forms
    for args in [(5, "X", BF16, (4, 64), -1), (torch.zeros(4, 64, dtype=BF16), "X", None, (4, 64), -1), (torch.zeros(4, 64, dtype=BF16), "X", BF16, [4, 64], -1),
                 (torch.zeros(4, 64, dtype=BF16), "X", BF16, (1 << 80, 64), -1), (torch.zeros(4),), ()]:
        got = []
        for f in (python, compiled):
            try:
                got.append(f(*args))
            except Exception as e:                    # noqa: BLE001 (the same kind from either)
                got.append(type(e))
        assert got[0] == got[1], args


def test_the_stream_without_a_device(forms):
    from activation_epilogue_tcgen05_b200 import _operands
    if torch.cuda.is_available():
        device, stream = _operands.device_and_stream(None)
        assert (device, stream) == (torch.cuda.current_device(), torch.cuda.current_stream().cuda_stream)
    else:
        with pytest.raises((RuntimeError, AssertionError)):
            _operands.device_and_stream(None)
