"""The compiled checks put in place by the first call, whichever thread makes it."""
import os
import subprocess
import sys

import pytest

from activation_epilogue_tcgen05_b200 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# torch's look-ups replaced, so that a machine without a GPU gets as far as the checks; device -1 is the CPU's
START = """
import sys, threading
import torch
from activation_epilogue_tcgen05_b200 import gemm_epi as g
torch.cuda.current_device, torch._C._cuda_getCurrentRawStream = (lambda: -1), (lambda device: 5)
BF16, flat = torch.bfloat16, torch.zeros(256, dtype=torch.bfloat16)
python = g._operand, g._device_and_stream
"""


def run(code):
    assert build.build_operands()
    r = subprocess.run([sys.executable, "-c", START + code], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
    return r.stdout


def test_first_calls_of_many_threads():
    """After each round of first calls, what the compiled form hands on still ends in the Python form: flat shapes and refusals."""
    run("""
sys.setswitchinterval(1e-6)
for turn in range(300):
    g._operand, g._device_and_stream, g._current = *python, None
    if sys.modules.pop("activation_epilogue_tcgen05_b200._operands", None):        # the import is part of a first call
        del sys.modules["activation_epilogue_tcgen05_b200"]._operands
    gate, wrong = threading.Barrier(16), []
    def first():
        gate.wait()
        try:
            assert g._device_and_stream(7) == (-1, 7)
        except BaseException as e:
            wrong.append(e)
    threads = [threading.Thread(target=first) for _ in range(16)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not wrong, (turn, wrong[0])
    _operands = sys.modules["activation_epilogue_tcgen05_b200._operands"]
    assert g._operand is _operands.operand and g._device_and_stream is _operands.device_and_stream
    assert g._operand(flat, "X", BF16, (4, 64), -1) == flat.data_ptr(), turn
    assert g._device_and_stream(7) == (-1, 7)
    try:
        g._operand(flat, "X", BF16, (4, 32), -1)
        raise SystemExit("accepted")
    except g.GemmEpiError as e:
        assert e.status == g.ERR_ARG
""")


def test_the_compiled_forms_are_not_taken_for_the_python_ones():
    run("""
assert g._device_and_stream(7) == (-1, 7)
from activation_epilogue_tcgen05_b200 import _operands
for forms in ((_operands.operand, g._device_and_stream), (python[0], _operands.device_and_stream), (_operands.operand, python[1]), (3, python[1])):
    try:
        _operands.set_python_forms(*forms)
        raise SystemExit(f"taken: {forms}")
    except TypeError:
        pass
assert g._operand(flat, "X", BF16, (4, 64), -1) == flat.data_ptr() and g._device_and_stream(7) == (-1, 7)
""")


def test_the_names_stand_for_the_python_forms_until_then():
    assert "function" in run("print(type(g._operand).__name__, g._compiled_checks(), g._compiled_checks(), type(g._operand).__name__)")
