"""What the objects take for an operand's shape (CPU tensors: the device index of one is -1)."""
import pytest
import torch

from activation_epilogue_tcgen05_b200 import gemm_epi as g

BF16 = torch.bfloat16


@pytest.mark.parametrize("shape", [(4, 64), (256,), (2, 2, 64), (4, 8, 8), (1, 4, 64), (4, 64, 1), (2, 2, 4, 16), (1, 1, 4, 64)])
def test_shapes_of_the_same_rows(shape):
    t = torch.zeros(shape, dtype=BF16)
    assert g._operand(t, "t", BF16, (4, 64), -1) == t.data_ptr()


@pytest.mark.parametrize("shape", [(64, 4), (8, 32), (32, 8), (2, 128), (2, 64, 2), (16, 16), (4, 65), (255,), (0, 64), ()])
def test_other_shapes_are_refused(shape):
    with pytest.raises(g.GemmEpiError) as e:
        g._operand(torch.zeros(shape, dtype=BF16), "t", BF16, (4, 64), -1)
    assert e.value.status == g.ERR_ARG


def test_vectors_and_single_rows():
    for shape in ((64,), (1, 64), (64, 1), (8, 8)):
        t = torch.zeros(shape, dtype=BF16)
        assert g._operand(t, "t", BF16, (64,), -1) == t.data_ptr()
        assert g._operand(t, "t", BF16, (1, 64), -1) == t.data_ptr()
    for shape in ((), (1,), (1, 1)):
        assert g._operand(torch.zeros(shape), "t", torch.float32, (1,), -1)
    for bad in (torch.zeros(63, dtype=BF16), torch.zeros(64), torch.zeros(8, 16, dtype=BF16)[:, ::2], torch.zeros(2, 64, dtype=BF16)):
        with pytest.raises(g.GemmEpiError):
            g._operand(bad, "t", BF16, (64,), -1)
    assert g._operand(None, "t", BF16, (64,), -1, True) is None
    with pytest.raises(g.GemmEpiError) as e:
        g._operand(None, "t", BF16, (64,), -1)
    assert e.value.status == g.ERR_NULL
