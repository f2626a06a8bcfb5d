"""What the header promises of the norm, the extended epilogue and the epilogue's backward beyond their formulas:
what the reported maximum counts, which scales are read, the limits of the arguments, values far from one."""
import math

import pytest
import torch


from activation_epilogue_tcgen05_b200 import gemm_epi as g

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.get_device_capability() != (10, 0):
        pytest.skip("needs sm_100")
    from activation_epilogue_tcgen05_b200 import build
    build.build()


def f32(*v):
    return torch.tensor(v, dtype=torch.float32, device="cuda")


# ------------------------------------------------------------------ the maximum of an e4m3 output
# A bias of 10 that the products take almost wholly away: |y| is at most 2.125 in D, and act(bias) = 10 in the rows and
# columns of a tile that D does not have.  Every value is a small multiple of 1/8, so fp32 holds each y exactly.
def cancelled(m, n, axis):
    a, b = torch.zeros(m, 32), torch.zeros(32, n)
    a[:, 3] = torch.tensor([0.875, 1.0, 1.125])[torch.arange(m) % 3]
    b[3] = -9.0
    y = 10.0 + a @ b
    bias = torch.full((m if axis == "row" else n,), 10.0, dtype=torch.bfloat16, device="cuda")
    return a.to(E4M3).cuda(), b.to(E4M3).cuda(), bias, y


# ------------------------------------------------------------------ scales
@pytest.mark.parametrize("out_e4m3", [False, True])
@pytest.mark.parametrize("m,kw", [(5, {}), (129, dict(kernel="tc1", block_n=128)), (300, dict(kernel="tc2", block_n=256))])
def test_row_scales_take_the_place_of_the_scale_of_a(m, kw, out_e4m3):
    """With one scale a row s_A is not read: whatever it holds, the same bits."""
    a, b, bias, _ = cancelled(m, 272, "col")
    rows, got = torch.linspace(0.25, 1.0, m, device="cuda"), []
    with g.Plan(m, 272, 32, "e4m3", "gelu_bias", "col", out_e4m3=out_e4m3, **kw) as p:
        for sa in (1.0, 3.0, math.nan, math.inf):
            s, sb, so, amax = f32(sa), f32(1), f32(0.0625), f32(0)
            p.set_scales(s, sb)
            if out_e4m3:
                p.set_out_scale(so, amax)
            D = torch.zeros(m, 272, dtype=E4M3 if out_e4m3 else torch.bfloat16, device="cuda")
            p.run_ext(a, b, bias, D, scale_rows=rows)
            p.check()
            got.append((D.view(torch.uint8), amax))
    for D, amax in got[1:]:
        assert torch.equal(D, got[0][0]) and torch.equal(amax, got[0][1])
