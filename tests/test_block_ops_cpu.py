"""The norm and the epilogue's backward on a machine without a GPU: refusals (made before the device
is looked at), scratch sizes, and the 64-bit formulas against differences."""
import ctypes

import pytest
import torch

import block_ref as ref

P = 0x10000          # an aligned address that no call here reads


@pytest.fixture(scope="module")
def g():
    from activation_epilogue_tcgen05_b200 import build, gemm_epi
    build.build()
    gemm_epi.lib()
    return gemm_epi


def norm_rc(g, m=4, d=64, dtype=1, out=0, eps=1e-6, X=P, R=None, gamma=P, S=None, Y=2 * P, scale=None, amax=None):
    return g.lib().gemm_epi_rmsnorm(m, d, dtype, out, eps, X, R, gamma, S, Y, scale, amax, None)


def bwd_rc(g, m=4, d=64, dtype=1, eps=1e-6, dY=P, S=P, gamma=P, dS=None, dX=P, dgamma=None, ws=None):
    return g.lib().gemm_epi_rmsnorm_bwd(m, d, dtype, eps, dY, S, gamma, dS, dX, dgamma, ws, None)


def dact_rc(g, m=4, n=64, dtype=1, epi=4, axis=1, dD=P, Z=P, aux=None, dZ=P, dbias=None, ws=None):
    return g.lib().gemm_epi_dact(m, n, dtype, epi, axis, dD, Z, aux, dZ, dbias, ws, None)


@pytest.mark.parametrize("kw,code", [
    (dict(m=0), "ERR_ARG"), (dict(m=-1), "ERR_ARG"), (dict(d=0), "ERR_ARG"), (dict(m=1 << 31), "ERR_ARG"),
    (dict(dtype=2), "ERR_ARG"), (dict(dtype=-1), "ERR_ARG"), (dict(out=3), "ERR_ARG"), (dict(out=-1), "ERR_ARG"),
    (dict(eps=0.0), "ERR_ARG"), (dict(eps=-1e-6), "ERR_ARG"), (dict(eps=float("nan")), "ERR_ARG"),
    (dict(eps=float("inf")), "ERR_ARG"), (dict(d=60), "ERR_ALIGN"), (dict(d=72, out=2, scale=P), "ERR_ALIGN"),
    (dict(d=16392), "ERR_UNSUPPORTED"), (dict(X=None), "ERR_NULL"), (dict(gamma=None), "ERR_NULL"),
    (dict(Y=None), "ERR_NULL"), (dict(out=1), "ERR_NULL"), (dict(out=2), "ERR_NULL"),
    (dict(S=3 * P), "ERR_ARG"),                       # a sum without a residual
    (dict(R=P, S=2 * P), "ERR_ARG"),                  # S over Y
    (dict(out=2, scale=P, Y=P), "ERR_ARG"), (dict(out=1, scale=P, R=2 * P), "ERR_ARG"),
    (dict(X=P + 8), "ERR_ALIGN"), (dict(R=P + 2), "ERR_ALIGN"), (dict(gamma=P + 4), "ERR_ALIGN"),
    (dict(R=P, S=P + 8), "ERR_ALIGN"), (dict(Y=P + 8), "ERR_ALIGN"), (dict(out=2, scale=P + 2), "ERR_ALIGN"),
    (dict(out=1, scale=P, amax=P + 2), "ERR_ALIGN"),
])
def test_norm_refusals(g, kw, code):
    assert norm_rc(g, **kw) == getattr(g, code)


@pytest.mark.parametrize("kw,code", [
    (dict(m=0), "ERR_ARG"), (dict(d=-8), "ERR_ARG"), (dict(dtype=2), "ERR_ARG"), (dict(eps=0.0), "ERR_ARG"),
    (dict(d=4), "ERR_ALIGN"), (dict(d=16392), "ERR_UNSUPPORTED"), (dict(dY=None), "ERR_NULL"), (dict(S=None), "ERR_NULL"),
    (dict(gamma=None), "ERR_NULL"), (dict(dX=None), "ERR_NULL"), (dict(m=2000, dgamma=P), "ERR_NULL"),
    (dict(dY=P + 8), "ERR_ALIGN"), (dict(dS=P + 8), "ERR_ALIGN"), (dict(dgamma=P, ws=P + 4), "ERR_ALIGN"),
])
def test_norm_bwd_refusals(g, kw, code):
    assert bwd_rc(g, **kw) == getattr(g, code)


@pytest.mark.parametrize("kw,code", [
    (dict(m=0), "ERR_ARG"), (dict(n=0), "ERR_ARG"), (dict(dtype=3), "ERR_ARG"), (dict(epi=10), "ERR_ARG"),
    (dict(epi=-1), "ERR_ARG"), (dict(axis=2), "ERR_ARG"), (dict(n=60), "ERR_ALIGN"), (dict(dD=None), "ERR_NULL"),
    (dict(Z=None), "ERR_NULL"), (dict(epi=3), "ERR_NULL"), (dict(dZ=None), "ERR_NULL"), (dict(m=2000, dbias=P), "ERR_NULL"),
    (dict(epi=1, dZ=None), "ERR_NULL"), (dict(epi=1, dbias=P, ws=P), "ERR_ARG"), (dict(Z=P + 8), "ERR_ALIGN"),
    (dict(epi=7, aux=P + 4), "ERR_ALIGN"), (dict(dbias=P, ws=P + 8), "ERR_ALIGN"),
])
def test_dact_refusals(g, kw, code):
    assert dact_rc(g, **kw) == getattr(g, code)


def test_valid_calls_without_a_gpu_report_no_device(g):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert norm_rc(g) == norm_rc(g, R=P, S=P) == norm_rc(g, Y=P) == norm_rc(g, out=2, scale=P) == g.ERR_NO_DEVICE
    assert bwd_rc(g) == bwd_rc(g, dgamma=P, dS=P) == bwd_rc(g, m=2000, dgamma=P, ws=P, dS=P) == g.ERR_NO_DEVICE
    assert dact_rc(g) == dact_rc(g, epi=1, dZ=None, dbias=P, ws=P) == dact_rc(g, epi=3, aux=P, Z=None) == g.ERR_NO_DEVICE


def test_scratch_sizes(g):
    for m, d in [(1, 8), (37, 1000), (64, 1024), (16, 4096), (1024, 64)]:
        assert g.gemm_epi_rmsnorm_workspace_bytes(m, d) == 0         # one cluster: no partial rows
    for m, d in [(1, 16384), (65, 1024), (17, 4096), (1025, 64), (65537, 128), (2_000_000, 4096)]:
        b = g.gemm_epi_rmsnorm_workspace_bytes(m, d)
        assert b > 0 and b % (4 * d) == 0 and b // (4 * d) <= m      # whole rows of fp32, no more than the input's
        assert b <= 4 * d * 148 * 4
    assert g.gemm_epi_rmsnorm_workspace_bytes(0, 64) == g.gemm_epi_rmsnorm_workspace_bytes(4, 16392) == 0
    for m, n in [(1, 8), (1023, 4104), (8192, 14336), (1 << 20, 64), (16, 1 << 20), ((1 << 31) - 1, 8)]:
        col, row = (g.gemm_epi_dact_workspace_bytes(m, n, a) for a in (1, 0))
        assert row in (0, (n + 255) // 256 * m * 4)                  # 0: a block takes whole rows
        assert (row == 0) == (m >= 1776 or n <= 6144)
        runs = col // (4 * n)
        assert col == runs * 4 * n and runs != 1 and runs <= min(65535, (m + 31) // 32)      # 0: one run
        assert m > 64 or runs == 0
    assert g.gemm_epi_dact_workspace_bytes(4, 64, 2) == g.gemm_epi_dact_workspace_bytes(4, 0, 1) == 0
    assert g.gemm_epi_dact_workspace_bytes(4, 60, 1) == g.gemm_epi_rmsnorm_workspace_bytes(2000, 60) == 0


def test_objects_refuse_unknown_names(g):
    with pytest.raises(g.GemmEpiError):
        g.RmsNorm(4, 64, "e4m3")
    with pytest.raises(KeyError):
        g.RmsNorm(4, 64, out="int8")
    with pytest.raises(KeyError):
        g.ActBackward(4, 64, "bf16", "swish")


def test_norm_formula_against_differences():
    gen = torch.Generator().manual_seed(3)
    x, r, dy, v = (torch.randn(5, 24, generator=gen, dtype=torch.float64) for _ in range(4))
    gamma, w = (torch.randn(24, generator=gen, dtype=torch.float64) for _ in range(2))
    dx, dg, _, _ = ref.norm_bwd(dy, x + r, gamma, None, 1e-3)

    def f(t, u):
        return float((ref.norm(x + t * v, r, gamma + u * w, 1e-3)[1] * dy).sum())

    h = 1e-5
    assert abs((f(h, 0) - f(-h, 0)) / (2 * h) - float((dx * v).sum())) < 1e-7
    assert abs((f(0, h) - f(0, -h)) / (2 * h) - float((dg * w).sum())) < 1e-7


@pytest.mark.parametrize("name", ["gelu_bias", "tanh", "relu_bias", "bias"])
def test_slopes_against_differences(name):
    z = torch.linspace(-4, 4, 801, dtype=torch.float64) + 0.003
    h = 1e-5
    diff = (ref.act(name, z + h) - ref.act(name, z - h)) / (2 * h)
    assert float((diff - ref.act_slope(name, z)).abs().max()) < 1e-8


def test_extended_entry_points_reject_bad_handles(g):
    for bad in (None, ctypes.c_void_p(0x1000)):
        assert g.lib().gemm_epi_run_ext(bad, P, P, P, P, None, P, None, None) == g.ERR_ARG
        assert g.lib().gemm_epi_run_ext(bad, P, P, P, None, None, P, None, None) == g.ERR_ARG
        assert g.lib().gemm_epi_mlp_run_prenorm(bad, P, P, P, 1e-6, P, P, P, P, P, P, None, P, P, None) == g.ERR_ARG
