"""The layer norm, 8-bit integer products and 8-bit checkpoints on a machine without a GPU: refusals (made before the device is
looked at), scratch sizes, plan choices, and the 64-bit formulas against differences."""
import ctypes

import pytest
import torch

import block8_ref as ref8
from block_ref import act

P = 0x10000          # an aligned address that no call here reads


@pytest.fixture(scope="module")
def g():
    from activation_epilogue_tcgen05_b200 import build, gemm_epi
    build.build()
    gemm_epi.lib()
    return gemm_epi


def ln_rc(g, m=4, d=64, dtype=1, out=0, eps=1e-5, X=P, R=None, gamma=P, beta=None, S=None, Y=2 * P, scale=None, amax=None):
    return g.lib().gemm_epi_layernorm(m, d, dtype, out, eps, X, R, gamma, beta, S, Y, scale, amax, None)


def bwd_rc(g, m=4, d=64, dtype=1, eps=1e-5, dY=P, S=P, gamma=P, dS=None, dX=P, dgamma=None, dbeta=None, ws=None):
    return g.lib().gemm_epi_layernorm_bwd(m, d, dtype, eps, dY, S, gamma, dS, dX, dgamma, dbeta, ws, None)


def quant_rc(g, m=4, d=64, dtype=1, out=4, X=P, Q=2 * P, scale=P):
    return g.lib().gemm_epi_quant_rows(m, d, dtype, out, X, Q, scale, None)


def save_rc(g, m=4, n=64, dtype=1, epi=4, Z=P, H=2 * P, codes=3 * P, exps=4 * P):
    return g.lib().gemm_epi_ckpt_save(m, n, dtype, epi, Z, H, codes, exps, None)


def load_rc(g, m=4, n=64, dtype=1, epi=4, codes=3 * P, exps=4 * P, X=P):
    return g.lib().gemm_epi_ckpt_load(m, n, dtype, epi, codes, exps, X, None)


def dact_rc(g, m=4, n=64, dtype=1, epi=4, axis=1, dD=P, codes=3 * P, exps=4 * P, dZ=P, H=None, dbias=None, ws=None):
    return g.lib().gemm_epi_dact_ckpt(m, n, dtype, epi, axis, dD, codes, exps, dZ, H, dbias, ws, None)


SIZES = [(dict(m=0), "ERR_ARG"), (dict(m=-1), "ERR_ARG"), (dict(m=1 << 31), "ERR_ARG"), (dict(dtype=-1), "ERR_ARG"), (dict(dtype=3), "ERR_ARG"),
         (dict(dtype=4), "ERR_ARG")]


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(d=0), "ERR_ARG"), (dict(dtype=2), "ERR_ARG"), (dict(out=3), "ERR_ARG"), (dict(out=5), "ERR_ARG"), (dict(out=-1), "ERR_ARG"),
    (dict(eps=0.0), "ERR_ARG"), (dict(eps=float("nan")), "ERR_ARG"), (dict(eps=float("inf")), "ERR_ARG"), (dict(d=60), "ERR_ALIGN"),
    (dict(d=72, out=4, scale=P), "ERR_ALIGN"), (dict(d=16392), "ERR_UNSUPPORTED"), (dict(X=None), "ERR_NULL"), (dict(gamma=None), "ERR_NULL"),
    (dict(Y=None), "ERR_NULL"), (dict(out=1), "ERR_NULL"), (dict(out=4), "ERR_NULL"), (dict(S=3 * P), "ERR_ARG"), (dict(R=P, S=2 * P), "ERR_ARG"),
    (dict(out=4, scale=P, Y=P), "ERR_ARG"), (dict(out=2, scale=P, R=2 * P), "ERR_ARG"), (dict(X=P + 8), "ERR_ALIGN"),
    (dict(beta=P + 8), "ERR_ALIGN"), (dict(gamma=P + 4), "ERR_ALIGN"), (dict(Y=P + 8), "ERR_ALIGN"), (dict(out=4, scale=P + 2), "ERR_ALIGN")])
def test_layer_norm_refusals(g, kw, code):
    assert ln_rc(g, **kw) == getattr(g, code)


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(d=-8), "ERR_ARG"), (dict(eps=0.0), "ERR_ARG"), (dict(d=4), "ERR_ALIGN"), (dict(d=16392), "ERR_UNSUPPORTED"), (dict(dY=None), "ERR_NULL"),
    (dict(S=None), "ERR_NULL"), (dict(gamma=None), "ERR_NULL"), (dict(dX=None), "ERR_NULL"), (dict(m=2000, dgamma=P), "ERR_NULL"),
    (dict(m=2000, dbeta=P), "ERR_NULL"), (dict(dgamma=P, dbeta=P), "ERR_ARG"), (dict(dY=P + 8), "ERR_ALIGN"), (dict(dbeta=P + 8), "ERR_ALIGN"),
    (dict(dgamma=P, ws=P + 4), "ERR_ALIGN")])
def test_layer_norm_bwd_refusals(g, kw, code):
    assert bwd_rc(g, **kw) == getattr(g, code)


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(dtype=2), "ERR_ARG"), (dict(d=0), "ERR_ARG"), (dict(d=1 << 31), "ERR_ARG"), (dict(out=0), "ERR_ARG"), (dict(out=1), "ERR_ARG"),
    (dict(out=3), "ERR_ARG"), (dict(d=72), "ERR_ALIGN"), (dict(X=None), "ERR_NULL"), (dict(Q=None), "ERR_NULL"), (dict(scale=None), "ERR_NULL"),
    (dict(Q=P), "ERR_ARG"), (dict(X=P + 8), "ERR_ALIGN"), (dict(Q=P + 8), "ERR_ALIGN"), (dict(scale=P + 1), "ERR_ALIGN")])
def test_quant_rows_refusals(g, kw, code):
    assert quant_rc(g, **kw) == getattr(g, code)


SHARED = SIZES + [(dict(n=0), "ERR_ARG"), (dict(n=1 << 31), "ERR_ARG"), (dict(epi=10), "ERR_ARG"), (dict(epi=-1), "ERR_ARG"), (dict(n=60), "ERR_ALIGN"),
                  (dict(m=1 << 27, n=1 << 10), "ERR_UNSUPPORTED"), (dict(codes=None), "ERR_NULL"), (dict(exps=None), "ERR_NULL"),
                  (dict(codes=P + 8), "ERR_ALIGN")]


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(Z=None), "ERR_NULL"), (dict(codes=P), "ERR_ARG"), (dict(codes=2 * P), "ERR_ARG"), (dict(exps=P), "ERR_ARG"), (dict(exps=2 * P), "ERR_ARG"),
    (dict(exps=3 * P), "ERR_ARG"), (dict(Z=P + 8), "ERR_ALIGN"), (dict(H=P + 8), "ERR_ALIGN")])
def test_save_refusals(g, kw, code):
    assert save_rc(g, **kw) == getattr(g, code)


@pytest.mark.parametrize("kw,code", SHARED + [(dict(X=None), "ERR_NULL"), (dict(X=3 * P), "ERR_ARG"), (dict(X=4 * P), "ERR_ARG"), (dict(X=P + 8), "ERR_ALIGN")])
def test_load_refusals(g, kw, code):
    assert load_rc(g, **kw) == getattr(g, code)


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(axis=2), "ERR_ARG"), (dict(epi=0), "ERR_ARG"), (dict(epi=1), "ERR_ARG"), (dict(epi=3), "ERR_ARG"), (dict(epi=7), "ERR_ARG"),
    (dict(dD=None), "ERR_NULL"), (dict(dZ=None), "ERR_NULL"), (dict(m=2000, dbias=P), "ERR_NULL"), (dict(H=P), "ERR_ARG"), (dict(dZ=3 * P), "ERR_ARG"),
    (dict(H=3 * P), "ERR_ARG"), (dict(H=4 * P), "ERR_ARG"), (dict(dD=P + 8), "ERR_ALIGN"), (dict(H=P + 8), "ERR_ALIGN"), (dict(dbias=P + 2, ws=P), "ERR_ALIGN")])
def test_dact_ckpt_refusals(g, kw, code):
    assert dact_rc(g, **kw) == getattr(g, code)


def test_valid_calls_without_a_gpu_report_no_device(g):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    none = g.ERR_NO_DEVICE
    assert ln_rc(g) == ln_rc(g, beta=P, R=P, S=P) == ln_rc(g, out=4, scale=P) == ln_rc(g, Y=P) == none
    assert bwd_rc(g) == bwd_rc(g, dgamma=P) == bwd_rc(g, dbeta=P) == bwd_rc(g, m=2000, dgamma=P, dbeta=2 * P, ws=P, dS=P) == none
    assert quant_rc(g) == quant_rc(g, out=2) == quant_rc(g, d=1 << 20) == none
    assert save_rc(g) == save_rc(g, H=None) == save_rc(g, H=P) == save_rc(g, epi=0) == save_rc(g, dtype=2) == load_rc(g) == load_rc(g, epi=1) == none
    assert dact_rc(g) == dact_rc(g, H=2 * P, dbias=P, ws=P) == dact_rc(g, dZ=2 * P, H=P) == none
    assert g.lib().gemm_epi_rmsnorm(4, 64, 1, 4, 1e-6, P, None, P, None, 2 * P, P, None, None) == none


def test_sizes(g):
    assert [g.gemm_epi_ckpt_groups(n) for n in (-1, 0, 1, 8, 32, 40, 4104, 1 << 31)] == [0, 0, 1, 1, 1, 2, 129, 0]
    ws = g.gemm_epi_layernorm_workspace_bytes
    assert ws(0, 64) == ws(4, 60) == ws(4, 16392) == ws(1 << 31, 64) == 0
    assert ws(8192, 4096) == 148 * 2 * 4096 * 4                # one block an SM, two rows of sums each
    assert ws(16, 4096) == ws(64, 1024) == 0                   # one cluster
    for m, d in [(17, 4096), (300, 4096), (2000, 64), (40000, 128), (5, 16384)]:
        assert ws(m, d) % (8 * d) == 0 and 0 < ws(m, d) <= 148 * 8 * d


def plan_rc(g, m, n, k, epi=1, layout=0, opts=None):
    h = ctypes.c_void_p()
    return g.lib().gemm_epi_plan_opts(m, n, k, g.I8, epi, 1, layout, ctypes.byref(opts) if opts else None, ctypes.byref(h))


def test_plans_of_8_bit_integers(g):
    opts = lambda **kw: g.Options(**{**dict(kernel=0, block_n=0, split_k=0, max_ctas=0, inject_stall=0, stream_k=0, out_e4m3=0), **kw})  # noqa: E731
    assert plan_rc(g, 64, 64, 40) == plan_rc(g, 64, 56, 64) == g.ERR_ALIGN
    assert plan_rc(g, 64, 64, 131072) == g.ERR_UNSUPPORTED
    assert plan_rc(g, 64, 64, 64, epi=10) == plan_rc(g, 64, 64, 64, epi=11) == plan_rc(g, 64, 64, 64, layout=2) == g.ERR_UNSUPPORTED
    assert plan_rc(g, 64, 64, 64, opts=opts(out_e4m3=1)) == plan_rc(g, 640, 512, 64, opts=opts(block_n=512)) == g.ERR_UNSUPPORTED
    if not torch.cuda.is_available():
        for epi in range(10):
            assert plan_rc(g, 64, 64, 131056, epi=epi) == plan_rc(g, 500, 272, 528, epi=epi, layout=1) == g.ERR_NO_DEVICE
    L, h = g.lib(), ctypes.c_void_p()
    assert L.gemm_epi_mlp_plan(64, 64, 128, g.I8, 4, 0, ctypes.byref(h)) == g.ERR_UNSUPPORTED
    assert L.gemm_epi_run_noalloc(64, 64, 64, g.I8, 1, 0, 0, P, P, P, P, P, P, None, 0, None) == g.ERR_ARG
    for bad in (None, ctypes.c_void_p(0x1000)):
        assert L.gemm_epi_run_scaled(bad, P, P, P, None, P, P, P, None, None) == g.ERR_ARG


def test_plans_choose_as_for_e4m3(g):
    """One byte an element: the same kernels, tiles and splits, without the 512-wide ones."""
    for m, n, k, layout in [(1, 4096, 4096, "nk"), (16, 4096, 14336, "kn"), (64, 6144, 4096, "nk"), (65, 4096, 4096, "kn"), (777, 1040, 528, "nk"),
                            (8192, 14336, 4096, "kn"), (8192, 4096, 14336, "nk"), (65536, 8192, 16384, "kn")]:
        a, b = (g.plan_preview(m, n, k, t, "gelu_bias", "col", layout) for t in ("e4m3", "i8"))
        for key in ("kernel", "block_m", "block_n", "block_k", "split_k", "grid", "cluster", "tiles", "sk_tiles", "sk_split", "group_m", "group_n"):
            assert a[key] == b[key], (m, n, k, key)


# ------------------------------------------------------------------ the formulas
@pytest.mark.parametrize("mean", [0.0, 30.0])
def test_layer_norm_gradients_against_differences(mean):
    gen = torch.Generator().manual_seed(1)
    m, d, eps, h = 3, 12, 1e-3, 1e-6
    s, dy, gamma, beta = (torch.randn(*k, generator=gen, dtype=torch.float64) for k in ((m, d), (m, d), (d,), (d,)))
    s = s + mean
    dx, dg, db, *_ = ref8.layer_norm_bwd(dy, s, gamma, None, eps)
    loss = lambda s, gamma, beta: float((ref8.layer_norm(s, None, gamma, beta, eps)[1] * dy).sum())  # noqa: E731
    for got, k in ((dx, 0), (dg, 1), (db, 2)):
        for i in range(got.numel()):
            args = [s.clone(), gamma.clone(), beta.clone()]
            args[k].view(-1)[i] += h
            up = loss(*args)
            args[k].view(-1)[i] -= 2 * h
            assert abs((up - loss(*args)) / (2 * h) - float(got.view(-1)[i])) < 1e-6


def test_checkpoint_formula():
    """The kept z is within half a step of z, the step at most 1/64 of the largest magnitude; powers of two and their borders."""
    gen = torch.Generator().manual_seed(2)
    z = torch.randn(40, 96, generator=gen, dtype=torch.float64) * torch.exp2(torch.randint(-20, 20, (40, 3), generator=gen).double()).repeat_interleave(32, 1)
    z[:, 0], z[:, 32], z[:, 64] = 2.0 ** 9, 127 * 2.0 ** 4, 127.5 * 2.0 ** 4
    q, e, k = ref8.checkpoint(z)
    step = torch.exp2(e - 133).repeat_interleave(32, 1)
    assert (q.abs() <= 127).all() and ((k - z).abs() <= step / 2).all() and torch.equal(k, ref8.kept(q, e))
    top = z.view(40, 3, 32).abs().amax(2).repeat_interleave(32, 1)
    assert (step <= top / 63.4).all() and (step >= top / 127).all()
    only = torch.zeros(3, 32, dtype=torch.float64)
    only[0, 0], only[1, 0], only[2, 0] = 64.0, 127.0, 127.5
    assert ref8.checkpoint(only)[1].view(-1).tolist() == [133, 133, 134]
    assert ref8.checkpoint(torch.zeros(1, 40, dtype=torch.float64))[1].tolist() == [[7, 7]]


def test_product_formula():
    gen = torch.Generator().manual_seed(3)
    a, b = (torch.randint(-128, 128, k, generator=gen).to(torch.int8) for k in ((5, 16), (16, 8)))
    rows, cols, bias, r = (torch.rand(k, generator=gen) for k in (5, 8, 8, (5, 8)))
    x, _, y, _ = ref8.product_i8(a, b, rows, cols, bias, "col", "gelu_bias", r)
    want = sum(int(a[2, k]) * int(b[k, 3]) for k in range(16)) * float(rows[2]) * float(cols[3]) + float(bias[3])
    assert abs(float(x[2, 3]) - want) < 1e-9 and abs(float(y[2, 3]) - (float(act("gelu", torch.tensor(want, dtype=torch.float64))) + float(r[2, 3]))) < 1e-9
