"""Products of 8-bit integers with scales for each token and channel on the GPU, against the formula in 64 bits: the sums are exact,
so the bounds are those of the epilogue's few fp32 operations and the one rounding of D.  And the operators of 8 bits run
together as a block uses them."""
import numpy as np
import pytest
import torch

import block8_ref as ref
import block_ref
from block_ref import close, rounded
from helpers import aux_padding_bits, unpack_aux
from test_gpu_block_ops import Guarded, _cuda, randn  # noqa: F401

from activation_epilogue_tcgen05_b200 import gemm_epi as g

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def codes(m, k, seed, low=-128):
    return torch.randint(low, 128, (m, k), generator=torch.Generator().manual_seed(seed)).to(torch.int8).cuda()


def scales(count, seed):
    return torch.exp(torch.randn(count, generator=torch.Generator().manual_seed(seed))).cuda() / 2000


def problem(m, n, k, epilogue, axis, layout, seed=0):
    a, b = codes(m, k, seed), codes(*((k, n) if layout == "kn" else (n, k)), seed + 1)
    bias = randn(m if axis == "row" else n, seed=seed + 2) if epilogue in g.HAS_BIAS else None
    return a, b, scales(m, seed + 3), scales(n, seed + 4), bias


def run(m, n, k, epilogue="bias", axis="col", layout="kn", residual=False, in_place=False, seed=0, plan_args={}, stream=None, plan=None):
    a, b, rows, cols, bias = problem(m, n, k, epilogue, axis, layout, seed)
    R = randn(m, n, seed=seed + 5) if residual else None
    D = Guarded(m * n, BF16)
    if in_place:
        D.t.copy_(R.view(-1))
    aux = torch.full((m, g.aux_pitch_words(n)), -1, dtype=torch.int32, device="cuda") if epilogue in g.HAS_AUX else None
    own = plan or g.Plan(m, n, k, "i8", epilogue, axis, layout, **plan_args)
    own.run_i8(a, b, bias, D.t, rows, cols, residual=D.t if in_place else R, aux=aux, stream=stream)
    own.check(stream)
    info = own.info
    if plan is None:
        own.close()
    assert D.intact()
    cpu = lambda t: None if t is None else t.cpu()  # noqa: E731
    x, off, y, oy = ref.product_i8(a.cpu(), b.cpu() if layout == "kn" else b.cpu().t(), rows.cpu(), cols.cpu(), cpu(bias), axis, epilogue, cpu(R))
    close(D.t.view(m, n), y, rounded(y, "bf16", oy), "D")
    if aux is not None:
        words = aux.cpu().numpy().view(np.uint32)
        sure = (x.abs() > off).numpy()
        assert (unpack_aux(words, m, n) == (x > 0).numpy())[sure].all() and aux_padding_bits(words, m, n) == 0
    return D.t.view(m, n), info


EPILOGUES = ["none", "bias", "relu_bias", "relu_aux_bias", "gelu_bias", "tanh_bias", "relu", "relu_aux", "gelu", "tanh"]


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("kernel,args", [("tc1", dict(block_n=128)), ("tc1", dict(block_n=256)), ("tc2", dict(block_n=256)), ("splitk", {})])
@pytest.mark.parametrize("epilogue", EPILOGUES)
def test_every_kernel(kernel, args, layout, epilogue):
    m = 77 if kernel == "splitk" else 300
    for axis, residual in (("col", True), ("row", False)):
        run(m, 272, 336, epilogue, axis, layout, residual, plan_args=dict(kernel=kernel, **args))


def test_pairs_with_narrow_tiles():
    run(300, 272, 336, layout="nk", residual=True, plan_args=dict(kernel="tc2", block_n=128))
    with pytest.raises(g.GemmEpiError) as e:
        g.Plan(300, 272, 336, "i8", "bias", "col", "kn", kernel="tc2", block_n=128)
    assert e.value.status == g.ERR_UNSUPPORTED


@pytest.mark.parametrize("m,n,k", [(1, 16, 16), (1, 128, 4096), (2, 144, 16), (17, 1040, 272), (64, 4096, 1040), (65, 16, 144), (129, 2048, 16),
                                   (1000, 512, 2048), (777, 1040, 528), (2049, 1296, 400), (4100, 272, 144), (300, 8208, 272)])
@pytest.mark.parametrize("layout", ["kn", "nk"])
def test_sizes(m, n, k, layout):
    run(m, n, k, "gelu_bias", "col", layout, residual=True, seed=m)
    run(m, n, k, "none", layout=layout, seed=n)


@pytest.mark.parametrize("split", [1, 2, 3, 4, 8])
@pytest.mark.parametrize("m", [3, 16])
def test_split_sums_of_small_m(m, split):
    run(m, 400, 2064, "bias", "row", "nk", residual=True, plan_args=dict(kernel="splitk", split_k=split))


@pytest.mark.parametrize("m,split", [(30, 4), (60, 4), (100, 2)])
def test_split_sums_of_more_rows(m, split):
    run(m, 400, 2064, "gelu_bias", "col", "kn", residual=True, plan_args=dict(kernel="splitk", split_k=split))


@pytest.mark.parametrize("kernel", ["tc1", "tc2"])
def test_split_tails(kernel):
    _, info = run(700, 1536, 4112, "bias", "col", "nk", residual=True, plan_args=dict(kernel=kernel, stream_k="on"))
    assert info["sk_tiles"] > 0


@pytest.mark.parametrize("m", [16, 256])
def test_the_largest_sums(m):
    """k at its limit and every code -128 (2^31 - 2^18), or signs that alternate: int32 holds them."""
    k, n = 131056, 16
    a, b = torch.full((m, k), -128, dtype=torch.int8, device="cuda"), torch.full((n, k), -128, dtype=torch.int8, device="cuda")
    b[1] = 127
    b[2, ::2] = 127
    one = torch.ones(max(m, n), device="cuda")
    D = torch.empty(m, n, dtype=BF16, device="cuda")
    with g.Plan(m, n, k, "i8", "none", "col", "nk") as plan:
        plan.run_i8(a, b, None, D, one[:m], one[:n])
        plan.check()
    want = (a[:1].cpu().double() @ b.cpu().double().t()).to(torch.float32).to(BF16)
    assert torch.equal(D.cpu(), want.expand(m, n)) and float(want[0, 0]) == 2.0 ** 31


def test_exact_where_the_output_holds_the_sum():
    m, n, k = 200, 272, 1024
    gen = torch.Generator().manual_seed(1)
    a, b = (torch.randint(-1, 2, s, generator=gen).to(torch.int8) for s in ((m, k), (n, k)))
    D, one = torch.empty(m, n, dtype=BF16, device="cuda"), torch.ones(300, device="cuda")
    with g.Plan(m, n, k, "i8", "none", "col", "nk") as plan:
        plan.run_i8(a.cuda(), b.cuda(), None, D, one[:m], one[:n])
        plan.check()
    assert torch.equal(D.cpu(), (a.double() @ b.double().t()).to(BF16))


@pytest.mark.parametrize("m", [16, 500])
def test_residual_in_place_from_run_to_run_and_captured(m):
    first, _ = run(m, 1040, 2064, "gelu_bias", "col", "nk", residual=True, in_place=True)
    again, _ = run(m, 1040, 2064, "gelu_bias", "col", "nk", residual=True, in_place=False)
    assert torch.equal(first, again)
    a, b, rows, cols, bias = problem(m, 1040, 2064, "gelu_bias", "col", "nk")
    R, D = randn(m, 1040, seed=5), torch.empty(m, 1040, dtype=BF16, device="cuda")
    with g.Plan(m, 1040, 2064, "i8", "gelu_bias", "col", "nk") as plan:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        plan.run_i8(a, b, bias, D, rows, cols, residual=R, stream=side)
        side.synchronize()
        assert torch.equal(D, first)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            plan.run_i8(a, b, bias, D, rows, cols, residual=R)
        for _ in range(3):
            D.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(D, first)
        plan.check()
        del graph


def test_scales_that_are_not_finite_stay_in_their_row_and_column():
    m, n, k = 70, 272, 336
    a, b, rows, cols, _ = problem(m, n, k, "none", "col", "nk")
    for size in (m, 20):
        D = torch.empty(size, n, dtype=BF16, device="cuda")
        r, c = rows[:size].clone(), cols.clone()
        r[3], c[100] = float("nan"), float("nan")
        with g.Plan(size, n, k, "i8", "none", "col", "nk") as plan:
            plan.run_i8(a[:size].contiguous(), b, None, D, r, c)
            plan.check()
        lost = torch.zeros(size, n, dtype=torch.bool)
        lost[3], lost[:, 100] = True, True
        assert torch.equal(D.cpu().isnan(), lost)


def test_a_wait_that_runs_out_is_reported():
    a, b, rows, cols, bias = problem(300, 272, 336, "bias", "col", "kn")
    D, R = torch.zeros(300, 272, dtype=BF16, device="cuda"), randn(300, 272)
    with g.Plan(300, 272, 336, "i8", "bias", "col", "kn", kernel="tc1", inject_stall=1) as plan:
        plan.run_i8(a, b, bias, D, rows, cols, residual=R)
        with pytest.raises(g.GemmEpiError) as e:
            plan.check()
        assert e.value.status == g.ERR_TIMEOUT
    run(300, 272, 336, residual=True)


def test_calls_that_do_not_take_such_a_plan():
    a, b, rows, cols, bias = problem(64, 64, 64, "bias", "col", "kn")
    D, one = torch.zeros(64, 64, dtype=BF16, device="cuda"), torch.ones(64, device="cuda")
    with g.Plan(64, 64, 64, "i8", "bias", "col", "kn") as plan, g.Plan(64, 64, 64, "bf16", "bias", "col", "kn") as other:
        calls = [lambda: plan.run(a, b, bias, D), lambda: plan.run(a, b, bias, D, fused=False), lambda: plan.run_ext(a, b, bias, D, residual=D),
                 lambda: plan.run_ext(a, b, bias, D, scale_rows=rows), lambda: plan.set_scales(one, one), lambda: plan.run_bwd(a, b, D, D),
                 lambda: other.run_i8(a, b, bias, D, rows, cols), lambda: plan.run_i8(a, b, bias, D, rows, cols[:63]),
                 lambda: plan.run_i8(a, b, bias, D, rows.half(), cols), lambda: plan.run_i8(a.view(torch.uint8), b, bias, D, rows, cols),
                 lambda: g.gemm_epi_run_scaled(other.handle, a.data_ptr(), b.data_ptr(), bias.data_ptr(), None, rows.data_ptr(), cols.data_ptr(), D.data_ptr(), None, None)]
        for call in calls:
            with pytest.raises(g.GemmEpiError) as e:
                call()
            assert e.value.status == g.ERR_ARG
        args = [a.data_ptr(), b.data_ptr(), bias.data_ptr(), None, rows.data_ptr(), cols.data_ptr(), D.data_ptr(), None, None]
        for at, value, code in ((4, None, g.ERR_NULL), (5, None, g.ERR_NULL), (4, rows.data_ptr() + 2, g.ERR_ALIGN), (5, cols.data_ptr() + 4, g.ERR_ALIGN),
                                (3, D.data_ptr() + 2, g.ERR_ALIGN), (2, None, g.ERR_NULL), (0, None, g.ERR_NULL), (6, None, g.ERR_NULL)):
            bad = list(args)
            bad[at] = value
            assert g.lib().gemm_epi_run_scaled(plan.handle, *bad) == code
        torch.cuda.synchronize()
        assert not D.any()


def test_the_grid_wide_form_is_not_read(monkeypatch):
    monkeypatch.setenv("GEMM_EPI_SK_GRID", "1")
    _, info = run(16, 1040, 2064, "bias", "col", "nk", residual=True)
    assert info["cluster"] > 1


# ------------------------------------------------------------------ together
def quantised(w):
    """(codes, scales) of the rows of a weight (n, k), by the framework."""
    q, s = torch.empty(w.shape, dtype=torch.int8, device="cuda"), torch.empty(w.shape[0], device="cuda")
    g.QuantRows(*w.shape, out="i8_rows").run(w, q, s)
    return q, s


@pytest.mark.parametrize("m", [1, 16, 300])
def test_a_served_block(m):
    """Layer norm -> up-projection with GELU -> rows quantised -> down-projection into the residual stream, in 8-bit integers: each
    stage against the formula on what it was given, and the whole against the block in 64 bits on the weights that the codes stand for."""
    dm, ff = 512, 1552
    x, r, gamma, beta, b1, b2 = (randn(*s, seed=i) for i, s in enumerate([(m, dm), (m, dm), (dm,), (dm,), (ff,), (dm,)]))
    (q1, s1), (q2, s2) = quantised(randn(ff, dm, seed=7, scale=0.05)), quantised(randn(dm, ff, seed=8, scale=0.03))
    S, H, Y = torch.empty_like(x), torch.empty(m, ff, dtype=BF16, device="cuda"), torch.empty_like(x)
    n8, ns = torch.empty(m, dm, dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    h8, hs = torch.empty(m, ff, dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    norm, quant = g.LayerNorm(m, dm, out="i8_rows"), g.QuantRows(m, ff)
    with g.Plan(m, ff, dm, "i8", "gelu_bias", "col", "nk") as up, g.Plan(m, dm, ff, "i8", "bias", "col", "nk") as down:
        def block():
            norm.run(x, gamma, n8, beta=beta, residual=r, S=S, scale=ns)
            up.run_i8(n8, q1, b1, H, ns, s1)
            quant.run(H, h8, hs)
            down.run_i8(h8, q2, b2, Y, hs, s2, residual=S)

        block()
        up.check(), down.check()
        cpu = lambda *t: [v.cpu() for v in t]  # noqa: E731
        ref.check_layer_norm("i8_rows", "bf16", x, r, gamma, beta, 1e-5, n8, S, ns)
        a, w, sa, sw, b, h = cpu(n8, q1, ns, s1, b1, H)
        _, _, y, oy = ref.product_i8(a, w.t(), sa, sw, b, "col", "gelu_bias", None)
        close(h, y, rounded(y, "bf16", oy), "H")
        ref.check_out("i8_rows", "bf16", h.double(), 0 * h.double(), h8, hs)
        a, w, sa, sw, b, res = cpu(h8, q2, hs, s2, b2, S)
        _, _, y, oy = ref.product_i8(a, w.t(), sa, sw, b, "col", "bias", res)
        close(Y, y, rounded(y, "bf16", oy), "Y")
        # the whole: each operand is off by half a code (1/254 of its row's largest), which random signs average over a sum
        s, n, _ = ref.layer_norm(x.cpu(), r.cpu(), gamma.cpu(), beta.cpu(), 1e-5)
        w1, w2 = q1.cpu().double() * s1.cpu().double()[:, None], q2.cpu().double() * s2.cpu().double()[:, None]
        hh = block_ref.act("gelu", n @ w1.t() + b1.cpu().double())
        whole = hh @ w2.t() + b2.cpu().double() + s
        assert float((Y.cpu().double() - whole).norm() / whole.norm()) < 0.02
        first = Y.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            block()
        Y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, first)
        del graph


def test_a_trained_block():
    """Layer norm -> up-projection -> GELU, z kept in 8 bits; backward through GELU and norm from what was kept.  The gradients
    against those of the formula in 64 bits with the kept z; against those of z itself they are off by what half a code does."""
    m, dm, ff = 500, 256, 1032
    x, gamma, beta, b1, dH = (randn(*s, seed=i) for i, s in enumerate([(m, dm), (dm,), (dm,), (ff,), (m, ff)]))
    w = randn(ff, dm, seed=9, scale=0.06)
    n, z, h, hb, dz, dn, dx = (torch.empty(*s, dtype=BF16, device="cuda") for s in [(m, dm), (m, ff), (m, ff), (m, ff), (m, ff), (m, dm), (m, dm)])
    codes8, exps = torch.empty(m, ff, dtype=torch.int8, device="cuda"), torch.empty(m, 33, dtype=torch.uint8, device="cuda")
    db1, dgamma, dbeta = (torch.empty(k, dtype=BF16, device="cuda") for k in (ff, dm, dm))
    norm, ck, back = g.LayerNorm(m, dm), g.ActCheckpoint(m, ff), g.ActBackward(m, ff, "bf16", "gelu_bias", "col")
    with g.Plan(m, ff, dm, "bf16", "bias", "col", "nk") as up, g.Plan(m, dm, ff, "bf16", "none", "col", "kn") as down:
        norm.run(x, gamma, n, beta=beta)
        up.run(n, w, b1, z)
        ck.save(z, codes8, exps, H=h)
        kept = ref.kept(codes8.cpu(), exps.cpu())
        z16 = z.cpu().double()
        z.zero_()                                          # (it is gone; the checkpoint is what the backward pass has)
        back.run_ckpt(dH, codes8, exps, dz, H=hb, dbias=db1)
        down.run(dz, w, None, dn)
        norm.run_bwd(dn, x, gamma, dx, dgamma=dgamma, dbeta=dbeta)
        up.check(), down.check()
    ref.check_layer_norm("same", "bf16", x, None, gamma, beta, 1e-5, n)
    ref.check_act("gelu_bias", "bf16", z16, h)
    ref.check_act("gelu_bias", "bf16", kept, hb, 1e-6)
    block_ref.check_dact("gelu_bias", "col", "bf16", dH, kept, dz, db1)
    ref.check_layer_norm_bwd("bf16", dn, x, gamma, None, 1e-5, dx, dgamma, dbeta)
    exact = dH.cpu().double() * block_ref.act_slope("gelu", z16)
    assert float((dz.cpu().double() - exact).norm() / exact.norm()) < 0.02
