"""The extended epilogue (residual, scales by row) against the formula in 64 bits, and the pre-norm
MLP block in both directions.

The product's own allowance is the library's: TOL of tests/helpers.py around alpha * A.B (fp32 sums of
k products).  Integer-valued operands make A.B exact in fp32, so there the only errors are those of the
epilogue: one rounding of D, and fp32 arithmetic before it.
"""
import numpy as np
import pytest
import torch

import block_ref as ref
from block_ref import T16
from helpers import unpack_aux

from activation_epilogue_tcgen05_b200 import gemm_epi as g

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
IN = {**T16, "e4m3": E4M3}
OUT = {"f16": "f16", "bf16": "bf16", "e4m3": "bf16"}
EPILOGUES = ["none", "bias", "relu_bias", "relu_aux_bias", "gelu_bias", "tanh_bias", "relu", "relu_aux", "gelu", "tanh"]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.get_device_capability() != (10, 0):
        pytest.skip("needs sm_100")
    from activation_epilogue_tcgen05_b200 import build
    build.build()


class Case:
    """Integer operands (|a|, |b| <= 3: every partial sum is an integer below 2^24), real bias and residual."""

    def __init__(self, m, n, k, dtype, epilogue, axis="col", layout="kn", rows=False, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.m, self.n, self.k, self.dtype, self.epilogue, self.axis, self.layout = m, n, k, dtype, epilogue, axis, layout
        o = OUT[dtype]
        a, b = torch.randint(-3, 4, (m, k), generator=gen).float(), torch.randint(-3, 4, (k, n), generator=gen).float()
        self.a, self.b = a.to(IN[dtype]).cuda(), (b if layout == "kn" else b.t().contiguous()).to(IN[dtype]).cuda()
        self.bias = torch.randn(m if axis == "row" else n, generator=gen).to(T16[o]).cuda()
        self.res = (2 * torch.randn(m, n, generator=gen)).to(T16[o]).cuda()
        self.rows = (torch.rand(m, generator=gen) * 0.2 + 0.01).cuda() if rows else None
        self.sa, self.sb = torch.tensor([0.25], device="cuda"), torch.tensor([0.125 if not rows else 0.37], device="cuda")
        self.ab = a.double() @ b.double()

    def plan(self, scales=True, **kw):
        p = g.Plan(self.m, self.n, self.k, self.dtype, self.epilogue, self.axis, self.layout, **kw)
        if scales:
            p.set_scales(self.sa, self.sb)
        return p

    def pre(self):
        alpha = self.sa.cpu().double() if self.rows is None else self.rows.cpu().double()[:, None]
        z = self.ab * (alpha * self.sb.cpu().double())
        off = 3 * 2.0 ** -24 * z.abs()                                   # the scales' product, times the sum
        if self.epilogue in g.HAS_BIAS:
            bias = self.bias.cpu().double()
            z = z + (bias[:, None] if self.axis == "row" else bias)
            off = off + 2.0 ** -24 * z.abs()
        return z, off

    def want(self, residual=True):
        """(D, allowance): |act'| <= 1.13, the activations' own error as documented beside them."""
        z, off = self.pre()
        y = ref.act(self.epilogue, z)
        kind = self.epilogue.split("_")[0]
        # GELU: erfc within 1.5e-7 and its exponential's argument within 2^-21 of a value that |x| scales
        own = {"gelu": 2.0 ** -20 * z.abs().clamp(max=8) + 2.0 ** -24 * y.abs(), "tanh": 2.0 ** -22 * y.abs()}.get(kind, 0 * y)
        off = 1.13 * off + own
        if residual:
            y = y + self.res.cpu().double()
            off = off + 2.0 ** -24 * y.abs()
        return y, ref.rounded(y, OUT[self.dtype], off)

    def out(self):
        return torch.full((self.m, self.n), float("nan"), dtype=T16[OUT[self.dtype]], device="cuda")

    def aux(self):
        return torch.full((self.m * g.aux_pitch_words(self.n),), -1515870811, dtype=torch.int32, device="cuda") \
            if self.epilogue in g.HAS_AUX else None

    def check(self, plan=None, **kw):
        D, aux = self.out(), self.aux()
        own = plan is None
        plan = plan or self.plan(**kw)
        plan.run_ext(self.a, self.b, self.bias, D, residual=self.res, scale_rows=self.rows, aux=aux)
        plan.check()
        info = plan.info
        if own:
            plan.close()
        ref.close(D, *self.want(), what=f"{self.epilogue} {info}")
        if aux is not None:
            z, off = self.pre()
            words = aux.cpu().numpy().view(np.uint32)
            bits = torch.from_numpy(unpack_aux(words, self.m, self.n).astype(np.int64))
            sure = z.abs() > 2 * off
            assert torch.equal(bits[sure].bool(), (z > 0)[sure])
        return info


@pytest.mark.parametrize("axis,layout", [("col", "kn"), ("row", "nk")])
@pytest.mark.parametrize("epilogue", EPILOGUES)
@pytest.mark.parametrize("dtype", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("m,kw", [(300, dict(kernel="tc1", block_n=128)), (300, dict(kernel="tc2", block_n=256)), (17, dict(kernel="splitk"))])
def test_every_epilogue(m, kw, dtype, epilogue, axis, layout):
    Case(m, 336, 272, dtype, epilogue, axis, layout).check(**kw)


@pytest.mark.parametrize("dtype,layout", [("f16", "nk"), ("bf16", "kn"), ("e4m3", "kn"), ("e4m3", "nk")])
@pytest.mark.parametrize("kw", [dict(kernel="tc1", block_n=256), dict(kernel="tc2", block_n=128), dict(kernel="tc2", block_n=512),
                                dict(kernel="tc1", block_n=128, stream_k="on"), dict(kernel="tc2", block_n=256, stream_k="on"),
                                dict(kernel="tc2", block_n=256, max_ctas=4), dict(kernel="tc2", block_n=512, max_ctas=2),
                                dict(kernel="tc1", block_n=256, max_ctas=3, stream_k="off")])
def test_every_tile_and_schedule(kw, dtype, layout):
    if kw["kernel"] == "tc2" and kw["block_n"] == 128 and (dtype, layout) == ("e4m3", "kn"):
        pytest.skip("not instantiated: a 64-column e4m3 half-tile is narrower than one 128-byte box")
    Case(700, 1040, 1040, dtype, "gelu_bias", "col", layout, rows=True).check(**kw)


@pytest.mark.parametrize("dtype", ["f16", "e4m3"])
@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 31, 33, 64, 65, 128])
@pytest.mark.parametrize("split", [0, 1, 2])
def test_small_m(m, split, dtype):
    Case(m, 1552, 784, dtype, "bias", "col", "nk", rows=True).check(kernel="splitk", split_k=split)


@pytest.mark.parametrize("split", [3, 4, 8])
def test_small_m_larger_clusters(split):
    Case(9, 272, 1040, "bf16", "relu_aux_bias", "row", "kn", rows=True).check(kernel="splitk", split_k=split)


@pytest.mark.parametrize("m,n,k", [(1, 16, 16), (1, 8, 8), (2, 8, 4096), (129, 8, 8), (257, 4104, 24), (1000, 264, 8), (64, 24, 1000)])
def test_odd_sizes(m, n, k):
    dtype = "bf16" if n % 16 or k % 16 else "e4m3"
    info = Case(m, n, k, dtype, "gelu_bias", rows=True).check()
    assert info["kernel"] in (1, 2, 3)


@pytest.mark.parametrize("m", [5, 300])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "e4m3"])
def test_the_pieces_alone(m, dtype):
    """A residual without row scales, row scales without a residual, neither (gemm_epi_run's bits)."""
    c = Case(m, 272, 144, dtype, "gelu_bias", rows=True)
    with c.plan() as p:
        D, E = c.out(), c.out()
        p.run_ext(c.a, c.b, c.bias, D, scale_rows=c.rows)
        ref.close(D, *c.want(residual=False), what="row scales")
        p.run_ext(c.a, c.b, c.bias, D)
        p.run(c.a, c.b, c.bias, E)
        assert torch.equal(D, E)
        c.rows = None
        c.check(plan=p)
        p.check()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_16_bit_plans_without_scales(dtype):
    """alpha is 1, or the row's scale alone."""
    for rows in (False, True):
        c = Case(150, 272, 144, dtype, "none", rows=rows)
        c.sa = c.sb = torch.ones(1, device="cuda")
        c.check(scales=False)


@pytest.mark.parametrize("m,kw", [(3, {}), (40, {}), (700, dict(kernel="tc1", block_n=128)), (700, dict(kernel="tc2", block_n=256)),
                                  (700, dict(kernel="tc2", block_n=512, max_ctas=4)), (520, dict(kernel="tc1", block_n=256, stream_k="on"))])
@pytest.mark.parametrize("n", [264, 1032])
def test_residual_in_place(m, n, kw):
    c = Case(m, n, 520, "bf16", "bias")
    D, E = c.out(), c.res.clone()
    with c.plan(**kw) as p:
        p.run_ext(c.a, c.b, c.bias, D, residual=c.res)
        p.run_ext(c.a, c.b, c.bias, E, residual=E)
        p.check()
    assert torch.equal(D, E)


def test_only_the_output_is_written():
    for m in (3, 130):
        c = Case(m, 72, 64, "bf16", "bias")
        raw = torch.full((m * 72 + 256,), 7.0, dtype=torch.bfloat16, device="cuda")
        with c.plan() as p:
            p.run_ext(c.a, c.b, c.bias, raw[128:-128], residual=c.res)
            p.check()
        ref.close(raw[128:-128].view(m, 72), *c.want())
        assert bool((raw[:128] == 7).all() and (raw[-128:] == 7).all())


@pytest.mark.parametrize("m", [20, 300])
@pytest.mark.parametrize("epilogue", ["none", "bias", "relu_bias", "gelu_bias"])
def test_e4m3_output_with_row_scales(m, epilogue):
    c = Case(m, 272, 144, "e4m3", epilogue, rows=True)
    s_out, amax = torch.tensor([0.05], device="cuda"), torch.full((1,), 9e9, device="cuda")
    D = torch.zeros(m, 272, dtype=torch.uint8, device="cuda").view(E4M3)
    with c.plan(out_e4m3=True) as p:
        p.set_out_scale(s_out, amax)
        p.run_ext(c.a, c.b, c.bias, D, scale_rows=c.rows)
        p.check()
        with pytest.raises(g.GemmEpiError) as e:
            p.run_ext(c.a, c.b, c.bias, D, residual=c.res, scale_rows=c.rows)
        assert e.value.status == g.ERR_UNSUPPORTED
    y, tol = c.want(residual=False)
    z, off = c.pre()
    v = (y / 0.05000000074505806)
    ref.close(D, v.clamp(-448, 448), ref.rounded(v, "e4m3", 2.0 ** -20 * (v.abs() + z.abs() * 20)), "e4m3")
    assert abs(float(amax) - float(y.abs().max())) <= 2.0 ** -19 * float(z.abs().max())


def test_real_operands_at_a_long_k():
    """Real operands: the library's bound for the product, the residual's rounding beside it."""
    from helpers import tolerance
    m, n, k = 333, 520, 4096
    gen = torch.Generator().manual_seed(5)
    a, b = torch.randn(m, k, generator=gen).bfloat16(), (torch.randn(k, n, generator=gen) / 64).bfloat16()
    r = torch.randn(m, n, generator=gen).bfloat16()
    D = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    with g.Plan(m, n, k, "bf16", "none") as p:
        p.run_ext(a.cuda(), b.cuda(), None, D, residual=r.cuda())
        p.check()
    z = a.double() @ b.double()
    tol = torch.from_numpy(tolerance(z.numpy(), "bf16", k, float(a.double().std()), float(b.double().std())))
    want = z + r.double()
    ref.close(D, want, tol + ref.U["bf16"] * want.abs())


def test_captured_and_replayed_and_on_a_side_stream():
    for m in (16, 600):
        c = Case(m, 1032, 520, "bf16", "gelu_bias", rows=True)
        with c.plan() as p:
            D = c.out()
            p.run_ext(c.a, c.b, c.bias, D, residual=c.res, scale_rows=c.rows)
            p.check()
            st = torch.cuda.Stream()
            st.wait_stream(torch.cuda.current_stream())
            E = c.out()
            st.wait_stream(torch.cuda.current_stream())
            p.run_ext(c.a, c.b, c.bias, E, residual=c.res, scale_rows=c.rows, stream=st)
            p.check(st)
            assert torch.equal(D, E)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                p.run_ext(c.a, c.b, c.bias, E, residual=c.res, scale_rows=c.rows)
            for k in range(3):
                c.res.copy_(c.res * 0.5)
                c.rows.mul_(1.5)
                graph.replay()
                p.check()
                ref.close(E, *c.want())
            del graph


@pytest.mark.parametrize("kernel,block_n", [("tc1", 128), ("tc2", 256)])
def test_a_wait_that_runs_out_is_reported(kernel, block_n):
    """The accumulator never comes: the kernel gives up after about a second, with the residual's load landed, and says so; the
    next run of the same sizes is right."""
    c = Case(300, 336, 272, "bf16", "bias")
    D = torch.full((300, 336), 5.0, dtype=torch.bfloat16, device="cuda")
    with c.plan(kernel=kernel, block_n=block_n, inject_stall=1) as p:
        p.run_ext(c.a, c.b, c.bias, D, residual=c.res)
        with pytest.raises(g.GemmEpiError) as e:
            p.check()
        assert e.value.status == g.ERR_TIMEOUT
    assert bool((D == 5).all())
    c.check(kernel=kernel, block_n=block_n)


def test_refusals():
    c = Case(130, 272, 144, "bf16", "bias", rows=True)
    D = c.out()
    with c.plan() as p:
        for kw in (dict(residual=c.res.cpu()), dict(residual=c.res[:, :136]), dict(residual=c.res.float()), dict(scale_rows=c.rows[:4]),
                   dict(scale_rows=c.rows.double()), dict(residual=c.res.t())):
            with pytest.raises(g.GemmEpiError):
                p.run_ext(c.a, c.b, c.bias, D, **kw)
        with pytest.raises(g.GemmEpiError):
            p.run_ext(c.a, c.b, None, D, residual=c.res)
        rc = g.lib().gemm_epi_run_ext(p.handle, c.a.data_ptr(), c.b.data_ptr(), c.bias.data_ptr(), c.res.data_ptr() + 2, None, D.data_ptr(),
                                      None, None)
        assert rc == g.ERR_ALIGN
        rc = g.lib().gemm_epi_run_ext(p.handle, c.a.data_ptr(), c.b.data_ptr(), c.bias.data_ptr(), None, c.rows.data_ptr() + 2, D.data_ptr(),
                                      None, None)
        assert rc == g.ERR_ALIGN
    with g.Plan(136, 272, 144, "bf16", "bias", a_layout="km") as p:
        rc = g.lib().gemm_epi_run_ext(p.handle, c.a.data_ptr(), c.b.data_ptr(), c.bias.data_ptr(), c.res.data_ptr(), None, D.data_ptr(), None,
                                      None)
        assert rc == g.ERR_UNSUPPORTED
    with g.Plan(130, 272, 144, "bf16", "drelu") as p:
        rc = g.lib().gemm_epi_run_ext(p.handle, c.a.data_ptr(), c.b.data_ptr(), None, c.res.data_ptr(), None, D.data_ptr(), None, None)
        assert rc == g.ERR_ARG


# ------------------------------------------------------------------ the block, forward and backward
def mlp_inputs(m, dm, ff, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed)
    t = T16[dtype]
    x, r = torch.randn(m, dm, generator=gen).to(t), (2 * torch.randn(m, dm, generator=gen)).to(t)
    gamma = (1 + 0.2 * torch.randn(dm, generator=gen)).to(t)
    w1, w2 = (torch.randn(dm, ff, generator=gen) / dm ** 0.5), (torch.randn(ff, dm, generator=gen) / ff ** 0.5)
    b1, b2 = (0.1 * torch.randn(ff, generator=gen)).to(t), (0.1 * torch.randn(dm, generator=gen)).to(t)
    return x, r, gamma, w1, b1, w2, b2


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("act", ["gelu_bias", "relu_bias", "bias"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m", [1, 33, 300])
def test_prenorm_block_16_bit(m, dtype, act, residual):
    dm, ff, eps = 256, 528, 1e-5
    x, r, gamma, w1, b1, w2, b2 = mlp_inputs(m, dm, ff, dtype)
    r = r if residual else None
    w1, w2 = w1.to(T16[dtype]), w2.to(T16[dtype])
    dev = [None if t is None else t.cuda() for t in (x, r, gamma, w1, b1, w2, b2)]
    e = lambda *s: torch.full(s, float("nan"), dtype=T16[dtype], device="cuda")      # noqa: E731
    S, N, H, Y = e(m, dm) if residual else None, e(m, dm), e(m, ff), e(m, dm)
    with g.MlpPlan(m, dm, ff, dtype, act) as p:
        p.run_prenorm(dev[0], dev[2], *dev[3:], N, H, Y, residual=dev[1], S=S, eps=eps)
        p.check()
        # each stage against the formula applied to what the stage before it wrote
        ref.check_norm("same", dtype, x, r, gamma, eps, N, S)
        u = ref.U[dtype]
        z = N.cpu().double() @ w1.double() + b1.double()
        h = ref.act(act, z)
        # fp32 sums of dm (ff) products: 2^-24 sqrt-free bound dm * 2^-24 * sum |terms|
        mag = N.cpu().double().abs() @ w1.double().abs() + b1.double().abs()
        ref.close(H, h, ref.rounded(h, dtype, 1.13 * dm * 2.0 ** -24 * mag + 2.0 ** -20), "H")
        s = (S if residual else dev[0]).cpu().double()
        y = H.cpu().double() @ w2.double() + b2.double() + s
        mag = H.cpu().double().abs() @ w2.double().abs() + b2.double().abs() + s.abs()
        ref.close(Y, y, ref.rounded(y, dtype, ff * 2.0 ** -24 * mag), "Y")
        assert u
        # the stream updated in place gives the same bits
        if residual:
            a, b = dev[0].clone(), dev[1].clone()
            p.run_prenorm(a, dev[2], *dev[3:], N, H, b, residual=b, S=b, eps=eps)
            assert torch.equal(b, Y)
        else:
            a = dev[0].clone()
            p.run_prenorm(a, dev[2], *dev[3:], N, H, a, eps=eps)
            assert torch.equal(a, Y)
        p.check()


@pytest.mark.parametrize("m", [1, 40, 300])
@pytest.mark.parametrize("act", ["gelu_bias", "relu_bias"])
def test_prenorm_block_e4m3(m, act):
    dm, ff, eps = 256, 528, 1e-5
    x, r, gamma, w1, b1, w2, b2 = mlp_inputs(m, dm, ff, "bf16")
    s1, s2 = w1.abs().max() / 448, w2.abs().max() / 448
    q1, q2 = (w1 / s1).to(E4M3), (w2 / s2).to(E4M3)
    sc = [torch.tensor([float(v)], device="cuda") for v in (1.0, s1, 4.0 / 448, s2)]
    amax = torch.zeros(1, device="cuda")
    e = lambda *s: torch.full(s, float("nan"), dtype=torch.bfloat16, device="cuda")      # noqa: E731
    S, Y, rows = e(m, dm), e(m, dm), torch.zeros(m, device="cuda")
    N, H = torch.empty(m, dm, dtype=E4M3, device="cuda"), torch.empty(m, ff, dtype=E4M3, device="cuda")
    x, r, gamma, b1, b2 = (t.cuda() for t in (x, r, gamma, b1, b2))
    with g.MlpPlan(m, dm, ff, "e4m3", act) as p:
        p.set_scales(sc[0], sc[1], sc[2], amax, sc[3])
        p.run_prenorm(x, gamma, q1.cuda(), b1, q2.cuda(), b2, N, H, Y, residual=r, S=S, scale_rows=rows, eps=eps)
        p.check()
        with pytest.raises(g.GemmEpiError):
            p.run_prenorm(x, gamma, q1.cuda(), b1, q2.cuda(), b2, N, H, Y, residual=r, S=S, eps=eps)      # no row scales
    ref.check_norm("e4m3_rows", "bf16", x, r, gamma, eps, N, S, rows)
    n = N.cpu().double() * rows.cpu().double()[:, None]
    d1, d2 = q1.double() * sc[1].cpu().double(), q2.double() * sc[3].cpu().double()
    z = n @ d1 + b1.cpu().double()
    h = ref.act(act, z)
    mag = n.abs() @ d1.abs() + b1.cpu().double().abs()
    sh = sc[2].cpu().double()
    v = h / sh
    ref.close(H, v.clamp(-448, 448), ref.rounded(v, "e4m3", (1.13 * dm * 2.0 ** -24 * mag + 2.0 ** -20) / sh), "H")
    hq = H.cpu().double() * sh
    y = hq @ d2 + b2.cpu().double() + S.cpu().double()
    mag = hq.abs() @ d2.abs() + b2.cpu().double().abs() + S.cpu().double().abs()
    ref.close(Y, y, ref.rounded(y, "bf16", ff * 2.0 ** -24 * mag), "Y")


@pytest.mark.parametrize("m", [8, 260])
def test_prenorm_block_captured_and_replayed(m):
    """The serving loop: the stream updated in place by two blocks in one graph, replayed, against the same calls made one by
    one; then the backward calls in a graph of their own."""
    dm, ff, eps = 256, 528, 1e-5
    x, r, gamma, w1, b1, w2, b2 = (t.to(torch.bfloat16).cuda() for t in mlp_inputs(m, dm, ff, "bf16"))
    N, H = torch.empty(m, dm, dtype=torch.bfloat16, device="cuda"), torch.empty(m, ff, dtype=torch.bfloat16, device="cuda")
    with g.MlpPlan(m, dm, ff, "bf16", "gelu_bias") as p:
        def step(a, b):
            p.run_prenorm(a, gamma, w1, b1, w2, b2, N, H, a, residual=b, S=b, eps=eps)     # b = a + b, a = mlp(norm(b)) + b
            p.run_prenorm(a, gamma, w1, b1, w2, b2, N, H, a, eps=eps)

        a, b = x.clone(), r.clone()
        for _ in range(3):
            step(a, b)
        p.check()
        c, d = x.clone(), r.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(c, d)
        c.copy_(x)
        d.copy_(r)
        for _ in range(3):
            graph.replay()
        p.check()
        assert torch.equal(a, c) and torch.equal(b, d) and bool(torch.isfinite(a.float()).all())
        del graph
    dZ, dX, db, dg, dbr = (torch.empty_like(t) for t in (x, x, gamma, gamma, x[:, 0].contiguous()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.ActBackward(m, dm, "bf16", "gelu", "col").run(x, dZ=dZ, z=r, dbias=db)
        g.ActBackward(m, dm, "bf16", "bias", "row").run(dZ, dbias=dbr)
        g.RmsNorm(m, dm, eps=eps).run_bwd(dZ, r, gamma, dX, dgamma=dg, dS=x)
    for _ in range(2):
        x.mul_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        ref.check_dact("gelu", "col", "bf16", x, r, dZ, db)
        ref.check_dact("bias", "row", "bf16", dZ, r, None, dbr)
        ref.check_norm_bwd("bf16", dZ, r, gamma, x, eps, dX, dg)


def test_prenorm_block_refusals():
    m, dm, ff = 4, 64, 128
    x, r, gamma, w1, b1, w2, b2 = (t.to(torch.bfloat16).cuda() for t in mlp_inputs(m, dm, ff, "bf16"))
    N, S, Y, H = (torch.empty(m, k, dtype=torch.bfloat16, device="cuda") for k in (dm, dm, dm, ff))
    with g.MlpPlan(m, dm, ff, "bf16", "gelu_bias") as p:
        for kw in (dict(residual=r), dict(residual=r, S=N), dict(N=x), dict(N=Y), dict(eps=0.0), dict(H=N), dict(gamma=gamma[:32]),
                   dict(residual=x[:2])):
            a = {**dict(X=x, gamma=gamma, W1=w1, b1=b1, W2=w2, b2=b2, N=N, H=H, Y=Y), **kw}
            with pytest.raises(g.GemmEpiError):
                p.run_prenorm(**a)


@pytest.mark.parametrize("act", ["relu_aux_bias", "gelu_bias"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_block_trained(dtype, act):
    """Forward and backward of y = x + W2 act(W1 norm(x) + b1) + b2 with the framework's calls alone, every gradient
    against the formula on what the calls before it wrote, and the whole against central differences."""
    m, dm, ff, eps = 200, 256, 528, 1e-3
    t, o = T16[dtype], dtype
    x, _, gamma, w1, b1, w2, b2 = mlp_inputs(m, dm, ff, dtype, seed=3)
    w1, w2 = w1.to(t), w2.to(t)
    dy = torch.randn(m, dm, generator=torch.Generator().manual_seed(9)).to(t)
    X, G, W1, B1, W2, B2, DY = (v.cuda() for v in (x, gamma, w1, b1, w2, b2, dy))
    e = lambda *s: torch.full(s, float("nan"), dtype=t, device="cuda")                       # noqa: E731
    N, H, Y, Z = e(m, dm), e(m, ff), e(m, dm), e(m, ff)
    aux = torch.zeros(m * g.aux_pitch_words(ff), dtype=torch.int32, device="cuda")
    norm, gelu = g.RmsNorm(m, dm, dtype, eps=eps), act == "gelu_bias"
    plans = []

    def product(m_, n_, k_, epi, a, b, bias, d, layout="kn", res=None, mask=None, a_layout="mk"):
        p = g.Plan(m_, n_, k_, dtype, epi, "col", layout, a_layout=a_layout)
        plans.append(p)
        if res is None:
            p.run(a, b, bias, d, mask)
        else:
            p.run_ext(a, b, bias, d, residual=res, aux=mask)

    norm.run(X, G, N)
    product(m, ff, dm, act, N, W1, B1, H, mask=aux if not gelu else None)
    if gelu:
        product(m, ff, dm, "bias", N, W1, B1, Z)
    product(m, dm, ff, "bias", H, W2, B2, Y, res=X)
    # backward: the residual's gradient is DY itself
    dB2, dH, dZ, dB1, dN, dX, dG = e(dm), e(m, ff), e(m, ff), e(ff), e(m, dm), e(m, dm), e(dm)
    dW1, dW2 = e(dm, ff), e(ff, dm)
    g.ActBackward(m, dm, dtype, "bias", "col").run(DY, dbias=dB2)
    product(ff, dm, m, "none", H, DY, None, dW2, a_layout="km")
    product(m, ff, dm, "none", DY, W2, None, dH, layout="nk")
    g.ActBackward(m, ff, dtype, act, "col").run(dH, dZ=dZ, z=Z if gelu else None, aux=None if gelu else aux, dbias=dB1)
    product(dm, ff, m, "none", N, dZ, None, dW1, a_layout="km")
    product(m, dm, ff, "none", dZ, W1, None, dN, layout="nk")
    norm.run_bwd(dN, X, G, dX, dgamma=dG, dS=DY)
    torch.cuda.synchronize()
    for p in plans:
        p.check()
        p.close()
    # each call against the formula
    ref.check_dact("bias", "col", o, DY, torch.zeros(m, dm), None, dB2)
    z = N.cpu().double() @ w1.double() + b1.double()
    slope = (torch.from_numpy(unpack_aux(aux.cpu().numpy().view(np.uint32), m, ff).astype(np.float64)) if not gelu else None)
    ref.check_dact(act, "col", o, dH, Z if gelu else z, dZ, dB1, slope=slope)
    ref.check_norm_bwd(o, dN, X, G, DY, eps, dX, dG)
    # the whole against differences of the 64-bit loss sum(dy * y): the 16-bit stages between are each off
    # by half a step, U, of their value; a gradient passes 7 of them, so 8 U of its terms' size bounds it
    gen = torch.Generator().manual_seed(4)
    names = ["x", "gamma", "w1", "b1", "w2", "b2"]
    vals = dict(zip(names, (v.double() for v in (x, gamma, w1, b1, w2, b2))))
    grads = dict(zip(names, (v.cpu().double() for v in (dX, dG, dW1, dB1, dW2, dB2))))

    # ReLU's slope jumps at z = 0, and the forward's z comes from N rounded to 16 bits: off by at most U of
    # sum |n w| (and fp32 sums).  Elements that near zero take either branch, and each that is taken otherwise moves a
    # difference by its whole term, which no step size bounds: the gradient is that of the branches that the
    # forward took (its mask), so the differences are taken along them, and the branches are checked by themselves.
    if not gelu:
        n = ref.norm(x, None, gamma, eps)[1]
        z = n @ w1.double() + b1.double()
        near = ref.U[o] * 1.01 * (n.abs() @ w1.double().abs()) + 2.0 ** -20
        assert bool(((slope > 0) == (z > 0))[z.abs() > near].all())

    def loss(v):
        _, n = ref.norm(v["x"], None, v["gamma"], eps)
        z = n @ v["w1"] + v["b1"]
        return float((((ref.act(act, z) if gelu else z * slope) @ v["w2"] + v["b2"] + v["x"]) * dy.double()).sum())

    for k in names:
        d = torch.randn(vals[k].shape, generator=gen, dtype=torch.float64)
        h = 1e-6
        diff = (loss({**vals, k: vals[k] + h * d}) - loss({**vals, k: vals[k] - h * d})) / (2 * h)
        # independent errors of the terms d * grad: 8 U of the root of their squares' sum, 6 sigma
        allow = 6 * 8 * ref.U[o] * float((grads[k] * d).norm()) + 1e-4
        assert abs(diff - float((grads[k] * d).sum())) <= allow, (k, diff, float((grads[k] * d).sum()), allow)
