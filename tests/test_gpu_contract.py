"""What the header promises of the norm, the extended epilogue and the epilogue's backward beyond their formulas:
what the reported maximum counts, which scales are read, the limits of the arguments, values far from one."""
import math

import pytest
import torch

import block_ref as ref
from block_ref import T16

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


def randn(*shape, seed=0, dtype="bf16", scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=gen) * scale).to(T16[dtype]).cuda()


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


@pytest.mark.parametrize("rows", [False, True])
@pytest.mark.parametrize("epilogue", ["bias", "relu_bias", "gelu_bias"])
@pytest.mark.parametrize("axis", ["col", "row"])
@pytest.mark.parametrize("m,n,kw", [(129, 272, dict(kernel="tc1", block_n=128)), (129, 272, dict(kernel="tc1", block_n=256)),
                                    (300, 272, dict(kernel="tc2", block_n=256)), (1, 16, dict(kernel="tc1", block_n=128)),
                                    (300, 400, dict(kernel="tc2", block_n=256, max_ctas=2)),
                                    (128, 272, dict(kernel="tc1", block_n=256)), (256, 272, dict(kernel="tc2", block_n=256)), (17, 272, dict(kernel="splitk")),
                                    (300, 272, {}), (5, 144, {})])
def test_the_reported_maximum_is_over_the_output(m, n, kw, axis, epilogue, rows):
    a, b, bias, y = cancelled(m, n, axis)
    want = ref.act(epilogue, y.double()).abs().max()
    D, amax = torch.zeros(m, n, dtype=torch.uint8, device="cuda").view(E4M3), f32(9e9)
    with g.Plan(m, n, 32, "e4m3", epilogue, axis, out_e4m3=True, **kw) as p:
        p.set_scales(f32(1), f32(2 if rows else 1))
        p.set_out_scale(f32(0.0625), amax)
        if rows:
            p.run_ext(a, b, bias, D, scale_rows=torch.full((m,), 0.5, device="cuda"))
        else:
            p.run(a, b, bias, D)
        p.check()
    # GELU alone computes: its erfc is within 1.5e-7 (of a value that |x| / 2 scales) and fp32
    assert abs(float(amax) - float(want)) <= (2.0 ** -20 * 2.125 if epilogue == "gelu_bias" else 0.0)


@pytest.mark.parametrize("prenorm", [False, True])
@pytest.mark.parametrize("act", ["relu_bias", "gelu_bias"])
@pytest.mark.parametrize("m", [5, 129, 300])
def test_the_blocks_reported_maximum_is_over_h(m, act, prenorm):
    dm, ff = 256, 528
    w1 = torch.zeros(dm, ff)
    w1[0] = -9.0
    q1, q2 = w1.to(E4M3).cuda(), torch.zeros(ff, dm).to(E4M3).cuda()
    b1, b2 = torch.full((ff,), 10.0, dtype=torch.bfloat16, device="cuda"), torch.zeros(dm, dtype=torch.bfloat16, device="cuda")
    amax, rows = f32(9e9), torch.zeros(m, device="cuda")
    N = torch.zeros(m, dm).cuda()
    N[:, 0] = 1
    X, N = N.bfloat16(), N.to(E4M3)
    H, Y = torch.zeros(m, ff, dtype=torch.uint8, device="cuda").view(E4M3), torch.zeros(m, dm, dtype=torch.bfloat16, device="cuda")
    gamma = torch.full((dm,), 0.0625, dtype=torch.bfloat16, device="cuda")        # the norm of a row is 16 in its one column
    with g.MlpPlan(m, dm, ff, "e4m3", act) as p:
        p.set_scales(f32(1), f32(1), f32(0.0625), amax, f32(1))
        if prenorm:
            p.run_prenorm(X, gamma, q1, b1, q2, b2, N, H, Y, scale_rows=rows, eps=1e-12)
        else:
            p.run(N, q1, b1, q2, b2, H, Y)
        p.check()
    # h = act(10 - 9 * 1); before a GELU or ReLU of slope up to 1.13 the norm's 1 is off by at most a few 2^-24
    want = float(ref.act(act, torch.ones((), dtype=torch.float64)))
    assert abs(float(amax) - want) <= 1.13 * 9 * 2.0 ** -20


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


@pytest.mark.parametrize("d", [64, 1024, 8192])
def test_norm_with_the_smallest_scales(d):
    """Any scale above 0: a quotient beyond fp32 saturates, and 0 / scale is 0."""
    x, gamma = randn(5, d, seed=1), torch.ones(d, dtype=torch.bfloat16, device="cuda")
    x[1] = 0
    x[2, ::3] = 0
    for scale in (1e-37, 1e-42):
        Y = torch.empty(5, d, dtype=torch.uint8, device="cuda").view(E4M3)
        g.RmsNorm(5, d, "bf16", "e4m3").run(x, gamma, Y, scale=f32(scale))
        assert torch.equal(Y.float(), 448 * torch.sign(x.float()))
    g.RmsNorm(5, d, "bf16", "e4m3").run(x, gamma, Y, scale=f32(math.nan))
    assert bool(Y.float().isnan().all())               # a scale that is no number shows


@pytest.mark.parametrize("m,kw", [(5, {}), (129, dict(kernel="tc1", block_n=128)), (300, dict(kernel="tc2", block_n=256))])
def test_e4m3_output_with_the_smallest_scales(m, kw):
    a, b, bias, y = cancelled(m, 272, "col")
    for scale in (1e-37, 1e-42):
        with g.Plan(m, 272, 32, "e4m3", "relu_bias", "col", out_e4m3=True, **kw) as p:
            p.set_scales(f32(1), f32(1))
            p.set_out_scale(f32(scale), None)
            for rows in (torch.ones(m, device="cuda"), None):
                D = torch.empty(m, 272, dtype=torch.uint8, device="cuda").view(E4M3)
                p.run_ext(a, b, bias, D, scale_rows=rows)
                p.check()
                assert torch.equal(D.float().cpu(), 448.0 * (y > 0))
                p.set_out_scale(f32(math.nan), None)
                p.run_ext(a, b, bias, D, scale_rows=rows)
                p.check()
                assert bool(D.float().isnan().all())
                p.set_out_scale(f32(scale), None)


# ------------------------------------------------------------------ the norm
def test_norm_of_a_sum_whose_rounding_would_show():
    """S rounds 256.99 down to 256 and 257.01 up to 258: a norm taken of the rounded S would be off by two half-steps in the
    columns that round the other way, twice what Y's own rounding may be."""
    r = torch.full((4, 256), 256.0, dtype=torch.bfloat16)
    x = torch.full((4, 256), 0.98828125, dtype=torch.bfloat16)
    x[:, ::16] = 1.0078125
    gamma = torch.linspace(0.5, 2.0, 256).bfloat16()
    Y, S = torch.empty(4, 256, dtype=torch.bfloat16, device="cuda"), torch.empty(4, 256, dtype=torch.bfloat16, device="cuda")
    g.RmsNorm(4, 256).run(x.cuda(), gamma.cuda(), Y, residual=r.cuda(), S=S)
    ref.check_norm("same", "bf16", x, r, gamma, 1e-6, Y, S)
    s = S.cpu()
    assert set(s.float().unique().tolist()) == {256.0, 258.0}
    wrong = ref.norm(s, None, gamma, 1e-6)[1].bfloat16()
    with pytest.raises(AssertionError):
        ref.check_norm("same", "bf16", x, r, gamma, 1e-6, wrong, s)


@pytest.mark.parametrize("eps", [1e-30, 1e-38, 1e-40, 1e-44])
@pytest.mark.parametrize("m,d", [(3, 64), (3, 1024), (200, 4096), (2, 8192)])
def test_norm_and_its_backward_with_the_smallest_eps(m, d, eps):
    """eps may be any positive number: a row of zeros beside it has rho = eps^-1/2, which fp32 holds although its square is beyond it."""
    x, gamma = randn(m, d, seed=1), randn(d, seed=2)
    x[1] = 0
    Y, dX, dg = torch.empty_like(x), torch.empty_like(x), torch.empty_like(gamma)
    op = g.RmsNorm(m, d, eps=eps)
    op.run(x, gamma, Y)
    e = float(torch.tensor(eps, dtype=torch.float32))
    ref.check_norm("same", "bf16", x, None, gamma, e, Y)
    dy, ds = randn(m, d, seed=3), randn(m, d, seed=4)
    dy[1] *= 1e-12
    op.run_bwd(dy, x, gamma, dX, dgamma=dg, dS=ds)
    ref.check_norm_bwd("bf16", dy, x, gamma, ds, e, dX, dg)


def column_sums(make, m, step):
    """Sums over m rows of a term's rows in 64 bits, `step` rows at a time: (sum, sum of magnitudes)."""
    total = size = 0.0
    for i in range(0, m, step):
        t = make(i, min(m, i + step))
        total, size = total + t.sum(0), size + t.abs().sum(0)
    return total.cpu(), size.cpu()


def test_norm_bwd_sums_over_many_rows():
    """dgamma of hundreds of rows to each of the 148 blocks.  A sum of N terms in fp32 is off by at most N 2^-24 of the sum of
    their magnitudes: a thread adds m / 148 rows, its results pass 148 more; a term is off by at most 2^-20 of itself (the
    sum of squares has d positive terms in chains of at most 64, whose root halves its error, and four more operations)."""
    m, d = 37000, 8208
    gen = torch.Generator(device="cuda").manual_seed(7)
    s = torch.randn(m, d, generator=gen, device="cuda", dtype=torch.bfloat16)
    dy = torch.randn(m, d, generator=gen, device="cuda", dtype=torch.bfloat16)
    gamma = randn(d, seed=8)
    dX, dg = torch.empty_like(s), torch.empty_like(gamma)
    op = g.RmsNorm(m, d)
    op.run_bwd(dy, s, gamma, dX, dgamma=dg)

    def terms(i, j):
        v = s[i:j].double()
        return dy[i:j].double() * v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6)

    want, size = column_sums(terms, m, 1000)
    ref.close(dg, want, ref.rounded(want, "bf16", ((m / 148 + 148) * 2.0 ** -24 + 2.0 ** -20) * size), "dgamma")
    again = torch.empty_like(dg)
    op.run_bwd(dy, s, gamma, dX, dgamma=again)
    assert torch.equal(again, dg)


def test_bias_gradient_of_many_rows_in_one_run():
    """So many strips that every row is in one run: a lane adds m / 8 rows in a chain, then the 8 warps' sums."""
    m, n = 1500, 303360
    gen = torch.Generator(device="cuda").manual_seed(9)
    dd = torch.randn(m, n, generator=gen, device="cuda", dtype=torch.bfloat16)
    db = torch.empty(n, dtype=torch.bfloat16, device="cuda")
    assert g.gemm_epi_dact_workspace_bytes(m, n, g.BIAS_COL) == 0
    g.ActBackward(m, n, "bf16", "bias", "col").run(dd, dbias=db)
    want, size = column_sums(lambda i, j: dd[i:j].double(), m, 100)
    ref.close(db, want, ref.rounded(want, "bf16", (m / 8 + 8) * 2.0 ** -24 * size), "dbias")


# ------------------------------------------------------------------ slopes far from zero
# e^-(z^2 / 2) is computed as 2^-q, q = (z c)^2: c and z c are rounded and squared, q is rounded, 5 half-steps of q in all, so
# off by ln 2 q 5 2^-24 <= 1.25 z^2 2^-23 of itself, and ex2.approx by 2^-22; the fraction beside it is fitted to the larger of
# 1.8e-7 and 3.6e-5 of itself and computed to 2^-21 of one half, which is absolute where its two terms cancel (near z = -0.75).
# tanh: e^-2|z| = 2^-q with q = 2 |z| log2 e of two roundings, ln 2 q 2^-23 <= |z| 2^-21.
def slope_allowance(name, z, slope):
    if name == "gelu":
        return slope.abs() * (1.25 * z * z * 2.0 ** -23 + 2.0 ** -20 + 3.6e-5) + (2.0 ** -21 + 1.8e-7) * torch.exp(-z * z / 2)
    return slope.abs() * (z.abs() * 2.0 ** -21 + 2.0 ** -20)


@pytest.mark.parametrize("axis", ["row", "col"])
@pytest.mark.parametrize("epilogue,far", [("gelu", 12.5), ("tanh_bias", 40.0)])
def test_slopes_have_their_digits_far_out(epilogue, far, axis):
    """bf16 holds the slopes of saturated units: GELU's to z = -12.5, tanh's to |z| = 40, with every digit of the type."""
    z = torch.linspace(-far, far, 4096).bfloat16().view(16, 256)
    dd = (2.0 ** torch.arange(-2, 2, 1 / 64)).bfloat16().view(1, 256).expand(16, 256).contiguous()
    dZ, db = torch.empty_like(z, device="cuda"), torch.empty(16 if axis == "row" else 256, dtype=torch.bfloat16, device="cuda")
    g.ActBackward(16, 256, "bf16", epilogue, axis).run(dd.cuda(), dZ=dZ, z=z.cuda(), dbias=db)
    name, zd, ddd = epilogue.split("_")[0], z.double(), dd.double()
    if name == "gelu":       # Phi(z) = erfc(-z / sqrt 2) / 2, without cancellation on the left
        slope = torch.special.erfc(-zd / math.sqrt(2)) / 2 + zd * torch.exp(-zd * zd / 2) / math.sqrt(2 * math.pi)
    else:
        slope = 1 / torch.cosh(zd) ** 2
    off = ddd * slope_allowance(name, zd, slope)
    want = ddd * slope
    ref.close(dZ, want, ref.rounded(want, "bf16", off + 2.0 ** -24 * want.abs()), "dZ")
    dim = 1 if axis == "row" else 0
    ref.close(db, want.sum(dim), ref.rounded(want.sum(dim), "bf16", off.sum(dim) + ref.F32 * want.abs().sum(dim)), "dbias")


@pytest.mark.parametrize("epilogue,left,right", [("gelu", 0.0, 1.0), ("tanh", 0.0, 0.0), ("relu", 0.0, 1.0)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_slopes_at_infinity(dtype, epilogue, left, right):
    """A pre-activation that overflowed its 16 bits has the slope of the side that it is on."""
    z = randn(8, 64, seed=1, dtype=dtype)
    z[:, 5], z[:, 6], z[:, 7], z[:, 8] = math.inf, -math.inf, 65504.0, -65504.0
    dd = torch.full_like(z, 3.0)
    dZ, db = torch.empty_like(z), torch.empty(64, dtype=z.dtype, device="cuda")
    g.ActBackward(8, 64, dtype, epilogue, "col").run(dd, dZ=dZ, z=z, dbias=db)
    assert bool((dZ[:, [5, 7]] == 3 * right).all()) and bool((dZ[:, [6, 8]] == 3 * left).all())
    assert db[5:9].tolist() == [24 * right, 24 * left] * 2 and bool(torch.isfinite(db.float()).all())


# ------------------------------------------------------------------ plans
@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("epilogue", ["bias", "relu_aux_bias"])
@pytest.mark.parametrize("m,n,k", [(700, 1040, 520), (1025, 2056, 136)])
def test_plans_that_chose_wide_tiles_by_themselves(m, n, k, epilogue, layout):
    """Few SMs make a plan choose 512-wide tiles; its runs with a residual then take 256-wide ones, with ring stages, tiles and a
    raster of their own.  Its plain runs, before and after, keep their bits."""
    from test_gpu_ext import Case
    for rows in (False, True):
        c = Case(m, n, k, "bf16", epilogue, "col", layout, rows=rows)
        with c.plan(max_ctas=4) as p:
            assert p.info["block_n"] == 512 and p.info["kernel"] == g.KERNEL_TC2
            plain = []
            for _ in range(2):
                D = c.out()
                p.run(c.a, c.b, c.bias, D, c.aux())
                plain.append(D)
                c.check(plan=p)
                if rows:
                    E, aux = c.out(), c.aux()
                    p.run_ext(c.a, c.b, c.bias, E, scale_rows=c.rows, aux=aux)
                    p.check()
                    ref.close(E, *c.want(residual=False), what="row scales alone")
            assert torch.equal(*plain)


def test_the_grid_wide_small_m_form_has_no_extended_epilogue(monkeypatch):
    from test_gpu_ext import Case
    c = Case(9, 272, 1040, "bf16", "bias", rows=True)
    x = torch.zeros(9, 64, dtype=torch.bfloat16, device="cuda")
    w1, w2 = torch.zeros(64, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(128, 64, dtype=torch.bfloat16, device="cuda")
    gamma, b1 = x[0].contiguous(), w1[0].contiguous()
    H, N, Y = torch.zeros(9, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros_like(x), torch.zeros_like(x)
    monkeypatch.setenv("GEMM_EPI_SK_GRID", "1")
    with c.plan() as p, g.MlpPlan(9, 64, 128, "bf16", "bias") as mlp:
        for call in (lambda: p.run_ext(c.a, c.b, c.bias, c.out(), residual=c.res),
                     lambda: p.run_ext(c.a, c.b, c.bias, c.out(), scale_rows=c.rows),
                     lambda: mlp.run_prenorm(x, gamma, w1, b1, w2, gamma, N, H, Y)):
            with pytest.raises(g.GemmEpiError) as e:
                call()
            assert e.value.status == g.ERR_UNSUPPORTED
        D = c.out()
        p.run_ext(c.a, c.b, c.bias, D)              # without either, gemm_epi_run
        p.check()
    c.rows = None
    ref.close(D, *c.want(residual=False))


# ------------------------------------------------------------------ shapes
def test_objects_refuse_tensors_of_another_shape():
    """As many values in another shape, transposed ones above all, are refused; flat buffers and split axes are the same rows."""
    x, gamma, Y = randn(4, 64), randn(64), randn(4, 64)
    op = g.RmsNorm(4, 64)
    for bad in (randn(64, 4), randn(8, 32), randn(32, 8), randn(2, 64, 2)):
        for kw in (dict(X=bad), dict(Y=bad), dict(residual=bad)):
            with pytest.raises(g.GemmEpiError) as e:
                op.run(**{**dict(X=x, gamma=gamma, Y=Y), **kw})
            assert e.value.status == g.ERR_ARG
        with pytest.raises(g.GemmEpiError):
            op.run_bwd(x, bad, gamma, Y)
        with pytest.raises(g.GemmEpiError):
            g.ActBackward(4, 64, "bf16", "gelu").run(x, dZ=Y, z=bad)
    op.run(x, gamma, Y)
    for shape in ((256,), (2, 2, 64), (4, 8, 8), (1, 4, 64), (4, 64, 1), (2, 2, 4, 16)):
        Z = torch.empty_like(Y)
        op.run(x.view(shape), gamma.view(1, 64), Z.view(shape))
        assert torch.equal(Z, Y)
    a, b, bias, D = randn(32, 64), randn(64, 48), randn(48), torch.empty(32, 48, dtype=torch.bfloat16, device="cuda")
    res, out = randn(32, 48), []
    for layout in ("kn", "nk"):
        with g.Plan(32, 48, 64, "bf16", "bias", "col", layout) as p:
            right, wrong = (b, b.t().contiguous()) if layout == "kn" else (b.t().contiguous(), b)
            with pytest.raises(g.GemmEpiError):
                p.run_ext(a, wrong, bias, D, residual=res)
            with pytest.raises(g.GemmEpiError):
                p.run_ext(a.view(64, 32), right, bias, D, residual=res)
            with pytest.raises(g.GemmEpiError):
                p.run_ext(a, right, bias, D, residual=res.view(48, 32))
            p.run_ext(a, right, bias.view(1, 48), D, residual=res)
            p.check()
            out.append(D.clone())
    assert torch.equal(*out)
    x2, w1, w2, b1 = randn(4, 64), randn(64, 128), randn(128, 64), randn(128)
    N, H, Y2 = torch.empty_like(x2), torch.empty(4, 128, dtype=torch.bfloat16, device="cuda"), torch.empty_like(x2)
    with g.MlpPlan(4, 64, 128, "bf16", "bias") as p:
        with pytest.raises(g.GemmEpiError):
            p.run_prenorm(x2, gamma, w2, b1, w1, gamma, N, H, Y2)
        p.run_prenorm(x2, gamma, w1, b1, w2, gamma, N, H, Y2)
        p.check()
