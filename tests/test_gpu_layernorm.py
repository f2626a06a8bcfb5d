"""The layer norm, its backward and rows quantised alone on the GPU, against the formulas in 64 bits (block8_ref, where the bounds
are derived)."""
import pytest
import torch

import block8_ref as ref
import block_ref
from block_ref import T16
from test_gpu_block_ops import E4M3, SHAPES, Guarded, _cuda, randn  # noqa: F401

from activation_epilogue_tcgen05_b200 import gemm_epi as g

pytestmark = pytest.mark.gpu
EPS = 1e-5
OUT_T = {"e4m3": E4M3, "e4m3_rows": E4M3, "i8_rows": torch.int8}


def run_norm(x, r, gamma, beta, dtype, out, eps=EPS, scale=None, amax=None, keep=True, stream=None):
    m, d = x.shape
    Y = Guarded(m * d, OUT_T.get(out, T16[dtype]))
    S = Guarded(m * d, T16[dtype]) if r is not None and keep else None
    rows = Guarded(m, torch.float32) if out.endswith("rows") else None
    g.LayerNorm(m, d, dtype, out, eps).run(x, gamma, Y.t, beta=beta, residual=r, S=S and S.t, scale=rows.t if rows else scale,
                                           amax=amax, stream=stream)
    torch.cuda.synchronize()
    assert all(b.intact() for b in (Y, S, rows) if b is not None)
    return Y.t.view(m, d), S and S.t.view(m, d), rows.t if rows else scale


@pytest.mark.parametrize("out", ["same", "e4m3", "e4m3_rows", "i8_rows"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,d", SHAPES)
def test_layer_norm(m, d, dtype, residual, out):
    x, gamma, beta = randn(m, d, seed=1, dtype=dtype, scale=2.0) + 1.5, randn(d, seed=2, dtype=dtype), randn(d, seed=4, dtype=dtype)
    r = randn(m, d, seed=3, dtype=dtype, scale=3.0) if residual else None
    beta = beta if m % 2 else None
    scale = torch.tensor([2.0 / 448], device="cuda") if out == "e4m3" else None       # the largest values saturate
    amax = torch.full((1,), 1e9, device="cuda") if out == "e4m3" else None
    Y, S, sc = run_norm(x, r, gamma, beta, dtype, out, scale=scale, amax=amax)
    ref.check_layer_norm(out, dtype, x, r, gamma, beta, EPS, Y, S, sc, amax)


@pytest.mark.parametrize("m,d", [(5, 8), (3, 1000), (2, 4104), (3, 6144), (2, 6152), (3, 12288), (2, 12296), (3, 16376)])
def test_lengths_that_are_no_multiple_of_16(m, d):
    x, gamma, beta, r = randn(m, d, seed=1), randn(d, seed=2), randn(d, seed=3), randn(m, d, seed=4)
    Y, S, _ = run_norm(x, r, gamma, beta, "bf16", "same")
    ref.check_layer_norm("same", "bf16", x, r, gamma, beta, EPS, Y, S)


@pytest.mark.parametrize("dtype,mean,spread", [("bf16", 256.0, 1.0), ("bf16", -3e4, 200.0), ("f16", 1000.0, 0.5), ("f16", 0.0, 1e-4)])
@pytest.mark.parametrize("d", [64, 1024, 4096])
def test_means_far_from_zero(d, dtype, mean, spread):
    """A mean of hundreds of deviations: mean s^2 - mean^2 would have few digits left."""
    x, gamma, beta = (randn(9, d, seed=5, dtype="bf16").float() * spread + mean).to(T16[dtype]), randn(d, seed=6, dtype=dtype), randn(d, seed=7, dtype=dtype)
    Y, _, _ = run_norm(x, None, gamma, beta, dtype, "same")
    ref.check_layer_norm("same", dtype, x, None, gamma, beta, EPS, Y)
    dy, dX = randn(9, d, seed=8, dtype=dtype), torch.empty_like(x)
    dg, db = torch.empty_like(gamma), torch.empty_like(gamma)
    g.LayerNorm(9, d, dtype, eps=EPS).run_bwd(dy, x, gamma, dX, dgamma=dg, dbeta=db)
    ref.check_layer_norm_bwd(dtype, dy, x, gamma, None, EPS, dX, dg, db)


def test_the_sum_is_not_rounded_first():
    """x + r that cancels to below the type's step of r: the norm sees the difference."""
    r = torch.full((4, 256), 256.0, dtype=torch.bfloat16, device="cuda")
    x, gamma = randn(4, 256, seed=6, scale=0.25), torch.ones(256, dtype=torch.bfloat16, device="cuda")
    Y, S, _ = run_norm(x, r, gamma, None, "bf16", "same")
    ref.check_layer_norm("same", "bf16", x, r, gamma, None, EPS, Y, S)


@pytest.mark.parametrize("out", ["same", "e4m3", "e4m3_rows", "i8_rows"])
@pytest.mark.parametrize("d", [64, 512, 4096])
def test_constant_rows_and_rows_of_zeros(d, out):
    """A row without a deviation is beta; with beta 0 as well a row of zeros, whose scale is 1."""
    x = randn(5, d, seed=4)
    x[1], x[2], x[3] = 0, 3.0, 1e-38
    gamma, beta = randn(d, seed=5), randn(d, seed=6)
    scale = torch.tensor([0.01], device="cuda") if out == "e4m3" else None
    for b in (beta, None):
        Y, _, sc = run_norm(x, None, gamma, b, "bf16", out, scale=scale)
        if b is None and out.endswith("rows"):
            assert sc[1:4].tolist() == [1.0] * 3 and not Y[1:4].float().any()
            ref.check_layer_norm(out, "bf16", x[[0, 4]], None, gamma, b, EPS, Y[[0, 4]], None, sc[[0, 4]])
        else:
            ref.check_layer_norm(out, "bf16", x, None, gamma, b, EPS, Y, None, sc)


@pytest.mark.parametrize("eps", [1e-12, 1e-3, 1.0, 1e4])
def test_eps(eps):
    x, gamma, beta = randn(5, 384, seed=7, scale=0.01), randn(384, seed=8), randn(384, seed=9)
    Y, _, _ = run_norm(x, None, gamma, beta, "bf16", "same", eps=eps)
    ref.check_layer_norm("same", "bf16", x, None, gamma, beta, eps, Y)


@pytest.mark.parametrize("out", ["same", "e4m3_rows", "i8_rows"])
def test_values_that_are_not_finite_stay_in_their_row(out):
    x, gamma = randn(8, 1024, seed=1), randn(1024, seed=2)
    want, _, sw = run_norm(x, None, gamma, None, "bf16", out)
    x[2, 5], x[5, 700] = float("nan"), float("inf")
    Y, _, sc = run_norm(x, None, gamma, None, "bf16", out)
    keep = [0, 1, 3, 4, 6, 7]
    assert torch.equal(Y[keep].float(), want[keep].float())
    if out == "same":
        assert Y[2].isnan().all() and Y[5].isnan().all()
    else:
        assert torch.equal(sc[keep], sw[keep]) and not sc[[2, 5]].isfinite().any()


@pytest.mark.parametrize("d", [128, 1024, 4096])
def test_in_place(d):
    x, r, gamma, beta = randn(67, d, seed=9), randn(67, d, seed=10), randn(d, seed=11), randn(d, seed=12)
    Y, S, _ = run_norm(x, r, gamma, beta, "bf16", "same")
    for s_over, y_over in [("r", "x"), ("x", "r")]:
        b = {"x": x.clone(), "r": r.clone()}
        g.LayerNorm(67, d).run(b["x"], gamma, b[y_over], beta=beta, residual=b["r"], S=b[s_over])
        assert torch.equal(b[s_over], S) and torch.equal(b[y_over], Y)
    assert torch.equal(run_norm(x, r, gamma, beta, "bf16", "same", keep=False)[0], Y)


def test_offsets_beyond_32_bits():
    m, d = 140_000, 16_384             # 2.3 G elements, 4.6 GB
    x = torch.zeros(m, d, dtype=torch.bfloat16, device="cuda")
    last, gamma, beta = randn(3, d, seed=12), randn(d, seed=13), randn(d, seed=14)
    x[-3:] = last
    g.LayerNorm(m, d, eps=EPS).run(x, gamma, x, beta=beta)
    ref.check_layer_norm("same", "bf16", last, None, gamma, beta, EPS, x[-3:])
    assert torch.equal(x[m // 2], beta)
    q, sc = torch.empty(m, d, dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    x[-3:] = last
    g.QuantRows(m, d).run(x, q, sc)
    ref.check_out("i8_rows", "bf16", last.cpu().double(), 0 * last.cpu().double(), q[-3:], sc[-3:])


# ------------------------------------------------------------------ backward
def run_bwd(dy, s, gamma, ds, dtype, eps=EPS, want="gb", workspace=None, stream=None):
    m, d = dy.shape
    dX, dg, db = Guarded(m * d, T16[dtype]), Guarded(d, T16[dtype]), Guarded(d, T16[dtype])
    g.LayerNorm(m, d, dtype, eps=eps).run_bwd(dy, s, gamma, dX.t, dgamma=dg.t if "g" in want else None, dbeta=db.t if "b" in want else None,
                                              dS=ds, workspace=workspace, stream=stream)
    torch.cuda.synchronize()
    assert dX.intact() and dg.intact() and db.intact()
    return dX.t.view(m, d), dg.t if "g" in want else None, db.t if "b" in want else None


# one cluster (a row on 8, 32, 128, 512 threads; one turn and two), few rows with partial sums, and every shape of many rows
BWD = [(1, 8), (3, 64), (1000, 64), (1024, 56), (256, 256), (37, 1000), (64, 1024), (8, 4096), (16, 4096), (16, 2056),
       (1100, 64), (300, 256), (70, 1024), (17, 4096), (37, 2048), (3, 8192), (2, 16384),
       (26, 5000), (3, 6144),
       (40000, 64), (20011, 128), (20011, 104), (9001, 256), (5003, 512), (2001, 1024), (1203, 2048), (601, 4096), (600, 4008), (450, 5000), (400, 6144),
       (333, 8192), (151, 8200), (150, 12288), (150, 16384)]


@pytest.mark.parametrize("skip", [False, True])
@pytest.mark.parametrize("m,d", BWD)
def test_layer_norm_bwd(m, d, skip):
    dtype = "f16" if (m + d // 8) % 2 else "bf16"
    dy, s, gamma = randn(m, d, seed=1, dtype=dtype), randn(m, d, seed=2, dtype=dtype, scale=2.0) + 1.0, randn(d, seed=3, dtype=dtype)
    ds = randn(m, d, seed=4, dtype=dtype) if skip else None
    dX, dg, db = run_bwd(dy, s, gamma, ds, dtype)
    ref.check_layer_norm_bwd(dtype, dy, s, gamma, ds, EPS, dX, dg, db)


@pytest.mark.parametrize("m,d", [(37, 1000), (8, 4096), (500, 4096), (3000, 512)])
def test_either_gradient_may_be_left_out(m, d):
    dy, s, gamma = randn(m, d, seed=1), randn(m, d, seed=2), randn(d, seed=3)
    dX, dg, db = run_bwd(dy, s, gamma, None, "bf16")
    for want in ("g", "b", ""):
        x, a, b = run_bwd(dy, s, gamma, None, "bf16", want=want)
        assert (a is None or torch.equal(a, dg)) and (b is None or torch.equal(b, db))
        # (a call without sums may deal its rows otherwise, but dX is a row's own)
        ref.check_layer_norm_bwd("bf16", dy, s, gamma, None, EPS, x)


@pytest.mark.parametrize("m,d", [(64, 1024), (601, 4096), (151, 16384)])
def test_bwd_in_place_and_from_run_to_run(m, d):
    dy, s, gamma, ds = (randn(*k, seed=i) for i, k in enumerate([(m, d), (m, d), (d,), (m, d)]))
    dX, dg, db = run_bwd(dy, s, gamma, ds, "bf16")
    for over in range(3):
        t = [dy.clone(), s.clone(), ds.clone()]
        a, b = torch.empty_like(dg), torch.empty_like(db)
        g.LayerNorm(m, d, eps=EPS).run_bwd(t[0], t[1], gamma, t[over], dgamma=a, dbeta=b, dS=t[2])
        assert torch.equal(t[over], dX) and torch.equal(a, dg) and torch.equal(b, db)


def test_bwd_constant_rows():
    """No deviation: u is 0 and the gradient is that of the mean's removal over sqrt(eps)."""
    dy, s, gamma = randn(6, 512, seed=1), torch.full((6, 512), 5.0, dtype=torch.bfloat16, device="cuda"), randn(512, seed=2)
    dX, dg, db = run_bwd(dy, s, gamma, None, "bf16")
    ref.check_layer_norm_bwd("bf16", dy, s, gamma, None, EPS, dX, dg, db)


def test_bwd_scratch_that_is_too_small_is_refused():
    dy, s, gamma = randn(601, 4096, seed=1), randn(601, 4096, seed=2), randn(4096, seed=3)
    with pytest.raises(g.GemmEpiError) as e:
        run_bwd(dy, s, gamma, None, "bf16", workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == g.ERR_ARG


# ------------------------------------------------------------------ rows quantised alone
@pytest.mark.parametrize("out", ["i8_rows", "e4m3_rows"])
@pytest.mark.parametrize("m,d", SHAPES + [(3, 16400), (2, 40000), (1, 131072)])
def test_quant_rows(m, d, out):
    dtype = "f16" if m % 2 else "bf16"
    x = randn(m, d, seed=3, dtype=dtype, scale=3.0)
    x[0, d // 2] = 0
    q, sc = Guarded(m * d, OUT_T[out]), Guarded(m, torch.float32)
    g.QuantRows(m, d, dtype, out).run(x, q.t, sc.t)
    torch.cuda.synchronize()
    assert q.intact() and sc.intact()
    ref.check_out(out, dtype, x.cpu().double(), 0 * x.cpu().double(), q.t.view(m, d), sc.t)


@pytest.mark.parametrize("d", [64, 4096, 20000])
def test_quant_rows_of_zeros_and_of_values_that_are_not_finite(d):
    x = randn(6, d, seed=3)
    x[1], x[2], x[3, 7], x[4, d - 1] = 0, 1e-38, float("nan"), float("-inf")
    q, sc = torch.empty(6, d, dtype=torch.int8, device="cuda"), torch.empty(6, device="cuda")
    g.QuantRows(6, d).run(x, q, sc)
    assert sc[1:3].tolist() == [1.0, 1.0] and not q[1:3].any() and not sc[3:5].isfinite().any()
    keep = x[[0, 5]].cpu().double()
    ref.check_out("i8_rows", "bf16", keep, 0 * keep, q[[0, 5]], sc[[0, 5]])


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("m,d", [(1, 16), (257, 64), (5, 128), (7, 208), (2, 256), (65, 512), (9, 1008), (3, 2048), (33, 4096), (3, 8192), (3, 16384)])
def test_rms_norm_to_8_bit_integers(m, d, residual):
    x, gamma = randn(m, d, seed=1, scale=2.0), randn(d, seed=2)
    r = randn(m, d, seed=3) if residual else None
    q, sc = Guarded(m * d, torch.int8), Guarded(m, torch.float32)
    g.RmsNorm(m, d, out="i8_rows").run(x, gamma, q.t, residual=r, S=torch.empty_like(x) if residual else None, scale=sc.t)
    torch.cuda.synchronize()
    assert q.intact() and sc.intact()
    _, y = block_ref.norm(x.cpu(), None if r is None else r.cpu(), gamma.cpu(), 1e-6)
    ref.check_out("i8_rows", "bf16", y, block_ref.F32 * y.abs(), q.t.view(m, d), sc.t)


# ------------------------------------------------------------------ streams and graphs
def test_on_a_given_stream_and_captured():
    m, d = 601, 1024
    dy, s, gamma, beta = randn(m, d, seed=1), randn(m, d, seed=2), randn(d, seed=3), randn(d, seed=4)
    want = run_norm(s, None, gamma, beta, "bf16", "i8_rows") + run_bwd(dy, s, gamma, None, "bf16")
    fwd, bwd = g.LayerNorm(m, d, out="i8_rows"), g.LayerNorm(m, d, eps=EPS)
    q, sc, dX, dg, db = torch.empty(m, d, dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda"), torch.empty_like(dy), torch.empty_like(gamma), torch.empty_like(gamma)

    def both(stream=None):
        fwd.run(s, gamma, q, beta=beta, scale=sc, stream=stream)
        bwd.run_bwd(dy, s, gamma, dX, dgamma=dg, dbeta=db, stream=stream)

    def check():
        torch.cuda.synchronize()
        for got, w in zip((q, sc, dX, dg, db), (want[0], want[2], want[3], want[4], want[5])):
            assert torch.equal(got, w)
            got.zero_()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    both(side)
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for _ in range(2):
        graph.replay()
        check()


# ------------------------------------------------------------------ rows that are not finite, to 8-bit integers
@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("d", [16, 64, 128, 1008, 4096, 16384])
def test_a_row_that_is_not_finite_has_no_finite_scale(d, residual, norm):
    """Its codes say nothing, so the scale has to: rows of NaN, a NaN among zeros, infinities, and every row beside a gain that is NaN."""
    m = 11
    x, gamma = randn(m, d, seed=1), randn(d, seed=2)
    r = randn(m, d, seed=3) if residual else None
    plan = (g.RmsNorm if norm == "rms" else g.LayerNorm)(m, d, out="i8_rows")

    def run(x, gamma):
        q, sc = torch.empty(m, d, dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
        plan.run(x, gamma, q, residual=r, scale=sc)
        return q, sc

    want, scales = run(x, gamma)
    assert scales.isfinite().all()
    bad = x.clone()
    bad[0], bad[3] = float("nan"), 0
    bad[3, d - 1], bad[6, d // 2], bad[8] = float("nan"), float("inf"), float("-inf")
    if residual:
        r[3] = 0
    q, sc = run(bad, gamma)
    keep = [1, 2, 4, 5, 7, 9, 10]
    assert torch.equal(q[keep], want[keep]) and torch.equal(sc[keep], scales[keep]) and not sc[[0, 3, 6, 8]].isfinite().any()
    odd = gamma.clone()
    odd[d // 3] = float("nan")
    assert not run(x, odd)[1].isfinite().any()
    x[5] = 0
    if residual:
        r[5] = 0
    assert not run(x, odd)[1].isfinite().any()


# ------------------------------------------------------------------ the backward's mean
@pytest.mark.parametrize("dtype,mean,spread", [("bf16", 1000.0, 0.0), ("f16", 30000.0, 0.0), ("f16", 1000.0, 0.5), ("bf16", 256.0, 2.0), ("f16", 0.0, 1.0)])
@pytest.mark.parametrize("m,d", [(9, 40), (9, 200), (9, 1000), (9, 4000), (17, 4000), (1300, 56), (40000, 56), (20011, 104), (9001, 248), (5003, 504),
                                 (2500, 1000), (1203, 2040), (601, 4040), (601, 4096), (400, 6200), (333, 8200), (180, 12400)])
def test_bwd_means_far_from_the_deviations(m, d, dtype, mean, spread):
    """Constant and nearly constant rows of a large mean, whose own rounding is not part of u (block8_ref.layer_norm_bwd_close).  Every
    seventh row begins with an outlier."""
    s = (randn(m, d, seed=5, dtype="bf16").float() * spread + mean).to(T16[dtype])
    s[::7, 0] = mean / 2 + 3
    dy, gamma = randn(m, d, seed=6, dtype=dtype), randn(d, seed=7, dtype=dtype)
    dX, dg, db = run_bwd(dy, s, gamma, None, dtype)
    dx, wg, wb, ox, og, ob = ref.layer_norm_bwd_close(dtype, dy.cpu(), s.cpu(), gamma.cpu(), EPS)
    block_ref.close(dX, dx, block_ref.rounded(dx, dtype, ox), "dX")
    block_ref.close(dg, wg, block_ref.rounded(wg, dtype, og), "dgamma")
    block_ref.close(db, wb, block_ref.rounded(wb, dtype, ob), "dbeta")


# ------------------------------------------------------------------ codes at ties
@pytest.mark.parametrize("dtype,bits", [("bf16", 8), ("f16", 11)])
def test_int8_codes_are_the_nearest(dtype, bits):
    """Every mantissa as a row's largest value, every mantissa beside it at nine sizes: the code is the one nearest to the exact quotient
    127 v / top, and the even one at a tie but for f16's, where 127 divides top's digits (they may go up)."""
    low = 2 ** (bits - 1)
    digits = torch.arange(low, 2 * low, dtype=torch.int64)
    top = digits[:, None]                                            # in units of 2^-8 below
    v = torch.cat([digits << (8 - s) for s in range(9)])[None, :].expand(low, -1)
    v = torch.where(v > top << 8, 0, v)                              # (256 v is what stands for a value v)
    x = torch.cat([(top << 8), v, torch.zeros(low, 15, dtype=torch.int64)], 1).double() / 2 ** 12
    x[1::2] *= -1
    x16 = x.to(T16[dtype])
    assert torch.equal(x16.double(), x)
    q, sc = torch.empty(x.shape, dtype=torch.int8, device="cuda"), torch.empty(low, device="cuda")
    g.QuantRows(low, x.shape[1], dtype).run(x16.cuda(), q, sc)
    got = q.cpu().long()
    got[1::2] *= -1
    num, den = 127 * torch.cat([(top << 8), v, torch.zeros(low, 15, dtype=torch.int64)], 1), top << 8
    floor, rest = num // den, num % den
    tie = 2 * rest == den
    want = torch.where(2 * rest < den, floor, torch.where(tie, floor + (floor & 1), floor + 1))
    may_go_up = tie & (top % 127 == 0) & (dtype == "f16")
    assert tie.any() and torch.equal(got[~may_go_up], want[~may_go_up]) and ((got == want) | (got == floor + 1))[may_go_up].all()
