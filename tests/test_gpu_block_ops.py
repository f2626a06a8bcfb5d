"""The norm, its backward and the epilogue's backward on the GPU, against the formulas in 64 bits
(block_ref, where the bounds are derived)."""
import pytest
import torch

import block_ref as ref
from block_ref import T16

from activation_epilogue_tcgen05_b200 import gemm_epi as g

pytestmark = pytest.mark.gpu
EPS = 1e-6
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.get_device_capability() != (10, 0):
        pytest.skip("needs sm_100")
    from activation_epilogue_tcgen05_b200 import build
    build.build()


def randn(*shape, seed=0, dtype="bf16", scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=gen) * scale).to(T16[dtype]).cuda()


class Guarded:
    """A buffer between two guard bands that a call must leave as they were."""

    def __init__(self, count, dtype):
        size = torch.empty((), dtype=dtype).element_size()
        self.raw = torch.full((count * size + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        self.t = self.raw[256:256 + count * size].view(dtype)

    def intact(self):
        return bool((self.raw[:256] == 0xA5).all() and (self.raw[-256:] == 0xA5).all())


def run_norm(x, r, gamma, dtype, out, eps=EPS, scale=None, amax=None, keep=True, stream=None):
    m, d = x.shape
    Y = Guarded(m * d, T16[dtype] if out == "same" else E4M3)
    S = Guarded(m * d, T16[dtype]) if r is not None and keep else None
    rows = Guarded(m, torch.float32) if out == "e4m3_rows" else None
    g.RmsNorm(m, d, dtype, out, eps).run(x, gamma, Y.t, residual=r, S=S and S.t, scale=rows.t if rows else scale,
                                         amax=amax, stream=stream)
    torch.cuda.synchronize()
    assert all(b.intact() for b in (Y, S, rows) if b is not None)
    return Y.t.view(m, d), S and S.t.view(m, d), rows.t if rows else scale


# every row length's own kernel (a few threads of a warp, a warp, several warps; full and ragged), and the limits
SHAPES = [(1, 16), (3, 16), (257, 64), (5, 128), (1023, 128), (7, 208), (2, 256), (65, 512), (9, 1008), (3, 1024), (4, 1040), (2, 2048),
          (1, 4096), (33, 4096), (5, 4112), (3, 8192), (2, 8208), (2, 14336), (3, 16384)]


@pytest.mark.parametrize("out", ["same", "e4m3", "e4m3_rows"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,d", SHAPES)
def test_norm(m, d, dtype, residual, out):
    x, gamma = randn(m, d, seed=1, dtype=dtype, scale=2.0), randn(d, seed=2, dtype=dtype)
    r = randn(m, d, seed=3, dtype=dtype, scale=3.0) if residual else None
    scale = torch.tensor([2.0 / 448], device="cuda") if out == "e4m3" else None       # the largest values saturate
    amax = torch.full((1,), 1e9, device="cuda") if out == "e4m3" else None
    Y, S, sc = run_norm(x, r, gamma, dtype, out, scale=scale, amax=amax)
    ref.check_norm(out, dtype, x, r, gamma, EPS, Y, S, sc, amax)


@pytest.mark.parametrize("m,d", [(5, 8), (3, 1000), (2, 4104), (3, 16376)])
def test_norm_lengths_that_are_no_multiple_of_16(m, d):
    x, gamma, r = randn(m, d, seed=1), randn(d, seed=2), randn(m, d, seed=3)
    Y, S, _ = run_norm(x, r, gamma, "bf16", "same")
    ref.check_norm("same", "bf16", x, r, gamma, EPS, Y, S)


@pytest.mark.parametrize("out", ["same", "e4m3", "e4m3_rows"])
@pytest.mark.parametrize("d", [64, 512, 4096])
def test_norm_rows_of_zeros_and_of_tiny_and_large_values(d, out):
    x = randn(6, d, seed=4, dtype="bf16")
    x[1] = 0
    x[2] = 1e-38                       # squares vanish beside eps; below any scale in use
    x[3] *= 1e15
    x[4] = 0
    x[4, d - 1] = 7.0                  # one value carries the row
    gamma = randn(d, seed=5, dtype="bf16")
    gamma[0] = 0
    scale = torch.tensor([0.01], device="cuda") if out == "e4m3" else None
    Y, _, sc = run_norm(x, None, gamma, "bf16", out, scale=scale)
    if out == "e4m3_rows":
        # a row whose largest y is below 1e-35 times its rho counts as zeros
        assert float(sc[1]) == 1.0 and float(sc[2]) == 1.0 and not Y[1:3].float().any()
        keep = [0, 3, 4, 5]
        ref.check_norm(out, "bf16", x[keep], None, gamma, EPS, Y[keep], None, sc[keep])
    else:
        ref.check_norm(out, "bf16", x, None, gamma, EPS, Y, None, sc)


def test_norm_takes_the_unrounded_sum():
    """x + r that cancels to below the type's step of r: the norm sees the difference, S its rounding."""
    r = torch.full((4, 256), 256.0, dtype=torch.bfloat16, device="cuda")
    x = randn(4, 256, seed=6, scale=0.25)
    gamma = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    Y, S, _ = run_norm(x - 0, r, gamma, "bf16", "same")
    ref.check_norm("same", "bf16", x, r, gamma, EPS, Y, S)


@pytest.mark.parametrize("eps", [1e-12, 1e-5, 1.0, 1e4])
def test_norm_eps(eps):
    x, gamma = randn(5, 384, seed=7, scale=0.01), randn(384, seed=8)
    Y, _, _ = run_norm(x, None, gamma, "bf16", "same", eps=eps)
    ref.check_norm("same", "bf16", x, None, gamma, eps, Y)


@pytest.mark.parametrize("d", [128, 1024, 4096])
def test_norm_in_place(d):
    """The stream updated in place (S over the residual, Y over x) gives the same bits."""
    x, r, gamma = randn(67, d, seed=9), randn(67, d, seed=10), randn(d, seed=11)
    Y, S, _ = run_norm(x, r, gamma, "bf16", "same")
    for s_over, y_over in [("r", "x"), ("x", "r")]:
        b = {"x": x.clone(), "r": r.clone()}
        g.RmsNorm(67, d).run(b["x"], gamma, b[y_over], residual=b["r"], S=b[s_over])
        assert torch.equal(b[s_over], S) and torch.equal(b[y_over], Y)
    b = x.clone()
    g.RmsNorm(67, d).run(b, gamma, b)
    assert torch.equal(b, run_norm(x, None, gamma, "bf16", "same")[0])
    assert torch.equal(run_norm(x, r, gamma, "bf16", "same", keep=False)[0], Y)


def test_norm_offsets_beyond_32_bits():
    m, d = 140_000, 16_384             # 2.3 G elements, 4.6 GB
    x = torch.zeros(m, d, dtype=torch.bfloat16, device="cuda")
    last = randn(3, d, seed=12)
    x[-3:] = last
    gamma = randn(d, seed=13)
    g.RmsNorm(m, d).run(x, gamma, x)
    ref.check_norm("same", "bf16", last, None, gamma, EPS, x[-3:])
    assert not x[:4].any() and not x[70_000:70_004].any()


def test_norm_of_a_side_stream_and_of_a_replayed_graph():
    x, r, gamma = randn(300, 2048, seed=14), randn(300, 2048, seed=15), randn(2048, seed=16)
    want = [t.clone() for t in run_norm(x, r, gamma, "bf16", "e4m3_rows")]
    got = run_norm(x, r, gamma, "bf16", "e4m3_rows", stream=torch.cuda.Stream())
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    op, Y, S = g.RmsNorm(300, 2048, out="e4m3"), torch.empty(300, 2048, dtype=E4M3, device="cuda"), torch.empty_like(x)
    scale, amax = torch.tensor([0.01], device="cuda"), torch.zeros(1, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op.run(x, gamma, Y, residual=r, S=S, scale=scale, amax=amax)
    for k in range(3):                 # smaller inputs later: the maximum starts anew in each replay
        x.mul_(0.5)
        gamma.mul_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        ref.check_norm("e4m3", "bf16", x, r, gamma, EPS, Y, S, scale, amax)


# ------------------------------------------------------------------ backward of the norm
def run_norm_bwd(dy, s, gamma, ds, dtype, eps=EPS, want=True, **kw):
    m, d = s.shape
    dX, dg = Guarded(m * d, T16[dtype]), Guarded(d, T16[dtype]) if want else None
    nbytes = g.gemm_epi_rmsnorm_workspace_bytes(m, d)
    ws = Guarded(nbytes, torch.uint8)
    g.RmsNorm(m, d, dtype, eps=eps).run_bwd(dy, s, gamma, dX.t, dgamma=dg and dg.t, dS=ds, workspace=ws.t, **kw)
    torch.cuda.synchronize()
    assert all(b.intact() for b in (dX, dg, ws) if b is not None)
    return dX.t.view(m, d), dg and dg.t


@pytest.mark.parametrize("skip", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,d", SHAPES + [(5, 8), (37, 1000), (64, 1024), (65, 1024), (16, 4096), (17, 4096), (256, 256), (257, 248), (1024, 64), (1025, 64), (700, 4104), (1500, 264), (301, 16376)])
def test_norm_bwd(m, d, dtype, skip):
    dy, s, gamma = randn(m, d, seed=1, dtype=dtype), randn(m, d, seed=2, dtype=dtype, scale=2.0), randn(d, seed=3, dtype=dtype)
    ds = randn(m, d, seed=4, dtype=dtype) if skip else None
    dX, dg = run_norm_bwd(dy, s, gamma, ds, dtype)
    ref.check_norm_bwd(dtype, dy, s, gamma, ds, EPS, dX, dg)
    assert torch.equal(run_norm_bwd(dy, s, gamma, ds, dtype, want=False)[0], dX)
    again = run_norm_bwd(dy, s, gamma, ds, dtype)
    assert torch.equal(again[0], dX) and torch.equal(again[1], dg)         # the order of the sums is fixed


def test_norm_bwd_rows_of_zeros():
    dy, s, gamma = randn(4, 256, seed=1), randn(4, 256, seed=2), randn(256, seed=3)
    s[1] = 0
    dy[2] = 0
    dX, dg = run_norm_bwd(dy, s, gamma, None, "bf16", eps=1e-3)
    ref.check_norm_bwd("bf16", dy, s, gamma, None, 1e-3, dX, dg)


@pytest.mark.parametrize("over", ["dy", "s", "ds"])
@pytest.mark.parametrize("d", [64, 1024, 8192])
def test_norm_bwd_in_place(d, over):
    b = {"dy": randn(40, d, seed=1), "s": randn(40, d, seed=2), "ds": randn(40, d, seed=3)}
    gamma = randn(d, seed=4)
    dX, dg = run_norm_bwd(b["dy"], b["s"], gamma, b["ds"], "bf16")
    dg2 = torch.empty_like(gamma)
    g.RmsNorm(40, d).run_bwd(b["dy"], b["s"], gamma, b[over], dgamma=dg2, dS=b["ds"])
    assert torch.equal(b[over], dX) and torch.equal(dg2, dg)


@pytest.mark.parametrize("over", ["dy", "s", "ds"])
@pytest.mark.parametrize("m,d", [(5000, 64), (3000, 1024), (1500, 4096), (400, 16384)])
def test_norm_bwd_in_place_over_many_rows(m, d, over):
    """A block's later rows are on their way while an earlier one is overwritten."""
    b = {"dy": randn(m, d, seed=1), "s": randn(m, d, seed=2), "ds": randn(m, d, seed=3)}
    gamma = randn(d, seed=4)
    dX, dg = run_norm_bwd(b["dy"], b["s"], gamma, b["ds"], "bf16")
    ref.check_norm_bwd("bf16", b["dy"], b["s"], gamma, b["ds"], EPS, dX, dg)
    dg2 = torch.empty_like(gamma)
    g.RmsNorm(m, d).run_bwd(b["dy"], b["s"], gamma, b[over], dgamma=dg2, dS=b["ds"])
    assert torch.equal(b[over], dX) and torch.equal(dg2, dg)


def test_scratch_of_a_given_stream():
    """Scratch from torch's allocator belongs to the stream of the call: a Stream, its raw handle, the default."""
    dy, s, gamma = randn(500, 1024, seed=1), randn(500, 1024, seed=2), randn(1024, seed=3)
    dX, dg = run_norm_bwd(dy, s, gamma, None, "bf16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for st in (side, side.cuda_stream, torch.cuda.default_stream(), 0):
        out, dgamma, db = torch.empty_like(dy), torch.empty_like(gamma), torch.empty_like(gamma)
        side.wait_stream(torch.cuda.current_stream())
        for _ in range(3):
            g.RmsNorm(500, 1024).run_bwd(dy, s, gamma, out, dgamma=dgamma, stream=st)
            g.ActBackward(500, 1024, "bf16", "bias", "col").run(dy, dbias=db, stream=st)
        torch.cuda.synchronize()
        assert torch.equal(out, dX) and torch.equal(dgamma, dg)
        ref.check_dact("bias", "col", "bf16", dy, torch.zeros(500, 1024), None, db)


def test_norm_gradients_against_differences():
    """Along random directions, the kernel's gradients against central differences of the forward formula."""
    m, d = 6, 512
    x, gamma, dy = randn(m, d, seed=1, dtype="f16"), randn(d, seed=2, dtype="f16"), randn(m, d, seed=3, dtype="f16")
    dX, dg = (t.cpu().double() for t in run_norm_bwd(dy, x, gamma, None, "f16", eps=1e-3))
    X, G, W = x.cpu().double(), gamma.cpu().double(), dy.cpu().double()
    gen = torch.Generator().manual_seed(5)
    v, w = torch.randn(m, d, generator=gen, dtype=torch.float64), torch.randn(d, generator=gen, dtype=torch.float64)
    f = lambda t, u: float((ref.norm(X + t * v, None, G + u * w, 1e-3)[1] * W).sum())     # noqa: E731
    h = 1e-5
    # the gradients' own roundings (half a step each) and fp32, weighted by the direction
    _, _, size, dsize = ref.norm_bwd(W, X, G, None, 1e-3)
    allow = float((ref.rounded(dX, "f16", ref.F32 * size) * v.abs()).sum()) + 1e-6
    assert abs((f(h, 0) - f(-h, 0)) / (2 * h) - float((dX * v).sum())) <= allow
    allow = float((ref.rounded(dg, "f16", ref.F32 * dsize) * w.abs()).sum()) + 1e-6
    assert abs((f(0, h) - f(0, -h)) / (2 * h) - float((dg * w).sum())) <= allow


def test_norm_bwd_two_graphs_at_once():
    """Two captured calls on two streams, each with scratch of its own from torch's allocator, replayed together."""
    op, sets, graphs = g.RmsNorm(900, 1024), [], []
    for k in range(2):
        t = [randn(900, 1024, seed=10 * k + i) for i in range(2)] + [randn(1024, seed=10 * k + 2)]
        sets.append(t + [torch.empty_like(t[0]), torch.empty_like(t[2])])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            dy, s, gamma, dX, dg = sets[k]
            op.run_bwd(dy, s, gamma, dX, dgamma=dg)
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for dy, s, gamma, dX, dg in sets:
        ref.check_norm_bwd("bf16", dy, s, gamma, None, EPS, dX, dg)


# ------------------------------------------------------------------ backward of the epilogue
DACT = ["none", "bias", "relu_bias", "relu", "relu_aux_bias", "relu_aux", "gelu_bias", "gelu", "tanh_bias", "tanh"]


def run_dact(dd, z, dtype, epilogue, axis, bias=True, **kw):
    m, n = dd.shape
    plain, mask = epilogue in ("none", "bias"), "aux" in epilogue
    dZ = None if plain else Guarded(m * n, T16[dtype])
    db = Guarded(m if axis == "row" else n, T16[dtype]) if bias else None
    ws = Guarded(g.gemm_epi_dact_workspace_bytes(m, n, g.AXIS[axis]), torch.uint8)
    g.ActBackward(m, n, "e4m3" if dtype == "bf16" and m % 2 else dtype, epilogue, axis).run(
        dd, dZ=dZ and dZ.t, z=None if plain or mask else z, aux=ref.pack_mask(z) if mask else None, dbias=db and db.t,
        workspace=ws.t if bias else None, **kw)
    torch.cuda.synchronize()
    assert all(b.intact() for b in (dZ, db, ws) if b is not None)
    return dZ and dZ.t.view(m, n), db and db.t


@pytest.mark.parametrize("axis", ["row", "col"])
@pytest.mark.parametrize("epilogue", DACT)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,n", [(1, 8), (3, 264), (129, 40), (130, 1000)])
def test_dact(m, n, dtype, epilogue, axis):
    dd, z = randn(m, n, seed=1, dtype=dtype), randn(m, n, seed=2, dtype=dtype, scale=2.0)
    z[0, 0] = 0.0
    dZ, db = run_dact(dd, z, dtype, epilogue, axis)
    ref.check_dact(epilogue, axis, dtype, dd, z, dZ, db)
    again = run_dact(dd, z, dtype, epilogue, axis)
    assert (dZ is None or torch.equal(again[0], dZ)) and torch.equal(again[1], db)
    if dZ is not None:
        assert torch.equal(run_dact(dd, z, dtype, epilogue, axis, bias=False)[0], dZ)


@pytest.mark.parametrize("axis", ["row", "col"])
@pytest.mark.parametrize("m,n", [(5000, 256), (16, 16384), (1, 20000), (2049, 2056), (70000, 8),
                                 (1775, 6152), (1776, 6152), (7, 40000), (2, 2048), (5, 4096), (301, 6144), (2001, 16392), (64, 4104), (65, 4104), (33, 70000)])
def test_dact_long_and_wide(m, n, axis):
    dd, z = randn(m, n, seed=3), randn(m, n, seed=4)
    dZ, db = run_dact(dd, z, "bf16", "gelu_bias", axis)
    ref.check_dact("gelu_bias", axis, "bf16", dd, z, dZ, db)


@pytest.mark.parametrize("epilogue", ["gelu", "tanh", "relu"])
def test_dact_far_from_zero(epilogue):
    """Slopes far out on both sides: 0 and 1 (tanh: 0), never NaN."""
    z = torch.linspace(-60000, 60000, 4096).to(torch.float16).cuda().view(16, 256)
    dd = torch.ones_like(z)
    dZ, db = run_dact(dd, z, "f16", epilogue, "col")
    ref.check_dact(epilogue, "col", "f16", dd, z, dZ, db)


@pytest.mark.parametrize("m", [70, 20000])
@pytest.mark.parametrize("over", ["dd", "z"])
def test_dact_in_place(over, m):
    b = {"dd": randn(m, 520, seed=5), "z": randn(m, 520, seed=6)}
    want = run_dact(b["dd"], b["z"], "bf16", "gelu_bias", "col")
    db = torch.empty(520, dtype=torch.bfloat16, device="cuda")
    g.ActBackward(m, 520, "bf16", "gelu_bias", "col").run(b["dd"], dZ=b[over], z=b["z"], dbias=db)
    assert torch.equal(b[over], want[0]) and torch.equal(db, want[1])


def test_dact_ignores_the_masks_padding():
    dd, z = randn(9, 200, seed=7), randn(9, 200, seed=8)
    aux = ref.pack_mask(z)
    full = aux.view(9, -1).clone()
    full[:, 200 // 32] |= -1 << (200 % 32)
    full[:, 200 // 32 + 1:] = -1
    out = []
    for a in (aux, full.view(-1)):
        dZ, db = torch.empty_like(dd), torch.empty(9, dtype=torch.bfloat16, device="cuda")
        g.ActBackward(9, 200, "bf16", "relu_aux", "row").run(dd, dZ=dZ, aux=a, dbias=db)
        out.append((dZ, db))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])


@pytest.mark.parametrize("axis", ["row", "col"])
def test_dact_offsets_beyond_32_bits(axis):
    m, n = 140_000, 16_384
    dd = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
    last = randn(2, n, seed=9)
    dd[-2:] = last
    db = torch.empty(m if axis == "row" else n, dtype=torch.bfloat16, device="cuda")
    g.ActBackward(m, n, "bf16", "bias", axis).run(dd, dbias=db)
    ref.check_dact("bias", axis, "bf16", last, torch.zeros(2, n), None, db[-2:] if axis == "row" else db)
    assert axis == "col" or not db[:-2].any()


# ------------------------------------------------------------------ refusals of the objects
def test_objects_refuse_tensors_that_do_not_fit():
    op, x, gamma = g.RmsNorm(4, 64), randn(4, 64), randn(64)
    y = torch.empty_like(x)
    bad = [dict(X=x.cpu()), dict(X=x.half()), dict(X=x[:3]), dict(X=randn(64, 4).t()), dict(gamma=gamma[:32]), dict(Y=y.float()),
           dict(residual=x[:, :32]), dict(X=None), dict(Y=randn(4, 128)[:, :64])]
    for kw in bad:
        with pytest.raises(g.GemmEpiError):
            op.run(**{**dict(X=x, gamma=gamma, Y=y), **kw})
    with pytest.raises(g.GemmEpiError):
        g.RmsNorm(4, 64, out="e4m3_rows").run(x, gamma, torch.empty(4, 64, dtype=E4M3, device="cuda"))       # no scales
    with pytest.raises(g.GemmEpiError):
        b = randn(2000, 64)
        g.RmsNorm(2000, 64).run_bwd(b, b, gamma, torch.empty_like(b), dgamma=torch.empty_like(gamma),
                                    workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(g.GemmEpiError):
        g.ActBackward(4, 64, "bf16", "gelu").run(x, dZ=y)                                                  # no z
    with pytest.raises(g.GemmEpiError):
        g.ActBackward(4, 64, "bf16", "relu_aux").run(x, dZ=y, aux=torch.zeros(3, dtype=torch.int32, device="cuda"))
