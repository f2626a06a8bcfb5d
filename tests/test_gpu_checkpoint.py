"""Activation checkpoints in 8 bits and the epilogue's backward from them on the GPU, against the formulas in 64 bits."""
import pytest
import torch

import block8_ref as ref
import block_ref
from block_ref import T16
from test_gpu_block_ops import Guarded, _cuda, randn  # noqa: F401

from activation_epilogue_tcgen05_b200 import gemm_epi as g

pytestmark = pytest.mark.gpu
SIZES = [(1, 8), (3, 24), (5, 32), (7, 40), (2, 256), (129, 264), (1000, 72), (33, 1000), (1023, 4104), (3, 14336), (2000, 96)]
EPILOGUES = ["none", "relu_bias", "gelu_bias", "tanh"]


def pre(m, n, dtype, seed=1):
    """Values of many sizes: groups of 32 columns apart by powers of two, some values 0."""
    z = randn(m, n, seed=seed, dtype=dtype).float()
    size = torch.exp2(torch.randint(-9, 3, (m, -(-n // 32)), generator=torch.Generator().manual_seed(seed)).float()).cuda()
    z = z * size.repeat_interleave(32, dim=1)[:, :n]
    z[:, ::7] = 0
    return z.to(T16[dtype])


def save(z, dtype, epilogue, H=True, stream=None):
    m, n = z.shape
    codes, exps, h = Guarded(m * n, torch.int8), Guarded(m * -(-n // 32), torch.uint8), Guarded(m * n, T16[dtype])
    g.ActCheckpoint(m, n, dtype, epilogue).save(z, codes.t, exps.t, H=h.t if H else None, stream=stream)
    torch.cuda.synchronize()
    assert codes.intact() and exps.intact() and h.intact()
    return codes.t.view(m, n), exps.t.view(m, -1), h.t.view(m, n)


@pytest.mark.parametrize("epilogue", EPILOGUES)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,n", SIZES)
def test_save_and_load(m, n, dtype, epilogue):
    z = pre(m, n, dtype)
    codes, exps, h = save(z, dtype, epilogue)
    q, e, k = ref.checkpoint(z.cpu())
    assert torch.equal(codes.cpu().double(), q) and torch.equal(exps.cpu().double(), e)
    ref.check_act(epilogue, dtype, z, h)
    ck = g.ActCheckpoint(m, n, dtype, epilogue)
    for act in (False, True):
        x = Guarded(m * n, T16[dtype])
        ck.load(codes, exps, x.t, act=act)
        torch.cuda.synchronize()
        assert x.intact()
        if act:
            ref.check_act(epilogue, dtype, k, x.t.view(m, n))
        else:
            assert torch.equal(x.t.view(m, n).cpu(), k.to(T16[dtype]))


def test_every_bf16_value():
    """Each alone in its group: its own code and exponent, restored to within half a step; NaN, infinities and what is above
    127 * 2^121 as NaN."""
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    z = torch.zeros(65536, 32, dtype=torch.bfloat16)
    z[:, 3] = v
    codes, exps, _ = save(z.cuda(), "bf16", "none", H=False)
    x = torch.empty(65536, 32, dtype=torch.bfloat16, device="cuda")
    g.ActCheckpoint(65536, 32).load(codes, exps, x)
    x, d = x.cpu(), v.double()
    bad = ~(d.abs() <= 127 * 2.0 ** 121)
    assert (exps.cpu().view(-1)[bad] == 255).all() and x[bad].isnan().all()
    q, e, k = ref.checkpoint(z[~bad])
    assert torch.equal(exps.cpu()[~bad].double(), e) and torch.equal(codes.cpu()[~bad].double(), q) and torch.equal(x[~bad].double(), k)


def test_f16_values_up_to_the_largest():
    z = torch.zeros(4, 64, dtype=torch.float16)
    z[0, 0], z[1, 1], z[2, 40], z[3, 3] = 65504, -65504, float("inf"), 2.0 ** -24
    codes, exps, _ = save(z.cuda(), "f16", "none", H=False)
    x = torch.empty(4, 64, dtype=torch.float16, device="cuda")
    g.ActCheckpoint(4, 64, "f16").load(codes, exps, x)
    x = x.cpu()
    assert x[0, 0] == 65504 and x[1, 1] == -65504 and x[2, 32:].isnan().all() and not x[2, :32].any() and x[3, 3] == 2.0 ** -24


def test_a_group_that_is_not_finite_leaves_its_neighbours():
    z = pre(5, 160, "bf16")
    codes, exps, h = save(z, "bf16", "gelu_bias")
    z[1, 40], z[3, 100] = float("nan"), float("-inf")
    c, e, _ = save(z, "bf16", "gelu_bias")
    assert int(e[1, 1]) == 255 and int(e[3, 3]) == 255
    x, dz, hh, dd = (torch.empty_like(z) for _ in range(4))
    dd.fill_(1.0)
    g.ActCheckpoint(5, 160).load(c, e, x)
    g.ActBackward(5, 160, "bf16", "gelu_bias", "col").run_ckpt(dd, c, e, dz, H=hh)
    lost = torch.zeros(5, 160, dtype=torch.bool)
    lost[1, 32:64] = lost[3, 96:128] = True
    for t in (x, dz, hh):
        assert torch.equal(t.cpu().isnan(), lost)
    keep = torch.ones(5, 5, dtype=torch.bool)
    keep[1, 1] = keep[3, 3] = False
    assert torch.equal(e.cpu()[keep], exps.cpu()[keep]) and torch.equal(c.cpu()[~lost], codes.cpu()[~lost])


def test_save_in_place():
    z = pre(77, 1000, "bf16")
    codes, exps, h = save(z, "bf16", "gelu_bias")
    c, e = torch.empty_like(codes), torch.empty_like(exps)
    g.ActCheckpoint(77, 1000).save(z, c, e, H=z)
    assert torch.equal(c, codes) and torch.equal(e, exps) and torch.equal(z, h)


def test_offsets_beyond_32_bits():
    m, n = 140_000, 16_384
    z = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
    last = pre(2, n, "bf16")
    z[-2:] = last
    codes, exps = torch.empty(m, n, dtype=torch.int8, device="cuda"), torch.empty(m, n // 32, dtype=torch.uint8, device="cuda")
    g.ActCheckpoint(m, n).save(z, codes, exps)
    q, e, k = ref.checkpoint(last.cpu())
    assert torch.equal(codes[-2:].cpu().double(), q) and torch.equal(exps[-2:].cpu().double(), e) and not codes[: m // 2].any()
    z.fill_(1)
    g.ActCheckpoint(m, n).load(codes, exps, z)
    assert torch.equal(z[-2:].cpu().double(), k) and not z[m // 2].any()
    dbias = torch.empty(n, dtype=torch.bfloat16, device="cuda")
    z.fill_(1)
    g.ActBackward(m, n, "bf16", "relu_bias", "col").run_ckpt(z, codes, exps, z, dbias=dbias)
    assert torch.equal(z[-2:].cpu() > 0, k > 0) and not z[m // 2].any()


# ------------------------------------------------------------------ backward
@pytest.mark.parametrize("recompute", [False, True])
@pytest.mark.parametrize("axis", ["row", "col", None])
@pytest.mark.parametrize("epilogue", ["relu_bias", "gelu_bias", "tanh_bias"])
@pytest.mark.parametrize("m,n", SIZES + [(300, 16384), (4000, 520), (1024, 1024), (20000, 8), (1025, 264), (1024, 1032)])
def test_backward(m, n, epilogue, axis, recompute):
    dtype = "f16" if (m + n) % 3 == 0 else "bf16"
    dd, z = randn(m, n, seed=2, dtype=dtype), pre(m, n, dtype, seed=3)
    codes, exps, _ = save(z, dtype, "none", H=False)
    k = ref.kept(codes.cpu(), exps.cpu())
    dZ, H = Guarded(m * n, T16[dtype]), Guarded(m * n, T16[dtype])
    db = Guarded(m if axis == "row" else n, T16[dtype])
    g.ActBackward(m, n, dtype, epilogue, axis or "col").run_ckpt(dd, codes, exps, dZ.t, H=H.t if recompute else None,
                                                               dbias=db.t if axis else None)
    torch.cuda.synchronize()
    assert dZ.intact() and H.intact() and db.intact()
    block_ref.check_dact(epilogue, axis or "col", dtype, dd, k, dZ.t.view(m, n), db.t if axis else None)
    if recompute:
        # GELU: the slope's tail (within 1e-6, block_ref) times |z|; tanh 2^-21 of itself
        ref.check_act(epilogue, dtype, k, H.t.view(m, n), {"gelu_bias": 1e-6, "tanh_bias": 2.0 ** -21, "relu_bias": 0.0}[epilogue])


@pytest.mark.parametrize("epilogue", ["gelu_bias", "tanh_bias", "relu_bias"])
def test_the_gradient_is_that_of_the_kept_value(epilogue):
    """Without rounding between: dZ from the checkpoint against the kernel that reads the same z in 16 bits, bit for bit."""
    z = pre(500, 1000, "bf16", seed=4)
    codes, exps, _ = save(z, "bf16", "none", H=False)
    kept, dd = torch.empty_like(z), randn(500, 1000, seed=5)
    g.ActCheckpoint(500, 1000).load(codes, exps, kept)
    for axis, size in (("row", 500), ("col", 1000)):
        plan = g.ActBackward(500, 1000, "bf16", epilogue, axis)
        out = [torch.empty_like(z), torch.empty(size, dtype=torch.bfloat16, device="cuda"), torch.empty_like(z), torch.empty(size, dtype=torch.bfloat16, device="cuda")]
        plan.run(dd, dZ=out[0], z=kept, dbias=out[1])
        plan.run_ckpt(dd, codes, exps, out[2], dbias=out[3])
        assert torch.equal(out[0], out[2]) and torch.equal(out[1], out[3])


def test_backward_in_place_captured_and_on_a_stream():
    m, n = 700, 1032
    dd, z = randn(m, n, seed=6), pre(m, n, "bf16", seed=7)
    codes, exps, _ = save(z, "bf16", "none", H=False)
    plan = g.ActBackward(m, n, "bf16", "gelu_bias", "col")
    dZ, H, db = torch.empty_like(dd), torch.empty_like(dd), torch.empty(n, dtype=torch.bfloat16, device="cuda")
    plan.run_ckpt(dd, codes, exps, dZ, H=H, dbias=db)
    a, b, c = dd.clone(), torch.empty_like(dd), torch.empty_like(db)
    plan.run_ckpt(a, codes, exps, a, H=b, dbias=c)
    assert torch.equal(a, dZ) and torch.equal(b, H) and torch.equal(c, db)
    a = dd.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    plan.run_ckpt(a, codes, exps, b, H=a, dbias=c, stream=side)
    side.synchronize()
    assert torch.equal(b, dZ) and torch.equal(a, H) and torch.equal(c, db)
    ck, graph = g.ActCheckpoint(m, n), torch.cuda.CUDAGraph()
    cc, ee = torch.zeros_like(codes), torch.zeros_like(exps)
    with torch.cuda.graph(graph):
        ck.save(z, cc, ee, H=b)
        plan.run_ckpt(dd, cc, ee, a, dbias=c)
    for _ in range(2):
        for t in (cc, ee, a, b, c):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(cc, codes) and torch.equal(ee, exps) and torch.equal(a, dZ) and torch.equal(c, db)


def test_operands_are_checked():
    z, plan = randn(4, 64), g.ActCheckpoint(4, 64)
    codes, exps = torch.empty(4, 64, dtype=torch.int8, device="cuda"), torch.empty(4, 2, dtype=torch.uint8, device="cuda")
    for bad in (dict(Z=z.half()), dict(Z=z.t()), dict(codes=codes.view(torch.uint8)), dict(exps=exps[:, :1]), dict(exps=exps.cpu()), dict(codes=None)):
        with pytest.raises(g.GemmEpiError) as e:
            plan.save(**{**dict(Z=z, codes=codes, exps=exps), **bad})
        assert e.value.status in (g.ERR_ARG, g.ERR_NULL)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m", [1, 37, 5000])
def test_order_of_a_rows_sum(m, dtype):
    """dbias along rows adds eight neighbours as ((0+1)+(2+3)) + ((4+5)+(6+7)) in fp32, from a checkpoint as from D: the large
    values of a row cancel, so that another order leaves other bits."""
    d = randn(m, 8, seed=5, dtype=dtype) * 2.0 ** -12
    d[:, 0], d[:, 4] = randn(m, seed=6, dtype=dtype) * 1024, randn(m, seed=7, dtype=dtype) * 64
    d[:, 2], d[:, 6] = -d[:, 0], -d[:, 4]
    f = d.float()
    want = (((f[:, 0] + f[:, 1]) + (f[:, 2] + f[:, 3])) + ((f[:, 4] + f[:, 5]) + (f[:, 6] + f[:, 7]))).to(T16[dtype])
    other = (((f[:, 0] + f[:, 2]) + (f[:, 1] + f[:, 3])) + ((f[:, 4] + f[:, 6]) + (f[:, 5] + f[:, 7]))).to(T16[dtype])
    assert not torch.equal(want, other)
    got = Guarded(m, T16[dtype])
    g.ActBackward(m, 8, dtype, "bias", "row").run(d, dbias=got.t)
    torch.cuda.synchronize()
    assert got.intact() and torch.equal(got.t, want)
    one = torch.ones_like(d)                                     # z > 0: ReLU's slope is 1
    codes, exps, _ = save(one, dtype, "relu_bias")
    got, dz = Guarded(m, T16[dtype]), Guarded(m * 8, T16[dtype])
    g.ActBackward(m, 8, dtype, "relu_bias", "row").run_ckpt(d, codes, exps, dz.t.view(m, 8), dbias=got.t)
    torch.cuda.synchronize()
    assert got.intact() and dz.intact() and torch.equal(got.t, want) and torch.equal(dz.t.view(m, 8), d)


# ------------------------------------------------------------------ the ends of the range
# one for each kernel and shape of the backward: columns, no bias, rows whole in a block (two and four rows), narrow rows by
# warps, rows by strips
ENDS = [("col", 37, 1000), (None, 37, 1000), ("row", 37, 1000), ("row", 1800, 1032), ("row", 1024, 1024), ("row", 3000, 96), ("row", 40, 6152)]


@pytest.mark.parametrize("epilogue", ["relu_bias", "gelu_bias"])
@pytest.mark.parametrize("axis,m,n", ENDS)
def test_f16_values_beside_the_gradient_up_to_the_largest(axis, m, n, epilogue):
    """A z near f16's largest number is kept as 65536 in steps of 1024: act(z) beside dZ is drawn back to a number, as load's is."""
    z = pre(m, n, "f16", seed=8)
    z[0, :4] = torch.tensor([65504.0, 65056.0, 64992.0, -65504.0])
    z[m - 1, n - 1], z[m // 2, 40], z[m // 2, 41] = 65504.0, -65504.0, 65504.0
    z[m // 3, 64:72] = float("inf")
    codes, exps, _ = save(z, "f16", "none", H=False)
    dd, dZ, H, X = randn(m, n, seed=9, dtype="f16"), torch.empty_like(z), torch.empty_like(z), torch.empty_like(z)
    db = torch.empty(m if axis == "row" else n, dtype=torch.float16, device="cuda") if axis else None
    g.ActBackward(m, n, "f16", epilogue, axis or "col").run_ckpt(dd, codes, exps, dZ, H=H, dbias=db)
    g.ActCheckpoint(m, n, "f16", epilogue).load(codes, exps, X, act=True)
    lost = (exps == 255).repeat_interleave(32, dim=1)[:, :n]
    assert lost.any() and torch.equal(H.isnan(), lost) and torch.equal(X.isnan(), lost)
    assert not H.isinf().any() and not X.isinf().any() and H[0, 0] == 65504 and H[m - 1, n - 1] == 65504 and H[m // 2, 41] == 65504
    # (in the large groups every kept value is 0 or beyond 16, where both activations are max(z, 0) without a rounding)
    large = (exps >= 143).repeat_interleave(32, dim=1)[:, :n] & ~lost
    assert large.any() and torch.equal(H[large], X[large])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("epilogue", ["relu_bias", "gelu_bias", "tanh_bias"])
@pytest.mark.parametrize("axis,m,n", ENDS)
def test_a_group_that_is_not_finite_shows_in_the_gradient(axis, m, n, epilogue, dtype):
    """dZ, act(z) and dbias are NaN where a group's z is lost, whatever the activation, and what they were elsewhere."""
    z, dd = pre(m, n, dtype, seed=10), randn(m, n, seed=11, dtype=dtype)
    plan = g.ActBackward(m, n, dtype, epilogue, axis or "col")

    def run(z, recompute):
        codes, exps, _ = save(z, dtype, "none", H=False)
        dZ, H = torch.empty_like(z), torch.empty_like(z)
        db = torch.empty(m if axis == "row" else n, dtype=T16[dtype], device="cuda") if axis else None
        plan.run_ckpt(dd, codes, exps, dZ, H=H if recompute else None, dbias=db)
        return dZ, H, db

    want = run(z, True)
    bad, lost = z.clone(), torch.zeros(m, n, dtype=torch.bool, device="cuda")
    for i, j, v in ((0, 33, "inf"), (m // 2, n - 1, "-inf"), (m - 1, 0, "nan")) + (((m // 3, 70, "3.389e38"),) if dtype == "bf16" else ()):
        bad[i, j] = float(v)
        lost[i, j // 32 * 32: j // 32 * 32 + 32] = True
    assert bad[m // 3, 70].isfinite()
    for recompute in (True, False):
        dZ, H, db = run(bad, recompute)
        assert torch.equal(dZ.isnan(), lost) and torch.equal(dZ[~lost], want[0][~lost])
        assert not recompute or (torch.equal(H.isnan(), lost) and torch.equal(H[~lost], want[1][~lost]))
        if axis:
            touched = lost.any(1 if axis == "row" else 0)
            assert torch.equal(db.isnan(), touched) and torch.equal(db[~touched], want[2][~touched])
