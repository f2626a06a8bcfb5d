"""The operators around the MLP's products from their formulas, in 64 bits on the CPU, and the
bounds that the kernels' outputs are held to.

A rounding to nearest is off by at most half a step: U * |value| for normal numbers, TINY near
zero (half the smallest step of the type).  Everything before the one rounding is fp32: a sum of
squares (only positive terms) or any sum of N terms is off by at most N * 2^-24 of the sum of the
terms' magnitudes, and the kernels add at most 64 terms in a chain (a thread's own, then trees of
at most 32), so F32 = 2^-17 covers a sum and the few operations around it.
"""
import math

import torch

U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -4}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "e4m3": 2.0 ** -10}
F32 = 2.0 ** -17
T16 = {"f16": torch.float16, "bf16": torch.bfloat16}


def rounded(v, dtype, extra):
    """Allowance for `v` rounded once to `dtype` after being off by `extra`."""
    return U[dtype] * (v.abs() + extra) + TINY[dtype] + extra


def close(got, want, tol, what=""):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    bad = ~((got - want).abs() <= tol)            # NaN counts as bad
    if bad.any():
        i = tuple(int(k) for k in bad.nonzero()[0])
        t = tol[i] if torch.is_tensor(tol) and tol.ndim else tol
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; first {i}: got {float(got[i])!r}, "
                             f"want {float(want[i])!r}, allowed {float(t)!r}")


def norm(x, r, gamma, eps):
    """(s, y) in 64 bits."""
    s = x.double() if r is None else x.double() + r.double()
    return s, s / torch.sqrt((s * s).mean(1, keepdim=True) + eps) * gamma.double()


def check_norm(out, dtype, x, r, gamma, eps, Y, S=None, scale=None, amax=None):
    x, gamma = x.cpu(), gamma.cpu()
    r = None if r is None else r.cpu()
    s, y = norm(x, r, gamma, eps)
    if S is not None:
        close(S, s, rounded(s, dtype, 2.0 ** -24 * s.abs()), "S")
    if out == "same":
        close(Y, y, rounded(y, dtype, F32 * y.abs()), "Y")
        return
    if out == "e4m3":
        v = y / scale.cpu().double()
        if amax is not None:
            close(amax, y.abs().max().reshape(1), F32 * y.abs().max(), "amax")
    else:
        top = y.abs().amax(1)
        want = torch.where(top > 0, top / 448, torch.ones_like(top))
        close(scale, want, F32 * want, "scale")
        v = y / want[:, None]
    close(Y, v.clamp(-448, 448), rounded(v, "e4m3", F32 * v.abs()), "Y")


def norm_bwd(dy, s, gamma, ds, eps):
    """(dx, dgamma, bound of dx before its rounding, sum of |terms| of dgamma)."""
    dy, s, g = dy.double(), s.double(), gamma.double()
    rho = 1 / torch.sqrt((s * s).mean(1, keepdim=True) + eps)
    a = dy * g
    dx = rho * a - s * rho ** 3 * (a * s).mean(1, keepdim=True)
    size = rho * a.abs() + s.abs() * rho ** 3 * (a * s).abs().mean(1, keepdim=True)
    if ds is not None:
        dx = dx + ds.double()
        size = size + ds.double().abs()
    t = dy * s * rho
    return dx, t.sum(0), size, t.abs().sum(0)


def check_norm_bwd(dtype, dy, s, gamma, ds, eps, dX, dgamma=None):
    dx, dg, size, dsize = norm_bwd(dy.cpu(), s.cpu(), gamma.cpu(), None if ds is None else ds.cpu(), eps)
    close(dX, dx, rounded(dx, dtype, F32 * size), "dX")
    if dgamma is not None:
        close(dgamma, dg, rounded(dg, dtype, F32 * dsize), "dgamma")


def act(name, z):
    name = name.replace("_aux", "").replace("_bias", "")
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "gelu":
        return z * torch.special.ndtr(z)
    if name == "tanh":
        return torch.tanh(z)
    return z                                       # none, bias


def act_slope(name, z):
    name = name.replace("_aux", "").replace("_bias", "")
    if name == "relu":
        return (z > 0).double()
    if name == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "tanh":
        return 1 / torch.cosh(z) ** 2
    return torch.ones_like(z)


# The slopes' own error before the rounding.  GELU: Abramowitz & Stegun 7.1.26 is within 1.5e-7 of
# erf (half of it on Phi), the hardware's reciprocal and exponential within 2^-22 of values below
# 1, and the exponent's rounding within 18 * 2^-24 of a term below 0.25: 1e-6 covers them.  tanh:
# tanhf is within 2 units of 2^-24, so 1 - tanh^2 within 2^-21.
SLOPE = {"gelu": 1e-6, "tanh": 2.0 ** -21}


def check_dact(epilogue, axis, dtype, dd, z, dZ, dbias, slope=None):
    dd = dd.cpu().double()
    s = act_slope(epilogue, z.cpu().double()) if slope is None else slope
    dz = dd * s
    off = dd.abs() * SLOPE.get(epilogue.split("_")[0], 0.0)
    if dZ is not None:
        close(dZ, dz, rounded(dz, dtype, off + 2.0 ** -24 * dz.abs()), "dZ")
    if dbias is not None:
        dim = 1 if axis == "row" else 0
        want = dz.sum(dim)
        close(dbias, want, rounded(want, dtype, off.sum(dim) + F32 * dz.abs().sum(dim)), "dbias")


def pack_mask(z):
    """The library's packed mask of z > 0 as int32 words, on z's device."""
    from activation_epilogue_tcgen05_b200 import workloads
    m = (z.cpu().double() > 0).to(torch.uint8).numpy()
    return torch.from_numpy(workloads.pack_mask(m).view("int32")).to(z.device)
