"""The layer norm, products of 8-bit integers and 8-bit checkpoints from their formulas, in 64 bits on the CPU, and the bounds
that the kernels' outputs are held to (block_ref's: half a step of the output's type for its one rounding, F32 = 2^-17 for
an fp32 sum and the few operations around it)."""
import torch

from block_ref import F32, TINY, U, act, close, rounded

E24 = 2.0 ** -24


# ------------------------------------------------------------------ layer norm
def layer_norm(x, r, gamma, beta, eps):
    """(s, y, what y may be off by before its rounding) in 64 bits.

    The mean is put right by the sum of the differences from it, so (s - mean) is off by F32 of the differences' mean magnitude and
    of itself.  Where s is a sum, it is rounded to fp32: e = 2^-24 max |s| moves a difference by 2 e at most and rho by 2 e rho of
    itself."""
    s = x.double() if r is None else x.double() + r.double()
    c = s - s.mean(1, keepdim=True)
    rho = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + eps)
    u, g = c * rho, gamma.double()
    b = torch.zeros_like(g) if beta is None else beta.double()
    y = u * g + b
    e = 0.0 if r is None else E24 * s.abs().amax(1, keepdim=True) * rho
    off = g.abs() * (F32 * (u.abs() + u.abs().mean(1, keepdim=True)) + e * (2 + 2 * u.abs())) + F32 * (y.abs() + b.abs())
    return s, y, off


def check_layer_norm(out, dtype, x, r, gamma, beta, eps, Y, S=None, scale=None, amax=None):
    cpu = lambda t: None if t is None else t.cpu()  # noqa: E731
    s, y, off = layer_norm(cpu(x), cpu(r), cpu(gamma), cpu(beta), eps)
    if S is not None:
        close(S, s, rounded(s, dtype, E24 * s.abs()), "S")
    check_out(out, dtype, y, off, Y, scale, amax)


def check_out(out, dtype, y, off, Y, scale=None, amax=None):
    """Y (and its scale) against the values y, known to within off."""
    if out == "same":
        close(Y, y, rounded(y, dtype, off), "Y")
    elif out == "e4m3":
        v, o = y / scale.cpu().double(), off / scale.cpu().double()
        if amax is not None:
            close(amax, y.abs().max().reshape(1), off.max() + F32 * y.abs().max(), "amax")
        close(Y, v.clamp(-448, 448), rounded(v, "e4m3", o + F32 * v.abs()), "Y")
    else:
        top, most = (448, None) if out == "e4m3_rows" else (127, 127)
        big = y.abs().amax(1)
        want = torch.where(big > 0, big / top, torch.ones_like(big))
        close(scale, want, off.amax(1) / top + F32 * want, "scale")
        v, o = y / want[:, None], off / want[:, None]
        o = o + v.abs() * (o.amax(1, keepdim=True) / top + F32)            # the scale's own error
        if most is None:
            close(Y, v.clamp(-448, 448), rounded(v, "e4m3", o), "Y")
        else:
            close(Y, v, 0.5 + o, "Y")
            got = Y.cpu().double().abs().amax(1)
            assert (got[big > 0] == 127).all() and (got[big == 0] == 0).all()


def layer_norm_bwd(dy, s, gamma, ds, eps):
    """(dx, dgamma, dbeta, and what each may be off by before its rounding).

    The mean is off by d = F32 mean |s|, u by d rho."""
    dy, s, g = dy.double(), s.double(), gamma.double()
    c = s - s.mean(1, keepdim=True)
    rho = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + eps)
    u, a = c * rho, dy * g
    mean = lambda t: t.mean(1, keepdim=True)  # noqa: E731
    dx = rho * (a - mean(a) - u * mean(a * u))
    du = F32 * mean(s.abs()) * rho
    off = F32 * rho * (a.abs() + mean(a.abs()) + u.abs() * mean((a * u).abs())) + rho * du * (mean((a * u).abs()) + (u.abs() + du) * mean(a.abs()))
    if ds is not None:
        dx = dx + ds.double()
        off = off + E24 * ds.double().abs() + E24 * dx.abs()
    return (dx, (dy * u).sum(0), dy.sum(0), off, F32 * (dy * u).abs().sum(0) + (du * dy.abs()).sum(0), F32 * dy.abs().sum(0))


def check_layer_norm_bwd(dtype, dy, s, gamma, ds, eps, dX, dgamma=None, dbeta=None):
    dx, dg, db, ox, og, ob = layer_norm_bwd(dy.cpu(), s.cpu(), gamma.cpu(), None if ds is None else ds.cpu(), eps)
    close(dX, dx, rounded(dx, dtype, ox), "dX")
    if dgamma is not None:
        close(dgamma, dg, rounded(dg, dtype, og), "dgamma")
    if dbeta is not None:
        close(dbeta, db, rounded(db, dtype, ob), "dbeta")


# ------------------------------------------------------------------ products of 8-bit integers
def act_off(name, x, off):
    """What act(x) may be off by: x's own error times the steepest slope (1.13), and the activation's own: erfc within 1.5e-7 (half
    of it on Phi) and the hardware's reciprocal and exponential for GELU, 2^-21 for tanh."""
    own = {"gelu": 3e-7 * x.abs(), "tanh": 2.0 ** -21 * x.abs().clamp(max=1.0)}.get(name.split("_")[0], 0.0)
    return 1.13 * off + own


def product_i8(a, b_kn, rows, cols, bias, axis, epilogue, residual):
    """(pre-activation, its bound, output, its bound before the rounding).  The integer sum is exact; it is rounded to fp32, and so
    is each product and sum after it."""
    acc = a.double() @ b_kn.double()
    lin = acc * rows.double()[:, None] * cols.double()
    x = lin if bias is None else lin + (bias.double()[:, None] if axis == "row" else bias.double())
    off = 4 * E24 * lin.abs() + E24 * x.abs()
    y = act(epilogue, x)
    oy = act_off(epilogue, x, off)
    if residual is not None:
        y = y + residual.double()
        oy = oy + E24 * y.abs()
    return x, off, y, oy


# ------------------------------------------------------------------ checkpoints
def checkpoint(z):
    """(codes, exponents, kept z) in 64 bits of a finite z."""
    m, n = z.shape
    g = -(-n // 32)
    p = torch.nn.functional.pad(z.double(), (0, 32 * g - n)).view(m, g, 32)
    top = p.abs().amax(2)
    e = torch.full((m, g), 7.0, dtype=torch.float64)
    for cand in range(254, 6, -1):          # the smallest that fits
        e = torch.where(top <= 127 * 2.0 ** (cand - 133), float(cand), e)
    step = torch.exp2(e - 133)[:, :, None]
    q = torch.round(p / step)
    return q.view(m, -1)[:, :n], e, (q * step).view(m, -1)[:, :n]


def kept(codes, exps):
    """The values that codes and exponents stand for."""
    n = codes.shape[1]
    step = torch.exp2(exps.double() - 133).repeat_interleave(32, dim=1)[:, :n]
    return codes.double() * step


def check_act(epilogue, dtype, z, H, own=None):
    """H = act(z) of values z that are known exactly."""
    z = z.cpu().double()
    y = act(epilogue, z)
    off = act_off(epilogue, z, 0.0) if own is None else own * z.abs()
    close(H, y, U[dtype] * (y.abs() + off) + TINY[dtype] + off, "H")


def layer_norm_bwd_close(dtype, dy, s, gamma, eps):
    """(dx, dgamma, dbeta, and what each may be off by before its rounding) from differences c = s - mean that keep their digits
    whatever the mean.

    A row's values are multiples of the smallest one's unit.  Where their magnitudes add up to at most 2^24 units their sum is exact in
    fp32 (rows beyond 8192 are added up as two, neither more than 5/8 of the row).  Otherwise a value passes at most 32 roundings,
    and the mean is off by D = 2^-19 mean |s|.  It is held in two numbers, the second one at most t = 2^-22 |mean| and off by 2^-22
    of itself.  c is off by E = D + F32 |u / rho|, an eighth of it allowed for what is smaller still, and 2^-22 t; mean c^2 by F32 of
    itself, by (D + t)^2 where t is left in it, so rho by r = 2 F32 + (D + t)^2 rho^2 of itself, its own roundings among it; mean a c by
    A = F32 (mean |a c| + t mean |a|) + mean |a| E."""
    dy, s, g = dy.double(), s.double(), gamma.double()
    mean = lambda v: v.mean(1, keepdim=True)  # noqa: E731
    unit = torch.where(s == 0, torch.inf, torch.exp2(torch.frexp(s)[1].double() - {"f16": 11, "bf16": 8}[dtype])).amin(1, keepdim=True)
    exact = s.abs().sum(1, keepdim=True) * (0.625 if s.shape[1] > 8192 else 1.0) <= 2.0 ** 24 * unit
    D = torch.where(exact, 0.0, 2.0 ** -19 * mean(s.abs()))
    c = s - mean(s)
    rho = 1 / torch.sqrt(mean(c * c) + eps)
    u, a = c * rho, dy * g
    ac = mean(a * c)
    dx = rho * (a - mean(a) - rho * rho * c * ac)
    t = 4 * E24 * mean(s).abs()
    E = 1.125 * (D + F32 * c.abs()) + 4 * E24 * t
    r = 2 * F32 + ((D + t) * rho) ** 2
    A = 1.125 * F32 * mean((a * c).abs()) + F32 * t * mean(a.abs()) + mean(a.abs() * E)
    most = (1 + r) ** 3
    off = rho * ((r + F32) * (a.abs() + mean(a.abs())) + most * rho * rho * (E * (ac.abs() + A) + c.abs() * A)
                 + (most - 1 + F32) * rho * rho * ((c.abs() + t) * ac.abs()))
    og = F32 * (dy * u).abs().sum(0) + (dy.abs() * (rho * (1 + r) * E + r * u.abs() + F32 * t * rho)).sum(0)
    return dx, (dy * u).sum(0), dy.sum(0), off, og, F32 * dy.abs().sum(0)
