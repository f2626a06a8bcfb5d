"""The work of a transformer's MLP around a layer norm, with 8-bit integers: in the products that serve it, and in what training keeps of it.

* ``norm``        s = x + r, y = (s - mean) / sd * gamma + beta; y in 16 bits, or in e4m3 with a given scale or one scale a row
* ``norm_bwd``    the gradients of ``norm`` with respect to x (and r), gamma and beta, the skip path's gradient added
* ``product_i8``  D = act(s_i t_j (A.B)_ij + bias) + R on 8-bit integers, one scale a token (row of A) and one a channel (column of B)
* ``linear_i8``   the same from 16-bit rows, quantised on the way: as they are, or after ``norm``
* ``checkpoint``  a pre-activation z on its way through the activation, kept in 8 bits with one power of two for 32 columns, and what it restores
* ``act_bwd8``    the gradients through the activation and the bias from that checkpoint, the activation's value recomputed beside them

``own`` chooses between the plain torch form and the package's kernels.
"""
import math

import torch

own = False

T16 = {"f16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn
EPS = 1e-5
GROUP = 32          # columns of a checkpoint that share a power of two


# ------------------------------------------------------------------ cases
def listed():
    def norm(name, m, d, dtype, residual, out):
        return {"name": name, "op": "norm", "m": m, "d": d, "dtype": dtype, "residual": residual, "out": out}

    def norm_bwd(name, m, d, dtype, skip):
        return {"name": name, "op": "norm_bwd", "m": m, "d": d, "dtype": dtype, "skip": skip}

    def product(name, m, n, k, epilogue, axis, layout, residual):
        return {"name": name, "op": "product_i8", "m": m, "n": n, "k": k, "epilogue": epilogue, "axis": axis, "layout": layout,
                "residual": residual}

    def linear(name, m, n, k, epilogue, layout, norm):
        return {"name": name, "op": "linear_i8", "m": m, "n": n, "k": k, "epilogue": epilogue, "axis": "col", "layout": layout, "norm": norm}

    def checkpoint(name, m, n, dtype, epilogue, act):
        return {"name": name, "op": "checkpoint", "m": m, "n": n, "dtype": dtype, "epilogue": epilogue, "act": act}

    def act_bwd(name, m, n, dtype, epilogue, axis, recompute):
        return {"name": name, "op": "act_bwd8", "m": m, "n": n, "dtype": dtype, "epilogue": epilogue, "axis": axis, "recompute": recompute}

    return [
        # one sequence decoding: the norm between two blocks, where only latency counts
        norm("norm_token", 1, 4096, "bf16", True, "same"),
        # a prompt's rows on their way into an FP8 up-projection
        norm("norm_prompt_rows8", 8192, 4096, "bf16", True, "e4m3_rows"),
        # a short ragged batch of a narrow model
        norm_bwd("norm_bwd_small_odd", 37, 1000, "f16", False),
        # a training batch, the skip connection's gradient joining
        norm_bwd("norm_bwd_train", 8192, 4096, "bf16", True),
        # sixteen sequences decoding: output projection back into the residual stream
        product("product_decode", 16, 4096, 4096, "bias", "col", "nk", True),
        # a prompt through the down-projection, back into the residual stream
        product("product_prompt", 8192, 4096, 14336, "bias", "col", "kn", True),
        # ragged in every direction, tokens quantised as they come
        linear("linear_odd_gelu", 777, 1040, 528, "gelu_bias", "nk", False),
        # a prompt from the residual stream through norm and up-projection
        linear("linear_prompt_norm", 8192, 14336, 4096, "gelu_bias", "nk", True),
        # a small ragged batch kept and restored, the activation taken again on the way back
        checkpoint("checkpoint_odd", 1023, 4104, "f16", "tanh_bias", True),
        # a training batch of the up-projection kept through the forward pass and restored as it was
        checkpoint("checkpoint_train", 8192, 14336, "bf16", "gelu_bias", False),
        # odd sizes, the bias along the rows
        act_bwd("act_bwd_odd", 1023, 4104, "f16", "gelu_bias", "row", False),
        # a training batch through the GELU, whose value the weight's gradient needs again
        act_bwd("act_bwd_train", 8192, 14336, "bf16", "gelu_bias", "col", True),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "product_i8", "linear_i8", "checkpoint", "act_bwd8"])
    dtype = rng.choice(["f16", "bf16"])
    if op == "norm":
        d = 16 * _log(rng, 4, 1024)
        return {"op": op, "m": min(_log(rng, 1, 65536), 2**25 // d), "d": d, "dtype": dtype, "residual": rng.random() < 0.7,
                "out": rng.choice(["same", "e4m3", "e4m3_rows"])}
    if op == "norm_bwd":
        d = 8 * _log(rng, 8, 2048)
        return {"op": op, "m": min(_log(rng, 1, 65536), 2**25 // d), "d": d, "dtype": dtype, "skip": rng.random() < 0.7}
    if op in ("product_i8", "linear_i8"):
        n, k = 16 * _log(rng, 8, 1024), 16 * _log(rng, 8, 1024)
        case = {"op": op, "m": max(1, min(_log(rng, 1, 8192), 2**38 // (n * k))), "n": n, "k": k,
                "epilogue": rng.choice(["none", "bias", "relu_bias", "gelu_bias", "tanh_bias"]),
                "axis": rng.choice(["row", "col"]), "layout": rng.choice(["kn", "nk"])}
        return {**case, "residual": rng.random() < 0.5} if op == "product_i8" else {**case, "norm": rng.random() < 0.5}
    n = 8 * _log(rng, 16, 2048)
    case = {"op": op, "m": min(_log(rng, 1, 16384), 2**26 // n), "n": n, "dtype": dtype,
            "epilogue": rng.choice(["relu_bias", "gelu_bias", "tanh_bias"])}
    if op == "checkpoint":
        return {**case, "act": rng.random() < 0.5}
    return {**case, "axis": rng.choice(["row", "col"]), "recompute": rng.random() < 0.5}


def work(case):
    op, m = case["op"], case["m"]
    if op == "norm":
        d = case["d"]
        out = {"same": 2 * m * d, "e4m3": m * d + 8, "e4m3_rows": m * d + 4 * m}[case["out"]]
        return {"bytes": 2 * m * d + (4 * m * d if case["residual"] else 0) + 4 * d + out, "flops": 9 * m * d}
    if op == "norm_bwd":
        d = case["d"]
        return {"bytes": (8 if case["skip"] else 6) * m * d + 6 * d, "flops": 18 * m * d}
    if op in ("product_i8", "linear_i8"):
        n, k = case["n"], case["k"]
        bias = 0 if case["epilogue"] == "none" else 2 * (m if case["axis"] == "row" else n)
        if op == "product_i8":      # codes and scales of both operands, the residual, the output
            return {"bytes": k * (m + n) + 4 * (m + n) + bias + (4 if case["residual"] else 2) * m * n, "flops": 2 * m * n * k}
        # the 16-bit rows (and what the norm needs) in place of their codes
        return {"bytes": 2 * k * m + k * n + 4 * n + bias + 2 * m * n + (4 * k if case["norm"] else 0), "flops": 2 * m * n * k}
    n = case["n"]
    held = m * n + m * -(-n // GROUP)
    if op == "checkpoint":          # z in, the activation and the codes out; the codes in, what they stand for out
        return {"bytes": 4 * m * n + held + held + 2 * m * n, "flops": 16 * m * n}
    return {"bytes": 2 * m * n + held + (4 if case["recompute"] else 2) * m * n + 2 * (m if case["axis"] == "row" else n), "flops": 20 * m * n}


# ------------------------------------------------------------------ inputs
def _stream(m, d, gen):
    """Rows of a residual stream: channels of unlike size and mean, a few of them large."""
    size = torch.exp(0.5 * torch.randn(d, generator=gen, device="cuda"))
    size[:: max(1, d // 7)] *= 8.0
    return (torch.randn(m, d, generator=gen, device="cuda") + 0.5 * torch.randn(d, generator=gen, device="cuda")) * size


def _keep(z):
    """(codes, exponents) of a checkpoint: the smallest power of two in which every value of a group is at most 127, from 2^-126 on."""
    m, n = z.shape
    groups = torch.nn.functional.pad(z.float(), (0, -n % GROUP)).view(m, -1, GROUP)
    exps = ((groups.abs().amax(dim=2).view(torch.int32) + 0x1FFFF) >> 23).clamp(min=7)
    codes = torch.round(torch.ldexp(groups, (133 - exps)[:, :, None])).to(torch.int8)
    return codes.view(m, -1)[:, :n].contiguous(), exps.to(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def empty(*shape, dtype):
        return torch.empty(shape, device="cuda", dtype=dtype)

    op, m, s = case["op"], case["m"], {"case": case}
    t = T16[case.get("dtype", "bf16")]
    if op == "norm":
        d, out = case["d"], case["out"]
        s["x"] = (0.5 * randn(m, d) if case["residual"] else _stream(m, d, gen)).to(t)
        s["gamma"], s["beta"] = (1 + 0.1 * randn(d)).to(t), (0.1 * randn(d)).to(t)
        s["y"] = empty(m, d, dtype=t if out == "same" else E4M3)
        if case["residual"]:
            s["residual"] = _stream(m, d, gen).to(t)
            s["sum"] = empty(m, d, dtype=t)
        if out == "e4m3":       # a scale from calibration: a little less than the largest value, which then saturates
            s["scale"] = torch.full((1,), 4.5 / 448, device="cuda")
            s["amax"] = empty(1, dtype=torch.float32)
        elif out == "e4m3_rows":
            s["scale"] = empty(m, dtype=torch.float32)
    elif op == "norm_bwd":
        d = case["d"]
        s["dy"], s["sum"], s["gamma"] = randn(m, d).to(t), _stream(m, d, gen).to(t), (1 + 0.1 * randn(d)).to(t)
        s["ds"] = randn(m, d).to(t) if case["skip"] else None
        s["dx"], s["dgamma"], s["dbeta"] = empty(m, d, dtype=t), empty(d, dtype=t), empty(d, dtype=t)
    elif op in ("product_i8", "linear_i8"):
        n, k = case["n"], case["k"]
        w = randn(n, k) * torch.exp(0.3 * randn(n, 1)) / math.sqrt(k)       # channels of unlike size
        top = w.abs().amax(dim=1, keepdim=True)
        s["scale_cols"] = (top / 127).reshape(-1)
        w = torch.round(w * (127 / top)).to(torch.int8)
        s["b"] = w.t().contiguous() if case["layout"] == "kn" else w
        if op == "product_i8":
            a = randn(m, k) * torch.exp(0.5 * randn(m, 1))
            top = a.abs().amax(dim=1, keepdim=True)
            s["a"], s["scale_rows"] = torch.round(a * (127 / top)).to(torch.int8), (top / 127).reshape(-1)
            s["residual"] = randn(m, n).to(t) if case["residual"] else None
        else:
            s["x"] = (_stream(m, k, gen) if case["norm"] else randn(m, k) * torch.exp(0.5 * randn(m, 1))).to(t)
            if case["norm"]:
                s["gamma"], s["beta"] = (1 + 0.1 * randn(k)).to(t), (0.1 * randn(k)).to(t)
            s["a"], s["scale_rows"] = empty(m, k, dtype=torch.int8), empty(m, dtype=torch.float32)
        s["bias"] = None if case["epilogue"] == "none" else (0.1 * randn(m if case["axis"] == "row" else n)).to(t)
        s["out"] = empty(m, n, dtype=t)
    else:
        n = case["n"]
        z = randn(m, n).to(t)
        if op == "checkpoint":
            s["z"], s["h"], s["restored"] = z, empty(m, n, dtype=t), empty(m, n, dtype=t)
            s["codes"], s["exps"] = empty(m, n, dtype=torch.int8), empty(m, -(-n // GROUP), dtype=torch.uint8)
        else:
            s["dd"] = randn(m, n).to(t)
            s["codes"], s["exps"] = _keep(z)
            s["dz"], s["h"] = empty(m, n, dtype=t), empty(m, n, dtype=t) if case["recompute"] else None
            s["dbias"] = empty(m if case["axis"] == "row" else n, dtype=t)
    if own:
        _plans(case, s)
    return s


def _plans(case, s):
    """The handles that a program keeps for calls of these sizes."""
    from activation_epilogue_tcgen05_b200 import gemm_epi as g

    op, m = case["op"], case["m"]
    if op == "norm":
        s["plan"] = g.LayerNorm(m, case["d"], case["dtype"], out=case["out"], eps=EPS)
    elif op == "norm_bwd":
        s["plan"] = g.LayerNorm(m, case["d"], case["dtype"], eps=EPS)
    elif op == "checkpoint":
        s["plan"] = g.ActCheckpoint(m, case["n"], case["dtype"], case["epilogue"])
    elif op == "act_bwd8":
        s["plan"] = g.ActBackward(m, case["n"], case["dtype"], case["epilogue"], case["axis"])
    else:
        s["plan"] = g.Plan(m, case["n"], case["k"], "i8", case["epilogue"], case["axis"], case["layout"])
        if op == "linear_i8":
            s["first"] = g.LayerNorm(m, case["k"], out="i8_rows", eps=EPS) if case["norm"] else g.QuantRows(m, case["k"], out="i8_rows")


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "norm_bwd": _own_norm_bwd, "product_i8": _own_product, "linear_i8": _own_linear,
                "checkpoint": _own_checkpoint, "act_bwd8": _own_act_bwd}[op](state)
    return {"norm": _norm, "norm_bwd": _norm_bwd, "product_i8": _product, "linear_i8": _linear,
            "checkpoint": _checkpoint, "act_bwd8": _act_bwd}[op](state["case"], state)


def _own_norm(s):
    s["plan"].run(s["x"], s["gamma"], s["y"], beta=s["beta"], residual=s.get("residual"), S=s.get("sum"), scale=s.get("scale"), amax=s.get("amax"))
    return {"y": s["y"], "sum": s.get("sum"), "scale": s["scale"] if s["case"]["out"] == "e4m3_rows" else None, "amax": s.get("amax")}


def _own_norm_bwd(s):
    s["plan"].run_bwd(s["dy"], s["sum"], s["gamma"], s["dx"], dgamma=s["dgamma"], dbeta=s["dbeta"], dS=s["ds"])
    return {"dx": s["dx"], "dgamma": s["dgamma"], "dbeta": s["dbeta"]}


def _own_product(s):
    s["plan"].run_i8(s["a"], s["b"], s["bias"], s["out"], s["scale_rows"], s["scale_cols"], residual=s["residual"])
    return {"out": s["out"]}


def _own_linear(s):
    if s["case"]["norm"]:
        s["first"].run(s["x"], s["gamma"], s["a"], beta=s["beta"], scale=s["scale_rows"])
    else:
        s["first"].run(s["x"], s["a"], s["scale_rows"])
    s["plan"].run_i8(s["a"], s["b"], s["bias"], s["out"], s["scale_rows"], s["scale_cols"])
    return {"out": s["out"]}


def _own_checkpoint(s):
    s["plan"].save(s["z"], s["codes"], s["exps"], H=s["h"])
    s["plan"].load(s["codes"], s["exps"], s["restored"], act=s["case"]["act"])
    return {"h": s["h"], "restored": s["restored"]}


def _own_act_bwd(s):
    s["plan"].run_ckpt(s["dd"], s["codes"], s["exps"], s["dz"], H=s["h"], dbias=s["dbias"])
    return {"dz": s["dz"], "h": s["h"], "dbias": s["dbias"]}


def _layer_norm(h, gamma, beta):
    h = h - h.mean(dim=1, keepdim=True)
    return h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS) * gamma.float() + beta.float()


def _norm(case, s):
    t = T16[case["dtype"]]
    h = s["x"].float()
    if case["residual"]:
        h = h + s["residual"].float()
    y = _layer_norm(h, s["gamma"], s["beta"])
    total, scale, amax = h.to(t) if case["residual"] else None, None, None
    if case["out"] == "same":
        y = y.to(t)
    elif case["out"] == "e4m3":
        amax = y.abs().max().reshape(1)
        y = (y / s["scale"]).clamp(-448, 448).to(E4M3)
    else:
        top = y.abs().amax(dim=1)
        scale = torch.where(top > 0, top / 448, torch.ones_like(top))
        y = (y / scale[:, None]).clamp(-448, 448).to(E4M3)
    return {"y": y, "sum": total, "scale": scale, "amax": amax}


def _norm_bwd(case, s):
    t = T16[case["dtype"]]
    h, dy = s["sum"].float(), s["dy"].float()
    h = h - h.mean(dim=1, keepdim=True)
    r = torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS)
    unit, a = h * r, dy * s["gamma"].float()
    dx = r * (a - a.mean(dim=1, keepdim=True) - unit * (a * unit).mean(dim=1, keepdim=True))
    if s["ds"] is not None:
        dx = dx + s["ds"].float()
    return {"dx": dx.to(t), "dgamma": (dy * unit).sum(dim=0).to(t), "dbeta": dy.sum(dim=0).to(t)}


def _act(epilogue, x):
    if epilogue == "relu_bias":
        return x.clamp_min(0)
    if epilogue == "gelu_bias":
        return 0.5 * x * torch.erfc(x * -math.sqrt(0.5))
    return torch.tanh(x) if epilogue == "tanh_bias" else x


def _scaled(case, s, a, scale_rows):
    """The product of codes, its scales, bias and activation, in fp32."""
    x = a.float() @ (s["b"].float() if case["layout"] == "kn" else s["b"].float().t())
    x = x * scale_rows[:, None] * s["scale_cols"]
    if s["bias"] is not None:
        x = x + (s["bias"].float()[:, None] if case["axis"] == "row" else s["bias"].float())
    return _act(case["epilogue"], x)


def _product(case, s):
    x = _scaled(case, s, s["a"], s["scale_rows"])
    if s["residual"] is not None:
        x = x + s["residual"].float()
    return {"out": x.to(torch.bfloat16)}


def _linear(case, s):
    y = s["x"].float()
    if case["norm"]:
        y = _layer_norm(y, s["gamma"], s["beta"])
    top = y.abs().amax(dim=1)
    top = torch.where(top > 0, top, torch.full_like(top, 127.0))
    codes = torch.round(y * (127 / top)[:, None])
    return {"out": _scaled(case, s, codes, top / 127).to(torch.bfloat16)}


def _restore(codes, exps):
    steps = torch.ldexp(torch.ones((), device="cuda"), exps.to(torch.int32) - 133)
    return codes.float() * steps.repeat_interleave(GROUP, dim=1)[:, : codes.shape[1]]


def _checkpoint(case, s):
    t = T16[case["dtype"]]
    h = _act(case["epilogue"], s["z"].float()).to(t)
    z = _restore(*_keep(s["z"]))
    return {"h": h, "restored": (_act(case["epilogue"], z) if case["act"] else z).to(t)}


def _act_bwd(case, s):
    t, e = T16[case["dtype"]], case["epilogue"]
    dz, z = s["dd"].float(), _restore(s["codes"], s["exps"])
    if e == "relu_bias":
        dz = dz * (z > 0)
    elif e == "gelu_bias":
        dz = dz * (0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi)))
    else:
        y = torch.tanh(z)
        dz = dz * (1 - y * y)
    return {"dz": dz.to(t), "h": _act(e, z).to(t) if case["recompute"] else None,
            "dbias": dz.sum(dim=1 if case["axis"] == "row" else 0).to(t)}


# ------------------------------------------------------------------ from the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    wide = {k: v.to(torch.float64) for k, v in s.items() if isinstance(v, torch.Tensor) and k not in ("y", "out", "dx", "dz", "h", "restored", "z", "dd")}
    op = case["op"]

    def unit_of(h):
        c = h - h.sum(dim=1, keepdim=True) / h.shape[1]
        sd = torch.sqrt(torch.linalg.vecdot(c, c) / h.shape[1] + EPS)[:, None]
        return c / sd, sd

    if op == "norm":
        h = wide["x"] + wide["residual"] if case["residual"] else wide["x"]
        y = torch.addcmul(wide["beta"], unit_of(h)[0], wide["gamma"])
        top = torch.maximum(y.amax(dim=1), -y.amin(dim=1))
        by_row, given = case["out"] == "e4m3_rows", case["out"] == "e4m3"
        scale = torch.where(top == 0, 1.0, top / 448.0)
        return {"y": torch.clamp(y / scale[:, None], -448, 448) if by_row else torch.clamp(y / wide["scale"], -448, 448) if given else y,
                "sum": h if case["residual"] else None, "scale": scale if by_row else None, "amax": top.max().reshape(1) if given else None}
    if op == "norm_bwd":
        unit, sd = unit_of(wide["sum"])
        dy, d = wide["dy"], case["d"]
        dunit = dy * wide["gamma"]          # d unit / d h = (1 - 1 1^T / d - unit unit^T / d) / sd
        dx = (dunit - dunit.sum(dim=1, keepdim=True) / d - unit * (torch.linalg.vecdot(dunit, unit) / d)[:, None]) / sd
        return {"dx": dx + wide["ds"] if case["skip"] else dx, "dgamma": torch.einsum("ij,ij->j", dy, unit), "dbeta": torch.einsum("ij->j", dy)}
    act = {"relu_bias": lambda v: torch.where(v > 0, v, 0.0), "gelu_bias": lambda v: v * torch.special.ndtr(v), "tanh_bias": torch.tanh}
    act = act.get(case["epilogue"], lambda v: v)
    if op in ("product_i8", "linear_i8"):
        if op == "product_i8":
            a, rows = wide["a"], wide["scale_rows"]
        else:
            y = torch.addcmul(wide["beta"], unit_of(wide["x"])[0], wide["gamma"]) if case["norm"] else wide["x"]
            top = torch.maximum(y.amax(dim=1), -y.amin(dim=1))
            rows = torch.where(top == 0, 1.0, top / 127.0)
            a = torch.round(y / rows[:, None])
        x = torch.einsum("ik,kj->ij" if case["layout"] == "kn" else "ik,jk->ij", a, wide["b"])
        x = torch.einsum("ij,i,j->ij", x, rows, wide["scale_cols"])
        if s["bias"] is not None:
            x += wide["bias"].unsqueeze(1 if case["axis"] == "row" else 0)
        x = act(x)
        return {"out": x + wide["residual"] if case.get("residual") else x}
    m, n = case["m"], case["n"]
    if op == "checkpoint":
        z, restored = s["z"].to(torch.float64), torch.empty(m, n, device="cuda", dtype=torch.float64)
        for j in range(0, n, GROUP):
            part = z[:, j : j + GROUP]
            frac, power = torch.frexp(part.abs().amax(dim=1, keepdim=True))      # amax = 2 frac * 2^(power - 1)
            step = torch.exp2((power - 7 + (2 * frac > 127 / 64).to(power.dtype)).clamp(min=-126).to(torch.float64))
            restored[:, j : j + GROUP] = torch.round(part / step) * step
        return {"h": act(z), "restored": act(restored) if case["act"] else restored}
    z = wide["codes"] * torch.exp2(wide["exps"] - 133)[:, torch.arange(n, device="cuda") // GROUP]
    if case["epilogue"] == "relu_bias":
        slope = torch.heaviside(z, torch.zeros((), dtype=torch.float64, device="cuda"))
    elif case["epilogue"] == "gelu_bias":
        slope = torch.special.ndtr(z) + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)
    else:
        slope = torch.cosh(z).pow(-2)
    dz = s["dd"].to(torch.float64) * slope
    return {"dz": dz, "h": act(z) if case["recompute"] else None, "dbias": torch.einsum("ij->i" if case["axis"] == "row" else "ij->j", dz)}
