"""The work of the operators around an MLP block: the norm before it, the product with a residual that ends it, and their gradients.

* ``norm``      s = x + r, y = s / rms(s) * gamma; y in 16 bits, or in e4m3 with a given scale or with one scale a row
* ``norm_bwd``  the gradients of ``norm`` with respect to x (and r) and gamma, the skip path's gradient added
* ``product``   D = act(alpha A.B + bias) + R on 16-bit operands, or on e4m3 operands with one scale a row of A
* ``act_bwd``   the gradients through the activation and the bias of ``product``

``own`` chooses between the plain torch form and the package's kernels.
"""
import math

import torch

own = False

T16 = {"f16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    def norm(name, m, d, dtype, residual, out):
        return {"name": name, "op": "norm", "m": m, "d": d, "dtype": dtype, "residual": residual, "out": out}

    def norm_bwd(name, m, d, dtype, skip):
        return {"name": name, "op": "norm_bwd", "m": m, "d": d, "dtype": dtype, "skip": skip}

    def product(name, m, n, k, dtype, epilogue, axis, layout, rows):
        return {"name": name, "op": "product", "m": m, "n": n, "k": k, "dtype": dtype, "epilogue": epilogue, "axis": axis, "layout": layout,
                "rows": rows}

    def act_bwd(name, m, n, dtype, epilogue, axis):
        return {"name": name, "op": "act_bwd", "m": m, "n": n, "dtype": dtype, "epilogue": epilogue, "axis": axis}

    return [
        # one sequence decoding: the norm between two blocks, where only latency counts
        norm("norm_token", 1, 4096, "bf16", True, "same"),
        # a prompt's rows on their way into an FP8 up-projection
        norm("norm_prompt_rows8", 8192, 4096, "bf16", True, "e4m3_rows"),
        # the norm of a long training batch of a wide model
        norm("norm_train_wide", 16384, 8192, "bf16", True, "same"),
        # short rows, an odd number of them (a norm per attention head), with a calibrated scale
        norm("norm_heads_tensor8", 65537, 128, "f16", False, "e4m3"),
        # a short ragged batch of a narrow model
        norm_bwd("norm_bwd_small_odd", 37, 1000, "f16", False),
        # a training batch, the skip connection's gradient joining
        norm_bwd("norm_bwd_train", 8192, 4096, "bf16", True),
        # the same for rows as wide as an MLP's intermediate
        norm_bwd("norm_bwd_wide", 4096, 14336, "f16", True),
        # sixteen sequences decoding: output projection back into the residual stream
        product("product_decode", 16, 4096, 4096, "f16", "bias", "col", "nk", False),
        # a prompt through the FP8 down-projection, the activations quantised by rows
        product("product_prompt_rows8", 8192, 4096, 14336, "e4m3", "bias", "col", "kn", True),
        # ragged in every direction, an activation before the residual
        product("product_odd_gelu", 777, 1032, 520, "bf16", "gelu_bias", "col", "kn", False),
        # a training batch through the GELU of the up-projection
        act_bwd("act_bwd_gelu_train", 8192, 14336, "bf16", "gelu_bias", "col"),
        # odd sizes through ReLU's sign mask, the bias along the rows
        act_bwd("act_bwd_relu_mask_odd", 1023, 4104, "f16", "relu_aux_bias", "row"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "product", "act_bwd"])
    dtype = rng.choice(["f16", "bf16"])
    if op == "norm":
        d = 16 * _log(rng, 4, 1024)
        return {"op": op, "m": min(_log(rng, 1, 65536), 2**27 // d), "d": d, "dtype": dtype, "residual": rng.random() < 0.7,
                "out": rng.choice(["same", "e4m3", "e4m3_rows"])}
    if op == "norm_bwd":
        d = 8 * _log(rng, 8, 2048)
        return {"op": op, "m": min(_log(rng, 1, 65536), 2**27 // d), "d": d, "dtype": dtype, "skip": rng.random() < 0.7}
    if op == "product":
        dtype = rng.choice(["f16", "bf16", "e4m3"])
        n, k = 16 * _log(rng, 8, 1024), 16 * _log(rng, 8, 1024)
        return {"op": op, "m": max(1, min(_log(rng, 1, 8192), 2**38 // (n * k))), "n": n, "k": k, "dtype": dtype,
                "epilogue": rng.choice(["none", "bias", "relu_bias", "gelu_bias", "tanh_bias"]), "axis": rng.choice(["row", "col"]),
                "layout": rng.choice(["kn", "nk"]), "rows": dtype == "e4m3" and rng.random() < 0.7}
    n = 8 * _log(rng, 16, 2048)
    return {"op": op, "m": min(_log(rng, 1, 16384), 2**27 // n), "n": n, "dtype": dtype,
            "epilogue": rng.choice(["bias", "relu_bias", "relu_aux_bias", "gelu_bias", "tanh_bias"]), "axis": rng.choice(["row", "col"])}


def work(case):
    if case["op"] == "norm":
        m, d = case["m"], case["d"]
        out = {"same": 2 * m * d, "e4m3": m * d + 8, "e4m3_rows": m * d + 4 * m}[case["out"]]
        return {"bytes": 2 * m * d + (4 * m * d if case["residual"] else 0) + 2 * d + out, "flops": 6 * m * d}
    if case["op"] == "norm_bwd":
        m, d = case["m"], case["d"]
        return {"bytes": (8 if case["skip"] else 6) * m * d + 4 * d, "flops": 12 * m * d}
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        e = 1 if case["dtype"] == "e4m3" else 2
        bias = 0 if case["epilogue"] == "none" else 2 * (m if case["axis"] == "row" else n)
        return {"bytes": e * k * (m + n) + 4 * m * n + bias + (4 * m if case["rows"] else 0), "flops": 2 * m * n * k}
    m, n, epilogue = case["m"], case["n"], case["epilogue"]
    side = {"bias": 0, "relu_aux_bias": m * n // 8}.get(epilogue, 2 * m * n)
    return {"bytes": 2 * m * n + side + (0 if epilogue == "bias" else 2 * m * n) + 2 * (m if case["axis"] == "row" else n), "flops": 10 * m * n}


# ------------------------------------------------------------------ inputs
def _stream(m, d, gen):
    """Rows of a residual stream: channels of unlike size, a few of them large."""
    size = torch.exp(0.5 * torch.randn(d, generator=gen, device="cuda"))
    size[:: max(1, d // 7)] *= 8.0
    return torch.randn(m, d, generator=gen, device="cuda") * size


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def empty(*shape, dtype):
        return torch.empty(shape, device="cuda", dtype=dtype)

    op, m, s = case["op"], case["m"], {"case": case}
    t = T16.get(case["dtype"], torch.bfloat16)
    if op == "norm":
        d, out = case["d"], case["out"]
        s["x"] = (0.5 * randn(m, d) if case["residual"] else _stream(m, d, gen)).to(t)
        s["gamma"] = (1 + 0.1 * randn(d)).to(t)
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
        s["dx"], s["dgamma"] = empty(m, d, dtype=t), empty(d, dtype=t)
    elif op == "product":
        n, k, dtype = case["n"], case["k"], case["dtype"]
        a, b = randn(m, k) * torch.exp(0.5 * randn(m, 1)), randn(*((k, n) if case["layout"] == "kn" else (n, k))) / math.sqrt(k)
        if dtype == "e4m3":
            top = a.abs().amax(dim=1, keepdim=True) if case["rows"] else a.abs().max()
            s["scale_a"], s["scale_b"] = (top / 448).reshape(-1), (b.abs().max() / 448).reshape(1)
            s["a"], s["b"] = (a * (448 / top)).clamp(-448, 448).to(E4M3), (b / s["scale_b"]).clamp(-448, 448).to(E4M3)
        else:
            s["a"], s["b"] = a.to(t), b.to(t)
        s["bias"] = None if case["epilogue"] == "none" else (0.1 * randn(m if case["axis"] == "row" else n)).to(t)
        s["residual"], s["out"] = randn(m, n).to(t), empty(m, n, dtype=t)
    else:
        n = case["n"]
        s["dd"], z = randn(m, n).to(t), randn(m, n).to(t)
        s["aux"] = s["z"] = None
        if case["epilogue"] == "relu_aux_bias":
            words = -(-n // 128) * 4
            bits = torch.zeros(m, words * 32, device="cuda", dtype=torch.int64)
            bits[:, :n] = z > 0
            bits = (bits.view(m, words, 32) << torch.arange(32, device="cuda")).sum(-1)
            s["aux"] = torch.where(bits >= 2**31, bits - 2**32, bits).to(torch.int32)
        elif case["epilogue"] != "bias":
            s["z"] = z
        s["dz"] = None if case["epilogue"] == "bias" else empty(m, n, dtype=t)
        s["dbias"] = empty(m if case["axis"] == "row" else n, dtype=t)
    if own:
        s["plan"] = _plan(case, s)
    return s


def _plan(case, s):
    """The handle that a program keeps for calls of these sizes."""
    from activation_epilogue_tcgen05_b200 import gemm_epi as g

    if case["op"] == "norm":
        return g.RmsNorm(case["m"], case["d"], case["dtype"], out=case["out"], eps=EPS)
    if case["op"] == "norm_bwd":
        return g.RmsNorm(case["m"], case["d"], case["dtype"], eps=EPS)
    if case["op"] == "act_bwd":
        return g.ActBackward(case["m"], case["n"], case["dtype"], case["epilogue"], case["axis"])
    plan = g.Plan(case["m"], case["n"], case["k"], case["dtype"], case["epilogue"], case["axis"], case["layout"])
    if case["dtype"] == "e4m3":
        plan.set_scales(s["scale_b"] if case["rows"] else s["scale_a"], s["scale_b"])     # with scales by row, that of A is not read
    return plan


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "norm_bwd": _own_norm_bwd, "product": _own_product, "act_bwd": _own_act_bwd}[op](state)
    return {"norm": _norm, "norm_bwd": _norm_bwd, "product": _product, "act_bwd": _act_bwd}[op](state["case"], state)


def _own_norm(s):
    s["plan"].run(s["x"], s["gamma"], s["y"], residual=s.get("residual"), S=s.get("sum"), scale=s.get("scale"), amax=s.get("amax"))
    return {"y": s["y"], "sum": s.get("sum"), "scale": s["scale"] if s["case"]["out"] == "e4m3_rows" else None, "amax": s.get("amax")}


def _own_norm_bwd(s):
    s["plan"].run_bwd(s["dy"], s["sum"], s["gamma"], s["dx"], dgamma=s["dgamma"], dS=s["ds"])
    return {"dx": s["dx"], "dgamma": s["dgamma"]}


def _own_product(s):
    s["plan"].run_ext(s["a"], s["b"], s["bias"], s["out"], residual=s["residual"], scale_rows=s["scale_a"] if s["case"]["rows"] else None)
    return {"out": s["out"]}


def _own_act_bwd(s):
    s["plan"].run(s["dd"], dZ=s["dz"], z=s["z"], aux=s["aux"], dbias=s["dbias"])
    return {"dz": s["dz"], "dbias": s["dbias"]}


def _norm(case, s):
    t = T16[case["dtype"]]
    h = s["x"].float()
    if case["residual"]:
        h = h + s["residual"].float()
    y = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS) * s["gamma"].float()
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
    r = torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS)
    a = dy * s["gamma"].float()
    dx = r * a - h * (r * r * r * (a * h).mean(dim=1, keepdim=True))
    if s["ds"] is not None:
        dx = dx + s["ds"].float()
    return {"dx": dx.to(t), "dgamma": (dy * h * r).sum(dim=0).to(t)}


def _product(case, s):
    a, b = s["a"].float(), s["b"].float()
    x = a @ (b if case["layout"] == "kn" else b.t())
    if case["dtype"] == "e4m3":
        x = x * (s["scale_a"].reshape(-1, 1) * s["scale_b"])
    if s["bias"] is not None:
        x = x + (s["bias"].float()[:, None] if case["axis"] == "row" else s["bias"].float())
    e = case["epilogue"]
    if e == "relu_bias":
        x = x.clamp_min(0)
    elif e == "gelu_bias":
        x = 0.5 * x * (1 + torch.erf(x * math.sqrt(0.5)))
    elif e == "tanh_bias":
        x = torch.tanh(x)
    return {"out": (x + s["residual"].float()).to(s["residual"].dtype)}


def _act_bwd(case, s):
    t, e = T16[case["dtype"]], case["epilogue"]
    dz, z = s["dd"].float(), None if s["z"] is None else s["z"].float()
    if e == "relu_bias":
        dz = dz * (z > 0)
    elif e == "relu_aux_bias":
        bits = (s["aux"][:, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
        dz = dz * bits.reshape(case["m"], -1)[:, : case["n"]]
    elif e == "gelu_bias":
        dz = dz * (0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi)))
    elif e == "tanh_bias":
        y = torch.tanh(z)
        dz = dz * (1 - y * y)
    return {"dz": None if e == "bias" else dz.to(t), "dbias": dz.sum(dim=1 if case["axis"] == "row" else 0).to(t)}


# ------------------------------------------------------------------ from the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    wide = {k: v.to(torch.float64) for k, v in s.items() if isinstance(v, torch.Tensor) and v.dtype != torch.int32 and k not in ("y", "out", "dx", "dz")}
    if case["op"] == "norm":
        h = wide["x"] + wide["residual"] if case["residual"] else wide["x"]
        y = h.div_(torch.sqrt(torch.linalg.vecdot(h, h) / case["d"] + EPS)[:, None]) if not case["residual"] else \
            h / torch.sqrt(torch.linalg.vecdot(h, h) / case["d"] + EPS)[:, None]
        y = y * wide["gamma"]
        top = torch.maximum(y.amax(dim=1), -y.amin(dim=1))
        by_row, given = case["out"] == "e4m3_rows", case["out"] == "e4m3"
        scale = torch.where(top == 0, 1.0, top / 448.0)
        return {"y": torch.clamp(y / scale[:, None], -448, 448) if by_row else torch.clamp(y / wide["scale"], -448, 448) if given else y,
                "sum": h if case["residual"] else None, "scale": scale if by_row else None, "amax": top.max().reshape(1) if given else None}
    if case["op"] == "norm_bwd":
        h, dy, g = wide["sum"], wide["dy"], wide["gamma"]
        rms = torch.sqrt(torch.linalg.vecdot(h, h) / case["d"] + EPS)[:, None]
        unit = h / rms                      # y = unit * gamma; d unit / d h = (1 - unit unit^T / d) / rms
        dunit = dy * g
        dx = (dunit - unit * (torch.linalg.vecdot(dunit, unit) / case["d"])[:, None]) / rms
        return {"dx": dx + wide["ds"] if case["skip"] else dx, "dgamma": torch.einsum("ij,ij->j", dy, unit)}
    if case["op"] == "product":
        x = torch.einsum("ik,kj->ij" if case["layout"] == "kn" else "ik,jk->ij", wide["a"], wide["b"])
        if case["dtype"] == "e4m3":
            x *= wide["scale_b"]
            x *= wide["scale_a"][:, None] if case["rows"] else wide["scale_a"]
        if "bias" in wide:
            x += wide["bias"].unsqueeze(1 if case["axis"] == "row" else 0)
        act = {"relu_bias": lambda v: torch.where(v > 0, v, 0.0), "gelu_bias": lambda v: v * torch.special.ndtr(v), "tanh_bias": torch.tanh}
        return {"out": act.get(case["epilogue"], lambda v: v)(x) + wide["residual"]}
    e = case["epilogue"]
    if e == "bias":
        slope = 1.0
    elif e == "relu_aux_bias":
        byte = s["aux"].contiguous().view(torch.uint8)      # little-endian words: bit b of byte k is column 8 k + b
        slope = torch.stack([(byte >> b) & 1 for b in range(8)], dim=-1).reshape(case["m"], -1)[:, : case["n"]].to(torch.float64)
    elif e == "relu_bias":
        slope = torch.heaviside(wide["z"], torch.zeros((), dtype=torch.float64, device="cuda"))
    elif e == "gelu_bias":
        slope = torch.special.ndtr(wide["z"]) + wide["z"] * torch.exp(-wide["z"].square() / 2) / math.sqrt(2 * math.pi)
    else:
        slope = torch.cosh(wide["z"]).pow(-2)
    dz = wide["dd"] * slope
    return {"dz": None if e == "bias" else dz, "dbias": torch.einsum("ij->i" if case["axis"] == "row" else "ij->j", dz)}
