"""ctypes binding of the C ABI in ``include/gemm_epi.h`` (argument marshalling only).

The functions keep the C names and signatures; every step of the computation
runs in the CUDA library.  ``Plan`` is a small convenience wrapper that takes
torch tensors (device memory, the current stream) and passes their raw
pointers through the same entry points.

If ``libgemm_epi.so`` has not been built, loading raises ``RuntimeError``:
there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import math
import os
import sys
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libgemm_epi.so")

# enums (include/gemm_epi.h)
F16, BF16, E4M3, I8 = 0, 1, 2, 4
I8_MAX_K = 131071
NONE, BIAS, RELU_BIAS, RELU_AUX_BIAS, GELU_BIAS = 0, 1, 2, 3, 4
TANH_BIAS, RELU, RELU_AUX, GELU, TANH = 5, 6, 7, 8, 9
DRELU, DRELU_BGRAD = 10, 11
BIAS_ROW, BIAS_COL = 0, 1
B_KN, B_NK = 0, 1
A_KM = 2          # layout flag: A stored (k, m)
KERNEL_AUTO, KERNEL_TC1, KERNEL_TC2, KERNEL_SPLITK = 0, 1, 2, 3
OK, ERR_ARG, ERR_ALIGN, ERR_NULL, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT, ERR_NO_DEVICE = \
    0, -1, -2, -3, -4, -5, -6, -7

DTYPE = {"f16": F16, "bf16": BF16, "e4m3": E4M3, "i8": I8}
EPILOGUE = {"none": NONE, "bias": BIAS, "relu_bias": RELU_BIAS, "relu_aux_bias": RELU_AUX_BIAS,
            "gelu_bias": GELU_BIAS, "tanh_bias": TANH_BIAS, "relu": RELU, "relu_aux": RELU_AUX,
            "gelu": GELU, "tanh": TANH, "drelu": DRELU, "drelu_bgrad": DRELU_BGRAD}
HAS_BIAS = {"bias", "relu_bias", "relu_aux_bias", "gelu_bias", "tanh_bias"}
HAS_AUX = {"relu_aux_bias", "relu_aux"}
BACKWARD = {"drelu", "drelu_bgrad"}
AXIS = {"row": BIAS_ROW, "col": BIAS_COL}
LAYOUT = {"kn": B_KN, "nk": B_NK}
KERNEL = {"auto": KERNEL_AUTO, "tc1": KERNEL_TC1, "tc2": KERNEL_TC2, "splitk": KERNEL_SPLITK}
STREAM_K = {"auto": 0, "off": 1, "on": 2}
NORM_SAME, NORM_E4M3, NORM_E4M3_ROWS, NORM_I8_ROWS = 0, 1, 2, 4
NORM_OUT = {"same": NORM_SAME, "e4m3": NORM_E4M3, "e4m3_rows": NORM_E4M3_ROWS, "i8_rows": NORM_I8_ROWS}
CKPT_GROUP = 32   # columns of a checkpoint that share an exponent

# every symbol include/gemm_epi.h declares
EXPORTS = ("gemm_epi_plan", "gemm_epi_plan_ex", "gemm_epi_plan_opts", "gemm_epi_set_scales",
           "gemm_epi_run", "gemm_epi_unfused_run", "gemm_epi_check", "gemm_epi_plan_query",
           "gemm_epi_free", "gemm_epi_status_string", "gemm_epi_aux_pitch_bytes",
           "gemm_epi_version", "gemm_epi_run_noalloc", "gemm_epi_run_bwd", "gemm_epi_unfused_run_bwd",
           "gemm_epi_set_out_scale", "gemm_epi_mlp_plan", "gemm_epi_mlp_set_scales", "gemm_epi_mlp_run",
           "gemm_epi_mlp_check", "gemm_epi_mlp_query", "gemm_epi_mlp_free", "gemm_epi_mlp_unfused_run",
           "gemm_epi_plan_preview", "gemm_epi_rmsnorm", "gemm_epi_rmsnorm_workspace_bytes",
           "gemm_epi_rmsnorm_bwd", "gemm_epi_dact_workspace_bytes", "gemm_epi_dact", "gemm_epi_run_ext",
           "gemm_epi_mlp_run_prenorm", "gemm_epi_run_scaled", "gemm_epi_layernorm", "gemm_epi_layernorm_workspace_bytes",
           "gemm_epi_layernorm_bwd", "gemm_epi_quant_rows", "gemm_epi_ckpt_groups", "gemm_epi_ckpt_save", "gemm_epi_ckpt_load",
           "gemm_epi_dact_ckpt")


class Options(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int32), ("block_n", ctypes.c_int32),
                ("split_k", ctypes.c_int32), ("max_ctas", ctypes.c_int32),
                ("inject_stall", ctypes.c_int32), ("stream_k", ctypes.c_int32),
                ("out_e4m3", ctypes.c_int32)]


class PlanInfo(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int32) for f in
                ("kernel", "block_m", "block_n", "block_k", "stages", "split_k", "grid", "cluster",
                 "threads", "smem_bytes", "tiles", "sk_tiles", "sk_split", "group_m", "group_n")]

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


class GemmEpiError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


_lib = None
_lock = threading.Lock()


def lib():
    """Load libgemm_epi.so (raises RuntimeError when it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with "
                    "`python -m activation_epilogue_tcgen05_b200.build` (no fallback exists)")
            L = ctypes.CDLL(LIB_PATH)
            i64, i32, vp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
            pp = ctypes.POINTER(vp)
            L.gemm_epi_plan.argtypes = [i64, i64, i64, i32, i32, i32, pp]
            L.gemm_epi_plan_ex.argtypes = [i64, i64, i64, i32, i32, i32, i32, pp]
            L.gemm_epi_plan_opts.argtypes = [i64, i64, i64, i32, i32, i32, i32,
                                             ctypes.POINTER(Options), pp]
            L.gemm_epi_set_scales.argtypes = [vp, vp, vp]
            L.gemm_epi_run.argtypes = [vp, vp, vp, vp, vp, vp, vp]
            L.gemm_epi_unfused_run.argtypes = [vp, vp, vp, vp, vp, vp, vp]
            L.gemm_epi_run_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp]
            L.gemm_epi_unfused_run_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp]
            L.gemm_epi_set_out_scale.argtypes = [vp, vp, vp]
            L.gemm_epi_mlp_plan.argtypes = [i64, i64, i64, i32, i32, i32, pp]
            L.gemm_epi_mlp_set_scales.argtypes = [vp, vp, vp, vp, vp, vp]
            L.gemm_epi_mlp_run.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp]
            L.gemm_epi_mlp_unfused_run.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
            L.gemm_epi_mlp_check.argtypes = [vp, vp]
            L.gemm_epi_mlp_query.argtypes = [vp, ctypes.POINTER(PlanInfo), ctypes.POINTER(PlanInfo)]
            L.gemm_epi_mlp_free.argtypes = [vp]
            L.gemm_epi_check.argtypes = [vp, vp]
            L.gemm_epi_plan_query.argtypes = [vp, ctypes.POINTER(PlanInfo)]
            L.gemm_epi_plan_preview.argtypes = [i64, i64, i64, i32, i32, i32, i32,
                                                ctypes.POINTER(Options), i32, ctypes.POINTER(PlanInfo)]
            L.gemm_epi_free.argtypes = [vp]
            L.gemm_epi_status_string.argtypes = [i32]
            L.gemm_epi_status_string.restype = ctypes.c_char_p
            L.gemm_epi_aux_pitch_bytes.argtypes = [i64]
            L.gemm_epi_aux_pitch_bytes.restype = i64
            L.gemm_epi_version.argtypes = []
            L.gemm_epi_run_noalloc.argtypes = [i64, i64, i64, i32, i32, i32, i32, vp, vp, vp, vp,
                                               vp, vp, vp, i32, vp]
            L.gemm_epi_rmsnorm.argtypes = [i64, i64, i32, i32, ctypes.c_float, vp, vp, vp, vp, vp, vp, vp, vp]
            L.gemm_epi_rmsnorm_bwd.argtypes = [i64, i64, i32, ctypes.c_float, vp, vp, vp, vp, vp, vp, vp, vp]
            L.gemm_epi_rmsnorm_workspace_bytes.argtypes = [i64, i64]
            L.gemm_epi_rmsnorm_workspace_bytes.restype = i64
            L.gemm_epi_dact.argtypes = [i64, i64, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp]
            L.gemm_epi_dact_workspace_bytes.argtypes = [i64, i64, i32]
            L.gemm_epi_dact_workspace_bytes.restype = i64
            L.gemm_epi_run_ext.argtypes = [vp] * 9
            L.gemm_epi_mlp_run_prenorm.argtypes = [vp, vp, vp, vp, ctypes.c_float] + [vp] * 10
            f32 = ctypes.c_float
            L.gemm_epi_run_scaled.argtypes = [vp] * 10
            L.gemm_epi_layernorm.argtypes = [i64, i64, i32, i32, f32] + [vp] * 9
            L.gemm_epi_layernorm_workspace_bytes.argtypes = [i64, i64]
            L.gemm_epi_layernorm_workspace_bytes.restype = i64
            L.gemm_epi_layernorm_bwd.argtypes = [i64, i64, i32, f32] + [vp] * 9
            L.gemm_epi_quant_rows.argtypes = [i64, i64, i32, i32, vp, vp, vp, vp]
            L.gemm_epi_ckpt_groups.argtypes = [i64]
            L.gemm_epi_ckpt_groups.restype = i64
            L.gemm_epi_ckpt_save.argtypes = [i64, i64, i32, i32, vp, vp, vp, vp, vp]
            L.gemm_epi_ckpt_load.argtypes = [i64, i64, i32, i32, vp, vp, vp, vp]
            L.gemm_epi_dact_ckpt.argtypes = [i64, i64, i32, i32, i32] + [vp] * 8
            for name in ("gemm_epi_run_scaled", "gemm_epi_layernorm", "gemm_epi_layernorm_bwd", "gemm_epi_quant_rows", "gemm_epi_ckpt_save",
                         "gemm_epi_ckpt_load", "gemm_epi_dact_ckpt", "gemm_epi_run_ext", "gemm_epi_mlp_run_prenorm", "gemm_epi_rmsnorm", "gemm_epi_rmsnorm_bwd", "gemm_epi_dact",
                         "gemm_epi_plan", "gemm_epi_plan_ex", "gemm_epi_plan_opts",
                         "gemm_epi_set_scales", "gemm_epi_run", "gemm_epi_unfused_run",
                         "gemm_epi_check", "gemm_epi_plan_query", "gemm_epi_free",
                         "gemm_epi_version", "gemm_epi_run_noalloc", "gemm_epi_run_bwd",
                         "gemm_epi_unfused_run_bwd", "gemm_epi_set_out_scale", "gemm_epi_mlp_plan",
                         "gemm_epi_mlp_set_scales", "gemm_epi_mlp_run", "gemm_epi_mlp_check",
                         "gemm_epi_mlp_query", "gemm_epi_mlp_free", "gemm_epi_mlp_unfused_run"):
                getattr(L, name).restype = i32
            _lib = L
    return _lib


# ---------------------------------------------------------------- C-named wrappers
def gemm_epi_plan(m, n, k, dtype, epilogue, bias_axis) -> int:
    h = ctypes.c_void_p()
    _check(lib().gemm_epi_plan(m, n, k, dtype, epilogue, bias_axis, ctypes.byref(h)), "gemm_epi_plan")
    return h.value


def gemm_epi_plan_ex(m, n, k, dtype, epilogue, bias_axis, b_layout) -> int:
    h = ctypes.c_void_p()
    _check(lib().gemm_epi_plan_ex(m, n, k, dtype, epilogue, bias_axis, b_layout, ctypes.byref(h)),
           "gemm_epi_plan_ex")
    return h.value


def gemm_epi_plan_opts(m, n, k, dtype, epilogue, bias_axis, b_layout, opts: Options | None) -> int:
    h = ctypes.c_void_p()
    _check(lib().gemm_epi_plan_opts(m, n, k, dtype, epilogue, bias_axis, b_layout,
                                    ctypes.byref(opts) if opts is not None else None,
                                    ctypes.byref(h)), "gemm_epi_plan_opts")
    return h.value


def gemm_epi_set_scales(plan, d_scale_a, d_scale_b) -> None:
    _check(lib().gemm_epi_set_scales(plan, d_scale_a, d_scale_b), "gemm_epi_set_scales")


def gemm_epi_run(plan, A, B, bias, D, aux, stream) -> None:
    _check(lib().gemm_epi_run(plan, A, B, bias, D, aux, stream), "gemm_epi_run")


def gemm_epi_run_ext(plan, A, B, bias, R, d_scale_rows, D, aux, stream) -> None:
    _check(lib().gemm_epi_run_ext(plan, A, B, bias, R, d_scale_rows, D, aux, stream), "gemm_epi_run_ext")


def gemm_epi_run_scaled(plan, A, B, bias, R, d_scale_rows, d_scale_cols, D, aux, stream) -> None:
    _check(lib().gemm_epi_run_scaled(plan, A, B, bias, R, d_scale_rows, d_scale_cols, D, aux, stream), "gemm_epi_run_scaled")


def gemm_epi_unfused_run(plan, A, B, bias, D, aux, stream) -> None:
    _check(lib().gemm_epi_unfused_run(plan, A, B, bias, D, aux, stream), "gemm_epi_unfused_run")


def gemm_epi_run_bwd(plan, A, B, aux, D, dbias, stream) -> None:
    _check(lib().gemm_epi_run_bwd(plan, A, B, aux, D, dbias, stream), "gemm_epi_run_bwd")


def gemm_epi_unfused_run_bwd(plan, A, B, aux, D, dbias, stream) -> None:
    _check(lib().gemm_epi_unfused_run_bwd(plan, A, B, aux, D, dbias, stream), "gemm_epi_unfused_run_bwd")


def gemm_epi_set_out_scale(plan, d_scale_out, d_amax) -> None:
    _check(lib().gemm_epi_set_out_scale(plan, d_scale_out, d_amax), "gemm_epi_set_out_scale")


def gemm_epi_mlp_plan(m, d_model, d_ff, dtype, act, w_layout) -> int:
    h = ctypes.c_void_p()
    _check(lib().gemm_epi_mlp_plan(m, d_model, d_ff, dtype, act, w_layout, ctypes.byref(h)),
           "gemm_epi_mlp_plan")
    return h.value


def gemm_epi_mlp_set_scales(mlp, d_scale_x, d_scale_w1, d_scale_h, d_amax_h, d_scale_w2) -> None:
    _check(lib().gemm_epi_mlp_set_scales(mlp, d_scale_x, d_scale_w1, d_scale_h, d_amax_h, d_scale_w2),
           "gemm_epi_mlp_set_scales")


def gemm_epi_mlp_run(mlp, X, W1, b1, W2, b2, H, Y, stream) -> None:
    _check(lib().gemm_epi_mlp_run(mlp, X, W1, b1, W2, b2, H, Y, stream), "gemm_epi_mlp_run")


def gemm_epi_mlp_run_prenorm(mlp, X, R, gamma, eps, W1, b1, W2, b2, S, N, d_scale_rows, H, Y, stream) -> None:
    _check(lib().gemm_epi_mlp_run_prenorm(mlp, X, R, gamma, eps, W1, b1, W2, b2, S, N, d_scale_rows, H, Y, stream),
           "gemm_epi_mlp_run_prenorm")


def gemm_epi_mlp_unfused_run(mlp, X, W1, b1, W2, b2, H, Y, H_wide, stream) -> None:
    _check(lib().gemm_epi_mlp_unfused_run(mlp, X, W1, b1, W2, b2, H, Y, H_wide, stream),
           "gemm_epi_mlp_unfused_run")


def gemm_epi_mlp_check(mlp, stream) -> None:
    _check(lib().gemm_epi_mlp_check(mlp, stream), "gemm_epi_mlp_check")


def gemm_epi_mlp_query(mlp) -> tuple:
    up, down = PlanInfo(), PlanInfo()
    _check(lib().gemm_epi_mlp_query(mlp, ctypes.byref(up), ctypes.byref(down)), "gemm_epi_mlp_query")
    return up.as_dict(), down.as_dict()


def gemm_epi_mlp_free(mlp) -> None:
    _check(lib().gemm_epi_mlp_free(mlp), "gemm_epi_mlp_free")


def gemm_epi_check(plan, stream) -> None:
    _check(lib().gemm_epi_check(plan, stream), "gemm_epi_check")


def gemm_epi_plan_query(plan) -> dict:
    info = PlanInfo()
    _check(lib().gemm_epi_plan_query(plan, ctypes.byref(info)), "gemm_epi_plan_query")
    return info.as_dict()


def gemm_epi_plan_preview(m, n, k, dtype, epilogue, bias_axis, b_layout, opts: Options | None,
                          num_sms: int) -> dict:
    info = PlanInfo()
    _check(lib().gemm_epi_plan_preview(m, n, k, dtype, epilogue, bias_axis, b_layout,
                                       ctypes.byref(opts) if opts is not None else None, num_sms,
                                       ctypes.byref(info)), "gemm_epi_plan_preview")
    return info.as_dict()


def plan_preview(m, n, k, dtype="bf16", epilogue="bias", bias_axis="row", b_layout="kn", num_sms=148,
                 kernel="auto", block_n=0, split_k=0, max_ctas=0, stream_k="auto", out_e4m3=False,
                 a_layout="mk") -> dict:
    """The kernel choice a plan would make on a device with ``num_sms`` SMs, computed on the
    host (no device needed); the same names as :class:`Plan`, the same keys as ``Plan.info``."""
    opts = Options(KERNEL[kernel], int(block_n), int(split_k), int(max_ctas), 0, STREAM_K[stream_k],
                   1 if out_e4m3 else 0)
    layout = LAYOUT[b_layout] | (A_KM if a_layout == "km" else 0)
    return gemm_epi_plan_preview(int(m), int(n), int(k), DTYPE[dtype], EPILOGUE[epilogue], AXIS[bias_axis],
                                 layout, opts, int(num_sms))


def gemm_epi_free(plan) -> None:
    _check(lib().gemm_epi_free(plan), "gemm_epi_free")


def gemm_epi_status_string(status: int) -> str:
    return lib().gemm_epi_status_string(status).decode()


def gemm_epi_aux_pitch_bytes(n: int) -> int:
    return lib().gemm_epi_aux_pitch_bytes(n)


def gemm_epi_version() -> int:
    return lib().gemm_epi_version()


def gemm_epi_run_noalloc(m, n, k, dtype, epilogue, bias_axis, b_layout, A, B, bias, d_scale_a,
                         d_scale_b, D, aux, wait, stream) -> None:
    """Allocation-free fused run (see include/gemm_epi.h); raises on a non-zero status."""
    _check(lib().gemm_epi_run_noalloc(m, n, k, dtype, epilogue, bias_axis, b_layout, A, B, bias,
                                      d_scale_a, d_scale_b, D, aux, wait, stream),
           "gemm_epi_run_noalloc")


def gemm_epi_rmsnorm(m, d, dtype, out_mode, eps, X, R, gamma, S, Y, d_scale, d_amax, stream) -> None:
    _check(lib().gemm_epi_rmsnorm(m, d, dtype, out_mode, eps, X, R, gamma, S, Y, d_scale, d_amax, stream),
           "gemm_epi_rmsnorm")


def gemm_epi_rmsnorm_workspace_bytes(m: int, d: int) -> int:
    return lib().gemm_epi_rmsnorm_workspace_bytes(m, d)


def gemm_epi_rmsnorm_bwd(m, d, dtype, eps, dY, S, gamma, dS, dX, dgamma, workspace, stream) -> None:
    _check(lib().gemm_epi_rmsnorm_bwd(m, d, dtype, eps, dY, S, gamma, dS, dX, dgamma, workspace, stream),
           "gemm_epi_rmsnorm_bwd")


def gemm_epi_layernorm(m, d, dtype, out_mode, eps, X, R, gamma, beta, S, Y, d_scale, d_amax, stream) -> None:
    _check(lib().gemm_epi_layernorm(m, d, dtype, out_mode, eps, X, R, gamma, beta, S, Y, d_scale, d_amax, stream),
           "gemm_epi_layernorm")


def gemm_epi_layernorm_workspace_bytes(m: int, d: int) -> int:
    return lib().gemm_epi_layernorm_workspace_bytes(m, d)


def gemm_epi_layernorm_bwd(m, d, dtype, eps, dY, S, gamma, dS, dX, dgamma, dbeta, workspace, stream) -> None:
    _check(lib().gemm_epi_layernorm_bwd(m, d, dtype, eps, dY, S, gamma, dS, dX, dgamma, dbeta, workspace, stream),
           "gemm_epi_layernorm_bwd")


def gemm_epi_quant_rows(m, d, dtype, out_mode, X, Q, d_scale, stream) -> None:
    _check(lib().gemm_epi_quant_rows(m, d, dtype, out_mode, X, Q, d_scale, stream), "gemm_epi_quant_rows")


def gemm_epi_ckpt_groups(n: int) -> int:
    return lib().gemm_epi_ckpt_groups(n)


def gemm_epi_ckpt_save(m, n, dtype, epilogue, Z, H, codes, exps, stream) -> None:
    _check(lib().gemm_epi_ckpt_save(m, n, dtype, epilogue, Z, H, codes, exps, stream), "gemm_epi_ckpt_save")


def gemm_epi_ckpt_load(m, n, dtype, epilogue, codes, exps, X, stream) -> None:
    _check(lib().gemm_epi_ckpt_load(m, n, dtype, epilogue, codes, exps, X, stream), "gemm_epi_ckpt_load")


def gemm_epi_dact_ckpt(m, n, dtype, epilogue, bias_axis, dD, codes, exps, dZ, H, dbias, workspace, stream) -> None:
    _check(lib().gemm_epi_dact_ckpt(m, n, dtype, epilogue, bias_axis, dD, codes, exps, dZ, H, dbias, workspace, stream),
           "gemm_epi_dact_ckpt")


def gemm_epi_dact_workspace_bytes(m: int, n: int, bias_axis: int) -> int:
    return lib().gemm_epi_dact_workspace_bytes(m, n, bias_axis)


def gemm_epi_dact(m, n, dtype, epilogue, bias_axis, dD, Z, aux, dZ, dbias, workspace, stream) -> None:
    _check(lib().gemm_epi_dact(m, n, dtype, epilogue, bias_axis, dD, Z, aux, dZ, dbias, workspace, stream),
           "gemm_epi_dact")


def status_string(status: int) -> str:
    try:
        return gemm_epi_status_string(status)
    except Exception:  # library not loadable: still report the number
        return "status"


def _check(rc: int, what: str) -> None:
    if rc != OK:
        raise GemmEpiError(rc, what)


# ---------------------------------------------------------------- torch convenience
def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


class Plan:
    """Owns one gemm_epi plan; ``run`` passes torch tensors' device pointers.

    ``dtype``/``epilogue``/``bias_axis``/``b_layout``/``kernel`` take the
    names used across the package ("bf16", "relu_aux_bias", "row", "kn", ...).
    """

    def __init__(self, m, n, k, dtype="bf16", epilogue="bias", bias_axis="row", b_layout="kn",
                 kernel="auto", block_n=0, split_k=0, max_ctas=0, inject_stall=0, stream_k="auto",
                 out_e4m3=False, a_layout="mk"):
        self.m, self.n, self.k = int(m), int(n), int(k)
        self.dtype, self.epilogue, self.bias_axis = dtype, epilogue, bias_axis
        self.a_layout, self.b_layout = a_layout, b_layout
        opts = Options(KERNEL[kernel], int(block_n), int(split_k), int(max_ctas), int(inject_stall),
                       STREAM_K[stream_k], 1 if out_e4m3 else 0)
        layout = LAYOUT[b_layout] | (A_KM if a_layout == "km" else 0)
        self.handle = gemm_epi_plan_opts(self.m, self.n, self.k, DTYPE[dtype], EPILOGUE[epilogue],
                                         AXIS[bias_axis], layout, opts)
        self.out_e4m3 = bool(out_e4m3)
        self._scales = self._ext = self._i8 = None

    @property
    def info(self) -> dict:
        return gemm_epi_plan_query(self.handle)

    def set_scales(self, scale_a, scale_b):
        """fp32 device scalars (torch tensors); kept alive by the plan object."""
        self._scales = (scale_a, scale_b)
        gemm_epi_set_scales(self.handle, _ptr(scale_a), _ptr(scale_b))

    def set_out_scale(self, scale_out, amax=None):
        """FP8-output plans: fp32 device scalars (the output scale; the amax word or None)."""
        self._out = (scale_out, amax)
        gemm_epi_set_out_scale(self.handle, _ptr(scale_out), _ptr(amax))

    def run(self, A, B, bias, D, aux=None, stream=None, fused=True):
        s = _stream_ptr(stream)
        f = gemm_epi_run if fused else gemm_epi_unfused_run
        f(self.handle, _ptr(A), _ptr(B), _ptr(bias), _ptr(D), _ptr(aux), s)

    def run_ext(self, A, B, bias, D, residual=None, scale_rows=None, aux=None, stream=None):
        """D = act(alpha_i * A.B + bias) + residual; ``scale_rows``: m fp32 values, one scale a row of A
        (see gemm_epi_run_ext in include/gemm_epi.h).  ``residual`` may be D."""
        dev, s = _device_and_stream(stream)
        if self._ext is None:
            self._ext = self._ext_operands()
        t, a, b, wide, bias_of, out, d, f32, rows, i32, mask = self._ext
        gemm_epi_run_ext(self.handle, _operand(A, "Plan.run_ext: A", t, a, dev), _operand(B, "Plan.run_ext: B", t, b, dev),
                         None if bias_of is None else _operand(bias, "Plan.run_ext: bias", wide, bias_of, dev),
                         None if residual is None else _operand(residual, "Plan.run_ext: residual", wide, d, dev),
                         None if scale_rows is None else _operand(scale_rows, "Plan.run_ext: scale_rows", f32, rows, dev),
                         _operand(D, "Plan.run_ext: D", out, d, dev),
                         None if mask is None else _operand(aux, "Plan.run_ext: aux", i32, mask, dev), s)

    def run_i8(self, A, B, bias, D, scale_rows, scale_cols, residual=None, aux=None, stream=None):
        """dtype "i8": D = act(scale_rows_i * scale_cols_j * (A.B)_ij + bias) + residual; ``scale_rows``: m fp32 values,
        ``scale_cols``: n of them (see gemm_epi_run_scaled in include/gemm_epi.h).  ``residual`` may be D."""
        dev, s = _device_and_stream(stream)
        if self._i8 is None:
            if self.dtype != "i8":
                raise GemmEpiError(ERR_ARG, f"Plan.run_i8: a plan of {self.dtype!r}")
            self._i8 = self._ext_operands() + ((self.n,),)
        t, a, b, wide, bias_of, out, d, f32, rows, i32, mask, cols = self._i8
        gemm_epi_run_scaled(self.handle, _operand(A, "Plan.run_i8: A", t, a, dev), _operand(B, "Plan.run_i8: B", t, b, dev),
                        None if bias_of is None else _operand(bias, "Plan.run_i8: bias", wide, bias_of, dev),
                        None if residual is None else _operand(residual, "Plan.run_i8: residual", wide, d, dev),
                        _operand(scale_rows, "Plan.run_i8: scale_rows", f32, rows, dev),
                        _operand(scale_cols, "Plan.run_i8: scale_cols", f32, cols, dev),
                        _operand(D, "Plan.run_i8: D", out, d, dev),
                        None if mask is None else _operand(aux, "Plan.run_i8: aux", i32, mask, dev), s)

    def _ext_operands(self):
        """Types and shapes of run_ext's operands: of A and B, of the bias (None without one) and the residual, of D,
        of the row scales, of the mask (None without one)."""
        import torch
        t = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "i8": torch.int8}[self.dtype]
        wide = torch.bfloat16 if self.dtype in ("e4m3", "i8") else t
        m, n, k = self.m, self.n, self.k
        return (t, (k, m) if self.a_layout == "km" else (m, k), (n, k) if self.b_layout == "nk" else (k, n),
                wide, (m if self.bias_axis == "row" else n,) if self.epilogue in HAS_BIAS else None,
                t if self.out_e4m3 else wide, (m, n), torch.float32, (m,),
                torch.int32, (m, aux_pitch_words(n)) if self.epilogue in HAS_AUX else None)

    def run_bwd(self, A, B, aux, D, dbias=None, stream=None, fused=True):
        """Backward plans (``drelu``/``drelu_bgrad``): D = mask ? alpha*A.B : 0 (+ dbias)."""
        s = _stream_ptr(stream)
        f = gemm_epi_run_bwd if fused else gemm_epi_unfused_run_bwd
        f(self.handle, _ptr(A), _ptr(B), _ptr(aux), _ptr(D), _ptr(dbias), s)

    def check(self, stream=None):
        gemm_epi_check(self.handle, _stream_ptr(stream))

    def close(self):
        if getattr(self, "handle", None):
            gemm_epi_free(self.handle)
            self.handle = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _stream_ptr(stream):
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream) if hasattr(stream, "cuda_stream") else stream


def aux_pitch_words(n: int) -> int:
    return gemm_epi_aux_pitch_bytes(n) // 4


class MlpPlan:
    """Owns one MLP-block handle (gemm_epi_mlp_*): H = act(X.W1 + b1), Y = H.W2 + b2."""

    def __init__(self, m, d_model, d_ff, dtype="bf16", act="gelu_bias", w_layout="kn"):
        self.m, self.d_model, self.d_ff = int(m), int(d_model), int(d_ff)
        self.dtype, self.act, self.w_layout = dtype, act, w_layout
        self.handle = gemm_epi_mlp_plan(self.m, self.d_model, self.d_ff, DTYPE[dtype], EPILOGUE[act],
                                        LAYOUT[w_layout])
        self._scales = None

    @property
    def info(self) -> tuple:
        return gemm_epi_mlp_query(self.handle)

    def set_scales(self, scale_x, scale_w1, scale_h, amax_h, scale_w2):
        self._scales = (scale_x, scale_w1, scale_h, amax_h, scale_w2)
        gemm_epi_mlp_set_scales(self.handle, _ptr(scale_x), _ptr(scale_w1), _ptr(scale_h), _ptr(amax_h),
                                _ptr(scale_w2))

    def run(self, X, W1, b1, W2, b2, H, Y, stream=None, fused=True, H_wide=None):
        """fused=False: the unfused baseline (H_wide: bf16 (m, d_ff) scratch, e4m3 plans)."""
        if fused:
            gemm_epi_mlp_run(self.handle, _ptr(X), _ptr(W1), _ptr(b1), _ptr(W2), _ptr(b2), _ptr(H), _ptr(Y),
                             _stream_ptr(stream))
        else:
            gemm_epi_mlp_unfused_run(self.handle, _ptr(X), _ptr(W1), _ptr(b1), _ptr(W2), _ptr(b2), _ptr(H),
                                     _ptr(Y), _ptr(H_wide), _stream_ptr(stream))

    def run_prenorm(self, X, gamma, W1, b1, W2, b2, N, H, Y, residual=None, S=None, scale_rows=None, eps=1e-6, stream=None):
        """S = X + residual, N = rmsnorm(S) * gamma, H = act(N.W1 + b1), Y = H.W2 + b2 + S (S is X without
        a residual); e4m3: ``scale_rows``, m fp32 values of scratch for N's scales by row."""
        import torch
        dev, s = _device_and_stream(stream)
        t = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[self.dtype]
        wide = torch.bfloat16 if self.dtype == "e4m3" else t
        m, dm, ff, w = self.m, self.d_model, self.d_ff, "MlpPlan.run_prenorm: "
        w1, w2 = ((ff, dm), (dm, ff)) if self.w_layout == "nk" else ((dm, ff), (ff, dm))
        gemm_epi_mlp_run_prenorm(
            self.handle, _operand(X, w + "X", wide, (m, dm), dev), _operand(residual, w + "residual", wide, (m, dm), dev, True),
            _operand(gamma, w + "gamma", wide, (dm,), dev), float(eps), _operand(W1, w + "W1", t, w1, dev),
            _operand(b1, w + "b1", wide, (ff,), dev), _operand(W2, w + "W2", t, w2, dev), _operand(b2, w + "b2", wide, (dm,), dev),
            _operand(S, w + "S", wide, (m, dm), dev, True), _operand(N, w + "N", t, (m, dm), dev),
            _operand(scale_rows, w + "scale_rows", torch.float32, (m,), dev, True), _operand(H, w + "H", t, (m, ff), dev),
            _operand(Y, w + "Y", wide, (m, dm), dev), s)

    def check(self, stream=None):
        gemm_epi_mlp_check(self.handle, _stream_ptr(stream))

    def close(self):
        if getattr(self, "handle", None):
            gemm_epi_mlp_free(self.handle)
            self.handle = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _operand(t, name, dtype, shape, device, optional=False):
    """Device address of a tensor that has to be dense values of ``dtype`` on the current device (None
    for an optional one left out), ``shape`` its (rows, columns) or (length,): flat, or with an axis
    split, the rows are the same; another shape of as many values is a mistake."""
    if t is None:
        if optional:
            return None
        raise GemmEpiError(ERR_NULL, name)
    if (t.dtype is not dtype or (t.shape != shape and not _same_rows(t.shape, shape)) or not t.is_contiguous()
            or t.get_device() != device):
        raise GemmEpiError(ERR_ARG, f"{name}: wanted contiguous {shape} {dtype} on cuda:{device}, got "
                                    f"{tuple(t.shape)} {t.dtype} on {t.device}, strides {t.stride()}")
    return t.data_ptr()


def _same_rows(got, want):
    """Whether contiguous values of shape ``got`` are the rows of ``want``: as many of them, and flat or with
    an axis's end where a row ends."""
    if math.prod(got) != math.prod(want):
        return False
    if len(want) == 1 or len(got) <= 1:
        return True
    n = 1
    for k in got:
        if n == want[0]:
            return True
        n *= k
    return n == want[0]


_current = None


def _device_and_stream(stream):
    """(current device index, raw stream): the device's current stream when none is given."""
    global _current
    if _current is None:               # looked up once: 0.15 us of every call
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)     # 0.1 us; a Stream object costs 1.3 us
        _current = torch.cuda.current_device, raw or (lambda d: torch.cuda.current_stream(d).cuda_stream)
        _compiled_checks()
    device = _current[0]()
    return device, _current[1](device) if stream is None else getattr(stream, "cuda_stream", stream)


_python_forms = _operand, _device_and_stream
_install = threading.Lock()


def _compiled_checks() -> bool:
    """Put the compiled forms of ``_operand`` and ``_device_and_stream`` (binding/operands.cpp) in their place, where
    build.py has made them for this torch and Python; they hand what is not in order to the forms here, and a call of six
    operands takes 2 us less.  Threads may make their first calls together."""
    global _operand, _device_and_stream
    with _install:
        if _operand is not _python_forms[0]:
            return True
        try:
            from . import _operands
        except ImportError:
            return False
        import torch
        if getattr(_operands, "built_for", None) != f"{torch.__version__} {sys.version}":
            return False
        _operands.set_python_forms(*_python_forms)
        _operand, _device_and_stream = _operands.operand, _operands.device_and_stream
    return True


def _scratch(nbytes, device, stream):
    """Scratch of one call.  Memory that is handed out to the stream that uses it may be given
    back as soon as the call is enqueued; a stream that is not the current one is made the
    current one for the allocation."""
    import torch
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(getattr(stream, "value", stream) or 0), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


class _Norm:
    """Sizes and types of a norm's operands."""

    def __init__(self, m, d, dtype="bf16", out="same", eps=1e-6):
        import torch
        self.m, self.d, self.dtype, self.out, self.eps = int(m), int(d), dtype, out, float(eps)
        if dtype not in ("f16", "bf16"):
            raise GemmEpiError(ERR_ARG, f"{type(self).__name__}: dtype {dtype!r}")
        self._t = torch.float16 if dtype == "f16" else torch.bfloat16
        self._dt, self._mode = DTYPE[dtype], NORM_OUT[out]
        self._out_t = self._t if out == "same" else torch.int8 if out == "i8_rows" else torch.float8_e4m3fn
        self._f32 = torch.float32
        self._shape, self._row, self._one = (self.m, self.d), (self.d,), (1,)
        self._scales = (self.m,) if out in ("e4m3_rows", "i8_rows") else (1,)


class RmsNorm(_Norm):
    """Root-mean-square norm of (m, d) rows with the residual's addition before it, and its backward
    (gemm_epi_rmsnorm, gemm_epi_rmsnorm_bwd).  ``dtype``: "f16" or "bf16"; ``out``: "same", "e4m3" (a given
    scale), "e4m3_rows" or "i8_rows" (one scale a row, written).  The object holds sizes only."""

    def __init__(self, m, d, dtype="bf16", out="same", eps=1e-6):
        super().__init__(m, d, dtype, out, eps)
        self._scratch_bytes = gemm_epi_rmsnorm_workspace_bytes(self.m, self.d)

    def run(self, X, gamma, Y, residual=None, S=None, scale=None, amax=None, stream=None):
        """S = X + residual (X without one), Y = S / rms(S) * gamma; ``scale`` and ``amax`` as in
        include/gemm_epi.h.  S or Y may be X or residual."""
        dev, s = _device_and_stream(stream)
        shape, t = self._shape, self._t
        gemm_epi_rmsnorm(self.m, self.d, self._dt, self._mode, self.eps, _operand(X, "RmsNorm.run: X", t, shape, dev),
                         _operand(residual, "RmsNorm.run: residual", t, shape, dev, True),
                         _operand(gamma, "RmsNorm.run: gamma", t, self._row, dev),
                         _operand(S, "RmsNorm.run: S", t, shape, dev, True),
                         _operand(Y, "RmsNorm.run: Y", self._out_t, shape, dev),
                         _operand(scale, "RmsNorm.run: scale", self._f32, self._scales, dev, True),
                         _operand(amax, "RmsNorm.run: amax", self._f32, self._one, dev, True), s)

    def run_bwd(self, dY, S, gamma, dX, dgamma=None, dS=None, workspace=None, stream=None):
        """dX (of X and of the residual alike) and, if given, dgamma, from the sum S of the forward run
        (X without a residual); dS: the skip connection's gradient.  ``workspace``: a uint8 tensor of
        gemm_epi_rmsnorm_workspace_bytes(m, d) bytes, taken from torch's allocator when left out."""
        dev, s = _device_and_stream(stream)
        shape, t = self._shape, self._t
        if dgamma is None or not self._scratch_bytes:
            workspace = None
        else:
            workspace = _workspace(workspace, self._scratch_bytes, "RmsNorm.run_bwd", dev, stream)
        gemm_epi_rmsnorm_bwd(self.m, self.d, self._dt, self.eps, _operand(dY, "RmsNorm.run_bwd: dY", t, shape, dev),
                             _operand(S, "RmsNorm.run_bwd: S", t, shape, dev),
                             _operand(gamma, "RmsNorm.run_bwd: gamma", t, self._row, dev),
                             _operand(dS, "RmsNorm.run_bwd: dS", t, shape, dev, True),
                             _operand(dX, "RmsNorm.run_bwd: dX", t, shape, dev),
                             _operand(dgamma, "RmsNorm.run_bwd: dgamma", t, self._row, dev, True),
                             None if workspace is None else workspace.data_ptr(), s)


class LayerNorm(_Norm):
    """Layer norm of (m, d) rows with the residual's addition before it, and its backward (gemm_epi_layernorm,
    gemm_epi_layernorm_bwd).  Arguments as for :class:`RmsNorm`.  The object holds sizes only."""

    def __init__(self, m, d, dtype="bf16", out="same", eps=1e-5):
        super().__init__(m, d, dtype, out, eps)
        self._scratch_bytes = gemm_epi_layernorm_workspace_bytes(self.m, self.d)

    def run(self, X, gamma, Y, beta=None, residual=None, S=None, scale=None, amax=None, stream=None):
        """S = X + residual (X without one), Y = (S - mean) / deviation * gamma + beta; ``scale`` and ``amax`` as in
        include/gemm_epi.h.  S or Y may be X or residual."""
        dev, s = _device_and_stream(stream)
        shape, t = self._shape, self._t
        gemm_epi_layernorm(self.m, self.d, self._dt, self._mode, self.eps, _operand(X, "LayerNorm.run: X", t, shape, dev),
                           _operand(residual, "LayerNorm.run: residual", t, shape, dev, True),
                           _operand(gamma, "LayerNorm.run: gamma", t, self._row, dev),
                           _operand(beta, "LayerNorm.run: beta", t, self._row, dev, True),
                           _operand(S, "LayerNorm.run: S", t, shape, dev, True),
                           _operand(Y, "LayerNorm.run: Y", self._out_t, shape, dev),
                           _operand(scale, "LayerNorm.run: scale", self._f32, self._scales, dev, True),
                           _operand(amax, "LayerNorm.run: amax", self._f32, self._one, dev, True), s)

    def run_bwd(self, dY, S, gamma, dX, dgamma=None, dbeta=None, dS=None, workspace=None, stream=None):
        """dX (of X and of the residual alike) and, if given, dgamma and dbeta, from the sum S of the forward run (X
        without a residual); dS: the skip connection's gradient.  ``workspace``: a uint8 tensor of
        gemm_epi_layernorm_workspace_bytes(m, d) bytes, taken from torch's allocator when left out."""
        dev, s = _device_and_stream(stream)
        shape, t = self._shape, self._t
        if (dgamma is None and dbeta is None) or not self._scratch_bytes:
            workspace = None
        else:
            workspace = _workspace(workspace, self._scratch_bytes, "LayerNorm.run_bwd", dev, stream)
        gemm_epi_layernorm_bwd(self.m, self.d, self._dt, self.eps, _operand(dY, "LayerNorm.run_bwd: dY", t, shape, dev),
                               _operand(S, "LayerNorm.run_bwd: S", t, shape, dev),
                               _operand(gamma, "LayerNorm.run_bwd: gamma", t, self._row, dev),
                               _operand(dS, "LayerNorm.run_bwd: dS", t, shape, dev, True),
                               _operand(dX, "LayerNorm.run_bwd: dX", t, shape, dev),
                               _operand(dgamma, "LayerNorm.run_bwd: dgamma", t, self._row, dev, True),
                               _operand(dbeta, "LayerNorm.run_bwd: dbeta", t, self._row, dev, True),
                               None if workspace is None else workspace.data_ptr(), s)


class QuantRows:
    """(m, d) rows quantised with one scale each (gemm_epi_quant_rows): ``out`` "i8_rows" or "e4m3_rows".  The object holds
    sizes only."""

    def __init__(self, m, d, dtype="bf16", out="i8_rows"):
        import torch
        self.m, self.d, self.dtype, self.out = int(m), int(d), dtype, out
        if dtype not in ("f16", "bf16") or out not in ("i8_rows", "e4m3_rows"):
            raise GemmEpiError(ERR_ARG, f"QuantRows: dtype {dtype!r}, out {out!r}")
        self._t, self._f32 = torch.float16 if dtype == "f16" else torch.bfloat16, torch.float32
        self._out_t = torch.int8 if out == "i8_rows" else torch.float8_e4m3fn
        self._dt, self._mode, self._shape, self._scales = DTYPE[dtype], NORM_OUT[out], (self.m, self.d), (self.m,)

    def run(self, X, Q, scale, stream=None):
        """Q = the codes of X / scale, scale: m fp32 values, written."""
        dev, s = _device_and_stream(stream)
        gemm_epi_quant_rows(self.m, self.d, self._dt, self._mode, _operand(X, "QuantRows.run: X", self._t, self._shape, dev),
                            _operand(Q, "QuantRows.run: Q", self._out_t, self._shape, dev),
                            _operand(scale, "QuantRows.run: scale", self._f32, self._scales, dev), s)


class ActCheckpoint:
    """Checkpoints of an (m, n) pre-activation in 8 bits (gemm_epi_ckpt_save, gemm_epi_ckpt_load): ``codes`` (m, n) int8 and
    ``exps`` (m, groups) uint8, ``groups`` of 32 columns each.  ``dtype`` ("bf16" for an "i8" plan, whose z is) and ``epilogue``
    are the forward plan's.  The object holds sizes only."""

    def __init__(self, m, n, dtype="bf16", epilogue="gelu_bias"):
        import torch
        self.m, self.n, self.dtype, self.epilogue = int(m), int(n), dtype, epilogue
        self.groups = gemm_epi_ckpt_groups(self.n)
        self._dt, self._epi = DTYPE[dtype], EPILOGUE[epilogue]
        self._t, self._i8, self._u8 = torch.float16 if dtype == "f16" else torch.bfloat16, torch.int8, torch.uint8
        self._shape, self._exps = (self.m, self.n), (self.m, self.groups)

    def save(self, Z, codes, exps, H=None, stream=None):
        """Z kept as codes and exps; H = act(Z), if given (H may be Z)."""
        dev, s = _device_and_stream(stream)
        gemm_epi_ckpt_save(self.m, self.n, self._dt, self._epi, _operand(Z, "ActCheckpoint.save: Z", self._t, self._shape, dev),
                           _operand(H, "ActCheckpoint.save: H", self._t, self._shape, dev, True),
                           _operand(codes, "ActCheckpoint.save: codes", self._i8, self._shape, dev),
                           _operand(exps, "ActCheckpoint.save: exps", self._u8, self._exps, dev), s)

    def load(self, codes, exps, X, act=False, stream=None):
        """X = z as kept, or (``act``) act(z)."""
        dev, s = _device_and_stream(stream)
        gemm_epi_ckpt_load(self.m, self.n, self._dt, self._epi if act else NONE,
                           _operand(codes, "ActCheckpoint.load: codes", self._i8, self._shape, dev),
                           _operand(exps, "ActCheckpoint.load: exps", self._u8, self._exps, dev),
                           _operand(X, "ActCheckpoint.load: X", self._t, self._shape, dev), s)


class ActBackward:
    """Backward of a forward plan's epilogue (gemm_epi_dact, gemm_epi_dact_ckpt): dZ = dD * act'(z) and dbias, the names as
    for :class:`Plan` (``dtype`` "bf16" for an "i8" plan, whose z is).  The object holds sizes only."""

    def __init__(self, m, n, dtype="bf16", epilogue="bias", bias_axis="row"):
        import torch
        self.m, self.n, self.dtype, self.epilogue, self.bias_axis = int(m), int(n), dtype, epilogue, bias_axis
        self._args = (DTYPE[dtype], EPILOGUE[epilogue], AXIS[bias_axis])
        self._t = torch.float16 if dtype == "f16" else torch.bfloat16
        self._i32 = torch.int32
        self._shape, self._len = (self.m, self.n), (self.m if bias_axis == "row" else self.n,)
        self._aux_words = (self.m, aux_pitch_words(self.n))
        self._i8, self._u8, self._exps = torch.int8, torch.uint8, (self.m, gemm_epi_ckpt_groups(self.n))
        self._scratch_bytes = gemm_epi_dact_workspace_bytes(self.m, self.n, AXIS[bias_axis])

    def run(self, dD, dZ=None, z=None, aux=None, dbias=None, workspace=None, stream=None):
        """``z``: the pre-activation (ReLU, GELU, tanh); ``aux``: the forward's packed mask as int32 words
        (relu_aux, relu_aux_bias); dZ: left out without an activation; dbias: left out if not wanted;
        ``workspace``: as for RmsNorm.run_bwd (gemm_epi_dact_workspace_bytes)."""
        dev, s = _device_and_stream(stream)
        shape, t = self._shape, self._t
        if dbias is None or not self._scratch_bytes:
            workspace = None
        else:
            workspace = _workspace(workspace, self._scratch_bytes, "ActBackward.run", dev, stream)
        gemm_epi_dact(self.m, self.n, *self._args, _operand(dD, "ActBackward.run: dD", t, shape, dev),
                      _operand(z, "ActBackward.run: z", t, shape, dev, True),
                      _operand(aux, "ActBackward.run: aux", self._i32, self._aux_words, dev, True),
                      _operand(dZ, "ActBackward.run: dZ", t, shape, dev, True),
                      _operand(dbias, "ActBackward.run: dbias", t, self._len, dev, True),
                      None if workspace is None else workspace.data_ptr(), s)

    def run_ckpt(self, dD, codes, exps, dZ, H=None, dbias=None, workspace=None, stream=None):
        """The same from z's checkpoint (:class:`ActCheckpoint`): dZ = dD * act'(z), dbias and, if given, H = act(z), with
        z as kept (relu, gelu and tanh epilogues without a mask)."""
        dev, s = _device_and_stream(stream)
        shape, t = self._shape, self._t
        if dbias is None or not self._scratch_bytes:
            workspace = None
        else:
            workspace = _workspace(workspace, self._scratch_bytes, "ActBackward.run_ckpt", dev, stream)
        gemm_epi_dact_ckpt(self.m, self.n, *self._args, _operand(dD, "ActBackward.run_ckpt: dD", t, shape, dev),
                           _operand(codes, "ActBackward.run_ckpt: codes", self._i8, shape, dev),
                           _operand(exps, "ActBackward.run_ckpt: exps", self._u8, self._exps, dev),
                           _operand(dZ, "ActBackward.run_ckpt: dZ", t, shape, dev),
                           _operand(H, "ActBackward.run_ckpt: H", t, shape, dev, True),
                           _operand(dbias, "ActBackward.run_ckpt: dbias", t, self._len, dev, True),
                           None if workspace is None else workspace.data_ptr(), s)


def _workspace(given, nbytes, what, device, stream):
    if given is None:
        return _scratch(nbytes, device, stream)
    if given.numel() * given.element_size() < nbytes or not given.is_contiguous() or given.get_device() != device:
        raise GemmEpiError(ERR_ARG, f"{what}: workspace of {nbytes} contiguous bytes on cuda:{device} wanted")
    return given
