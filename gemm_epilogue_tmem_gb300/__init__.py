"""Python binding of libgf.so, the fused GEMM + epilogue library for GB300.

Argument marshalling only: every step of the path runs in the CUDA kernels
behind the C ABI declared in ``include/gf.h``. The functions keep the C names
(``gf_matmul_plan``, ``gf_matmul_execute``, ``gf_plan_free`` ...) and take
either torch tensors (device memory) or raw integer device pointers. There is
no CPU fallback: importing works without a GPU, but the library must be built
(``build()``) and every call fails loudly when it is missing.
"""
from __future__ import annotations

import ctypes
import os

from ._build import LIB, build

__all__ = [
    "GF_OK", "GF_ERR_INVALID_VALUE", "GF_ERR_UNSUPPORTED", "GF_ERR_NO_DEVICE", "GF_ERR_CUDA",
    "GF_ERR_OUT_OF_MEMORY", "GF_ERR_DEVICE_TIMEOUT",
    "GF_F16", "GF_BF16",
    "GF_EPILOG_NONE", "GF_EPILOG_RELU_BIAS", "GF_EPILOG_RELU_AUX_BIAS", "GF_EPILOG_DRELU_BGRAD",
    "GF_EPILOG_BIAS", "GF_EPILOG_GELU_BIAS", "GF_EPILOG_GELU_AUX_BIAS", "GF_EPILOG_DGELU_BGRAD",
    "GF_BIAS_COL", "GF_BIAS_ROW", "GF_B_KN", "GF_B_NK", "GF_BGRAD_TWO_PASS", "GF_BGRAD_ATOMIC",
    "GF_OPT_BGRAD_MODE", "GF_OPT_WAIT_LIMIT_US", "GF_OPT_TILE_N", "GF_OPT_FAULT_DROP_LOAD",
    "GF_OPT_KERNEL", "GF_OPT_GROUP_M", "GF_OPT_L2_HINTS", "GF_OPT_SCHEDULE", "GF_OPT_SPLIT_K",
    "GF_OPT_PDL", "GF_OPT_RASTER",
    "GfError", "Plan", "build", "lib", "gf_matmul_plan", "gf_matmul_plan_ex",
    "gf_matmul_execute", "gf_plan_status", "gf_plan_set_option", "gf_plan_describe",
    "gf_plan_free", "gf_status_string", "gf_last_error", "gf_drelu_bgrad_noalloc",
    "gf_noalloc_status",
    "gf_swiglu_plan", "gf_swiglu_execute", "gf_dswiglu_plan", "gf_dswiglu_execute",
    "GF_NOALLOC_MAX_PARTIALS",
    "GF_FP8_EPILOG_NONE", "GF_FP8_EPILOG_SWIGLU_QUANT",
    "gf_moe_plan", "gf_moe_dispatch_execute", "gf_moe_dispatch_fp8_execute",
    "gf_moe_dispatch_grad_execute", "gf_moe_combine_execute", "gf_moe_combine_grad_execute",
    "gf_fp8_quantize", "gf_fp8_matmul_plan", "gf_fp8_matmul_execute",
    "GF_F32", "GF_ACT_NONE", "GF_ACT_RELU", "GF_ACT_GELU", "GF_ACT_SILU",
    "GF_SCORE_SOFTMAX", "GF_SCORE_SIGMOID",
    "gf_matmul_residual_plan", "gf_matmul_residual_execute",
    "gf_dact_bgrad_plan", "gf_dact_bgrad_execute",
    "gf_rmsnorm_plan", "gf_rmsnorm_execute", "gf_rmsnorm_grad_execute",
    "gf_route_plan", "gf_route_execute", "gf_route_grad_execute",
]

# gf_status
GF_OK, GF_ERR_INVALID_VALUE, GF_ERR_UNSUPPORTED, GF_ERR_NO_DEVICE = 0, 1, 2, 3
GF_ERR_CUDA, GF_ERR_OUT_OF_MEMORY, GF_ERR_DEVICE_TIMEOUT = 4, 5, 6
# gf_dtype
GF_F16, GF_BF16, GF_F32 = 0, 1, 2
# gf_epilog
GF_EPILOG_NONE, GF_EPILOG_RELU_BIAS, GF_EPILOG_RELU_AUX_BIAS = 0, 1, 2
GF_EPILOG_DRELU_BGRAD, GF_EPILOG_BIAS = 3, 4
GF_EPILOG_GELU_BIAS, GF_EPILOG_GELU_AUX_BIAS, GF_EPILOG_DGELU_BGRAD = 5, 6, 7
# gf_bias_axis, gf_b_layout, gf_bgrad_mode
GF_BIAS_COL, GF_BIAS_ROW = 0, 1
GF_B_KN, GF_B_NK = 0, 1
GF_BGRAD_TWO_PASS, GF_BGRAD_ATOMIC = 0, 1
# gf_option
GF_OPT_BGRAD_MODE, GF_OPT_WAIT_LIMIT_US, GF_OPT_TILE_N, GF_OPT_FAULT_DROP_LOAD = 0, 1, 2, 3
GF_OPT_KERNEL, GF_OPT_GROUP_M, GF_OPT_L2_HINTS, GF_OPT_SCHEDULE = 4, 5, 6, 7
GF_OPT_SPLIT_K, GF_OPT_PDL, GF_OPT_RASTER = 8, 9, 10
# gf_fp8_epilog
GF_FP8_EPILOG_NONE, GF_FP8_EPILOG_SWIGLU_QUANT = 0, 1
# gf_activation, gf_score
GF_ACT_NONE, GF_ACT_RELU, GF_ACT_GELU, GF_ACT_SILU = 0, 1, 2, 3
GF_SCORE_SOFTMAX, GF_SCORE_SIGMOID = 0, 1
# fp32 partial sums the allocation-free DRELU_BGRAD entry point can hold
GF_NOALLOC_MAX_PARTIALS = 2097152


class GfError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {gf_status_string(status)}")


_lib = None
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int
_F32 = ctypes.c_float


def lib(path: str | None = None):
    """Load libgf.so (built in-tree by ``build()``); raise if it is missing."""
    global _lib
    if _lib is None:
        p = path or LIB
        if not os.path.exists(p):
            raise RuntimeError(
                f"libgf.so not found at {p}: build it with gemm_epilogue_tmem_gb300.build()")
        L = ctypes.CDLL(p)
        L.gf_matmul_plan.restype = _P
        L.gf_matmul_plan.argtypes = [_I64, _I64, _I64, _I32, _I32, _I32]
        L.gf_matmul_plan_ex.restype = _P
        L.gf_matmul_plan_ex.argtypes = [_I64, _I64, _I64, _I32, _I32, _I32, _I32]
        L.gf_matmul_execute.restype = _I32
        L.gf_matmul_execute.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _P]
        L.gf_plan_status.restype = _I32
        L.gf_plan_status.argtypes = [_P, _P]
        L.gf_plan_set_option.restype = _I32
        L.gf_plan_set_option.argtypes = [_P, _I32, _I64]
        L.gf_plan_describe.restype = _I32
        L.gf_plan_describe.argtypes = [_P, _P, _P, _P, _P, _P]
        L.gf_plan_k_splits.restype = _I32
        L.gf_plan_k_splits.argtypes = [_P, _P]
        L.gf_plan_launches.restype = _I32
        L.gf_plan_launches.argtypes = [_P, _P]
        L.gf_plan_free.restype = None
        L.gf_plan_free.argtypes = [_P]
        L.gf_status_string.restype = ctypes.c_char_p
        L.gf_status_string.argtypes = [_I32]
        L.gf_last_error.restype = _I32
        L.gf_last_error.argtypes = []
        L.gf_swiglu_plan.restype = _P
        L.gf_swiglu_plan.argtypes = [_I64, _I64, _I64, _I32, _I32]
        L.gf_swiglu_execute.restype = _I32
        L.gf_swiglu_execute.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P]
        L.gf_dswiglu_plan.restype = _P
        L.gf_dswiglu_plan.argtypes = [_I64, _I64, _I64, _I32]
        L.gf_dswiglu_execute.restype = _I32
        L.gf_dswiglu_execute.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P]
        L.gf_matmul_autotune.restype = _I32
        L.gf_matmul_autotune.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I32]
        L.gf_drelu_bgrad_noalloc.restype = _I32
        L.gf_drelu_bgrad_noalloc.argtypes = [_I64, _I64, _I64, _I32, _I32, _P, _P, _P, _P, _P, _P]
        L.gf_noalloc_status.restype = _I32
        L.gf_noalloc_status.argtypes = [_P]
        L.gf_moe_plan.restype = _P
        L.gf_moe_plan.argtypes = [_I64, _I64, _I64, _I64, _I32]
        L.gf_moe_dispatch_execute.restype = _I32
        L.gf_moe_dispatch_execute.argtypes = [_P] * 8
        L.gf_moe_dispatch_fp8_execute.restype = _I32
        L.gf_moe_dispatch_fp8_execute.argtypes = [_P] * 9
        L.gf_moe_dispatch_grad_execute.restype = _I32
        L.gf_moe_dispatch_grad_execute.argtypes = [_P] * 5
        L.gf_moe_combine_execute.restype = _I32
        L.gf_moe_combine_execute.argtypes = [_P] * 6
        L.gf_moe_combine_grad_execute.restype = _I32
        L.gf_moe_combine_grad_execute.argtypes = [_P] * 9
        L.gf_fp8_quantize.restype = _I32
        L.gf_fp8_quantize.argtypes = [_I64, _I64, _I32, _I32, _P, _P, _P, _P]
        L.gf_fp8_matmul_plan.restype = _P
        L.gf_fp8_matmul_plan.argtypes = [_I64, _I64, _I64, _I64, _I32, _I32]
        L.gf_fp8_matmul_execute.restype = _I32
        L.gf_fp8_matmul_execute.argtypes = [_P] * 11
        L.gf_matmul_residual_plan.restype = _P
        L.gf_matmul_residual_plan.argtypes = [_I64, _I64, _I64, _I32, _I32, _I32]
        L.gf_matmul_residual_execute.restype = _I32
        L.gf_matmul_residual_execute.argtypes = [_P] * 8
        L.gf_dact_bgrad_plan.restype = _P
        L.gf_dact_bgrad_plan.argtypes = [_I64, _I64, _I32, _I32]
        L.gf_dact_bgrad_execute.restype = _I32
        L.gf_dact_bgrad_execute.argtypes = [_P] * 6
        L.gf_rmsnorm_plan.restype = _P
        L.gf_rmsnorm_plan.argtypes = [_I64, _I64, _I32, _F32]
        L.gf_rmsnorm_execute.restype = _I32
        L.gf_rmsnorm_execute.argtypes = [_P] * 9
        L.gf_rmsnorm_grad_execute.restype = _I32
        L.gf_rmsnorm_grad_execute.argtypes = [_P] * 8
        L.gf_route_plan.restype = _P
        L.gf_route_plan.argtypes = [_I64, _I64, _I64, _I32, _I32, _I32, _F32, _I64, _I64, _I32, _I64]
        L.gf_route_execute.restype = _I32
        L.gf_route_execute.argtypes = [_P] * 6
        L.gf_route_grad_execute.restype = _I32
        L.gf_route_grad_execute.argtypes = [_P] * 6
        _lib = L
    return _lib


def _ptr(x) -> int | None:
    """torch tensor / int / None -> device address (or NULL)."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


_current_stream = None  # () -> the address of the current device's current stream


def _bind_current_stream():
    """torch's own getter of the raw stream where it has one (it makes no
    Stream object: 0.1 against 2.9 us a call), else the public one."""
    global _current_stream
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    device = getattr(torch._C, "_cuda_getDevice", None)
    if raw is None or device is None:
        _current_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
    else:
        torch.cuda.init()
        _current_stream = lambda: raw(device())  # noqa: E731
    return _current_stream


def _stream(stream) -> int | None:
    if stream is None:
        return (_current_stream or _bind_current_stream())()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


class Plan:
    """Owns a gf_plan* and frees it when collected (or on ``free()``)."""

    def __init__(self, handle: int, m: int, n: int, k: int, dtype: int, epilog: int,
                 bias_axis: int, b_layout: int):
        self.handle = handle
        self.m, self.n, self.k = m, n, k
        self.dtype, self.epilog, self.bias_axis, self.b_layout = dtype, epilog, bias_axis, b_layout

    def free(self) -> None:
        if self.handle:
            lib().gf_plan_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def gf_status_string(status: int) -> str:
    return lib().gf_status_string(status).decode()


def gf_last_error() -> int:
    return int(lib().gf_last_error())


def gf_matmul_plan_ex(m: int, n: int, k: int, dtype: int, epilog: int, bias_axis: int = GF_BIAS_COL,
                      b_layout: int = GF_B_KN) -> Plan:
    h = lib().gf_matmul_plan_ex(m, n, k, dtype, epilog, bias_axis, b_layout)
    if not h:
        raise GfError(gf_last_error(), "gf_matmul_plan_ex")
    return Plan(h, m, n, k, dtype, epilog, bias_axis, b_layout)


def gf_matmul_plan(m: int, n: int, k: int, dtype: int, epilog: int,
                   bias_axis: int = GF_BIAS_COL) -> Plan:
    h = lib().gf_matmul_plan(m, n, k, dtype, epilog, bias_axis)
    if not h:
        raise GfError(gf_last_error(), "gf_matmul_plan")
    return Plan(h, m, n, k, dtype, epilog, bias_axis, GF_B_KN)


def gf_matmul_execute(plan: Plan, A, B, bias=None, out=None, aux_in=None, aux_out=None,
                      bgrad=None, stream=None) -> None:
    """Enqueue the planned GEMM + epilogue; raises GfError on a non-OK status."""
    rc = lib().gf_matmul_execute(plan.handle, _ptr(A), _ptr(B), _ptr(bias), _ptr(out),
                                 _ptr(aux_in), _ptr(aux_out), _ptr(bgrad), _stream(stream))
    if rc != GF_OK:
        raise GfError(rc, "gf_matmul_execute")


def gf_matmul_autotune(plan: Plan, A, B, bias=None, out=None, aux_in=None, aux_out=None,
                       bgrad=None, stream=None, reps: int = 3) -> dict:
    """Time the library's kernel/tile/schedule candidates on these buffers,
    keep the fastest in the plan and return its description."""
    rc = lib().gf_matmul_autotune(plan.handle, _ptr(A), _ptr(B), _ptr(bias), _ptr(out),
                                  _ptr(aux_in), _ptr(aux_out), _ptr(bgrad), _stream(stream), reps)
    if rc != GF_OK:
        raise GfError(rc, "gf_matmul_autotune")
    return gf_plan_describe(plan)


def gf_swiglu_plan(m: int, n: int, k: int, dtype: int, save_gu: bool = False) -> Plan:
    """Gate+up SwiGLU forward plan: h[m, n] = silu(x Wg^T) * (x Wu^T), x [m, k]."""
    h = lib().gf_swiglu_plan(m, n, k, dtype, 1 if save_gu else 0)
    if not h:
        raise GfError(gf_last_error(), "gf_swiglu_plan")
    return Plan(h, m, n, k, dtype, -1, GF_BIAS_COL, GF_B_NK)


def gf_swiglu_execute(plan: Plan, x, Wg, Wu, h, g_out=None, u_out=None, stream=None) -> None:
    rc = lib().gf_swiglu_execute(plan.handle, _ptr(x), _ptr(Wg), _ptr(Wu), _ptr(h), _ptr(g_out),
                                 _ptr(u_out), _stream(stream))
    if rc != GF_OK:
        raise GfError(rc, "gf_swiglu_execute")


def gf_dswiglu_plan(m: int, n: int, k: int, dtype: int) -> Plan:
    """dSwiGLU backward plan: dh = dout Wd with the dSwiGLU as its epilogue."""
    h = lib().gf_dswiglu_plan(m, n, k, dtype)
    if not h:
        raise GfError(gf_last_error(), "gf_dswiglu_plan")
    return Plan(h, m, n, k, dtype, -2, GF_BIAS_COL, GF_B_KN)


def gf_dswiglu_execute(plan: Plan, dout, Wd, g, u, d_gate, d_up, stream=None) -> None:
    rc = lib().gf_dswiglu_execute(plan.handle, _ptr(dout), _ptr(Wd), _ptr(g), _ptr(u),
                                  _ptr(d_gate), _ptr(d_up), _stream(stream))
    if rc != GF_OK:
        raise GfError(rc, "gf_dswiglu_execute")


def gf_plan_status(plan: Plan, stream=None) -> int:
    """Synchronise the stream and return the plan's status (GF_OK, GF_ERR_DEVICE_TIMEOUT ...)."""
    return int(lib().gf_plan_status(plan.handle, _stream(stream)))


def gf_plan_set_option(plan: Plan, option: int, value: int) -> None:
    rc = lib().gf_plan_set_option(plan.handle, option, value)
    if rc != GF_OK:
        raise GfError(rc, "gf_plan_set_option")


def gf_plan_describe(plan: Plan) -> dict:
    vals = [ctypes.c_int32() for _ in range(4)]
    ws = ctypes.c_int64()
    rc = lib().gf_plan_describe(plan.handle, *(ctypes.byref(v) for v in vals), ctypes.byref(ws))
    if rc != GF_OK:
        raise GfError(rc, "gf_plan_describe")
    ks = ctypes.c_int32()
    rc = lib().gf_plan_k_splits(plan.handle, ctypes.byref(ks))
    if rc != GF_OK:
        raise GfError(rc, "gf_plan_k_splits")
    nl = ctypes.c_int32()
    rc = lib().gf_plan_launches(plan.handle, ctypes.byref(nl))
    if rc != GF_OK:
        raise GfError(rc, "gf_plan_launches")
    return {"tile_m": vals[0].value, "tile_n": vals[1].value, "stages": vals[2].value,
            "grid": vals[3].value, "workspace_bytes": ws.value, "k_splits": ks.value,
            "launches": nl.value}


def gf_plan_free(plan: Plan) -> None:
    plan.free()


def gf_drelu_bgrad_noalloc(m: int, n: int, k: int, dtype: int, b_layout: int, A, B, out, aux_in,
                           bgrad, stream=None) -> None:
    """DRELU_BGRAD without any device allocation (fixed scratch inside the
    library; see include/gf.h). Raises GfError on a non-OK status."""
    rc = lib().gf_drelu_bgrad_noalloc(m, n, k, dtype, b_layout, _ptr(A), _ptr(B), _ptr(out),
                                      _ptr(aux_in), _ptr(bgrad), _stream(stream))
    if rc != GF_OK:
        raise GfError(rc, "gf_drelu_bgrad_noalloc")


def gf_noalloc_status(stream=None) -> int:
    """Synchronise the stream and return the status of the most recent
    gf_drelu_bgrad_noalloc on this device (GF_OK, GF_ERR_DEVICE_TIMEOUT ...)."""
    return int(lib().gf_noalloc_status(_stream(stream)))


# ------------------------------------------------------- expert routing, e4m3
# Tensors of the calls below are checked against the plan: element size and
# kind, number of elements, contiguous, on a GPU. Raw addresses are not.
_I32_KIND, _F32_KIND, _E4M3_KIND = "i32", "f32", "e4m3"
_TENSOR_KINDS = {
    _I32_KIND: ("torch.int32",), _F32_KIND: ("torch.float32",),
    _E4M3_KIND: ("torch.float8_e4m3fn", "torch.uint8"),
    GF_F16: ("torch.float16",), GF_BF16: ("torch.bfloat16",), GF_F32: ("torch.float32",),
}
_kinds = {}  # kind -> its torch dtypes


def _arg(x, kind, count: int, what: str) -> int | None:
    """Device address of x, a tensor of `count` elements of `kind` (or an address, or None)."""
    if x is None or type(x) is int:
        return x
    try:
        if x.dtype in _kinds[kind] and x.numel() == count and x.is_cuda and x.is_contiguous():
            return x.data_ptr()
    except KeyError:  # the first tensor
        import torch
        _kinds.update({k: tuple(getattr(torch, n.split(".")[1]) for n in v)
                       for k, v in _TENSOR_KINDS.items()})
        return _arg(x, kind, count, what)
    raise GfError(GF_ERR_INVALID_VALUE,
                  f"{what}: a contiguous CUDA tensor of {count} elements of "
                  f"{' or '.join(_TENSOR_KINDS[kind])} is needed, not {x.dtype} {tuple(x.shape)}")


def _check(rc: int, what: str) -> None:
    if rc != GF_OK:
        raise GfError(rc, what)


def gf_moe_plan(tokens: int, topk: int, experts: int, hidden: int, dtype: int) -> Plan:
    """Expert-routing plan: `tokens` rows of `hidden` elements, `topk` of `experts` each."""
    h = lib().gf_moe_plan(tokens, topk, experts, hidden, dtype)
    if not h:
        raise GfError(gf_last_error(), "gf_moe_plan")
    plan = Plan(h, tokens, experts, hidden, dtype, -3, GF_BIAS_COL, GF_B_KN)
    plan.topk, plan.slots = topk, tokens * topk
    return plan


def _moe(plan: Plan, what: str) -> None:
    if not hasattr(plan, "slots"):
        raise GfError(GF_ERR_INVALID_VALUE, f"{what}: not a plan of gf_moe_plan")


def gf_moe_dispatch_execute(plan: Plan, expert, x, offsets, row_of, slot_of, rows,
                            stream=None) -> None:
    """Sort the slots by expert and copy the tokens' rows to their places
    (x and rows None: the sort alone); see include/gf.h."""
    what = "gf_moe_dispatch_execute"
    _moe(plan, what)
    _check(lib().gf_moe_dispatch_execute(
        plan.handle, _arg(expert, _I32_KIND, plan.slots, what), _arg(x, plan.dtype, plan.m * plan.k, what),
        _arg(offsets, _I32_KIND, plan.n + 1, what), _arg(row_of, _I32_KIND, plan.slots, what),
        _arg(slot_of, _I32_KIND, plan.slots, what), _arg(rows, plan.dtype, plan.slots * plan.k, what),
        _stream(stream)), what)


def gf_moe_dispatch_fp8_execute(plan: Plan, expert, x, offsets, row_of, slot_of, rows, scale,
                                stream=None) -> None:
    """Dispatch with rows quantised to e4m3, one fp32 scale per 128 elements."""
    what = "gf_moe_dispatch_fp8_execute"
    _moe(plan, what)
    _check(lib().gf_moe_dispatch_fp8_execute(
        plan.handle, _arg(expert, _I32_KIND, plan.slots, what), _arg(x, plan.dtype, plan.m * plan.k, what),
        _arg(offsets, _I32_KIND, plan.n + 1, what), _arg(row_of, _I32_KIND, plan.slots, what),
        _arg(slot_of, _I32_KIND, plan.slots, what), _arg(rows, _E4M3_KIND, plan.slots * plan.k, what),
        _arg(scale, _F32_KIND, plan.slots * -(-plan.k // 128), what), _stream(stream)), what)


def gf_moe_dispatch_grad_execute(plan: Plan, row_of, d_rows, d_x, stream=None) -> None:
    """d_x[t] = sum of its slots' d_rows."""
    what = "gf_moe_dispatch_grad_execute"
    _moe(plan, what)
    _check(lib().gf_moe_dispatch_grad_execute(
        plan.handle, _arg(row_of, _I32_KIND, plan.slots, what),
        _arg(d_rows, plan.dtype, plan.slots * plan.k, what),
        _arg(d_x, plan.dtype, plan.m * plan.k, what), _stream(stream)), what)


def gf_moe_combine_execute(plan: Plan, row_of, weight, rows, out, stream=None) -> None:
    """out[t] = sum of its slots' rows, weighted."""
    what = "gf_moe_combine_execute"
    _moe(plan, what)
    _check(lib().gf_moe_combine_execute(
        plan.handle, _arg(row_of, _I32_KIND, plan.slots, what), _arg(weight, _F32_KIND, plan.slots, what),
        _arg(rows, plan.dtype, plan.slots * plan.k, what),
        _arg(out, plan.dtype, plan.m * plan.k, what), _stream(stream)), what)


def gf_moe_combine_grad_execute(plan: Plan, offsets, row_of, weight, rows, d_out, d_rows, d_weight,
                                stream=None) -> None:
    """Gradients of combine: d_rows and d_weight."""
    what = "gf_moe_combine_grad_execute"
    _moe(plan, what)
    _check(lib().gf_moe_combine_grad_execute(
        plan.handle, _arg(offsets, _I32_KIND, plan.n + 1, what), _arg(row_of, _I32_KIND, plan.slots, what),
        _arg(weight, _F32_KIND, plan.slots, what), _arg(rows, plan.dtype, plan.slots * plan.k, what),
        _arg(d_out, plan.dtype, plan.m * plan.k, what),
        _arg(d_rows, plan.dtype, plan.slots * plan.k, what),
        _arg(d_weight, _F32_KIND, plan.slots, what), _stream(stream)), what)


def gf_fp8_quantize(m: int, k: int, dtype: int, block_rows: int, x, q, scale, stream=None) -> None:
    """e4m3 values and one power-of-two scale per block of block_rows x 128."""
    what = "gf_fp8_quantize"
    if dtype not in (GF_F16, GF_BF16) or block_rows < 1:
        raise GfError(GF_ERR_INVALID_VALUE, what)
    blocks = -(-m // block_rows) * -(-k // 128)
    _check(lib().gf_fp8_quantize(m, k, dtype, block_rows, _arg(x, dtype, m * k, what),
                                 _arg(q, _E4M3_KIND, m * k, what), _arg(scale, _F32_KIND, blocks, what),
                                 _stream(stream)), what)


def gf_fp8_matmul_plan(m: int, n: int, k: int, groups: int, dtype: int,
                       epilog: int = GF_FP8_EPILOG_NONE) -> Plan:
    """Block-scaled e4m3 product plan: m rows in `groups` groups, each with a B [n, k] of its own."""
    h = lib().gf_fp8_matmul_plan(m, n, k, groups, dtype, epilog)
    if not h:
        raise GfError(gf_last_error(), "gf_fp8_matmul_plan")
    plan = Plan(h, m, n, k, dtype, -4, GF_BIAS_COL, GF_B_NK)
    plan.groups, plan.quant = groups, epilog == GF_FP8_EPILOG_SWIGLU_QUANT
    plan.kb, plan.nb = -(-k // 128), -(-n // 128)
    return plan


def gf_fp8_matmul_execute(plan: Plan, A, a_scale, B, b_scale, B2=None, b2_scale=None, offsets=None,
                          out=None, out_scale=None, stream=None) -> None:
    """Enqueue the planned product; B2 and out_scale for GF_FP8_EPILOG_SWIGLU_QUANT."""
    what = "gf_fp8_matmul_execute"
    if not hasattr(plan, "groups"):
        raise GfError(GF_ERR_INVALID_VALUE, f"{what}: not a plan of gf_fp8_matmul_plan")
    m, n, k, groups = plan.m, plan.n, plan.k, plan.groups
    scales = groups * plan.nb * plan.kb
    _check(lib().gf_fp8_matmul_execute(
        plan.handle, _arg(A, _E4M3_KIND, m * k, what), _arg(a_scale, _F32_KIND, m * plan.kb, what),
        _arg(B, _E4M3_KIND, groups * n * k, what), _arg(b_scale, _F32_KIND, scales, what),
        _arg(B2, _E4M3_KIND, groups * n * k, what), _arg(b2_scale, _F32_KIND, scales, what),
        _arg(offsets, _I32_KIND, groups + 1, what),
        _arg(out, _E4M3_KIND if plan.quant else plan.dtype, m * n, what),
        _arg(out_scale, _F32_KIND, m * plan.nb, what), _stream(stream)), what)


# ------------------------------------------- a block's norm, router, residual
def _of(plan: Plan, kind: str, what: str) -> None:
    if getattr(plan, "block", None) != kind:
        raise GfError(GF_ERR_INVALID_VALUE, f"{what}: not a plan of gf_{kind}_plan")


def _block_plan(handle, kind: str, m: int, n: int, k: int, dtype: int) -> Plan:
    if not handle:
        raise GfError(gf_last_error(), f"gf_{kind}_plan")
    plan = Plan(handle, m, n, k, dtype, -5, GF_BIAS_COL, GF_B_KN)
    plan.block = kind
    return plan


def gf_matmul_residual_plan(m: int, n: int, k: int, dtype: int, act: int = GF_ACT_NONE,
                            b_layout: int = GF_B_KN) -> Plan:
    """out = act(A B + bias) + residual plan."""
    plan = _block_plan(lib().gf_matmul_residual_plan(m, n, k, dtype, act, b_layout),
                       "matmul_residual", m, n, k, dtype)
    plan.b_layout = b_layout
    return plan


def gf_matmul_residual_execute(plan: Plan, A, B, residual, out, bias=None, z_out=None,
                               stream=None) -> None:
    """out = act(A B + bias) + residual; z_out keeps what the activation takes."""
    what = "gf_matmul_residual_execute"
    _of(plan, "matmul_residual", what)
    m, n, k, dtype = plan.m, plan.n, plan.k, plan.dtype
    _check(lib().gf_matmul_residual_execute(
        plan.handle, _arg(A, dtype, m * k, what), _arg(B, dtype, n * k, what),
        _arg(bias, dtype, n, what), _arg(residual, dtype, m * n, what),
        _arg(out, dtype, m * n, what), _arg(z_out, dtype, m * n, what), _stream(stream)), what)


def gf_dact_bgrad_plan(m: int, n: int, dtype: int, act: int) -> Plan:
    """Plan of the gradients of an activation's argument and of the bias in it."""
    return _block_plan(lib().gf_dact_bgrad_plan(m, n, dtype, act), "dact_bgrad", m, n, 0, dtype)


def gf_dact_bgrad_execute(plan: Plan, d_out, z=None, d_z=None, bgrad=None, stream=None) -> None:
    """d_z = d_out * act'(z) and bgrad, its column sums (GF_ACT_NONE: bgrad alone)."""
    what = "gf_dact_bgrad_execute"
    _of(plan, "dact_bgrad", what)
    count, dtype = plan.m * plan.n, plan.dtype
    _check(lib().gf_dact_bgrad_execute(
        plan.handle, _arg(d_out, dtype, count, what), _arg(z, dtype, count, what),
        _arg(d_z, dtype, count, what), _arg(bgrad, _F32_KIND, plan.n, what), _stream(stream)), what)


def gf_rmsnorm_plan(rows: int, hidden: int, dtype: int, eps: float = 1e-6) -> Plan:
    """Root-mean-square norm plan: `rows` rows of `hidden` elements."""
    return _block_plan(lib().gf_rmsnorm_plan(rows, hidden, dtype, eps), "rmsnorm", rows, hidden,
                       hidden, dtype)


def gf_rmsnorm_execute(plan: Plan, x, weight, residual=None, residual_out=None, out=None, out8=None,
                       out_scale=None, stream=None) -> None:
    """r = x + residual, and its norm in 16 bits (out) and / or e4m3 (out8, out_scale)."""
    what = "gf_rmsnorm_execute"
    _of(plan, "rmsnorm", what)
    count, dtype = plan.m * plan.n, plan.dtype
    _check(lib().gf_rmsnorm_execute(
        plan.handle, _arg(x, dtype, count, what), _arg(residual, dtype, count, what),
        _arg(weight, dtype, plan.n, what), _arg(residual_out, dtype, count, what),
        _arg(out, dtype, count, what), _arg(out8, _E4M3_KIND, count, what),
        _arg(out_scale, _F32_KIND, plan.m * -(-plan.n // 128), what), _stream(stream)), what)


def gf_rmsnorm_grad_execute(plan: Plan, d_out, r, weight, d_x, d_weight=None, d_residual=None,
                            stream=None) -> None:
    """Gradients of the norm: d_x (of x and of the residual) and d_weight."""
    what = "gf_rmsnorm_grad_execute"
    _of(plan, "rmsnorm", what)
    count, dtype = plan.m * plan.n, plan.dtype
    _check(lib().gf_rmsnorm_grad_execute(
        plan.handle, _arg(d_out, dtype, count, what), _arg(r, dtype, count, what),
        _arg(weight, dtype, plan.n, what), _arg(d_residual, dtype, count, what),
        _arg(d_x, dtype, count, what), _arg(d_weight, _F32_KIND, plan.n, what), _stream(stream)), what)


def gf_route_plan(tokens: int, experts: int, topk: int, dtype: int, score: int = GF_SCORE_SOFTMAX,
                  renorm: bool = True, scale: float = 1.0, groups: int = 1, topk_groups: int = 1,
                  group_best: int = 2, ld: int | None = None) -> Plan:
    """Router plan: `topk` of `experts` for each token, from logits with rows `ld` elements apart."""
    ld = experts if ld is None else ld
    plan = _block_plan(lib().gf_route_plan(tokens, experts, topk, dtype, score, 1 if renorm else 0,
                                           scale, groups, topk_groups, group_best, ld),
                       "route", tokens, experts, topk, dtype)
    plan.ld, plan.choices = ld, tokens * topk
    return plan


def gf_route_execute(plan: Plan, logits, expert, weight, bias=None, stream=None) -> None:
    """The tokens' experts and weights; the bias takes part in the choice alone."""
    what = "gf_route_execute"
    _of(plan, "route", what)
    _check(lib().gf_route_execute(
        plan.handle, _arg(logits, plan.dtype, plan.m * plan.ld, what), _arg(bias, _F32_KIND, plan.n, what),
        _arg(expert, _I32_KIND, plan.choices, what), _arg(weight, _F32_KIND, plan.choices, what),
        _stream(stream)), what)


def gf_route_grad_execute(plan: Plan, logits, expert, d_weight, d_logits, stream=None) -> None:
    """The gradient of the logits from that of the weights."""
    what = "gf_route_grad_execute"
    _of(plan, "route", what)
    _check(lib().gf_route_grad_execute(
        plan.handle, _arg(logits, plan.dtype, plan.m * plan.ld, what),
        _arg(expert, _I32_KIND, plan.choices, what), _arg(d_weight, _F32_KIND, plan.choices, what),
        _arg(d_logits, plan.dtype, plan.m * plan.ld, what), _stream(stream)), what)
