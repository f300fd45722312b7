"""Thin ctypes binding of the C ABI in include/moe.h.

Argument marshalling only: every step of the layer runs in the CUDA library
``libqeffn.so`` (built in-tree by ``build.py``).  Functions keep the C names;
device buffers are passed as torch CUDA tensors (or raw integer addresses),
streams as torch streams (or raw handles).  A non-zero status raises
``MoeError``.  There is no fallback: if the library is missing, importing
this module fails.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libqeffn.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = -1
MOE_ERR_OOM = -2
MOE_ERR_CUDA = -3
MOE_ERR_NOT_LOADED = -4
MOE_ERR_TOO_MANY_TOKENS = -5
MOE_ERR_DEVICE_TIMEOUT = -6
MOE_ERR_UNSUPPORTED = -7
MOE_Q4B32 = 1
MOE_Q3B32 = 2
MOE_Q2B32 = 3
MOE_FLAG_NO_DECODE_KERNEL = 1
MOE_FLAG_NO_TENSOR_PREFILL = 2
MOE_FLAG_NO_MULTI_DECODE = 8
MOE_FLAG_SPLIT_DECODE = 16
MOE_FLAG_TEST_WITHHOLD = 256
MOE_FLAG_TRACE = 4
MOE_L2_STREAM = 0
MOE_L2_KEEP_SHARED = 1
MOE_ROUTE_STATIC_MAX_LOGITS = 65536
MOE_BF16 = 1
MOE_FP16 = 2
MOE_FP32 = 3
MOE_ACT_SILU = 1
MOE_ACT_GELU_TANH = 2
MOE_ACT_GELU = 3
MOE_FFN_GRAD_FP32 = 1
MOE_FFN_GRAD_ADD = 2
ACTS = {"silu": MOE_ACT_SILU, "gelu_tanh": MOE_ACT_GELU_TANH, "gelu": MOE_ACT_GELU}
FORMATS = {"q4": MOE_Q4B32, "q3": MOE_Q3B32, "q2": MOE_Q2B32}

EXPORTED = [
    "moe_create", "moe_load_layer", "moe_forward", "moe_forward_stack",
    "moe_forward_stack_host", "moe_destroy", "moe_get_device_error",
    "moe_status_string", "moe_last_error", "moe_timing_enable", "moe_timing_read",
    "moe_trace_read", "moe_route_static", "moe_set_l2_policy",
    "moe_ffn_workspace", "moe_ffn_forward", "moe_ffn_backward", "moe_quantize_s8",
    "moe_matmul_s8_workspace", "moe_matmul_s8", "moe_ffn_s8_workspace", "moe_ffn_s8_forward",
    "moe_ffn_get_device_error",
]


class moe_config(ctypes.Structure):
    _fields_ = [("d_model", ctypes.c_int), ("n_experts", ctypes.c_int), ("d_ff", ctypes.c_int),
                ("top_k", ctypes.c_int), ("n_shared", ctypes.c_int), ("d_ff_shared", ctypes.c_int),
                ("n_layers", ctypes.c_int), ("max_tokens", ctypes.c_int), ("fmt", ctypes.c_int),
                ("device_mem_limit", ctypes.c_longlong), ("flags", ctypes.c_int)]


class moe_layer_weights(ctypes.Structure):
    _fields_ = [("router_w", ctypes.c_void_p), ("router_bias", ctypes.c_void_p),
                ("codes", ctypes.c_void_p * 3), ("scales", ctypes.c_void_p * 3),
                ("sh_codes", ctypes.c_void_p * 3), ("sh_scales", ctypes.c_void_p * 3),
                ("on_device", ctypes.c_int)]


class moe_stack_record(ctypes.Structure):
    _fields_ = [("x_bf16", ctypes.c_void_p), ("y_bf16", ctypes.c_void_p), ("y_f32", ctypes.c_void_p),
                ("ids", ctypes.c_void_p), ("w", ctypes.c_void_p), ("rows", ctypes.c_void_p),
                ("n_rows", ctypes.c_int)]


class moe_ffn(ctypes.Structure):
    _fields_ = [("d_model", ctypes.c_int), ("d_ff", ctypes.c_int), ("dtype", ctypes.c_int), ("act", ctypes.c_int),
                ("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p)]


class moe_ffn_s8(ctypes.Structure):
    _fields_ = [("d_model", ctypes.c_int), ("d_ff", ctypes.c_int), ("dtype", ctypes.c_int), ("act", ctypes.c_int),
                ("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p),
                ("s_gate", ctypes.c_void_p), ("s_up", ctypes.c_void_p), ("s_down", ctypes.c_void_p)]


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status}) {last_error()}")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python quantized_expert_ffn_token_b200/build.py`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i = ctypes.c_void_p, ctypes.c_int
    L.moe_create.argtypes = [ctypes.POINTER(moe_config), i, ctypes.POINTER(vp)]
    L.moe_load_layer.argtypes = [vp, i, ctypes.POINTER(moe_layer_weights), vp]
    L.moe_forward.argtypes = [vp, i, vp, i, vp, vp, vp, vp, vp]
    L.moe_forward_stack.argtypes = [vp, i, i, vp, i, vp, ctypes.POINTER(moe_stack_record), vp]
    L.moe_forward_stack_host.argtypes = [vp, i, i, vp, i, vp, vp]
    L.moe_destroy.argtypes = [vp]
    L.moe_get_device_error.argtypes = [vp, ctypes.POINTER(i)]
    L.moe_timing_enable.argtypes = [vp, i]
    L.moe_set_l2_policy.argtypes = [vp, i]
    L.moe_timing_read.argtypes = [vp, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_longlong),
                                  ctypes.POINTER(ctypes.c_longlong), ctypes.c_char_p, i]
    L.moe_trace_read.argtypes = [vp, ctypes.POINTER(ctypes.c_ulonglong), i, ctypes.POINTER(i)]
    L.moe_route_static.argtypes = [vp, i, i, vp, vp, i, i, vp, vp, vp]
    ll, pll = ctypes.c_longlong, ctypes.POINTER(ctypes.c_longlong)
    pf, p8 = ctypes.POINTER(moe_ffn), ctypes.POINTER(moe_ffn_s8)
    L.moe_ffn_workspace.argtypes = [pf, i, i, pll]
    L.moe_ffn_forward.argtypes = [pf, vp, ll, i, vp, ll, vp, vp, vp, ll, vp]
    L.moe_ffn_backward.argtypes = [pf, vp, ll, vp, vp, vp, ll, i, vp, ll, vp, vp, vp, i, vp, ll, vp]
    L.moe_quantize_s8.argtypes = [vp, i, ll, i, i, vp, vp, vp]
    L.moe_matmul_s8_workspace.argtypes = [i, i, i, pll]
    L.moe_matmul_s8.argtypes = [vp, vp, i, vp, vp, i, i, vp, vp, i, ll, vp, ll, vp]
    L.moe_ffn_s8_workspace.argtypes = [p8, i, pll]
    L.moe_ffn_s8_forward.argtypes = [p8, vp, ll, i, vp, ll, vp, ll, vp]
    L.moe_ffn_get_device_error.argtypes = [ctypes.POINTER(i)]
    L.moe_status_string.argtypes = [i]
    L.moe_status_string.restype = ctypes.c_char_p
    L.moe_last_error.argtypes = []
    L.moe_last_error.restype = ctypes.c_char_p
    for n in ("moe_create", "moe_load_layer", "moe_forward", "moe_forward_stack",
              "moe_forward_stack_host", "moe_destroy", "moe_get_device_error",
              "moe_timing_enable", "moe_timing_read", "moe_trace_read", "moe_route_static",
              "moe_set_l2_policy", "moe_ffn_workspace", "moe_ffn_forward", "moe_ffn_backward", "moe_quantize_s8",
              "moe_matmul_s8_workspace", "moe_matmul_s8", "moe_ffn_s8_workspace", "moe_ffn_s8_forward",
              "moe_ffn_get_device_error"):
        getattr(L, n).restype = i
    return L


lib = _load()


def _ptr(t) -> int | None:
    """Address of a tensor's data (None for None); ints pass through."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _stream(s) -> int | None:
    if s is None:
        return None
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(status: int, what: str) -> None:
    if status != MOE_OK:
        raise MoeError(status, what)


def status_string(status: int) -> str:
    return lib.moe_status_string(status).decode()


def last_error() -> str:
    return lib.moe_last_error().decode()


def moe_create(cfg: moe_config, device: int = 0) -> ctypes.c_void_p:
    h = ctypes.c_void_p()
    _check(lib.moe_create(ctypes.byref(cfg), device, ctypes.byref(h)), "moe_create")
    return h


def moe_load_layer(ctx, layer: int, w: moe_layer_weights, stream=None) -> None:
    _check(lib.moe_load_layer(ctx, layer, ctypes.byref(w), _stream(stream)), "moe_load_layer")


def moe_forward(ctx, layer: int, x, T: int, y, y_f32=None, ids=None, w=None, stream=None) -> None:
    _check(lib.moe_forward(ctx, layer, _ptr(x), T, _ptr(y), _ptr(y_f32), _ptr(ids), _ptr(w),
                           _stream(stream)), "moe_forward")


def moe_forward_stack(ctx, layer0: int, n_layers: int, x, T: int, resid_out, rec=None,
                      stream=None) -> None:
    _check(lib.moe_forward_stack(ctx, layer0, n_layers, _ptr(x), T, _ptr(resid_out),
                                 ctypes.byref(rec) if rec is not None else None, _stream(stream)),
           "moe_forward_stack")


def moe_forward_stack_host(ctx, layer0: int, n_layers: int, x_host, T: int, resid_host,
                           stream=None) -> None:
    _check(lib.moe_forward_stack_host(ctx, layer0, n_layers, _ptr(x_host), T, _ptr(resid_host),
                                      _stream(stream)), "moe_forward_stack_host")


def moe_destroy(ctx) -> None:
    _check(lib.moe_destroy(ctx), "moe_destroy")


def moe_set_l2_policy(ctx, mode: int) -> None:
    """L2 eviction priorities of the decode kernels' weight copies (see include/moe.h)."""
    _check(lib.moe_set_l2_policy(ctx, mode), "moe_set_l2_policy")


def moe_get_device_error(ctx) -> int:
    code = ctypes.c_int(0)
    _check(lib.moe_get_device_error(ctx, ctypes.byref(code)), "moe_get_device_error")
    return code.value


def moe_timing_enable(ctx, on: bool = True) -> None:
    _check(lib.moe_timing_enable(ctx, 1 if on else 0), "moe_timing_enable")


def moe_timing_read(ctx) -> dict:
    ms = ctypes.c_double()
    timed = ctypes.c_longlong()
    allk = ctypes.c_longlong()
    name = ctypes.create_string_buffer(128)
    _check(lib.moe_timing_read(ctx, ctypes.byref(ms), ctypes.byref(timed), ctypes.byref(allk), name, 128),
           "moe_timing_read")
    return {"ms": ms.value, "timed_launches": timed.value, "all_launches": allk.value,
            "kernel": name.value.decode()}


def moe_trace_read(ctx, n_max: int = 1 << 16):
    """Phase trace records as a list of 24-tuples (see include/moe.h)."""
    buf = (ctypes.c_ulonglong * (24 * n_max))()
    n = ctypes.c_int(0)
    _check(lib.moe_trace_read(ctx, buf, n_max, ctypes.byref(n)), "moe_trace_read")
    return [tuple(buf[24 * i:24 * i + 24]) for i in range(n.value)]


def moe_route_static(x, T: int, d_model: int, router_w, router_bias, n_experts: int, top_k: int,
                     ids, w, stream=None) -> None:
    """Allocation-free routing (see include/moe.h): device buffers in, ids/w out."""
    _check(lib.moe_route_static(_ptr(x), T, d_model, _ptr(router_w), _ptr(router_bias), n_experts,
                                top_k, _ptr(ids), _ptr(w), _stream(stream)), "moe_route_static")


def make_record(x=None, y=None, y_f32=None, ids=None, w=None, rows=None) -> moe_stack_record:
    r = moe_stack_record()
    r.x_bf16, r.y_bf16, r.y_f32 = _ptr(x), _ptr(y), _ptr(y_f32)
    r.ids, r.w = _ptr(ids), _ptr(w)
    r.rows = _ptr(rows)
    r.n_rows = 0 if rows is None else int(rows.numel())
    return r


# ---- dense feed-forward (see include/moe.h) ---------------------------------------------------------------------
# Tensors carry their sizes here: activations are 2-d CUDA tensors whose rows may lie apart (a slice of a wider
# buffer); everything else is contiguous.  Shapes and types are checked before an address leaves Python.

class _TorchTypes:
    """torch's types, looked up when a tensor first comes: the binding itself needs no torch."""

    def __getattr__(self, name):      # called until the attributes are there
        import torch
        self.int8, self.float32 = torch.int8, torch.float32
        self.dtypes = {torch.bfloat16: MOE_BF16, torch.float16: MOE_FP16, torch.float32: MOE_FP32}
        return object.__getattribute__(self, name)


_types = _TorchTypes()


def __getattr__(name):
    if name == "DTYPES":              # moe_dtype of a torch dtype
        return _types.dtypes
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")


def _int(n: int) -> int:
    """n as a C int.  ctypes takes a size modulo 2^32; past its range it becomes the nearest C int, which is
    outside every call's limits."""
    return n if -0x80000000 <= n <= 0x7FFFFFFF else 0x7FFFFFFF if n > 0 else -0x80000000


def _dtype(t) -> int:
    try:
        return _types.dtypes[t.dtype]
    except KeyError:
        raise ValueError(f"dtype {t.dtype}: bf16, fp16 or fp32 expected") from None


def _rows(t, T: int, cols: int, dtype, what: str):
    """(address, row distance) of the first T rows of a [>= T][cols] CUDA tensor of the given torch dtype."""
    shape = t.shape
    if len(shape) != 2 or shape[1] != cols or shape[0] < T or t.dtype is not dtype or not t.is_cuda:
        raise ValueError(f"{what}: a CUDA tensor [{T}, {cols}] of {dtype} expected")
    if t.is_contiguous():
        return t.data_ptr(), 0
    ld, inner = t.stride()
    if cols > 1 and inner != 1:
        raise ValueError(f"{what}: elements of a row must be contiguous")
    if T <= 1:
        return t.data_ptr(), 0
    if ld < cols:
        raise ValueError(f"{what}: rows overlap")
    return t.data_ptr(), ld


def _full(t, shape, dtype, what: str):
    """Address of a contiguous CUDA tensor of this shape and torch dtype."""
    if t.dtype is dtype and t.is_cuda and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{what}: a contiguous CUDA tensor {list(shape)} of {dtype} expected")


def _space(ws):
    if ws is None:
        return None, 0
    if ws.is_cuda and ws.is_contiguous():
        return ws.data_ptr(), ws.numel() * ws.element_size()
    raise ValueError("workspace: a contiguous CUDA tensor expected")


def _act(act) -> int:
    return ACTS[act] if isinstance(act, str) else int(act)


def make_ffn(w_gate, w_up, w_down, act="silu") -> moe_ffn:
    """The block over its weights [d_ff, d_model], [d_ff, d_model], [d_model, d_ff] (kept alive by the result)."""
    I, d = w_gate.shape
    f = moe_ffn()
    f.d_model, f.d_ff, f.dtype, f.act = _int(d), _int(I), _dtype(w_gate), _act(act)
    f.torch_dtype = w_gate.dtype
    f.w_gate = _full(w_gate, (I, d), f.torch_dtype, "w_gate")
    f.w_up = _full(w_up, (I, d), f.torch_dtype, "w_up")
    f.w_down = _full(w_down, (d, I), f.torch_dtype, "w_down")
    f.keep = (w_gate, w_up, w_down)
    return f


def moe_ffn_workspace(f: moe_ffn, T: int, backward: bool = False) -> int:
    n = ctypes.c_longlong()
    _check(lib.moe_ffn_workspace(f, _int(T), 1 if backward else 0, ctypes.byref(n)), "moe_ffn_workspace")
    return n.value


def moe_ffn_forward(f: moe_ffn, x, T: int, y, gate=None, up=None, workspace=None, stream=None) -> None:
    dt, d, I = f.torch_dtype, f.d_model, f.d_ff
    xp, lx = _rows(x, T, d, dt, "x")
    yp, ly = _rows(y, T, d, dt, "y")
    gp = None if gate is None else _full(gate, (T, I), dt, "gate")
    up_ = None if up is None else _full(up, (T, I), dt, "up")
    wp, wn = _space(workspace)
    _check(lib.moe_ffn_forward(f, xp, lx, _int(T), yp, ly, gp, up_, wp, wn, _stream(stream)),
           "moe_ffn_forward")


def moe_ffn_backward(f: moe_ffn, x, gate, up, dy, T: int, dx=None, dw_gate=None, dw_up=None, dw_down=None,
                     add: bool = False, workspace=None, stream=None) -> None:
    """Gradients of the block; fp32 weight-gradient tensors select fp32 sums, ``add`` adds to what they hold."""
    dt, d, I = f.torch_dtype, f.d_model, f.d_ff
    xp, lx = (None, 0) if x is None else _rows(x, T, d, dt, "x")
    dyp, ldy = _rows(dy, T, d, dt, "dy")
    dxp, ldx = (None, 0) if dx is None else _rows(dx, T, d, dt, "dx")
    gp, up_ = _full(gate, (T, I), dt, "gate"), _full(up, (T, I), dt, "up")
    flags = MOE_FFN_GRAD_ADD if add else 0
    wdt = dt
    if dw_gate is not None and _dtype(dw_gate) == MOE_FP32:
        flags |= MOE_FFN_GRAD_FP32
        wdt = dw_gate.dtype
    dg = None if dw_gate is None else _full(dw_gate, (I, d), wdt, "dw_gate")
    du = None if dw_up is None else _full(dw_up, (I, d), wdt, "dw_up")
    dd = None if dw_down is None else _full(dw_down, (d, I), wdt, "dw_down")
    wp, wn = _space(workspace)
    _check(lib.moe_ffn_backward(f, xp, lx, gp, up_, dyp, ldy, _int(T), dxp, ldx, dg, du, dd, flags, wp, wn,
                                _stream(stream)), "moe_ffn_backward")


def _codes(t, shape, what: str):
    return _full(t, shape, _types.int8, what)


def _scales(t, n: int, what: str):
    return _full(t, (n,), _types.float32, what)


def moe_quantize_s8(x, q, scale, stream=None) -> None:
    """Rows of x (bf16, fp16, fp32) as 8-bit codes q [rows, cols] and scales [rows]."""
    rows, cols = x.shape
    xp, lx = _rows(x, rows, cols, x.dtype, "x")
    _check(lib.moe_quantize_s8(xp, _dtype(x), lx, _int(rows), _int(cols), _codes(q, (rows, cols), "q"),
                               _scales(scale, rows, "scale"), _stream(stream)), "moe_quantize_s8")


def moe_matmul_s8_workspace(T: int, N: int, K: int) -> int:
    n = ctypes.c_longlong()
    _check(lib.moe_matmul_s8_workspace(_int(T), _int(N), _int(K), ctypes.byref(n)), "moe_matmul_s8_workspace")
    return n.value


def moe_matmul_s8(a, a_scale, w, w_scale, y, bias=None, workspace=None, stream=None) -> None:
    """y [T, N] = scaled product of 8-bit a [T, K] and w [N, K], plus bias [N]."""
    T, K = a.shape
    N = w.shape[0]
    yp, ly = _rows(y, T, N, y.dtype, "y")
    wp, wn = _space(workspace)
    _check(lib.moe_matmul_s8(_codes(a, (T, K), "a"), _scales(a_scale, T, "a_scale"), _int(T), _codes(w, (N, K), "w"),
                             _scales(w_scale, N, "w_scale"), _int(N), _int(K),
                             None if bias is None else _scales(bias, N, "bias"),
                             yp, _dtype(y), ly, wp, wn, _stream(stream)), "moe_matmul_s8")


def make_ffn_s8(w_gate, s_gate, w_up, s_up, w_down, s_down, act="silu", dtype=None) -> moe_ffn_s8:
    """The block over 8-bit weights and their row scales; ``dtype``: torch.bfloat16 or torch.float16 of x and y."""
    I, d = w_gate.shape
    f = moe_ffn_s8()
    f.d_model, f.d_ff, f.dtype, f.act = _int(d), _int(I), _types.dtypes.get(dtype, 0), _act(act)
    f.torch_dtype = dtype
    f.w_gate, f.s_gate = _codes(w_gate, (I, d), "w_gate"), _scales(s_gate, I, "s_gate")
    f.w_up, f.s_up = _codes(w_up, (I, d), "w_up"), _scales(s_up, I, "s_up")
    f.w_down, f.s_down = _codes(w_down, (d, I), "w_down"), _scales(s_down, d, "s_down")
    f.keep = (w_gate, s_gate, w_up, s_up, w_down, s_down)
    return f


def moe_ffn_s8_workspace(f: moe_ffn_s8, T: int) -> int:
    n = ctypes.c_longlong()
    _check(lib.moe_ffn_s8_workspace(f, _int(T), ctypes.byref(n)), "moe_ffn_s8_workspace")
    return n.value


def moe_ffn_s8_forward(f: moe_ffn_s8, x, T: int, y, workspace=None, stream=None) -> None:
    xp, lx = _rows(x, T, f.d_model, f.torch_dtype, "x")
    yp, ly = _rows(y, T, f.d_model, f.torch_dtype, "y")
    wp, wn = _space(workspace)
    _check(lib.moe_ffn_s8_forward(f, xp, lx, _int(T), yp, ly, wp, wn, _stream(stream)),
           "moe_ffn_s8_forward")


def moe_ffn_get_device_error() -> int:
    code = ctypes.c_int(0)
    _check(lib.moe_ffn_get_device_error(ctypes.byref(code)), "moe_ffn_get_device_error")
    return code.value
