"""Dense feed-forward operators: refusals (no GPU needed) and, on the GPU, every
operator against its definition in 64 bits.

Tolerances.  ``u`` is the largest relative error of one rounding to the type
(half a step: bf16 2^-8, fp16 2^-11, fp32 2^-24).  An output is rounded once:
at most u |y|.  An operand that the kernel rounds (h, dg, du) carries an
independent error of at most u times itself into every sum it enters; a sum
of n such terms c_k e_k, |e_k| <= u, is a sum of bounded independent errors,
and exceeds 6 u sqrt(sum c_k^2) with probability below 2 e^-18 (Hoeffding).
fp32 accumulation adds at most n 2^-24 of the sum of magnitudes; ``U32`` = 2^-19
of it covers every n used here (at most 2^5 partial sums deep per output in
any kernel).  An activation carries at most ``UACT`` of itself: CUDA documents
__expf(x) within 2 + 1.17 |x| units in the last place, |x| < 89 where it is not
zero, i.e. 107 * 2^-23 < 2^-16.
"""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

from quantized_expert_ffn_token_b200 import capi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
U32 = 2.0 ** -19
UACT = 2.0 ** -16
ACTS = ["silu", "gelu_tanh", "gelu"]


# ---- definitions in 64 bits --------------------------------------------------------------------------------------

def act64(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu_tanh":
        return z * torch.sigmoid((8 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3))   # (1 + tanh v) / 2, exact in the tail
    return z * 0.5 * torch.special.erfc(-z * 0.5 ** 0.5)                     # exact in the tail


def ffn64(x, wg, wu, wd, act):
    g, u = x @ wg.T, x @ wu.T
    return (act64(g, act) * u) @ wd.T


def quantize64(x):
    """Codes and scales of rows, as the header defines them (fp32 scale and quotients, correctly rounded)."""
    x = x.double()
    s = (x.abs().amax(1) / 127).float().double()
    q = (x / torch.where(s > 0, s, torch.ones_like(s))[:, None]).float().double().round()
    return torch.where(s[:, None] > 0, q, torch.zeros_like(q)), s


def check(got, want, tol, what=""):
    """|got - want| <= tol element by element (tol: a tensor)."""
    got = got.double()
    assert torch.isfinite(got).all(), what
    bad = (got - want).abs() > tol
    if bad.any():
        i = torch.nonzero(bad)[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {i}: "
                             f"{got[tuple(i)].item()} for {want[tuple(i)].item()}, tolerance {tol[tuple(i)].item()}")


def sum_tol(a, b, u):
    """Six sigma of sum_k a_k b_k over the last index of a [M][K] and b [N][K], a's entries off by at most u each,
    and the fp32 accumulation."""
    return 6 * u * ((a * a) @ (b * b).T).sqrt() + U32 * (a.abs() @ b.abs().T)


# ---- refusals (host checks: no device) ---------------------------------------------------------------------------

def _ffn(d=256, I=512, dtype=capi.MOE_BF16, act=capi.MOE_ACT_SILU, w=0x10000):
    return capi.moe_ffn(d, I, dtype, act, w, w, w)


def test_ffn_refusals():
    L, P, ws = capi.lib, 0x20000, 0x100000
    n = ctypes.c_longlong()
    inv, uns = capi.MOE_ERR_INVALID_ARG, capi.MOE_ERR_UNSUPPORTED

    def fwd(f, x=P, ldx=0, T=4, y=P, ldy=0, g=None, u=None, w=ws, wn=1 << 40):
        return L.moe_ffn_forward(ctypes.byref(f) if f else None, x, ldx, T, y, ldy, g, u, w, wn, None)

    assert fwd(None) == inv
    assert fwd(_ffn(dtype=capi.MOE_FP32)) == inv
    assert fwd(_ffn(act=0)) == inv and "act" in capi.last_error()
    assert fwd(_ffn(d=0)) == inv
    assert fwd(_ffn(d=252)) == uns
    assert fwd(_ffn(I=516)) == uns
    assert fwd(_ffn(d=65544)) == uns
    assert fwd(_ffn(), T=-1) == inv
    assert fwd(_ffn(), T=(1 << 30) + 1) == uns
    assert fwd(_ffn(), x=None) == inv
    assert fwd(_ffn(w=None)) == inv
    assert fwd(_ffn(), g=P) == inv
    assert fwd(_ffn(), ldx=248) == inv           # shorter than a row
    assert fwd(_ffn(), ldx=260) == inv           # rows off 16 bytes
    assert fwd(_ffn(), x=P + 2) == inv
    assert fwd(_ffn(), w=None) == inv
    assert fwd(_ffn(), wn=16) == inv and "workspace" in capi.last_error()
    assert fwd(_ffn(), w=ws + 128) == inv
    assert fwd(_ffn(), T=0, x=None, w=None) == capi.MOE_OK
    assert L.moe_ffn_workspace(ctypes.byref(_ffn()), -1, 0, ctypes.byref(n)) == inv
    assert L.moe_ffn_workspace(ctypes.byref(_ffn()), 4, 0, None) == inv
    sizes = []
    for T in (0, 1, 100, 8192):
        assert L.moe_ffn_workspace(ctypes.byref(_ffn()), T, 1, ctypes.byref(n)) == capi.MOE_OK
        sizes.append(n.value)
    assert sizes == sorted(sizes)

    def bwd(f, flags=0, T=4, x=P, dx=P, dw=(P, P, P), wn=1 << 40, ldy=0):
        return L.moe_ffn_backward(ctypes.byref(f), x, 0, P, P, P, ldy, T, dx, 0, *dw, flags, ws, wn, None)

    assert bwd(_ffn(), flags=4) == inv
    assert bwd(_ffn(), flags=capi.MOE_FFN_GRAD_ADD) == inv
    assert bwd(_ffn(), dw=(P, None, P)) == inv
    assert bwd(_ffn(), x=None) == inv
    assert bwd(_ffn(), ldy=100) == inv
    assert bwd(_ffn(), wn=100) == inv
    assert bwd(_ffn(), T=-2) == inv
    assert bwd(_ffn(), dx=None, dw=(None, None, None)) == capi.MOE_OK   # nothing wanted


def test_s8_refusals():
    L, P, ws = capi.lib, 0x20000, 0x100000
    inv, uns = capi.MOE_ERR_INVALID_ARG, capi.MOE_ERR_UNSUPPORTED
    n = ctypes.c_longlong()

    def mm(a=P, T=4, N=64, K=64, y=P, dt=capi.MOE_BF16, ld=0, w=ws, s=P):
        return L.moe_matmul_s8(a, s, T, P, s, N, K, None, y, dt, ld, w, 1 << 40, None)

    assert mm(dt=0) == inv
    assert mm(T=-1) == inv
    assert mm(K=24) == uns
    assert mm(N=12) == uns
    assert mm(K=65552) == uns
    assert mm(a=None) == inv
    assert mm(a=P + 1) == inv
    assert mm(s=P + 2) == inv
    assert mm(ld=32) == inv
    assert mm(T=0) == capi.MOE_OK
    assert L.moe_matmul_s8_workspace(4, 0, 64, ctypes.byref(n)) == inv
    q = lambda dt=capi.MOE_BF16, ld=0, r=4, c=64, x=P: L.moe_quantize_s8(x, dt, ld, r, c, P, P, None)  # noqa: E731
    assert q(dt=4) == inv
    assert q(c=0) == inv
    assert q(r=-1) == inv
    assert q(ld=63) == inv
    assert q(x=P + 1) == inv
    assert q(c=65537) == uns
    assert q(r=0) == capi.MOE_OK
    f = capi.moe_ffn_s8(256, 520, capi.MOE_BF16, capi.MOE_ACT_SILU, P, P, P, P, P, P)
    assert L.moe_ffn_s8_workspace(ctypes.byref(f), 4, ctypes.byref(n)) == uns
    f.d_ff = 512
    assert L.moe_ffn_s8_workspace(ctypes.byref(f), 4, ctypes.byref(n)) == capi.MOE_OK
    assert L.moe_ffn_s8_forward(ctypes.byref(f), P, 0, 4, P, 0, ws, n.value - 1, None) == inv
    f.s_up = None
    assert L.moe_ffn_s8_forward(ctypes.byref(f), P, 0, 4, P, 0, ws, n.value, None) == inv
    assert L.moe_ffn_get_device_error(None) == inv


def test_binding_refuses_wrong_tensors():
    w = torch.zeros(64, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError):   # not on a CUDA device
        capi.make_ffn(w, w, torch.zeros(32, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        capi.moe_quantize_s8(torch.zeros(4, 32), torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4))


def test_reference_gradient_is_the_formulas():
    """The backward formulas that the GPU tests use, against differences of the forward definition."""
    gen = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, wg, wu, wd, dy = rnd(5, 6), rnd(7, 6), rnd(7, 6), rnd(6, 7), rnd(5, 6)
    for act in ACTS:
        grads = dict(zip(("x", "wg", "wu", "wd"), grads64(x, x @ wg.T, x @ wu.T, dy, wg, wu, wd, act)))
        p = {"x": x, "wg": wg, "wu": wu, "wd": wd}
        for name in p:
            v, e = rnd(*p[name].shape), 1e-5
            loss = lambda s: (ffn64(**{**p, name: p[name] + s * v}, act=act) * dy).sum()  # noqa: E731
            want = (loss(e) - loss(-e)) / (2 * e)
            assert abs((grads[name] * v).sum() - want) <= 1e-7 * (1 + abs(want))


def grads64(x, g, u, dy, wg, wu, wd, act):
    z = g.detach().clone().requires_grad_(True)
    a = act64(z, act)
    (d,) = torch.autograd.grad(a.sum(), z)
    a = a.detach()
    dh = dy @ wd
    dg, du = dh * u * d, dh * a
    return dg @ wg + du @ wu, dg.T @ x, du.T @ x, dy.T @ (a * u)


# ---- on the GPU --------------------------------------------------------------------------------------------------

def _mk(seed, T, d, I, dt):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda r, c, s=1.0: (torch.randn(r, c, generator=gen, device="cuda") * s).to(dt)  # noqa: E731
    return (rnd(T, d), rnd(I, d, d ** -0.5), rnd(I, d, d ** -0.5), rnd(d, I, I ** -0.5), rnd(T, d), rnd)


def _ws(n):
    return torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")


def _forward(f, x, save=True, stream=None):
    T, d, I = x.shape[0], f.d_model, f.d_ff
    y = torch.full((T, d), float("nan"), dtype=x.dtype, device="cuda")
    g = torch.full((T, I), float("nan"), dtype=x.dtype, device="cuda") if save else None
    u = torch.full_like(g, float("nan")) if save else None
    capi.moe_ffn_forward(f, x, T, y, g, u, _ws(capi.moe_ffn_workspace(f, T)), stream)
    return y, g, u


SHAPES = [(1, 8, 8), (1, 256, 512), (2, 72, 40), (4, 2560, 512), (7, 264, 1000), (16, 512, 136), (17, 136, 264),
          (32, 1024, 520), (33, 256, 256), (65, 520, 392), (128, 384, 640), (129, 512, 1032), (300, 1032, 776),
          (513, 640, 264), (1000, 264, 2056)]
DT = [torch.bfloat16, torch.float16]


def check_forward(x, wg, wu, wd, act, y, g, u):
    dt = x.dtype
    X, G, W, D = x.double(), wg.double(), wu.double(), wd.double()
    g64, u64 = X @ G.T, X @ W.T
    eg, eu = U32 * (X.abs() @ G.abs().T), U32 * (X.abs() @ W.abs().T)
    h64 = act64(g64, act) * u64
    y64 = h64 @ D.T
    if g is not None:
        check(g, g64, U[dt] * g64.abs() + eg + 1e-7, "gate")
        check(u, u64, U[dt] * u64.abs() + eu + 1e-7, "up")
    # |act'| <= 1.13: errors of the fp32 sums g and u pass into h and on into y
    eh = 1.13 * eg * u64.abs() + act64(g64, act).abs() * eu + UACT * h64.abs()
    tiny = 2.0 ** -24 if dt == torch.float16 else 0.0       # fp16 subnormal spacing of h and y
    check(y, y64, U[dt] * y64.abs() + sum_tol(h64, D, U[dt]) + eh @ D.abs().T + tiny * (1 + D.abs().sum(1)), "y")
    # roundings of y and of h, one u each in the relative 2-norm (on average: with few elements the bound above decides)
    assert y.numel() < 4096 or (y.double() - y64).norm() <= 2 * U[dt] * y64.norm() + tiny * y64.numel()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DT, ids=["bf16", "fp16"])
@pytest.mark.parametrize("T,d,I", SHAPES)
def test_forward(T, d, I, dt):
    for act in (ACTS if T in (4, 65) else [ACTS[(T + d) % 3]]):
        x, wg, wu, wd, _, _ = _mk(T + d + I, T, d, I, dt)
        f = capi.make_ffn(wg, wu, wd, act)
        y, g, u = _forward(f, x)
        check_forward(x, wg, wu, wd, act, y, g, u)
        y2, _, _ = _forward(f, x, save=False)
        assert torch.equal(y, y2)        # keeping g and u changes nothing, and the same call gives the same bits
    assert capi.moe_ffn_get_device_error() == 0


def _backward(f, x, g, u, dy, dw_dtype=None, dx=True, dw=True, fill=float("nan"), add=False, stream=None):
    T, d, I = x.shape[0], f.d_model, f.d_ff
    o = lambda r, c, t: torch.full((r, c), fill, dtype=t, device="cuda")  # noqa: E731
    t = dw_dtype or x.dtype
    out = [o(T, d, x.dtype) if dx else None] + ([o(I, d, t), o(I, d, t), o(d, I, t)] if dw else [None] * 3)
    capi.moe_ffn_backward(f, x, g, u, dy, T, *out, add=add, stream=stream,
                          workspace=_ws(capi.moe_ffn_workspace(f, T, backward=True)))
    return out


def check_backward(x, g, u, dy, wg, wu, wd, act, out, dw_dtype=None, base=0.0):
    dt = x.dtype
    uo = U[dw_dtype or dt]
    X, G, W, D, g64, u64, dy64 = (v.double() for v in (x, wg, wu, wd, g, u, dy))
    z = g64.clone().requires_grad_(True)
    a = act64(z, act)
    (dact,) = torch.autograd.grad(a.sum(), z)
    a = a.detach()
    dh = dy64 @ D
    edh = U32 * (dy64.abs() @ D.abs())
    dg, du, h = dh * u64 * dact, dh * a, a * u64
    # errors of dg, du before they are rounded: the fp32 sum dh, and a few fp32 steps in act and act', whose
    # terms (at most max(1, |g|) in size where they cancel) are bounded by 2 + |g| e^-|g| < 3 of fp32's
    edg, edu = edh * (u64 * dact).abs() + 3 * UACT * (dh * u64).abs(), edh * a.abs() + UACT * du.abs()
    tiny = 2.0 ** -24 if dt == torch.float16 else 0.0
    want = [dg @ G + du @ W, dg.T @ X, du.T @ X, dy64.T @ h]
    tol = [sum_tol(dg, G.T, U[dt]) + sum_tol(du, W.T, U[dt]) + edg @ G.abs() + edu @ W.abs()
           + tiny * (1 + G.abs().sum(0) + W.abs().sum(0)),
           sum_tol(dg.T, X.T, U[dt]) + edg.T @ X.abs() + tiny * (1 + X.abs().sum(0)),
           sum_tol(du.T, X.T, U[dt]) + edu.T @ X.abs() + tiny * (1 + X.abs().sum(0)),
           sum_tol(h.T, dy64.T, U[dt]).T + UACT * (dy64.abs().T @ h.abs()) + tiny * (1 + dy64.abs().sum(0))[:, None]]
    for i, name in enumerate(("dx", "dw_gate", "dw_up", "dw_down")):
        if out[i] is None:
            continue
        w = want[i] + (base if i else 0.0)
        r = (U[dt] if i == 0 else uo)
        check(out[i], w, r * w.abs() + tol[i] + 1e-30, name)
        # the output's rounding and the operand's (dx: two operands, independent), one u each on average: a sum over
        # few elements can lie anywhere within the bound above
        assert w.numel() < 4096 or (out[i].double() - w).norm() <= 2 * U[dt] * w.norm() + tiny * w.numel(), name


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DT, ids=["bf16", "fp16"])
@pytest.mark.parametrize("T,d,I", SHAPES)
def test_backward(T, d, I, dt):
    for act in (ACTS if T in (4, 65) else [ACTS[(T + I) % 3]]):
        x, wg, wu, wd, dy, rnd = _mk(T + 3 * d + I, T, d, I, dt)
        g, u = rnd(T, I, 2.0), rnd(T, I)
        f = capi.make_ffn(wg, wu, wd, act)
        out = _backward(f, x, g, u, dy)
        check_backward(x, g, u, dy, wg, wu, wd, act, out)
        again = _backward(f, x, g, u, dy)
        assert all(torch.equal(p, q) for p, q in zip(out, again))
        # dx alone may split its reduction, and then sums in another order
        check_backward(x, g, u, dy, wg, wu, wd, act, _backward(f, x, g, u, dy, dw=False))
        only_dw = _backward(f, x, g, u, dy, dx=False)
        assert all(torch.equal(p, q) for p, q in zip(only_dw[1:], out[1:]))
    assert capi.moe_ffn_get_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T,d,I", [(5, 64, 72), (200, 264, 520), (700, 512, 256)])
def test_backward_fp32_sums(T, d, I):
    x, wg, wu, wd, dy, rnd = _mk(7, T, d, I, torch.bfloat16)
    g, u = rnd(T, I), rnd(T, I)
    f = capi.make_ffn(wg, wu, wd)
    out = _backward(f, x, g, u, dy, dw_dtype=torch.float32)
    check_backward(x, g, u, dy, wg, wu, wd, "silu", out, dw_dtype=torch.float32)
    added = _backward(f, x, g, u, dy, dw_dtype=torch.float32, fill=0.5, add=True)
    for p, q in zip(added[1:], out[1:]):
        assert torch.equal(p, 0.5 + q)


@pytest.mark.gpu
def test_no_rows():
    d, I = 64, 72
    x, wg, wu, wd, dy, rnd = _mk(1, 0, d, I, torch.bfloat16)
    f = capi.make_ffn(wg, wu, wd)
    capi.moe_ffn_forward(f, x, 0, x)
    z = torch.empty(0, I, dtype=x.dtype, device="cuda")
    for t in (torch.bfloat16, torch.float32):
        out = _backward(f, x, z, z, dy, dw_dtype=t)
        assert all(not v.any() for v in out[1:])
    kept = _backward(f, x, z, z, dy, dw_dtype=torch.float32, fill=3.0, add=True)
    assert all((v == 3.0).all() for v in kept[1:])
    q, s = torch.empty(0, 32, dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda")
    capi.moe_quantize_s8(torch.empty(0, 32, device="cuda"), q, s)
    w, ws = torch.ones(16, 32, dtype=torch.int8, device="cuda"), torch.ones(16, device="cuda")
    capi.moe_matmul_s8(q, s, w, ws, torch.empty(0, 16, device="cuda"))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 3, 20, 150, 300])
def test_strided_rows_and_padding(T):
    """x, y, dy and dx as slices of wider buffers; what lies around them stays."""
    d, I, dt = 136, 264, torch.bfloat16
    x, wg, wu, wd, dy, rnd = _mk(T, T, d, I, dt)
    f = capi.make_ffn(wg, wu, wd)
    y, g, u = _forward(f, x)
    wide = lambda v: torch.nn.functional.pad(v, (8, 16, 0, 5), value=7.0)[:, 8:8 + d]  # noqa: E731
    xw, dyw = wide(x), wide(dy)
    buf = torch.full((T + 5, d + 24), 7.0, dtype=dt, device="cuda")
    capi.moe_ffn_forward(f, xw, T, buf[:, 8:8 + d], workspace=_ws(capi.moe_ffn_workspace(f, T)))
    assert torch.equal(buf[:T, 8:8 + d], y)
    assert (buf[T:] == 7).all() and (buf[:, :8] == 7).all() and (buf[:, 8 + d:] == 7).all()
    out = _backward(f, x, g, u, dy)
    buf.fill_(7.0)
    dw = [torch.empty_like(v) for v in out[1:]]
    capi.moe_ffn_backward(f, xw, g, u, dyw, T, buf[:, 8:8 + d], *dw,
                          workspace=_ws(capi.moe_ffn_workspace(f, T, backward=True)))
    assert torch.equal(buf[:T, 8:8 + d], out[0])
    assert (buf[T:] == 7).all() and (buf[:, :8] == 7).all() and (buf[:, 8 + d:] == 7).all()
    assert all(torch.equal(p, q) for p, q in zip(dw, out[1:]))
    with pytest.raises(ValueError):
        capi.moe_ffn_forward(f, x[:1].expand(2, d), 2, buf[:, 8:8 + d])


@pytest.mark.gpu
@pytest.mark.parametrize("T", [2, 40, 260])
def test_a_bad_token_stays_in_its_row(T):
    """A NaN or an infinity in one row reaches that row of y alone, and every weight gradient's columns it feeds."""
    d, I, dt = 128, 256, torch.bfloat16
    x, wg, wu, wd, dy, rnd = _mk(T, T, d, I, dt)
    f = capi.make_ffn(wg, wu, wd)
    y, g, u = _forward(f, x)
    x2 = x.clone()
    x2[1, 5] = float("nan")
    y2, _, _ = _forward(f, x2)
    keep = torch.arange(T, device="cuda") != 1
    assert torch.equal(y2[keep], y[keep]) and y2[1].isnan().all()
    out, g2 = _backward(f, x, g, u, dy), g.clone()
    g2[1, 3] = float("nan")
    out2 = _backward(f, x, g2, u, dy)
    assert torch.equal(out2[0][keep], out[0][keep]) and out2[0][1].isnan().all()
    assert out2[1][3].isnan().all() and torch.equal(out2[1][4:], out[1][4:])


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T", [3, 64])
def test_far_pre_activations(act, T):
    """Gates far out on both sides: the activation is 0 or the identity there, and so is its gradient."""
    d, I, dt = 64, 64, torch.bfloat16
    x, wg, wu, wd, dy, rnd = _mk(T, T, d, I, dt)
    g, u = rnd(T, I), rnd(T, I)
    g[0, :8] = torch.tensor([1e4, -1e4, 1e20, -1e20, 300.0, -300.0, 88.0, -88.0], device="cuda").to(dt)
    f = capi.make_ffn(wg, wu, wd, act)
    out = _backward(f, x, g, u, dy)
    assert all(torch.isfinite(v).all() for v in out)
    eye = torch.eye(64, device="cuda", dtype=dt)
    f = capi.make_ffn(eye, eye, eye, act)
    # with both weights the identity, h = act(g) g; 1e20 squared is above bf16's largest value, so that entry of h is
    # infinite: the row's sums hold infinity times one, or infinity times zero (NaN)
    y, _, _ = _forward(f, g)
    assert not torch.isfinite(y[0]).any()
    g2 = g.clone()
    g2[0, 2:4] = 0
    y2, _, _ = _forward(f, g2)
    G = g2.double()
    want = act64(G, act) * G
    want[0, :8] = torch.where(G[0, :8] > 0, G[0, :8] ** 2, torch.zeros_like(G[0, :8]))
    assert torch.equal(y[1:], y2[1:])
    assert ((y2.double() - want).abs() <= 2.1 * U[dt] * want.abs() + 1e-12).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 2560), (3, 7), (5, 33), (17, 264), (64, 4096), (9, 1001), (2, 65536),
                                       (700, 520)])
def test_quantize(rows, cols, dt):
    gen = torch.Generator(device="cuda").manual_seed(rows * cols)
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    x[:, ::97] *= 20
    if rows > 2:
        x[1] = 0
        x[2] = torch.randint(-127, 128, (cols,), generator=gen, device="cuda") * 0.5     # ties and exact codes
        x[2, 0] = 63.5
    x = x.to(dt)
    buf = torch.full((rows, cols + 3), 1e3, device="cuda").to(dt)
    buf[:, 1:cols + 1] = x
    for src in (x, buf[:, 1:cols + 1]):      # contiguous, and at a row distance that is no multiple of 16 bytes
        q = torch.full((rows, cols), -128, dtype=torch.int8, device="cuda")
        s = torch.full((rows,), -1.0, device="cuda")
        capi.moe_quantize_s8(src, q, s)
        q64, s64 = quantize64(x)
        assert torch.equal(s.double(), s64)
        assert torch.equal(q.double(), q64)


@pytest.mark.gpu
def test_quantize_odd_values():
    x = torch.ones(6, 64, device="cuda")
    x[0, 3], x[1, 60], x[2, 0] = float("nan"), float("inf"), -float("inf")
    x[3] *= 1e-45
    x[4] *= 3e38
    x[5] *= 1e-38
    q, s = torch.empty(6, 64, dtype=torch.int8, device="cuda"), torch.empty(6, device="cuda")
    capi.moe_quantize_s8(x, q, s)
    assert s[:3].isnan().all() and not q[:4].any() and s[3] == 0
    assert (q[4:] == 127).all() and torch.isfinite(s[4:]).all()


MM = [(1, 8, 16), (1, 2560, 512), (3, 72, 48), (8, 10240, 256), (16, 264, 528), (17, 136, 80), (32, 520, 1040),
      (33, 256, 256), (100, 1000, 400), (128, 264, 2048), (129, 520, 1040), (300, 776, 4096), (777, 264, 528)]


@pytest.mark.gpu
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16, torch.float32], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,N,K", MM)
def test_matmul_s8(T, N, K, out):
    gen = torch.Generator(device="cuda").manual_seed(T + N + K)
    a = torch.randint(-128, 128, (T, K), generator=gen, device="cuda").to(torch.int8)
    w = torch.randint(-128, 128, (N, K), generator=gen, device="cuda").to(torch.int8)
    a[0], w[0] = -128, -128                      # the largest sum there is
    sa = torch.rand(T, generator=gen, device="cuda") * 1e-3
    sw = torch.rand(N, generator=gen, device="cuda") * 1e-2
    bias = torch.randn(N, generator=gen, device="cuda")
    p = (a.double() @ w.double().T) * sa.double()[:, None] * sw.double()[None]
    for b in (None, bias):
        buf = torch.full((T + 2, N + 8), 7.0, dtype=out, device="cuda")
        y = buf[:T, :N]
        capi.moe_matmul_s8(a, sa, w, sw, y, b, _ws(capi.moe_matmul_s8_workspace(T, N, K)))
        want = p if b is None else p + b.double()
        # the sum, the scales' product and their product round to fp32, then the bias, then the output
        tiny = 2.0 ** -24 if out == torch.float16 else 0.0
        check(y, want, 3.01 * 2.0 ** -24 * p.abs() + (U[out] * 1.001 + 2.0 ** -24) * want.abs() + tiny, "y")
        assert (buf[T:] == 7).all() and (buf[:, N:] == 7).all()
    assert capi.moe_ffn_get_device_error() == 0


def check_ffn_s8(x, wq, act, y):
    (wg, sg), (wu, su), (wd, sd) = wq
    qx, sx = quantize64(x)
    mm = lambda q, s, w, sw: (q @ w.double().T) * s[:, None] * sw.double()[None]  # noqa: E731
    h = act64(mm(qx, sx, wg, sg), act) * mm(qx, sx, wu, su)
    qh, sh = quantize64(h)
    want = mm(qh, sh, wd, sd)
    # h is fp32 in the kernel, within 2^-18 of itself: a quotient that lies this near to a half may round to the
    # other code
    frac = (h / torch.where(sh > 0, sh, torch.ones_like(sh))[:, None]).abs() % 1
    near = ((frac - 0.5).abs() <= 127 * 2.0 ** -18).double()
    tiny = 2.0 ** -24 if x.dtype == torch.float16 else 0.0
    other = mm(near, sh, wd.abs(), sd) + 2.0 ** -18 * mm(qh.abs(), sh, wd.abs(), sd)
    # the value that is rounded last is at most |want| + other, and the rounding is relative to it
    tol = other + (U[x.dtype] + 2.0 ** -17) * (want.abs() + other)
    check(y, want, tol + tiny, "y")
    assert y.numel() < 4096 or (y.double() - want).norm() <= 2 * U[x.dtype] * want.norm() + 1.01 * other.norm() + tiny * want.numel()


def _quantized(w):
    q = torch.empty(w.shape, dtype=torch.int8, device="cuda")
    s = torch.empty(w.shape[0], device="cuda")
    capi.moe_quantize_s8(w.contiguous(), q, s)
    return q, s


@pytest.mark.gpu
@pytest.mark.parametrize("T,d,I", [(1, 16, 16), (1, 2560, 1024), (4, 272, 528), (17, 512, 144), (33, 144, 272),
                                   (130, 528, 1040), (300, 1040, 784)])
def test_ffn_s8(T, d, I):
    for dt, act in ((torch.bfloat16, "silu"), (torch.float16, "gelu_tanh"), (torch.bfloat16, "gelu")):
        x, wg, wu, wd, _, _ = _mk(T + d + I, T, d, I, dt)
        wq = [_quantized(w) for w in (wg, wu, wd)]
        f = capi.make_ffn_s8(*wq[0], *wq[1], *wq[2], act, dt)
        y = torch.full((T, d), float("nan"), dtype=dt, device="cuda")
        capi.moe_ffn_s8_forward(f, x, T, y, _ws(capi.moe_ffn_s8_workspace(f, T)))
        check_ffn_s8(x, wq, act, y)
    assert capi.moe_ffn_get_device_error() == 0


@pytest.mark.gpu
def test_ffn_s8_rows_of_zeros_and_nans():
    T, d, I = 5, 64, 128
    x, wg, wu, wd, _, _ = _mk(3, T, d, I, torch.bfloat16)
    x[1] = 0
    x[3, 7] = float("inf")
    wq = [_quantized(w) for w in (wg, wu, wd)]
    f = capi.make_ffn_s8(*wq[0], *wq[1], *wq[2], "silu", torch.bfloat16)
    y = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    capi.moe_ffn_s8_forward(f, x, T, y, _ws(capi.moe_ffn_s8_workspace(f, T)))
    assert not y[1].any() and y[3].isnan().all() and torch.isfinite(y[[0, 2, 4]]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 4, 48, 320])
def test_captured_calls_replay(T):
    """The whole set in one graph: forward, backward, quantised block; replays on new inputs, no allocation."""
    d, I, dt = 256, 520, torch.bfloat16
    I8 = 528
    x, wg, wu, wd, dy, rnd = _mk(9, T, d, I, dt)
    f = capi.make_ffn(wg, wu, wd)
    wq = [_quantized(w) for w in (rnd(I8, d, d ** -0.5), rnd(I8, d, d ** -0.5), rnd(d, I8, I8 ** -0.5))]
    f8 = capi.make_ffn_s8(*wq[0], *wq[1], *wq[2], "silu", dt)
    ws = [_ws(capi.moe_ffn_workspace(f, T)), _ws(capi.moe_ffn_workspace(f, T, True)),
          _ws(capi.moe_ffn_s8_workspace(f8, T))]
    y, y8, g, u = torch.empty_like(x), torch.empty_like(x), x.new_empty(T, I), x.new_empty(T, I)
    out = [torch.empty_like(v) for v in (x, wg, wu, wd)]

    def calls(stream):
        capi.moe_ffn_forward(f, x, T, y, g, u, ws[0], stream)
        capi.moe_ffn_backward(f, x, g, u, dy, T, *out, workspace=ws[1], stream=stream)
        capi.moe_ffn_s8_forward(f8, x, T, y8, ws[2], stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        calls(side)
    for seed in (1, 2):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        x.copy_(torch.randn(T, d, generator=gen, device="cuda"))
        dy.copy_(torch.randn(T, d, generator=gen, device="cuda"))
        for v in (y, y8, g, u, *out):
            v.fill_(float("nan"))
        for w in ws:
            w.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        check_forward(x, wg, wu, wd, "silu", y, g, u)
        check_backward(x, g, u, dy, wg, wu, wd, "silu", out)
        check_ffn_s8(x, wq, "silu", y8)
    assert capi.moe_ffn_get_device_error() == 0


@pytest.mark.gpu
def test_capture_in_a_fresh_process():
    """A process whose first calls of the operators are captured ones."""
    code = """
import sys, torch
sys.path.insert(0, {root!r})
from tests.test_dense_ffn import *
from tests.test_dense_ffn import _mk, _ws, _quantized
T, d, I, dt = 150, 256, 512, torch.bfloat16
x, wg, wu, wd, dy, rnd = _mk(1, T, d, I, dt)
f = capi.make_ffn(wg, wu, wd)
y, g, u = torch.empty_like(x), x.new_empty(T, I), x.new_empty(T, I)
out = [torch.empty_like(v) for v in (x, wg, wu, wd)]
ws, wb = _ws(capi.moe_ffn_workspace(f, T)), _ws(capi.moe_ffn_workspace(f, T, True))
q, s, x1, y1 = torch.empty(T, d, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda"), x[:3].clone(), y[:3].clone()
st = torch.cuda.Stream()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=st):
    capi.moe_ffn_forward(f, x, T, y, g, u, ws, st)
    capi.moe_ffn_backward(f, x, g, u, dy, T, *out, workspace=wb, stream=st)
    capi.moe_quantize_s8(x, q, s, st)
    capi.moe_ffn_forward(f, x1, 3, y1, workspace=ws, stream=st)
graph.replay()
torch.cuda.synchronize()
check_forward(x, wg, wu, wd, "silu", y, g, u)
check_backward(x, g, u, dy, wg, wu, wd, "silu", out)
check_forward(x1, wg, wu, wd, "silu", y1, None, None)
assert torch.equal(q.double(), quantize64(x)[0])
print("captured")
""".format(root=ROOT)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Intermediates of more than 2^31 elements: the last rows are as they are in a call of their own."""
    T, d, I, dt = 33100, 64, 65536, torch.bfloat16
    x, wg, wu, wd, dy, _ = _mk(5, T, d, I, dt)
    f = capi.make_ffn(wg, wu, wd)
    y, g, u = _forward(f, x)
    n = 40
    check_forward(x[-n:], wg, wu, wd, "silu", y[-n:], g[-n:], u[-n:])
    dx = torch.full_like(x, float("nan"))
    ws = _ws(capi.moe_ffn_workspace(f, T, True))
    capi.moe_ffn_backward(f, x, g, u, dy, T, dx, workspace=ws)
    check_backward(x[-n:], g[-n:], u[-n:], dy[-n:], wg, wu, wd, "silu", [dx[-n:], None, None, None])
    del y, u, dx, ws
    wq = [_quantized(w) for w in (wg, wu, wd)]
    f8 = capi.make_ffn_s8(*wq[0], *wq[1], *wq[2], "silu", dt)
    y8 = torch.full_like(x, float("nan"))
    capi.moe_ffn_s8_forward(f8, x, T, y8, _ws(capi.moe_ffn_s8_workspace(f8, T)))
    check_ffn_s8(x[-n:], wq, "silu", y8[-n:])


@pytest.mark.gpu
def test_two_streams_at_once():
    """Calls on two streams, a workspace each, at sizes of every path."""
    d, I, dt = 512, 1024, torch.bfloat16
    jobs = []
    for i, T in enumerate((2, 90, 600, 5)):
        x, wg, wu, wd, dy, _ = _mk(i, T, d, I, dt)
        f = capi.make_ffn(wg, wu, wd)
        jobs.append((x, f, _forward(f, x)[0], torch.empty_like(x), _ws(capi.moe_ffn_workspace(f, T))))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(20):
        for (x, f, _, y, ws), s in zip(jobs, streams):
            capi.moe_ffn_forward(f, x, x.shape[0], y, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for _, _, want, y, _ in jobs:
        assert torch.equal(y, want)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [6, 150])
def test_train_then_serve(T):
    """The operators together: steps of gradient descent on the 16-bit block with fp32 master weights, whose
    gradients agree with differences of the definition; then the trained weights quantised and served in 8 bits."""
    d, I, dt = 128, 256, torch.bfloat16
    x, wg, wu, wd, target, rnd = _mk(11, T, d, I, dt)
    master = [w.float() for w in (wg, wu, wd)]
    for step in range(3):
        w16 = [w.to(dt) for w in master]
        f = capi.make_ffn(*w16)
        y, g, u = _forward(f, x)
        dy = ((y.float() - target.float()) / T).to(dt)
        out = _backward(f, x, g, u, dy, dw_dtype=torch.float32)
        check_backward(x, g, u, dy, *w16, "silu", out, dw_dtype=torch.float32)
        # differences of the definition along the gradients' own direction; g and u were rounded on the way (u of
        # bf16 each, entering dg and du once), as were dg, du, h
        W = [w.double() for w in w16]
        for i, v in enumerate(out[1:]):
            v, e = v.double() / v.double().norm(), 1e-4
            at = lambda s: (ffn64(x.double(), *[w + s * v if j == i else w for j, w in enumerate(W)], "silu")  # noqa: E731
                            * dy.double()).sum()
            want = (at(e) - at(-e)) / (2 * e)
            assert abs((out[1 + i].double() * v).sum() - want) <= 4 * U[dt] * abs(want)
        for w, v in zip(master, out[1:]):
            w -= 0.1 * v
    wq = [_quantized(w) for w in master]
    f8 = capi.make_ffn_s8(*wq[0], *wq[1], *wq[2], "silu", dt)
    y8 = torch.empty_like(x)
    capi.moe_ffn_s8_forward(f8, x, T, y8, _ws(capi.moe_ffn_s8_workspace(f8, T)))
    check_ffn_s8(x, wq, "silu", y8)
    # the block step by step through the product's own entry point gives the same numbers
    qx, sx = _quantized(x)
    g, u = (torch.empty(T, I, device="cuda") for _ in range(2))
    for o, (q, s) in ((g, wq[0]), (u, wq[1])):
        capi.moe_matmul_s8(qx, sx, q, s, o, workspace=_ws(capi.moe_matmul_s8_workspace(T, I, d)))
    h = g / (1 + torch.exp(-g)) * u
    qh, sh = _quantized(h)
    y9 = torch.empty_like(x)
    capi.moe_matmul_s8(qh, sh, *wq[2], y9, workspace=_ws(capi.moe_matmul_s8_workspace(T, d, I)))
    assert (y9.double() - y8.double()).norm() <= 2 * U[dt] * y8.double().norm()
