"""The 16-bit block at sizes of training steps, every result whole: CTA pairs with one sub-tile of the gate, its gradient,
dx and the down product, several waves of tiles and both accumulators in turn, weight gradients over thousands of rows,
and fp32 sums of them; and the 8-bit block on CTA pairs.

Tolerances.  Roundings as test_dense_ffn.py counts them.  Accumulation: a tile adds K / 16 MMAs to one fp32 accumulator; one
is off by at most 2^-22 of the partial sum (a last place for the sum, another for the alignment of its addends), with
any sign.  The partial sum after j MMAs of 16 products of independent centred entries with standard deviation s stays
below 6 s sqrt(16 j), so that all together are off by at most 2^-22 * 6 * 4 s * (2 / 3) (K / 16)^1.5 = 2^-24 K * sqrt(K) s,
and sqrt(K) s is the root of the sum of the squared products: ``acc_tol``.
"""
import pytest
import torch

from quantized_expert_ffn_token_b200 import capi
from tests.test_dense_ffn import (ACTS, U, UACT, _backward, _forward, _mk, _quantized, _ws, act64, check, check_ffn_s8)

DT = [torch.bfloat16, torch.float16]
# tokens, d, I: the second with sizes that end inside tiles, the third a ragged batch, the last with a short d, a
# reduction over many rows and few columns
SHAPES = [(1500, 1024, 4096), (2100, 1032, 2056), (1001, 2560, 5120), (6000, 2048, 4104), (8200, 264, 1000)]


def root(a, b):
    """sqrt(sum_k (a_k b_k)^2) of the rows of a and b."""
    return ((a * a) @ (b * b).T).sqrt()


def acc_tol(a, b):
    return 2.0 ** -24 * a.shape[1] * root(a, b)


def near(got, want, tol, u, tiny, what):
    """Element by element, and the outputs' and operands' roundings (one u each, independent) in the 2-norm."""
    check(got, want, u[1] * want.abs() + tol + tiny, what)
    assert (got.double() - want).norm() <= 2 * u[0] * want.norm() + tiny * want.numel(), what


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DT, ids=["bf16", "fp16"])
@pytest.mark.parametrize("T,d,I", SHAPES)
def test_forward_at_training_sizes(T, d, I, dt):
    act = ACTS[(T + d + (dt is torch.float16)) % 3]
    x, wg, wu, wd, _, _ = _mk(T + d + I, T, d, I, dt)
    f = capi.make_ffn(wg, wu, wd, act)
    y, g, u = _forward(f, x)
    X, G, W, D = x.double(), wg.double(), wu.double(), wd.double()
    g64, u64 = X @ G.T, X @ W.T
    eg, eu = acc_tol(X, G), acc_tol(X, W)
    r, tiny = U[dt], 2.0 ** -24 if dt is torch.float16 else 0.0
    near(g, g64, eg, (r, r), tiny, "gate")
    near(u, u64, eu, (r, r), tiny, "up")
    a = act64(g64, act)
    h = a * u64
    # |act'| <= 1.13
    eh = 1.13 * eg * u64.abs() + a.abs() * eu + UACT * h.abs() + tiny
    near(y, h @ D.T, 6 * r * root(h, D) + acc_tol(h, D) + eh @ D.abs().T, (r, r), tiny, "y")
    assert torch.equal(_forward(f, x, save=False)[0], y)
    assert capi.moe_ffn_get_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DT, ids=["bf16", "fp16"])
@pytest.mark.parametrize("T,d,I", SHAPES)
def test_backward_at_training_sizes(T, d, I, dt):
    act = ACTS[(T + I + (dt is torch.float16)) % 3]
    x, wg, wu, wd, dy, rnd = _mk(T + 3 * d + I, T, d, I, dt)
    g, u = rnd(T, I, 2.0), rnd(T, I)
    f = capi.make_ffn(wg, wu, wd, act)
    X, G, W, D, g64, u64, dy64 = (v.double() for v in (x, wg, wu, wd, g, u, dy))
    z = g64.clone().requires_grad_(True)
    a = act64(z, act)
    (dact,) = torch.autograd.grad(a.sum(), z)
    a = a.detach()
    dh, h = dy64 @ D, a * u64
    dg, du = dh * u64 * dact, dh * a
    edh = acc_tol(dy64, D.T)
    r, tiny = U[dt], 2.0 ** -24 if dt is torch.float16 else 0.0
    edg = edh * (u64 * dact).abs() + 3 * UACT * (dh * u64).abs() + tiny
    edu = edh * a.abs() + UACT * du.abs() + tiny
    eh = UACT * h.abs() + tiny
    want = [dg @ G + du @ W, dg.T @ X, du.T @ X, dy64.T @ h]

    def summed(p, q):       # the operand that is rounded, and the accumulation
        return 6 * r * root(p, q) + acc_tol(p, q)

    # dx: one accumulator holds both sums, 2 I products
    tol = [summed(dg, G.T) + summed(du, W.T) + 2.0 ** -24 * I * (root(dg, G.T) + root(du, W.T)) + edg @ G.abs() + edu @ W.abs(),
           summed(dg.T, X.T) + edg.T @ X.abs(), summed(du.T, X.T) + edu.T @ X.abs(),
           summed(h.T, dy64.T).T + dy64.abs().T @ eh]
    names = ("dx", "dw_gate", "dw_up", "dw_down")
    out = _backward(f, x, g, u, dy)
    for i, name in enumerate(names):
        near(out[i], want[i], tol[i], (r, r), tiny, name)
    assert all(torch.equal(p, q) for p, q in zip(out, _backward(f, x, g, u, dy)))
    for i, v in enumerate(_backward(f, x, g, u, dy, dx=False)):
        assert v is None or torch.equal(v, out[i])
    near(_backward(f, x, g, u, dy, dw=False)[0], want[0], tol[0], (r, r), tiny, "dx alone")
    wide = _backward(f, x, g, u, dy, dw_dtype=torch.float32)
    added = _backward(f, x, g, u, dy, dw_dtype=torch.float32, fill=0.5, add=True)
    assert torch.equal(wide[0], out[0])
    for i in (1, 2, 3):
        near(wide[i], want[i], tol[i], (r, 2.0 ** -24), tiny, names[i] + " in fp32")
        assert torch.equal(added[i], 0.5 + wide[i])
        assert torch.equal(wide[i].to(dt), out[i])        # the same sums, rounded
    assert capi.moe_ffn_get_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T,d,I,act", [(2100, 2064, 4112, "silu"), (4100, 1040, 2064, "gelu_tanh"), (1500, 512, 4096, "gelu")])
def test_ffn_s8_at_prompt_sizes(T, d, I, act):
    x, wg, wu, wd, _, _ = _mk(T + d + I, T, d, I, torch.bfloat16)
    wq = [_quantized(w) for w in (wg, wu, wd)]
    f = capi.make_ffn_s8(*wq[0], *wq[1], *wq[2], act, torch.bfloat16)
    y = torch.full((T, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    capi.moe_ffn_s8_forward(f, x, T, y, _ws(capi.moe_ffn_s8_workspace(f, T)))
    check_ffn_s8(x, wq, act, y)
    assert capi.moe_ffn_get_device_error() == 0
