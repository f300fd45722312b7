"""Workloads of the dense feed-forward operators: the gated block in 16 bits (forward and backward pass), the 8-bit
integer product with a scale for each token and channel, alone and behind the quantisation of its rows, and the gated
block in 8 bits.

``own`` chooses what ``run`` calls: False computes the plain form (elementary torch operations in fp32, rounded once
at the end), True the library's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one token through a dense layer of four times the hidden size: all weight bytes, no reuse
        {"name": "ffn_t1", "op": "ffn", "T": 1, "d": 2560, "I": 10240, "dtype": "bf16", "act": "silu", "save": False},
        # four drafted tokens through a block of one expert's size: the smallest call, launch and latency bound
        {"name": "ffn_t4_small", "op": "ffn", "T": 4, "d": 2560, "I": 512, "dtype": "fp16", "act": "silu", "save": False},
        # a prompt of odd length: between weight-bound and compute-bound
        {"name": "ffn_t333", "op": "ffn", "T": 333, "d": 2560, "I": 6912, "dtype": "bf16", "act": "gelu_tanh",
         "save": False},
        # a training step's forward pass, its pre-activations kept for the backward pass
        {"name": "ffn_train", "op": "ffn", "T": 8192, "d": 4096, "I": 12288, "dtype": "bf16", "act": "silu", "save": True},
        # that step's backward pass
        {"name": "ffn_bwd_train", "op": "ffn_bwd", "T": 8192, "d": 4096, "I": 12288, "dtype": "bf16", "act": "silu"},
        # the backward pass of a short ragged batch
        {"name": "ffn_bwd_t1001", "op": "ffn_bwd", "T": 1001, "d": 2560, "I": 5120, "dtype": "fp16", "act": "gelu_tanh"},
        # a decode batch through one projection
        {"name": "mm_s8_t16", "op": "matmul_s8", "T": 16, "K": 2560, "N": 10240, "out": "bf16", "bias": False},
        # a long prompt through one projection
        {"name": "mm_s8_t8192", "op": "matmul_s8", "T": 8192, "K": 4096, "N": 12288, "out": "bf16", "bias": False},
        # one token, quantised on the way in
        {"name": "linear_s8_t1", "op": "linear_s8", "T": 1, "K": 2560, "N": 10240, "out": "bf16", "bias": False,
         "dtype": "bf16"},
        # a ragged prompt, quantised on the way in, with a bias and an fp32 result
        {"name": "linear_s8_t777", "op": "linear_s8", "T": 777, "K": 2560, "N": 5120, "out": "fp32", "bias": True,
         "dtype": "bf16"},
        # one token through the block in 8 bits
        {"name": "ffn_s8_t1", "op": "ffn_s8", "T": 1, "d": 2560, "I": 10240, "dtype": "bf16", "act": "silu"},
        # a prompt chunk through the block in 8 bits
        {"name": "ffn_s8_t4096", "op": "ffn_s8", "T": 4096, "d": 4096, "I": 12288, "dtype": "bf16", "act": "silu"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ffn", "ffn", "ffn_bwd", "matmul_s8", "linear_s8", "ffn_s8"])
    T = _log(rng, 1, 8192)
    a, b = 16 * _log(rng, 16, 256), 16 * _log(rng, 16, 768)   # rows of 8-bit weights come in 16-byte units
    if op in ("ffn", "ffn_bwd"):                              # rows of 16-bit weights too: odd multiples of 8
        a, b = a - 8 * rng.randrange(2), b - 8 * rng.randrange(2)
    case = {"op": op, "T": T}
    if op in ("matmul_s8", "linear_s8"):
        case.update(K=a, N=b - 8 * rng.randrange(2), out=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                    bias=rng.random() < 0.3)
    else:
        case.update(d=a, I=b, act=rng.choice(["silu", "silu", "gelu_tanh", "gelu"]))
    if op != "matmul_s8":
        case["dtype"] = rng.choice(["bf16", "bf16", "fp16"])
    if op == "ffn":
        case["save"] = rng.random() < 0.4
    return case


# ---- inputs -----------------------------------------------------------------------------------------------------

def _tokens(gen, T, d, dt):
    """Normalised activations with a few channels of ten times the rest's size, as a residual stream has them."""
    x = torch.randn(T, d, generator=gen, device="cuda")
    wide = torch.randint(0, d, (max(1, d // 512),), generator=gen, device="cuda")
    x[:, wide] *= 10.0
    return x.to(dt)


def _weight(gen, rows, cols, dt):
    return (torch.randn(rows, cols, generator=gen, device="cuda") / math.sqrt(cols)).to(dt)


def _weight_s8(gen, rows, cols):
    """Channel-wise 8-bit weights: codes and one scale a row."""
    w = torch.randn(rows, cols, generator=gen, device="cuda") / math.sqrt(cols)
    s = w.abs().amax(1) / 127.0
    return torch.round(w / s[:, None]).to(torch.int8), s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, T = case["op"], case["T"]
    st = {"case": case}
    if op in ("matmul_s8", "linear_s8"):
        K, N = case["K"], case["N"]
        st["w"], st["ws"] = _weight_s8(gen, N, K)
        st["bias"] = torch.randn(N, generator=gen, device="cuda") if case["bias"] else None
        if op == "matmul_s8":
            st["a"] = torch.randn(T, K, generator=gen, device="cuda").mul_(32).round_().clamp_(-127, 127).to(torch.int8)
            st["as"] = torch.rand(T, generator=gen, device="cuda") * 0.05 + 0.01
        else:
            st["x"] = _tokens(gen, T, K, DTYPES[case["dtype"]])
            st["a"] = torch.empty(T, K, dtype=torch.int8, device="cuda")
            st["as"] = torch.empty(T, device="cuda")
        st["y"] = torch.empty(T, N, dtype=DTYPES[case["out"]], device="cuda")
    else:
        d, I, dt = case["d"], case["I"], DTYPES[case["dtype"]]
        st["x"] = _tokens(gen, T, d, dt)
        if op == "ffn_s8":
            for name, rows, cols in (("wg", I, d), ("wu", I, d), ("wd", d, I)):
                st[name], st[name + "_s"] = _weight_s8(gen, rows, cols)
        else:
            st["wg"], st["wu"], st["wd"] = _weight(gen, I, d, dt), _weight(gen, I, d, dt), _weight(gen, d, I, dt)
        if op == "ffn_bwd":
            st["gate"], st["up"] = st["x"] @ st["wg"].T, st["x"] @ st["wu"].T
            st["dy"] = torch.randn(T, d, generator=gen, device="cuda").to(dt)
            st["dx"] = torch.empty_like(st["x"])
            for name in ("wg", "wu", "wd"):
                st["d" + name] = torch.empty_like(st[name])
        else:
            st["y"] = torch.empty_like(st["x"])
            if case.get("save"):
                st["gate"], st["up"] = (torch.empty(T, I, dtype=dt, device="cuda") for _ in range(2))
    if own:
        st["plan"] = _plan(st)
    return st


# ---- the library's calls ------------------------------------------------------------------------------------------

def _plan(st):
    """The weights' handle and the workspace that a program keeps between calls."""
    from quantized_expert_ffn_token_b200 import capi
    c = st["case"]
    op, T = c["op"], c["T"]
    if op in ("matmul_s8", "linear_s8"):
        f, size = None, capi.moe_matmul_s8_workspace(T, c["N"], c["K"])
    elif op == "ffn_s8":
        f = capi.make_ffn_s8(st["wg"], st["wg_s"], st["wu"], st["wu_s"], st["wd"], st["wd_s"], c["act"], st["x"].dtype)
        size = capi.moe_ffn_s8_workspace(f, T)
    else:
        f = capi.make_ffn(st["wg"], st["wu"], st["wd"], c["act"])
        size = capi.moe_ffn_workspace(f, T, backward=op == "ffn_bwd")
    return capi, f, torch.empty(size, dtype=torch.uint8, device="cuda")


def _run_own(st):
    capi, f, ws = st["plan"]
    c = st["case"]
    op, T, stream = c["op"], c["T"], torch.cuda.current_stream()
    if op == "ffn":
        capi.moe_ffn_forward(f, st["x"], T, st["y"], st.get("gate"), st.get("up"), ws, stream)
        return (st["y"], st["gate"], st["up"]) if c["save"] else st["y"]
    if op == "ffn_bwd":
        capi.moe_ffn_backward(f, st["x"], st["gate"], st["up"], st["dy"], T, st["dx"], st["dwg"], st["dwu"], st["dwd"],
                              workspace=ws, stream=stream)
        return st["dx"], st["dwg"], st["dwu"], st["dwd"]
    if op == "ffn_s8":
        capi.moe_ffn_s8_forward(f, st["x"], T, st["y"], ws, stream)
        return st["y"]
    if op == "linear_s8":
        capi.moe_quantize_s8(st["x"], st["a"], st["as"], stream)
    capi.moe_matmul_s8(st["a"], st["as"], st["w"], st["ws"], st["y"], st["bias"], ws, stream)
    return st["y"]


# ---- the plain form -----------------------------------------------------------------------------------------------

def _act(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    if act == "gelu_tanh":
        return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))
    return 0.5 * g * (1 + torch.erf(g * math.sqrt(0.5)))


def _act_grad(g, act):
    if act == "silu":
        s = 1 / (1 + torch.exp(-g))
        return s * (1 + g * (1 - s))
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (g + 0.044715 * g * g * g))
        return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)
    return 0.5 * (1 + torch.erf(g * math.sqrt(0.5))) + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)


def _quantize(x):
    x = x.float()
    top = x.abs().amax(1)
    s = top / torch.full_like(top, 127.0)   # a division, not a product with the rounded 1/127
    q = torch.round(x / torch.where(s > 0, s, torch.ones_like(s))[:, None])
    return torch.where(s[:, None] > 0, q, torch.zeros_like(q)), s


def _matmul_s8(a, a_scale, w, w_scale, bias=None):
    y = (a.float() @ w.float().T) * (a_scale[:, None] * w_scale[None, :])
    return y if bias is None else y + bias


def _run_plain(st):
    c = st["case"]
    op = c["op"]
    if op == "matmul_s8":
        return _matmul_s8(st["a"], st["as"], st["w"], st["ws"], st["bias"]).to(DTYPES[c["out"]])
    if op == "linear_s8":
        q, s = _quantize(st["x"])
        return _matmul_s8(q, s, st["w"], st["ws"], st["bias"]).to(DTYPES[c["out"]])
    act, dt = c["act"], DTYPES[c["dtype"]]
    if op == "ffn_s8":
        q, s = _quantize(st["x"])
        h = _act(_matmul_s8(q, s, st["wg"], st["wg_s"]), act) * _matmul_s8(q, s, st["wu"], st["wu_s"])
        q, s = _quantize(h)
        return _matmul_s8(q, s, st["wd"], st["wd_s"]).to(dt)
    x, wg, wu, wd = st["x"].float(), st["wg"].float(), st["wu"].float(), st["wd"].float()
    if op == "ffn":
        g, u = x @ wg.T, x @ wu.T
        y = ((_act(g, act) * u) @ wd.T).to(dt)
        return (y, g.to(dt), u.to(dt)) if c["save"] else y
    g, u, dy = st["gate"].float(), st["up"].float(), st["dy"].float()
    a = _act(g, act)
    dh = dy @ wd
    dg, du = dh * u * _act_grad(g, act), dh * a
    return ((dg @ wg + du @ wu).to(dt), (dg.T @ x).to(dt), (du.T @ x).to(dt), (dy.T @ (a * u)).to(dt))


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without --------------------------------------------------------------------------------

def work(case):
    op, T = case["op"], case["T"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    if op in ("matmul_s8", "linear_s8"):
        K, N = case["K"], case["N"]
        rows = T * K + 4 * T if op == "matmul_s8" else size[case["dtype"]] * T * K
        return {"bytes": rows + N * K + 4 * N * (2 if case["bias"] else 1) + size[case["out"]] * T * N,
                "flops": 2 * T * N * K}
    d, I = case["d"], case["I"]
    if op == "ffn_s8":
        return {"bytes": 4 * T * d + 3 * d * I + 4 * (2 * I + d), "flops": 6 * T * d * I}
    if op == "ffn":
        return {"bytes": 2 * (2 * T * d + 3 * d * I + (2 * T * I if case["save"] else 0)), "flops": 6 * T * d * I}
    return {"bytes": 2 * (3 * T * d + 2 * T * I + 6 * d * I), "flops": 12 * T * d * I}


# ---- the definition in 64 bits ------------------------------------------------------------------------------------

def _phi(g, act):
    """The activation and its derivative: g P(g) and P(g) + g P'(g) with P the gate's weight."""
    if act == "silu":
        P = torch.special.expit(g)
        dP = P * torch.special.expit(-g)
    elif act == "gelu_tanh":
        z = math.sqrt(8 / math.pi) * (g + 0.044715 * g ** 3)      # (1 + tanh v) / 2 = expit(2 v)
        P = torch.special.expit(z)
        dP = P * torch.special.expit(-z) * math.sqrt(8 / math.pi) * (1 + 0.134145 * g ** 2)
    else:
        P = torch.special.ndtr(g)
        dP = torch.exp(-g ** 2 / 2) / math.sqrt(2 * math.pi)
    return g * P, P + g * dP


def _codes64(x):
    """Codes and scales of rows: the scale is the fp32 number nearest max|x| / 127, and the quotients are rounded
    to fp32 before they are rounded to whole numbers."""
    x = x.double()
    s = (x.abs().max(dim=1).values / 127).float().double()
    safe = s.clone()
    safe[s == 0] = 1
    q = (x / safe.unsqueeze(1)).float().double().round()
    q[s == 0] = 0
    return q, s


def _product64(q, s, w, ws):
    return torch.einsum("tk,nk->tn", q, w.double()) * s.unsqueeze(1) * ws.double().unsqueeze(0)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("matmul_s8", "linear_s8"):
        q, s = (st["a"].double(), st["as"].double()) if op == "matmul_s8" else _codes64(st["x"])
        y = _product64(q, s, st["w"], st["ws"])
        return y + st["bias"].double() if case["bias"] else y
    if op == "ffn_s8":
        q, s = _codes64(st["x"])
        h = _phi(_product64(q, s, st["wg"], st["wg_s"]), case["act"])[0] * _product64(q, s, st["wu"], st["wu_s"])
        q, s = _codes64(h)
        return _product64(q, s, st["wd"], st["wd_s"])
    x, wd = st["x"].double(), st["wd"].double()
    if op == "ffn":
        g = torch.einsum("td,id->ti", x, st["wg"].double())
        u = torch.einsum("td,id->ti", x, st["wu"].double())
        y = torch.einsum("ti,di->td", _phi(g, case["act"])[0] * u, wd)
        return (y, g, u) if case["save"] else y
    g, u, dy = st["gate"].double(), st["up"].double(), st["dy"].double()
    a, da = _phi(g, case["act"])
    dwd = torch.einsum("td,ti->di", dy, a * u)
    dh = torch.einsum("td,di->ti", dy, wd)
    dg, du = dh * u * da, dh * a
    dx = torch.einsum("ti,id->td", dg, st["wg"].double()) + torch.einsum("ti,id->td", du, st["wu"].double())
    return dx, torch.einsum("ti,td->id", dg, x), torch.einsum("ti,td->id", du, x), dwd
