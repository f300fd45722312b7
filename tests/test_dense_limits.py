"""Dense feed-forward operators at the ends of their ranges: what the calls document, at the values and sizes where
it is easiest to break."""
import gc
import os
import random
import shutil
import subprocess
import sys
import weakref

import pytest
import torch

from quantized_expert_ffn_token_b200 import capi
from tests.test_dense_ffn import _backward, _forward, _mk, _ws, check_backward, quantize64

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# ---- sizes: refused before a device is touched -------------------------------------------------------------------

P = 0x100000            # an aligned address that no device has: a call that gets as far as looking at it fails otherwise


@pytest.mark.parametrize("N", [(1 << 30) + 8, (1 << 31) - 16, (1 << 31) - 8])
@pytest.mark.parametrize("T", [1, 16, 200])
def test_product_refuses_more_columns_than_its_indices_hold(T, N):
    """Row and column indices of the kernels are 32-bit: the last block of 8 or 16 rows of w would start past 2^31."""
    st = capi.lib.moe_matmul_s8(P, P, T, P, P, N, 16, None, P, capi.MOE_BF16, 0, None, 0, None)
    assert st == capi.MOE_ERR_UNSUPPORTED and "N" in capi.last_error()


class Huge:
    """What the binding looks at of a CUDA tensor of any size."""
    is_cuda = True

    def __init__(self, *shape, dtype=torch.bfloat16):
        self.shape, self.dtype = torch.Size(shape), dtype

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return P


BIG = (1 << 32) + 4     # 4 in 32 bits


def test_binding_passes_no_size_cut_to_32_bits():
    """Sizes above 2^31 are refused as those above 2^30 are; a size taken modulo 2^32 would be answered in part."""
    i8, f32 = torch.int8, torch.float32

    def refused(call):
        with pytest.raises(capi.MoeError) as e:
            call()
        assert e.value.status == capi.MOE_ERR_UNSUPPORTED

    refused(lambda: capi.moe_quantize_s8(Huge(BIG, 1), Huge(BIG, 1, dtype=i8), Huge(BIG, dtype=f32)))
    refused(lambda: capi.moe_quantize_s8(Huge(1, BIG), Huge(1, BIG, dtype=i8), Huge(1, dtype=f32)))

    def product(T, N, K):
        return lambda: capi.moe_matmul_s8(Huge(T, K, dtype=i8), Huge(T, dtype=f32), Huge(N, K, dtype=i8),
                                          Huge(N, dtype=f32), Huge(T, N))
    refused(product(BIG, 8, 16))
    refused(product(2, BIG + 4, 16))
    refused(product(2, 8, BIG + 12))
    f = capi.make_ffn(Huge(16, 8), Huge(16, 8), Huge(8, 16))
    x, h = Huge(BIG, 8), Huge(BIG, 16)
    refused(lambda: capi.moe_ffn_forward(f, x, BIG, x))
    refused(lambda: capi.moe_ffn_backward(f, x, h, h, x, BIG, x))
    with pytest.raises(capi.MoeError):
        capi.moe_ffn_forward(f, x, 4 - (1 << 32), x)
    w, s = Huge(16, 16, dtype=i8), Huge(16, dtype=f32)
    f8 = capi.make_ffn_s8(w, s, w, s, w, s, "silu", torch.bfloat16)
    refused(lambda: capi.moe_ffn_s8_forward(f8, Huge(BIG, 16), BIG, Huge(BIG, 16)))
    # the workspace of more rows than there are 32-bit sizes is no smaller than that of 2^31 - 1
    top = (1 << 31) - 1
    assert capi.moe_ffn_workspace(f, BIG, True) == capi.moe_ffn_workspace(f, top, True)
    assert capi.moe_ffn_s8_workspace(f8, BIG) == capi.moe_ffn_s8_workspace(f8, top)
    # widths: refused when the handle is used
    wide = BIG + 4
    f = capi.make_ffn(Huge(wide, 8), Huge(wide, 8), Huge(8, wide))
    refused(lambda: capi.moe_ffn_workspace(f, 4))


# ---- bounded waits -------------------------------------------------------------------------------------------------

def _host_program(tmp_path, body):
    """Compiles and runs host code over the kernels' schedule header; its output's lines."""
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    src, exe = tmp_path / "schedule.cu", tmp_path / "schedule"
    src.write_text('#include <stdio.h>\n#include "dense_schedule.cuh"\nusing namespace qeffn::dense;\n' + body)
    csrc = os.path.join(ROOT, "quantized_expert_ffn_token_b200", "csrc")
    subprocess.check_call([nvcc, "-std=c++17", "-I", csrc, "-o", str(exe), str(src)])
    return subprocess.check_output([str(exe)], text=True).splitlines()


def test_wait_for_a_tile_outlasts_its_reduction(tmp_path):
    """The epilogue waits for a tile's whole reduction at once.  Weight gradients reduce over up to 2^30 rows, 64 a step;
    a step on a CTA pair with 128 columns takes at least 256 cycles (128 rows x 64 values x 1 column in 2) and is modelled
    at 1.18 * 345 = 408.  The limit leaves twice that at every length, and stays near two seconds for the usual ones."""
    steps = [1, 128, 1 << 13, 1 << 20, 1 << 24]
    out = _host_program(tmp_path, "int main() { for (long long k : {%s}) printf(\"%%lld\\n\", tile_wait_cycles(k)); }"
                        % ", ".join(f"{k}LL" for k in steps))
    for k, limit in zip(steps, map(int, out)):
        assert limit >= 2 * 408 * k
    assert int(out[1]) < 4.01e9


# ---- the order of tiles -----------------------------------------------------------------------------------------------

def test_every_tile_is_dealt_once(tmp_path):
    """The kernels' own order, run on the host: over all clusters every tile comes once and ascending, the tiles of the
    long product first and evenly, and a cluster with one long tile less takes the extra rounds of short ones."""
    rng = random.Random(5)
    cases = []
    for _ in range(1500):
        big, small = rng.choice([0, rng.randrange(200)]), rng.randrange(800)
        P = rng.randint(1, min(74, max(1, big + small)))
        r = big % P
        rounds = rng.randint(0, small // (P - r)) if r else 0
        cases.append((big + small, big, rounds, P))
    rows = ", ".join("{%d, %d, %d, %d}" % c for c in cases)
    out = _host_program(tmp_path, """
template <bool G> void deal(const int *q) {
    for (int c = 0; c < q[3]; ++c) {
        Order<G> order(q[0], q[1], q[2], c, q[3]);
        int k = 0;
        for (int t; (t = order.at(k)) >= 0 && k <= q[0]; ++k) printf("%%d ", t);
        printf("\\n");
    }
}
int main() {
    static const int q[][4] = {%s};
    for (const int *p : q) deal<true>(p), deal<false>(p);
}
""" % rows)
    lines = iter(out)
    for n, big, rounds, P in cases:
        group = [list(map(int, next(lines).split())) for _ in range(P)]
        single = [list(map(int, next(lines).split())) for _ in range(P)]
        for dealt in (group, single):
            assert sorted(t for d in dealt for t in d) == list(range(n))
            assert all(d == sorted(d) for d in dealt)
        long = [sum(t < big for t in d) for d in group]
        assert max(long) - min(long) <= 1
        if big % P:
            assert min(len(d) - m for d, m in zip(group, long) if m == min(long)) >= rounds


# ---- handles ------------------------------------------------------------------------------------------------------

def test_a_handle_frees_its_weights_with_its_last_reference():
    """A handle keeps its weights alive, and gives them up at once: the cyclic collector does not see device memory, so
    a handle per training step must not wait for it."""
    i8, f32 = torch.int8, torch.float32
    w = [Huge(16, 16) for _ in range(3)]
    q = [t for _ in range(3) for t in (Huge(16, 16, dtype=i8), Huge(16, dtype=f32))]
    gc.collect()
    gc.disable()
    try:
        for tensors, make in ((w, lambda: capi.make_ffn(*w)),
                              (q, lambda: capi.make_ffn_s8(*q, "silu", torch.bfloat16))):
            watch = [weakref.ref(t) for t in tensors]
            f = make()
            tensors.clear()
            assert all(r() is not None for r in watch)
            assert (capi.moe_ffn_workspace if tensors is w else capi.moe_ffn_s8_workspace)(f, 4) > 0
            del f
            assert all(r() is None for r in watch)
    finally:
        gc.enable()


# ---- the binding without torch ------------------------------------------------------------------------------------

def test_binding_imports_without_torch():
    """The binding is ctypes: a program that passes addresses needs no torch, and pays for no import of it."""
    code = """
import ctypes, sys
sys.modules["torch"] = None          # importing it raises ImportError
from quantized_expert_ffn_token_b200 import capi
assert capi.lib.moe_quantize_s8(None, capi.MOE_BF16, 0, 4, 8, None, None, None) == capi.MOE_ERR_INVALID_ARG
h = ctypes.c_void_p()
assert capi.lib.moe_create(None, 0, ctypes.byref(h)) == capi.MOE_ERR_INVALID_ARG
print(sorted(capi.EXPORTED)[0])
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and r.stdout.startswith("moe_"), r.stderr[-2000:]
    assert capi.DTYPES == {torch.bfloat16: capi.MOE_BF16, torch.float16: capi.MOE_FP16, torch.float32: capi.MOE_FP32}


# ---- rows whose scale is a small subnormal number ----------------------------------------------------------------

UNIT = 2.0 ** -149      # fp32's smallest positive number


@pytest.mark.gpu
@pytest.mark.parametrize("cols", [64, 33, 4096])      # 16-byte loads, element by element, several loads a thread
def test_codes_of_tiny_rows_stay_in_range(cols):
    """scale = max / 127 in whole units of 2^-149, so that a quotient may lie above 127 (190 for a maximum of 190 units):
    its code is 127, and never wraps.  All numbers here are whole multiples of the unit, and the quotients of their
    multiples are the same in any precision that holds them: int and fp64 arithmetic are exact."""
    tops = [1, 63, 64, 127, 128, 150, 190, 191, 317, 318, 16065, 65536, 10 ** 6]
    gen = torch.Generator().manual_seed(cols)
    units = torch.stack([torch.randint(-t, t + 1, (cols,), generator=gen) for t in tops]).double()
    for i, t in enumerate(tops):
        units[i, 0], units[i, 1], units[i, 2] = t, -t, 0
    x = (units * UNIT).float()
    assert torch.equal(x.double(), units * UNIT)
    s = (units.abs().amax(1) / 127).round()                         # half to even, as the fp32 division rounds here
    quot = (units / torch.where(s > 0, s, torch.ones_like(s))[:, None]).float().double()
    want = torch.where(s[:, None] > 0, quot.round().clamp(-127, 127), torch.zeros_like(quot))
    assert (quot.abs() > 127.5).any()                               # the range that this test is for
    q = torch.empty(len(tops), cols, dtype=torch.int8, device="cuda")
    scale = torch.empty(len(tops), device="cuda")
    capi.moe_quantize_s8(x.cuda(), q, scale)
    assert torch.equal(scale.double().cpu(), s * UNIT)
    assert torch.equal(q.cpu().double(), want)


# ---- the largest number of rows ----------------------------------------------------------------------------------

@pytest.mark.gpu
def test_weight_gradients_over_the_largest_batch():
    """2^30 rows, all zero but for some in front, in the middle and at the end: the gradients are those of these rows
    alone (a row of zeros adds exact zeros), and no wait gives up on the way.  Inputs may share memory: x is dy and gate
    is up, which keeps the test below 90 GB."""
    T, d, I, dt = 1 << 30, 8, 8, torch.bfloat16
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 100e9:
        pytest.skip("needs 100 GB of device memory")
    gen = torch.Generator(device="cuda").manual_seed(30)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(dt)  # noqa: E731
    wg, wu, wd = rnd(I, d), rnd(I, d), rnd(d, I)
    x, g = torch.zeros(T, d, dtype=dt, device="cuda"), torch.zeros(T, I, dtype=dt, device="cuda")
    at = torch.cat([torch.arange(s, s + 40, device="cuda") for s in (0, 12345, T // 2 - 20, 3 * (T // 4), T - 40)])
    x[at], g[at] = rnd(at.numel(), d), rnd(at.numel(), I)
    f = capi.make_ffn(wg, wu, wd)
    ws = torch.empty(capi.moe_ffn_workspace(f, T, True), dtype=torch.uint8, device="cuda")
    out = [torch.full(s, float("nan"), device="cuda") for s in ((I, d), (I, d), (d, I))]
    capi.moe_ffn_backward(f, x, g, g, x, T, None, *out, workspace=ws)
    assert capi.moe_ffn_get_device_error() == 0
    check_backward(x[at], g[at], g[at], x[at], wg, wu, wd, "silu", [None] + out, dw_dtype=torch.float32)
    del x, g, ws
    torch.cuda.empty_cache()


# ---- padding ---------------------------------------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 13, 31, 129, 333])
def test_nothing_outside_the_batch_is_read(T):
    """A padded batch: NaN in the rows behind the last one and in the columns beside x and dy changes nothing, and the
    padding of the outputs stays as it is."""
    d, I, dt = 136, 264, torch.bfloat16
    x, wg, wu, wd, dy, rnd = _mk(T, T, d, I, dt)
    f = capi.make_ffn(wg, wu, wd)
    y, g, u = _forward(f, x)
    want = _backward(f, x, g, u, dy)

    def padded(v):
        buf = torch.full((T + 9, d + 24), float("nan"), dtype=v.dtype, device="cuda")
        buf[:T, 8:8 + d] = v
        return buf, buf[:, 8:8 + d]

    def unchanged(buf, v):
        return torch.equal(buf[:T, 8:8 + d], v) and bool(buf[T:].isnan().all() and buf[:, :8].isnan().all()
                                                          and buf[:, 8 + d:].isnan().all())

    (_, xp), (_, dyp), (yb, yp), (dxb, dxp) = padded(x), padded(dy), padded(y * 0), padded(y * 0)
    capi.moe_ffn_forward(f, xp, T, yp, workspace=_ws(capi.moe_ffn_workspace(f, T)))
    assert unchanged(yb, y)
    dw = [torch.full_like(v, float("nan")) for v in want[1:]]
    capi.moe_ffn_backward(f, xp, g, u, dyp, T, dxp, *dw, workspace=_ws(capi.moe_ffn_workspace(f, T, True)))
    assert unchanged(dxb, want[0])
    assert all(torch.equal(p, q) for p, q in zip(dw, want[1:]))


# ---- graphs ----------------------------------------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 200])
def test_captured_between_copies_and_on_two_streams(T):
    """A graph whose calls come after a copy and a fill, run in two branches (a workspace each) and join again, replayed
    on other inputs; and two such graphs in flight at once."""
    d, I, dt = 256, 512, torch.bfloat16
    graphs = []
    for seed in (1, 2):
        x, wg, wu, wd, dy, rnd = _mk(seed, T, d, I, dt)
        f = capi.make_ffn(wg, wu, wd)
        src, y, g, u = torch.empty_like(x), torch.empty_like(x), x.new_empty(T, I), x.new_empty(T, I)
        q, s = torch.empty(T, d, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
        out = [torch.empty_like(v) for v in (x, wg, wu, wd)]
        ws = _ws(capi.moe_ffn_workspace(f, T)), _ws(capi.moe_ffn_workspace(f, T, True))
        a, b = torch.cuda.Stream(), torch.cuda.Stream()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=a):
            x.copy_(src)                      # a copy node, then a kernel of torch's, then the block
            y.zero_()
            capi.moe_ffn_forward(f, x, T, y, g, u, ws[0], a)
            b.wait_stream(a)
            capi.moe_quantize_s8(y, q, s, b)
            capi.moe_ffn_backward(f, x, g, u, y, T, *out, workspace=ws[1], stream=a)
            a.wait_stream(b)
        graphs.append((graph, f, src, x, y, g, u, q, s, out, rnd, a, (wg, wu, wd), ws))
    for _ in range(3):
        for graph, f, src, *_ in graphs:
            src.copy_(torch.randn_like(src.float()))
        torch.cuda.synchronize()
        for graph, *_, a, _, _ in graphs:
            with torch.cuda.stream(a):
                graph.replay()
        torch.cuda.synchronize()
        for graph, f, src, x, y, g, u, q, s, out, rnd, a, w, ws in graphs:
            y2, g2, u2 = _forward(f, src)
            assert torch.equal(y, y2) and torch.equal(g, g2) and torch.equal(u, u2)
            assert all(torch.equal(p, r) for p, r in zip(out, _backward(f, src, g2, u2, y2)))
            q64, s64 = quantize64(y2)
            assert torch.equal(q.double(), q64) and torch.equal(s.double(), s64)
    assert capi.moe_ffn_get_device_error() == 0
