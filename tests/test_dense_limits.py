"""Dense feed-forward operators at the ends of their ranges: what the calls document, at the values and sizes where
it is easiest to break."""
import pytest
import torch

from quantized_expert_ffn_token_b200 import capi


# ---- sizes: refused before a device is touched -------------------------------------------------------------------

P = 0x100000            # an aligned address that no device has: a call that gets as far as looking at it fails otherwise


@pytest.mark.parametrize("N", [(1 << 30) + 8, (1 << 31) - 16, (1 << 31) - 8])
@pytest.mark.parametrize("T", [1, 16, 200])
def test_product_refuses_more_columns_than_its_indices_hold(T, N):
    """Row and column indices of the kernels are 32-bit: the last block of 8 or 16 rows of w would start past 2^31."""
    st = capi.lib.moe_matmul_s8(P, P, T, P, P, N, 16, None, P, capi.MOE_BF16, 0, None, 0, None)
    assert st == capi.MOE_ERR_UNSUPPORTED and "N" in capi.last_error()


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
