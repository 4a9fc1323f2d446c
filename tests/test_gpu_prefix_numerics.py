"""Shared-prefix decode attention where the reference of a row moves, or the values' sizes differ, by far: each output against
the definition in 64 bits, held to the sum of w |v| of its own row instead of the largest |v|.

An output is sum w v / sum w. Each weight enters the second product rounded to 16 bits, and so does (E4M3) each value times
its scale; the exponent of a weight is off by the logits' fp32 sums, `err`, absolute. So it is off by (rounding + 2 err) of
sum w |v| / sum w, and by 2^-8 of itself for its own rounding to bf16. The rounding is 2^-8 on a bf16 cache, and on an E4M3
cache 3 * 2^-11 (weight, scale, and their product with the code), stated as 2^-9."""
import numpy as np
import pytest
import torch

from decode_attention_mfa_gb300 import capi
from test_gpu_prefix import DIM, HEADS, KV, PAGE, SCALE, Batch

pytestmark = pytest.mark.gpu


def check(b, err, heads=slice(None), floor=0.0):
    """floor: what an output may be off by besides, of the row's largest w |v|."""
    capi.mfa_check_device_errors(b.ws)
    for i in range(b.B):
        n = int(b.lens[i])
        ids = torch.from_numpy(b.table[i, :-(-n // PAGE)]).long().cuda()
        k, v = (c[ids].view(torch.float8_e4m3fn).double() * b.scales[j][ids].double().unsqueeze(-1) if b.fp8
                else c[ids].double() for j, c in enumerate(b.cache))
        k, v = k.reshape(-1, DIM)[:n], v.reshape(-1, DIM)[:n]
        logits = b.q[i, heads].double() @ k.T * SCALE
        lse = torch.logsumexp(logits, 1)
        w = torch.exp(logits - lse[:, None])
        out, size = w @ v, w @ v.abs()
        got = b.out[i, heads].double()
        top = (w * v.abs().amax(1)).amax(1, keepdim=True)
        bound = (2 ** -9 if b.fp8 else 2 ** -8) * size + 2 * err * size + 2 ** -8 * out.abs() + floor * top
        assert torch.isfinite(got).all(), i
        worst = ((got - out).abs() / bound).max()
        assert worst <= 1.0, (i, float(worst))
        assert float((b.lse[i, heads].double() - lse).abs().max()) <= err, i


@KV
def test_a_reference_that_moves_twice_in_a_unit(fp8):
    """One head has logits of -inf alone in the first two pages (a unit of the kernel) and finite ones behind them; the other
    heads' rise by 6 in the first half of a page and by 12 more in the second, so that O, which holds values of 2^16 from the
    first pages, is scaled twice in a unit: left out once, it would be off by 0.4. Logits are sums of 256 products below 16 *
    300 / 16: off by 2^-15 of 300."""
    b = Batch([3], [4], np.full(3, 4 * PAGE + 20), fp8, seed=41)
    pages = torch.from_numpy(b.table[0, :4]).long().cuda()
    b.q[:, :, 0] = 0.0
    b.q[:, 5, 0] = 2.0 ** 20
    b.q[:, :, 1] = 1.0
    if fp8:  # codes of at most 448 times a scale; 448 * 2^112 * 2^20 is past the fp32 range
        b.scales[0][~b.unused] = 2.0 ** -6
        b.cache[0][:, :, 0] = 0
        b.cache[0][:, :, 1] = 0
        step = {96.0: 0x44, 288.0: 0x51}  # 3, 9: times 32 of the scale below
    else:
        b.cache[0][:, :, 0] = 0.0
        b.cache[0][:, :, 1] = 0.0
    if fp8:
        b.scales[1][pages[:2]] *= 2.0 ** 16
        # the second dimension alone counts for these two pages: scale 32
        for half, code in ((slice(0, 32), step[96.0]), (slice(32, 64), step[288.0])):
            b.cache[0][pages[2:], half] = 0
            b.cache[0][pages[2:], half, 1] = code
            b.scales[0][pages[2:], half] = 32.0
        b.cache[0][pages[:2]] = 0
        b.cache[0][pages[:2], :, 0] = 0xFE
        b.scales[0][pages[:2]] = 2.0 ** 112
        for x in b.q:
            x[torch.arange(HEADS, device="cuda") != 5, 0] = 0.0
    else:
        b.cache[1][pages[:2]] *= 2.0 ** 16
        b.cache[0][pages[2:], :32, 1] = 96.0
        b.cache[0][pages[2:], 32:, 1] = 288.0
        b.cache[0][pages[:2], :, 0] = -2.0 ** 120
    b.call(hints=(0, 0))
    others = [h for h in range(HEADS) if h != 5]
    check(b, 300 * 2 ** -15, others)
    # the odd head does have no finite logit in the first unit
    b.d["lens"].fill_(2 * PAGE)
    b.d["pages"].fill_(2)
    b.call(hints=(0, 0))
    capi.mfa_check_device_errors(b.ws)
    assert not torch.isfinite(b.lse[:, 5]).any() and torch.isfinite(b.lse[:, others]).all()
