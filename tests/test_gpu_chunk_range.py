"""Attention of chunks of new tokens where the sizes of weights and values differ by far, each against the definition in 64
bits with tolerances from the roundings on the way (a rounding to bf16 is off by at most 2^-8 of the value, to f16 2^-11)."""
import numpy as np
import pytest
import torch

from decode_attention_mfa_gb300 import capi
from test_gpu_chunk import KV, Step, _with_logits, values

pytestmark = pytest.mark.gpu
LN2 = float(np.log(2.0))


# ---------------------------------------------------------------- small weights behind long contexts
@KV
@pytest.mark.parametrize("at", [100, 131000])
@pytest.mark.parametrize("below", [20.0, 24.0, 25.5])
def test_many_small_weights_beside_a_large_one(below, at, kv):
    """One key of weight 1 whose value is 0, and 131375 of weight 2^-below whose value is 1, all rounded the same way: the output
    is what these have together. 304 tokens are as many row tiles as there are pairs of CTAs, so that a tile's keys are not
    many pairs' with references of their own."""
    s = Step([304], [131072], kv, seed=31)
    n = int(s.lens[0])
    logits = torch.full((n,), -below * LN2, device="cuda")
    logits[at] = 0.0
    v = torch.ones(n, device="cuda")
    v[at] = 0.0
    _with_logits(s, 0, logits, v)
    s.call()
    capi.mfa_check_device_errors(s.ws)
    s.starts[0] = 300  # the last four tokens, one tile's: the reference takes 64 heads of them
    s.new[0] = 4
    out, lse, _, _ = s.reference(0)
    got, got_lse = s.out[300:304].double(), s.lse[300:304].double()
    # the output's rounding, 2^-8; weights and values by 2^-8 (bf16) or 2^-11 each (f16, and 2^-11 for the scale) of their mean;
    # on a quantised cache a weight below 2^-18 is held to 2^-29 of the largest, 1, instead
    parts = 2 * 2 ** -8 if kv == "bf16" else 3 * 2 ** -11
    bound = (2 ** -8 + parts) * out.abs() + (0 if kv == "bf16" else n * 2 ** -29)
    assert ((got - out).abs() <= bound).all(), float(((got - out).abs() / bound).max())
    assert float((got_lse - lse).abs().max()) <= 1e-4  # fp32 sums of 131375 weights, 2^-24 of each partial sum


@KV
@pytest.mark.parametrize("new,held", [(1, 262143), (3, 131072), (2, 200001)])
def test_long_contexts(new, held, kv):
    Step([new], [held], kv, seed=held).run()


# ---------------------------------------------------------------- values of any size
@pytest.mark.parametrize("power", [-108, -90, -40, 40, 90, 110, 127])
@pytest.mark.parametrize("rise", [0.0, 9.0, 14.0, 16.5, 30.0, -30.0])
@pytest.mark.parametrize("new,held", [(5, 40000), (70, 300), (304, 30000)])
def test_values_of_any_size(new, held, rise, power):
    """Values up to the largest bf16, behind logits that are 2^(rise / ln 2) larger from the second unit of 128 keys on, so that
    weights grow as far as they may before the reference moves, and then stay there: no finite value gives an infinite output."""
    s = Step([new], [held], seed=32)
    n = int(s.lens[0])
    logits = torch.full((n,), rise, device="cuda")
    logits[:128] = 0.0
    v = torch.full((n,), 1.9921875 * 2.0 ** power, device="cuda")  # 2^127: the largest bf16
    if held != 300:
        v[::3] *= -1.0
    _with_logits(s, 0, logits, v)
    s.call()
    if new > 70:  # the reference takes 64 heads of each token that it is asked for
        s.starts[0], s.new[0] = new - 4, 4
        s.out[:new - 4] = 7.0
        s.lse[:new - 4] = 7.0
    s.check()


@pytest.mark.parametrize("steps", [1, 7, 90])
def test_sums_near_what_moves_a_reference(steps):
    """Weights that grow by 2^20 in all, in steps between whole units: each unit's sum, and what the units before it left, is near
    what moves the reference (a weight of 2^-9 each), behind it again, and much smaller ones follow to the end."""
    s = Step([9, 304], [60000, 9000], seed=35)
    for b in range(2):
        n = int(s.lens[b])
        unit = torch.arange(n, device="cuda") // 128
        logits = LN2 * (20.0 * (unit.clamp(max=steps) / steps) - 45.0 * (unit > 2 * steps))
        logits += 0.3 * torch.randn(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(steps))
        _with_logits(s, b, logits)
    s.cache[1] *= 2.0 ** 124
    s.call()
    s.check(which=[0])
    s.starts[1], s.new[1] = int(s.starts[2]) - 4, 4
    out, lse, top, _ = s.reference(1)
    got, got_lse = s.out[s.starts[1]:s.starts[2]].double(), s.lse[s.starts[1]:s.starts[2]].double()
    assert ((got - out).abs() <= 2 ** -8 * (top + out.abs()) + 2 ** -12 * top).all()
    assert float((got_lse - lse).abs().max()) <= 1e-3


@pytest.mark.parametrize("sigma", [1.0, 4.0])
def test_large_values_and_logits_of_any_spread(sigma):
    s = Step([40, 1], [20000, 20000], seed=33, q_scale=sigma)
    s.cache[1] *= 2.0 ** 124
    s.call()
    capi.mfa_check_device_errors(s.ws)
    for b in range(2):
        out, lse, top, _ = s.reference(b)
        got, got_lse = (x[s.starts[b]:s.starts[b + 1]].double() for x in (s.out, s.lse))
        # besides the weights' and the output's rounding, the logits' fp32 sums: 2^-15 of scale * sum |q k|, about 10 sigma
        assert ((got - out).abs() <= 2 ** -8 * (top + out.abs()) + 2 * 10 * sigma * 2 ** -15 * top).all(), b
        assert float((got_lse - lse).abs().max()) <= 1e-3 * sigma, b


@pytest.mark.parametrize("kv,power", [("fp8", 100), ("fp8", 101), ("fp8", 104), ("fp8", 112), ("fp4", 100), ("fp4", 110), ("fp4", 112), ("fp4", 115)])
@pytest.mark.parametrize("new,held,at", [(7, 121, 125), (3, 0, 2), (4, 0, 0), (6, 125, 128), (40, 300, 50), (2, 5000, 5001)])
def test_value_scales_at_the_end_of_their_range(new, held, at, kv, power):
    """One position's V scale is the largest that the weights can take, 2^101 (E2M1 2^110), or above: the tokens that see it get
    the attention, or no number where f16 does not hold a value above, and never a finite output without it; the others do not
    notice it."""
    s = Step([new], [held], kv, seed=34)
    s.call()
    clean = s.out.clone()
    s.scales[1].view(-1)[s.row(0, at)] = 2.0 ** power
    s.call()
    capi.mfa_check_device_errors(s.ws)
    out, _, top, limit = s.reference(0)
    sees = limit > at
    assert sees.any() and torch.equal(s.out[~sees], clean[~sees])
    got = s.out.double()[sees]
    # as f16: the codes times the scale less the 2^100 that the weight takes at most, times 2^6 (E2M1 2^3)
    code = values(s.cache[1].view(-1, s.cache[1].shape[-1])[s.row(0, at)], torch.ones((), device="cuda"), kv)
    held_as = code * torch.tensor(2.0 ** (power - 100 + (6 if kv == "fp8" else 3)), device="cuda").half().double()
    fits = held_as.abs() < 65520
    assert fits.all() or power > (101 if kv == "fp8" else 110)
    # weights, values and their scales as f16, another 2^-8 of the largest value (that position's)
    bound = 2 ** -8 * (2 * top[sees] + out[sees].abs()) + 2 ** -12 * top[sees]
    assert ((got - out[sees]).abs() <= bound)[..., fits].all()
    assert not torch.isfinite(got[..., ~fits]).any()
