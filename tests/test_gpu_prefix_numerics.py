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


def keyed(n, pages, own, fp8, seed):
    """A batch whose logits are set key by key, and normal ones to begin with. Returns it and set_keys(logit, power): both
    [num_pages, 64]; K's rows become their second dimension alone, V's rows are taken times 2^power."""
    b = Batch([n], [pages], np.full(n, pages * PAGE + own), fp8, seed=seed)
    b.q[:, :, 1] = 1.0
    used = ~b.unused

    def set_keys(logit, power):
        k = (logit / SCALE)[used]
        if fp8:
            b.cache[0][used] = 0
            codes = b.cache[0][used]
            codes[:, 1] = torch.where(k < 0, 0xB8, 0x38).to(torch.uint8)
            b.cache[0][used] = codes
            b.scales[0][used] = k.abs()
            b.scales[1][used] = torch.ldexp(b.scales[1][used], power[used])
        else:
            rows = torch.zeros((int(used.sum()), DIM), device="cuda")
            rows[:, 1] = k
            b.cache[0][used] = rows.bfloat16()
            b.cache[1][used] = torch.ldexp(b.cache[1][used].float(), power[used].unsqueeze(-1)).bfloat16()

    gen = torch.Generator(device="cuda").manual_seed(seed)
    shape = (b.num_pages, PAGE)
    return b, set_keys, torch.randn(shape, generator=gen, device="cuda"), lambda lo, hi: torch.randint(
        lo, hi + 1, shape, generator=gen, device="cuda")


@KV
@pytest.mark.parametrize("power", [12, 24, 60])
def test_large_values_without_weight_leave_small_ones_whole(power, fp8):
    """On every page one value of 2^power times the others' size at a logit of -56 (2^-81): it counts for nothing, or for all
    there is, and the others keep their bits either way. Logits of up to 56 are single products."""
    b, set_keys, logit, _ = keyed(3, 5, 100, fp8, 43)
    p = torch.zeros((b.num_pages, PAGE), device="cuda", dtype=torch.int64)
    logit[:, 5] = -56.0
    p[:, 5] = power
    set_keys(logit, p)
    b.call()
    check(b, 56 * 2 ** -15)


@KV
@pytest.mark.parametrize("power", [-6, -10, -14])
def test_rows_of_zeros_beside_small_values(power, fp8):
    """Values of nothing but zeros, whose scale is 1 as the append writes it, at logits 4 or more above the others', whose
    values are small: the zeros add nothing, and take nothing from the others. E4M3: a weight is a multiple of 2^-24 where
    the zeros' is 2^4, the others' largest 2^-5.8 of that (logits of 7 and 3) and, of values below 2^-16 of a scale, 2^x less:
    their scales are at least 2^-9 (the largest of 256 normal values over 448, times exp(-1.5)) times 2^power, so x is at
    least power + 7 where that is negative. Some 400 keys are then off by 2^-25 of 2^(4 - 5.8 + x) each, and V' of two keys
    differ by at most 2 where x is not 0, and by 2^7 where it is: 2^(8.7 - 25 + 1.8 + 7) = 2^-7.5 at power -6, and
    2^(8.7 - 25 + 1.8 + 1 - x) = 2^(-13.5 - x) below."""
    b, set_keys, logit, _ = keyed(3, 5, 100, fp8, 44)
    logit.clamp_(-3.0, 3.0)
    logit[:, ::16] = 7.0
    set_keys(logit, torch.full((b.num_pages, PAGE), power, device="cuda"))
    rows = torch.zeros_like(b.unused)
    rows[:, ::16] = True
    rows &= ~b.unused
    b.cache[1][rows] = 0
    if fp8:
        b.scales[1][rows] = 1.0
    b.call()
    check(b, 7 * 2 ** -15, floor=(2.0 ** -7.5 if power == -6 else 2.0 ** (-13.5 - (power + 7))) if fp8 else 0.0)


@KV
@pytest.mark.parametrize("lo,hi", [(-40, 20), (-110, 90)])
def test_values_of_all_sizes_in_a_page(lo, hi, fp8):
    """Sizes drawn key by key over a range that no 16-bit format holds; some scales are zero. The result is the large ones',
    and the rest is off by 2^-28 of them for each of some 400 keys (a step of 2^-25 of a weight where the largest is 2^4 or
    more, and a value twice as large)."""
    b, set_keys, logit, draw = keyed(3, 5, 100, fp8, 45)
    set_keys(logit, draw(lo, hi))
    if fp8:
        b.scales[1][:, 7::16] *= 0.0
        b.scales[1][b.unused] = float("nan")
    b.call()
    check(b, 5 * 2 ** -15, floor=2.0 ** -19)


@KV
@pytest.mark.parametrize("lo,hi", [(-16, 0), (-40, 20)])
def test_sizes_that_weights_make_up_for(lo, hi, fp8):
    """The smaller the value the larger its weight, so that each of some 400 keys counts as much as any other. Logits of up to
    28 are single products. (bf16: the weights span 2^60, which its exponents hold.)"""
    b, set_keys, logit, draw = keyed(3, 5, 100, fp8, 46)
    power = draw(lo, hi)
    set_keys(logit - power * float(np.log(2.0)), power)
    b.call()
    check(b, 32 * 2 ** -15)
