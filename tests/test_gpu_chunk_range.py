"""Attention of chunks of new tokens where the sizes of weights and values differ by far, each against the definition in 64
bits with tolerances from the roundings on the way (a rounding to bf16 is off by at most 2^-8 of the value, to f16 2^-11)."""
import numpy as np
import pytest
import torch

from decode_attention_mfa_gb300 import capi
from test_gpu_chunk import KV, Step, _with_logits

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
