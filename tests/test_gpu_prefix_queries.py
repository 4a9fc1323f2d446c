"""Shared-prefix decode attention with queries at the end of their range."""
import pytest
import torch

from decode_attention_mfa_gb300 import capi
from test_gpu_prefix import HEADS, KV, SCALE, Batch, lens_of

pytestmark = pytest.mark.gpu


@KV
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("sizes,pages", [([6], [4]), ([3, 1], [2, 0])])
def test_a_query_that_is_no_number_makes_its_own_row_so_and_no_other(sizes, pages, what, fp8):
    b = Batch(sizes, pages, lens_of(sizes, pages, 150, 3), fp8, seed=51)
    b.d["lens"].clamp_(min=1)
    b.q[1, 7, 3] = what
    b.q[-1, 63, 200] = what
    b.call()
    capi.mfa_check_device_errors(b.ws)
    bad = torch.zeros((b.B, HEADS), dtype=torch.bool, device="cuda")
    bad[1, 7] = bad[-1, 63] = True
    assert torch.isnan(b.out[bad]).all() and torch.isnan(b.lse[bad]).all()
    assert torch.isfinite(b.out[~bad]).all() and torch.isfinite(b.lse[~bad]).all()


@KV
@pytest.mark.parametrize("power", [-126, -60, 60, 100])
def test_query_norms(power, fp8):
    """Queries of any power of two, the scale undoing it where fp32 holds it."""
    b = Batch([5], [3], lens_of([5], [3], 150, 4), fp8, seed=52)
    b.q.copy_((b.q.double() * 2.0 ** power).bfloat16())
    b.run(scale=SCALE * 2.0 ** min(max(-power, -100), 120))


def test_the_largest_queries():
    """Rows with the largest bf16 number, 1.992 * 2^127, on an E4M3 cache, whose products of codes are far from fp32's range. The
    scale, 2^-131, is below fp32's normal range: times log2 e it is off by 2^-19 of itself, the logits (below 40) by 8e-5."""
    b = Batch([5], [3], lens_of([5], [3], 150, 4), True, seed=53)
    b.q.clamp_(-1.9921875, 1.9921875)
    b.q[:, ::2, 0] = 1.9921875
    b.q *= 2.0 ** 126
    b.q *= 2.0
    assert torch.isfinite(b.q).all()
    b.run(scale=SCALE * 2.0 ** -127)
