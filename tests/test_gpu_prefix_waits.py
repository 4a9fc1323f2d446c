"""The shared-prefix kernel's way out when a wait inside it gives up."""
import pytest
import torch

from decode_attention_mfa_gb300 import capi
from test_gpu_prefix import KV, Batch, lens_of

pytestmark = pytest.mark.gpu


@KV
def test_waits_without_a_budget_give_up_and_the_next_call_is_whole(fp8):
    """Ten calls whose waits have no budget: a call is right or reports a wait that gave up, at least one of them does report
    it (a copy takes longer than two looks at its barrier), and a call with the usual budget behind each is whole."""
    sizes, pages = [6, 5], [40, 30]
    b = Batch(sizes, pages, lens_of(sizes, pages, 200, 6), fp8, seed=42)
    b.workspace()
    gave_up = 0
    try:
        for _ in range(10):
            capi.mfa_set_wait_budget_ns(0)
            b.call()
            torch.cuda.synchronize()
            capi.mfa_set_wait_budget_ns(2_000_000_000)
            try:
                b.check()
            except capi.MFAError as e:
                assert e.status == 7
                gave_up += 1
            b.out.fill_(7.0)
            b.run()
    finally:
        capi.mfa_set_wait_budget_ns(2_000_000_000)
    assert gave_up >= 1
