"""Chunk attention as a server calls it: a pool and page tables far larger than the step, which take the kernel whose pieces may
come in another order (a tile's rest last), first where the step's own pages fit L2 and the order stays, then where it does not."""
import numpy as np
import pytest
import torch

import test_gpu_chunk as base
from decode_attention_mfa_gb300 import capi
from test_gpu_chunk import KV, PAGE, Step, _poison

pytestmark = pytest.mark.gpu


class PoolStep(Step):
    """A step whose pool and tables have room for more than twice what L2 holds."""

    def __init__(self, new, held, kv="bf16", **kw):
        pages = {"bf16": 1400, "fp8": 2800, "fp4": 5600}[kv]
        super().__init__(new, held, kv, spare_cols=-(-pages // len(new)), **kw)
        fill = [float("nan")] if kv == "bf16" else [0x7F if kv == "fp8" else 0x77]
        more = lambda x, what: torch.cat([x, torch.full((pages, *x.shape[1:]), what, dtype=x.dtype, device="cuda")])  # noqa: E731
        self.cache = [more(c, fill[0]) for c in self.cache]
        self.scales = [more(c, float("nan")) for c in self.scales]
        self.num_pages += pages
        torch.cuda.synchronize()  # (calls on other streams read these)


AS_BEFORE = {
    "lengths": lambda kv: [base.test_one_chunk(n, h, kv) for n in (1, 2, 5, 13) for h in (0, 61, 124, 127, 128, 700)],
    "prompt": lambda kv: base.test_whole_prompt(513, kv),
    "long": lambda kv: base.test_long_context(40, 16384, kv),
    "ragged": base.test_ragged_batch,
    "decode": base.test_decode_tokens_only,
    "unseeing": base.test_more_tokens_than_positions,
    "peaked": base.test_peaked_rows,
    "rising": base.test_rising_and_falling_logits,
    "bad tables": base.test_bad_pages_and_lengths,
    "same bits": base.test_repeated_calls_give_the_same_bits,
    "graph": base.test_captured_and_replayed_with_other_lengths,
    "two at once": base.test_two_calls_at_once,
    "waits": base.test_waits_without_a_budget_give_up_and_the_next_call_is_whole,
    "later nan": lambda kv: [base.test_a_later_position_never_reaches_an_earlier_token(*c, float("nan"), kv)
                             for c in ((8, 60, 62), (8, 60, 67), (7, 121, 127), (131, 40, 100))],
    "later inf": lambda kv: base.test_a_later_position_never_reaches_an_earlier_token(6, 125, 128, float("inf"), kv),
    "seen nan": lambda kv: [base.test_a_value_that_is_no_number_reaches_every_token_that_sees_it(*c, float("nan"), kv)
                            for c in ((6, 125, 128), (3, 0, 2), (2000, 37, 1900))],
    "queries": lambda kv: base.test_query_rows_do_not_meet(kv, float("inf")),
}


@KV
@pytest.mark.parametrize("what", list(AS_BEFORE))
def test_as_with_a_pool_of_the_steps_size(what, kv, monkeypatch):
    monkeypatch.setattr(base, "Step", PoolStep)
    AS_BEFORE[what](kv)


@pytest.mark.parametrize("B", [31, 32, 33, 513])
def test_batch_sizes(B, monkeypatch):
    monkeypatch.setattr(base, "Step", PoolStep)
    base.test_batch_sizes(B)


@KV
def test_the_same_bits_in_a_pool_of_any_size(kv):
    """Where the step's pages fit L2 the order of the pieces is the same, and so is every bit."""
    args = ([37, 1, 200, 5, 0, 64], [900, 4000, 11, 64, 70, 0], kv)
    a, b = Step(*args, seed=41), PoolStep(*args, seed=41)
    a.call()
    b.call()
    assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse)


@KV
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_poisoned_ends_where_a_tiles_rest_comes_last(kv, what):
    """Sequences whose pages are more than L2 holds, the last position but one of each no number: tokens before it come out as
    without it, bit for bit, the two that see it do not."""
    new = [9, 1, 30, 61, 4, 17, 2, 9, 40, 0, 5, 12, 3, 700]
    s = Step(new, [30000 + 777 * (i % 5) for i in range(13)] + [9000], kv, seed=8, pad=2)
    s.call()
    s.check(which=[0, 4, 9, 12])
    clean, clean_lse = s.out.clone(), s.lse.clone()
    keep, hit = [], []
    for b, n in enumerate(new):
        rows = list(range(int(s.starts[b]), int(s.starts[b + 1])))
        if n < 2:
            keep += rows
            continue
        for i in range(2):
            _poison(s, i, b, int(s.lens[b]) - 2, what)
        keep += rows[:-2]
        hit += rows[-2:]
    s.call()
    capi.mfa_check_device_errors(s.ws)
    assert torch.equal(s.out[keep], clean[keep]) and torch.equal(s.lse[keep], clean_lse[keep])
    assert torch.isfinite(s.out[keep]).all()
    if what != what:
        assert torch.isnan(s.out[hit]).all()
    else:
        assert (~torch.isfinite(s.out[hit])).any(-1).all()


@KV
def test_values_no_numbers_at_the_ends_where_a_tiles_rest_comes_last(kv):
    """V alone: the LSE does not notice, every row that sees it has it, whichever of its tile's parts holds the tile's end."""
    s = Step([9, 30, 4, 17, 200], [40000, 31000, 30777, 42001, 50003], kv, seed=9)
    s.call()
    clean_lse = s.lse.clone()
    for b in range(s.B):
        _poison(s, 1, b, int(s.lens[b]) - 3, float("nan"))
    s.call()
    capi.mfa_check_device_errors(s.ws)
    for b in range(s.B):
        r = int(s.starts[b + 1])
        assert torch.isnan(s.out[r - 3:r]).all() and torch.isfinite(s.out[int(s.starts[b]):r - 3]).all()
        assert torch.equal(s.lse[int(s.starts[b]):r - 3], clean_lse[int(s.starts[b]):r - 3])
    # On an E2M1 cache the scale is NaN, its exponent 255, of which the weights take the most they can, 2^100: references are near
    # 112, exponents near -100, each rounded to half a step, 2^-18, as are the reference, the logarithm of the sum and their sum:
    # 4 * 2^-18 * ln 2 = 1.1e-5.
    assert float((s.lse - clean_lse).abs().max()) <= (1.1e-5 if kv == "fp4" else 0.0)


def test_the_pools_are_large_enough():
    """What the host's rule takes for more than L2 holds: units of two pages of K and V in 80 MB."""
    for kv, row in (("bf16", 512), ("fp8", 256), ("fp4", 128)):
        s = PoolStep([3, 1], [100, 7], kv)
        assert min(s.B * s.table.shape[1], s.num_pages) / 2 > (80 << 20) // (4 * PAGE * row)
        assert np.all(s.table[:, 2:] == -1)
