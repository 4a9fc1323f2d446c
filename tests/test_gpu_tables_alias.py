"""Page tables whose lengths or whose count of free pages alone replace their inputs, over one block and over several: every
block has read both before either is written. Whole numbers, compared for equality."""
import numpy as np
import pytest
import torch

from decode_attention_mfa_gb300 import capi
from test_gpu_tables import POISON, dev, errors, make, release_plain, reserve_plain, workspace

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,longest_new", [(9, 30), (1024, 400)])
@pytest.mark.parametrize("lens_replaced", [False, True])
def test_one_of_the_outputs_replaces_its_input(batch, longest_new, lens_replaced):
    rng = np.random.default_rng(batch)
    lens, table, free, n_free = make(rng, batch, 40, 1500, extra=batch * 8)
    n_new = rng.integers(0, longest_new, batch).astype(np.int32)
    most = int(n_new.sum()) + 5
    ws = workspace()
    d_lens, d_n, d_table, d_free = dev(lens), dev([n_free]), dev(table), dev(free)
    lens_out = d_lens if lens_replaced else torch.full_like(d_lens, POISON)
    n_out = torch.full_like(d_n, POISON) if lens_replaced else d_n
    starts = torch.full((batch + 1,), POISON, dtype=torch.int32, device="cuda")
    slots = torch.full((most,), POISON, dtype=torch.int64, device="cuda")
    capi.mfa_reserve_pages(dev(n_new), d_lens, d_table, d_free, d_n, batch, table.shape[1], len(free), most, starts, slots,
                           lens_out, n_out, ws)
    table, want_slots, want_starts, want_lens, left, err = reserve_plain(n_new, lens, table, free, n_free, table.shape[1], most)
    assert (d_table.cpu().numpy() == table).all() and (slots.cpu().numpy() == want_slots).all()
    assert (starts.cpu().numpy() == want_starts).all()
    assert (lens_out.cpu().numpy() == want_lens).all() and n_out.tolist() == [left] and errors(ws) == err
    # the input that was not replaced is as it was
    assert d_n.tolist() == [n_free] if lens_replaced else (d_lens.cpu().numpy() == lens).all()

    finished = (rng.random(batch) < 0.5).astype(np.int32)
    d_lens, d_n = dev(want_lens), dev([left])
    lens_out = d_lens if lens_replaced else torch.full_like(d_lens, POISON)
    n_out = torch.full_like(d_n, POISON) if lens_replaced else d_n
    capi.mfa_release_pages(dev(finished), None, d_lens, d_table, d_free, d_n, batch, table.shape[1], len(free), lens_out, n_out,
                           ws)
    want_free, after, top, err = release_plain(finished, None, want_lens, table, free, left, table.shape[1])
    assert (d_free.cpu().numpy() == want_free).all()
    assert (lens_out.cpu().numpy() == after).all() and n_out.tolist() == [top] and errors(ws) == err
    assert d_n.tolist() == [left] if lens_replaced else (d_lens.cpu().numpy() == want_lens).all()
