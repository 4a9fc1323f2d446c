"""Page tables, slot maps and slot appends (mfa_reserve_pages, mfa_kv_append_slots*, mfa_release_pages)
against plain implementations on the host. Everything here is a whole number or a copy, so results are
compared for equality."""
import numpy as np
import pytest
import torch

from decode_attention_mfa_gb300 import capi

pytestmark = pytest.mark.gpu
PAGE = 64
POISON = -77


def reserve_plain(n_new, lens, table, free, n_free, max_pages, max_new):
    """The definition, one request after the other. Returns outputs and the error bits."""
    table, err, bad_page = table.copy(), 0, False
    starts, slots, out = [0], np.full(max_new, -1, np.int64), lens.copy()
    wanted = taken = 0
    num_pages = len(free)
    for b, (n, length) in enumerate(zip(n_new.tolist(), lens.tolist())):
        err |= 2 if n < 0 else 0
        starts.append(starts[-1] + max(n, 0))
        if n < 0 or length < 0 or length + n > max_pages * PAGE or starts[-1] > max_new:
            err |= 2
            continue
        held, after = -(-length // PAGE), -(-(length + n) // PAGE)
        wanted += after - held
        if after > held and wanted > n_free:
            err |= 8
            continue
        for j in range(held, after):
            table[b, j] = free[n_free - 1 - taken]
            taken += 1
        for t in range(n):
            page = int(table[b, (length + t) // PAGE])
            if 0 <= page < num_pages:
                slots[starts[b] + t] = page * PAGE + (length + t) % PAGE
            else:
                bad_page = True
        out[b] = length + n
    bad_page |= any(not 0 <= p < num_pages for p in free[n_free - taken:n_free].tolist())
    return table, slots, np.minimum(starts, 2 ** 31 - 1), out, n_free - taken, err | (1 if bad_page else 0)


def release_plain(finished, keep, lens, table, free, n_free, max_pages):
    free, out, err, top, wanted = free.copy(), lens.copy(), 0, n_free, n_free
    for b, length in enumerate(lens.tolist()):
        if not finished[b]:
            continue
        k = 0 if keep is None else int(keep[b])
        if length < 0 or length > max_pages * PAGE or k < 0:
            err |= 2
            continue
        held = -(-length // PAGE)
        k = min(k, held)
        wanted += held - k
        if held > k and wanted > len(free):
            err |= 2
            continue
        for j in range(k, held):
            err |= 0 if 0 <= table[b, j] < len(free) else 1
            free[top] = table[b, j]
            top += 1
        out[b] = min(length, k * PAGE)
    return free, out, top, err


def make(rng, batch, max_pages, longest, extra=None):
    lens = rng.integers(0, min(longest, max_pages * PAGE) + 1, batch).astype(np.int32)
    used = -(-lens // PAGE)
    extra = int(rng.integers(0, 3 * batch + 2)) if extra is None else extra
    total = int(used.sum()) + extra + 1
    order = rng.permutation(total).astype(np.int32)
    table = np.full((batch, max_pages), POISON, np.int32)
    at = 0
    for b in range(batch):
        table[b, :used[b]] = order[at:at + used[b]]
        at += used[b]
    free = np.full(total, POISON, np.int32)
    free[:extra] = order[at:at + extra]
    return lens, table, free, extra


def dev(x, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype).cuda()


def workspace():
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    capi.mfa_workspace_init(ws, 256)
    return ws


def errors(ws):
    return int(ws[:4].view(torch.int32).item())


def reserve(n_new, lens, table, free, n_free, max_new, ws, alias=False, stream=None):
    batch, max_pages = table.shape
    d = dict(new=dev(n_new), lens=dev(lens), table=dev(table), free=dev(free), n=dev([n_free]),
             starts=torch.full((batch + 1,), POISON, dtype=torch.int32, device="cuda"),
             slots=torch.full((max_new + 3,), POISON, dtype=torch.int64, device="cuda"))
    d["lens_out"] = d["lens"] if alias else torch.full_like(d["lens"], POISON)
    d["n_out"] = d["n"] if alias else torch.full_like(d["n"], POISON)
    capi.mfa_reserve_pages(d["new"], d["lens"], d["table"], d["free"], d["n"], batch, max_pages, len(free), max_new,
                           d["starts"], d["slots"], d["lens_out"], d["n_out"], ws, stream)
    return d


def check_reserve(n_new, lens, table, free, n_free, max_new, alias=False):
    ws = workspace()
    d = reserve(n_new, lens, table, free, n_free, max_new, ws, alias)
    t, slots, starts, out, left, err = reserve_plain(n_new, lens, table, free, n_free, table.shape[1], max_new)
    assert (d["table"].cpu().numpy() == t).all()
    assert (d["slots"].cpu().numpy() == np.concatenate([slots, [POISON] * 3])).all()
    assert (d["starts"].cpu().numpy() == starts).all()
    assert (d["lens_out"].cpu().numpy() == out).all()
    assert int(d["n_out"].item()) == left
    assert errors(ws) == err
    assert int(ws[64:68].view(torch.int32).item()) == 0  # the arrival counter is back at zero
    return d


@pytest.mark.parametrize("batch", [1, 2, 31, 33, 511, 512, 513, 1024])
@pytest.mark.parametrize("alias", [False, True])
def test_reserve_matches_plain(batch, alias):
    rng = np.random.default_rng(batch)
    lens, table, free, n_free = make(rng, batch, 40, 1500, extra=batch * 3)
    n_new = rng.integers(0, 120, batch).astype(np.int32)
    n_new[rng.random(batch) < 0.2] = 0
    lens[rng.random(batch) < 0.1] &= ~63  # full last pages
    check_reserve(n_new, lens, table, free, n_free, int(n_new.sum()) + 70, alias)


def test_reserve_many_tokens_over_several_blocks():
    rng = np.random.default_rng(5)
    lens, table, free, n_free = make(rng, 300, 64, 700, extra=300 * 16)
    n_new = rng.integers(0, 900, 300).astype(np.int32)
    check_reserve(n_new, lens, table, free, n_free, int(n_new.sum()), alias=True)


def test_reserve_single_tokens_and_none():
    rng = np.random.default_rng(6)
    lens, table, free, n_free = make(rng, 128, 20, 1000, extra=128)
    check_reserve(np.ones(128, np.int32), lens, table, free, n_free, 128)
    check_reserve(np.zeros(128, np.int32), lens, table, free, n_free, 0)
    check_reserve(np.zeros(128, np.int32), lens, table, free, n_free, 9)


def test_reserve_with_too_few_pages_serves_the_first():
    rng = np.random.default_rng(7)
    for extra in (0, 1, 17):
        lens, table, free, n_free = make(rng, 90, 20, 600, extra=extra)
        check_reserve(rng.integers(0, 80, 90).astype(np.int32), lens, table, free, n_free, 90 * 80)


def test_reserve_refuses_requests_one_by_one():
    """Bad lengths and counts, rows past max_new and a full table leave their request as it is; the others are served."""
    rng = np.random.default_rng(8)
    lens, table, free, n_free = make(rng, 40, 10, 500, extra=200)
    n_new = rng.integers(1, 60, 40).astype(np.int32)
    n_new[3], lens[7], lens[11], n_new[13], n_new[21] = -4, -1, 10 * PAGE + 1, 10 * PAGE + 1, 2 ** 31 - 1
    lens[19], n_new[19] = 10 * PAGE, 1
    check_reserve(n_new, lens, table, free, n_free, 2000)
    lens[30], n_new[21] = 5, 4
    check_reserve(n_new, lens, table, free, n_free, int(np.maximum(n_new, 0)[:32].sum()) - 1)


def test_reserve_reports_bad_page_ids():
    rng = np.random.default_rng(9)
    lens, table, free, n_free = make(rng, 12, 10, 300, extra=40)
    lens[2] = 70
    table[2, 1] = len(free)
    free[n_free - 2] = -5
    check_reserve(rng.integers(1, 100, 12).astype(np.int32), lens, table, free, n_free, 1300)
    # a stack pointer outside its array is reported and read as the nearest valid one
    ws = workspace()
    d = reserve(np.zeros(12, np.int32), lens, table, free, len(free) + 5, 0, ws)
    assert errors(ws) == 2 and int(d["n_out"].item()) == len(free)


@pytest.mark.parametrize("batch,share,keep", [(1, 1.0, None), (64, 0.5, 3), (700, 0.1, 0), (1024, 1.0, 5), (9, 0.0, None)])
@pytest.mark.parametrize("alias", [False, True])
def test_release_matches_plain(batch, share, keep, alias):
    rng = np.random.default_rng(batch)
    lens, table, free, n_free = make(rng, batch, 30, 1900)
    finished = (rng.random(batch) < share).astype(np.int32) * 5
    kept = None if keep is None else rng.integers(0, keep + 1, batch).astype(np.int32)
    check_release(finished, kept, lens, table, free, n_free, alias)


def check_release(finished, keep, lens, table, free, n_free, alias=False):
    batch, max_pages = table.shape
    ws = workspace()
    d_free, d_lens, d_n, d_table = dev(free), dev(lens), dev([n_free]), dev(table)
    lo = d_lens if alias else torch.full_like(d_lens, POISON)
    no = d_n if alias else torch.full_like(d_n, POISON)
    capi.mfa_release_pages(dev(finished), None if keep is None else dev(keep), d_lens, d_table, d_free, d_n, batch,
                           max_pages, len(free), lo, no, ws)
    f, out, top, err = release_plain(finished, keep, lens, table, free, n_free, max_pages)
    assert (d_free.cpu().numpy() == f).all()
    assert (lo.cpu().numpy() == out).all()
    assert int(no.item()) == top
    assert errors(ws) == err
    assert (d_table.cpu().numpy() == table).all()


def test_release_refusals():
    rng = np.random.default_rng(10)
    lens, table, free, n_free = make(rng, 20, 10, 600, extra=5)
    finished = np.ones(20, np.int32)
    keep = rng.integers(0, 3, 20).astype(np.int32)
    lens[3], lens[5], keep[9], lens[11] = -1, 10 * PAGE + 1, -2, 200
    table[11, int(max(0, keep[11]))] = -1
    check_release(finished, keep, lens, table, free, n_free)
    # more pages than the stack's array holds: the first requests are taken
    lens, table, free, n_free = make(rng, 20, 10, 600, extra=5)
    check_release(finished, None, lens, table, free[:40].copy(), n_free)


def slots_case(rows, pages, seed):
    rng = np.random.default_rng(seed)
    slots = rng.permutation(pages * PAGE)[:rows].astype(np.int64)
    slots[rng.random(rows) < 0.1] = -1
    return slots


@pytest.mark.parametrize("rows", [1, 3, 4, 5, 129, 2000])
@pytest.mark.parametrize("stride", [256, 512, 264])
def test_append_slots_bf16(rows, stride):
    slots = slots_case(rows, 40, rows)
    kv = torch.randn((rows, stride), device="cuda").bfloat16()
    k = kv[:, :256]
    v = torch.randn((rows, 256), device="cuda").bfloat16()
    kc = torch.full((40, PAGE, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    ws = workspace()
    capi.mfa_kv_append_slots(k, v, stride, 256, dev(slots, torch.int64), rows, kc, vc, 40, ws)
    rk, rv = torch.full_like(kc, 7.0).view(-1, 256), torch.full_like(vc, 7.0).view(-1, 256)
    ok = slots >= 0
    rk[slots[ok]], rv[slots[ok]] = k[ok], v[ok]
    assert torch.equal(kc.view(-1, 256), rk) and torch.equal(vc.view(-1, 256), rv)
    assert errors(ws) == 0


def test_append_slots_out_of_range_and_special_values():
    """A slot past the cache is skipped and reported; infinities, NaN and signed zeros are copied as they are."""
    k = torch.randn((6, 256), device="cuda").bfloat16()
    k[0, :4] = torch.tensor([float("inf"), float("-inf"), float("nan"), -0.0])
    kc = torch.zeros((2, PAGE, 256), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    ws = workspace()
    slots = torch.tensor([127, 128, 2 ** 40, -2 ** 62, 5, -1], device="cuda")
    capi.mfa_kv_append_slots(k, k, 256, 256, slots, 6, kc, vc, 2, ws)
    want = torch.zeros_like(kc).view(-1, 256)
    want[127], want[5] = k[0], k[4]
    assert torch.equal(kc.view(torch.int16).view(-1, 256), want.view(torch.int16)) and torch.equal(vc.view(torch.int16), kc.view(torch.int16))
    assert errors(ws) == 1
    with pytest.raises(capi.MFAError) as e:
        capi.mfa_check_device_errors(ws)
    assert e.value.status == 5
    capi.mfa_kv_append_slots(k, k, 256, 256, slots, 0, kc, vc, 2, ws)  # no rows: nothing to do


@pytest.mark.parametrize("rows", [1, 7, 500])
def test_append_slots_fp8_equals_the_append_by_lengths(rows):
    """The same rows through mfa_kv_append_fp8 give the same codes and scales, bit for bit."""
    pages = -(-rows // PAGE)
    k = torch.randn((rows, 256), device="cuda").bfloat16() * 3
    v = torch.randn((rows, 2, 256), device="cuda").bfloat16()[:, 1]
    k[0] = 0  # a zero row: scale 1
    a = [torch.zeros((pages, PAGE, 256), dtype=torch.uint8, device="cuda") for _ in range(4)]
    s = [torch.zeros((pages, PAGE), device="cuda") for _ in range(4)]
    order = torch.randperm(pages, device="cuda").int()
    ws = workspace()
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    capi.mfa_kv_append_fp8(k, v.contiguous(), rows, a[0], a[1], s[0], s[1], order.view(1, -1), lens, 1, pages, pages, ws)
    at = torch.arange(rows, device="cuda")
    slots = order.long()[at // PAGE] * PAGE + at % PAGE
    capi.mfa_kv_append_slots_fp8(k, v, 256, 512, slots, rows, a[2], a[3], s[2], s[3], pages, ws)
    for i in range(2):
        assert torch.equal(a[i], a[i + 2]) and torch.equal(s[i], s[i + 2])


def test_serving_loop_captured_and_replayed():
    """reserve -> append -> attention in place, captured once and replayed on another stream: lengths, tables and
    caches after six steps are those of the host's bookkeeping, and release returns every page."""
    B, max_pages, num_pages = 5, 6, 32
    rng = np.random.default_rng(3)
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(num_pages, device="cuda").int()
    pages0 = free.clone().cpu()
    n_free = dev([num_pages])
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    new = torch.zeros(B, dtype=torch.int32, device="cuda")
    rows = 5 * 40
    k = torch.zeros((rows, 256), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    kc = torch.zeros((num_pages, PAGE, 256), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    q = torch.randn((B, 64, 256), device="cuda").bfloat16()
    out, lse = torch.zeros_like(q), torch.zeros((B, 64), device="cuda")
    starts = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    slots = torch.zeros(rows, dtype=torch.int64, device="cuda")
    nbytes = capi.mfa_decode_workspace_bytes(B, 384)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        capi.mfa_workspace_init(ws, nbytes)

        def step():
            capi.mfa_reserve_pages(new, lens, table, free, n_free, B, max_pages, num_pages, rows, starts, slots, lens,
                                   n_free, ws)
            capi.mfa_kv_append_slots(k, v, 256, 256, slots, rows, kc, vc, num_pages, ws)
            capi.mfa_decode_attention(q, kc, vc, table, lens, out, lse, 1 / 16, B, max_pages, num_pages, 384, ws, nbytes)

        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
        held = [np.zeros((0, 256), np.float32) for _ in range(B)]
        for _ in range(6):
            count = rng.integers(0, 41, B).astype(np.int32)
            rows_now = torch.randn((rows, 256)).bfloat16()
            new.copy_(torch.from_numpy(count))
            k.copy_(rows_now)
            v.copy_(rows_now * 2)
            graph.replay()
            at = np.concatenate([[0], np.cumsum(count)])
            held = [np.concatenate([h, rows_now[at[b]:at[b + 1]].float().numpy()]) for b, h in enumerate(held)]
        stream.synchronize()
        capi.mfa_check_device_errors(ws)
        assert lens.tolist() == [len(h) for h in held]
        for b, h in enumerate(held):
            ids = table[b, :-(-len(h) // PAGE)].long()
            got = kc[ids].reshape(-1, 256)[:len(h)].float().cpu().numpy()
            assert (got == h).all() and (vc[ids].reshape(-1, 256)[:len(h)].float().cpu().numpy() == 2 * h).all()
            if len(h):
                logits = q[b].double().cpu().numpy() @ h.T.astype(np.float64) / 16
                w = np.exp(logits - logits.max(1, keepdims=True))
                ref = (w / w.sum(1, keepdims=True)) @ (2.0 * h)
                # bf16 output and bf16 P: half a step each, 2^-8, of |values| that average below the largest
                assert np.abs(out[b].float().cpu().numpy() - ref).max() <= 2 ** -7 * np.abs(2 * h).max()
        capi.mfa_release_pages(torch.ones(B, dtype=torch.int32, device="cuda"), None, lens, table, free, n_free, B,
                               max_pages, num_pages, lens, n_free, ws)
        stream.synchronize()
    assert lens.tolist() == [0] * B and int(n_free.item()) == num_pages
    assert sorted(free.tolist()) == sorted(pages0.tolist())


def test_append_slots_fp8_codes_of_all_kinds_of_rows():
    """Codes and scales are those of mfa_kv_append_fp8, bit for bit, over 40,000 random rows (more than the sizes at which
    a warp takes one row) and rows of every scale, with signed zeros, subnormals, infinities and NaN among their values."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    rows, pages = 40960, 640
    k = torch.randn((rows, 256), generator=gen, device="cuda") * torch.exp2(torch.randint(-20, 20, (rows, 1), generator=gen, device="cuda"))
    v = torch.randn((rows, 256), generator=gen, device="cuda") * torch.rand((rows, 256), generator=gen, device="cuda") ** 8
    k, v = k.bfloat16(), v.bfloat16()
    exps = torch.arange(-132, 128, device="cuda").double()  # 260 rows, one of each scale that bf16 has
    v[:260] = (torch.randn((260, 256), generator=gen, device="cuda").double().clamp(-1, 1) * torch.exp2(exps).unsqueeze(1)).bfloat16()
    v[300:310, ::3] = -0.0
    v[310], v[311] = 0.0, -0.0
    v[312, 5], v[313, 7], v[314, 9] = float("inf"), float("-inf"), float("nan")
    v[315] = float("nan")
    a = [torch.zeros((pages, PAGE, 256), dtype=torch.uint8, device="cuda") for _ in range(4)]
    s = [torch.zeros((pages, PAGE), device="cuda") for _ in range(4)]
    ws = workspace()
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    table = torch.arange(pages, device="cuda").int().view(1, -1)
    capi.mfa_kv_append_fp8(k, v, rows, a[0], a[1], s[0], s[1], table, lens, 1, pages, pages, ws)
    capi.mfa_kv_append_slots_fp8(k, v, 256, 256, torch.arange(rows, device="cuda"), rows, a[2], a[3], s[2], s[3], pages, ws)
    for i in range(2):
        assert torch.equal(s[i].view(torch.int32), s[i + 2].view(torch.int32))
        assert torch.equal(a[i], a[i + 2])
