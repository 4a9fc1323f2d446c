"""Shared-prefix decode attention (mfa_decode_attention_prefix*) against the definition in 64 bits.

Tolerances, from the roundings on the way: each weight enters the second product as bf16, off by at most 2^-8 of
itself, and O is divided by the sum of what entered, so an output is off by at most 2^-8 of the weighted mean of
|v - out|, which is at most (t^2 - out^2) / t with t the largest |v|, below t; the output is rounded to bf16, off by at
most 2^-8 of itself; the fp32 sums of 256 products and the exponentials add less than 2^-12 of
either. On an E4M3 cache the weights and the scaled values are f16 (2^-11 each, and 2^-11 for the scale) and the queries
are held to 2^-18.8 of the largest: together no more than another 2^-8 of the largest |v|. The LSE is off by the logits' fp32 sums, 2^-15 of
scale * sum |q k| (about 10 here), below 1e-3."""
import numpy as np
import pytest
import torch

from decode_attention_mfa_gb300 import capi

pytestmark = pytest.mark.gpu
PAGE, HEADS, DIM = 64, 64, 256
SCALE = 1.0 / 16.0
LSE_ABS = 1e-3


class Batch:
    """Groups (first sequence, sequences, prefix pages) of a batch and its sequences' lengths, on the device."""

    def __init__(self, sizes, pages, lens, fp8=False, seed=0, starts=None, spare_cols=1):
        rng = np.random.default_rng(seed)
        self.B, self.fp8 = len(lens), fp8
        self.starts = np.concatenate([[0], np.cumsum(sizes)]) if starts is None else np.asarray(starts)
        self.pages, self.lens = np.asarray(pages), np.asarray(lens)
        shared = np.zeros(self.B, np.int64)
        group = np.full(self.B, -1)
        for g, n in enumerate(self.pages):
            shared[self.starts[g]:self.starts[g + 1]] = n
            group[self.starts[g]:self.starts[g + 1]] = g
        own = np.maximum(0, -(-self.lens // PAGE) - shared)
        total = int(self.pages.sum() + own.sum()) + 3
        order = rng.permutation(total)
        self.table = np.full((self.B, max(1, int((shared + own).max())) + spare_cols), -1, np.int32)
        at = int(self.pages.sum())
        first = np.concatenate([[0], np.cumsum(self.pages)])
        for b in range(self.B):
            if group[b] >= 0:
                self.table[b, :shared[b]] = order[first[group[b]]:first[group[b]] + shared[b]]
            self.table[b, shared[b]:shared[b] + own[b]] = order[at:at + own[b]]
            at += own[b]
        gen = torch.Generator(device="cuda").manual_seed(seed + 1)
        self.num_pages = total
        self.q = torch.randn((self.B, HEADS, DIM), generator=gen, device="cuda").bfloat16()
        rows = [torch.randn((total, PAGE, DIM), generator=gen, device="cuda").bfloat16() for _ in range(2)]
        # rows that no sequence holds are poisoned: a stale row is never read
        used = np.zeros((total, PAGE), bool)
        for b in range(self.B):
            n = int(self.lens[b])
            for j in range(-(-n // PAGE)):
                used[self.table[b, j], :min(PAGE, n - j * PAGE)] = True
        self.unused = torch.from_numpy(~used).cuda()
        self.scales = []
        if fp8:
            self.cache = []
            for x in rows:
                x = x.float() * torch.exp(0.5 * torch.randn((total, PAGE, 1), generator=gen, device="cuda"))
                s = x.abs().amax(-1) / 448.0
                codes = (x / s.unsqueeze(-1)).to(torch.float8_e4m3fn).view(torch.uint8)
                codes[self.unused] = 0x7F
                s[self.unused] = float("nan")
                self.cache.append(codes)
                self.scales.append(s)
        else:
            for x in rows:
                x[self.unused] = float("nan")
            self.cache = rows
        i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a)).int().cuda()  # noqa: E731
        self.d = dict(table=i32(self.table), lens=i32(self.lens), starts=i32(self.starts), pages=i32(self.pages))
        self.out = torch.full((self.B, HEADS, DIM), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((self.B, HEADS), 7.0, device="cuda")
        self.hints = (int(self.pages.max()) * PAGE, int(max(1, (self.lens - shared * PAGE).max())))
        self.ws = None

    def workspace(self, hints=None):
        n = capi.mfa_decode_prefix_workspace_bytes(self.B, len(self.pages), *(hints or self.hints))
        self.ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        capi.mfa_workspace_init(self.ws, n)
        self.ws[256:] = 0xFF  # what the scratch holds between calls is not used: NaN floats, page counts of -1
        torch.cuda.synchronize()

    def call(self, scale=SCALE, hints=None, stream=None):
        if self.ws is None:
            self.workspace(hints)
        fn = capi.mfa_decode_attention_prefix_fp8 if self.fp8 else capi.mfa_decode_attention_prefix
        fn(self.q, *self.cache, *self.scales, self.d["table"], self.d["lens"], self.d["starts"], self.d["pages"],
           len(self.pages), self.out, self.lse, scale, self.B, self.table.shape[1], self.num_pages, *(hints or self.hints),
           self.ws, self.ws.numel(), stream)

    def reference(self, b, scale=SCALE):
        n = int(self.lens[b])
        ids = torch.from_numpy(self.table[b, :-(-n // PAGE)]).long().cuda()
        rows = []
        for i, c in enumerate(self.cache):
            if self.fp8:
                x = c[ids].view(torch.float8_e4m3fn).double() * self.scales[i][ids].double().unsqueeze(-1)
            else:
                x = c[ids].double()
            rows.append(x.reshape(-1, DIM)[:n])
        logits = self.q[b].double() @ rows[0].T * scale
        lse = torch.logsumexp(logits, 1)
        return torch.exp(logits - lse[:, None]) @ rows[1], lse, rows[1].abs().max()

    def check(self, scale=SCALE, which=None):
        capi.mfa_check_device_errors(self.ws)
        for b in range(self.B) if which is None else which:
            if self.lens[b] == 0:
                assert (self.out[b] == 0).all() and torch.isneginf(self.lse[b]).all()
                continue
            out, lse, top = self.reference(b, scale)
            got = self.out[b].double()
            bound = 2 ** -8 * ((2 if self.fp8 else 1) * top + out.abs()) + 2 ** -12 * top
            assert torch.isfinite(got).all(), b
            assert ((got - out).abs() <= bound).all(), (b, float((got - out).abs().max()), float(bound.min()))
            assert float((got - out).norm() / out.norm()) <= 5e-3 * (2 if self.fp8 else 1), b
            assert float((self.lse[b].double() - lse).abs().max()) <= LSE_ABS, b

    def run(self, **kw):
        self.call(**kw)
        self.check(kw.get("scale", SCALE))
        return self


def lens_of(sizes, pages, suffix, seed=0):
    rng = np.random.default_rng(seed)
    return np.concatenate([p * PAGE + rng.integers(0, suffix + 1, n) for n, p in zip(sizes, pages)]).astype(np.int64)


KV = pytest.mark.parametrize("fp8", [False, True])


@KV
@pytest.mark.parametrize("n,pages", [(2, 1), (2, 2), (4, 2), (4, 3), (3, 4), (5, 5), (8, 16), (9, 7), (17, 31), (64, 64), (6, 400)])
def test_one_group(n, pages, fp8):
    Batch([n], [pages], lens_of([n], [pages], 150, n), fp8, seed=n).run()


@KV
@pytest.mark.parametrize("suffix", [0, 1, 64, 65])
def test_suffix_lengths(suffix, fp8):
    """No token behind the prefix, one, a whole page, one more."""
    Batch([6], [9], np.full(6, 9 * PAGE + suffix), fp8).run()


@KV
def test_groups_of_every_kind(fp8):
    """Odd sizes, a group of one, one without shared pages, one whose prefix is a single page."""
    sizes, pages = [7, 1, 19, 3, 2, 4], [5, 9, 40, 0, 1, 2]
    Batch(sizes, pages, lens_of(sizes, pages, 700, 4), fp8, seed=9).run()


@KV
def test_many_small_groups(fp8):
    """More row tiles than pairs of CTAs: pairs work through several pieces each."""
    rng = np.random.default_rng(1)
    sizes, pages = rng.integers(1, 6, 130).tolist(), rng.integers(1, 12, 130).tolist()
    Batch(sizes, pages, lens_of(sizes, pages, 90, 4), fp8, seed=3).run()


@KV
def test_sequences_that_end_inside_the_prefix_and_empty_slots(fp8):
    """They see their own tokens and nothing else, wherever in the group they stand; a group left with one whole prefix
    is read through its own rows."""
    sizes, pages = [5, 4, 6, 2], [6, 10, 3, 8]
    lens = lens_of(sizes, pages, 100, 5)
    lens[0], lens[2], lens[4] = 0, 1, 6 * PAGE - 1   # the first of its group among them
    lens[5:8] = 65, 0, 640 - 64                      # one of four holds the prefix
    lens[9:15] = 0                                   # none does
    lens[15], lens[16] = 8 * PAGE, 8 * PAGE + 1
    Batch(sizes, pages, lens, fp8, seed=5).run()


@KV
def test_all_empty_and_single(fp8):
    Batch([4], [3], np.zeros(4, np.int64), fp8).run()
    Batch([1], [3], np.array([200]), fp8).run()
    Batch([1], [0], np.array([1]), fp8).run()


@KV
def test_sequences_outside_the_groups(fp8):
    lens = np.array([10, 300, 5 * PAGE + 3, 5 * PAGE, 6 * PAGE, 77, 0, 128])
    Batch(None, [5], lens, fp8, starts=[2, 5]).run()


@KV
def test_shared_pages_beyond_the_prefix_and_long_rows(fp8):
    """prefix_pages may be fewer than the pages really shared; table rows may be longer than needed."""
    b = Batch([4], [12], lens_of([4], [12], 40, 1), fp8, spare_cols=33)
    b.d["pages"].fill_(5)
    b.run()


@KV
@pytest.mark.parametrize("hints", [(0, 0), (64, 64), (1 << 20, 1 << 20)])
def test_hints_size_the_grids_only(hints, fp8):
    sizes, pages = [6, 5], [30, 4]
    Batch(sizes, pages, lens_of(sizes, pages, 400, 8), fp8).run(hints=hints)


@KV
@pytest.mark.parametrize("scale", [-SCALE, 0.0, 0.5])
def test_scales(scale, fp8):
    sizes, pages = [6, 3], [7, 4]
    Batch(sizes, pages, lens_of(sizes, pages, 100, 8), fp8).run(scale=scale)


@KV
def test_moving_maximum(fp8):
    """Logits that grow along the prefix (the reference maximum moves at every unit) and fall again in the suffix."""
    b = Batch([5], [40], lens_of([5], [40], 200, 3), fp8)
    gain = torch.zeros(b.num_pages, device="cuda")
    ids = torch.from_numpy(b.table[0, :40]).long().cuda()
    gain[ids] = torch.linspace(0.0, 6.0, 40, device="cuda")
    if fp8:
        b.scales[0] *= (0.2 + gain).unsqueeze(-1)
    else:
        b.cache[0].copy_((b.cache[0].float() * (0.2 + gain).view(-1, 1, 1)).bfloat16())
    # the logits reach about 8 * 4 * sqrt(256) / 16: the LSE's bound grows with them
    b.call()
    capi.mfa_check_device_errors(b.ws)
    for i in range(5):
        out, lse, top = b.reference(i)
        assert ((b.out[i].double() - out).abs() <= 2 ** -7 * (2 if fp8 else 1) * top).all()
        assert float((b.lse[i].double() - lse).abs().max()) <= 1e-2


@KV
def test_whole_batch_of_1024(fp8):
    """The largest batch, in groups of four and one large group."""
    sizes = [4] * 100 + [200] + [2] * 212
    pages = [2] * 100 + [3] + [1] * 212
    b = Batch(sizes, pages, lens_of(sizes, pages, 70, 8), fp8)
    b.call()
    b.check(which=range(0, 1024, 7))


@KV
def test_bad_groups_and_pages_are_reported(fp8):
    """Group starts that decrease or leave the batch, page counts out of range and bad page ids set the error word;
    sequences that they do not concern keep their values."""
    sizes, pages = [4, 4, 4], [4, 3, 2]
    lens = lens_of(sizes, pages, 100, 2)
    b = Batch(sizes, pages, lens, fp8)
    for starts, counts in (([0, 4, 2, 12], [4, 3, 2]), ([-3, 4, 8, 90], [4, 3, 2]), ([0, 4, 8, 12], [4, 3, 1 << 30])):
        b.d["starts"].copy_(torch.tensor(starts))
        b.d["pages"].copy_(torch.tensor(counts))
        b.call()
        with pytest.raises(capi.MFAError) as e:
            capi.mfa_check_device_errors(b.ws)
        assert e.value.status == 6
        b.check(which=range(4))
    b = Batch(sizes, pages, lens, fp8)
    b.table[5, 0] = b.num_pages + 7
    b.table[4, 1] = -2
    b.d["table"].copy_(torch.from_numpy(b.table))
    b.call()
    with pytest.raises(capi.MFAError) as e:
        capi.mfa_check_device_errors(b.ws)
    assert e.value.status == 5
    b.check(which=list(range(4)) + list(range(8, 12)))


@KV
def test_captured_and_replayed_with_new_lengths_and_groups(fp8):
    """One graph, replayed on another stream with other lengths and groups of the same batch; two graphs share one
    workspace in turn; every replay gives what a direct call gives, bit for bit."""
    sizes, pages = [6, 6], [20, 10]
    a = Batch(sizes, pages, lens_of(sizes, pages, 300, 2), fp8)
    a.run()
    first = a.out.clone(), a.lse.clone()
    stream = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(stream):
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                a.call()
            graphs.append(g)
        for g in graphs * 2:
            a.out.zero_()
            g.replay()
            stream.synchronize()
            assert torch.equal(a.out, first[0]) and torch.equal(a.lse, first[1])
        a.lens = np.maximum(0, a.lens - np.arange(12) * 37)
        a.d["lens"].copy_(torch.from_numpy(a.lens))
        a.d["pages"].copy_(torch.tensor([13, 0]))
        graphs[0].replay()
        stream.synchronize()
        a.check()


@KV
def test_nothing_of_one_sequence_reaches_another(fp8):
    """NaN and infinities in the pages, scales and query of one sequence change no bit of the others' results, although
    they share tiles, units and MMAs; its own results are NaN."""
    sizes, pages = [6, 5], [5, 3]
    lens = lens_of(sizes, pages, 200, 6)
    lens[7] = 100  # ends inside its prefix: read on its own
    lens[[1, 4, 8]] += 70
    b = Batch(sizes, pages, lens, fp8, seed=11).run()
    clean = b.out.clone(), b.lse.clone()
    for bad in (1, 4, 7, 8):
        own = [int(x) for x in b.table[bad, (0 if bad == 7 else pages[0 if bad < 6 else 1]):-(-int(lens[bad]) // PAGE)]]
        if bad == 7:  # its pages are the group's: its query alone is its own
            own = []
        keep = [c.clone() for c in b.cache], [x.clone() for x in b.scales], b.q.clone()
        for i, c in enumerate(b.cache):
            if own and fp8:
                c[own[0]] = 0x7F
                b.scales[i][own[-1]] = float("inf") if i else float("nan")
            elif own:
                c[own[0]] = float("nan")
                c[own[-1], 0] = float("inf")
        b.q[bad, 5] = float("nan")
        b.call()
        capi.mfa_check_device_errors(b.ws)
        others = [i for i in range(11) if i != bad]
        assert torch.equal(b.out[others], clean[0][others]) and torch.equal(b.lse[others], clean[1][others]), bad
        assert torch.isnan(b.out[bad, 5].float()).all()
        if own:
            assert torch.isnan(b.out[bad].float()).any(dim=1).all()
        for c, k in zip(b.cache, keep[0]):
            c.copy_(k)
        for c, k in zip(b.scales, keep[1]):
            c.copy_(k)
        b.q.copy_(keep[2])
    b.run()


@KV
def test_nan_in_the_prefix_reaches_all_who_see_it_and_no_one_else(fp8):
    sizes, pages = [6, 5], [5, 3]
    lens = lens_of(sizes, pages, 200, 6)
    lens[2] = 64  # sees the first page of its group's prefix
    b = Batch(sizes, pages, lens, fp8, seed=12).run()
    clean = b.out.clone()
    page = int(b.table[0, 3])
    b.cache[1][page, 17] = 0x7F if fp8 else float("nan")
    b.call()
    capi.mfa_check_device_errors(b.ws)
    hit = [0, 1, 3, 4, 5]
    assert torch.isnan(b.out[hit].float()).all()
    others = [i for i in range(11) if i not in hit]
    assert torch.equal(b.out[others], clean[others])


@KV
def test_small_weights_beside_a_large_one(fp8):
    """One key with most of the weight and a value of nearly nothing (as the first token of a text often has) beside
    thousands of small weights: what these add up to is kept."""
    n, pages = 4, 130
    b = Batch([n], [pages], np.full(n, pages * PAGE + 40), fp8, seed=13)
    first = int(b.table[0, 0])
    q = b.q.float().mean(dim=(0, 1))
    for i in range(n):
        b.q[i] = (b.q[i].float() * 0.1 + q / q.norm() * 16).bfloat16()
    key = q / q.norm()
    if fp8:
        s = key.abs().max() * 12.0 / 448
        b.cache[0][first, 0] = (key * 12.0 / s).to(torch.float8_e4m3fn).view(torch.uint8)
        b.scales[0][first, 0] = s
        b.scales[1][first, 0] *= 1e-4
    else:
        b.cache[0][first, 0] = (key * 12.0).bfloat16()
        b.cache[1][first, 0] *= 1e-4
    b.call()
    capi.mfa_check_device_errors(b.ws)
    for i in range(n):
        out, lse, top = b.reference(i)
        got = b.out[i].double()
        # the weights are rounded one by one (bf16: 2^-8 of each), so the result is off by a like part of itself
        assert float((got - out).norm() / out.norm()) <= 2 ** -7, i
        assert float((b.lse[i].double() - lse).abs().max()) <= LSE_ABS


@KV
def test_a_wait_that_gives_up_is_reported_and_the_next_call_is_whole(fp8):
    """Without a budget for waits a call either reports one that gave up or gave up none and is right: how long a wait is
    lies with the memory, which copies on another stream keep busy here. It ends either way, and the next call is whole."""
    sizes, pages = [6, 5], [40, 30]
    b = Batch(sizes, pages, lens_of(sizes, pages, 200, 6), fp8, seed=14)
    b.workspace()
    busy = [torch.empty(1 << 28, dtype=torch.uint8, device="cuda") for _ in range(2)]
    side = torch.cuda.Stream()
    try:
        for _ in range(10):
            with torch.cuda.stream(side):
                for _ in range(4):
                    busy[0].copy_(busy[1])
            capi.mfa_set_wait_budget_ns(0)
            b.call()
            torch.cuda.synchronize()
            try:
                b.check()
            except capi.MFAError as e:
                assert e.status == 7
                capi.mfa_set_wait_budget_ns(2_000_000_000)
                b.run()
    finally:
        capi.mfa_set_wait_budget_ns(2_000_000_000)
    b.run()


@KV
def test_two_calls_at_once_with_workspaces_of_their_own(fp8):
    sizes, pages = [9, 4], [33, 20]
    a = Batch(sizes, pages, lens_of(sizes, pages, 300, 1), fp8, seed=15)
    b = Batch(sizes, pages, lens_of(sizes, pages, 300, 2), fp8, seed=16)
    a.workspace()
    b.workspace()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for x, s in zip((a, b), streams):
            x.call(stream=s)
    torch.cuda.synchronize()
    a.check()
    b.check()


@KV
def test_a_first_unit_of_infinite_logits_leaves_later_low_ones_whole(fp8):
    """Two pages (a unit of the kernel) whose logits are all -inf come first, and then logits near -224: a reference of the
    first unit's would send all their exponentials to zero. Queries of 1 and -1 but for one of 1024, so that two E4M3 terms
    hold them exactly. The LSE, and with it each weight, is off by 2^-15 of scale * sum |q k|, which is below 256."""
    n, pages = 3, 6
    b = Batch([n], [pages], np.full(n, pages * PAGE + 30), fp8, seed=17)
    b.q.copy_(torch.sign(b.q.float()).bfloat16())
    b.q[:, :, 0] = 1.0
    b.q[:, :, 1] = 1024.0
    low = torch.from_numpy(b.table[0, :2]).long().cuda()
    if fp8:
        b.scales[0].fill_(2 ** -7)      # values of up to 3.5
        b.cache[0][:, :, 1] = 0xFE      # -448
        b.cache[0][low] = 0
        b.cache[0][low, :, 0] = 0xB8    # -1
        b.scales[0][low] = float("inf")
        # 0 * inf is NaN: the other codes of these rows meet the scale as a part of the sum only
    else:
        b.cache[0][:, :, 1] = -3.5
        b.cache[0][low, :, 0] = float("-inf")
    b.call(hints=(0, 0))
    capi.mfa_check_device_errors(b.ws)
    for i in range(n):
        length = int(b.lens[i]) - 2 * PAGE
        ids = torch.from_numpy(b.table[i, 2:-(-int(b.lens[i]) // PAGE)]).long().cuda()
        k, v = (c[ids].view(torch.float8_e4m3fn).double() * x[ids].double().unsqueeze(-1) if fp8 else c[ids].double()
                for c, x in zip(b.cache, b.scales or [None] * 2))
        k, v = k.reshape(-1, DIM)[:length], v.reshape(-1, DIM)[:length]
        logits = b.q[i].double() @ k.T * SCALE
        lse = torch.logsumexp(logits, 1)
        out = torch.exp(logits - lse[:, None]) @ v
        assert float(lse.max()) < -150
        err = 256 * 2 ** -15
        assert float((b.lse[i].double() - lse).abs().max()) <= err
        bound = (2 ** -8 * (2 if fp8 else 1) + 2 * err) * v.abs().max() + 2 ** -8 * out.abs()
        assert ((b.out[i].double() - out).abs() <= bound).all()


@KV
@pytest.mark.parametrize("first,count", [(0, 32), (32, 32), (0, 63)])
def test_infinite_logits_beside_low_ones_in_a_page(first, count, fp8):
    """Keys of one page whose logits are -inf, the others' near -224 (as above); nothing else is there to set a reference."""
    b = Batch([2], [1], np.full(2, PAGE), fp8, seed=23)
    b.q.copy_(torch.sign(b.q.float()).bfloat16())
    b.q[:, :, 0] = 1.0
    b.q[:, :, 1] = 1024.0
    page, off = int(b.table[0, 0]), slice(first, first + count)
    if fp8:
        b.scales[0].fill_(2 ** -7)
        b.cache[0][:, :, 1] = 0xFE
        b.cache[0][page, off] = 0
        b.cache[0][page, off, 0] = 0xB8
        b.scales[0][page, off] = float("inf")
    else:
        b.cache[0][:, :, 1] = -3.5
        b.cache[0][page, off, 0] = float("-inf")
    b.call()
    capi.mfa_check_device_errors(b.ws)
    rest = [i for i in range(PAGE) if not first <= i < first + count]
    k, v = (c[page].view(torch.float8_e4m3fn).double() * x[page].double().unsqueeze(-1) if fp8 else c[page].double()
            for c, x in zip(b.cache, b.scales or [None] * 2))
    for i in range(2):
        logits = b.q[i].double() @ k[rest].T * SCALE
        lse = torch.logsumexp(logits, 1)
        out = torch.exp(logits - lse[:, None]) @ v[rest]
        err = 256 * 2 ** -15
        assert float((b.lse[i].double() - lse).abs().max()) <= err
        bound = (2 ** -8 * (2 if fp8 else 1) + 2 * err) * v.abs().max() + 2 ** -8 * out.abs()
        assert ((b.out[i].double() - out).abs() <= bound).all()


@KV
def test_serving_steps_over_a_shared_prefix(fp8):
    """What a server does: a prompt is appended once, its pages are entered in the rows of all who share it, and then
    steps of reserve, append by slots and attention are replayed from one graph; requests end, keep the shared pages and
    give back their own. Lengths, caches and results follow the host's bookkeeping."""
    sizes, pages, B, cols, num_pages, rows = [3, 4], [3, 2], 7, 8, 64, 7 * 24
    b = Batch(sizes, pages, np.repeat(pages, sizes) * PAGE, fp8, seed=18, spare_cols=5)  # the prompts alone
    i32 = dict(dtype=torch.int32, device="cuda")
    kv = [torch.zeros((num_pages, PAGE, DIM), dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda") for _ in range(2)]
    scales = [torch.zeros((num_pages, PAGE), device="cuda") for _ in range(2 * fp8)]
    ids = torch.randperm(num_pages, generator=torch.Generator().manual_seed(1)).int().cuda()
    free, n_free = ids.clone(), torch.tensor([num_pages], **i32)
    table = torch.full((B, cols), -1, **i32)
    lens, new, done = (torch.zeros(B, **i32) for _ in range(3))
    starts = torch.zeros(B + 1, **i32)
    slots = torch.zeros(max(rows, 5 * PAGE), dtype=torch.int64, device="cuda")
    fused = torch.zeros((5 * PAGE, 2 * DIM), dtype=torch.bfloat16, device="cuda")
    keep = torch.tensor(np.repeat(pages, sizes), **i32)
    hints = (max(pages) * PAGE, 3 * PAGE)
    b.workspace(hints)
    append = capi.mfa_kv_append_slots_fp8 if fp8 else capi.mfa_kv_append_slots
    attend = capi.mfa_decode_attention_prefix_fp8 if fp8 else capi.mfa_decode_attention_prefix

    def take(most):
        capi.mfa_reserve_pages(new, lens, table, free, n_free, B, cols, num_pages, most, starts, slots, lens, n_free, b.ws)
        append(fused, fused[:, DIM:], 2 * DIM, 2 * DIM, slots, most, *kv, *scales, num_pages, b.ws)

    def step():
        take(rows)
        attend(b.q, *kv, *scales, table, lens, b.d["starts"], b.d["pages"], 2, b.out, b.lse, SCALE, B, cols, num_pages,
               *hints, b.ws, b.ws.numel())

    # the prompts, for the first request of each group, and then shared with the others
    prompt = torch.randn((5 * PAGE, 2 * DIM)).bfloat16()
    new.copy_(torch.tensor([3 * PAGE, 0, 0, 2 * PAGE, 0, 0, 0]))
    fused.copy_(prompt)
    take(5 * PAGE)
    for g, first in enumerate((0, 3)):
        table[first:first + sizes[g], :pages[g]] = table[first, :pages[g]].clone()
    lens.copy_(keep * PAGE)
    held = [prompt[:3 * PAGE]] * 3 + [prompt[3 * PAGE:]] * 4
    new.zero_()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
    rng = np.random.default_rng(3)
    for turn in range(6):
        count = rng.integers(0, 25, B)
        now = torch.randn((5 * PAGE, 2 * DIM)).bfloat16()
        with torch.cuda.stream(stream):
            new.copy_(torch.from_numpy(count))
            fused.copy_(now)
            graph.replay()
        stream.synchronize()
        capi.mfa_check_device_errors(b.ws)
        at = np.concatenate([[0], np.cumsum(count)])
        held = [torch.cat([h, now[at[i]:at[i + 1]]]) for i, h in enumerate(held)]
        assert lens.tolist() == [len(h) for h in held]
        b.cache, b.scales, b.table, b.lens = kv, scales, table.cpu().numpy(), lens.cpu().numpy()
        for i, h in enumerate(held):
            pg = table[i, :-(-len(h) // PAGE)].long()
            for c, (x, cache) in enumerate(zip((h[:, :DIM], h[:, DIM:]), kv)):
                got = cache[pg].reshape(-1, DIM)[:len(h)]
                if fp8:  # codes as tests of the append pin them; here: within half a step of E4M3 of the row's largest
                    s = scales[c][pg].reshape(-1)[:len(h), None]
                    x = x.float().cuda()
                    top = x.abs().amax(1, keepdim=True)
                    assert ((got.view(torch.float8_e4m3fn).float() * s - x).abs() <= 2 ** -4 * 1.01 * top).all()
                else:
                    assert torch.equal(got.cpu(), x)
        b.check()
        if turn == 3:  # two requests end and new ones take their places, behind the same prompts
            done.zero_()
            done[[1, 5]] = 1
            own = [-(-len(held[i]) // PAGE) - int(keep[i]) for i in (1, 5)]
            left = int(n_free.item())
            with torch.cuda.stream(stream):
                capi.mfa_release_pages(done, keep, lens, table, free, n_free, B, cols, num_pages, lens, n_free, b.ws)
            stream.synchronize()
            assert int(n_free.item()) == left + sum(own)
            for i in (1, 5):
                held[i] = held[i][:int(keep[i]) * PAGE]
    with torch.cuda.stream(stream):  # all end; the first of each group gives the prompt back as well
        done.fill_(1)
        keep[0] = keep[3] = 0
        capi.mfa_release_pages(done, keep, lens, table, free, n_free, B, cols, num_pages, lens, n_free, b.ws)
    stream.synchronize()
    capi.mfa_check_device_errors(b.ws)
    assert int(n_free.item()) == num_pages and sorted(free.tolist()) == list(range(num_pages))


@KV
def test_as_many_groups_as_sequences_and_empty_groups(fp8):
    """1024 groups of one share nothing, whatever their counts of pages; groups without a sequence change nothing."""
    rng = np.random.default_rng(8)
    lens = rng.integers(0, 200, 1024)
    b = Batch([1] * 1024, rng.integers(0, 4, 1024), lens, fp8, seed=19)
    b.call()
    b.check(which=range(0, 1024, 11))
    starts = [0, 0, 5, 5, 5, 9, 12, 12]
    pages = [7, 3, 9, 0, 4, 2, 1]
    lens = np.concatenate([np.full(5, 3 * PAGE + 10), np.full(4, 4 * PAGE + 70), np.full(3, 2 * PAGE), [100]])
    Batch(None, pages, lens, fp8, seed=20, starts=starts, spare_cols=9).run()  # counts of pages within the table rows


@KV
def test_lengths_out_of_range_are_clamped_and_reported(fp8):
    """A negative length is an empty sequence, one beyond its table row ends with the row; the others keep their values."""
    b = Batch([5], [4], lens_of([5], [4], 100, 2), fp8, seed=21, spare_cols=0)
    true = b.lens.copy()
    full = b.table.shape[1] * PAGE
    row = int(np.argmax(true))
    other = (row + 1) % 5
    b.d["lens"][other] = -5
    b.call()
    with pytest.raises(capi.MFAError) as e:
        capi.mfa_check_device_errors(b.ws)
    assert e.value.status == 6
    b.lens[other] = 0
    b.check()
    b.lens = true
    b.d["lens"].copy_(torch.from_numpy(true))
    b.d["lens"][row] = 2 ** 31 - 1
    for i, c in enumerate(b.cache):  # the rest of its last page counts then
        last = int(b.table[row, -1])
        c[last] = 0x38 if fp8 else 1.0
        if fp8:
            b.scales[i][last] = 1.0
    b.call()
    with pytest.raises(capi.MFAError) as e:
        capi.mfa_check_device_errors(b.ws)
    assert e.value.status == 6
    b.lens = true.copy()
    b.lens[row] = full
    b.check()


@KV
def test_pages_at_the_far_end_of_a_large_cache(fp8):
    """Pages whose rows lie past 2^31 elements: rows appended by slot are where the attention reads them."""
    num_pages, n, own = 131072 + 40, 4, 70
    sizes, pages = [n], [3]
    b = Batch(sizes, pages, np.full(n, 3 * PAGE + own), fp8, seed=22)
    far = torch.arange(num_pages - b.num_pages, num_pages, device="cuda")
    kv = [torch.empty((num_pages, PAGE, DIM), dtype=c.dtype, device="cuda") for c in b.cache]
    scales = [torch.empty((num_pages, PAGE), device="cuda") for _ in b.scales]
    for big, c in zip(kv + scales, b.cache + b.scales):
        big[far] = c
    b.table = np.where(b.table >= 0, b.table + num_pages - b.num_pages, -1).astype(np.int32)
    b.d["table"].copy_(torch.from_numpy(b.table))
    b.cache, b.scales, b.num_pages = kv, scales, num_pages
    b.run()
    # one more token for each, behind its last
    rows = torch.randn((n, DIM), device="cuda").bfloat16()
    slots = torch.tensor([int(b.table[i, b.lens[i] // PAGE]) * PAGE + int(b.lens[i]) % PAGE for i in range(n)], device="cuda")
    append = capi.mfa_kv_append_slots_fp8 if fp8 else capi.mfa_kv_append_slots
    append(rows, rows, DIM, DIM, slots, n, *kv, *scales, num_pages, b.ws)
    b.lens = b.lens + 1
    b.d["lens"].copy_(torch.from_numpy(b.lens))
    b.run()
    if not fp8:
        assert torch.equal(kv[0].view(-1, DIM)[slots], rows)
